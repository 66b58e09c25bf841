"""Units read from the 8-bit cache where the rest of the library takes them: a
host store that the look-ahead step serves from, the dense anchor's cache, and
the cache's own attention, all against the oracle on the same units."""
import numpy as np
import pytest
import torch

import oracle
from sparse_kv_block_gb300 import oasis as ob
from sparse_kv_block_gb300 import workload
from tests import _harness as H
from tests import _q8 as Q
from tests.test_q8 import dev, gen  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [[1000, 37], [1024, 512]])
def test_units_serve_the_step_and_the_dense_anchor(dev, lens):  # noqa: F811
    sh = workload.SHAPES["tiny"]
    R, NB = sh.R, sh.NBmax
    nb = [-(-n // 16) for n in lens]
    cache = ob.Q8Cache(ob.make_q8_config(sum(nb) + 2, NB, sh.Hq, sh.Hkv, out_fp32=True))
    table = Q.table_of(lens, sum(nb) + 2, NB, gen(sum(lens))).to(dev)
    m = torch.tensor(lens, dtype=torch.int32, device=dev)
    units = torch.zeros(R, sh.Hkv, NB, 2, 16, 128, dtype=torch.bfloat16, device=dev)

    def through_the_cache(host):
        """[R][Hkv][NBmax][2][16][d]: each request's tokens are written and read back in place."""
        tok = host.to(dev).permute(0, 2, 4, 3, 1, 5).reshape(R, NB * 16, 2, sh.Hkv, 128)
        for r, n in enumerate(lens):
            cache.oasis_q8_write(tok[r, :n, 0], tok[r, :n, 1], Q.slots_of(table.cpu(), r, 0, n).to(dev))
        units.copy_(host)
        cache.oasis_q8_read(table, m, units)
        assert cache.oasis_q8_sync() == 0
        assert not torch.equal(units.cpu(), host)
        host.copy_(units)

    L = H.make_layer(sh, seed=5, lens=lens, steps=3, out_fp32=True, mutate_host=through_the_cache)
    H.check_summaries(L)
    # the dense anchor and the cache's own attention, the normal query and the draft
    out = torch.empty((R, sh.Hq, 128), dtype=torch.float32, device=dev)
    outd = torch.empty_like(out)
    q, qd = L.q[0].to(dev), L.qd[0].to(dev)
    L.eng.oasis_dense_attn(units, 0, q, qd, out, outd)
    L.eng.oasis_sync()
    both = torch.empty((2, R, sh.Hq, 128), dtype=torch.float32, device=dev)
    cache.oasis_q8_attn(torch.stack([q, qd]), table, m, both)
    assert cache.oasis_q8_sync() == 0
    every = np.broadcast_to(np.arange(NB, dtype=np.int32), (R, sh.Hkv, NB)).copy()
    qb, qdb = workload.bf16_bits(L.q[0]), workload.bf16_bits(L.qd[0])
    ref = {(r, h): {"attn": oracle.attention_rh(L.hb, L.lens, every, qb, qdb, r, h)}
           for r in range(R) for h in range(sh.Hkv)}
    H.check_attention([out.cpu().numpy(), outd.cpu().numpy()], ref, sh.G)
    H.check_attention(list(both.cpu().numpy()), ref, sh.G)
    for t in range(3):
        H.run_staged_step(L, t, dev)
    L.eng.close()
