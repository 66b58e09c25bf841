"""Arguments of the 8-bit cache's calls at and past their limits, on the host."""
import __graft_entry__
import pytest

from sparse_kv_block_gb300 import oasis as ob


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


@pytest.mark.parametrize("scale,ok", [(0.0, True), (1e-30, True), (2.3e38, True), (2.4e38, False), (3.4e38, False)])
def test_scale_times_log2_e_is_finite(scale, ok):
    """The kernels hold scale * log2(e) in fp32: a scale past 2^128 / log2(e) = 2.36e38 would make
    every score of a zero query NaN."""
    c = ob.make_q8_config(num_pages=10, max_blocks=4, Hq=8, Hkv=2, softmax_scale=scale)
    m = ob.oasis_q8_config_error(c)
    assert (m is None) == ok
    if not ok:
        assert "softmax_scale" in m
        with pytest.raises(ob.OasisError):
            ob.oasis_q8_query_sizes(c)
