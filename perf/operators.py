"""The decode operators over a quantised KV cache in HBM, as they are measured.

Five operators, all of the serving side (head dim d = 128, blocks of B = 16 tokens):

* write   keys and values of T tokens, rounded to 8-bit floats (e4m3, one
          power-of-two scale per token and KV head) and placed in paged blocks;
* read    the valid tokens of R requests back as 16- or 32-bit units
          [R][Hkv][blocks][2][B][d];
* attn    attention of S queries a request (the normal one and its drafts)
          over the paged 8-bit cache;
* prefix  the same for a batch whose requests share one long prefix, held
          once in bf16 units, before their own 8-bit suffixes;
* verify  which drafted tokens the target's probabilities accept, and the
          token that follows, from given random numbers.

A page is one KV head's block: 2048 bytes of key codes [16 tokens][128] (the
two halves of an odd token's row exchanged), 2048 bytes of value codes
[128][16 tokens], 16 key exponents and 16 value exponents (a code c stands for
c * 2^(byte - 127)).
"""
import math

import torch

own = False

D, B = 128, 16
HALF = 2048
PAGE = 2 * HALF + 2 * B
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 128 requests appends a token each; k and v are slices of one
        # projection's output (32 query heads before them)
        dict(name="write_step", op="write", T=128, Hkv=8, dtype="bf16", run=1, fused=32),
        # a long prompt's keys and values go to whole pages in order
        dict(name="write_prompt", op="write", T=32768, Hkv=8, dtype="bf16", run=2048, fused=0),
        # one short context is fetched back for inspection or a move
        dict(name="read_short", op="read", R=1, len=100, Hkv=8, ragged=False, dtype="bf16"),
        # a ragged batch leaves the cache for 16-bit units (a prefix, a host store)
        dict(name="read_batch", op="read", R=16, len=16384, Hkv=8, ragged=True, dtype="bf16"),
        # one request's single token: latency
        dict(name="attn_one", op="attn", R=1, S=1, Hq=32, Hkv=8, len=4096, ragged=False, causal=False, dtype="bf16"),
        # a ragged batch verifies three drafts causally
        dict(name="attn_drafts", op="attn", R=24, S=4, Hq=32, Hkv=8, len=9001, ragged=True, causal=True, dtype="fp16"),
        # a full serving batch: normal and draft query over 16K tokens a request
        dict(name="attn_batch", op="attn", R=64, S=2, Hq=32, Hkv=8, len=16384, ragged=False, causal=False, dtype="bf16"),
        # few requests share a system prompt
        dict(name="prefix_few", op="prefix", R=3, S=1, Hq=32, Hkv=8, prefix=2048, len=300, ragged=True, causal=False, dtype="bf16"),
        # a mid-size batch with three drafts behind an odd prefix
        dict(name="prefix_drafts", op="prefix", R=20, S=4, Hq=32, Hkv=8, prefix=8191, len=777, ragged=True, causal=True, dtype="bf16"),
        # many requests ask about one long document
        dict(name="prefix_batch", op="prefix", R=128, S=1, Hq=32, Hkv=8, prefix=32768, len=512, ragged=True, causal=False, dtype="bf16"),
        # one request's three drafts over a small vocabulary
        dict(name="verify_one", op="verify", R=1, n=3, V=32000, dtype="fp32", point=False),
        # a serving batch over a large vocabulary
        dict(name="verify_batch", op="verify", R=128, n=3, V=151936, dtype="fp32", point=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(32, 8), (8, 2), (16, 16), (24, 8), (40, 8), (8, 1), (28, 4)]


def draw(rng):
    op = rng.choice(["write", "read", "attn", "prefix", "verify"])
    Hq, Hkv = rng.choice(HEADS)
    if op == "write":
        return dict(op=op, T=_log(rng, 1, 16384), Hkv=Hkv, dtype=rng.choice(list(DTYPES)),
                    run=_log(rng, 1, 2048), fused=rng.choice([0, Hq]))
    if op == "verify":
        return dict(op=op, R=_log(rng, 1, 96), n=rng.randint(1, 6), V=_log(rng, 1000, 130000),
                    dtype=rng.choice(list(DTYPES)), point=rng.random() < 0.25)
    R, S = _log(rng, 1, 96), rng.randint(1, 4)
    most = 40 // Hkv if op == "read" else min(480 // Hkv, 4096 // (S * Hq))
    n = _log(rng, 17, min(32768, max(18, 16384 * most // R)))
    if op == "read":
        return dict(op=op, R=R, len=n, Hkv=Hkv, ragged=rng.random() < 0.7, dtype=rng.choice(list(DTYPES)))
    d = dict(op=op, R=R, S=S, Hq=Hq, Hkv=Hkv, len=n, ragged=rng.random() < 0.7,
             causal=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp16"]))
    if op == "prefix":
        d.update(prefix=_log(rng, 17, 32768), len=_log(rng, 1, 1024), dtype="bf16")
        while d["R"] * d["S"] * Hq > 4096:
            d["R"] = max(1, d["R"] // 2)
    return d


def _lens(case):
    """Tokens of each request: all of them, or a spread over (0, len] with an empty request
    where there are several."""
    R, n = case["R"], case["len"]
    if not case["ragged"]:
        return [n] * R
    out = [max(1, int(n * ((r + 1) * 0.6180339887 % 1.0))) for r in range(R)]
    out[0] = n
    if R > 2:
        out[R // 2] = 0
    return out


def work(case):
    op = case["op"]
    if op == "write":
        e = case["T"] * case["Hkv"]
        return {"bytes": e * (2 * D * SIZE[case["dtype"]] + 2 * D + 2) + 8 * case["T"], "flops": 0}
    if op == "verify":
        # n draft probabilities and n target ones a request; then the target's row and, where a
        # draft was refused (about 1 - 0.7^n of the requests), the draft's row too
        row = case["V"] * SIZE[case["dtype"]]
        second = 0.0 if case["point"] else 1.0 - 0.7 ** case["n"]
        return {"bytes": case["R"] * (row * (1.0 + second) + 16 * case["n"]), "flops": 2 * case["R"] * case["V"]}
    tokens = sum(_lens(case))
    if op == "read":
        return {"bytes": tokens * case["Hkv"] * (2 * D + 2 + 2 * D * SIZE[case["dtype"]]), "flops": 0}
    rows = case["S"] * case["R"] * case["Hq"]
    b = tokens * case["Hkv"] * (2 * D + 2) + 2 * rows * D * SIZE[case["dtype"]]
    f = 4 * case["S"] * case["Hq"] * D * tokens
    if op == "prefix":
        b += case["prefix"] * case["Hkv"] * 2 * D * 2
        f += 4 * rows * D * case["prefix"]
    return {"bytes": b, "flops": f}


# ------------------------------------------------- the page format, in torch
def _quantise(x):
    """(codes, exponents) of rows of d values: the exponent e is the least with max |x| <= 448 * 2^e,
    held in [-100, 120]; the code is x * 2^-e, rounded to e4m3."""
    m, k = torch.frexp(x.float().abs().amax(-1))
    e = torch.where(m <= 0.875, k - 9, k - 8)
    e = torch.where(m == 0, torch.full_like(e, -100), e).clamp(-100, 120)
    return torch.ldexp(x.float(), -e.unsqueeze(-1)).to(torch.float8_e4m3fn), e


def _swap(k):
    """Exchange the halves of the odd tokens' rows of key codes [..., 16, 128] (bytes)."""
    odd = (torch.arange(B, device=k.device) & 1).bool()[:, None]
    return torch.where(odd, k.roll(D // 2, -1), k)


def _pages_of(k, v):
    """Pages [n][Hkv][PAGE] of keys and values [n][Hkv][16][128]."""
    kc, ke = _quantise(k)
    vc, ve = _quantise(v)
    n, h = k.shape[:2]
    return torch.cat([_swap(kc.view(torch.uint8)).reshape(n, h, HALF),
                      vc.view(torch.uint8).transpose(2, 3).reshape(n, h, HALF),
                      (ke + 127).to(torch.uint8), (ve + 127).to(torch.uint8)], -1)


def _values(pages, dtype):
    """(keys, values) [..., 16, 128] that pages [..., PAGE] stand for."""
    lead = pages.shape[:-1]
    kc = _swap(pages[..., :HALF].reshape(*lead, B, D)).view(torch.float8_e4m3fn).to(dtype)
    vc = pages[..., HALF:2 * HALF].reshape(*lead, D, B).transpose(-1, -2).contiguous().view(torch.float8_e4m3fn).to(dtype)
    ex = torch.ldexp(torch.ones((), dtype=dtype, device=pages.device), pages[..., 2 * HALF:].int() - 127)
    return kc * ex[..., :B, None], vc * ex[..., B:, None]


def _whole(pages):
    """A pool as its codes' values and its exponents."""
    return {"codes": pages[..., :2 * HALF].view(torch.float8_e4m3fn), "exponents": pages[..., 2 * HALF:]}


# ----------------------------------------------------------------- inputs
def _cache(case, g, lens):
    """Pages of random keys and values (5 % of the blocks lean towards their head's direction,
    token sizes vary), a page table in random order, and head directions."""
    Hkv = case["Hkv"]
    nb = [-(-n // B) for n in lens]
    total = sum(nb) + 3
    dev = "cuda"
    u = torch.randn(Hkv, D, generator=g, device=dev)
    u = u / u.norm(dim=1, keepdim=True)
    k = torch.randn(total, Hkv, B, D, generator=g, device=dev)
    k += (torch.rand(total, Hkv, 1, 1, generator=g, device=dev) < 0.05) * 3.0 * u[:, None, :]
    v = torch.randn(total, Hkv, B, D, generator=g, device=dev)
    v *= torch.exp2(0.5 * torch.randn(total, Hkv, B, 1, generator=g, device=dev))
    pages = _pages_of(k, v)
    del k, v
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(lens), max(1, max(nb))), -1, dtype=torch.int32, device=dev)
    at = 0
    for r, n in enumerate(nb):
        table[r, :n] = order[at:at + n]
        if lens[r] % B:  # what was there before the last block's tokens: anything
            pages[order[at + n - 1].long(), :, HALF:2 * HALF].view(Hkv, D, B)[:, :, lens[r] % B:] = 0x7F
        at += n
    return pages, table, torch.tensor(lens, dtype=torch.int32, device=dev), u


def _handle(case, pages, table):
    from sparse_kv_block_gb300.oasis import Q8Cache, make_q8_config
    blocks = table.shape[1] if table is not None else 1
    cfg = make_q8_config(num_pages=pages.shape[0], max_blocks=blocks, Hq=case.get("Hq", case["Hkv"]), Hkv=case["Hkv"])
    return Q8Cache(cfg, pages=pages)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    op, dev = case["op"], "cuda"
    s = dict(case=case)
    if op == "write":
        T, Hkv = case["T"], case["Hkv"]
        dt = DTYPES[case["dtype"]]
        x = torch.randn(T, case["fused"] + 2 * Hkv, D, generator=g, device=dev)
        x *= torch.exp2(2.0 * torch.randn(T, case["fused"] + 2 * Hkv, 1, generator=g, device=dev))
        x = x.to(dt)
        s["k"], s["v"] = x[:, case["fused"]:case["fused"] + Hkv], x[:, case["fused"] + Hkv:]
        # runs of consecutive tokens, each from a block's beginning or (runs shorter than a
        # block) from anywhere inside one
        run = case["run"]
        per = -(-run // B) + (1 if run < B else 0)
        runs = -(-T // run)
        first = torch.randperm(runs, generator=g, device=dev) * per * B
        if run < B:
            first = first + torch.randint(0, B, (runs,), generator=g, device=dev)
        t = torch.arange(T, device=dev)
        s["slots"] = first[t // run] + t % run
        s["pages"] = torch.zeros(runs * per, Hkv, PAGE, dtype=torch.uint8, device=dev)
        if own:
            s["cache"] = _handle(case, s["pages"], None)
        return s
    if op == "verify":
        R, n, V = case["R"], case["n"], case["V"]
        dt = DTYPES[case["dtype"]]
        z = 2.5 * torch.randn(R, n + 1, V, generator=g, device=dev)
        p = torch.softmax(z, -1)
        z = z[:, :n] + 0.75 * torch.randn(R, n, V, generator=g, device=dev)
        q = torch.softmax(z, -1)
        s["drafts"] = torch.multinomial((p[:, :n] if case["point"] else q).reshape(R * n, V), 1, generator=g).view(R, n).to(torch.int32)
        s["p"], s["q"] = p.to(dt), None if case["point"] else q.to(dt)
        s["u_accept"] = torch.rand(R, n, generator=g, device=dev)
        s["u_sample"] = torch.rand(R, generator=g, device=dev)
        s["tokens"] = torch.empty(R, n + 1, dtype=torch.int32, device=dev)
        s["n_accept"] = torch.empty(R, dtype=torch.int32, device=dev)
        return s
    lens = _lens(case)
    s["pages"], s["table"], s["lens"], u = _cache(case, g, lens)
    if own:
        s["cache"] = _handle(case, s["pages"], s["table"])
    if op == "read":
        s["out"] = torch.zeros(case["R"], case["Hkv"], s["table"].shape[1], 2, B, D, dtype=DTYPES[case["dtype"]], device=dev)
        return s
    dt = DTYPES[case["dtype"]]
    G = case["Hq"] // case["Hkv"]
    q = torch.randn(case["S"], case["R"], case["Hq"], D, generator=g, device=dev)
    s["q"] = (q + 8.0 * u.repeat_interleave(G, 0)).to(dt)
    s["out"] = torch.empty_like(s["q"])
    if op == "prefix":
        nb = -(-case["prefix"] // B)
        x = torch.randn(case["Hkv"], nb, 2, B, D, generator=g, device=dev)
        x[:, :, 0] += (torch.rand(case["Hkv"], nb, 1, 1, generator=g, device=dev) < 0.05) * 3.0 * u[:, None, None, :]
        s["prefix"] = x.to(torch.bfloat16)
        if own:
            s["ws"] = s["cache"].prefix_workspace(case["R"], case["S"], case["prefix"])
    return s


# ------------------------------------------------------------- one pass
def run(s):
    return globals()["_run_" + s["case"]["op"]](s)


def _run_write(s):
    if own:
        s["cache"].oasis_q8_write(s["k"], s["v"], s["slots"])
        return _whole(s["pages"])
    page, at = s["slots"] // B, s["slots"] % B
    pool = s["pages"]
    P, H = pool.shape[:2]
    kc, ke = _quantise(s["k"])
    vc, ve = _quantise(s["v"])
    kc = kc.view(torch.uint8)
    kc = torch.where((at & 1).bool()[:, None, None], kc.roll(D // 2, -1), kc)
    codes = pool[..., :2 * HALF]
    h = torch.arange(H, device=pool.device)
    i = torch.arange(D, device=pool.device)
    codes[page[:, None, None], h[:, None], at[:, None, None] * D + i] = kc
    codes[page[:, None, None], h[:, None], HALF + i * B + at[:, None, None]] = vc.view(torch.uint8)
    pool[page[:, None], h, 2 * HALF + at[:, None]] = (ke + 127).to(torch.uint8)
    pool[page[:, None], h, 2 * HALF + B + at[:, None]] = (ve + 127).to(torch.uint8)
    return _whole(pool)


def _run_read(s):
    out = s["out"]
    if own:
        s["cache"].oasis_q8_read(s["table"], s["lens"], out)
        return out
    k, v = _values(s["pages"][s["table"].clamp(min=0).long()], torch.float32)  # [R][NB][Hkv][16][128]
    kv = torch.stack([k, v], 3).transpose(1, 2).to(out.dtype)
    NB = out.shape[2]
    pos = torch.arange(NB * B, device=out.device).view(NB, 1, B, 1)
    out.copy_(torch.where(pos < s["lens"].view(-1, 1, 1, 1, 1, 1), kv, out))
    return out


def _suffix(s, dtype):
    """(scores, values, mask) of the paged tokens: [R][Hkv][S*G][N], [R][Hkv][N][d], [R][1][S*G][N]."""
    c = s["case"]
    S, R, Hq, _ = s["q"].shape
    Hkv = c["Hkv"]
    G = Hq // Hkv
    k, v = _values(s["pages"][s["table"].clamp(min=0).long()], dtype)
    N = k.shape[1] * B
    k = k.transpose(1, 2).reshape(R, Hkv, N, D)
    v = v.transpose(1, 2).reshape(R, Hkv, N, D)
    q = s["q"].to(dtype).view(S, R, Hkv, G, D).permute(1, 2, 0, 3, 4).reshape(R, Hkv, S * G, D)
    x = q @ k.transpose(-1, -2) / math.sqrt(D)
    pos = torch.arange(N, device=q.device)
    less = torch.arange(S - 1, -1, -1, device=q.device) if c["causal"] else torch.zeros(S, dtype=torch.long, device=q.device)
    limit = (s["lens"].view(R, 1) - less.view(1, S)).repeat_interleave(G, 1)  # [R][S*G]
    mask = (pos < limit.unsqueeze(-1)).unsqueeze(1)
    v = torch.where((pos < s["lens"].view(R, 1)).view(R, 1, N, 1), v, torch.zeros((), dtype=dtype, device=v.device))
    return q, torch.where(mask, x, -math.inf), v, mask


def _back(o, S, G):
    """[R][Hkv][S*G][d] -> [S][R][Hq][d]."""
    R, Hkv = o.shape[:2]
    return o.view(R, Hkv, S, G, D).permute(2, 0, 1, 3, 4).reshape(S, R, Hkv * G, D)


def _run_attn(s):
    c = s["case"]
    if own:
        s["cache"].oasis_q8_attn(s["q"], s["table"], s["lens"], s["out"], causal=c["causal"])
        return s["out"]
    _, x, v, mask = _suffix(s, torch.float32)
    m = x.amax(-1, keepdim=True)
    p = torch.where(mask, torch.exp(x - torch.where(torch.isinf(m), 0.0, m)), 0.0)
    l = p.sum(-1, keepdim=True)
    o = torch.where(l > 0, (p @ v) / l, 0.0)
    s["out"].copy_(_back(o, c["S"], c["Hq"] // c["Hkv"]))
    return s["out"]


def _run_prefix(s):
    c = s["case"]
    if own:
        s["cache"].oasis_prefix_attn(s["q"], s["prefix"], c["prefix"], s["table"], s["lens"], s["out"], s["ws"], causal=c["causal"])
        return s["out"]
    q, x, v, mask = _suffix(s, torch.float32)
    R, Hkv, n, _ = q.shape
    kv = s["prefix"].float()
    P = c["prefix"]
    k2 = kv[:, :, 0].reshape(Hkv, -1, D)[:, :P]
    v2 = kv[:, :, 1].reshape(Hkv, -1, D)[:, :P]
    y = q.transpose(0, 1).reshape(Hkv, R * n, D) @ k2.transpose(-1, -2) / math.sqrt(D)
    y = y.view(Hkv, R, n, P)
    m = torch.maximum(x.amax(-1), y.amax(-1).transpose(0, 1)).unsqueeze(-1)  # [R][Hkv][n][1]
    p = torch.where(mask, torch.exp(x - m), 0.0)
    r = torch.exp(y - m.transpose(0, 1))
    l = p.sum(-1, keepdim=True) + r.sum(-1, keepdim=True).transpose(0, 1)
    o = p @ v + (r.view(Hkv, R * n, P) @ v2).view(Hkv, R, n, D).transpose(0, 1)
    s["out"].copy_(_back(o / l, c["S"], c["Hq"] // Hkv))
    return s["out"]


def _run_verify(s):
    p, q = s["p"], s["q"]
    if own:
        from sparse_kv_block_gb300.oasis import oasis_verify_drafts
        oasis_verify_drafts(p, q, s["drafts"], s["u_accept"], s["u_sample"], s["tokens"], s["n_accept"])
        return s["tokens"], s["n_accept"]
    x = s["drafts"].long()
    R, n = x.shape
    px = p[:, :n].gather(2, x.unsqueeze(-1)).squeeze(-1).double()
    qx = q.gather(2, x.unsqueeze(-1)).squeeze(-1).double() if q is not None else torch.ones_like(px)
    ok = s["u_accept"].double() * qx < px
    k = ok.long().cumprod(1).sum(1)  # accepted drafts of each request
    rows = torch.arange(R, device=p.device)
    target = p[rows, k].double()
    j = k.clamp(max=n - 1)
    if q is not None:
        draft = q[rows, j].double()
    else:
        draft = torch.zeros_like(target).scatter_(1, x[rows, j].unsqueeze(1), 1.0)
    rest = torch.where((k < n).unsqueeze(1), (target - draft).clamp(min=0), target)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, target)
    cum = rest.cumsum(1)
    token = (cum <= s["u_sample"].double().unsqueeze(1) * cum[:, -1:]).sum(1)
    i = torch.arange(n + 1, device=p.device)
    drafts = torch.cat([x, x[:, :1]], 1)
    kk = k.unsqueeze(1)
    s["tokens"].copy_(torch.where(i < kk, drafts, torch.where(i == kk, token.unsqueeze(1), -1)))
    s["n_accept"].copy_(k)
    return s["tokens"], s["n_accept"]


# ------------------------------------------------- the definitions, in 64 bits
def _round_e4m3(x):
    """x (64 bits, |x| <= 448) to the nearest number of 4 significant bits, 2^-9 apart at least; ties to even."""
    a = x.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -30)))
    e = torch.where(torch.exp2(e + 1) <= a, e + 1, e)
    e = torch.where(torch.exp2(e) > a, e - 1, e).clamp(min=-6.0)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _exact_rows(x):
    x = x.double()
    a = x.abs().amax(-1)
    e = torch.ceil(torch.log2(a.clamp(min=2.0 ** -140) / 448.0))
    e = torch.where(448.0 * torch.exp2(e) < a, e + 1, e)
    e = torch.where(448.0 * torch.exp2(e - 1) >= a, e - 1, e).clamp(-100, 120)
    return _round_e4m3(x * torch.exp2(-e).unsqueeze(-1)), e


def _exact_token(pages, table, n):
    """Keys and values [Hkv][n][d] in 64 bits of one request's n tokens, straight from the bytes."""
    t = torch.arange(n, device=pages.device)
    page, j = table[t // B].long(), t % B
    i = torch.arange(D, device=pages.device)
    b = pages[page]  # [n][Hkv][PAGE]
    H = pages.shape[1]
    at = j[:, None] * D + (i + 64 * (j[:, None] & 1)) % D  # where dim i of token j stands
    k = b.gather(2, at[:, None].expand(n, H, D))
    v = b.gather(2, (HALF + i * B + j[:, None])[:, None].expand(n, H, D))
    ke = b.gather(2, (2 * HALF + j).view(n, 1, 1).expand(n, H, 1))
    ve = b.gather(2, (2 * HALF + B + j).view(n, 1, 1).expand(n, H, 1))

    def value(c, e):
        c, e = c.long(), e.double()
        sign = 1.0 - 2.0 * (c >> 7).double()
        ex, man = ((c >> 3) & 15).double(), (c & 7).double()
        a = torch.where(ex == 0, man * 2.0 ** -9, (8 + man) * torch.exp2(ex - 10))
        return (sign * a * torch.exp2(e - 127)).transpose(0, 1)
    return value(k, ke), value(v, ve)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "write":
        k, ke = _exact_rows(s["k"])
        v, ve = _exact_rows(s["v"])
        P, H = s["pages"].shape[:2]
        K = torch.zeros(P * B, H, D, dtype=torch.float64, device=k.device)
        V = torch.zeros_like(K)
        E = torch.zeros(P * B, H, 2, dtype=torch.uint8, device=k.device)
        K[s["slots"]], V[s["slots"]] = k, v
        E[s["slots"]] = torch.stack([ke + 127, ve + 127], -1).to(torch.uint8)
        K = K.view(P, B, H, 2, 64).permute(0, 2, 1, 3, 4).contiguous()
        K[:, :, 1::2] = K[:, :, 1::2].flip(3)
        V = V.view(P, B, H, D).permute(0, 2, 3, 1)
        return {"codes": torch.cat([K.reshape(P, H, HALF), V.reshape(P, H, HALF)], -1),
                "exponents": E.view(P, B, H, 2).permute(0, 2, 3, 1).reshape(P, H, 2 * B)}
    if op == "verify":
        return _exact_verify(s)
    lens = _lens(case)
    if op == "read":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        flat = out.permute(0, 1, 3, 2, 4, 5).reshape(case["R"], case["Hkv"], 2, -1, D)
        for r, n in enumerate(lens):
            if n:
                k, v = _exact_token(s["pages"], s["table"][r], n)
                flat[r, :, 0, :n], flat[r, :, 1, :n] = k, v
        NB = out.shape[2]
        return flat.view(case["R"], case["Hkv"], 2, NB, B, D).permute(0, 1, 3, 2, 4, 5).contiguous()
    S, R, Hq, Hkv = case["S"], case["R"], case["Hq"], case["Hkv"]
    G = Hq // Hkv
    out = torch.zeros(S, R, Hq, D, dtype=torch.float64, device="cuda")
    pre = None
    if op == "prefix":
        P = case["prefix"]
        pre = [s["prefix"][:, :, i].reshape(Hkv, -1, D)[:, :P].double() for i in (0, 1)]
    for r, n in enumerate(lens):
        k, v = _exact_token(s["pages"], s["table"][r], n) if n else (torch.zeros(Hkv, 0, D, dtype=torch.float64, device="cuda"),) * 2
        for i in range(S):
            t = max(0, n - (S - 1 - i)) if case["causal"] else n
            kk, vv = k[:, :t], v[:, :t]
            if pre is not None:
                kk, vv = torch.cat([pre[0], kk], 1), torch.cat([pre[1], vv], 1)
            if kk.shape[1]:
                x = torch.einsum("hgd,hnd->hgn", s["q"][i, r].double().view(Hkv, G, D), kk) / math.sqrt(D)
                w = torch.softmax(x, -1)
                out[i, r] = torch.einsum("hgn,hnd->hgd", w, vv).reshape(Hq, D)
    return out


def _exact_verify(s):
    x = s["drafts"].tolist()
    R, n = len(x), len(x[0])
    ua, us = s["u_accept"].tolist(), s["u_sample"].double().tolist()
    tokens, accepted = torch.full((R, n + 1), -1, dtype=torch.int32), torch.zeros(R, dtype=torch.int32)
    for r in range(R):
        at = 0
        while at < n:
            px = float(s["p"][r, at, x[r][at]])
            qx = float(s["q"][r, at, x[r][at]]) if s["q"] is not None else 1.0
            if not ua[r][at] * qx < px:
                break
            tokens[r, at] = x[r][at]
            at += 1
        w = s["p"][r, at].double()
        if at < n:
            if s["q"] is not None:
                left = w - s["q"][r, at].double()
            else:
                left = w.clone()
                left[x[r][at]] -= 1.0
            left = left.clamp(min=0)
            if float(left.sum()) > 0:
                w = left
        c = torch.cumsum(w, 0)
        tokens[r, at] = int(torch.searchsorted(c, us[r] * float(c[-1]), right=True))
        accepted[r] = at
    return tokens, accepted
