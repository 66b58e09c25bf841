"""The operators of a decode step with a tree of drafted tokens, as they are measured.

Four operators beside the 8-bit paged KV cache (head dim d = 128, blocks of B = 16 tokens):

* append    rotates T tokens' queries and keys by their positions (one or several position
            axes), writes the rotated queries out and rounds keys and values into the pages;
* tree      attention of a request's N drafted nodes over its pages: each sees the context
            before the tree and the nodes that its 64-bit word names;
* logprobs  log probability of a given token, entropy and the k largest alternatives of rows
            of logits;
* keep      moves an accepted path's keys and values to the tree's first places.

A page is one KV head's block: 2048 bytes of key codes [16 tokens][128] (e4m3, the two halves
of an odd token's row exchanged), 2048 bytes of value codes [128][16 tokens], 16 key exponents
and 16 value exponents (a code c stands for c * 2^(byte - 127)).
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
        # one decode step of 128 requests: a token each, every page another; q, k and v are slices
        # of one projection's output
        dict(name="append_step", op="append", T=128, Hq=32, Hkv=8, dtype="bf16", run=1, rot=128, axes=1, interleaved=False, far=16000),
        # 24 requests' drafted trees of 17 nodes, half of the dims rotated, in neighbouring pairs
        dict(name="append_tree", op="append", T=408, Hq=24, Hkv=8, dtype="fp16", run=17, rot=64, axes=1, interleaved=True, far=100000),
        # images of a prompt: positions in time, height and width
        dict(name="append_video", op="append", T=4999, Hq=28, Hkv=4, dtype="bf16", run=1250, rot=128, axes=3, interleaved=False, far=30000),
        # a long prompt's keys and values go to whole pages in order
        dict(name="append_prompt", op="append", T=16384, Hq=32, Hkv=8, dtype="bf16", run=2048, rot=128, axes=1, interleaved=False, far=0),
        # one request's small tree: latency
        dict(name="tree_one", op="tree", R=1, N=16, Hq=32, Hkv=8, len=4096, ragged=False, sizes=False, dtype="bf16"),
        # a ragged batch, trees of several sizes
        dict(name="tree_ragged", op="tree", R=24, N=13, Hq=28, Hkv=4, len=9001, ragged=True, sizes=True, dtype="fp16"),
        # a serving batch with large trees
        dict(name="tree_batch", op="tree", R=16, N=64, Hq=32, Hkv=8, len=16384, ragged=False, sizes=False, dtype="bf16"),
        # the tokens of one request's step, with five alternatives
        dict(name="logprobs_one", op="logprobs", rows=4, V=32000, k=5, dtype="fp32", skip=False),
        # 16 requests' trees of 16 nodes over a large vocabulary, some rows not wanted
        dict(name="logprobs_tree", op="logprobs", rows=256, V=151936, k=1, dtype="bf16", skip=True),
        # a serving batch's tokens with twenty alternatives
        dict(name="logprobs_batch", op="logprobs", rows=512, V=151936, k=20, dtype="bf16", skip=False),
        # one request's path
        dict(name="keep_one", op="keep", R=1, N=16, Hkv=8),
        # a serving batch's paths
        dict(name="keep_batch", op="keep", R=128, N=64, Hkv=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(32, 8), (8, 2), (16, 16), (24, 8), (40, 8), (8, 1), (28, 4)]


def draw(rng):
    op = rng.choice(["append", "tree", "logprobs", "keep"])
    Hq, Hkv = rng.choice(HEADS)
    if op == "append":
        dtype = rng.choice(list(DTYPES))
        return dict(op=op, T=_log(rng, 1, 6000 if dtype == "fp32" else 12000), Hq=Hq, Hkv=Hkv, dtype=dtype,
                    run=_log(rng, 1, 2048), rot=rng.choice([128, 128, 64, 32, 96]), axes=rng.randint(1, 3),
                    interleaved=rng.random() < 0.4, far=_log(rng, 1, 1000000))
    if op == "logprobs":
        V = _log(rng, 1000, 152000)
        return dict(op=op, rows=_log(rng, 1, min(512, 70000000 // V)), V=V, k=rng.randint(0, 20),
                    dtype=rng.choice(list(DTYPES)), skip=rng.random() < 0.4)
    if op == "keep":
        return dict(op=op, R=_log(rng, 1, 128), N=_log(rng, 1, 64), Hkv=Hkv)
    R, N = _log(rng, 1, 64), _log(rng, 1, 64)
    most = min(200000000 // (R * N * Hq), 2000000 // (R * Hkv))
    return dict(op=op, R=R, N=N, Hq=Hq, Hkv=Hkv, len=_log(rng, 17, min(32768, max(18, most))),
                ragged=rng.random() < 0.7, sizes=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp16"]))


def _lens(case):
    """Tokens of each request before its tree: all of them, or a spread over (0, len] with a
    request of none where there are several."""
    R, n = case["R"], case["len"]
    if not case["ragged"]:
        return [n] * R
    out = [max(1, int(n * ((r + 1) * 0.6180339887 % 1.0))) for r in range(R)]
    out[0] = n
    if R > 2:
        out[R // 2] = 0
    return out


def _sizes(case):
    """Nodes of each request's tree."""
    R, N = case["R"], case["N"]
    if not case["sizes"]:
        return [N] * R
    out = [max(1, int(N * ((r + 1) * 0.7548776662 % 1.0) + 0.5)) for r in range(R)]
    out[0] = N
    return out


def work(case):
    op = case["op"]
    if op == "append":
        e = SIZE[case["dtype"]]
        b = case["T"] * (D * e * 2 * (case["Hq"] + case["Hkv"]) + case["Hkv"] * (2 * D + 2) + 8 * (case["axes"] + 1))
        return {"bytes": b, "flops": 0}
    if op == "logprobs":
        rows = case["rows"] * (0.75 if case["skip"] else 1.0)
        return {"bytes": rows * (case["V"] * SIZE[case["dtype"]] + 12 + 8 * case["k"]), "flops": 4 * rows * case["V"]}
    if op == "keep":
        # a path of about six nodes
        return {"bytes": case["R"] * (min(6, case["N"]) * case["Hkv"] * 2 * (2 * D + 2) + 4 * case["N"]), "flops": 0}
    lens, sizes = _lens(case), _sizes(case)
    tokens = sum(lens) + sum(sizes)
    rows = sum(sizes) * case["Hq"]
    f = sum(4 * n * case["Hq"] * D * (t + n) for t, n in zip(lens, sizes))
    return {"bytes": tokens * case["Hkv"] * (2 * D + 2) + 2 * rows * D * SIZE[case["dtype"]], "flops": f}


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


def _values(pages):
    """(keys, values) [..., 16, 128] in fp32 that pages [..., PAGE] stand for."""
    lead = pages.shape[:-1]
    kc = _swap(pages[..., :HALF].reshape(*lead, B, D)).view(torch.float8_e4m3fn).float()
    vc = pages[..., HALF:2 * HALF].reshape(*lead, D, B).transpose(-1, -2).contiguous().view(torch.float8_e4m3fn).float()
    ex = torch.ldexp(torch.ones((), device=pages.device), pages[..., 2 * HALF:].int() - 127)
    return kc * ex[..., :B, None], vc * ex[..., B:, None]


def _whole(pages):
    """A pool as its codes' values and its exponents' powers of two."""
    return {"codes": pages[..., :2 * HALF].view(torch.float8_e4m3fn),
            "scales": pages[..., 2 * HALF:].view(torch.float8_e8m0fnu)}


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
        at += n
    return pages, table, torch.tensor(lens, dtype=torch.int32, device=dev), u


def _trees(g, R, N):
    """Parents [R][N] (-1: the context; a node's parent is one of the eight before it) and words
    [R][N]: bit j of node i's says that it sees node j (its ancestors and itself)."""
    dev = "cuda"
    i = torch.arange(N, device=dev)
    back = 1 + (torch.rand(R, N, generator=g, device=dev) * 8).long()
    parent = (i - back).clamp(min=-1)
    words = torch.zeros(R, N, dtype=torch.int64, device=dev)
    rows = torch.arange(R, device=dev)
    for n in range(N):
        p = parent[:, n]
        bit = -(1 << 63) if n == 63 else 1 << n
        words[:, n] = torch.where(p >= 0, words[rows, p.clamp(min=0)], 0) | bit
    return parent, words


def _handle(case, pages, table):
    from sparse_kv_block_gb300.oasis import Q8Cache, make_q8_config
    blocks = table.shape[1] if table is not None else 1
    cfg = make_q8_config(num_pages=pages.shape[0], max_blocks=blocks, Hq=case.get("Hq", case["Hkv"]), Hkv=case["Hkv"])
    return Q8Cache(cfg, pages=pages)


def _frequencies(case):
    """Radians a position of each pair, and each pair's axis: the axes' sections follow one
    another, a quarter of the pairs the first one's."""
    half = case["rot"] // 2
    f = [500000.0 ** (-2.0 * i / case["rot"]) for i in range(half)]
    first = half // 4
    rest = half - first
    axis = [0] * half if case["axes"] == 1 else [0 if i < first else 1 + (i - first) * (case["axes"] - 1) // rest for i in range(half)]
    return f, axis


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 29)
    op, dev = case["op"], "cuda"
    s = dict(case=case)
    if op == "append":
        T, Hq, Hkv = case["T"], case["Hq"], case["Hkv"]
        x = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=dev)
        x *= torch.exp2(2.0 * torch.randn(T, Hq + 2 * Hkv, 1, generator=g, device=dev))
        x = x.to(DTYPES[case["dtype"]])
        s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        # runs of consecutive tokens, each from a block's beginning or (runs shorter than a
        # block, and of an odd length) from anywhere inside one
        run = case["run"]
        inside = run < B or run % 2 == 1
        per = -(-run // B) + (1 if inside else 0)
        runs = -(-T // run)
        first = torch.randperm(runs, generator=g, device=dev) * per * B
        if inside:
            first = first + torch.randint(0, B, (runs,), generator=g, device=dev)
        t = torch.arange(T, device=dev)
        s["slots"] = first[t // run] + t % run
        start = torch.randint(0, case["far"] + 1, (runs,), generator=g, device=dev)
        pos = start[t // run] + t % run
        more = torch.randint(0, 64, (max(0, case["axes"] - 1), T), generator=g, device=dev)
        s["positions"] = torch.cat([pos[None], start[t // run] + more])
        s["frequency"], s["axis"] = _frequencies(case)
        s["frequencies"] = torch.tensor(s["frequency"], dtype=torch.float64, device=dev)
        s["axes"] = torch.tensor(s["axis"], device=dev)
        s["pages"] = torch.zeros(runs * per, Hkv, PAGE, dtype=torch.uint8, device=dev)
        s["q_out"] = torch.empty(T, Hq, D, dtype=x.dtype, device=dev)
        if own:
            from sparse_kv_block_gb300.oasis import make_rope
            s["cache"] = _handle(case, s["pages"], None)
            s["rope"] = make_rope(case["rot"], frequency=s["frequency"], axis=s["axis"], interleaved=case["interleaved"])
        return s
    if op == "logprobs":
        rows, V, k = case["rows"], case["V"], case["k"]
        z = 2.5 * torch.randn(rows, V, generator=g, device=dev)
        s["tokens"] = torch.multinomial(torch.softmax(z, -1), 1, generator=g).view(rows).to(torch.int32)
        if case["skip"]:
            s["tokens"][torch.arange(rows, device=dev) % 4 == 3] = -1
        s["logits"] = z.to(DTYPES[case["dtype"]])
        s["logprobs"] = torch.zeros(rows, device=dev)
        s["entropy"] = torch.zeros(rows, device=dev)
        s["top_ids"] = torch.zeros(rows, k, dtype=torch.int32, device=dev)
        s["top_logprobs"] = torch.zeros(rows, k, device=dev)
        return s
    if op == "keep":
        R, N = case["R"], case["N"]
        lens = [17 + (r * 7) % 41 + N for r in range(R)]
        s["pages"], s["table"], s["lens"], _ = _cache(case, g, lens)
        # each request's path: from a random node up to the context, in order
        parent, _ = _trees(g, R, N)
        leaf = torch.randint(0, N, (R,), generator=g, device=dev)
        path = [[] for _ in range(R)]
        up, at = parent.tolist(), leaf.tolist()
        for r in range(R):
            while at[r] >= 0:
                path[r].append(at[r])
                at[r] = up[r][at[r]]
        s["n_keep"] = torch.tensor([len(p) for p in path], dtype=torch.int32, device=dev)
        s["nodes"] = torch.tensor([p[::-1] + [0] * (N - len(p)) for p in path], dtype=torch.int32, device=dev)
        if own:
            s["cache"] = _handle(case, s["pages"], s["table"])
        return s
    before, sizes = _lens(case), _sizes(case)
    s["pages"], s["table"], s["lens"], u = _cache(case, g, [t + n for t, n in zip(before, sizes)])
    R, N, Hq, Hkv = case["R"], case["N"], case["Hq"], case["Hkv"]
    s["words"] = _trees(g, R, N)[1]
    s["sizes"] = torch.tensor(sizes, dtype=torch.int32, device=dev)
    q = torch.randn(R, N, Hq, D, generator=g, device=dev)
    s["q"] = (q + 8.0 * u.repeat_interleave(Hq // Hkv, 0)).to(DTYPES[case["dtype"]])
    s["out"] = torch.zeros_like(s["q"])
    if own:
        s["cache"] = _handle(case, s["pages"], s["table"])
    return s


# ------------------------------------------------------------- one pass
def run(s):
    return globals()["_run_" + s["case"]["op"]](s)


def _rotated(x, cos, sin, rot, interleaved):
    """x [T][H][128] in fp32 with its first `rot` dims rotated; cos, sin [T][rot / 2]."""
    c, n = cos.unsqueeze(1), sin.unsqueeze(1)
    y = x.clone()
    a = x[..., 0:rot:2] if interleaved else x[..., :rot // 2]
    b = x[..., 1:rot:2] if interleaved else x[..., rot // 2:rot]
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * n, a * n + b * c
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * n, a * n + b * c
    return y


def _run_append(s):
    c = s["case"]
    if own:
        s["cache"].oasis_q8_append(s["rope"], s["q"], s["k"], s["v"], s["positions"], s["slots"], s["q_out"])
        return {"q": s["q_out"], **_whole(s["pages"])}
    angle = s["positions"][s["axes"]].t().double() * s["frequencies"]  # [T][rot / 2]
    cos, sin = angle.cos().float(), angle.sin().float()
    s["q_out"].copy_(_rotated(s["q"].float(), cos, sin, c["rot"], c["interleaved"]))
    kc, ke = _quantise(_rotated(s["k"].float(), cos, sin, c["rot"], c["interleaved"]))
    vc, ve = _quantise(s["v"])
    page, at = s["slots"] // B, s["slots"] % B
    pool = s["pages"]
    H = pool.shape[1]
    kc = kc.view(torch.uint8)
    kc = torch.where((at & 1).bool()[:, None, None], kc.roll(D // 2, -1), kc)
    codes = pool[..., :2 * HALF]
    h = torch.arange(H, device=pool.device)
    i = torch.arange(D, device=pool.device)
    codes[page[:, None, None], h[:, None], at[:, None, None] * D + i] = kc
    codes[page[:, None, None], h[:, None], HALF + i * B + at[:, None, None]] = vc.view(torch.uint8)
    pool[page[:, None], h, 2 * HALF + at[:, None]] = (ke + 127).to(torch.uint8)
    pool[page[:, None], h, 2 * HALF + B + at[:, None]] = (ve + 127).to(torch.uint8)
    return {"q": s["q_out"], **_whole(pool)}


def _run_tree(s):
    if own:
        s["cache"].oasis_q8_tree_attn(s["q"], s["words"], s["table"], s["lens"], s["out"], tree_size=s["sizes"])
        return s["out"]
    R, N, Hq, _ = s["q"].shape
    Hkv = s["case"]["Hkv"]
    G = Hq // Hkv
    k, v = _values(s["pages"][s["table"].clamp(min=0).long()])
    L = k.shape[1] * B
    k = k.transpose(1, 2).reshape(R, Hkv, L, D)
    v = v.transpose(1, 2).reshape(R, Hkv, L, D)
    q = s["q"].float().view(R, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, N * G, D)
    x = q @ k.transpose(-1, -2) / math.sqrt(D)
    node = torch.arange(L, device=q.device) - (s["lens"] - s["sizes"])[:, None]  # [R][L]: which node a token is
    seen = (s["words"].unsqueeze(-1) >> node.clamp(0, 63).unsqueeze(1)) & 1  # [R][N][L]
    seen = ((node < 0).unsqueeze(1) | (seen == 1)) & (node < s["sizes"][:, None]).unsqueeze(1)
    mask = seen.repeat_interleave(G, 1).unsqueeze(1)  # [R][1][N * G][L]
    v = torch.where((node < s["sizes"][:, None]).view(R, 1, L, 1), v, 0.0)
    x = torch.where(mask, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.where(mask, torch.exp(x - torch.where(torch.isinf(m), 0.0, m)), 0.0)
    l = p.sum(-1, keepdim=True)
    o = torch.where(l > 0, (p @ v) / l, 0.0)
    o = o.view(R, Hkv, N, G, D).permute(0, 2, 1, 3, 4).reshape(R, N, Hq, D).to(s["out"].dtype)
    is_node = torch.arange(N, device=q.device) < s["sizes"][:, None]
    s["out"].copy_(torch.where(is_node[..., None, None], o, s["out"]))
    return s["out"]


def _run_logprobs(s):
    k = s["case"]["k"]
    outs = {n: s[n] for n in ("logprobs", "entropy") + (("top_ids", "top_logprobs") if k else ())}
    if own:
        from sparse_kv_block_gb300.oasis import oasis_token_logprobs
        oasis_token_logprobs(s["logits"], s["tokens"], **outs)
        return outs
    x = s["logits"].float()
    y = x - x.amax(-1, keepdim=True)
    e = torch.exp(y)
    total = e.sum(-1)
    lse = torch.log(total)
    want = s["tokens"] >= 0
    t = s["tokens"].clamp(min=0).long().unsqueeze(1)
    s["logprobs"].copy_(torch.where(want, y.gather(1, t).squeeze(1) - lse, s["logprobs"]))
    s["entropy"].copy_(torch.where(want, lse - (e * y).sum(-1) / total, s["entropy"]))
    if k:
        # the largest first, of equal ones the lowest index first
        bits = x.view(torch.int32).long()
        key = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF))
        key = key * (1 << 20) + (x.shape[1] - 1 - torch.arange(x.shape[1], device=x.device))
        ids = key.topk(k, -1).indices
        s["top_ids"].copy_(torch.where(want[:, None], ids.to(torch.int32), s["top_ids"]))
        s["top_logprobs"].copy_(torch.where(want[:, None], y.gather(1, ids) - lse[:, None], s["top_logprobs"]))
    return outs


def _run_keep(s):
    pool = s["pages"]
    if own:
        s["cache"].oasis_q8_keep(s["table"], s["lens"], s["nodes"], s["n_keep"], num_nodes=s["case"]["N"])
        return _whole(pool)
    R, M = s["nodes"].shape
    H = pool.shape[1]
    i = torch.arange(M, device=pool.device)
    base = (s["lens"] - s["case"]["N"]).long()[:, None]
    src = base + torch.where(i < s["n_keep"][:, None], s["nodes"].long(), i)  # the others stay where they are
    dst = base + i
    sp, dp = s["table"].gather(1, src // B).long().flatten(), s["table"].gather(1, dst // B).long().flatten()
    sj, dj = (src % B).flatten(), (dst % B).flatten()
    h = torch.arange(H, device=pool.device)
    d = torch.arange(D, device=pool.device)

    def places(page, j):
        key = j[:, None, None] * D + (d ^ (64 * (j[:, None, None] & 1)))
        value = HALF + d * B + j[:, None, None]
        ex = 2 * HALF + torch.stack([j, j + B], -1)[:, None]
        return page[:, None, None], h[:, None], torch.cat([key, value, ex], -1)
    pool[places(dp, dj)] = pool[places(sp, sj)]
    return _whole(pool)


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
    a = x.abs().amax(-1)
    e = torch.ceil(torch.log2(a.clamp(min=2.0 ** -140) / 448.0))
    e = torch.where(448.0 * torch.exp2(e) < a, e + 1, e)
    e = torch.where(448.0 * torch.exp2(e - 1) >= a, e - 1, e).clamp(-100, 120)
    return _round_e4m3(x * torch.exp2(-e).unsqueeze(-1)), e


def _code_values(b):
    """What bytes stand for as e4m3 numbers."""
    c = b.long()
    sign = 1.0 - 2.0 * (c >> 7).double()
    ex, man = ((c >> 3) & 15).double(), (c & 7).double()
    return sign * torch.where(ex == 0, man * 2.0 ** -9, (8 + man) * torch.exp2(ex - 10))


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
    ke = b.gather(2, (2 * HALF + j).view(n, 1, 1).expand(n, H, 1)).double()
    ve = b.gather(2, (2 * HALF + B + j).view(n, 1, 1).expand(n, H, 1)).double()
    return ((_code_values(k) * torch.exp2(ke - 127)).transpose(0, 1), (_code_values(v) * torch.exp2(ve - 127)).transpose(0, 1))


def exact(case, seed):
    return globals()["_exact_" + case["op"]](case, prepare(case, seed))


def _exact_append(case, s):
    T, Hkv, rot = case["T"], case["Hkv"], case["rot"]
    f, axis = _frequencies(case)
    pos = s["positions"].double()
    pair = [(2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2) for i in range(rot // 2)]
    q, k = s["q"].double().clone(), s["k"].double().clone()
    for x in (q, k):
        for i, (a, b) in enumerate(pair):
            w = pos[axis[i]] * f[i]
            z = torch.complex(x[:, :, a], x[:, :, b]) * torch.polar(torch.ones_like(w), w)[:, None]
            x[:, :, a], x[:, :, b] = z.real, z.imag
    K, ke = _exact_rows(k)
    V, ve = _exact_rows(s["v"].double())
    P = s["pages"].shape[0]
    KV = torch.zeros(2, P * B, Hkv, D, dtype=torch.float64, device=q.device)
    E = torch.full((2, P * B, Hkv), -127.0, dtype=torch.float64, device=q.device)
    KV[0, s["slots"]], KV[1, s["slots"]] = K, V
    E[0, s["slots"]], E[1, s["slots"]] = ke.double(), ve.double()
    kk = KV[0].view(P, B, Hkv, 2, 64).permute(0, 2, 1, 3, 4).contiguous()
    kk[:, :, 1::2] = kk[:, :, 1::2].flip(3)
    vv = KV[1].view(P, B, Hkv, D).permute(0, 2, 3, 1)
    return {"q": q, "codes": torch.cat([kk.reshape(P, Hkv, HALF), vv.reshape(P, Hkv, HALF)], -1),
            "scales": torch.exp2(E).view(2, P, B, Hkv).permute(1, 3, 0, 2).reshape(P, Hkv, 2 * B)}


def _exact_tree(case, s):
    R, N, Hq, Hkv = case["R"], case["N"], case["Hq"], case["Hkv"]
    G = Hq // Hkv
    out = torch.zeros(R, N, Hq, D, dtype=torch.float64, device="cuda")
    words = s["words"].tolist()
    for r, (t, n) in enumerate(zip(_lens(case), _sizes(case))):
        k, v = _exact_token(s["pages"], s["table"][r], t + n)
        see = torch.ones(n, t + n, dtype=torch.bool)
        for i in range(n):
            for j in range(n):
                see[i, t + j] = bool(words[r][i] >> j & 1)
        for h in range(Hkv):
            x = s["q"][r, :n, h * G:(h + 1) * G].double().transpose(0, 1) @ k[h].t() / math.sqrt(D)  # [G][n][t + n]
            w = torch.softmax(x.masked_fill(~see.to(x.device), -math.inf), -1)
            out[r, :n, h * G:(h + 1) * G] = (w @ v[h]).transpose(0, 1)
    return out


def _exact_logprobs(case, s):
    rows, V, k = case["rows"], case["V"], case["k"]
    outs = [torch.zeros(rows, dtype=torch.float64), torch.zeros(rows, dtype=torch.float64),
            torch.zeros(rows, k, dtype=torch.int32), torch.zeros(rows, k, dtype=torch.float64)]
    tokens = s["tokens"].tolist()
    for r in range(rows):
        if tokens[r] < 0:
            continue
        x = s["logits"][r].double()
        lse = torch.logsumexp(x, 0)
        p = torch.exp(x - lse)
        outs[0][r] = x[tokens[r]] - lse
        outs[1][r] = (p * (lse - x)).sum()
        for j in range(k):
            top = int((x == x.max()).nonzero()[0])
            outs[2][r, j], outs[3][r, j] = top, x[top] - lse
            x[top] = -math.inf
    return dict(zip(("logprobs", "entropy") + (("top_ids", "top_logprobs") if k else ()), outs))


def _exact_keep(case, s):
    pages = s["pages"].cpu()
    new = pages.clone()
    table, lens = s["table"].tolist(), s["lens"].tolist()
    for r, (nodes, n) in enumerate(zip(s["nodes"].tolist(), s["n_keep"].tolist())):
        base = lens[r] - case["N"]
        for i in range(n):
            (a, x), (b, y) = divmod(base + nodes[i], B), divmod(base + i, B)
            src, dst = pages[table[r][a]], new[table[r][b]]
            row = src[:, x * D:(x + 1) * D]
            dst[:, y * D:(y + 1) * D] = row if (x - y) % 2 == 0 else torch.cat([row[:, 64:], row[:, :64]], 1)
            dst[:, HALF + y:2 * HALF:B] = src[:, HALF + x:2 * HALF:B]
            dst[:, 2 * HALF + y], dst[:, 2 * HALF + B + y] = src[:, 2 * HALF + x], src[:, 2 * HALF + B + x]
    return {"codes": _code_values(new[..., :2 * HALF]), "scales": torch.exp2(new[..., 2 * HALF:].double() - 127)}
