"""Operators in front of the indexer's scores, as cases to measure: the page maps of a paged key
cache, FP8 quantisation in blocks of 128, the block-scaled FP8 product, norms and position
rotation of query and key heads, and the same in FP8 written into the indexer's key cache.

run() computes a case in plain torch operations in 32 bits, or, with `own` set, through
dsa_indexer_top_amd.binding.  exact() is the definition in 64 bits."""

import math

import torch

own = False

if torch.cuda.is_available():
    DEV = "cuda"
else:
    DEV = "cpu"

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
F8 = torch.float8_e4m3fn
BLOCK = 128                      # elements under one scale
FP8_MAX = 448.0
SCALE_MIN = 2.0 ** -126          # the scale of a block of zeros
EPS = 1e-6
N_POS = 65536                    # positions of the rotation table


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of 256 requests with contexts of up to 16384 tokens in 64-token pages:
        # one token each, eight requests finished since the last step
        dict(name="pages decode 256", op="pages", rows=256, page=64, ctx=16384, chunk=1, done=8),
        # a chunked prefill: 61 prompts get up to 8192 tokens each on top of up to 32768, in
        # 16-token pages
        dict(name="pages prefill 61 x 8192", op="pages", rows=61, page=16, ctx=32768, chunk=8192, done=3),
        # the hidden states of a small decode batch, an odd width
        dict(name="quant decode 33 x 2047", op="quant", rows=33, cols=2047, type="bf16"),
        # the hidden states of a prefill chunk
        dict(name="quant prefill 32768 x 4096", op="quant", rows=32768, cols=4096, type="bf16"),
        # one token's query projection to 64 heads of 128
        dict(name="product 1 x 8192 x 2048", op="product", m=1, n=8192, k=2048, out="bf16"),
        # a small decode batch, sizes that fill neither a tile nor a block
        dict(name="product 77 x 1000 x 1111", op="product", m=77, n=1000, k=1111, out="fp32"),
        # a prefill chunk's key projection: one head of 128 from wide hidden states
        dict(name="product 8192 x 128 x 4096", op="product", m=8192, n=128, k=4096, out="bf16"),
        # a prefill chunk's query projection
        dict(name="product 16384 x 8192 x 2048", op="product", m=16384, n=8192, k=2048, out="bf16"),
        # one token of a model with grouped heads, whole heads rotated in halves
        dict(name="heads 1 x 32+8", op="heads", tokens=1, q_heads=32, k_heads=8, dim=128, rot=128,
             pairs="half", norm="rms", type="bf16"),
        # a prefill chunk, half of each head rotated in neighbouring pairs, 16-bit floats
        dict(name="heads 8191 x 40+5", op="heads", tokens=8191, q_heads=40, k_heads=5, dim=128, rot=64,
             pairs="next", norm="layer", type="fp16"),
        # the indexer's queries and keys of a decode batch of 64, into a paged cache
        dict(name="indexer decode 64", op="indexer", tokens=64, slots=65536, pairs="half", type="bf16"),
        # ... and of a prefill chunk of 32768 tokens
        dict(name="indexer prefill 32768", op="indexer", tokens=32768, slots=65536, pairs="half",
             type="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "quant", "product", "product", "heads", "indexer"])
    if op == "pages":
        chunk = rng.choice([1, _log(rng, 2, 8192)])
        rows = _log(rng, 1, 1024 if chunk == 1 else max(1, min(1024, 61 * 8192 // chunk)))
        return dict(op=op, rows=rows, page=rng.choice([16, 32, 64, 128, 256]),
                    ctx=_log(rng, 64, max(64, min(32768, (1 << 22) // rows))), chunk=chunk,
                    done=rng.randint(0, rows // 4))
    if op == "quant":
        cols = _log(rng, 64, 8192)
        return dict(op=op, rows=_log(rng, 1, min(32768, 32768 * 4096 // (2 * cols))), cols=cols,
                    type=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "product":
        n, k = _log(rng, 64, 8192), _log(rng, 128, 8192)
        return dict(op=op, m=_log(rng, 1, max(1, min(16384, 16384 * 8192 * 2048 // (n * k)))), n=n, k=k,
                    out=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "heads":
        q, k, dim = _log(rng, 1, 64), _log(rng, 1, 16), rng.choice([64, 96, 128, 192, 256])
        return dict(op=op, tokens=_log(rng, 1, max(1, min(8191, 8191 * 45 * 64 // ((q + k) * dim)))),
                    q_heads=q, k_heads=k, dim=dim, rot=rng.choice([32, 64, dim]),
                    pairs=rng.choice(["half", "next"]), norm=rng.choice(["rms", "layer"]),
                    type=rng.choice(["bf16", "fp16", "fp32"]))
    return dict(op=op, tokens=_log(rng, 1, 32768), slots=65536, pairs=rng.choice(["half", "next"]),
                type=rng.choice(["bf16", "fp16"]))


def work(case):
    op = case["op"]
    if op == "pages":
        rows, tok = case["rows"], case["rows"] * (case["chunk"] + 1) // 2
        new = tok // case["page"] + (rows if case["chunk"] > 1 else 0) // 2
        # lengths in and out, table and list entries of the new pages, maps of the tokens
        return dict(bytes=rows * 20 + new * 8 + case["rows"] * case["chunk"] * 16, flops=0)
    if op == "quant":
        nb = -(-case["cols"] // BLOCK)
        size = 4 if case["type"] == "fp32" else 2
        return dict(bytes=case["rows"] * (case["cols"] * (size + 1) + nb * 4),
                    flops=2 * case["rows"] * case["cols"])
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        nb = -(-k // BLOCK)
        return dict(bytes=m * k + n * k + 4 * nb * (m + -(-n // BLOCK)) + m * n * (4 if case["out"] == "fp32" else 2),
                    flops=2 * m * n * k)
    if op == "heads":
        size = 4 if case["type"] == "fp32" else 2
        n = case["tokens"] * (case["q_heads"] + case["k_heads"]) * case["dim"]
        return dict(bytes=2 * size * n + case["tokens"] * (4 + 4 * case["rot"]), flops=8 * n)
    n = case["tokens"] * 65 * 128
    return dict(bytes=3 * n + case["tokens"] * (12 + 4 * 64 + 64 * 8 + 4), flops=10 * n)


# ---------------------------------------------------------------- inputs
def _rotation_table(n_pos, rot, dev):
    """cos | sin of every position's angles, float32, from 64-bit angles."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    a = torch.arange(n_pos, dtype=torch.float64, device=dev)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


def _quantise(x):
    """FP8 codes and scales of a float32 matrix (rows x blocks of 128), for making inputs."""
    m, k = x.shape
    nb = -(-k // BLOCK)
    p = torch.zeros(m, nb * BLOCK, device=x.device)
    p[:, :k] = x
    p = p.view(m, nb, BLOCK)
    s = (p.abs().amax(2) / FP8_MAX).clamp_min(SCALE_MIN)
    return (p / s[:, :, None]).view(m, nb * BLOCK)[:, :k].to(F8), s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=g)
    ints = lambda lo, hi, *s: torch.randint(lo, hi, s, device=DEV, generator=g)
    op = case["op"]
    s = dict(case)
    if op == "pages":
        R, P, ctx, chunk = case["rows"], case["page"], case["ctx"], case["chunk"]
        lens = ints(max(1, ctx // 4), ctx + 1, R).int()
        # decode: a few rows of the batch are padding; prefill: ragged chunks
        new = (ints(0, 16, R) > 0).int() if chunk == 1 else ints(1, chunk + 1, R).int()
        done = torch.zeros(R, dtype=torch.uint8, device=DEV)
        done[torch.randperm(R, device=DEV, generator=g)[:case["done"]]] = 1
        new = new * (1 - done.int())
        width = -(-(ctx + chunk) // P)
        used = (lens + P - 1) // P
        n_pages = R * width
        perm = torch.randperm(n_pages, device=DEV, generator=g).int()
        begin = used.cumsum(0) - used
        col = torch.arange(width, device=DEV)
        table = torch.where(col < used[:, None], perm[(begin[:, None] + col).clamp_max(n_pages - 1)], 0).int()
        total = int(used.sum())
        free = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
        free[:n_pages - total] = perm[total:]
        cap = R * chunk
        s.update(lens=lens, new=new, done_rows=done, table=table.contiguous(), free=free,
                 count=torch.full((1,), n_pages - total, dtype=torch.int32, device=DEV),
                 len_out=torch.empty_like(lens), count_out=torch.empty(1, dtype=torch.int32, device=DEV),
                 row_begin=torch.empty(R + 1, dtype=torch.int32, device=DEV),
                 slot=torch.empty(cap, dtype=torch.int64, device=DEV),
                 row=torch.empty(cap, dtype=torch.int32, device=DEV),
                 pos=torch.empty(cap, dtype=torch.int32, device=DEV),
                 status=torch.zeros(1, dtype=torch.int32, device=DEV),
                 ws=torch.empty(12 * (R + 64), dtype=torch.int32, device=DEV))
    elif op == "quant":
        M, K = case["rows"], case["cols"]
        ld = -(-K // 16) * 16
        x = (rnd(M, K) * torch.exp(rnd(M, 1))).to(TYPES[case["type"]])
        s.update(x=x, y=torch.zeros(M, ld, dtype=torch.uint8, device=DEV)[:, :K],
                 scale=torch.empty(-(-K // BLOCK), M, device=DEV).t())
    elif op == "product":
        M, N, K = case["m"], case["n"], case["k"]
        nb, nn, ld = -(-K // BLOCK), -(-N // BLOCK), -(-K // 16) * 16
        a8, a_scale = _quantise(rnd(M, K) * torch.exp(rnd(M, 1)))
        a = torch.zeros(M, ld, dtype=torch.uint8, device=DEV)
        a[:, :K] = a8.view(torch.uint8)
        b = torch.zeros(N, ld, dtype=torch.uint8, device=DEV)
        b[:, :K] = (rnd(N, K) * 100).clamp(-FP8_MAX, FP8_MAX).to(F8).view(torch.uint8)
        s.update(a=a[:, :K], a_scale=a_scale.t().contiguous().t(), b=b[:, :K],
                 b_scale=1e-3 * torch.exp(0.3 * rnd(nn, nb)),
                 c=torch.empty(M, N, dtype=TYPES[case["out"]], device=DEV))
    else:
        T = case["tokens"]
        Hq, Hk, D, rot = (case["q_heads"], case["k_heads"], case["dim"], case["rot"]) if op == "heads" else (64, 1, 128, 64)
        dt = TYPES[case["type"]]
        s.update(rot=rot, q=(rnd(T, Hq, D) * 2).to(dt), k=(rnd(T, Hk, D) * 2 + 0.5).to(dt),
                 pos=ints(0, N_POS, T).int(), cos_sin=_rotation_table(N_POS, rot, DEV),
                 k_weight=1 + 0.2 * rnd(D), k_bias=0.2 * rnd(D))
        if op == "heads":
            s.update(q_weight=1 + 0.2 * rnd(D), q_bias=0.2 * rnd(D),
                     q_out=torch.empty(T, Hq, D, dtype=dt, device=DEV),
                     k_out=torch.empty(T, Hk, D, dtype=dt, device=DEV))
        else:
            n = case["slots"]
            s.update(w=rnd(T, 64), slot=torch.randperm(n, device=DEV, generator=g)[:T].contiguous(),
                     q8=torch.empty(T, 64, 128, dtype=torch.uint8, device=DEV),
                     w_out=torch.empty(T, 64, device=DEV),
                     cache=(rnd(n, 128) * 50).to(F8).view(torch.uint8),
                     cache_scale=0.02 * torch.exp(0.5 * rnd(n)), w_mul=64 ** -0.5 * 128 ** -0.5)
    return s


# ---------------------------------------------------------------- plain forms
def _pages(s):
    P, table, R = s["page"], s["table"], s["rows"]
    done = s["done_rows"] != 0
    lens = torch.where(done, 0, s["lens"])
    # the finished requests' pages go on top of the stack of free pages
    back = torch.where(done, (s["lens"] + P - 1) // P, 0)
    back_begin = back.cumsum(0) - back
    col = torch.arange(table.shape[1], device=table.device)
    n = s["free"].shape[0]
    to = torch.where(col < back[:, None], s["count"] + back_begin[:, None] + col, n)
    stack = torch.cat([s["free"], s["free"].new_zeros(1)])
    stack[to] = table
    s["free"].copy_(stack[:n])
    count = s["count"] + back.sum()
    # new pages come off the top, requests in order
    old = (lens + P - 1) // P
    need = (lens + s["new"] + P - 1) // P - old
    nth = (need.cumsum(0) - need)[:, None] + col - old[:, None]
    fresh = (col >= old[:, None]) & (col < (old + need)[:, None])
    table.copy_(torch.where(fresh, stack[(count - 1 - nth).clamp(0, n)], table))
    s["len_out"].copy_(lens + s["new"])
    s["count_out"].copy_(count - need.sum())
    ends = s["new"].cumsum(0)
    s["row_begin"][0] = 0
    s["row_begin"][1:] = ends
    t = torch.arange(s["slot"].shape[0], device=table.device)
    row = torch.searchsorted(ends, t, right=True)
    real = row < R
    row_c = row.clamp_max(R - 1)
    pos = lens[row_c] + t - (ends - s["new"])[row_c]
    pos = torch.where(real, pos, 0)
    page = table[row_c, pos // P].long()
    s["slot"].copy_(torch.where(real, page * P + pos % P, -1))
    s["row"].copy_(torch.where(real, row, -1))
    s["pos"].copy_(torch.where(real, pos, -1))
    return _pages_out(s)


def _pages_out(s):
    return {k: s[k] for k in ("table", "free", "len_out", "count_out", "row_begin", "slot", "row", "pos", "status")}


def _blocks(x):
    m, k = x.shape
    nb = -(-k // BLOCK)
    if nb * BLOCK != k:
        x = torch.cat([x, x.new_zeros(m, nb * BLOCK - k)], 1)
    return x.view(m, nb, BLOCK)


def _to_fp8(x):
    """Codes and scales of the last dimension's blocks."""
    scale = (x.abs().amax(-1) / FP8_MAX).clamp_min(SCALE_MIN)
    return (x / scale[..., None]).to(F8), scale


def _quant(s):
    y, scale = _to_fp8(_blocks(s["x"].float()))
    s["y"].copy_(y.flatten(1)[:, :s["cols"]].view(torch.uint8))
    s["scale"].copy_(scale)
    return {"y": s["y"].view(F8), "scale": s["scale"]}


def _product(s):
    a, b = (_blocks(s[n].view(F8).float()) for n in ("a", "b"))
    a = (a * s["a_scale"][:, :, None]).flatten(1)
    rows = s["b_scale"].repeat_interleave(BLOCK, 0)[:s["n"]]
    b = (b * rows[:, :, None]).flatten(1)
    s["c"].copy_(torch.matmul(a, b.t()))
    return s["c"]


def _norm(x, kind, weight, bias):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    return x + bias if kind == "layer" else x


def _rotate(x, s):
    """The first `rot` values of each head turned by the token's angles."""
    rot = s["rot"]
    h = rot // 2
    cs = s["cos_sin"][s["pos"].long()][:, None, :]
    c, d = cs[..., :h], cs[..., h:]
    r = x[..., :rot]
    if s["pairs"] == "half":
        u, v = r[..., :h], r[..., h:]
        r = torch.cat([u * c - v * d, v * c + u * d], -1)
    else:
        u, v = r[..., 0::2], r[..., 1::2]
        r = torch.stack([u * c - v * d, v * c + u * d], -1).flatten(-2)
    return torch.cat([r, x[..., rot:]], -1)


def _heads(s):
    q = _rotate(_norm(s["q"].float(), s["norm"], s["q_weight"], s["q_bias"]), s)
    k = _rotate(_norm(s["k"].float(), s["norm"], s["k_weight"], s["k_bias"]), s)
    s["q_out"].copy_(q)
    s["k_out"].copy_(k)
    return {"q": s["q_out"], "k": s["k_out"]}


def _indexer(s):
    q, q_scale = _to_fp8(_rotate(s["q"].float(), s))
    k, k_scale = _to_fp8(_rotate(_norm(s["k"].float(), "layer", s["k_weight"], s["k_bias"]), s))
    s["q8"].copy_(q.view(torch.uint8))
    s["w_out"].copy_(s["w"] * q_scale * s["w_mul"])
    s["cache"][s["slot"]] = k[:, 0].view(torch.uint8)
    s["cache_scale"][s["slot"]] = k_scale[:, 0]
    return _indexer_out(s)


def _indexer_out(s):
    return {"q8": s["q8"].view(F8), "w_out": s["w_out"], "cache": s["cache"].view(F8),
            "cache_scale": s["cache_scale"]}


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    from dsa_indexer_top_amd import binding as B
    op = s["op"]
    if op == "pages":
        B.page_step(s["lens"], s["new"], s["table"], s["page"], s["free"], s["count"], s["len_out"],
                    s["count_out"], s["row_begin"], s["slot"], s["row"], s["pos"], s["status"], s["ws"],
                    done=s["done_rows"])
        return _pages_out(s)
    if op == "quant":
        B.quant_fp8(s["x"], s["y"], s["scale"])
        return {"y": s["y"].view(F8), "scale": s["scale"]}
    if op == "product":
        B.matmul_fp8(s["a"], s["a_scale"], s["b"], s["b_scale"], s["c"])
        return s["c"]
    next_pairs = s["pairs"] == "next"
    if op == "heads":
        norm = B.NORM_RMS if s["norm"] == "rms" else B.NORM_LAYER
        qb, kb = (None, None) if s["norm"] == "rms" else (s["q_bias"], s["k_bias"])
        B.qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["pos"], s["cos_sin"],
                       q_norm=norm, q_weight=s["q_weight"], q_bias=qb, k_norm=norm,
                       k_weight=s["k_weight"], k_bias=kb, eps=EPS, interleaved=next_pairs)
        return {"q": s["q_out"], "k": s["k_out"]}
    B.indexer_qk(s["q"], s["k"], s["w"], s["q8"], s["w_out"], s["cache"], s["cache_scale"], s["slot"],
                 s["pos"], s["cos_sin"], w_mul=s["w_mul"], k_norm=B.NORM_LAYER,
                 k_weight=s["k_weight"], k_bias=s["k_bias"], eps=EPS, interleaved=next_pairs)
    return _indexer_out(s)


PLAIN = {"pages": _pages, "quant": _quant, "product": _product, "heads": _heads, "indexer": _indexer}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits
def _turned(x, pos, table, rot, pairs):
    """Each pair (x_i, x_j) as a complex number times that of its angle."""
    x = x.clone()
    half = rot // 2
    angle = torch.complex(table[:, :half].double(), table[:, half:].double())[pos.long()][:, None]
    i = torch.arange(half, device=x.device)
    first, second = (i, i + half) if pairs == "half" else (2 * i, 2 * i + 1)
    z = torch.complex(x[..., first], x[..., second]) * angle
    x[..., first], x[..., second] = z.real, z.imag
    return x


def _normed(x, kind, weight, bias):
    if kind == "layer":
        d = x - x.sum(-1, keepdim=True) / x.shape[-1]
        return d / ((d * d).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double() + bias.double()
    return x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()


def exact(case, seed):
    op = case["op"]
    if op == "pages":
        return None                                # whole numbers only
    s = prepare(case, seed)
    if op == "quant":
        x = s["x"].double()
        M, K = x.shape
        scale = torch.stack([c.abs().max(1).values for c in x.split(BLOCK, 1)], 1) / FP8_MAX
        scale = scale.clamp_min(SCALE_MIN)
        # the values that the codes stand for, before their rounding
        return {"y": x / scale.repeat_interleave(BLOCK, 1)[:, :K], "scale": scale}
    if op == "product":
        a, b = s["a"].view(F8).double(), s["b"].view(F8).double()
        a = a * s["a_scale"].double().repeat_interleave(BLOCK, 1)[:, :case["k"]]
        n = torch.arange(case["n"], device=b.device) // BLOCK
        b = b * s["b_scale"].double()[n].repeat_interleave(BLOCK, 1)[:, :case["k"]]
        return a @ b.t()
    q, k = s["q"].double(), s["k"].double()
    turn = lambda x: _turned(x, s["pos"], s["cos_sin"], s["rot"], case["pairs"])
    if op == "heads":
        return {"q": turn(_normed(q, case["norm"], s["q_weight"], s["q_bias"])),
                "k": turn(_normed(k, case["norm"], s["k_weight"], s["k_bias"]))}
    q, k = turn(q), turn(_normed(k, "layer", s["k_weight"], s["k_bias"]))[:, 0]
    qs = (q.abs().max(-1).values / FP8_MAX).clamp_min(SCALE_MIN)
    ks = (k.abs().max(-1).values / FP8_MAX).clamp_min(SCALE_MIN)
    cache, cache_scale = s["cache"].view(F8).double(), s["cache_scale"].double()
    cache[s["slot"]] = k / ks[:, None]
    cache_scale[s["slot"]] = ks
    return {"q8": q / qs[..., None], "w_out": s["w"].double() * qs * s["w_mul"], "cache": cache,
            "cache_scale": cache_scale}
