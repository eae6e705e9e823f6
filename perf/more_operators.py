"""Operators behind the scores, as cases to measure: the blocks that scores select, attention over
listed tokens or blocks of a latent cache, attention of a batch over a shared prefix and each
request's own tokens, the attention weight that each listed token got, and its accumulation into the
pool's eviction order.

run() computes a case in plain torch operations in 32 bits, or, with `own` set, through
dsa_indexer_top_amd.binding.  exact() is the definition in 64 bits."""

import math

import torch

own = False

if torch.cuda.is_available():
    DEV = "cuda"
else:
    DEV = "cpu"

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
ROW, VAL = 576, 512              # values of a latent row, and those that are summed
SCALE = 192 ** -0.5              # heads of 128 + 64 values before they are absorbed
UNIT = 2.0 ** 32                 # an entry's weight is added up in units of 1 / UNIT
NINF = float("-inf")
WORKSPACE = 1 << 28              # bytes that a program keeps for its steps


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a small decode step: the blocks of 64 tokens that 4 requests attend to
        dict(name="blocks 4 x 8192", op="blocks", rows=4, ctx=8192, block=64, k=32, first=1, last=2),
        # a chunk of a prefill with contexts of up to 65536 tokens
        dict(name="blocks 4096 x 65536", op="blocks", rows=4096, ctx=65536, block=128, k=64, first=1, last=2),
        # one token of one request, the 16 heads that a GPU has of 128, 2048 selected pool slots
        dict(name="sparse 1 x 16", op="sparse", rows=1, heads=16, k=2048, block=1, ctx=0, type="bf16"),
        # a decode step of 8 requests: every head over the 2048 pool slots of each selection
        dict(name="sparse 8 x 128", op="sparse", rows=8, heads=128, k=2048, block=1, ctx=0, type="bf16"),
        # blocks of 64 tokens in a paged cache, lengths that end inside a block, heads that fill no tile
        dict(name="sparse blocks 37 x 20", op="sparse", rows=37, heads=20, k=29, block=64, ctx=9000, type="fp16"),
        # a chunk of a prefill: each of 2048 query tokens over its own 2048 positions of a paged cache
        dict(name="sparse 2048 x 128", op="sparse", rows=2048, heads=128, k=2048, block=1, ctx=16384, type="bf16"),
        # a few requests behind one system prompt
        dict(name="prefix 5 x 16", op="prefix", rows=5, heads=16, groups=1, prefix=3000, own=200, type="bf16"),
        # a batch of 64 in two groups, each behind a document of up to 32768 tokens
        dict(name="prefix 64 x 16 x 32768", op="prefix", rows=64, heads=16, groups=2, prefix=32768, own=2048,
             type="bf16"),
        # what each of the 2048 selected tokens of one request got from 16 heads
        dict(name="weights 1 x 16", op="weights", rows=1, heads=16, k=2048, block=1, ctx=0, type="bf16"),
        # ... and of a decode step of 64 requests from 128 heads
        dict(name="weights 64 x 128", op="weights", rows=64, heads=128, k=2048, block=1, ctx=0, type="bf16"),
        # the selection's weights of 8 requests onto a pool of 32768 slots
        dict(name="weigh 8 x 2048 of 32768", op="weigh", rows=8, k=2048, slots=32768),
        # ... of 64 requests onto a million slots
        dict(name="weigh 64 x 2048 of 1048576", op="weigh", rows=64, k=2048, slots=1 << 20),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(["blocks", "sparse", "sparse", "prefix", "weights", "weigh"])
    if op == "blocks":
        ctx = _log(rng, 1024, 131072)
        return dict(op=op, rows=_log(rng, 1, min(4096, (4096 * 65536) // ctx)), ctx=ctx,
                    block=rng.choice([16, 32, 64, 128]), k=_log(rng, 4, 128), first=rng.randint(0, 2), last=rng.randint(0, 3))
    if op in ("sparse", "weights"):
        heads = rng.choice([1, 8, 16, 32, 64, 128, rng.randint(2, 127)])
        block = rng.choice([1, 1, 16, 64])
        paged = block > 1 or rng.random() < 0.5
        k = _log(rng, 64, 4096) // block + 1
        most = (2048 if paged else 256) * 128 * 2048 // (heads * k * block)
        return dict(op=op, rows=_log(rng, 1, max(1, min(2048 if paged else 256, most))), heads=heads, k=k, block=block,
                    ctx=_log(rng, max(64, k * block // 2), 16384) if paged else 0, type=rng.choice(["bf16", "fp16"]))
    if op == "prefix":
        rows, heads = _log(rng, 1, 64), rng.choice([1, 8, 16, rng.randint(2, 31)])
        return dict(op=op, rows=rows, heads=heads, groups=rng.randint(1, max(1, min(4, rows))), prefix=_log(rng, 64, 32768),
                    own=_log(rng, 1, 2048), type=rng.choice(["bf16", "fp16"]))
    return dict(op=op, rows=_log(rng, 1, 64), k=_log(rng, 64, 2048), slots=_log(rng, 1 << 14, 1 << 20))


def work(case):
    """Whole lengths where prepare() draws them; the rows of a cache that several queries list count once."""
    op, rows = case["op"], case["rows"]
    if op == "blocks":
        mean = case["ctx"] * 3 // 4
        return dict(bytes=rows * (4 * mean + 4 + 4 * case["k"]), flops=rows * mean)
    if op == "weigh":
        n = min(rows * case["k"], case["slots"])
        return dict(bytes=n * 12 + case["slots"] * 13, flops=n)
    heads = case["heads"]
    if op == "prefix":
        once = case["groups"] * case["prefix"] * 7 // 8 + rows * case["own"] // 2
        pairs = rows * heads * (case["prefix"] * 7 // 8 + case["own"] // 2)
        return dict(bytes=2 * (once * ROW + rows * heads * (ROW + VAL)) + 4 * rows * heads, flops=2 * (ROW + VAL) * pairs)
    tok = case["k"] * case["block"]
    if case["ctx"]:
        tok = min(tok, case["ctx"] * 3 // 4)
    unique = min(rows * tok, REQUESTS * case["ctx"]) if case["ctx"] else rows * tok
    pairs = rows * heads * tok
    if op == "weights":
        return dict(bytes=2 * ROW * (unique + rows * heads) + 4 * rows * (heads + 2 * tok), flops=2 * ROW * pairs)
    return dict(bytes=2 * (ROW * (unique + rows * heads) + VAL * rows * heads) + 4 * rows * (heads + case["k"]),
                flops=2 * (ROW + VAL) * pairs)


# ---------------------------------------------------------------- inputs
PAGE = 64
REQUESTS = 4                     # that the query rows of a paged case belong to


def _pages(g, rows, tokens, first=0):
    """Page tables of `rows` requests of up to `tokens` tokens, their pages in no order, and the pages' number."""
    width = max(1, -(-tokens // PAGE))
    n = rows * width
    return (first + torch.randperm(n, device=DEV, generator=g).int()).view(rows, width), n


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=g)
    ints = lambda lo, hi, *s: torch.randint(lo, hi, s, device=DEV, generator=g)
    op, R = case["op"], case["rows"]
    s = dict(case, ws=torch.empty(WORKSPACE, dtype=torch.uint8, device=DEV))
    if op == "blocks":
        ctx, k = case["ctx"], case["k"]
        lens = ints(ctx // 2, ctx + 1, R).int()
        s.update(scores=rnd(R, ctx), lens=lens, idx=torch.empty(R, k, dtype=torch.int32, device=DEV))
        return s
    if op == "weigh":
        n, k = case["slots"], min(case["k"], case["slots"] // R)
        slot = torch.randperm(n, device=DEV, generator=g)[:R * k].int().view(R, k).clone()
        slot[ints(0, 64, R, k) == 0] = -1                       # selections shorter than k
        w = rnd(R, k).exp()
        flat = slot.flatten()
        free = (ints(0, 16, n) == 0).to(torch.uint8)
        free[flat[flat >= 0].long()] = 0                        # a listed slot holds a row
        fresh = torch.where(ints(0, 8, R * k) == 0, flat, -1).int()
        s.update(slot=slot, w=w / w.sum(1, keepdim=True) * 128, free=free, fresh=fresh.contiguous(), mass=rnd(n).exp(),
                 priority=torch.zeros(n, dtype=torch.int32, device=DEV), decay=0.9)
        return s
    H, dt = case["heads"], TYPES[case["type"]]
    s.update(q=rnd(R, H, ROW).to(dt), out=torch.empty(R, H, VAL, dtype=dt, device=DEV),
             lse=torch.empty(R, H, device=DEV))
    if op == "prefix":
        G, pre, n_own = case["groups"], case["prefix"], case["own"]
        begin = torch.linspace(0, R, G + 1, dtype=torch.float64, device=DEV).round().int()
        prefix_table, n0 = _pages(g, G, pre)
        own_table, n1 = _pages(g, R, n_own, n0)
        s.update(kv=rnd((n0 + n1) * PAGE, ROW).to(dt), begin=begin, prefix_table=prefix_table, own_table=own_table,
                 prefix_len=ints(max(1, pre * 3 // 4), pre + 1, G).int(), own_len=ints(0, n_own + 1, R).int())
        return s
    k, B, ctx = case["k"], case["block"], case["ctx"]
    if ctx:                                                     # positions or blocks of a paged cache
        table, n = _pages(g, REQUESTS, ctx)
        lens = ints(max(1, ctx // 2), ctx + 1, R).int()
        n_blk = (lens + B - 1) // B
        width = -(-ctx // B)
        order = torch.rand(R, width, device=DEV, generator=g)   # a random choice of each row's blocks
        order.masked_fill_(torch.arange(width, device=DEV) >= n_blk[:, None], 2.0)
        v, i = order.topk(min(k, width), 1, largest=False)
        idx = torch.full((R, k), -1, dtype=torch.int32, device=DEV)
        idx[:, :i.shape[1]] = torch.where(v < 1.5, i, width).sort(1).values.int()
        idx[idx >= width] = -1
        s.update(kv=rnd(n * PAGE, ROW).to(dt), table=table, lens=lens, req=(torch.arange(R, device=DEV) * REQUESTS // R).int(),
                 idx=idx)
    else:                                                       # slots of a pool
        n = max(65536, 2 * R * k)
        idx = torch.randperm(n, device=DEV, generator=g)[:R * k].int().view(R, k).clone()
        short = ints(k // 2, k + 1, R)
        short[0] = k
        idx[torch.arange(k, device=DEV) >= short[:, None]] = -1
        s.update(kv=rnd(n, ROW).to(dt), idx=idx)
    if op == "weights":
        s.update(w=torch.empty(R, k * B, device=DEV))
        s["lse"] = _lse(s)
    return s


# ---------------------------------------------------------------- plain forms
def _blocks(s):
    R, ctx, B, k = s["rows"], s["ctx"], s["block"], s["k"]
    nb = -(-ctx // B)
    x = torch.full((R, nb * B), NINF, device=s["scores"].device)
    x[:, :ctx] = torch.where(torch.arange(ctx, device=x.device) < s["lens"][:, None], s["scores"], NINF)
    m = x.view(R, nb, B).amax(2)
    b, n = torch.arange(nb, device=x.device), ((s["lens"] + B - 1) // B)[:, None]
    real = b < n
    m = torch.where((b < s["first"]) | (b >= n - s["last"]), math.inf, m)
    m = torch.where(real, m, NINF)
    order = m.sort(dim=1, descending=True, stable=True).indices[:, :k]
    order = torch.where(torch.gather(real, 1, order), order, nb).sort(1).values
    s["idx"].fill_(-1)
    s["idx"][:, :order.shape[1]] = torch.where(order < nb, order, -1).int()
    return s["idx"]


def _listed_rows(s):
    """Cache row of each listed token and whether there is one, [rows, k * block]."""
    B = s["block"]
    e = s["idx"].long()
    pos = (e[:, :, None] * B + torch.arange(B, device=e.device)).flatten(1)
    real = (e >= 0)[:, :, None].expand(-1, -1, B).flatten(1)
    if not s["ctx"]:
        return pos.clamp_min(0), real
    real = real & (pos < s["lens"][:, None])
    pos = torch.where(real, pos, 0)
    return s["table"][s["req"].long()[:, None], pos // PAGE].long() * PAGE + pos % PAGE, real


def _scores(s):
    """Scaled products of every head with its row's listed tokens, -inf where there is none, and the tokens' latents."""
    at, real = _listed_rows(s)
    kv = s["kv"][at].float()
    x = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * SCALE
    return x.masked_fill_(~real[:, None, :], NINF), kv


def _softmax(x):
    """Softmax over the last dimension and its log sum; rows without a token: zeros and -inf."""
    m = x.amax(-1, keepdim=True).clamp_min(-3e38)
    p = (x - m).exp()
    z = p.sum(-1, keepdim=True)
    return p / z.clamp_min(1e-38), (m + z.log()).squeeze(-1)


def _lse(s):
    x, _ = _scores(s)
    return _softmax(x)[1].contiguous()


def _sparse(s):
    x, kv = _scores(s)
    p, lse = _softmax(x)
    s["out"].copy_(torch.matmul(p, kv[:, :, :VAL]))
    s["lse"].copy_(lse)
    return {"out": s["out"], "lse": s["lse"]}


def _prefix(s):
    """The prefix of each group against all of the batch's heads, masked to the group's, then the own tokens."""
    R, H = s["rows"], s["heads"]
    q = s["q"].float()
    dev = q.device
    r = torch.arange(R, device=dev)
    grp = torch.searchsorted(s["begin"][1:].contiguous(), r.int(), right=True)
    pos = torch.arange(s["prefix"], device=dev)
    pre = s["kv"][s["prefix_table"].long()[:, pos // PAGE] * PAGE + pos % PAGE].float()            # [G, prefix, 576]
    x = torch.matmul(q.view(1, R * H, ROW), pre.transpose(1, 2)) * SCALE                           # [G, R H, prefix]
    here = (grp == torch.arange(s["groups"], device=dev)[:, None])[:, :, None] & (pos < s["prefix_len"][:, None])[:, None, :]
    x = x.view(-1, R, H, s["prefix"]).masked_fill_(~here[:, :, None, :], NINF)
    pos = torch.arange(s["own"], device=dev)
    mine = s["kv"][s["own_table"].long()[:, pos // PAGE] * PAGE + pos % PAGE].float()              # [R, own, 576]
    y = (torch.matmul(q, mine.transpose(1, 2)) * SCALE).masked_fill_(~(pos < s["own_len"][:, None])[:, None, :], NINF)
    m = torch.maximum(x.amax(-1).amax(0), y.amax(-1)).clamp_min(-3e38)[..., None]
    x, y = (x - m).exp(), (y - m).exp()
    z = x.sum(-1).sum(0) + y.sum(-1)
    o = torch.matmul(x.view(-1, R * H, s["prefix"]), pre[:, :, :VAL]).sum(0).view(R, H, VAL) + torch.matmul(y, mine[:, :, :VAL])
    s["out"].copy_(o / z.clamp_min(1e-38)[..., None])
    s["lse"].copy_(m[..., 0] + z.log())
    return {"out": s["out"], "lse": s["lse"]}


def _weights(s):
    x, _ = _scores(s)
    s["w"].copy_((x - s["lse"][:, :, None].clamp_min(-3e38)).exp().sum(1))
    return s["w"]


def _weigh(s):
    n = s["slots"]
    at = torch.where(s["slot"] >= 0, s["slot"], n).long().flatten()
    sums = torch.zeros(n + 1, dtype=torch.int64, device=at.device)
    sums.index_add_(0, at, (s["w"].flatten() * UNIT).round().long())
    old = torch.cat([s["mass"], s["mass"].new_zeros(1)]) * s["decay"]
    old[torch.where(s["fresh"] >= 0, s["fresh"], n).long()] = 0
    mass = old[:n] + sums[:n].float() / UNIT
    s["mass"].copy_(torch.where(s["free"] != 0, 0, mass))
    s["priority"].copy_(torch.where(s["free"] != 0, -1, s["mass"].view(torch.int32)))
    return {"mass": s["mass"], "priority": s["priority"]}


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    from dsa_indexer_top_amd import binding as B
    op = s["op"]
    if op == "blocks":
        B.block_topk(s["scores"], s["lens"], s["ctx"], s["block"], s["k"], s["idx"], s["ws"], n_first=s["first"],
                     n_last=s["last"])
        return s["idx"]
    if op == "weigh":
        B.pool_weigh(s["free"], s["priority"], s["mass"], s["slot"], s["w"], s["ws"], decay=s["decay"], fresh=s["fresh"])
        return {"mass": s["mass"], "priority": s["priority"]}
    if op == "prefix":
        B.prefix_attention(s["q"], s["kv"], s["out"], SCALE, s["begin"], s["prefix_len"], s["prefix_table"], s["own_len"],
                           s["own_table"], PAGE, s["prefix"], s["own"], s["ws"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    where = dict(block=s["block"])
    if s["ctx"]:
        where.update(length=s["lens"], page_table=s["table"], page_size=PAGE, req=s["req"])
    if op == "weights":
        B.attention_weights(s["q"], s["kv"], s["idx"], s["lse"], s["w"], SCALE, **where)
        return s["w"]
    B.sparse_attention(s["q"], s["kv"], s["idx"], s["out"], SCALE, s["ws"], lse=s["lse"], **where)
    return {"out": s["out"], "lse": s["lse"]}


PLAIN = {"blocks": _blocks, "sparse": _sparse, "prefix": _prefix, "weights": _weights, "weigh": _weigh}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits
def _rows_of(s, r):
    """Cache rows that query row r attends to, in list order, and their places in the list."""
    B, e = s["block"], s["idx"][r].long()
    j = torch.arange(e.numel() * B, device=e.device)
    pos = e[j // B] * B + j % B
    keep = e[j // B] >= 0
    if s["ctx"]:
        keep &= pos < s["lens"][r]
    j, pos = j[keep], pos[keep]
    if s["ctx"]:
        pos = s["table"][s["req"][r].long()][pos // PAGE].long() * PAGE + pos % PAGE
    return pos, j


def exact(case, seed):
    op = case["op"]
    if op == "blocks":
        return None                                # whole numbers only
    s = prepare(case, seed)
    R = case["rows"]
    if op == "weigh":
        mass = s["mass"].double() * s["decay"]
        mass[s["fresh"][s["fresh"] >= 0].long()] = 0
        take = s["slot"] >= 0
        mass.index_add_(0, s["slot"][take].long(), s["w"][take].double())
        mass[s["free"] != 0] = 0
        return {"mass": mass, "priority": None}
    q = s["q"].double()
    if op == "weights":
        w = torch.zeros(R, case["k"] * case["block"], dtype=torch.float64, device=q.device)
        for r in range(R):
            at, j = _rows_of(s, r)
            w[r, j] = torch.exp(SCALE * (s["kv"][at].double() @ q[r].t()) - s["lse"][r].double()).sum(1)
        return w
    out = torch.zeros(*s["out"].shape, dtype=torch.float64, device=q.device)
    lse = torch.full(s["lse"].shape, NINF, dtype=torch.float64, device=q.device)
    for r in range(R):
        if op == "sparse":
            at = _rows_of(s, r)[0]
        else:
            at = []
            for gi in range(case["groups"]):
                if s["begin"][gi] <= r < s["begin"][gi + 1]:
                    t = torch.arange(int(s["prefix_len"][gi]), device=q.device)
                    at.append(s["prefix_table"][gi].long()[t // PAGE] * PAGE + t % PAGE)
            t = torch.arange(int(s["own_len"][r]), device=q.device)
            at = torch.cat(at + [s["own_table"][r].long()[t // PAGE] * PAGE + t % PAGE])
        if at.numel():
            kv = s["kv"][at].double()
            x = SCALE * (q[r] @ kv.t())
            lse[r] = torch.logsumexp(x, 1)
            out[r] = torch.exp(x - lse[r][:, None]) @ kv[:, :VAL]
    return {"out": out, "lse": lse}
