"""Attention over listed rows, blocks and shared prefixes of a latent cache, and the weights of its tokens,
against the definition in 64 bits: heads that fill no tile, lengths from nothing on, lists with holes
and repetitions, pages that end inside a tile, NaN and infinities in rows that are passed over, strides, chunks,
graphs, streams."""

import numpy as np
import pytest
import torch

from attention_util import SCALE, TYPES, check, f64, rand, score_error
from dsa_indexer_top_amd import binding as B
from gpu_util import announce, dev, host
from oracle import attention as oa

pytestmark = pytest.mark.gpu


def workspace(n):
    return torch.empty(max(int(n), 256), dtype=torch.uint8, device="cuda")


def sparse(q, kv, idx, block=1, length=None, table=None, page=0, req=None, scale=SCALE, out=None, stream=None):
    """The call with a fresh workspace of just the size it asks for; q, kv on the device, the rest numpy."""
    R, H = q.shape[:2]
    out = torch.empty(R, H, 512, dtype=q.dtype, device="cuda") if out is None else out
    lse = torch.empty(R, H, device="cuda")
    ws = workspace(B.sparse_attention_workspace_bytes(R, H, idx.shape[1] * block))
    opt = lambda a: None if a is None else dev(np.asarray(a, np.int32))
    B.sparse_attention(q, kv, dev(np.asarray(idx, np.int32)), out, scale, ws, lse=lse, block=block, length=opt(length),
                       page_table=opt(table), page_size=page, req=opt(req), stream=stream)
    return out, lse


def lists(rng, R, k, n, holes=True):
    """k distinct rows of n for each query row, some of them missing."""
    idx = np.stack([rng.permutation(n)[:k] for _ in range(R)]).astype(np.int32).reshape(R, k)
    if holes and k:
        idx[rng.random((R, k)) < 0.2] = -1
    return idx


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("R,H,k", [(1, 1, 1), (2, 16, 63), (3, 5, 64), (2, 17, 65), (1, 32, 200), (2, 40, 130), (1, 64, 128),
                                   (1, 100, 70), (3, 16, 0)])
def test_listed_rows(t, R, H, k):
    rng = np.random.default_rng(R * 1000 + H + k)
    n = 2 * k + 5
    announce("sparse", t, R, H, k)
    q, kv, idx = rand(rng, (R, H, 576), t).cuda(), rand(rng, (n, 576), t).cuda(), lists(rng, R, k, n)
    out, lse = sparse(q, kv, idx)
    check(out, lse, q, kv, [r for _, r in oa.listed_rows(idx, 1, n)])


@pytest.mark.parametrize("t,R,H,k", [("bf16", 8, 128, 2048), ("fp16", 1, 16, 2048), ("bf16", 300, 16, 777), ("bf16", 70, 128, 1000)])
def test_listed_rows_full(t, R, H, k):
    rng = np.random.default_rng(7)
    n = 20000
    announce("sparse full", t, R, H, k)
    q, kv, idx = rand(rng, (R, H, 576), t).cuda(), rand(rng, (n, 576), t).cuda(), lists(rng, R, k, n)
    idx[0, 3:] = -1
    out, lse = sparse(q, kv, idx)
    check(out, lse, q, kv, [r for _, r in oa.listed_rows(idx, 1, n)])


def test_rows_without_tokens_and_repeated_tokens():
    rng = np.random.default_rng(3)
    q, kv = rand(rng, (5, 16, 576), "bf16").cuda(), rand(rng, (40, 576), "bf16").cuda()
    idx = np.full((5, 150), -1, np.int32)
    idx[1, 77] = 39                                        # one token, in the second tile
    idx[2] = 7                                             # one token 150 times
    idx[3, ::2] = rng.integers(0, 40, 75)
    idx[4, :4] = [40, 1 << 30, 2, -5]                      # rows behind the cache
    announce("no tokens, repeated tokens")
    out, lse = sparse(q, kv, idx)
    check(out, lse, q, kv, [r for _, r in oa.listed_rows(idx, 1, 40)])
    assert (host(out[0].float()) == 0).all() and np.isneginf(host(lse[0])).all()
    assert np.array_equal(host(out[1].float()), np.broadcast_to(host(kv[39, :512].float()), (16, 512)))
    assert np.array_equal(host(out[2].float()), np.broadcast_to(host(kv[7, :512].float()), (16, 512)))


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("block,page,k", [(1, 16, 90), (16, 16, 7), (64, 64, 3), (32, 16, 5), (64, 256, 4), (128, 64, 2), (1, 128, 64)])
def test_blocks_of_a_paged_cache(t, block, page, k):
    rng = np.random.default_rng(block * page + k)
    R, H, n_req, width = 6, 18, 3, -(-600 // page)
    announce("paged", t, block, page, k)
    pages = rng.permutation(n_req * width + 3)[:n_req * width].reshape(n_req, width)
    n_kv = (n_req * width + 3) * page
    kv = rand(rng, (n_kv, 576), t).cuda()
    q = rand(rng, (R, H, 576), t).cuda()
    length = np.array([0, 1, 130, 599, 600, 333])
    req = np.array([0, 2, 1, 0, 2, 1])
    idx = np.stack([rng.permutation(-(-640 // block))[:k] for _ in range(R)]).astype(np.int32)
    out, lse = sparse(q, kv, idx, block, length, pages, page, req)
    rows = [r for _, r in oa.listed_rows(idx, block, n_kv, length, pages, page, req)]
    check(out, lse, q, kv, rows)
    # the same rows without pages
    out2, _ = sparse(q, kv, np.array([np.concatenate([r, np.full(k * block - len(r), -1)]) for r in rows]))
    check(out2, None, q, kv, rows)


def test_what_is_passed_over_leaves_nothing():
    """NaN and infinities in rows that no position leads to, bad pages, requests that are none."""
    rng = np.random.default_rng(11)
    R, H, page, width = 5, 8, 16, 8
    n_kv = 20 * page
    kv = rand(rng, (n_kv, 576), "bf16").cuda()
    q = rand(rng, (R, H, 576), "bf16").cuda()
    table = rng.permutation(20)[:2 * width].reshape(2, width).astype(np.int32)
    table[0, 3], table[0, 5], table[1, 2] = -1, 20, 1 << 28
    length = np.array([100, 75, 128, 128, 40])
    req = np.array([0, 1, 2, -1, 0])
    idx = np.tile(np.arange(140, dtype=np.int32), (R, 1))
    rows = [r for _, r in oa.listed_rows(idx, 1, n_kv, length, table, page, req)]
    assert [len(r) for r in rows] == [68, 59, 0, 0, 40]
    used = np.unique(np.concatenate(rows))
    clean = kv.clone()
    bad = torch.full_like(kv, float("nan"))
    bad[::2] = float("inf")
    bad[used] = clean[used]
    announce("passed over")
    out, lse = sparse(q, bad, idx, 1, length, table, page, req)
    check(out, lse, q, clean, rows)
    w = torch.empty(R, 140, device="cuda")
    i = lambda a: dev(np.asarray(a, np.int32))
    B.attention_weights(q, bad, i(idx), lse, w, SCALE, length=i(length), page_table=i(table), page_size=page, req=i(req))
    assert np.isfinite(host(w)).all() and (host(w)[2:4] == 0).all()


def test_strides_and_neighbours_left_alone():
    rng = np.random.default_rng(5)
    R, H, n, k = 3, 7, 90, 70
    announce("strides")
    qb = rand(rng, (R, H + 2, 600), "bf16").cuda()
    q = qb[:, 1:H + 1, 8:584]
    kvb = rand(rng, (n, 640), "bf16").cuda()
    kv = kvb[:, 16:592]
    ob = torch.full((R, H + 1, 528), 9.0, dtype=torch.bfloat16, device="cuda")
    idx = lists(rng, R, k, n)
    wide = np.full((R, k + 3), 5, np.int32)
    wide[:, :k] = idx
    out, lse = ob[:, :H, 8:520], torch.empty(R, H, device="cuda")
    B.sparse_attention(q, kv, dev(wide)[:, :k], out, SCALE, workspace(B.sparse_attention_workspace_bytes(R, H, k)), lse=lse)
    check(out, lse, q, kv, [r for _, r in oa.listed_rows(idx, 1, n)])
    left = ob.clone()
    left[:, :H, 8:520] = 9.0
    assert (host(left.float()) == 9).all()


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_scales_and_wide_scores(scale):
    """No scale (the mean), a negative one, and scores of several hundred, whose maximum moves from tile to tile."""
    rng = np.random.default_rng(17)
    q, kv = rand(rng, (2, 16, 576), "bf16", 2.0).cuda(), rand(rng, (400, 576), "bf16", 2.0).cuda()
    idx = lists(rng, 2, 300, 400)
    announce("scale", scale)
    out, lse = sparse(q, kv, idx, scale=scale)
    check(out, lse, q, kv, [r for _, r in oa.listed_rows(idx, 1, 400)], scale)


def test_same_bits_again_and_without_lse():
    rng = np.random.default_rng(23)
    q, kv, idx = rand(rng, (4, 24, 576), "fp16").cuda(), rand(rng, (500, 576), "fp16").cuda(), lists(rng, 4, 400, 500)
    a, la = sparse(q, kv, idx)
    b, lb = sparse(q, kv, idx)
    assert np.array_equal(host(a.view(torch.int16)), host(b.view(torch.int16))) and np.array_equal(host(la), host(lb))
    out = torch.empty_like(a)
    B.sparse_attention(q, kv, dev(idx), out, SCALE, workspace(B.sparse_attention_workspace_bytes(4, 24, 400)))
    assert np.array_equal(host(a.view(torch.int16)), host(out.view(torch.int16)))


# ---------------------------------------------------------------- weights
@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("R,H,k,block", [(1, 1, 1, 1), (2, 16, 130, 1), (3, 33, 127, 1), (1, 128, 40, 1), (2, 20, 5, 64), (1, 7, 0, 1)])
def test_weights_of_tokens(t, R, H, k, block):
    rng = np.random.default_rng(R + H + k)
    announce("weights", t, R, H, k, block)
    n = (2 * k + 3) * block
    q, kv, idx = rand(rng, (R, H, 576), t).cuda(), rand(rng, (n, 576), t).cuda(), lists(rng, R, k, 2 * k + 3)
    length = rng.integers(n // 2, n + 1, R)
    out, lse = sparse(q, kv, idx, block, length)
    w = torch.full((R, k * block + 3), -7.0, device="cuda")
    B.attention_weights(q, kv, dev(idx), lse, w[:, :k * block], SCALE, block=block, length=dev(length.astype(np.int32)))
    listed = oa.listed_rows(idx, block, n, length)
    places, rows = [p for p, _ in listed], [r for _, r in listed]
    want = oa.token_weights(f64(q), f64(kv), places, rows, f64(lse), SCALE, k * block)
    _, want_lse, _, terms = oa.attention(f64(q), f64(kv), rows, SCALE)
    tol = want * score_error(terms, want_lse).max() + 1e-30
    got = host(w).astype(np.float64)
    assert (got[:, k * block:] == -7).all()
    assert (np.abs(got[:, :k * block] - want) <= tol).all()
    for r in range(R):
        if len(rows[r]):
            assert abs(got[r, :k * block].sum() - H) <= 1e-4 * H


@pytest.mark.parametrize("t,R,H,k", [("bf16", 40, 33, 1700), ("fp16", 300, 40, 130), ("bf16", 600, 20, 70)])
def test_weights_of_many_rows_full(t, R, H, k):
    rng = np.random.default_rng(R + H)
    announce("weights, many rows", t, R, H, k)
    n = 3000
    q, kv, idx = rand(rng, (R, H, 576), t).cuda(), rand(rng, (n, 576), t).cuda(), lists(rng, R, k, n)
    idx[1], idx[2, 1:] = -1, -1
    out, lse = sparse(q, kv, idx)
    w = torch.full((R, k), -7.0, device="cuda")
    B.attention_weights(q, kv, dev(idx), lse, w, SCALE)
    listed = oa.listed_rows(idx, 1, n)
    places, rows = [p for p, _ in listed], [r for _, r in listed]
    want = oa.token_weights(f64(q), f64(kv), places, rows, f64(lse), SCALE, k)
    _, want_lse, _, terms = oa.attention(f64(q), f64(kv), rows, SCALE)
    assert (np.abs(host(w) - want) <= want * score_error(terms, want_lse).max() + 1e-30).all()


# ---------------------------------------------------------------- shared prefixes
def prefix_case(rng, R, H, groups, prefix, own, page, t):
    """groups: (first row, last row) pairs as a begin list; prefix lengths and own lengths given."""
    G = len(prefix)
    pw, ow = max(1, -(-max(list(prefix) + [1]) // page)), max(1, -(-max(list(own) + [1]) // page))
    perm = rng.permutation(G * pw + R * ow + 2)
    pt, ot = perm[:G * pw].reshape(G, pw), perm[G * pw:G * pw + R * ow].reshape(R, ow)
    n_kv = len(perm) * page
    return dict(q=rand(rng, (R, H, 576), t).cuda(), kv=rand(rng, (n_kv, 576), t).cuda(), begin=np.asarray(groups, np.int32),
                plen=np.asarray(prefix, np.int32), ptab=pt.astype(np.int32), olen=np.asarray(own, np.int32),
                otab=ot.astype(np.int32), page=page)


def run_prefix(c, max_prefix=None, max_own=None):
    R, H = c["q"].shape[:2]
    out, lse = torch.empty(R, H, 512, dtype=c["q"].dtype, device="cuda"), torch.empty(R, H, device="cuda")
    mp = int(c["plen"].max(initial=0)) if max_prefix is None else max_prefix
    mo = int(c["olen"].max(initial=0)) if max_own is None else max_own
    mp, mo = max(mp, 0), max(mo, 0)
    ws = workspace(B.prefix_attention_workspace_bytes(R, H, len(c["plen"]), mp, mo))
    B.prefix_attention(c["q"], c["kv"], out, SCALE, dev(c["begin"]), dev(c["plen"]), dev(c["ptab"]), dev(c["olen"]), dev(c["otab"]),
                       c["page"], mp, mo, ws, lse=lse)
    return out, lse


def prefix_rows(c, plen=None, olen=None):
    return oa.prefix_rows(c["q"].shape[0], c["kv"].shape[0], c["page"], c["begin"], c["plen"] if plen is None else plen,
                          c["ptab"], c["olen"] if olen is None else olen, c["otab"])


@pytest.mark.parametrize("t,R,H,groups,prefix,own,page", [
    ("bf16", 1, 1, [0, 1], [1], [0], 16),
    ("bf16", 5, 16, [0, 5], [200], [0, 1, 64, 65, 30], 16),
    ("fp16", 6, 3, [0, 2, 6], [70, 129], [5, 0, 17, 1, 2, 3], 64),
    ("bf16", 7, 9, [1, 1, 4, 6], [50, 64, 0], [3, 0, 2, 90, 0, 0, 12], 16),
    ("fp16", 4, 40, [0, 4], [300], [10, 20, 30, 40], 128),
    ("bf16", 3, 16, [0], [], [100, 0, 7], 16),
    ("bf16", 2, 16, [0, 2], [0], [0, 0], 16),
])
def test_shared_prefixes(t, R, H, groups, prefix, own, page):
    rng = np.random.default_rng(R * H)
    announce("prefix", t, R, H, groups, prefix, own, page)
    c = prefix_case(rng, R, H, groups, prefix, own, page, t)
    out, lse = run_prefix(c)
    check(out, lse, c["q"], c["kv"], prefix_rows(c))


def test_prefix_lengths_beyond_their_bounds():
    rng = np.random.default_rng(2)
    c = prefix_case(rng, 4, 16, [0, 3, 4], [100, 90], [40, 30, 20, 10], 16, "bf16")
    c["plen"][0], c["olen"][1], c["olen"][2] = 1 << 30, -4, 1000
    announce("prefix clamped")
    out, lse = run_prefix(c, 80, 25)
    clamp = lambda a, n: np.clip(a, 0, n)
    check(out, lse, c["q"], c["kv"], prefix_rows(c, clamp(c["plen"], 80), clamp(c["olen"], 25)))


@pytest.mark.parametrize("t", ["bf16"])
def test_shared_prefixes_full(t):
    rng = np.random.default_rng(9)
    R, H = 64, 16
    c = prefix_case(rng, R, H, [0, 20, 64], [9000, 5001], list(rng.integers(0, 700, R)), 64, t)
    announce("prefix full")
    out, lse = run_prefix(c)
    check(out, lse, c["q"], c["kv"], prefix_rows(c))


# ---------------------------------------------------------------- graphs and streams
def test_graph_replays_with_new_inputs():
    """One captured graph of attention, weights and the shared prefix, replayed with other inputs between eager work."""
    rng = np.random.default_rng(31)
    R, H, n, k = 3, 16, 300, 200
    q, kv = rand(rng, (R, H, 576), "bf16").cuda(), rand(rng, (n, 576), "bf16").cuda()
    idx = dev(lists(rng, R, k, n))
    out, lse, w = torch.empty(R, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(R, H, device="cuda"), torch.empty(R, k, device="cuda")
    ws = workspace(B.sparse_attention_workspace_bytes(R, H, k))
    c = prefix_case(rng, R, H, [0, 3], [150], [4, 0, 33], 16, "bf16")
    c["q"], c["kv"] = q, kv
    c["ptab"], c["otab"] = c["ptab"] % 18, c["otab"] % 18
    pout, plse = torch.empty_like(out), torch.empty_like(lse)
    pws = workspace(B.prefix_attention_workspace_bytes(R, H, 1, 150, 33))
    pa = [dev(c[x]) for x in ("begin", "plen", "ptab", "olen", "otab")]

    def enqueue(st):
        B.sparse_attention(q, kv, idx, out, SCALE, ws, lse=lse, stream=st)
        B.attention_weights(q, kv, idx, lse, w, SCALE, stream=st)
        B.prefix_attention(q, kv, pout, SCALE, *pa, 16, 150, 33, pws, lse=plse, stream=st)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = B.CapturedGraph(enqueue, st)
    for i in range(3):
        announce("replay", i)
        q.copy_(rand(rng, (R, H, 576), "bf16").cuda())
        new = lists(rng, R, k, n)
        idx.copy_(dev(new))
        torch.cuda.synchronize()
        graph.launch(st)
        torch.cuda.synchronize()
        listed = oa.listed_rows(new, 1, n)
        check(out, lse, q, kv, [r for _, r in listed])
        check(pout, plse, q, kv, prefix_rows(c))
        want = oa.token_weights(f64(q), f64(kv), [p for p, _ in listed], [r for _, r in listed], f64(lse), SCALE, k)
        assert np.abs(host(w) - want).max() <= 1e-3
    graph.close()


def test_other_stream_and_two_calls_at_once():
    rng = np.random.default_rng(41)
    sets = []
    for i in range(2):
        q, kv, idx = rand(rng, (2, 16, 576), "bf16").cuda(), rand(rng, (900, 576), "bf16").cuda(), lists(rng, 2, 800, 900)
        sets.append((q, kv, idx, torch.cuda.Stream()))
    torch.cuda.synchronize()
    announce("two streams")
    got = []
    for q, kv, idx, st in sets:
        with torch.cuda.stream(st):
            got.append(sparse(q, kv, idx))                  # torch's current stream
    torch.cuda.synchronize()
    for (q, kv, idx, _), (out, lse) in zip(sets, got):
        check(out, lse, q, kv, [r for _, r in oa.listed_rows(idx, 1, 900)])


# ---------------------------------------------------------------- sizes where something else runs
@pytest.mark.parametrize("R,H,k", [(130, 5, 1700), (131, 64, 1600)])
def test_long_chunks_full(R, H, k):
    """Rows that are not cut, of more tokens than a workgroup looks up at once."""
    rng = np.random.default_rng(R)
    n = 4000
    announce("long chunks", R, H, k)
    assert B.sparse_attention_workspace_bytes(R, H, k) == 0
    q, kv, idx = rand(rng, (R, H, 576), "bf16").cuda(), rand(rng, (n, 576), "bf16").cuda(), lists(rng, R, k, n)
    idx[1, 1536:] = -1
    idx[2, :1540] = -1
    out, lse = sparse(q, kv, idx)
    check(out, lse, q, kv, [r for _, r in oa.listed_rows(idx, 1, n)])


@pytest.mark.parametrize("R,H,groups,prefix,own", [
    (64, 16, [0, 33, 64], [17500, 16001], 70),             # two groups of 32 queries for the prefixes alone
    (70, 128, [0, 64, 70], [900, 33], 50)])                # for prefixes and own tokens
def test_shared_prefixes_of_many_queries_full(R, H, groups, prefix, own):
    rng = np.random.default_rng(R + H)
    c = prefix_case(rng, R, H, groups, prefix, list(rng.integers(0, own, R)), 64, "bf16")
    announce("prefix, many queries", R, H)
    out, lse = run_prefix(c)
    check(out, lse, c["q"], c["kv"], prefix_rows(c))


def test_many_groups():
    """More groups than a wave looks through at once, some of them empty."""
    rng = np.random.default_rng(17)
    R = 90
    begin = np.sort(np.concatenate([[0], rng.integers(0, R + 1, 150), [R]]))
    c = prefix_case(rng, R, 2, begin, list(rng.integers(0, 40, 151)), [0] * 45 + [5] * 45, 16, "fp16")
    announce("prefix, many groups")
    out, lse = run_prefix(c)
    check(out, lse, c["q"], c["kv"], prefix_rows(c))


def test_an_empty_cache():
    rng = np.random.default_rng(18)
    q, idx = rand(rng, (2, 16, 576), "bf16").cuda(), np.zeros((2, 70), np.int32)
    kv = torch.empty(0, 576, dtype=torch.bfloat16, device="cuda")
    announce("no cache")
    out, lse = sparse(q, kv, idx)
    assert not host(out.float()).any() and np.isneginf(host(lse)).all()
    w = torch.full((2, 70), 3.0, device="cuda")
    B.attention_weights(q, kv, dev(idx), lse, w, SCALE)
    assert not host(w).any()


@pytest.mark.parametrize("t", ["bf16", "fp16"])
def test_scores_that_keep_rising(t):
    """Every tile has a token far above all before it, so that sums and results are scaled again and again; some heads'
    scores fall instead."""
    rng = np.random.default_rng(19)
    n, H = 700, 40
    announce("rising", t)
    q, kv = rand(rng, (2, H, 576), t, 0.02), rand(rng, (n, 576), t)
    kv[:, 575] = (torch.arange(n) // 7).to(kv.dtype)       # whole numbers up to 100
    q[:, :, 575] = 4.0
    q[:, 30:, 575] = -4.0
    q, kv = q.cuda(), kv.cuda()
    idx = np.stack([np.arange(n), rng.permutation(n)]).astype(np.int32)
    out, lse = sparse(q, kv, idx, scale=1.0)
    check(out, lse, q, kv, [r for _, r in oa.listed_rows(idx, 1, n)], scale=1.0)


def test_a_cache_behind_32_bits_full():
    """Rows on either side of 2^31 and 2^32 bytes, in a cache of 4.6 GB; only the listed ones are numbers."""
    rng = np.random.default_rng(20)
    n, R, H, k, page = 4000000, 3, 20, 300, 64
    marks = [0, (1 << 31) // 1152, (1 << 32) // 1152, n - 2]
    rows = np.unique(np.concatenate([rng.integers(0, n, 1500)] + [np.arange(max(m - 3, 0), min(m + 2, n)) for m in marks]))
    announce("4.6 GB")
    q, small = rand(rng, (R, H, 576), "bf16").cuda(), rand(rng, (len(rows), 576), "bf16").cuda()
    kv = torch.empty(n, 576, dtype=torch.bfloat16, device="cuda")
    kv.fill_(float("nan"))
    kv[torch.from_numpy(rows).cuda()] = small
    at = np.stack([rng.permutation(len(rows))[:k] for _ in range(R)])
    near = [r for m in marks for r in range(max(m - 3, 0), m + 2) if r < n]
    at[:, :len(near)] = np.searchsorted(rows, near)
    idx = rows[at].astype(np.int32)
    idx[0, 30], idx[1, 31] = -1, n                         # none, and one row behind the end
    listed = [a[(i >= 0) & (i < n)] for a, i in zip(at, idx)]
    out, lse = sparse(q, kv, idx)
    check(out, lse, q, small, listed)
    w = torch.empty(R, k, device="cuda")
    B.attention_weights(q, kv, dev(idx), lse, w, SCALE)
    places = [np.flatnonzero((i >= 0) & (i < n)) for i in idx]
    want = oa.token_weights(f64(q), f64(small), places, listed, f64(lse), SCALE, k)
    _, want_lse, _, terms = oa.attention(f64(q), f64(small), listed, SCALE)
    assert (np.abs(host(w) - want) <= want * score_error(terms, want_lse).max() + 1e-30).all()
    # pages: the last one and the one around 2^32 bytes
    pages = np.array([n // page - 1, (1 << 32) // 1152 // page, 3], np.int32)
    paged = np.concatenate([np.arange(p * page, (p + 1) * page) for p in pages])
    dense = rand(rng, (len(paged), 576), "bf16").cuda()
    kv[torch.from_numpy(paged).cuda()] = dense
    out, lse = torch.empty_like(out), torch.empty_like(lse)
    ws = workspace(B.prefix_attention_workspace_bytes(R, H, 1, 128, 64))
    B.prefix_attention(q, kv, out, SCALE, dev(np.array([0, 2], np.int32)), dev(np.array([120], np.int32)), dev(pages[None, :2].copy()),
                       dev(np.array([64, 10, 33], np.int32)), dev(np.full((3, 1), pages[2])), page, 128, 64, ws, lse=lse)
    own = 128 + np.arange(64)
    check(out, lse, q, dense, [np.concatenate([np.arange(120), own]), np.concatenate([np.arange(120), own[:10]]), own[:33]])


def test_two_graphs_of_one_workspace():
    """Captured apart, replayed in turn on one stream."""
    rng = np.random.default_rng(21)
    R, H, k, n = 2, 16, 500, 900
    q, kv = rand(rng, (R, H, 576), "bf16").cuda(), rand(rng, (n, 576), "bf16").cuda()
    ws = workspace(B.sparse_attention_workspace_bytes(R, H, k))
    st = torch.cuda.Stream()
    sets = []
    for _ in range(2):
        idx, out, lse = dev(lists(rng, R, k, n)), torch.empty(R, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(R, H, device="cuda")
        torch.cuda.synchronize()
        g = B.CapturedGraph(lambda s: B.sparse_attention(q, kv, idx, out, SCALE, ws, lse=lse, stream=s), st)
        sets.append((g, idx, out, lse))
    for i in range(3):
        announce("two graphs", i)
        q.copy_(rand(rng, (R, H, 576), "bf16"))
        torch.cuda.synchronize()
        for g, *_ in sets:
            g.launch(st)
        torch.cuda.synchronize()
        for _, idx, out, lse in sets:
            check(out, lse, q, kv, [r for _, r in oa.listed_rows(host(idx), 1, n)])
    for g, *_ in sets:
        g.close()


@pytest.mark.parametrize("begin", [[0, 4, 2], [-5, 2, 100], [4, 4, 0], [1 << 30, -(1 << 30), 3]])
def test_groups_that_are_none(begin):
    """Group bounds that are not ascending rows: whatever the rows get, nothing else is touched, and the next call is whole."""
    rng = np.random.default_rng(23)
    R, H = 4, 16
    c = prefix_case(rng, R, H, [0, 2, 4], [150, 90], [20, 0, 40, 1], 16, "bf16")
    out = torch.full((R + 2, H, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((R + 2, H), 3.0, device="cuda")
    ws = workspace(B.prefix_attention_workspace_bytes(R, H, 2, 150, 40))
    tables = [dev(c[x]) for x in ("plen", "ptab", "olen", "otab")]
    announce("groups", begin)
    for b in (np.asarray(begin, np.int32), c["begin"]):
        B.prefix_attention(c["q"], c["kv"], out[1:-1], SCALE, dev(b), *tables, 16, 150, 40, ws, lse=lse[1:-1])
        for x in (out, lse):
            assert (host(x[0].float()) == 3).all() and (host(x[-1].float()) == 3).all()
    check(out[1:-1], lse[1:-1], c["q"], c["kv"], prefix_rows(c))
