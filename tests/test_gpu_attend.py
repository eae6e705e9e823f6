"""Whole steps that go on behind the selection: decode steps over the pool with attention over the
selected rows and evictions by accumulated weight (runner.LoopRunner), and the indexer over a paged cache with attention
over what it selected, tokens or blocks, or over everything behind shared prefixes (runner.PagedIndexerRunner)."""

import numpy as np
import pytest
import torch

import oracle
from attention_util import SCALE, check, f64, rand, score_error
from dsa_indexer_top_amd import binding as B, inputs as gen
from dsa_indexer_top_amd.runner import LoopRunner, PagedIndexerRunner
from gpu_util import announce, assert_pool_equal, dev, host
from oracle import attention as oa, multistep as ms
from test_gpu_inputs import P, WIDTH, feed, weights

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- the pool
def bits(rng, shape):
    return rand(rng, shape, "bf16").view(torch.int16).numpy().view(np.uint16)


def loop_inputs(rows, length, steps, n_gpu, seed):
    """Steps whose latent rows are numbers (the generator's are any bits)."""
    m, host_kv = gen.make_multistep_inputs(rows, length, steps, n_gpu, seed=seed, drift=0.3)
    rng = np.random.default_rng(seed)
    host_kv = bits(rng, host_kv.shape)
    held = m.pool.to_host != oracle.INF
    m.pool.gpu_kv[held] = host_kv[m.pool.to_host[held]]
    for s in m.steps:
        s["new_kv"] = bits(rng, s["new_kv"].shape)
    return m, host_kv


@pytest.mark.parametrize("mode", ["eager", "graph"])
@pytest.mark.parametrize("rows,length,k,n_gpu,heads,decay", [(3, 300, 32, 120, 16, 0.5), (2, 700, 256, 600, 5, 1.0)])
def test_decode_steps_evict_by_weight(rows, length, k, n_gpu, heads, decay, mode):
    """Each step against the oracle's from the pool that the step before left: its selection, slots, evictions and
    rows; then attention over the slots, and mass and priorities of the weights bit for bit."""
    announce("attend, evict", rows, length, k, n_gpu, heads, mode)
    m, host_kv = loop_inputs(rows, length, 6, n_gpu, 61 + length)
    rng = np.random.default_rng(heads)
    cache = ms.KeyCache(m.k.copy(), None, m.key_begin.copy(), m.key_len.copy(), m.req_to_host.copy(), m.capacity)
    names = ("free", "priority", "to_host", "host_to_gpu", "indices_buf", "gpu_kv")
    state = oracle.PoolState(*(getattr(m.pool, n).copy() for n in names))
    mass = np.zeros(n_gpu, np.float32)
    r = LoopRunner(m, host_kv, k, device_step=mode == "graph", heads=dict(n_heads=heads, scale=SCALE, decay=decay))
    try:
        if mode == "graph":
            r.capture()
        evicted = 0
        for t, s in enumerate(m.steps):
            announce("step", t)
            r.heads.q.copy_(rand(rng, (rows, heads, 576), "bf16"))
            torch.cuda.synchronize()
            (r.replay_step if mode == "graph" else r.run_step)(s)
            got = r.results()
            assert got["status"] == 0
            before = state.host_to_gpu.copy()
            cache, state, host_kv, recs = ms.decode_loop(cache, state, host_kv, [s], k)
            evicted += int(((before != oracle.INF) & (state.host_to_gpu == oracle.INF)).sum())
            assert np.array_equal(got["topk_idx"], recs[0].idx) and np.array_equal(got["topk_slot"], recs[0].result.topk_slot)
            kv = r.kv.clone()
            listed = oa.listed_rows(got["topk_slot"], 1, n_gpu)
            places, at = [p for p, _ in listed], [x for _, x in listed]
            check(r.heads.out, r.heads.lse, r.heads.q, kv, at)
            w = host(r.weights)
            want = oa.token_weights(f64(r.heads.q), f64(kv), places, at, f64(r.heads.lse), SCALE, k)
            _, lse, _, terms = oa.attention(f64(r.heads.q), f64(kv), at, SCALE)
            assert (np.abs(w - want) <= want * score_error(terms, lse).max() + 1e-30).all()
            fresh = np.concatenate([got["miss_slot"], got["new_slot"]])
            mass, priority = oa.weigh(mass, state.free, got["topk_slot"], w, np.float32(decay), fresh)
            state.priority[:] = priority                   # what the next step evicts by
            assert np.array_equal(host(r.mass).view(np.int32), mass.view(np.int32)), "step %d mass" % t
            assert_pool_equal(oracle.PoolState(*(got["pool"][n] for n in names)), state, "step %d" % t)
        assert evicted > 5
    finally:
        r.close()


# ---------------------------------------------------------------- the paged cache
SHARED = 3                                                 # pages at the cache's end that no request is given


def make_runner(seed, n_rows, n_pages, max_new, topk, heads):
    rng = np.random.default_rng(seed)
    a = rng.uniform(0, 6.28, (WIDTH * P, 32))
    vec = lambda m: dev((m + 0.2 * rng.standard_normal(128)).astype(np.float32))
    r = PagedIndexerRunner(n_rows, P, WIDTH, n_pages, max_new, topk, *weights(rng),
                           dev(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)), vec(1.0), vec(0.0),
                           (64 * 128) ** -0.5, heads=heads)
    r.count.fill_(n_pages - SHARED)
    return r


def put_rows(r, rng, n):
    """The new tokens' latent rows at their slots, as a projection would leave them."""
    r.heads.q.copy_(rand(rng, r.heads.q.shape, "bf16").to(r.heads.q.dtype))
    if n:
        r.kv[r.slot[:n]] = rand(rng, (n, 576), "bf16").cuda().to(r.kv.dtype)


def expected_rows(r, whole):
    lens, table, n_kv = host(r.score_len), host(r.table), r.kv.shape[0]
    if whole:
        return oa.prefix_rows(r.n_rows, n_kv, P, host(r.group_begin), host(r.prefix_len), host(r.prefix_table), lens, table)
    return [x for _, x in oa.listed_rows(host(r.idx), max(r.block, 1), n_kv, lens, table, P)]


STEPS = [([40, 3, 0, 17], [0, 0, 0, 0]), ([1, 20, 33, 1], [0, 0, 0, 0]), ([1, 0, 1, 1], [0, 0, 0, 1]),
         ([0, 0, 0, 0], [0, 1, 0, 0]), ([1, 1, 1, 1], [0, 0, 0, 0])]


@pytest.mark.parametrize("dtype,block,topk", [(torch.bfloat16, 0, 24), (torch.float16, 0, 70), (torch.bfloat16, 16, 3)])
def test_paged_steps_with_attention(dtype, block, topk):
    rng = np.random.default_rng(31)
    r = make_runner(5, 4, 14 + SHARED, 64, topk, dict(n_heads=20, scale=SCALE, dtype=dtype, block=block, kept=(1, 1),
                                                      prefixes=(2, SHARED)))
    pages = r.kv.shape[0] // P
    r.kv[(pages - SHARED) * P:] = rand(rng, (SHARED * P, 576), "bf16").cuda().to(dtype)
    r.prefix_table.copy_(torch.tensor([[pages - 2, pages - 1, pages - 3], [pages - 3, -1, 0]], dtype=torch.int32))
    for i, (new, done) in enumerate(STEPS):
        announce("paged step", dtype, block, new, done)
        n = feed(r, rng, new, done)
        r.step()
        put_rows(r, rng, n)
        r.score()
        assert int(host(r.status)[0]) == 0 and host(r.table).max() < pages - SHARED
        idx, lens = host(r.idx), host(r.score_len)
        for row in range(4):
            s = host(r.scores)[row:row + 1]
            want = oa.block_topk(s, lens[row:row + 1], block, topk, 1, 1)[0] if block else oracle.topk_row(s[0, :lens[row]], topk)
            assert np.array_equal(idx[row], want), row
        check(r.heads.out, r.heads.lse, r.heads.q, r.kv, expected_rows(r, False))
        assert np.isneginf(host(r.heads.lse)[np.asarray(new) == 0]).all()
        for begin, length in (([0, 0, 0], [0, 0]), ([0, 3, 4], [37, 16])):
            r.group_begin.copy_(torch.tensor(begin, dtype=torch.int32))
            r.prefix_len.copy_(torch.tensor(length, dtype=torch.int32))
            r.attend_all()
            check(r.heads.out, r.heads.lse, r.heads.q, r.kv, expected_rows(r, True))


def test_paged_steps_as_one_graph():
    """Steps captured once: every replay leaves what the same eager steps leave in a second runner."""
    heads = dict(n_heads=16, scale=SCALE, block=16, kept=(0, 1))
    a, b = (make_runner(6, 3, 20 + SHARED, 24, 4, heads) for _ in range(2))
    main = torch.cuda.Stream()
    latent = [np.random.default_rng(9) for _ in range(2)]
    for r, g in zip((a, b), latent):
        n = feed(r, np.random.default_rng(1), [9, 1, 12], [0, 0, 0])
        torch.cuda.synchronize()
        r.step()
        put_rows(r, g, n)
    torch.cuda.synchronize()
    step = B.CapturedGraph(lambda st: a.step(st), main)
    score = B.CapturedGraph(lambda st: a.score(st), main)
    for i in range(4):
        announce("replay", i)
        for r in (a, b):
            feed(r, np.random.default_rng(10 + i), [1, 1, 1], [0, 0, int(i == 2)])
        torch.cuda.synchronize()
        step.launch(main)
        b.step()
        torch.cuda.synchronize()
        put_rows(a, latent[0], 3)
        put_rows(b, latent[1], 3)
        torch.cuda.synchronize()
        score.launch(main)
        b.score()
        for x in ("idx", "lens"):
            assert np.array_equal(host(getattr(a, x)), host(getattr(b, x))), x
        for x in ("out", "lse"):
            p, q = host(getattr(a.heads, x).float()), host(getattr(b.heads, x).float())
            assert np.array_equal(p, q), x
        check(a.heads.out, a.heads.lse, a.heads.q, a.kv, expected_rows(a, False))
    step.close()
    score.close()
