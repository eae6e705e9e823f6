"""Blocks that scores select, and the pool's eviction order by accumulated weight, against the oracle: bit for bit."""

import numpy as np
import pytest
import torch

import oracle
from dsa_indexer_top_amd import binding as B
from gpu_util import DevPool, announce, dev, host
from oracle import attention as oa

pytestmark = pytest.mark.gpu


def block_topk(scores, length, block, k, first=0, last=0, max_len=None, ld_pad=0):
    R, n = scores.shape
    buf = torch.full((R, n + ld_pad), 1e30, device="cuda")
    buf[:, :n] = dev(scores)
    idx = torch.empty(R, k, dtype=torch.int32, device="cuda")
    max_len = n if max_len is None else max_len
    ws = torch.empty(max(B.block_topk_workspace_bytes(R, max_len, block), 4), dtype=torch.uint8, device="cuda")
    B.block_topk(buf[:, :n], dev(np.asarray(length, np.int32)), max_len, block, k, idx, ws, n_first=first, n_last=last)
    return host(idx)


@pytest.mark.parametrize("block", [16, 32, 64, 128, 256, 512])
@pytest.mark.parametrize("first,last,pad", [(0, 0, 0), (1, 2, 3)])
def test_blocks(block, first, last, pad):
    rng = np.random.default_rng(block + first)
    announce("blocks", block, first, last, pad)
    R, n = 9, 1801
    scores = rng.standard_normal((R, n)).astype(np.float32)
    scores[3] = np.round(scores[3])                        # ties
    scores[4] = -np.abs(scores[4])
    scores[5, ::3] = -np.inf
    scores[6] = 0.0
    scores[6, ::2] = -0.0
    length = [n, 0, 1, n - 1, block, block + 1, n, -3, n // 2]
    for k in (1, 4, 40):
        got = block_topk(scores, length, block, k, first, last, ld_pad=pad)
        assert np.array_equal(got, oa.block_topk(scores, length, block, k, first, last)), k


def test_more_kept_blocks_than_k_and_clamped_lengths():
    rng = np.random.default_rng(1)
    scores = rng.standard_normal((3, 700)).astype(np.float32)
    announce("kept blocks")
    got = block_topk(scores, [700, 5000, 200], 16, 3, 5, 100)
    assert np.array_equal(got, oa.block_topk(scores, [700, 700, 200], 16, 3, 5, 100))
    got = block_topk(scores, [700, 5000, 200], 64, 6, 0, 1, max_len=500)
    assert np.array_equal(got, oa.block_topk(scores[:, :500], [500, 500, 200], 64, 6, 0, 1))


@pytest.mark.parametrize("R,n,block,k", [(1, 0, 16, 4), (2000, 300, 16, 8), (1, 131072, 64, 32), (3, 131071, 16, 4096)])
def test_blocks_full(R, n, block, k):
    rng = np.random.default_rng(n)
    announce("blocks full", R, n, block, k)
    scores = rng.standard_normal((R, n)).astype(np.float32)
    length = rng.integers(n // 2, n + 1, R)
    assert np.array_equal(block_topk(scores, length, block, k, 1, 1), oa.block_topk(scores, length, block, k, 1, 1))


# ---------------------------------------------------------------- eviction order
def weigh(mass, free, slot, w, decay, fresh=None):
    m, p = dev(mass), torch.full((len(mass),), 77, dtype=torch.int32, device="cuda")
    ws = torch.full((B.pool_weigh_workspace_bytes(len(mass)),), 0xAB, dtype=torch.uint8, device="cuda")
    B.pool_weigh(dev(free), p, m, dev(slot), dev(w), ws, decay=decay, fresh=None if fresh is None else dev(fresh))
    return host(m), host(p)


@pytest.mark.parametrize("n,entries,decay", [(1, 1, 1.0), (100, 0, 0.5), (257, 1000, 0.9), (5000, 300, 0.0), (3000, 20000, 1.0)])
def test_weigh(n, entries, decay):
    rng = np.random.default_rng(n + entries)
    announce("weigh", n, entries, decay)
    mass = np.exp(rng.standard_normal(n)).astype(np.float32)
    free = (rng.random(n) < 0.2).astype(np.uint8)
    slot = rng.integers(-2, n + 3, entries).astype(np.int32)           # repeated ones and some outside
    w = np.exp(3 * rng.standard_normal(entries)).astype(np.float32)
    fresh = rng.integers(-1, n + 1, max(1, n // 7)).astype(np.int32)
    for f in (None, fresh):
        got_m, got_p = weigh(mass, free, slot, w, decay, f)
        want_m, want_p = oa.weigh(mass, free, slot, w, np.float32(decay), () if f is None else f)
        assert np.array_equal(got_m.view(np.int32), want_m.view(np.int32))
        assert np.array_equal(got_p, want_p)


def test_weigh_odd_values():
    """NaN, negative, tiny and huge weights; masses that are no masses."""
    announce("weigh odd")
    mass = np.array([1, np.nan, -3, np.inf, 0, -0.0, 1e-38, 5], np.float32)
    slot = np.array([0, 1, 2, 3, 4, 5, 6, 7, 7], np.int32)
    w = np.array([np.nan, 2, -1, 3, 1e-12, -0.0, 2.0 ** -33, 1e9, np.inf], np.float32)
    got_m, got_p = weigh(mass, np.zeros(8, np.uint8), slot, w, 0.5)
    want_m, want_p = oa.weigh(mass, np.zeros(8), slot, w, np.float32(0.5))
    assert np.array_equal(got_m, want_m) and np.array_equal(got_p, want_p)
    assert (got_p >= 0).all() and got_m[7] == 2050.5 and got_m[3] == np.inf


def test_weigh_full():
    rng = np.random.default_rng(4)
    n, entries = 200000, 131072
    announce("weigh full")
    mass, free = np.exp(rng.standard_normal(n)).astype(np.float32), (rng.random(n) < 0.1).astype(np.uint8)
    slot, w = rng.integers(-1, n, entries).astype(np.int32), rng.random(entries).astype(np.float32)
    for _ in range(2):                                     # the same bits whatever the order of the adds
        got_m, got_p = weigh(mass, free, slot, w, 0.9)
        want_m, want_p = oa.weigh(mass, free, slot, w, np.float32(0.9))
        assert np.array_equal(got_m, want_m) and np.array_equal(got_p, want_p)


def test_pool_step_evicts_the_smallest_mass():
    """After echo_pool_weigh the pool step's evictions follow the accumulated weight, ties to the lower slot."""
    rng = np.random.default_rng(8)
    n_gpu, n_host, k = 60, 200, 20
    held = rng.permutation(n_host)[:55]
    free = np.ones(n_gpu, np.uint8)
    to_host = np.full(n_gpu, oracle.INF, np.int32)
    host_to_gpu = np.full(n_host, oracle.INF, np.int32)
    slots = rng.permutation(n_gpu)[:55]
    free[slots], to_host[slots] = 0, held
    host_to_gpu[held] = slots
    gpu_kv = rng.integers(0, 1 << 16, (n_gpu, 576)).astype(np.uint16)
    host_kv = rng.integers(0, 1 << 16, (n_host, 576)).astype(np.uint16)
    priority = np.where(free, -1, 3).astype(np.int32)
    mass = np.round(rng.random(n_gpu) * 8).astype(np.float32)          # ties among them
    p = DevPool(free, priority, to_host, host_to_gpu, np.full(n_gpu, -1, np.int32), gpu_kv, host_kv)
    try:
        announce("weigh, then a pool step")
        entries = slots[:30].astype(np.int32)
        w = np.round(rng.random(30) * 4).astype(np.float32)
        m = dev(mass)
        ws = torch.empty(B.pool_weigh_workspace_bytes(n_gpu), dtype=torch.uint8, device="cuda")
        B.pool_weigh(p.free, p.priority, m, dev(entries), dev(w), ws, decay=0.5)
        want_m, want_p = oa.weigh(mass, free, entries, w, np.float32(0.5))
        assert np.array_equal(host(m), want_m) and np.array_equal(host(p.priority), want_p)
        idx = np.sort(rng.permutation(n_host)[:k]).astype(np.int32)[None]
        st0 = oracle.PoolState(free.copy(), want_p.copy(), to_host.copy(), host_to_gpu.copy(), np.full(n_gpu, -1, np.int32), gpu_kv.copy())
        step = (1 << 31) - 2
        want_state, want = oracle.pool_step(st0, host_kv, idx, np.zeros(1, np.int64), np.arange(n_host, dtype=np.int32), step)
        i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
        topk_slot, mh, ms, nm = i32(k), i32(k), i32(k), i32(1)
        pw = torch.empty(B.pool_workspace_bytes(1, k, n_gpu), dtype=torch.uint8, device="cuda")
        B.pool_lookup_alloc(p.pool, dev(idx), dev(np.zeros(1, np.int64)), dev(np.arange(n_host, dtype=np.int32)), step, topk_slot,
                            mh, ms, nm, pw)
        B.recall(p.pool, mh, ms, nm, k)
        assert want.n_miss > 5
        assert np.array_equal(host(topk_slot), want.topk_slot.ravel()) and int(host(nm)[0]) == want.n_miss
        got = p.state()
        for name in ("free", "priority", "to_host", "host_to_gpu", "gpu_kv"):
            assert np.array_equal(getattr(got, name), getattr(want_state, name)), name
    finally:
        p.close()


@pytest.mark.parametrize("n,block", [(1023, 16), (1024, 16), (1025, 64), (2048, 256), (4097, 512), (9000, 1024), (9000, 4096),
                                     (2049, 16), (8193, 16)])
def test_blocks_around_a_waves_span(n, block):
    """Lengths around what a wave takes, blocks around it and above, and 129, 512 and 513 blocks of a row."""
    rng = np.random.default_rng(n + block)
    scores = np.round(8 * rng.standard_normal((5, n))).astype(np.float32)           # many ties
    length = [n, n - 1, max(0, n - block), n // 2 + 1, min(n, 1024)]
    announce("blocks, spans", n, block)
    for k, first, last in ((1, 0, 0), (3, 0, 1), (7, 2, 0), (100, 0, 0)):
        got = block_topk(scores, length, block, k, first, last, ld_pad=1)
        assert np.array_equal(got, oa.block_topk(scores, length, block, k, first, last)), k


@pytest.mark.parametrize("n,entries", [(700, 30000), (3000, 5), (40000, 20000), (200000, 9000)])
def test_weigh_either_way(n, entries):
    """Few entries and many, few slots and many: searched for in one launch, or added up in memory."""
    rng = np.random.default_rng(n)
    announce("weigh", n, entries)
    mass, free = rng.random(n).astype(np.float32), (rng.random(n) < 0.3).astype(np.uint8)
    slot = rng.integers(-1, n + 1, entries + 3).astype(np.int32)
    w = rng.random(entries + 3).astype(np.float32)
    fresh = rng.integers(-1, n + 1, 1300).astype(np.int32)
    for a in (0, 3):                                       # arrays that begin and end anywhere
        s, x = dev(slot)[a:a + entries], dev(w)[a:a + entries]
        m, p = dev(mass), torch.empty(n, dtype=torch.int32, device="cuda")
        ws = torch.full((B.pool_weigh_workspace_bytes(n),), 0x5A, dtype=torch.uint8, device="cuda")
        B.pool_weigh(dev(free), p, m, s, x, ws, decay=0.75, fresh=dev(fresh))
        want_m, want_p = oa.weigh(mass, free, slot[a:a + entries], w[a:a + entries], np.float32(0.75), fresh)
        assert np.array_equal(host(m).view(np.int32), want_m.view(np.int32)) and np.array_equal(host(p), want_p)


@pytest.mark.parametrize("R,n,block,k", [(3, 70000, 256, 20), (2, 66000, 4096, 5), (520, 66000, 1024, 9), (2, 65536, 128, 600)])
def test_long_rows_full(R, n, block, k):
    """Few long rows in two launches, many in one, and more asked for than there are."""
    rng = np.random.default_rng(n + R)
    scores = np.round(50 * rng.standard_normal((R, n)).astype(np.float32))
    length = rng.integers(0, n + 1, R)
    length[0] = n
    announce("long rows", R, n, block, k)
    assert np.array_equal(block_topk(scores, length, block, k, 1, 2), oa.block_topk(scores, length, block, k, 1, 2))
