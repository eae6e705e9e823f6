"""The indexer over a paged cache from hidden states to the selected tokens (runner.PagedIndexerRunner):
page maps, quantisation, projections, norms, rotation, FP8 keys into their pages, paged scores and
top-k in a row, with requests that come, grow, end and are taken over, eager and as one graph."""

import numpy as np
import pytest
import torch

import oracle
from dsa_indexer_top_amd import binding as B
from dsa_indexer_top_amd.runner import PagedIndexerRunner
from gpu_util import announce, dev, host
from oracle import blockfp8, pages

pytestmark = pytest.mark.gpu
HID, Q_HID, P, WIDTH = 200, 144, 16, 8


def weights(rng):
    def one(n, k):
        w = torch.from_numpy(np.clip(rng.standard_normal((n, k)) * 60, -448, 448)).float().to(torch.float8_e4m3fn)
        ld = -(-k // 16) * 16
        codes = torch.zeros((n, ld), dtype=torch.uint8)
        codes[:, :k] = w.view(torch.uint8)
        scale = np.exp(0.3 * rng.standard_normal((-(-n // 128), -(-k // 128)))).astype(np.float32) * np.float32(1e-3)
        return codes.cuda()[:, :k], dev(scale)
    return one(64 * 128, Q_HID), one(128, HID), one(64, HID)


def make_runner(rng, n_rows, n_pages, max_new, topk):
    a = rng.uniform(0, 6.28, (WIDTH * P, 32))
    cs = dev(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32))
    vec = lambda m: dev((m + 0.2 * rng.standard_normal(128)).astype(np.float32))
    return PagedIndexerRunner(n_rows, P, WIDTH, n_pages, max_new, topk, *weights(rng), cs, vec(1.0), vec(0.0),
                              (64 * 128) ** -0.5)


def feed(r, rng, new, done):
    """The step's states and lengths into the runner's buffers; the states of its real tokens."""
    n = int(np.sum(new))
    x, xq = rng.standard_normal(r.x.shape), rng.standard_normal(r.xq.shape)
    r.x.copy_(torch.from_numpy(x).to(torch.bfloat16))
    r.xq.copy_(torch.from_numpy(xq).to(torch.bfloat16))
    r.new_len.copy_(torch.from_numpy(np.asarray(new, np.int32)))
    r.done.copy_(torch.from_numpy(np.asarray(done, np.uint8)))
    return n


class Book:
    """What the requests hold, kept by the oracle: their pages, and the FP8 key rows made apart."""

    def __init__(self, r):
        n = r.n_rows
        self.state = dict(lens=np.zeros(n, np.int32), table=np.zeros((n, WIDTH), np.int32),
                          free_list=host(r.free).copy(), count=int(host(r.count)[0]))
        self.keys = [np.zeros((0, 132), np.uint8) for _ in range(n)]     # code row and scale bytes

    def step(self, r, new, done):
        s = self.state
        out = pages.page_step(s["lens"], np.asarray(new, np.int32), np.asarray(done), s["table"], s["free_list"],
                              s["count"], P, len(host(r.slot)))
        assert out["status"] == 0
        self.state = {k: out[k] for k in s}
        # the new tokens' key rows once more, without pages: slots 0, 1, 2, ...
        n = int(np.sum(new))
        c, sc = torch.zeros_like(r.k[:max(n, 1)]), torch.zeros_like(r.k_scale[:max(n, 1)])
        slot = torch.full_like(r.slot, -1)
        slot[:n] = torch.arange(n)
        q8, w_out = torch.zeros_like(r.q8), torch.zeros_like(r.w_out)
        m = r.q.shape[0]
        B.indexer_qk(r.q.view(m, 64, 128), r.kk.view(m, 1, 128), r.w, q8, w_out, c, sc, slot, r.pos, r.cos_sin,
                     w_mul=r.w_mul, k_norm=B.NORM_LAYER, k_weight=r.k_weight, k_bias=r.k_bias)
        rows = np.concatenate([host(c), host(sc)[:, None].view(np.uint8)], 1)
        t = 0
        for i in range(r.n_rows):
            old = self.keys[i][:0] if done[i] else self.keys[i]
            self.keys[i] = np.concatenate([old, rows[t:t + new[i]]])
            t += new[i]
        return out

    def check_cache(self, r):
        """The cache holds every request's rows at its pages, in order."""
        k, sc, table = host(r.k), host(r.k_scale), host(r.table)
        assert np.array_equal(host(r.lens), self.state["lens"]) and int(host(r.status)[0]) == 0
        for i, want in enumerate(self.keys):
            p = np.arange(len(want))
            slot = table[i][p // P] * P + p % P
            got = np.concatenate([k[slot], sc[slot][:, None].view(np.uint8)], 1)
            assert np.array_equal(got, want), i


def check_scores(r, book):
    """Paged scores against the oracle's of the gathered rows, and the top-k of the scores."""
    q, w, scores, idx = host(r.q8), host(r.w_out), host(r.scores), host(r.idx)
    for i, rows in enumerate(book.keys):
        k, sc = np.ascontiguousarray(rows[:, :128]), np.ascontiguousarray(rows[:, 128:]).view(np.float32)[:, 0]
        begin, n = np.zeros(1, np.int64), np.array([len(rows)], np.int32)
        want = oracle.index_scores(q[i:i + 1], w[i:i + 1], k, sc, begin, n)[0]
        T = oracle.error_scale(q[i:i + 1], w[i:i + 1], k, sc, begin, n)[0]
        got = scores[i, :len(rows)]
        assert (np.abs(got - want) <= 1e-4 * T).all(), i
        assert np.array_equal(idx[i], oracle.topk_row(got, r.topk)), i


# chunked prompts, then a token each, with two requests ending and being taken over
STEPS = [([40, 3, 0, 17], [0, 0, 0, 0]), ([1, 20, 33, 1], [0, 0, 0, 0]), ([1, 1, 1, 1], [0, 0, 0, 0]),
         ([1, 25, 1, 1], [0, 1, 0, 0]), ([1, 1, 1, 1], [0, 0, 1, 0]), ([1, 1, 1, 1], [0, 0, 0, 0])]


def test_steps_from_states_to_selected_tokens():
    rng = np.random.default_rng(21)
    r = make_runner(rng, 4, 14, 64, 24)
    book = Book(r)
    for new, done in STEPS:
        announce("step", new, done)
        feed(r, rng, new, done)
        r.step()
        book.step(r, new, done)
        book.check_cache(r)
        if all(n == 1 for n in new):
            r.score()
            check_scores(r, book)


def test_projections_of_a_step():
    """The step's queries, keys and head weights are the products of its quantised states."""
    rng = np.random.default_rng(22)
    r = make_runner(rng, 3, 10, 40, 8)
    n = feed(r, rng, [20, 0, 7], [0, 0, 0])
    r.step()
    for x8, xs, w, got, half in ((r.x8, r.xs, r.wk, r.kk, 2.0 ** -9), (r.x8, r.xs, r.ww, r.w, 2.0 ** -24),
                                 (r.xq8, r.xqs, r.wq, r.q, 2.0 ** -9)):
        want, T = blockfp8.matmul(host(x8)[:n], host(xs)[:n], host(w[0]), host(w[1]))
        # as for the product alone: 2^-23 a step of the sums, and 7 * 2^-13 of the largest product of
        # eight, at most T, from the FP8 matrix core
        tol = T * ((128 + xs.shape[1] + 11) * 2.0 ** -23 + (7 * 2.0 ** -13 if half > 2.0 ** -20 else 0))
        off = np.abs(got[:n].double().cpu().numpy() - want)
        assert (off <= tol + half * (np.abs(want) + tol)).all()


def test_step_and_scores_as_one_graph():
    """One token a step, captured once: every replay leaves what the same eager steps leave in a
    second runner, with eager work and synchronisation in between."""
    rng = np.random.default_rng(23)
    a = make_runner(np.random.default_rng(5), 3, 20, 24, 16)
    b = make_runner(np.random.default_rng(5), 3, 20, 24, 16)
    seeds = rng.integers(0, 1 << 30, 6)
    main = torch.cuda.Stream()
    for r in (a, b):
        feed(r, np.random.default_rng(int(seeds[0])), [9, 1, 12], [0, 0, 0])
        torch.cuda.synchronize()
        r.step()
    torch.cuda.synchronize()

    def both(stream):
        a.step(stream)
        a.score(stream)

    g = B.CapturedGraph(both, main)
    for i in range(1, 6):
        done = [0, 0, int(i == 3)]
        for r in (a, b):
            feed(r, np.random.default_rng(int(seeds[i])), [1, 1, 1], done)
        torch.cuda.synchronize()
        g.launch(main)
        torch.cuda.synchronize()
        b.step()
        b.score()
        for name in ("lens", "table", "free", "count", "slot", "pos", "row", "row_begin", "status", "k", "k_scale", "idx"):
            assert np.array_equal(host(getattr(a, name)), host(getattr(b, name))), (i, name)
        for name in ("q8", "w_out"):                     # the first step wrote 22 tokens, nothing the rest
            assert np.array_equal(host(getattr(a, name))[:22], host(getattr(b, name))[:22]), (i, name)
        for row, n in enumerate(host(a.lens)):
            assert np.array_equal(host(a.scores)[row, :n], host(b.scores)[row, :n]), (i, row)
    g.close()


def check_newest(r, book, new):
    """Every request that got tokens is scored with its newest one's query, the rest select nothing."""
    q, w, scores, idx = host(r.q8), host(r.w_out), host(r.scores), host(r.idx)
    ends = np.cumsum(new)
    for i, rows in enumerate(book.keys):
        if not new[i]:
            assert (idx[i] == -1).all(), i
            continue
        t = ends[i] - 1
        k, sc = np.ascontiguousarray(rows[:, :128]), np.ascontiguousarray(rows[:, 128:]).view(np.float32)[:, 0]
        begin, n = np.zeros(1, np.int64), np.array([len(rows)], np.int32)
        want = oracle.index_scores(q[t:t + 1], w[t:t + 1], k, sc, begin, n)[0]
        T = oracle.error_scale(q[t:t + 1], w[t:t + 1], k, sc, begin, n)[0]
        got = scores[i, :len(rows)]
        assert (np.abs(got - want) <= 1e-4 * T).all(), i
        assert np.array_equal(idx[i], oracle.topk_row(got, r.topk)), i


def test_scores_of_padded_and_ragged_batches():
    """Rows without a token (padding, finished, none yet) and chunks of several: no request is scored
    with another's query."""
    rng = np.random.default_rng(24)
    r = make_runner(rng, 4, 20, 64, 24)
    book = Book(r)
    for new, done in [([9, 0, 12, 30], [0, 0, 0, 0]), ([1, 0, 1, 1], [0, 0, 0, 0]), ([0, 5, 0, 1], [0, 0, 1, 0]),
                      ([0, 0, 0, 0], [0, 0, 0, 0]), ([0, 1, 20, 1], [1, 0, 0, 0]), ([1, 1, 1, 1], [0, 0, 0, 0])]:
        announce("padded step", new, done)
        feed(r, rng, new, done)
        r.step()
        book.step(r, new, done)
        r.score()
        check_newest(r, book, new)


def test_a_refused_step_selects_nothing():
    """Too few pages: nothing is handed out, and no stale query is scored; the next step is whole."""
    rng = np.random.default_rng(25)
    r = make_runner(rng, 3, 4, 90, 8)
    book = Book(r)
    feed(r, rng, [20, 1, 3], [0, 0, 0])               # four pages of 16
    r.step()
    book.step(r, [20, 1, 3], [0, 0, 0])
    r.score()
    check_newest(r, book, [20, 1, 3])
    feed(r, rng, [1, 30, 1], [0, 0, 0])
    r.step()
    r.score()
    assert int(host(r.status)[0]) == B.ST_NO_PAGES and (host(r.idx) == -1).all()
    assert np.array_equal(host(r.lens), book.state["lens"])
    feed(r, rng, [1, 1, 1], [0, 0, 0])
    r.step()
    book.step(r, [1, 1, 1], [0, 0, 0])
    r.score()
    check_newest(r, book, [1, 1, 1])


def test_padded_scores_in_a_graph():
    """Steps with padding rows replayed from one graph: equal to eager steps of a second runner."""
    a = make_runner(np.random.default_rng(6), 4, 20, 24, 16)
    b = make_runner(np.random.default_rng(6), 4, 20, 24, 16)
    main = torch.cuda.Stream()
    torch.cuda.synchronize()

    def both(stream):
        a.step(stream)
        a.score(stream)

    g = B.CapturedGraph(both, main)
    for i, (new, done) in enumerate([([5, 0, 9, 3], [0] * 4), ([1, 0, 0, 1], [0] * 4), ([0, 1, 1, 0], [0] * 4),
                                     ([1, 1, 0, 1], [0, 0, 1, 0]), ([0, 0, 0, 0], [0] * 4)]):
        for r in (a, b):
            feed(r, np.random.default_rng(40 + i), new, done)
        torch.cuda.synchronize()
        g.launch(main)
        torch.cuda.synchronize()
        b.step()
        b.score()
        for name in ("lens", "table", "idx", "q_last", "w_last", "score_len"):
            assert np.array_equal(host(getattr(a, name)), host(getattr(b, name))), (i, name)
        assert ((host(a.idx) >= 0).any(1) == (np.array(new) > 0)).all()
    g.close()


@pytest.mark.parametrize("heads", [0, 1, 3, 64])
def test_newest_queries_of_any_rows(heads):
    """Requests without tokens, and rows that reach behind the tokens there are, have length 0 and
    leave their outputs alone."""
    rng = np.random.default_rng(heads)
    n_tok = 11
    q, w = rng.integers(0, 256, (n_tok, heads, 128), dtype=np.uint8), rng.standard_normal((n_tok, heads)).astype(np.float32)
    begin = np.array([0, 0, 4, 5, 11, 11, 12, -3, -1], np.int32)
    lens = rng.integers(1, 100, 8).astype(np.int32)
    q_out = torch.full((8, heads, 128), 0xEE, dtype=torch.uint8, device="cuda")
    w_out = torch.full((8, heads), -77.0, device="cuda")
    len_out = torch.full((8,), -9, dtype=torch.int32, device="cuda")
    B.newest_queries(dev(q), dev(w), dev(begin), dev(lens), q_out, w_out, len_out)
    got = np.array([0, 1, 1, 1, 0, 0, 0, 0], bool)
    assert np.array_equal(host(len_out), np.where(got, lens, 0))
    last = begin[1:][got] - 1
    assert np.array_equal(host(q_out)[got], q[last]) and np.array_equal(host(w_out)[got], w[last])
    assert (host(q_out)[~got] == 0xEE).all() and (host(w_out)[~got] == -77).all()
