"""echo_page_step against the oracle: tables, stack, lengths and maps equal entry by entry, for
decode batches, ragged chunks, finished and taken-over rows, padding, one-workgroup and spread
forms, steps in place and steps that are refused."""

import numpy as np
import pytest
import torch

from dsa_indexer_top_amd import binding as B
from gpu_util import announce, dev, host
from oracle import pages as O

pytestmark = pytest.mark.gpu


def make_state(rng, n, ctx, page, max_pages, extra, lens=None):
    """Requests with pages handed out in a random order, and `extra` free pages."""
    lens = rng.integers(0, ctx + 1, n).astype(np.int32) if lens is None else np.asarray(lens, np.int32)
    used = -(-lens // page)
    n_pages = int(used.sum()) + extra
    perm = rng.permutation(n_pages).astype(np.int32)
    table = rng.integers(-5, n_pages + 5, (n, max_pages)).astype(np.int32)   # stale entries
    at = 0
    for r in range(n):
        table[r, :used[r]] = perm[at:at + used[r]]
        at += used[r]
    free = np.full(max(n_pages, 1), -7, np.int32)
    free[:extra] = perm[at:]
    return lens, table, free, extra


def run_step(lens, new, done, table, free, count, page, max_new, in_place=False, no_row=False, ws=None,
             stream=None):
    n = len(lens)
    i32 = torch.int32
    d = dict(lens=dev(lens), new=dev(new), table=dev(table), free=dev(free),
             count=dev(np.array([count], np.int32)))
    done_t = None if done is None else dev(done)
    len_out = d["lens"] if in_place else torch.full((n,), -9, dtype=i32, device="cuda")
    count_out = d["count"] if in_place else torch.full((1,), -9, dtype=i32, device="cuda")
    row_begin = torch.full((n + 1,), -9, dtype=i32, device="cuda")
    slot = torch.full((max_new,), -9, dtype=torch.int64, device="cuda")
    row = None if no_row else torch.full((max_new,), -9, dtype=i32, device="cuda")
    pos = torch.full((max_new,), -9, dtype=i32, device="cuda")
    status = torch.zeros(1, dtype=i32, device="cuda")
    if ws is None:
        ws = torch.empty(B.page_workspace_bytes(n, max_new), dtype=torch.uint8, device="cuda")
    B.page_step(d["lens"], d["new"], d["table"], page, d["free"], d["count"], len_out, count_out,
                row_begin, slot, row, pos, status, ws, done=done_t, stream=stream)
    return dict(table=host(d["table"]), free_list=host(d["free"]), lens=host(len_out),
                count=int(host(count_out)[0]), row_begin=host(row_begin), slot=host(slot),
                row=None if no_row else host(row), pos=host(pos), status=int(host(status)[0]))


def check(got, want, what=""):
    for k, v in want.items():
        if got[k] is not None:
            assert np.array_equal(got[k], v), (what, k, got[k], v)


CASES = [
    # rows, page, ctx, chunk, done, slack of the maps, max_new
    dict(n=1, page=16, ctx=40, chunk=1, done=0),
    dict(n=7, page=16, ctx=100, chunk=1, done=2),
    dict(n=64, page=64, ctx=500, chunk=1, done=9),
    dict(n=33, page=16, ctx=70, chunk=90, done=5),
    dict(n=513, page=32, ctx=80, chunk=3, done=100),
    dict(n=3, page=65536, ctx=200000, chunk=40, done=1),
    dict(n=2049, page=16, ctx=40, chunk=2, done=300),       # more requests than one workgroup holds
    dict(n=9, page=128, ctx=300, chunk=2000, done=2),       # more tokens than one workgroup maps
    dict(n=40, page=16, ctx=3000, chunk=30, done=30),       # more pages come back than threads
    dict(n=40, page=16, ctx=9000, chunk=200, done=33),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: "n%(n)d_p%(page)d_c%(chunk)d" % c)
@pytest.mark.parametrize("in_place", [False, True])
def test_step_matches_oracle(c, in_place):
    announce("pages", c, in_place)
    rng = np.random.default_rng(c["n"] + c["page"])
    n, page, chunk = c["n"], c["page"], c["chunk"]
    max_pages = -(-(c["ctx"] + chunk) // page) + 1
    lens, table, free, count = make_state(rng, n, c["ctx"], page, max_pages, n * (chunk // page + 2))
    new = rng.integers(0, chunk + 1, n).astype(np.int32)
    done = np.zeros(n, np.uint8)
    done[rng.permutation(n)[:c["done"]]] = rng.integers(1, 256, c["done"])
    max_new = int(new.sum()) + 5 if chunk < 100 else n * chunk
    want = O.page_step(lens, new, done, table, free, count, page, max_new)
    assert want["status"] == 0
    check(run_step(lens, new, done, table, free, count, page, max_new, in_place), want, c)


@pytest.mark.parametrize("max_new", [64, 9000])       # both forms
def test_lengths_at_page_borders_and_empty_rows(max_new):
    """Lengths of 0, 1, a page less one, a page, a page and one; no, one or a page of new tokens;
    runs of rows with nothing; no free page needed; the last page of the pool."""
    P = 16
    lens = np.array([0, 0, 1, 15, 16, 17, 0, 0, 0, 32, 31, 5], np.int32)
    new = np.array([0, 1, 0, 1, 1, 16, 0, 0, 0, 0, 1, 0], np.int32)
    done = np.array([0, 0, 0, 0, 0, 1, 1, 0, 0, 1, 0, 0], np.uint8)
    rng = np.random.default_rng(1)
    _, table, free, count = make_state(rng, len(lens), 0, P, 4, 1, lens=lens)
    # need: row 1, row 4, row 5 (taken over, 1 page) = 3; have 1 + back (2 + 2)
    want = O.page_step(lens, new, done, table, free, count, P, max_new)
    assert want["status"] == 0 and want["count"] == 2
    check(run_step(lens, new, done, table, free, count, P, max_new, no_row=max_new == 64), want)
    zeros = np.zeros_like(new)
    want = O.page_step(lens, zeros, zeros.astype(np.uint8), table, free, count, P, max_new)
    check(run_step(lens, zeros, None, table, free, count, P, max_new), want)


@pytest.mark.parametrize("max_new", [40, 9000])
@pytest.mark.parametrize("what", ["no pages", "negative len", "negative new", "wide", "wide sum", "tokens",
                                  "stack", "negative count", "huge"])
def test_refused_steps_change_nothing(what, max_new):
    P, n = 16, 6
    rng = np.random.default_rng(3)
    lens, table, free, count = make_state(rng, n, 0, P, 4, 8, lens=[16, 5, 0, 40, 64, 1])
    new = np.array([1, 2, 3, 4, 0, 6], np.int32)
    done = np.zeros(n, np.uint8)
    if what == "no pages":
        count = 1                                     # three are needed
    elif what == "negative len":
        lens[2] = -1
    elif what == "negative new":
        new[5] = -3
    elif what == "wide":
        lens[1] = 65
        done[1] = 1
    elif what == "wide sum":
        new[4] = 1
    elif what == "tokens":
        max_new = 15 if max_new == 40 else max_new
        if max_new != 15:
            pytest.skip("the table is narrower than these maps")
    elif what == "stack":
        count = len(free)
        done[3] = 1
    elif what == "negative count":
        count = -1
    else:
        new[:] = 0x7FFFFFFF
    want = O.page_step(lens, new, done, table, free, count, P, max_new)
    assert want["status"] != 0
    got = run_step(lens, new, done, table, free, count, P, max_new)
    if got["status"] & O.ST_BAD_LEN:                  # a bad length leaves the pages it asks for open
        want["status"] |= got["status"] & O.ST_NO_PAGES
    check(got, want, what)


def test_no_requests_and_no_room():
    e = np.zeros(0, np.int32)
    got = run_step(e, e, None, np.zeros((0, 4), np.int32), np.arange(5, dtype=np.int32), 5, 16, 3)
    assert got["count"] == 5 and list(got["slot"]) == [-1] * 3 and list(got["row_begin"]) == [0]
    lens, z = np.array([3], np.int32), np.zeros(1, np.int32)
    got = run_step(lens, z, None, np.zeros((1, 1), np.int32), np.arange(5, dtype=np.int32), 5, 16, 0)
    assert got["status"] == 0 and list(got["lens"]) == [3]


def test_many_steps_keep_the_pages_apart():
    """Requests come, grow and go for 25 steps in place: equal to the oracle after each, no page is
    held twice and none is lost."""
    rng = np.random.default_rng(11)
    n, P, width = 12, 16, 8
    lens, table, free, count = make_state(rng, n, 60, P, width, 60)
    every = len(free)
    for step in range(25):
        new = rng.integers(0, 30, n).astype(np.int32)
        done = (rng.random(n) < 0.2).astype(np.uint8)
        new = np.where(np.where(done, 0, lens) + new > width * P, 0, new).astype(np.int32)
        cap = 400 if step % 2 else 9000
        want = O.page_step(lens, new, done, table, free, count, P, cap)
        got = run_step(lens, new, done, table, free, count, P, cap, in_place=True)
        check(got, want, step)
        if got["status"]:
            continue
        lens, table, free, count = got["lens"], got["table"], got["free_list"], got["count"]
        held = [table[r, i] for r in range(n) for i in range(-(-int(lens[r]) // P))] + list(free[:count])
        assert sorted(held) == list(range(every))


def test_pages_past_32_bits_of_slots():
    """Rows of the cache beyond 2^31: slots are 64 bits."""
    P = 65536
    lens, new = np.array([P], np.int32), np.array([3], np.int32)
    table = np.array([[7, 0]], np.int32)
    free = np.arange(70000, dtype=np.int32)
    got = run_step(lens, new, None, table, free, 70000, P, 4)
    assert list(got["slot"]) == [69999 * P, 69999 * P + 1, 69999 * P + 2, -1]


@pytest.mark.parametrize("max_new", [64, 9000])
def test_captured_steps_advance_on_every_replay(max_new):
    """An in-place step captured once and replayed: lengths, tables and stack move on by one step a
    replay, with eager work in between."""
    rng = np.random.default_rng(5)
    n, P, width = 6, 16, 10
    lens, table, free, count = make_state(rng, n, 30, P, width, 40)
    new = np.array([1, 0, 17, 2, 1, 5], np.int32)
    i32 = torch.int32
    t = dict(lens=dev(lens), new=dev(new), table=dev(table), free=dev(free),
             count=dev(np.array([count], np.int32)))
    done = torch.zeros(n, dtype=torch.uint8, device="cuda")
    rb = torch.empty(n + 1, dtype=i32, device="cuda")
    slot = torch.empty(max_new, dtype=torch.int64, device="cuda")
    pos = torch.empty(max_new, dtype=i32, device="cuda")
    status = torch.zeros(1, dtype=i32, device="cuda")
    ws = torch.empty(B.page_workspace_bytes(n, max_new), dtype=torch.uint8, device="cuda")
    main = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = B.CapturedGraph(lambda st: B.page_step(t["lens"], t["new"], t["table"], P, t["free"], t["count"], t["lens"],
                                               t["count"], rb, slot, None, pos, status, ws, done=done, stream=st), main)
    for step in range(5):
        flags = np.zeros(n, np.uint8)
        flags[step] = step % 2
        done.copy_(torch.from_numpy(flags))
        want = O.page_step(lens, new, flags, table, free, count, P, max_new)
        assert want["status"] == 0
        torch.cuda.synchronize()
        g.launch(main)
        torch.cuda.synchronize()
        got = dict(table=host(t["table"]), free_list=host(t["free"]), lens=host(t["lens"]),
                   count=int(host(t["count"])[0]), row_begin=host(rb), slot=host(slot), row=None, pos=host(pos),
                   status=int(host(status)[0]))
        check(got, want, step)
        lens, table, free, count = want["lens"], want["table"], want["free_list"], want["count"]
    g.close()


@pytest.mark.parametrize("max_new", [0, 3, 9000])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_batch_of_no_requests_keeps_the_count(max_new, in_place):
    """The batch has drained: the stack's height and row_begin are written all the same, also where
    the maps have no room either, eagerly and in a replayed graph."""
    e = np.zeros(0, np.int32)
    got = run_step(e, e, None, np.zeros((0, 4), np.int32), np.arange(5, dtype=np.int32), 5, 16, max_new, in_place)
    assert got["count"] == 5 and list(got["row_begin"]) == [0] and got["status"] == 0
    assert (got["slot"] == -1).all() and (got["pos"] == -1).all()
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    free, count, begin = torch.arange(5, dtype=torch.int32).cuda(), z(1), torch.full((1,), -9, dtype=torch.int32).cuda()
    out = count if in_place else z(1)
    slot, pos, status = z(max_new).long(), z(max_new), z(1)
    ws = torch.empty(B.page_workspace_bytes(0, max_new), dtype=torch.uint8, device="cuda")
    lens, new, table = z(0), z(0), z(0, 4)
    main = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = B.CapturedGraph(lambda st: B.page_step(lens, new, table, 16, free, count, lens, out, begin, slot, None, pos,
                                               status, ws, stream=st), main)
    for n in (4, 2, 5):
        count.fill_(n)
        begin.fill_(-9)
        torch.cuda.synchronize()
        g.launch(main)
        torch.cuda.synchronize()
        assert int(host(out)[0]) == n and int(host(begin)[0]) == 0
    g.close()


@pytest.mark.parametrize("max_new", [4, 9000])
def test_no_pages_at_all(max_new):
    """A pool without pages and tables without columns (tensors of no elements): steps that need none
    go through, others are refused as any step that needs too many."""
    z, none = np.zeros(3, np.int32), np.zeros(0, np.int32)
    for table, free in ((np.zeros((3, 0), np.int32), none), (np.zeros((3, 2), np.int32), none),
                        (np.zeros((3, 0), np.int32), np.arange(4, dtype=np.int32))):
        n = len(free)
        want = O.page_step(z, z, z, table, free, n, 16, max_new)
        assert want["status"] == 0
        check(run_step(z, z, z.astype(np.uint8), table, free, n, 16, max_new), want)
        new = np.array([0, 1, 0], np.int32)
        want = O.page_step(z, new, z, table, free, n, 16, max_new)
        got = run_step(z, new, None, table, free, n, 16, max_new)
        assert want["status"] and got["status"] & want["status"]
        want["status"] = got["status"]
        check(got, want)


@pytest.mark.parametrize("max_new", [4000, 5007, 5008, 5020])
def test_too_many_tokens_in_two_launches(max_new):
    """More new tokens than maps where the maps take two launches: refused whole, and the step that just
    fits is done."""
    rng = np.random.default_rng(12)
    lens, table, free, count = make_state(rng, 6, 0, 16, 200, 400, lens=[16, 5, 0, 40, 64, 1])
    new = np.array([3000, 2, 0, 2000, 0, 6], np.int32)
    done = np.array([0, 0, 0, 1, 0, 0], np.uint8)
    want = O.page_step(lens, new, done, table, free, count, 16, max_new)
    assert (want["status"] == O.ST_BAD_LEN) == (max_new < 5008) and max_new > 3584
    check(run_step(lens, new, done, table, free, count, 16, max_new), want, max_new)


@pytest.mark.parametrize("n,chunk", [(2048, 3), (9001, 1), (65535, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_many_requests_full(n, chunk, in_place):
    """The plan of more requests than LDS holds, up to the most there may be, many of them finished."""
    rng = np.random.default_rng(n)
    lens, table, free, count = make_state(rng, n, 70, 16, 6, n)
    new = rng.integers(0, chunk + 1, n).astype(np.int32)
    done = (rng.random(n) < 0.2).astype(np.uint8)
    cap = int(new.sum()) + 7
    want = O.page_step(lens, new, done, table, free, count, 16, cap)
    assert want["status"] == 0
    check(run_step(lens, new, done, table, free, count, 16, cap, in_place), want, n)
    want = O.page_step(lens, new, done, table, free, count, 16, cap - 8)
    assert want["status"] == O.ST_BAD_LEN
    check(run_step(lens, new, done, table, free, count, 16, cap - 8, in_place), want, n)
