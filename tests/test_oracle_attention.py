"""Pins of the oracle behind the selection: softmaxes worked by hand, invariances, blocks, weights and masses."""

import numpy as np

from oracle import attention as oa


def latent(*first):
    """Rows that are 0 but for their first values."""
    x = np.zeros((len(first), 576))
    for i, v in enumerate(first):
        x[i, :len(v)] = v
    return x


def test_softmaxes_by_hand():
    q = latent([1.0])[None]                                # one row, one head: the score is scale * kv[t][0]
    kv = latent([0.0, 8.0], [np.log(3.0), 4.0], [5.0, -2.0])
    out, lse, size, terms = oa.attention(q, kv, [np.array([2])], 2.0)
    assert np.allclose(out[0, 0, :3], [5, -2, 0]) and np.isclose(lse[0, 0], 10) and np.isclose(size[0, 0, 1], 2)
    out, lse, _, terms = oa.attention(q, kv, [np.array([0, 1])], 1.0)      # weights 1/4 and 3/4
    assert np.allclose(out[0, 0, :2], [0.75 * np.log(3), 5]) and np.isclose(lse[0, 0], np.log(4)) and np.isclose(terms[0, 0], np.log(3))
    out, lse, _, _ = oa.attention(q, kv, [np.array([1, 1, 1, 0])], 1.0)    # one listed three times: 9/10
    assert np.isclose(out[0, 0, 1], 0.9 * 4 + 0.1 * 8) and np.isclose(lse[0, 0], np.log(10))
    out, lse, _, _ = oa.attention(q, kv, [np.array([], int)], 1.0)
    assert not out.any() and np.isneginf(lse[0, 0])
    assert out.shape == (1, 1, 512)                        # the last 64 values are no part of a token's value


def test_order_and_halves():
    rng = np.random.default_rng(0)
    q, kv = rng.standard_normal((2, 3, 576)), rng.standard_normal((40, 576))
    rows = [rng.permutation(40)[:25] for _ in range(2)]
    out, lse, _, _ = oa.attention(q, kv, rows, 0.07)
    again, lse2, _, _ = oa.attention(q, kv, [r[::-1] for r in rows], 0.07)
    assert np.allclose(out, again) and np.allclose(lse, lse2)
    a, la, _, _ = oa.attention(q, kv, [r[:11] for r in rows], 0.07)
    b, lb, _, _ = oa.attention(q, kv, [r[11:] for r in rows], 0.07)
    both = np.logaddexp(la, lb)
    assert np.allclose(both, lse)
    assert np.allclose(a * np.exp(la - both)[..., None] + b * np.exp(lb - both)[..., None], out)
    w = oa.token_weights(q, kv, [np.arange(25)] * 2, rows, lse, 0.07, 30)
    assert np.allclose(w.sum(1), 3) and not w[:, 25:].any()


def test_listed_rows_by_hand():
    table = np.array([[4, -1, 0], [2, 3, 1]])
    idx = np.array([[0, -1, 2], [1, 1, 7]])
    # pages of 2, blocks of 2: entry e is tokens 2 e and 2 e + 1, on page e of the table
    got = oa.listed_rows(idx, 2, 10, [5, 100], table, 2)
    assert got[0][0].tolist() == [0, 1, 4] and got[0][1].tolist() == [8, 9, 0]     # token 5 is behind the length
    assert got[1][0].tolist() == [0, 1, 2, 3] and got[1][1].tolist() == [6, 7, 6, 7]      # entry 7 is behind the table
    got = oa.listed_rows(idx, 2, 9, [5, 100], table, 2, req=[1, 9])
    assert got[0][1].tolist() == [4, 5, 2] and got[1][1].tolist() == []
    assert oa.listed_rows([[3, 0, 3, 11]], 1, 11)[0][1].tolist() == [3, 0, 3]
    assert oa.prefix_rows(3, 10, 2, [0, 2], [3], table[:1], [1, 0, 3], np.array([[3], [3], [1]]))[0].tolist() == [8, 9, 6]
    rows = oa.prefix_rows(3, 10, 2, [0, 2], [3], np.array([[4, 0]]), [1, 0, 3], np.array([[3], [3], [1]]))
    assert [r.tolist() for r in rows] == [[8, 9, 0, 6], [8, 9, 0], [2, 3]]


def test_blocks_by_hand():
    s = np.array([[1, 5, 2, 2, 9, 0, 3, 7, 5, 1]], np.float32)             # blocks of 2: 5 2 9 7 5
    pick = lambda n, k, first=0, last=0: oa.block_topk(s, [n], 2, k, first, last)[0].tolist()
    assert pick(10, 2) == [2, 3] and pick(10, 3) == [0, 2, 3] and pick(10, 4) == [0, 2, 3, 4]
    assert pick(7, 2) == [0, 2] and pick(7, 5) == [0, 1, 2, 3, -1]         # the last block has one token
    assert pick(10, 3, 0, 1) == [2, 3, 4] and pick(10, 2, 1, 2) == [0, 3] and pick(0, 2) == [-1, -1]


def test_masses_by_hand():
    mass, free = np.array([1, 2, 4, 8], np.float32), np.array([0, 0, 1, 0])
    m, p = oa.weigh(mass, free, [[1, 1], [2, -1]], [[0.5, 0.25], [3, 3]], np.float32(0.5), fresh=[3, 9])
    assert m.tolist() == [0.5, 1.75, 0, 0] and p.tolist() == [0x3F000000, 0x3FE00000, -1, 0]
    m, _ = oa.weigh(mass, np.zeros(4), [0, 1], [2000.0, -1.0], np.float32(1))
    assert m.tolist() == [1025, 2, 4, 8]                   # one entry counts up to 1024, none below 0
