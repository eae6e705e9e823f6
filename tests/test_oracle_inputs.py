"""Pins of the oracles in front of the scores: page steps worked by hand and their invariants, the
E4M3FN distances and block scales, a product by hand, norms and rotations by hand and by their
invariants."""

import numpy as np
import pytest
import torch

from oracle import blockfp8, heads, pages
from oracle.fp8 import E4M3FN_TABLE


def test_page_step_by_hand():
    """Pages of 16. Request 0 has 16 tokens on page 5 and gets 2: one new page. Request 1 (17 tokens
    on pages 2, 7) is done and the row gets 1 token. Request 2 has 3 tokens on page 0 and gets 1.
    Stack 4, 9: pages 2 and 7 are pushed, then popped again, 7 to request 0 and 2 to request 1."""
    table = np.array([[5, -1, -1], [2, 7, -1], [0, -1, -1]], np.int32)
    free = np.array([4, 9, -1, -1], np.int32)
    out = pages.page_step(np.array([16, 17, 3], np.int32), np.array([2, 1, 1], np.int32), np.array([0, 1, 0]),
                          table, free, 2, 16, 6)
    assert out["status"] == 0 and out["count"] == 2
    assert out["lens"].tolist() == [18, 1, 4] and out["row_begin"].tolist() == [0, 2, 3, 4]
    assert out["table"].tolist() == [[5, 7, -1], [2, 7, -1], [0, -1, -1]]
    assert out["free_list"].tolist() == [4, 9, 2, 7]
    assert out["slot"].tolist() == [7 * 16, 7 * 16 + 1, 2 * 16, 3, -1, -1]
    assert out["row"].tolist() == [0, 0, 1, 2, -1, -1] and out["pos"].tolist() == [16, 17, 0, 3, -1, -1]


def test_refused_page_step_changes_nothing():
    table, free = np.array([[3]], np.int32), np.array([1, 2], np.int32)
    for lens, new, done, count, cap, bits in (([16], [1], [0], 2, 4, pages.ST_BAD_LEN), ([-1], [1], [0], 2, 4, pages.ST_BAD_LEN),
                                              ([0], [5], [0], 2, 4, pages.ST_BAD_LEN), ([0], [1], [0], 0, 4, pages.ST_NO_PAGES),
                                              ([16], [0], [1], 2, 4, pages.ST_NO_PAGES)):
        out = pages.page_step(np.array(lens, np.int32), np.array(new, np.int32), np.array(done), table, free, count, 16, cap)
        assert out["status"] == bits, (lens, new)
        assert out["lens"].tolist() == lens and out["count"] == count and (out["slot"] == -1).all()
        assert np.array_equal(out["table"], table) and np.array_equal(out["free_list"], free)


def test_block_scales_and_distances():
    x = np.zeros((2, 130))
    x[0, :128] = np.linspace(-224, 100, 128)
    x[0, 128] = -896.0
    s = blockfp8.block_scales(x)
    assert s[0].tolist() == [0.5, 2.0] and (s[1] == 2.0 ** -126).all()
    assert blockfp8.spread(s, 130)[0, 127:].tolist() == [0.5, 2.0, 2.0]
    v = np.concatenate([np.random.default_rng(0).uniform(-448, 448, 4000), 2.0 ** np.arange(-12, 9) * 1.03])
    near = torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
    assert np.allclose(blockfp8.nearest_distance(v.astype(np.float32)), np.abs(v.astype(np.float32) - near), rtol=0, atol=1e-12)


def test_product_by_hand():
    one, two = int(np.flatnonzero(E4M3FN_TABLE == 1.0)[0]), int(np.flatnonzero(E4M3FN_TABLE == 2.0)[0])
    a, b = np.full((1, 130), one, np.uint8), np.full((129, 130), two, np.uint8)
    c, t = blockfp8.matmul(a, np.array([[3.0, 10.0]]), b, np.array([[1.0, 0.5], [2.0, 1.0]]))
    assert (c[0, :128] == 128 * 2 * 3 + 2 * 2 * 5).all() and c[0, 128] == 128 * 2 * 6 + 2 * 2 * 10
    assert np.array_equal(c, t)
    g = blockfp8.group_maxima(a, np.array([[3.0, 10.0]]), b, np.array([[1.0, 0.5], [2.0, 1.0]]))
    assert g[0, 0] == 16 * 2 * 3 + 2 * 5 and g[0, 128] == 16 * 2 * 6 + 2 * 10


def test_norms_by_hand():
    x = np.array([[3.0, -4.0]])
    v, _ = heads.norm(x, "rms", np.array([1.0, 2.0]), None, 0.0)
    assert np.allclose(v, [[3 / 12.5 ** 0.5, -8 / 12.5 ** 0.5]])
    v, _ = heads.norm(x, "layer", np.array([1.0, 2.0]), np.array([0.5, 0.0]), 0.0)
    assert np.allclose(v, [[1.5, -2.0]])
    assert np.array_equal(heads.norm(x, "none")[0], x)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_by_hand_and_invariants(inter):
    rng = np.random.default_rng(3)
    a, b = rng.uniform(-3, 3, (2, 4))
    cs = lambda t: np.concatenate([np.cos(t), np.sin(t)])[None]
    x = rng.standard_normal((1, 2, 12))
    pos = np.zeros(1, int)
    turn = lambda y, t: heads.rotate(y, np.abs(y), pos, cs(t), 3, inter)[0]
    y = turn(x, a)
    i, j = (3 + 2 * 1, 3 + 2 * 1 + 1) if inter else (3 + 1, 3 + 4 + 1)
    assert np.allclose(y[..., i], x[..., i] * np.cos(a[1]) - x[..., j] * np.sin(a[1]))
    assert np.allclose(y[..., j], x[..., j] * np.cos(a[1]) + x[..., i] * np.sin(a[1]))
    assert np.array_equal(y[..., :3], x[..., :3]) and np.array_equal(y[..., 11:], x[..., 11:])
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    assert np.allclose(turn(y, b), turn(x, a + b))
