"""Norms and rotation of query and key heads (echo_qk_norm_rope) and the indexer's FP8 form of them
(echo_indexer_qk) against the oracle in float64.

Tolerance (u = 2^-24), with T the magnitudes behind a value (oracle.heads): a mean over at most 256
values sums 8 in the lane and 5 times over lanes (13 roundings with the division), the same for the
mean of squares and half of it for its root, and scaling, bias, and the rotation's three steps add
less than 10: 40 u T, plus half a step of the output's type (for fp16 below its normal numbers
2^-25).  FP8 scales: the value's tolerance over 448 and 2 u of the scale; codes: off the nearest
E4M3FN number's distance by the value's tolerance over the scale and 4 u of the value."""

import numpy as np
import pytest
import torch

from dsa_indexer_top_amd import binding as B
from gpu_util import announce, dev, host
from oracle import heads as O
from oracle.blockfp8 import nearest_distance, SCALE_MIN
from oracle.fp8 import E4M3FN_TABLE

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
K = 40
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NORMS = {"none": B.NORM_NONE, "rms": B.NORM_RMS, "layer": B.NORM_LAYER}


def f64(t):
    torch.cuda.synchronize()
    return t.cpu().double().numpy()


def table(rng, n_pos, rot):
    a = rng.uniform(-np.pi, np.pi, (n_pos, rot // 2))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def close(got, want, T, kind):
    half = torch.finfo(TYPES[kind]).eps / 2
    floor = 2.0 ** -25 if kind == "fp16" else 0.0
    off = np.abs(got - want)
    tol = K * U * T
    assert (off <= tol + half * (np.abs(want) + tol) + floor).all(), np.max(off - tol - half * np.abs(want))


CASES = [
    # tokens, q heads, k heads, dim, rot, rot_begin, interleaved, q norm, k norm, weights, biases
    (1, 1, 1, 8, 0, 0, False, "rms", "layer", True, True),
    (1, 64, 1, 128, 64, 0, False, "none", "layer", True, True),
    (5, 3, 2, 16, 16, 0, True, "rms", "rms", True, False),
    (3, 7, 0, 64, 64, 0, False, "rms", "rms", True, False),
    (9, 0, 3, 64, 32, 16, True, "layer", "layer", False, True),
    (17, 5, 4, 96, 96, 0, False, "layer", "rms", True, True),
    (33, 6, 1, 128, 128, 0, True, "rms", "rms", True, True),
    (65, 2, 1, 192, 64, 128, True, "rms", "rms", True, False),
    (31, 3, 2, 192, 64, 128, False, "rms", "none", True, False),
    (12, 4, 2, 256, 256, 0, False, "layer", "layer", True, True),
    (20, 3, 1, 40, 32, 8, False, "rms", "layer", False, False),
    (4, 2, 2, 200, 16, 184, False, "none", "none", False, False),
    (60, 37, 2, 64, 64, 0, False, "rms", "layer", True, True),
]
# Enough heads for several loads a wave: a token's heads in whole and partial chunks, few heads.
FULL = [
    (4200, 37, 2, 64, 64, 0, False, "rms", "layer", True, True),
    (8300, 3, 17, 128, 64, 64, True, "layer", "rms", True, False),
    (9000, 1, 6, 96, 32, 8, False, "layer", "rms", True, True),
    (4200, 32, 2, 64, 32, 16, True, "rms", "rms", True, False),
    (8300, 32, 3, 128, 64, 0, False, "rms", "layer", True, True),
]


def make(rng, c, kind):
    n, hq, hk, d, rot, begin, inter, qn, kn, weights, biases = c
    t = TYPES[kind]
    q = torch.from_numpy(rng.standard_normal((n, hq, d)) * 3).to(t)
    k = torch.from_numpy(rng.standard_normal((n, hk, d)) + 0.7).to(t)
    vec = lambda on: rng.standard_normal(d).astype(np.float32) if on else None
    par = dict(q_weight=vec(weights), q_bias=vec(biases), k_weight=vec(weights), k_bias=vec(biases))
    cs = table(rng, 50, rot) if rot else None
    pos = rng.integers(0, 50, n).astype(np.int32)
    return q, k, par, cs, pos


def want_of(c, q, k, par, cs, pos, eps):
    n, hq, hk, d, rot, begin, inter, qn, kn, weights, biases = c
    out = []
    for x, kind, s in ((q, qn, "q"), (k, kn, "k")):
        v, T = O.norm(x.double().numpy(), kind, par[s + "_weight"], par[s + "_bias"], eps)
        if cs is not None:
            v, T = O.rotate(v, T, pos, cs, begin, inter)
        out += [v, T]
    return out


def call(c, q, k, par, cs, pos, qo, ko, eps, **kw):
    n, hq, hk, d, rot, begin, inter, qn, kn, weights, biases = c
    p = {name: None if v is None else dev(v) for name, v in par.items()}
    B.qk_norm_rope(q, k, qo, ko, dev(pos), None if cs is None else dev(cs), rot_begin=begin, interleaved=inter,
                   q_norm=NORMS[qn], k_norm=NORMS[kn], eps=eps, **p, **kw)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("c", CASES, ids=lambda c: "t%d_%d+%d_d%d_r%d_%s" % (c[0], c[1], c[2], c[3], c[4], c[7]))
def test_heads(c, kind):
    announce("heads", c, kind)
    rng = np.random.default_rng(c[0] * 100 + c[3])
    q, k, par, cs, pos = make(rng, c, kind)
    qo, ko = torch.full_like(q, -77.0, device="cuda"), torch.full_like(k, -77.0, device="cuda")
    call(c, q.cuda(), k.cuda(), par, cs, pos, qo, ko, 1e-5)
    wq, Tq, wk, Tk = want_of(c, q, k, par, cs, pos, 1e-5)
    close(f64(qo), wq, Tq, kind)
    close(f64(ko), wk, Tk, kind)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("c", FULL, ids=lambda c: "t%d_%d+%d_d%d" % c[:4])
def test_heads_full(c, kind):
    test_heads(c, kind)


def test_views_of_one_projection_in_place():
    """q and k as views of one [tokens, (5 + 2 + 2) * 64] buffer, turned in place; the values
    between them stay."""
    rng = np.random.default_rng(3)
    c = (19, 5, 2, 64, 64, 0, False, "rms", "layer", True, True)
    _, _, par, cs, pos = make(rng, c, "bf16")
    x = torch.from_numpy(rng.standard_normal((19, 9 * 64))).to(torch.bfloat16)
    b = x.cuda()
    q, k = b[:, :320].view(19, 5, 64), b[:, 320:448].view(19, 2, 64)
    call(c, q, k, par, cs, pos, q, k, 1e-6)
    wq, Tq, wk, Tk = want_of(c, x[:, :320].reshape(19, 5, 64), x[:, 320:448].reshape(19, 2, 64), par, cs, pos, 1e-6)
    got = f64(b)
    close(got[:, :320].reshape(19, 5, 64), wq, Tq, "bf16")
    close(got[:, 320:448].reshape(19, 2, 64), wk, Tk, "bf16")
    assert np.array_equal(got[:, 448:], x[:, 448:].double().numpy())


def test_heads_before_tokens():
    """Layouts [heads, tokens, dim] seen as [tokens, heads, dim]."""
    rng = np.random.default_rng(8)
    c = (23, 4, 2, 128, 64, 64, True, "rms", "rms", True, False)
    q, k, par, cs, pos = make(rng, c, "fp16")
    qt, kt = q.cuda().transpose(0, 1).contiguous().transpose(0, 1), k.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    qo = torch.full((4, 23, 128), -77.0, dtype=q.dtype, device="cuda").transpose(0, 1)
    ko = torch.full((23, 2, 128), -77.0, dtype=q.dtype, device="cuda")
    call(c, qt, kt, par, cs, pos, qo, ko, 1e-6)
    wq, Tq, wk, Tk = want_of(c, q, k, par, cs, pos, 1e-6)
    close(f64(qo), wq, Tq, "fp16")
    close(f64(ko), wk, Tk, "fp16")


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_padding_tokens_are_left_alone(kind):
    rng = np.random.default_rng(5)
    c = (40, 3, 1, 128, 64, 0, False, "rms", "rms", True, False)
    q, k, par, cs, pos = make(rng, c, kind)
    bad = rng.random(40) < 0.4
    pos[bad] = rng.choice([-1, -2 ** 31, 50, 2 ** 31 - 1], bad.sum())
    qo, ko = torch.full_like(q, -77.0, device="cuda"), torch.full_like(k, -77.0, device="cuda")
    call(c, q.cuda(), k.cuda(), par, cs, pos, qo, ko, 1e-6)
    assert (f64(qo)[bad] == -77).all() and (f64(ko)[bad] == -77).all()
    wq, Tq, wk, Tk = want_of(c, q, k, par, cs, np.where(bad, 0, pos), 1e-6)
    close(f64(qo)[~bad], wq[~bad], Tq[~bad], kind)
    close(f64(ko)[~bad], wk[~bad], Tk[~bad], kind)


def test_heads_of_zeros_and_bad_values_stay_apart():
    """A head of zeros is zero (RMS) or its bias (layer); NaN and infinities stay in their head."""
    rng = np.random.default_rng(6)
    c = (4, 5, 2, 64, 64, 0, False, "rms", "layer", True, True)
    q, k, par, cs, pos = make(rng, c, "fp32")
    par["q_bias"] = None
    q[1, 2] = 0
    q[2, 0, 5], q[3, 4, 63] = float("nan"), float("inf")
    k[0, 1] = 0
    qo, ko = torch.empty_like(q, device="cuda"), torch.empty_like(k, device="cuda")
    call(c, q.cuda(), k.cuda(), par, cs, pos, qo, ko, 1e-6)
    got = f64(qo)
    assert (got[1, 2] == 0).all()
    nan = np.isnan(got).any(-1)
    assert nan[2, 0] and nan[3, 4] and nan.sum() == 2
    wq, Tq, wk, Tk = want_of(c, torch.nan_to_num(q, 0.0, 0.0, 0.0), k, par, cs, pos, 1e-6)
    close(got[~nan], wq[~nan], Tq[~nan], "fp32")
    close(f64(ko), wk, Tk, "fp32")


# ---------------------------------------------------------------- the indexer's form
def check_fp8(codes, scale, v, T, what):
    """codes [..., 128] and scale [...] of values v with error magnitudes T."""
    amax = np.abs(v).max(-1)
    assert (np.abs(scale - np.maximum(amax / 448, SCALE_MIN)) <= K * U * T.max(-1) / 448 + 2 * U * scale).all(), what
    t = v / scale[..., None]
    off = np.abs(E4M3FN_TABLE[codes] - t)
    assert (off <= nearest_distance(t) + K * U * T / scale[..., None] + 4 * U * np.abs(t)).all(), what


INDEXER = [
    # tokens, heads, rot, rot_begin, interleaved, slots
    (1, 64, 64, 0, False, 3),
    (7, 64, 64, 0, True, 40),
    (50, 64, 64, 64, False, 50),
    (13, 3, 128, 0, False, 100),
    (6, 0, 64, 0, False, 9),
]
INDEXER_FULL = [(2300, 64, 64, 0, False, 2301), (2300, 64, 64, 64, True, 2300), (4300, 64, 64, 0, True, 4310)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("n,h,rot,begin,inter,slots", INDEXER)
def test_indexer_inputs(n, h, rot, begin, inter, slots, kind):
    announce("indexer", n, h, rot, begin, inter, slots, kind)
    rng = np.random.default_rng(n + h + rot)
    c = (n, h, 1, 128, rot, begin, inter, "none", "layer", True, True)
    q, k, par, cs, pos = make(rng, c, kind)
    w = rng.standard_normal((n, h + 2)).astype(np.float32)
    slot = rng.permutation(slots)[:n].astype(np.int64)
    lost = np.zeros(n, bool)                          # tokens without a cache row
    if n > 5:
        lost[[1, 4]] = True
        slot[1], slot[4] = -1, slots
    q8 = torch.full((n, h, 128), 0xEE, dtype=torch.uint8, device="cuda")
    w_out = torch.full((n, h), -77.0, device="cuda")
    cache = torch.full((slots, 128), 0xEE, dtype=torch.uint8, device="cuda")
    cache_scale = torch.full((slots,), -77.0, device="cuda")
    B.indexer_qk(q.cuda(), k.cuda(), dev(w)[:, 1:1 + h], q8, w_out, cache, cache_scale, dev(slot), dev(pos), dev(cs),
                 w_mul=0.37, rot_begin=begin, interleaved=inter, k_norm=B.NORM_LAYER,
                 k_weight=dev(par["k_weight"]), k_bias=dev(par["k_bias"]))
    wq, Tq, wk, Tk = want_of(c, q, k, par, cs, pos, 1e-6)
    if h:
        got_w = f64(w_out)
        base = np.float64(np.float32(0.37)) * w[:, 1:1 + h].astype(np.float64)
        scale = np.abs(wq).max(-1) / 448
        assert (np.abs(got_w - base * scale) <= np.abs(base) * (K * U * Tq.max(-1) / 448 + 6 * U * scale)).all()
        check_fp8(host(q8), np.where(base != 0, got_w / base, scale), wq, Tq + 4 * np.abs(wq), "q")
    rows = slot[~lost]
    check_fp8(host(cache)[rows], host(cache_scale)[rows].astype(np.float64), wk[~lost, 0], Tk[~lost, 0], "k")
    rest = np.setdiff1d(np.arange(slots), rows)
    assert (host(cache)[rest] == 0xEE).all() and (host(cache_scale)[rest] == -77).all()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("n,h,rot,begin,inter,slots", INDEXER_FULL)
def test_indexer_inputs_full(n, h, rot, begin, inter, slots, kind):
    test_indexer_inputs(n, h, rot, begin, inter, slots, kind)


def test_indexer_padding_tokens():
    rng = np.random.default_rng(1)
    n = 9
    c = (n, 64, 1, 128, 64, 0, False, "rms", "layer", True, True)
    q, k, par, cs, pos = make(rng, c, "bf16")
    pos[[0, 3, 8]] = [-1, 50, -7]
    slot = np.arange(n, dtype=np.int64)
    q8 = torch.full((n, 64, 128), 0xEE, dtype=torch.uint8, device="cuda")
    w_out = torch.full((n, 64), -77.0, device="cuda")
    cache = torch.full((n, 128), 0xEE, dtype=torch.uint8, device="cuda")
    cache_scale = torch.full((n,), -77.0, device="cuda")
    B.indexer_qk(q.cuda(), k.cuda(), torch.ones((n, 64), device="cuda"), q8, w_out, cache, cache_scale, dev(slot),
                 dev(pos), dev(cs), q_norm=B.NORM_RMS, q_weight=dev(par["q_weight"]), k_norm=B.NORM_LAYER)
    pad = np.zeros(n, bool)
    pad[[0, 3, 8]] = True
    assert (host(q8)[pad] == 0xEE).all() and (host(cache)[pad] == 0xEE).all()
    assert (f64(w_out)[pad] == -77).all() and (f64(cache_scale)[pad] == -77).all()
    assert (f64(w_out)[~pad] > 0).all() and (f64(cache_scale)[~pad] > 0).all()


@pytest.mark.parametrize("n", [1, 30])
def test_captured_heads_on_another_stream(n):
    """Captured on a side stream and replayed three times over changed inputs: each replay equals
    the eager call, with eager work in between."""
    rng = np.random.default_rng(2)
    c = (n, 64, 1, 128, 64, 0, False, "none", "layer", True, True)
    q, k, par, cs, pos = make(rng, c, "bf16")
    q, k, cs_d, pos_d = q.cuda(), k.cuda(), dev(cs), dev(pos)
    w, slot = torch.ones((n, 64), device="cuda"), dev(np.arange(n, dtype=np.int64))
    p = dict(k_weight=dev(par["k_weight"]), k_bias=dev(par["k_bias"]), k_norm=B.NORM_LAYER)
    outs = lambda: (torch.zeros((n, 64, 128), dtype=torch.uint8, device="cuda"), torch.zeros((n, 64), device="cuda"),
                    torch.zeros((n, 128), dtype=torch.uint8, device="cuda"), torch.zeros(n, device="cuda"))
    a, b = outs(), outs()
    main = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = B.CapturedGraph(lambda st: B.indexer_qk(q, k, w, *a, slot, pos_d, cs_d, stream=st, **p), main)
    for step in range(3):
        q.copy_(torch.from_numpy(rng.standard_normal((n, 64, 128))).to(q.dtype))
        torch.cuda.synchronize()
        g.launch(main)
        torch.cuda.synchronize()
        B.indexer_qk(q, k, w, *b, slot, pos_d, cs_d, **p)
        for x, y in zip(a, b):
            assert np.array_equal(host(x), host(y)), step
    g.close()


def test_no_positions_and_no_slots():
    """A table of no positions makes every token padding; a cache of no rows takes no key."""
    q, k = torch.ones((3, 2, 128), device="cuda"), torch.ones((3, 1, 128), device="cuda")
    pos, slot = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    full = lambda *s: torch.full(s, -77.0, device="cuda")
    codes = lambda *s: torch.full(s, 0xEE, dtype=torch.uint8, device="cuda")
    qo, ko = full(3, 2, 128), full(3, 1, 128)
    B.qk_norm_rope(q, k, qo, ko, pos, torch.zeros((0, 64), device="cuda"))
    assert (f64(qo) == -77).all() and (f64(ko) == -77).all()
    q8, w_out = codes(3, 2, 128), full(3, 2)
    B.indexer_qk(q, k, torch.ones((3, 2), device="cuda"), q8, w_out, codes(0, 128), full(0), slot, pos, None)
    assert (host(q8) == 0x7E).all()                   # 448: every value is the largest
    assert np.array_equal(host(w_out), np.full((3, 2), np.float32(1) / np.float32(448)))
