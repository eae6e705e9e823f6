"""FP8 in blocks of 128: echo_quant_fp8 and echo_matmul_fp8 against the oracle in float64.

Tolerances (u = 2^-24).  Scales are one division of fp32 numbers: equal to numpy's.  A code is the
E4M3FN number nearest to the fp32 quotient x / scale, bit for bit (the last tests here); against the
quotient in 64 bits it may be off the nearest number's distance by its rounding, 4 u |x / scale| at most.  A
product sums up to 128 terms in a block, nb blocks and 8 partial sums in fp32; should the matrix
core cut instead of rounding, each step is off by 2 u: (128 + nb + 8 + 3) * 2 u times the sum of
the terms' magnitudes, plus half a step of the output's type.

Sums for 16-bit outputs may come from the FP8 matrix core, which is not an fp32 sum of products.
Measured on gfx950: of eight neighbouring products with one of 2^16, another one of 2^e is in the sum
for e >= 3 and gone for e < 3; 225 * 2^-6 * 2^e (15/8 squared) is cut to a multiple of 8 = 2^(16-13),
towards zero, for either sign; products of other groups are kept to fp32.  So a product loses less
than 2^-13 of the power of two of its group's largest product, which is at most that product: a
group loses at most 7 * 2^-13 of its largest product's magnitude (the largest one's own last bits,
2^-6 of its power of two, are kept), and an output at most that summed over the groups."""

import numpy as np
import pytest
import torch

from dsa_indexer_top_amd import binding as B
from gpu_util import announce, dev, host
from oracle import blockfp8 as O
from oracle.fp8 import E4M3FN_TABLE

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF_STEP = {t: torch.finfo(d).eps / 2 for t, d in TYPES.items()}


def f64(t):
    torch.cuda.synchronize()
    return t.cpu().double().numpy()


def check_codes(codes, scale, x, what=""):
    """Codes and scales of x (float64 of what the kernel read)."""
    want = np.maximum(np.float32(448.0 * O.SCALE_MIN), np.stack(
        [np.abs(x[:, b:b + 128]).max(1) for b in range(0, x.shape[1], 128)], 1).astype(np.float32)) / np.float32(448)
    assert np.array_equal(scale, want), what
    t = x / O.spread(scale.astype(np.float64), x.shape[1])
    off = np.abs(E4M3FN_TABLE[codes] - t)
    assert (off <= O.nearest_distance(t) + 4 * U * np.abs(t)).all(), (what, np.max(off - O.nearest_distance(t)))


QUANT = [(1, 128), (1, 1), (3, 127), (5, 129), (33, 300), (2, 2047), (17, 1024), (260, 8), (1, 5000), (40, 2047)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,cols", QUANT)
def test_quant(rows, cols, kind):
    announce("quant", rows, cols, kind)
    rng = np.random.default_rng(rows * 1000 + cols)
    x = torch.from_numpy(rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)) * 2)).to(TYPES[kind])
    ld = cols + 1 if rows in (40, 4110) else -(-cols // 16) * 16     # rows at any address, or on 16 bytes
    y = torch.full((rows, ld), 0xEE, dtype=torch.uint8, device="cuda")
    scale = torch.full((rows, -(-cols // 128)), -1.0, device="cuda")
    B.quant_fp8(x.cuda(), y[:, :cols], scale)
    check_codes(host(y)[:, :cols], host(scale), x.double().numpy())
    assert (host(y)[:, cols:] == 0xEE).all()          # what stands behind a row is left


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,cols", [(4100, 2048), (4110, 2047)])
def test_quant_full(rows, cols, kind):
    """Enough blocks for several a wave."""
    test_quant(rows, cols, kind)


def test_quant_strides_and_odd_addresses():
    rng = np.random.default_rng(2)
    base = torch.from_numpy(rng.standard_normal((9, 701))).to(torch.bfloat16)
    x = base.cuda()[:, 3:3 + 391]                     # rows that start on 2 bytes
    y = torch.full((9, 400), 0xEE, dtype=torch.uint8, device="cuda")
    scale = torch.full((4, 9), -1.0, device="cuda")   # scales with blocks as rows
    B.quant_fp8(x, y[:, 1:392], scale.t())
    check_codes(host(y)[:, 1:392], host(scale).T, base[:, 3:394].double().numpy())
    assert (host(y)[:, 0] == 0xEE).all() and (host(y)[:, 392:] == 0xEE).all()


def test_quant_values_at_the_borders():
    """Zeros, subnormals, the largest numbers, halves between codes, infinities and NaN."""
    rows = [np.zeros(256), np.full(256, 1e-38), np.linspace(-448, 448, 256), np.full(256, 3.0e38),
            np.r_[448.0, np.arange(255) * 1.0625], np.full(256, 1e-45), np.r_[448.0, 2.0 ** -10 * np.arange(255)]]
    x = np.array(rows, np.float32)
    xt = torch.from_numpy(x)
    y = torch.empty((len(x), 256), dtype=torch.uint8, device="cuda")
    scale = torch.empty((len(x), 2), device="cuda")
    B.quant_fp8(xt.cuda(), y, scale)
    check_codes(host(y), host(scale), x.astype(np.float64))
    assert (host(scale) > 0).all() and (host(y)[0] & 0x7F == 0).all()
    # a block with a NaN or an infinity stands for NaN; its neighbours are as they would be
    for bad in (np.nan, np.inf, -np.inf):
        z = x[2:5].copy()
        z[1, 5] = bad
        B.quant_fp8(torch.from_numpy(z).cuda(), y[:3], scale[:3])
        with np.errstate(invalid="ignore"):
            v = E4M3FN_TABLE[host(y)[:3]] * O.spread(host(scale)[:3].astype(np.float64), 256)
        assert np.isnan(v[1, :128]).all() and not np.isnan(v[1, 128:]).any() and not np.isnan(v[[0, 2]]).any()


def product_case(rng, m, n, k, grid=False):
    """Codes with 16-byte rows whose bytes behind k are NaN codes, and scales."""
    ld = -(-k // 16) * 16
    a, b = (np.full((r, ld), 0x7F, np.uint8) for r in (m, n))
    if grid:                                          # whole numbers: every sum is exact
        codes = np.flatnonzero(np.isin(E4M3FN_TABLE, np.arange(-4, 5)))
        a[:, :k], b[:, :k] = (rng.choice(codes, (r, k)) for r in (m, n))
        scales = [2.0 ** rng.integers(-3, 4, s) for s in ((m, -(-k // 128)), (-(-n // 128), -(-k // 128)))]
    else:
        finite = np.flatnonzero(np.isfinite(E4M3FN_TABLE))
        a[:, :k], b[:, :k] = (rng.choice(finite, (r, k)) for r in (m, n))
        scales = [np.exp(rng.standard_normal(s)) for s in ((m, -(-k // 128)), (-(-n // 128), -(-k // 128)))]
    return a, b, scales[0].astype(np.float32), scales[1].astype(np.float32)


def check_product(got, a, sa, b, sb, k, half_step, what):
    want, T = O.matmul(a[:, :k], sa, b[:, :k], sb)
    tol = (128 + -(-k // 128) + 11) * 2 * U * T
    off = np.abs(got - want)
    assert (off <= tol + half_step * (np.abs(want) + tol)).all(), (what, np.max(off / np.maximum(T, 1e-30)))


# sizes about 16, the tiles' edges, one and several workgroups, K of part of a block
PRODUCT = [(1, 1, 1), (1, 16, 128), (1, 300, 130), (7, 33, 129), (16, 128, 256), (17, 130, 1100), (33, 17, 300),
           (64, 64, 128), (65, 129, 300), (100, 260, 31), (130, 128, 256), (129, 300, 400), (200, 1, 140),
           (257, 5, 128), (270, 270, 272)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("m,n,k", PRODUCT)
def test_product(m, n, k, kind):
    announce("product", m, n, k, kind)
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    a, b, sa, sb = product_case(rng, m, n, k)
    if kind == "fp16":                                # keep the sums below fp16's 65504
        sa *= np.float32(1e-4 / max(1.0, k / 128))
    c = torch.full((m, n + 3), -77.0, dtype=TYPES[kind], device="cuda")
    B.matmul_fp8(dev(a)[:, :k], dev(sa), dev(b)[:, :k], dev(sb), c[:, :n])
    # fp16 below its normal numbers rounds in steps of 2^-24
    half = HALF_STEP[kind]
    got = f64(c)
    want, T = O.matmul(a[:, :k], sa, b[:, :k], sb)
    tol = (128 + -(-k // 128) + 11) * 2 * U * T
    if kind != "fp32":
        tol = tol + 7 * 2.0 ** -13 * O.group_maxima(a[:, :k], sa, b[:, :k], sb)
    floor = 2.0 ** -25 if kind == "fp16" else 0.0
    assert (np.abs(got[:, :n] - want) <= tol + half * (np.abs(want) + tol) + floor).all()
    assert (got[:, n:] == -77.0).all()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("m,n,k", [(600, 530, 140), (520, 600, 1030), (33, 4100, 270)])
def test_product_of_more_tiles(m, n, k, kind):
    """More outputs than the chip's workgroups of 32 x 32: the wider tiles, and their waves sharing K."""
    test_product(m, n, k, kind)


@pytest.mark.parametrize("m,n,k", [(5, 40, 300), (40, 70, 500), (140, 140, 384)])
def test_product_exact_on_whole_numbers(m, n, k):
    """Small whole numbers and powers of two as scales: every partial sum is exact in fp32."""
    rng = np.random.default_rng(k)
    a, b, sa, sb = product_case(rng, m, n, k, grid=True)
    c = torch.empty((m, n), device="cuda")
    B.matmul_fp8(dev(a)[:, :k], dev(sa), dev(b)[:, :k], dev(sb), c)
    assert np.array_equal(f64(c), O.matmul(a[:, :k], sa, b[:, :k], sb)[0])


@pytest.mark.parametrize("m", [3, 50, 150])
def test_product_strides(m):
    """Scales with blocks as rows, wide rows of a, b and c, columns of c that allow no wide store."""
    rng = np.random.default_rng(m)
    n, k = 150, 260
    a, b, sa, sb = product_case(rng, m, n, k)
    at, bt = torch.full((m, 320), 0x7F, dtype=torch.uint8, device="cuda"), torch.full((n, 400), 0x7F, dtype=torch.uint8, device="cuda")
    at[:, 16:16 + k], bt[:, 32:32 + k] = dev(a)[:, :k], dev(b)[:, :k]
    c = torch.full((m, n + 7), -77.0, device="cuda")
    B.matmul_fp8(at[:, 16:16 + k], dev(sa.T).t(), bt[:, 32:32 + k], dev(sb.T).t(), c[:, 3:3 + n])
    got = f64(c)
    check_product(got[:, 3:3 + n], a, sa, b, sb, k, HALF_STEP["fp32"], m)
    assert (got[:, :3] == -77.0).all() and (got[:, 3 + n:] == -77.0).all()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("m,n", [(3, 150), (50, 150), (300, 270), (600, 530),
                                 *(pytest.param(m, n, id=f"full-{m}-{n}") for m, n in [(1200, 1010), (1700, 2050), (2200, 2010),
                                                                                   (4100, 8201)])])
def test_product_at_odd_addresses(m, n, kind):
    """The same bits whether or not a row starts at a multiple of a wide store; nothing beside them."""
    rng = np.random.default_rng(m)
    k = 140
    a, b, sa, sb = product_case(rng, m, n, k)
    ops = (dev(a)[:, :k], dev(sa), dev(b)[:, :k], dev(sb))
    want = torch.empty((m, -(-n // 8) * 8), dtype=TYPES[kind], device="cuda")[:, :n]
    B.matmul_fp8(*ops, want)
    c = torch.full((m, -(-n // 2) * 2 + 5), -77.0, dtype=TYPES[kind], device="cuda")
    B.matmul_fp8(*ops, c[:, 1:1 + n])
    assert torch.equal(c[:, 1:1 + n], want)
    assert (c[:, :1] == -77.0).all() and (c[:, 1 + n:] == -77.0).all()


@pytest.mark.parametrize("m", [2, 40, 140])
def test_product_nan_stays_in_its_row_and_column(m):
    rng = np.random.default_rng(9)
    n, k = 70, 200
    a, b, sa, sb = product_case(rng, m, n, k)
    a[1, 130] = 0x7F
    b[69, 5] = 0xFF
    c = torch.empty((m, n), device="cuda")
    B.matmul_fp8(dev(a)[:, :k], dev(sa), dev(b)[:, :k], dev(sb), c)
    nan = np.isnan(f64(c))
    assert nan[1].all() and nan[:, 69].all() and nan.sum() == n + m - 1


@pytest.mark.parametrize("m", [3, 200])
def test_product_of_nothing(m):
    c = torch.full((m, 20), 5.0, device="cuda")
    z = lambda r, w, t: torch.zeros((r, w), dtype=t, device="cuda")
    B.matmul_fp8(z(m, 0, torch.uint8), z(m, 0, torch.float32), z(20, 0, torch.uint8), z(1, 0, torch.float32), c)
    assert (f64(c) == 0).all()
    B.matmul_fp8(z(0, 64, torch.uint8), z(0, 1, torch.float32), z(20, 64, torch.uint8), z(1, 1, torch.float32), c[:0])


def test_quant_then_product_of_hidden_states():
    """bf16 states to FP8 and through a projection: within the quantiser's half steps of the
    product of the unquantised states (an E4M3FN code is off by at most 2^-4 of its value, or half
    a subnormal step, 2^-10 of the scale)."""
    rng = np.random.default_rng(4)
    m, n, k = 21, 130, 520
    x = torch.from_numpy(rng.standard_normal((m, k))).to(torch.bfloat16)
    _, b, _, sb = product_case(rng, 1, n, k)
    y = torch.empty((m, 528), dtype=torch.uint8, device="cuda")[:, :k]
    sa = torch.empty((5, m), device="cuda").t()
    c = torch.empty((m, n), device="cuda")
    B.quant_fp8(x.cuda(), y, sa)
    B.matmul_fp8(y, sa, dev(b)[:, :k], dev(sb), c)
    bv = E4M3FN_TABLE[b[:, :k]] * O.spread(np.repeat(sb.astype(np.float64), 128, 0)[:n], k)
    xv, s = x.double().numpy(), O.spread(host(sa).astype(np.float64), k)
    bound = (np.abs(xv) * 2.0 ** -4 + s * 2.0 ** -10) @ np.abs(bv).T * 1.001
    assert (np.abs(f64(c) - xv @ bv.T) <= bound).all()


# Every tile's shape at sizes that fill the chip with it, edges included (the products' last rows,
# columns and block are partial), and one whole number of tiles.
@pytest.mark.parametrize("m,n,k,kind", [
    (4100, 4111, 400, "bf16"), (4096, 4096, 384, "fp16"), (2000, 2100, 300, "fp32"), (2000, 2100, 777, "bf16"),
    (2048, 2048, 256, "fp32"), (1030, 2050, 700, "bf16"), (1024, 2048, 1152, "fp16"), (1024, 2048, 130, "fp32"),
    (640, 640, 1500, "bf16"), (640, 640, 1408, "fp32"), (33, 4000, 640, "bf16"), (32, 8192, 1111, "bf16"),
    (31, 1000, 2047, "fp32"), (16, 3001, 2048, "fp16"), (1200, 1010, 260, "bf16"), (1200, 1010, 1100, "fp32"),
    (2200, 2010, 700, "fp16"), (4100, 2570, 520, "bf16"), (64, 2047, 1500, "fp16"), (509, 510, 2047, "bf16"),
    (120, 101, 6001, "fp32")])
def test_product_full_size_tiles_exact(m, n, k, kind):
    """Whole numbers and powers of two as scales: exact in fp32 in any order and on either matrix
    core (a product is at most 2^4 times another's unit, far above 2^-13), so the result is the
    float64 one rounded once."""
    announce("product tiles", m, n, k, kind)
    g = torch.Generator().manual_seed(m + n + k)
    ld = -(-k // 16) * 16
    f8 = torch.float8_e4m3fn
    ints = lambda r: torch.randint(-4, 5, (r, k), generator=g).double()
    av, bv = ints(m), ints(n)
    code = lambda v: torch.cat([v.float().to(f8).view(torch.uint8), torch.full((v.shape[0], ld - k), 0x7F, dtype=torch.uint8)], 1)
    nb = -(-k // 128)
    sa = 2.0 ** torch.randint(-3, 1, (m, nb), generator=g)
    sb = 2.0 ** torch.randint(-3, 1, (-(-n // 128), nb), generator=g)
    c = torch.full((m, n), -77.0, dtype=TYPES[kind], device="cuda")
    B.matmul_fp8(code(av).cuda()[:, :k], sa.cuda(), code(bv).cuda()[:, :k], sb.cuda(), c)
    spread = lambda s: s.double().repeat_interleave(128, 1)[:, :k]
    want = (av * spread(sa)).cuda() @ (bv * spread(sb.repeat_interleave(128, 0)[:n])).cuda().t()
    assert torch.equal(c, want.to(TYPES[kind]))


# ---------------------------------------------------------------- codes bit for bit
def fp32_codes(x, scale):
    """The fp32 quotient of value and scale (one IEEE division) rounded to the nearest code."""
    with np.errstate(invalid="ignore"):
        q = x.astype(np.float32) / np.repeat(scale, 128, 1)[:, :x.shape[1]]
    return torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def quotients_at_ties(rng, n):
    """Blocks whose values over their scale lie on, and a few units in the last place beside, the
    numbers halfway between two codes; scales from 2^-126 to 2^118."""
    finite = np.unique(E4M3FN_TABLE[np.isfinite(E4M3FN_TABLE)])
    ties = ((finite[1:] + finite[:-1]) / 2).astype(np.float32)
    x = np.zeros((n, 128), np.float32)
    for r in range(n):
        d = np.float32(2.0 ** rng.integers(-126, 118) * rng.uniform(1, 2))
        if r % 3 == 0:                                # few bits, so that products with a tie are exact
            d = np.float32(2.0 ** rng.integers(-126, 118) * rng.integers(8, 16) / 8 * (1 + rng.integers(-4, 5) * 2.0 ** -23))
        x[r, 0] = np.float32(448) * d
        d = x[r, 0] / np.float32(448)
        v = (rng.choice(ties, 127).astype(np.float64) * d).astype(np.float32)
        steps = rng.integers(-3, 4, 127).astype(np.int32)
        v = np.where(np.abs(v) > 1e-44, (v.view(np.int32) + steps).view(np.float32), v)
        x[r, 1:] = np.clip(v, -x[r, 0], x[r, 0])
    return x


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,cols", [(70, 1024), (9, 391), (520, 1000)])
def test_quant_codes_are_the_rounded_quotients(rows, cols, kind):
    rng = np.random.default_rng(rows)
    x = torch.from_numpy(rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)) * 2)).to(TYPES[kind])
    x[1] = -x[0].abs()
    x[2, ::2], x[2, 1::2] = 0.0, -0.0
    y = torch.empty((rows, cols), dtype=torch.uint8, device="cuda")
    scale = torch.empty((rows, -(-cols // 128)), device="cuda")
    B.quant_fp8(x.cuda(), y, scale)
    assert np.array_equal(host(y), fp32_codes(x.float().numpy(), host(scale)))


def test_quant_codes_beside_ties():
    x = quotients_at_ties(np.random.default_rng(31), 600)
    x = np.concatenate([x, np.full((1, 128), 1e-45, np.float32), np.linspace(-1e-38, 1e-38, 128, dtype=np.float32)[None],
                        np.full((1, 128), 3.4e38, np.float32)])
    y = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
    scale = torch.empty((len(x), 1), device="cuda")
    B.quant_fp8(torch.from_numpy(x).cuda(), y, scale)
    assert np.array_equal(host(scale)[:, 0], np.maximum(np.abs(x).max(1), np.float32(448 * 2.0 ** -126)) / np.float32(448))
    assert np.array_equal(host(y), fp32_codes(x, host(scale)))


@pytest.mark.parametrize("kind", list(TYPES))
def test_indexer_codes_are_the_quantisers(kind):
    """Heads that are neither normed nor turned: the codes of echo_quant_fp8, one scale a head."""
    rng = np.random.default_rng(7)
    n, h = 11, 5
    x = torch.from_numpy(rng.standard_normal((n, h + 1, 128)) * np.exp(rng.standard_normal((n, h + 1, 1)) * 2)).to(TYPES[kind])
    if kind == "fp32":
        x.view(-1, 128)[:] = torch.from_numpy(quotients_at_ties(rng, n * (h + 1)))
    x = x.cuda()
    codes, scale = torch.empty((n * (h + 1), 128), dtype=torch.uint8, device="cuda"), torch.empty((n * (h + 1), 1), device="cuda")
    B.quant_fp8(x.view(-1, 128), codes, scale)
    q8, w_out = torch.empty((n, h, 128), dtype=torch.uint8, device="cuda"), torch.empty((n, h), device="cuda")
    k8, k_scale = torch.empty((n, 128), dtype=torch.uint8, device="cuda"), torch.empty(n, device="cuda")
    B.indexer_qk(x[:, :h], x[:, h:], torch.ones((n, h), device="cuda"), q8, w_out, k8, k_scale,
                 dev(np.arange(n, dtype=np.int64)), torch.zeros(n, dtype=torch.int32, device="cuda"), None)
    codes, scale = host(codes).reshape(n, h + 1, 128), host(scale).reshape(n, h + 1)
    assert np.array_equal(host(q8), codes[:, :h]) and np.array_equal(host(w_out), scale[:, :h])
    assert np.array_equal(host(k8), codes[:, h]) and np.array_equal(host(k_scale), scale[:, h])


def test_quant_codes_of_all_significands():
    """Every fp16 significand over every other's scale (bf16 has fewer), in random binades."""
    rng = np.random.default_rng(17)
    x = np.zeros((1024, 9, 128), np.float32)
    x[:, :, 0] = (8 + np.arange(1024) / 128)[:, None]
    x[:, :, 1:] = (1 + np.resize(np.arange(1024), 9 * 127) / 1024).reshape(9, 127) * 2.0 ** rng.integers(-9, 3, (1024, 9, 127))
    x = torch.from_numpy(x.reshape(1024, -1)).half()
    y = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
    scale = torch.empty((1024, 9), device="cuda")
    B.quant_fp8(x.cuda(), y, scale)
    assert np.array_equal(host(y), fp32_codes(x.float().numpy(), host(scale)))


@pytest.mark.parametrize("kind", list(TYPES))
def test_quant_blocks_of_all_sizes_side_by_side(kind):
    """Blocks of zeros, of tiny and huge values, infinities and NaN next to ordinary ones: every
    block's codes are its own."""
    rng = np.random.default_rng(12)
    x = rng.standard_normal((64, 128 * 9)).reshape(64, 9, 128)
    small, large = (2.0 ** -20, 2.0 ** 12) if kind == "fp16" else (2.0 ** -100, 2.0 ** 100)
    x *= rng.choice([0.0, 1.0, 1.0, small, large], (64, 9, 1))
    x[5, 2, 7], x[9, 0, 100], x[9, 8, 3] = np.nan, np.inf, -np.inf
    x[20, 4] = -0.0
    x = torch.from_numpy(x.reshape(64, -1)).to(TYPES[kind])
    y = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
    scale = torch.empty((64, 9), device="cuda")
    B.quant_fp8(x.cuda(), y, scale)
    s = host(scale)
    ok = np.isfinite(s)
    bad = np.zeros((64, 9), bool)
    bad[[5, 9, 9], [2, 0, 8]] = True
    assert np.array_equal(~ok, bad)
    want = fp32_codes(x.float().numpy(), s).reshape(64, 9, 128)
    got = host(y).reshape(64, 9, 128)
    assert np.array_equal(got[ok], want[ok])
    amax = np.abs(x.float().numpy().reshape(64, 9, 128)[ok]).max(1)
    assert np.array_equal(s[ok], np.maximum(amax, np.float32(448 * 2.0 ** -126)) / np.float32(448))
