"""Every kernel that echo_matmul_fp8 can take, by name (echo_matmul_fp8_form), against a float64 product:
random operands of all codes, wide rows, scales with blocks as rows, results at even and odd addresses,
NaN, and K beyond what a wave holds of the weight scales at once.

Tolerance, derived as in test_gpu_blockfp8.py: (128 + nb + 11) * 2 u times the sum of the terms'
magnitudes T for sums in fp32 (u = 2^-24, nb blocks); for 16-bit results of the FP8 matrix core (the
forms "split" and "tile") 7 * 2^-13 of the largest of eight neighbouring products, summed; half a step of
the result's type, and 2^-25 below fp16's normal numbers."""

import numpy as np
import pytest
import torch

from dsa_indexer_top_amd import binding as B
from gpu_util import announce, dev
from oracle.fp8 import E4M3FN_TABLE
from test_gpu_blockfp8 import HALF_STEP, TYPES, U

pytestmark = pytest.mark.gpu
CODE = {"bf16": B.BF16, "fp16": B.FP16, "fp32": B.FP32}

# form, m, n, k, types: sizes that end inside a tile, a block and a 16-byte piece of K, some blocks
# more than the form keeps in LDS
FORMS = [
    ("few 16x16", 9, 301, 300, TYPES),
    ("few 16x16", 100, 120, 1301, TYPES),
    ("few 32x16", 30, 2101, 300, TYPES),
    ("few 32x16", 60, 1999, 300, TYPES),
    ("few 32x32", 301, 499, 1170, TYPES),
    ("split 64x64", 601, 531, 1301, TYPES),
    ("tile 64x64", 601, 531, 630, TYPES),
    ("tile 64x128", 1090, 1101, 530, TYPES),
    ("tile 128x128, 3 stages", 1701, 2051, 530, ("bf16", "fp16")),
    ("tile 128x128", 2201, 2301, 260, ("bf16", "fp16")),
    ("tile 128x128", 1701, 2051, 260, ("fp32",)),
    ("tile 256x256", 2901, 2945, 260, ("bf16", "fp16")),
]
EACH = [pytest.param(f, m, n, k, t, id="%s-%dx%dx%d-%s" % (f.replace(" ", "_"), m, n, k, t))
        for f, m, n, k, types in FORMS for t in types]


def operands(rng, m, n, k, kind):
    """Codes in wider rows (NaN codes beside them) and scales with blocks as rows, on the device."""
    finite = np.flatnonzero(np.isfinite(E4M3FN_TABLE)).astype(np.uint8)
    nb = -(-k // 128)

    def codes(rows, before, after):
        ld = before + -(-k // 16) * 16 + after
        t = np.full((rows, ld), 0x7F, np.uint8)
        t[:, before:before + k] = rng.choice(finite, (rows, k))
        return dev(t)[:, before:before + k]

    scale = lambda r, x=1.0: dev((x * np.exp(rng.standard_normal((nb, r)))).astype(np.float32)).t()
    a, b = codes(m, 16, 32), codes(n, 48, 0)
    # fp16 keeps the sums below 65504
    return a, scale(m, 1e-4 / max(1.0, k / 128) if kind == "fp16" else 1.0), b, scale(-(-n // 128))


VALUES = torch.from_numpy(E4M3FN_TABLE.astype(np.float64))


def reference(a, sa, b, sb, exact):
    """(product, what a sum may be off) in float64."""
    k, n = a.shape[1], b.shape[0]
    spread = lambda s: s.double().repeat_interleave(128, 1)[:, :k]
    values = VALUES.to(a.device)
    av = values[a.long()] * spread(sa)
    bv = values[b.long()] * spread(sb).repeat_interleave(128, 0)[:n]
    nan = [v.isnan() for v in (av, bv)]
    rows, cols = nan[0].any(1), nan[1].any(1)
    av, bv = av.masked_fill(nan[0], 0.0), bv.masked_fill(nan[1], 0.0)
    want = av @ bv.t().contiguous()
    ab, bb = av.abs(), bv.abs()
    tol = (128 + -(-k // 128) + 11) * 2 * U * (ab @ bb.t().contiguous())
    if not exact:
        x, y = ab.float(), bb.float()                # rounded up below: the bound is a sum of positive terms
        most, one, total = (torch.empty(want.shape, device=a.device) for _ in range(3))
        total.zero_()
        for p in range(0, k, 8):
            torch.outer(x[:, p], y[:, p], out=most)
            for q in range(p + 1, min(p + 8, k)):
                torch.outer(x[:, q], y[:, q], out=one)
                torch.maximum(most, one, out=most)
            total += most
        tol += 7 * 2.0 ** -13 * 1.001 * total.double()
    want[rows] = float("nan")
    want[:, cols] = float("nan")
    return want, tol


def check(c, ops, m, n, k, kind, exact):
    want, tol = reference(*ops, exact)
    got = c.double()
    floor = 2.0 ** -25 if kind == "fp16" else 0.0
    ok = (got - want).abs() <= tol + HALF_STEP[kind] * (want.abs() + tol) + floor
    assert bool((ok | (got.isnan() & want.isnan())).all())


def product(form, m, n, k, kind, at, width, seed, bad=()):
    """One product into columns [at, at + n) of rows of `width`, checked; nothing beside it is written."""
    announce("product form", form, m, n, k, kind, at, width)
    assert B.matmul_fp8_form(m, n, k, CODE[kind]) == form
    ops = operands(np.random.default_rng(seed), m, n, k, kind)
    for side, row, col in bad:
        ops[2 * side][row, col] = 0x7F
    c = torch.full((m, width), -77.0, dtype=TYPES[kind], device="cuda")
    B.matmul_fp8(*ops, c[:, at:at + n])
    check(c[:, at:at + n], ops, m, n, k, kind, form.startswith("few") or kind == "fp32")
    assert bool((c[:, :at] == -77.0).all()) and bool((c[:, at + n:] == -77.0).all())


@pytest.mark.parametrize("form,m,n,k,kind", EACH)
def test_forms_full(form, m, n, k, kind):
    """Rows of an odd width that start at an odd address: every other one between two dwords."""
    product(form, m, n, k, kind, 1, n + 4 - n % 2, m + n)


@pytest.mark.parametrize("form,m,n,k,kind", EACH)
def test_forms_with_nan_full(form, m, n, k, kind):
    """Even rows; a NaN in one row of each operand, in the last block and the first, stays there."""
    product(form, m, n, k, kind, 0, n + 1 + n % 2, m + k, [(0, m - 1, k - 1), (1, n - 1, 0)])


# 64 blocks' weight scales are in a wave's registers at a time: 8192 of K in the tiles, 4 x 8192 where four
# waves share the blocks
@pytest.mark.parametrize("form,m,n,k,kind", [
    ("tile 64x128", 1090, 1100, 8500, "bf16"), ("tile 64x128", 1090, 1100, 8300, "fp32"),
    ("split 64x64", 513, 530, 33100, "fp16"), ("split 64x64", 513, 530, 33100, "fp32"),
    ("tile 128x128", 1701, 2051, 16500, "fp32"), ("tile 256x256", 2901, 2945, 8321, "bf16")])
def test_long_sums_full(form, m, n, k, kind):
    product(form, m, n, k, kind, 0, n, k)
