"""Inputs, oracles and tolerances of the tests of attention over latent rows."""

import numpy as np
import torch

from oracle import attention as oa

SCALE = 192 ** -0.5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def rand(rng, shape, t, size=1.0):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * np.float32(size)).to(TYPES[t])


def f64(t):
    return t.cpu().double().numpy()


def score_error(terms, lse):
    """Relative error of a weight, from its score's: products are exact in fp32, a score's 576 of them go through
    18 dependent additions of the matrix core, each of which adds 32 within itself (50 roundings of half a step,
    2^-24, of at most the sum of |products|); scale, maximum, difference, exponential and the sums over tokens, lanes,
    waves and chunks are at most 100 more roundings of a size of at most 1 + |score| each."""
    return 2.0 ** -24 * (50 * terms + 100 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0)) + terms / 16))


def check(out, lse, q, kv, rows, scale=SCALE):
    """out and lse against the definition in 64 bits.  out may be off by the rounding of its value (u, half a step of
    its type), of the weights (u of every term, or fp16's smallest half step), and by the scores' errors in weights
    and in their sum."""
    t = out.dtype
    u = torch.finfo(t).eps / 2
    tiny = 2.0 ** -25 if t == torch.float16 else 0.0       # fp16 weights below 2^-14
    want, want_lse, size, terms = oa.attention(f64(q), f64(kv), rows, scale)
    rel = score_error(terms, want_lse)[:, :, None]
    got = f64(out)
    n_abs = np.stack([np.abs(f64(kv)[r][:, :oa.VALUES]).sum(0) if len(r) else np.zeros(oa.VALUES) for r in rows])[:, None, :]
    tol = u * np.abs(want) + (u + 2 * rel) * size * (1 + u) + tiny * (n_abs + 1) + 1e-30
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%d values off, worst %g of its tolerance, first at %s" % (
        bad.sum(), np.nanmax(np.abs(got - want) / tol), np.argwhere(bad)[0])
    if lse is not None:
        g = f64(lse)
        none = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(g), none)
        d = np.abs(np.where(none, 0, g) - np.where(none, 0, want_lse))
        assert (d <= np.where(none, 0, rel[:, :, 0] + 1e-30)).all(), (d / rel[:, :, 0]).max()
