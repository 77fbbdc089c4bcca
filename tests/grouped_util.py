"""Shared by the tests of products over groups of rows: operands in padded rows, and the bound of one product.

Bound: the products of two 16-bit values are exact in float32 (at most 22 significand bits; values here stay
far from its range's ends), so |D - ref| comes from the float32 sum and the output's own rounding. A sum of K
terms in any order, each addition off by at most 2^-23 of its result (the matrix instructions may truncate),
is off by at most K 2^-23 sum|ab|; the output rounds once by at most half a step: 2^-8 (bf16), 2^-11 (f16),
2^-24 (f32) of the value, or 2^-25, half a subnormal step, of f16.
"""
import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


def up(n, to):
    return -(-n // to) * to


def padded(x, to=8, extra=0, fill=float("nan")):
    """x in rows of its last axis rounded up to a multiple of `to`, plus `extra`; the padding holds `fill`."""
    ld = up(x.shape[-1], to) + extra
    out = torch.full((*x.shape[:-1], ld), fill, dtype=x.dtype)
    out[..., :x.shape[-1]] = x
    return out


def tolerance(ref, mag, terms, d):
    """The bound above, per element: ref the 64-bit result, mag the 64-bit sum of |a b| (+ |D|)."""
    return (terms + 2) * 2.0 ** -23 * mag + HALF_STEP[d] * ref.abs() * (1 + 2.0 ** -7) + (2.0 ** -25 if d == "f16" else 0.0)


def check(got, ref, mag, terms, d, what=""):
    got = got.double().cpu()
    tol = tolerance(ref, mag, terms, d)
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(),
                           float(((got - ref).abs() / tol.clamp_min(1e-300)).nan_to_num(1e9).max()))


def silu_affine(x, scale, bias):
    return x / (1 + torch.exp(-x)) * scale + bias


def offsets_of(sizes, first=0):
    return [first] + list(first + np.cumsum(sizes).astype(int))
