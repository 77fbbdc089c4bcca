"""Shared by the cross entropy's tests: one call of each direction against 64 bits.

Bound, with u = 2^-24: products of 16-bit values are exact in float32, so a logit of K terms is off by at most
ez = K 2^-23 sum|x w| (any order, truncating additions). The exponent's fma rounds once, |z| log2(e) u, and the base-2
exponential by 2 u of its result; a row's N terms meet in at most 64 + N / 4096 + 32 additions one behind another. So
log-sum-exp is off by el = ez + (2 |lse| + N / 4096 + 160) u and a loss by ez more and a float's rounding. A probability is off by
r = ez + el + (4 |z| + 4 |lse| + 8) u of itself, G by |dloss| (p r + 2 u) and its rounding to the operands' format:
half a step of |G| for a 16-bit gradient, half a step of that again for a float32 one (two terms), in f16 also half a
subnormal step, 2^-25 of the largest |dloss| / 2^14. A sum over n terms of G times
the other operand adds n 2^-23 of sum|G| |operand|, and the output its own half step.
"""
import torch

import block_scaled_matrix_amd as bsm
from grouped_util import DT, HALF_STEP, up
from gpu_util import say

U = 2.0 ** -24


def inputs(rows, N, K, ab, seed, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, K, device="cuda", generator=g).to(DT[ab])
    w = (torch.randn(N, K, device="cuda", generator=g) * (spread * max(K, 1) ** -0.5)).to(DT[ab])
    labels = torch.randint(0, N, (rows,), device="cuda", generator=g, dtype=torch.int32)
    labels[torch.rand(rows, device="cuda", generator=g) < 0.15] = -1
    dloss = torch.randn(rows, device="cuda", generator=g) / max(rows, 1)
    return x, w, labels, dloss


def wide(x, extra=0, q=8, fill=float("nan")):
    t = torch.full((x.shape[0], up(x.shape[1], q) + q * extra), fill, dtype=x.dtype, device="cuda")
    t[:, :x.shape[1]] = x
    return t


def reference(x, w, labels):
    x, w = x.double(), w.double()
    K = x.shape[1]
    z = x @ w.T.contiguous()
    ez = K * 2.0 ** -23 * (x.abs() @ w.abs().T.contiguous()).amax(1) if K else torch.zeros(x.shape[0], device="cuda").double()
    lse = torch.logsumexp(z, 1)
    N = w.shape[0]
    has = (labels >= 0) & (labels < N)
    at = torch.where(has, labels, 0).long()
    loss = torch.where(has, lse - z.gather(1, at[:, None])[:, 0], 0.0)
    el = ez + (2 * lse.abs() + N / 4096 + 160) * U
    return z, ez, lse, el, loss, has, at


def check_loss(x, w, labels, ab, stream=None, extra=0):
    (rows, K), N = x.shape, w.shape[0]
    loss, lse = (torch.full((rows + 3,), float("nan"), device="cuda") for _ in range(2))
    xp, wp = wide(x, extra), wide(w, extra)
    work = torch.full((bsm.bsm_gemm_cross_entropy_workspace(rows, N),), 255, dtype=torch.uint8, device="cuda")
    say("cross entropy", rows, N, K, ab, extra)
    bsm.bsm_gemm_cross_entropy(rows, N, K, ab, xp, xp.stride(0), wp, wp.stride(0), labels, loss, lse, work, stream)
    torch.cuda.synchronize()
    z, ez, rl, el, rloss, has, _ = reference(x, w, labels)
    assert torch.isnan(loss[rows:]).all() and torch.isnan(lse[rows:]).all()
    assert ((lse[:rows].double() - rl).abs() <= el).all(), float(((lse[:rows].double() - rl).abs() / el).max())
    tol = torch.where(has, ez + el + 2 * U * rloss.abs(), 0.0)
    assert ((loss[:rows].double() - rloss).abs() <= tol).all(), float(((loss[:rows].double() - rloss).abs() - tol).max())
    return loss[:rows].clone(), lse[:rows].clone()


def check_grad(x, w, labels, dloss, lse, ab, dx_fmt=None, dw_fmt=None, accum=0, piece=0, extra=0, stream=None, want="xw"):
    (rows, K), N = x.shape, w.shape[0]
    dx_fmt, dw_fmt = dx_fmt or ab, dw_fmt or ab
    xp, wp = wide(x, extra), wide(w, extra)
    g = torch.Generator(device="cuda").manual_seed(rows + N + K)
    dw0 = torch.randn(N, up(K, 8) + 8 * extra, device="cuda", generator=g).to(DT[dw_fmt])
    dx = torch.full((rows, up(K, 8) + 8 * extra), 7.0, dtype=DT[dx_fmt], device="cuda")
    dw = dw0.clone() if accum else torch.full_like(dw0, float("nan"))
    if not accum:
        dw[:, K:] = dw0[:, K:]
    work = torch.full((bsm.bsm_gemm_cross_entropy_grad_workspace(rows, N, K, piece),), 255, dtype=torch.uint8, device="cuda")
    say("cross entropy grad", rows, N, K, ab, dx_fmt, dw_fmt, accum, piece, extra, want)
    bsm.bsm_gemm_cross_entropy_grad(rows, N, K, ab, xp, xp.stride(0), wp, wp.stride(0), labels, lse, dloss, piece, work, dx_fmt,
                                    dx if "x" in want else None, dx.stride(0), dw_fmt, dw if "w" in want else None, dw.stride(0),
                                    accum, stream)
    torch.cuda.synchronize()
    z, ez, rl, el, _, has, at = reference(x, w, labels)
    p = torch.exp(z - rl[:, None])
    d = torch.where(has, dloss.double(), 0.0)[:, None]
    G = p.clone()
    G[torch.arange(rows, device="cuda"), at] -= 1.0
    G = torch.where(has[:, None], G * d, 0.0)
    r = (ez + el)[:, None] + (4 * z.abs() + 4 * rl.abs()[:, None] + 8) * U

    def error(fmt):
        e = d.abs() * (p * r + 2 * U) + HALF_STEP[ab] ** (2 if fmt == "f32" else 1) * G.abs() * 1.01
        return torch.where(has[:, None], e + 2.0 ** -25 * float(d.abs().max()) * 2.0 ** -14, 0.0) if ab == "f16" else e

    X, W = x.double(), w.double()

    def compare(got, ref, err, mag, terms, fmt, what):
        tol = err + (terms + 4) * 2.0 ** -23 * mag + HALF_STEP[fmt] * ref.abs() * 1.01 + (2.0 ** -25 if fmt == "f16" else 2.0 ** -126)
        bad = ~((got.double() - ref).abs() <= tol)
        assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), float(((got.double() - ref).abs() / tol).max()))

    if "x" in want:
        compare(dx[:, :K], G @ W, error(dx_fmt) @ W.abs(), G.abs() @ W.abs(), 2 * N + 64, dx_fmt, "dX")
        assert (dx[:, K:] == 7.0).all()
    if "w" in want:
        ref, mag = G.T.contiguous() @ X, G.abs().T.contiguous() @ X.abs()
        if accum:
            ref, mag = ref + dw0[:, :K].double(), mag + dw0[:, :K].double().abs()
        compare(dw[:, :K], ref, error(dw_fmt).T.contiguous() @ X.abs(), mag, 2 * rows, dw_fmt, "dW")
        assert torch.equal(dw[:, K:], dw0[:, K:])
    return dx, dw
