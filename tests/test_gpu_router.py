"""GPU parity: a router's counts, offsets, balance loss and its gradient, against 64 bits.

Bound: u = 2^-24, half a step of float32. A probability is exp(l - max) / sum: the difference is off by |l - max| u, the
exponential by 4 u more, the sum of E terms by at most E u of itself, reciprocal and product by 3 u: in all
r = (2 |l - max| + 2 E + 16) u of it, where the second |l - max| and E come with the denominator's terms. The loss is a
sum of products of positive terms: r, 64 u for the float32 part of the sum, and its own rounding. The gradient is
c p (f - dot): f is off by 3 u f, dot by (r + E u) dot, p by r, the products by 4 u; then the output's half step.
"""
import pytest
import torch

import block_scaled_matrix_amd as bsm
from grouped_util import DT, HALF_STEP, up
from gpu_util import say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def reference(logits, ids, E, k, scale, g):
    """loss, counts with the rows kept, offsets, gradient, and the error bounds of loss and gradient (before rounding)."""
    x = logits.double()
    ok = (ids >= 0) & (ids < E)
    keep = ok.any(1)
    counts = torch.bincount(ids[ok].long(), minlength=E)
    n = int(keep.sum())
    top = x.amax(1, keepdim=True)
    e = torch.where(x == -torch.inf, 0.0, torch.exp(x - top))
    s = e.sum(1, keepdim=True)
    p = torch.where(s == 0, 0.0, e / s)
    p = torch.where(keep[:, None], p, 0.0)
    d = torch.where(torch.isfinite(x) & torch.isfinite(top), top - x, 0.0)
    r = (2 * d.amax(1, keepdim=True) + 2 * E + 16) * U if x.numel() else d
    f = counts.double() / max(k * n, 1)
    loss = scale * E * (f * p.sum(0)).sum() / max(n, 1)
    dot = (p * f).sum(1, keepdim=True)
    c = g * scale * E / max(n, 1)
    grad = c * p * (f - dot)
    bound = abs(c) * p * ((r + 4 * U) * (f + dot) + 3 * U * f + (r + E * U) * dot)
    ends = torch.cat((torch.zeros(1, dtype=torch.long), counts.cumsum(0)))
    loss_bound = (float(r.max()) if x.numel() else 0.0) * abs(float(loss)) + 66 * U * abs(float(loss))
    return loss, torch.cat((counts, torch.tensor([n]))), ends, grad, loss_bound, bound


def run(rows, E, k, fmt="f32", d_fmt=None, scale=1.0, g=0.7, accum=0, seed=0, logits=None, ids=None, extra=0, pad=0.1, offset=0,
        stream=None, dloss=True):
    gen = torch.Generator().manual_seed(seed)
    d_fmt = d_fmt or fmt
    if logits is None:
        logits = (torch.randn(rows, E, generator=gen) * 2).to(DT[fmt])
    if ids is None:
        ids = torch.randint(0, E, (rows, k), generator=gen, dtype=torch.int32)
        ids[rows - int(rows * pad):] = -1
    ldl, ldd = E + extra, E + (2 * extra)
    big = torch.full((rows * ldl + 8,), float("nan"), dtype=DT[fmt], device="cuda")
    lv = big[offset:offset + rows * ldl].view(rows, ldl)[:, :E]
    lv.copy_(logits)
    D0 = torch.randn(rows, ldd, generator=gen).to(DT[d_fmt])
    D = D0.cuda()
    counts, offsets = (torch.full((E + 1,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    loss = torch.full((1,), float("nan"), device="cuda")
    idd = ids.cuda()
    work = torch.full((bsm.bsm_router_balance_workspace(rows, E),), 255, dtype=torch.uint8, device="cuda")
    say("balance", rows, E, k, fmt, d_fmt, accum, extra, offset)
    bsm.bsm_router_balance(rows, E, k, fmt, lv, ldl, idd, scale, counts, offsets, loss, work, stream)
    gl = torch.tensor([g], device="cuda") if dloss else None
    bsm.bsm_router_balance_grad(rows, E, k, fmt, lv, ldl, idd, counts, scale, gl, d_fmt, D, ldd, accum, stream)
    torch.cuda.synchronize()
    rl, rc, ro, rd, lb, db = reference(logits, ids, E, k, scale, g if dloss else 1.0)
    assert torch.equal(counts.cpu().long(), rc) and torch.equal(offsets.cpu().long(), ro)
    assert abs(float(loss) - float(rl)) <= lb + U * abs(float(rl)), (float(loss), float(rl), lb)
    got = D.cpu()
    ref = rd + (D0[:, :E].double() if accum else 0)
    tol = db + (2 * U * (rd.abs() + D0[:, :E].double().abs()) if accum else 0) + HALF_STEP[d_fmt] * ref.abs() * (1 + 2.0 ** -7) + \
        (2.0 ** -25 if d_fmt == "f16" else 2.0 ** -126)
    err = (got[:, :E].double() - ref).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert torch.equal(got[:, E:], D0[:, E:]), "columns past E were written"
    return loss, counts, offsets, D


@pytest.mark.parametrize("E", [1, 2, 3, 8, 16, 17, 32, 33, 60, 64, 65, 128, 130, 255, 256, 257, 512, 513, 1000, 1024])
@pytest.mark.parametrize("rows", [1, 5, 64, 333])
def test_experts_and_rows(rows, E):
    run(rows, E, min(E, 4), seed=rows + E)


@pytest.mark.parametrize("rows,E,k", [(5000, 64, 6), (20011, 128, 8), (70001, 8, 2), (9999, 257, 3), (4096, 1024, 1)])
@pytest.mark.parametrize("fmt,d_fmt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16")])
def test_many_rows(rows, E, k, fmt, d_fmt):
    run(rows, E, k, fmt, d_fmt, seed=E)


@pytest.mark.parametrize("fmt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E", [7, 30, 62, 100, 250, 500, 1001])
def test_every_width(E, fmt):
    """Few rows, which one workgroup takes, and more of them."""
    run(9, E, 2, fmt, seed=E)
    run(40000 // E + 900, E, 2, fmt, seed=E)


@pytest.mark.parametrize("k", [1, 3, 16, 70])
def test_ids_a_row(k):
    run(100, 12, k, seed=k)


@pytest.mark.parametrize("fmt", ["f32", "bf16", "f16"])
def test_strides_and_alignment(fmt):
    for E, extra, offset in ((64, 8, 0), (64, 3, 0), (64, 0, 1), (61, 0, 0), (130, 1, 3)):
        run(77, E, 4, fmt, extra=extra, offset=offset)


def test_accumulates_and_scales():
    for fmt, d in (("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")):
        run(300, 40, 4, fmt, d, scale=0.01, g=-3.0, accum=1)
    run(300, 40, 4, dloss=False)


def test_no_rows_and_no_row_kept():
    run(0, 64, 4)
    run(9, 64, 4, ids=torch.full((9, 4), -1, dtype=torch.int32))
    run(20000, 64, 4, ids=torch.full((20000, 4), 64, dtype=torch.int32))


def test_ids_that_are_no_experts():
    g = torch.Generator().manual_seed(5)
    ids = torch.randint(-40, 80, (500, 3), generator=g, dtype=torch.int32)
    ids[7] = torch.tensor([2 ** 31 - 1, -2 ** 31, -1], dtype=torch.int32)
    ids[8] = torch.tensor([3, 3, 3], dtype=torch.int32)      # the same expert three times
    run(500, 20, 3, ids=ids)


def test_masked_logits():
    """Logits of -infinity and of the type's lowest value; a kept row with nothing left; NaN in a row that is not kept."""
    x = torch.randn(64, 24)
    x[:, 5] = -torch.inf
    x[3] = -torch.inf
    x[4] = torch.finfo(torch.float32).min
    x[5, :23] = torch.finfo(torch.float32).min
    ids = torch.randint(0, 24, (64, 2), dtype=torch.int32)
    ids[9] = -1
    run(64, 24, 2, logits=torch.where(torch.arange(64)[:, None] == 9, 0.0, x), ids=ids)
    y = x.clone()
    y[9] = float("nan")
    y[10:12] = x[10:12]
    a = run(64, 24, 2, logits=torch.where(torch.arange(64)[:, None] == 9, 0.0, y), ids=ids)
    E = 24
    lv = y.cuda()
    outs = [torch.empty(E + 1, dtype=torch.int32, device="cuda") for _ in range(2)] + [torch.empty(1, device="cuda")]
    bsm.bsm_router_balance(64, E, 2, "f32", lv, E, ids.cuda(), 1.0, *outs, None)
    d = torch.empty(64, E, device="cuda")
    bsm.bsm_router_balance_grad(64, E, 2, "f32", lv, E, ids.cuda(), outs[0], 1.0, None, "f32", d, E)
    assert torch.equal(outs[2], a[0]) and not d[9].any() and torch.isfinite(d).all()


def test_nan_and_infinity_show():
    for bad in (float("nan"), float("inf")):
        x = torch.randn(40, 10)
        x[6, 3] = bad
        ids = torch.zeros(40, 1, dtype=torch.int32).cuda()
        outs = [torch.empty(11, dtype=torch.int32, device="cuda") for _ in range(2)] + [torch.empty(1, device="cuda")]
        bsm.bsm_router_balance(40, 10, 1, "f32", x.cuda(), 10, ids, 1.0, *outs, None)
        d = torch.empty(40, 10, device="cuda")
        bsm.bsm_router_balance_grad(40, 10, 1, "f32", x.cuda(), 10, ids, outs[0], 1.0, None, "f32", d, 10)
        assert torch.isnan(outs[2]).all() and torch.isnan(d[6]).all() and torch.isfinite(d[7:]).all() and torch.isfinite(d[:6]).all()


def test_same_bits_on_every_call():
    a = run(30000, 100, 4, "bf16", seed=3)
    for _ in range(3):
        b = run(30000, 100, 4, "bf16", seed=3)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_gradient_against_differences():
    """d loss / d logit by central differences of the 64-bit loss."""
    rows, E, k = 6, 5, 2
    g = torch.Generator().manual_seed(1)
    x = torch.randn(rows, E, generator=g)
    ids = torch.randint(0, E, (rows, k), generator=g, dtype=torch.int32)
    D = run(rows, E, k, logits=x, ids=ids, g=1.0)[3].cpu()
    h = 1e-5
    for t in range(rows):
        for e in range(E):
            v = []
            for s in (h, -h):
                y = x.double().clone()
                y[t, e] += s
                v.append(float(reference(y, ids, E, k, 1.0, 1.0)[0]))
            assert abs((v[0] - v[1]) / (2 * h) - float(D[t, e])) < 1e-6      # (h^2 and 1e-16 / h, loss near 1)


def test_rows_past_32_bits():
    """Logits whose last rows lie past 2^31 elements."""
    rows, E, ld = 70001, 8, 31000
    x = torch.zeros(rows * ld, dtype=torch.bfloat16, device="cuda")
    v = x.view(rows, ld)
    v[-1, :8] = torch.arange(8, device="cuda").bfloat16()
    ids = torch.full((rows, 1), -1, dtype=torch.int32, device="cuda")
    ids[-1] = 3
    outs = [torch.empty(9, dtype=torch.int32, device="cuda") for _ in range(2)] + [torch.empty(1, device="cuda")]
    work = torch.empty(bsm.bsm_router_balance_workspace(rows, E), dtype=torch.uint8, device="cuda")
    say("balance past 2^31")
    bsm.bsm_router_balance(rows, E, 1, "bf16", x, ld, ids, 1.0, *outs, work)
    want = 8 * torch.softmax(torch.arange(8).double(), 0)[3]
    assert abs(float(outs[2]) - float(want)) < 60 * U and outs[0].tolist() == [0, 0, 0, 1, 0, 0, 0, 0, 1]
