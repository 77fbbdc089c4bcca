"""GPU parity: cross entropy of a projection onto a vocabulary and its gradients, against 64 bits (bounds in xent_util)."""
import pytest
import torch

import block_scaled_matrix_amd as bsm
from grouped_util import DT, up
from gpu_util import say
from xent_util import check_grad, check_loss, inputs, reference, wide

pytestmark = pytest.mark.gpu


def both(rows, N, K, ab="bf16", seed=0, extra=0, **kw):
    x, w, labels, dloss = inputs(rows, N, K, ab, seed + rows + N + K)
    _, lse = check_loss(x, w, labels, ab, extra=extra)
    return check_grad(x, w, labels, dloss, lse, ab, extra=extra, **kw)


@pytest.mark.parametrize("ab", ["bf16", "f16"])
@pytest.mark.parametrize("rows,N,K", [(1, 1, 1), (1, 2, 8), (2, 15, 7), (3, 16, 64), (5, 17, 65), (16, 63, 33), (17, 64, 136), (31, 65, 520),
                                      (33, 129, 40), (63, 250, 72), (64, 1000, 100), (65, 1000, 8), (130, 257, 264), (200, 4099, 1000),
                                      (300, 128, 24)])
def test_sizes(rows, N, K, ab):
    both(rows, N, K, ab)


@pytest.mark.parametrize("ab", ["bf16", "f16"])
@pytest.mark.parametrize("rows,N,K", [
    (4, 33000, 40), (64, 20001, 64), (700, 9001, 48),     # whole vocabularies: the loss on mid tiles of 32, 64 and 128 rows
    (4096, 4100, 40), (3900, 4500, 72),                   # logits on the large tile
    (4096, 300, 4096), (200, 4096, 4096), (2100, 5000, 2056),   # and the gradients on it, dX in one part and in several
    (1, 5000, 4096)])
def test_tiles(rows, N, K, ab):
    both(rows, N, K, ab, extra=rows % 2)


@pytest.mark.parametrize("ab", ["bf16", "f16"])
@pytest.mark.parametrize("rows,N,K", [(3, 700, 40), (130, 700, 200), (40, 3000, 64), (4096, 600, 4096)])
def test_formats_accumulation_and_pieces(rows, N, K, ab):
    for dx, dw, accum, piece in ((ab, "f32", 1, 256), ("f32", ab, 1, 0), ("f32", "f32", 0, 300), (ab, ab, 0, 1)):
        both(rows, N, K, ab, dx_fmt=dx, dw_fmt=dw, accum=accum, piece=piece, extra=1)


@pytest.mark.parametrize("ab", ["bf16", "f16"])
def test_float32_gradients_on_every_tile(ab):
    """G in two terms, made on 32-row and on large tiles; a float32 weight gradient on large tiles, added to and not."""
    both(24, 33000, 40, ab, dx_fmt="f32", dw_fmt="f32")
    both(4096, 4100, 40, ab, dx_fmt="f32", dw_fmt="f32")
    for accum in (0, 1):
        both(1700, 4096, 4096, ab, want="w", dw_fmt="f32", accum=accum)


def test_one_gradient_alone():
    """Of few rows, whose gradients otherwise share a launch, and of many."""
    for ab, f in (("bf16", "bf16"), ("f16", "f32")):
        both(300, 5000, 264, ab, want="x", dx_fmt=f, dw_fmt=f)
        both(300, 5000, 264, ab, want="w", dx_fmt=f, dw_fmt=f)
        both(4096, 520, 4096, ab, want="x", dx_fmt=f, dw_fmt=f)
        both(1700, 4096, 4096, ab, want="w", dx_fmt=f, dw_fmt=f)
    both(130, 700, 72, want="x")
    both(130, 700, 72, want="w", piece=256)
    both(130, 700, 72, want="")


def test_no_rows_and_no_width():
    x, w, labels, dloss = inputs(0, 40, 16, "bf16", 1)
    bsm.bsm_gemm_cross_entropy(0, 40, 16, "bf16", x, 16, w, 16, labels, dloss, dloss, None)
    for accum in (0, 1):
        dw = torch.full((40, 16), 3.0, dtype=torch.bfloat16, device="cuda")
        bsm.bsm_gemm_cross_entropy_grad(0, 40, 16, "bf16", None, 16, None, 16, None, None, None, 0, None, "bf16", None, 16, "bf16", dw, 16, accum)
        assert (dw == 3.0 * accum).all()
    loss, lse = torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    work = torch.empty(bsm.bsm_gemm_cross_entropy_workspace(5, 40), dtype=torch.uint8, device="cuda")
    labels = torch.tensor([0, 39, 40, -1, 7], dtype=torch.int32, device="cuda")
    bsm.bsm_gemm_cross_entropy(5, 40, 0, "bf16", None, 0, None, 0, labels, loss, lse, work)
    want = torch.log(torch.tensor(40.0))
    assert (lse.cpu() - want).abs().max() < 1e-6 and (loss.cpu() - want * torch.tensor([1.0, 1, 0, 0, 1])).abs().max() < 1e-6


@pytest.mark.parametrize("accum", [0, 1])
@pytest.mark.parametrize("dw_fmt", ["f16", "f32"])
def test_no_rows_in_f16(dw_fmt, accum):
    """An empty micro-batch: no weights, so no power of two for them, and no workspace."""
    N, K = 300, 200
    dw = torch.full((N + 1, K), 3.0, dtype=DT[dw_fmt], device="cuda")
    say("cross entropy grad of no rows", dw_fmt, accum)
    bsm.bsm_gemm_cross_entropy_grad(0, N, K, "f16", None, K, None, K, None, None, None, 0, None, "f16", None, K, dw_fmt, dw, K, accum)
    assert (dw[:N] == 3.0 * accum).all() and (dw[N] == 3.0).all()


@pytest.mark.parametrize("rows,N", [(40, 300), (500, 20000)])
def test_rows_without_a_label(rows, N):
    """No label at all; labels far outside; such a row's NaN stays in its row of logits."""
    x, w, labels, dloss = inputs(rows, N, 64, "bf16", 2)
    for bad in (-1, N, 2 ** 31 - 1, -2 ** 31):
        none = torch.full_like(labels, bad)
        loss, lse = check_loss(x, w, none, "bf16")
        assert not loss.any()
        dx, dw = check_grad(x, w, none, dloss, lse, "bf16")
        assert not dx[:, :64].any() and not dw[:, :64].any()
    # a padding row of NaN with a NaN weight: its G is 0, but X enters dW as 0 * NaN, so its X must be finite for dW
    labels[3] = -1
    dl = dloss.clone()
    dl[3] = float("nan")
    y = x.clone()
    y[3] = float("nan")
    _, lse = check_loss(x, w, labels, "bf16")
    loss2, lse2 = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    work = torch.empty(bsm.bsm_gemm_cross_entropy_workspace(rows, N), dtype=torch.uint8, device="cuda")
    bsm.bsm_gemm_cross_entropy(rows, N, 64, "bf16", y, 64, w, 64, labels, loss2, lse2, work)
    keep = torch.arange(rows, device="cuda") != 3
    assert torch.equal(lse2[keep], lse[keep]) and torch.isnan(lse2[3]) and loss2[3] == 0
    dx = torch.empty(rows, 64, dtype=torch.bfloat16, device="cuda")
    ref, _ = check_grad(x, w, labels, dloss, lse, "bf16")
    gw = torch.empty(bsm.bsm_gemm_cross_entropy_grad_workspace(rows, N, 64, 0), dtype=torch.uint8, device="cuda")
    bsm.bsm_gemm_cross_entropy_grad(rows, N, 64, "bf16", y, 64, w, 64, labels, lse2, dl, 0, gw, "bf16", dx, 64, "bf16", None, 64)
    assert torch.equal(dx, ref[:, :64]) and not dx[3].any()


@pytest.mark.parametrize("rows,N", [(20, 100), (20, 30000), (700, 9000)])
def test_large_and_infinite_logits(rows, N):
    """Logits far apart (probabilities that underflow), equal ones, and infinities of the operands."""
    x, w, labels, dloss = inputs(rows, N, 16, "bf16", 5, spread=120.0)
    loss, lse = check_loss(x, w, labels, "bf16")
    check_grad(x, w, labels, dloss, lse, "bf16")
    z = torch.zeros_like(w)
    _, lse = check_loss(x, z, labels, "bf16")
    check_grad(x, z, labels, dloss, lse, "bf16")
    # a column of -infinity for every row: probability 0
    x2, w2 = x.abs() + 0.5, w.clone()
    w2[7] = -float("inf")
    lab = torch.where(labels == 7, 8, labels)
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    work = torch.empty(bsm.bsm_gemm_cross_entropy_workspace(rows, N), dtype=torch.uint8, device="cuda")
    bsm.bsm_gemm_cross_entropy(rows, N, 16, "bf16", x2, 16, w2, 16, lab, loss, lse, work)
    keep = torch.cat((w2[:7], w2[8:]))
    want = torch.logsumexp(x2.double() @ keep.double().T.contiguous(), 1)
    assert ((lse.double() - want).abs() <= 1e-5 * want.abs()).all()      # (16 products of up to a few thousand)
    # NaN in one row of X, and +infinity in another, show in their rows alone
    x3 = x.clone()
    x3[2, 3] = float("nan")
    w3 = w.abs() + 0.01
    x3[5] = x3[5].abs()
    x3[5, 1] = float("inf")
    bsm.bsm_gemm_cross_entropy(rows, N, 16, "bf16", x3, 16, w3, 16, labels, loss, lse, work)
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad[2] = bad[5] = True
    assert torch.isnan(lse[bad]).all() and torch.isfinite(lse[~bad]).all()


@pytest.mark.parametrize("rows,N", [(20, 100), (20, 30000), (700, 9000)])
def test_logits_at_the_end_of_the_range(rows, N):
    """Beyond 2^127.5 or so they count as infinite: positive ones make lse NaN, negative ones add nothing."""
    x = torch.zeros(rows, 8, device="cuda").bfloat16()
    w = torch.zeros(N, 8, device="cuda").bfloat16()
    x[:, 0], x[:, 1] = 2.0 ** 100, 1.0
    w[1:, 0], w[0, 1] = -1.875 * 2.0 ** 27, 3.0        # z(., 0) = 3, all others -1.875 * 2^127
    x[1, 0] = -(2.0 ** 100)                            # this row's others: +1.875 * 2^127
    x[2, 0] = 2.0 ** 99                                # and half: in range, far below
    x[4, 1] = 0.0
    w[0, 0] = 0.0
    labels = torch.zeros(rows, dtype=torch.int32, device="cuda")
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    work = torch.empty(bsm.bsm_gemm_cross_entropy_workspace(rows, N), dtype=torch.uint8, device="cuda")
    say("logits at the end of the range", rows, N)
    bsm.bsm_gemm_cross_entropy(rows, N, 8, "bf16", x, 8, w, 8, labels, loss, lse, work)
    want = torch.full((rows,), 3.0, device="cuda")
    want[1], want[4] = float("nan"), 0.0
    assert torch.isnan(lse[1]) and torch.isnan(loss[1])
    keep = torch.arange(rows, device="cuda") != 1
    assert (lse[keep] - want[keep]).abs().max() < 1e-6 and loss[keep].abs().max() < 1e-6
    w[0, 0] = w[1, 0]                                  # nothing but such ones
    w[0, 1] = 0.0
    bsm.bsm_gemm_cross_entropy(rows, N, 8, "bf16", x, 8, w, 8, labels, loss, lse, work)
    assert (lse[[0, 3, 5]] == -float("inf")).all()


def test_many_rows_few_columns():
    """dX of 2^28 values and more: the sum of its parts takes several launches."""
    rows, K = 66001, 4096
    x, w, labels, dloss = inputs(rows, 3, K, "bf16", 6)
    lse = torch.zeros(rows, device="cuda")             # (not the loss's: G is what it makes of these)
    dx = torch.full((rows, K), 7.0, device="cuda")
    work = torch.empty(bsm.bsm_gemm_cross_entropy_grad_workspace(rows, 3, K, 0), dtype=torch.uint8, device="cuda")
    say("cross entropy grad", rows, 3, K)
    bsm.bsm_gemm_cross_entropy_grad(rows, 3, K, "bf16", x, K, w, K, labels, lse, dloss, 0, work, "f32", dx, K, "f32", None, K)
    for r in (slice(0, 300), slice(65300, 65700), slice(rows - 300, rows)):
        z = x[r].double() @ w.double().T.contiguous()
        has = (labels[r] >= 0)[:, None]
        G = torch.exp(z)
        G[torch.arange(z.shape[0], device="cuda"), labels[r].clamp(0).long()] -= 1.0
        G = torch.where(has, G * dloss[r].double()[:, None], 0.0)
        ref, mag = G @ w.double(), (torch.exp(z) + 1) * dloss[r].double().abs()[:, None]
        # z off by K 2^-23 sum |x w|, G by that, 2^-18 for its two terms and a few float32 steps; three terms of dX
        ez = (K * 2.0 ** -23 * (x[r].double().abs() @ w.double().abs().T.contiguous()) + 2.0 ** -18 + 2.0 ** -20).amax(1, keepdim=True)
        assert ((dx[r].double() - ref).abs() <= (mag * (ez + 2.0 ** -20)) @ w.double().abs()).all()


def test_f16_weights_of_every_size():
    """The weights' power of two: tiny, huge, zero and one row far above the rest."""
    x, w, labels, _ = inputs(90, 500, 40, "f16", 9)
    _, lse = check_loss(x, w, labels, "f16")
    for d in (torch.full((90,), 2.0 ** -40), torch.full((90,), 1e30), torch.zeros(90), torch.rand(90) * 1e-3, torch.full((90,), -1.0)):
        dx_fmt = dw_fmt = "f32"
        check_grad(x, w, labels, d.cuda(), lse, "f16", dx_fmt, dw_fmt)
    d = torch.full((90,), 1e-6)
    d[4] = 1.0
    check_grad(x, w, labels, d.cuda(), lse, "f16")


@pytest.mark.parametrize("rows,N,K", [(24, 30011, 256), (1500, 3000, 200), (4096, 4096, 64)])
def test_same_bits_on_every_call(rows, N, K):
    x, w, labels, dloss = inputs(rows, N, K, "bf16", 4)
    a = check_loss(x, w, labels, "bf16")
    g = check_grad(x, w, labels, dloss, a[1], "bf16")
    for _ in range(3):
        b = check_loss(x, w, labels, "bf16")
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    h = check_grad(x, w, labels, dloss, a[1], "bf16")
    assert torch.equal(g[0], h[0]) and torch.equal(g[1], h[1])


def test_gradient_against_differences():
    """d (sum of weighted losses) / dx and / dw by central differences of the 64-bit loss."""
    x, w, labels, dloss = inputs(5, 9, 6, "bf16", 3)
    _, lse = check_loss(x, w, labels, "bf16")
    dx, dw = check_grad(x, w, labels, dloss, lse, "bf16", "f32", "f32")
    f = lambda a, b: float((torch.where((labels >= 0) & (labels < 9), torch.logsumexp(a @ b.T, 1) -
                                        (a @ b.T).gather(1, labels.clamp(0, 8).long()[:, None])[:, 0], 0.0) * dloss.double()).sum())
    X, W, h = x.double(), w.double(), 1e-5
    for t, g, n in ((X, dx, 5), (W, dw, 9)):
        for i in range(n):
            for k in range(6):
                keep = float(t[i, k])
                t[i, k] = keep + h
                hi = f(X, W)
                t[i, k] = keep - h
                lo = f(X, W)
                t[i, k] = keep
                # G is rounded to bf16: 2^-8 of sum |G| |operand|, weights 0.2, values to 3
                assert abs((hi - lo) / (2 * h) - float(g[i, k])) < 2.0 ** -8 * 5


@pytest.mark.parametrize("ab", ["bf16", "f16"])
def test_gradient_against_differences_within_two_terms(ab):
    """The same of float32 gradients, at what G's two terms leave: the bound of xent_util for each element (the differences
    themselves are good to 1e-8: h^2 / 6 of a third derivative below 20, and 2^-52 of the loss over 2 h)."""
    rows, N, K = 5, 9, 6
    x, w, labels, dloss = inputs(rows, N, K, ab, 3)
    _, lse = check_loss(x, w, labels, ab)
    dx, dw = check_grad(x, w, labels, dloss, lse, ab, "f32", "f32")
    X, W, d = x.double().cpu(), w.double().cpu(), dloss.double().cpu()
    lab = labels.cpu().long()
    has = (lab >= 0) & (lab < N)

    def f(a, b):
        z = a @ b.T
        return float((torch.where(has, torch.logsumexp(z, 1) - z.gather(1, lab.clamp(0, N - 1)[:, None])[:, 0], 0.0) * d).sum())

    def differences(t):
        out, h = torch.empty_like(t), 1e-5
        for i in range(t.shape[0]):
            for k in range(t.shape[1]):
                keep = float(t[i, k])
                t[i, k] = keep + h
                hi = f(X, W)
                t[i, k] = keep - h
                out[i, k] = (hi - f(X, W)) / (2 * h)
                t[i, k] = keep
        return out

    z, ez, rl, el, _, _, at = (t.cpu() for t in reference(x, w, labels))
    p = torch.exp(z - rl[:, None])
    G = torch.where(has[:, None], (p - torch.nn.functional.one_hot(at, N)) * d[:, None], 0.0)
    r = (ez + el)[:, None] + (4 * z.abs() + 4 * rl.abs()[:, None] + 8) * 2.0 ** -24
    e = torch.where(has[:, None], d.abs()[:, None] * (p * r + 2.0 ** -23), 0.0) + (2.0 ** -16 if ab == "bf16" else 2.0 ** -22) * G.abs() * 1.01
    if ab == "f16":
        e = torch.where(has[:, None], e + 2.0 ** -39 * float(d.abs().max()), 0.0)
    sums = (2 * N + 2 * rows + 68) * 2.0 ** -23 * G.abs()
    for got, want, tol in ((dx, differences(X), (e + sums) @ W.abs()), (dw, differences(W), (e + sums).T @ X.abs())):
        miss = (got[:, :K].double().cpu() - want).abs() - (tol + 2.0 ** -24 * want.abs() + 1e-8)
        assert (miss <= 0).all(), float(miss.max())
        # (a gradient of zeros, or of another sign, would not pass)
        assert (want.abs() > 100 * (tol + 1e-8)).sum() > 0.7 * want.numel() and tol.max() < 1e-4


def float32_of_g(z, labels, lse, d):
    """G in 64 bits, and its bound: with lse given, p is off by (4 |z| + 4 |lse| + 8) u of itself; G's terms, as one sum of
    exact products, by 2^-22 of G at most (f16's two leave 2^-23, three additions 2^-23 each)."""
    p = torch.exp(z - lse.double()[:, None])
    G = p.clone()
    G[torch.arange(z.shape[0], device="cuda"), labels.long()] -= 1.0
    G *= d.double()[:, None]
    r = (4 * z.abs() + 4 * lse.double().abs()[:, None] + 8) * 2.0 ** -24
    return G, d.double()[:, None].abs() * (p * r + 2.0 ** -23) + (2.0 ** -23 + 3 * 2.0 ** -23) * G.abs() + 2.0 ** -39 * float(d.abs().max())


@pytest.mark.parametrize("ab", ["bf16", "f16"])
@pytest.mark.parametrize("rows,N,K,piece", [(40, 3000, 40, 0), (300, 5001, 304, 0), (300, 5001, 304, 1000), (1700, 4096, 4096, 0),
                                            (1700, 4096, 4096, 2048)])
def test_float32_weight_gradient_is_float32(rows, N, K, piece, ab):
    """X of unit rows: dW is G transposed, every sum one product, so that what G's terms leave shows as it is."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.eye(rows, K, device="cuda").to(DT[ab])
    w = (torch.rand(N, K, device="cuda", generator=g) * 2 - 1).to(DT[ab])
    labels = torch.randint(0, N, (rows,), device="cuda", generator=g, dtype=torch.int32)
    d = torch.rand(rows, device="cuda", generator=g) * 0.9 + 0.1
    z = w.double()[:, :rows].T.contiguous()
    lse = torch.logsumexp(z, 1).float()
    for accum in (0, 1):
        dw = torch.full((N, up(K, 8)), -1.0 if accum else float("nan"), device="cuda")
        work = torch.full((bsm.bsm_gemm_cross_entropy_grad_workspace(rows, N, K, piece),), 255, dtype=torch.uint8, device="cuda")
        xp, wp = wide(x), wide(w)
        say("float32 dW", rows, N, K, piece, ab, accum)
        bsm.bsm_gemm_cross_entropy_grad(rows, N, K, ab, xp, xp.stride(0), wp, wp.stride(0), labels, lse, d, piece, work, ab, None, up(K, 8),
                                        "f32", dw, dw.stride(0), accum)
        G, tol = float32_of_g(z, labels, lse, d)
        got = dw[:, :rows].double().T
        if accum:
            # (onto -1: each of up to three stores rounds at 1)
            assert ((got - (G - 1)).abs() <= tol + 3 * 2.0 ** -24 * 2).all()
        else:
            assert ((got - G).abs() <= tol).all(), float(((got - G).abs() / tol).max())
            small = G.abs() > 0
            assert float(((got - G).abs() / G.abs())[small].mean()) < 2.0 ** -21     # (two bf16 terms: 2^-18.6 in the mean)
            assert not dw[:, rows:K].any()


@pytest.mark.parametrize("ab", ["bf16", "f16"])
@pytest.mark.parametrize("rows,K,piece", [(40, 200, 0), (300, 1000, 0), (300, 1000, 300), (2300, 4096, 0)])
def test_float32_input_gradient_is_float32(rows, K, piece, ab):
    """W of unit rows: dX is G."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    N = K
    x = (torch.rand(rows, K, device="cuda", generator=g) * 2 - 1).to(DT[ab])
    w = torch.eye(N, device="cuda").to(DT[ab])
    labels = torch.randint(0, N, (rows,), device="cuda", generator=g, dtype=torch.int32)
    d = torch.rand(rows, device="cuda", generator=g) * 0.9 + 0.1
    z = x.double()
    lse = torch.logsumexp(z, 1).float()
    dx = torch.full((rows, K), float("nan"), device="cuda")
    work = torch.full((bsm.bsm_gemm_cross_entropy_grad_workspace(rows, N, K, piece),), 255, dtype=torch.uint8, device="cuda")
    say("float32 dX", rows, K, piece, ab)
    bsm.bsm_gemm_cross_entropy_grad(rows, N, K, ab, x, K, w, K, labels, lse, d, piece, work, "f32", dx, K, ab, None, K)
    G, tol = float32_of_g(z, labels, lse, d)
    assert ((dx.double() - G).abs() <= tol).all(), float(((dx.double() - G).abs() / tol).max())
    assert float(((dx.double() - G).abs() / G.abs()).mean()) < 2.0 ** -21
