"""GPU parity: fp16/bf16 products with a weight per group of rows and their weight gradient, against 64 bits.
The bound is derived in grouped_util. Padding, rows outside every group and the other groups' rows hold NaN or
values that would show, and untouched memory is checked to stay so."""
import pytest
import torch

import block_scaled_matrix_amd as bsm
from grouped_util import DT, check, offsets_of, padded, silu_affine, up
from gpu_util import say

pytestmark = pytest.mark.gpu


def case(sizes, N, K, ab, major, seed, first=0, behind=0, extra=0):
    g = torch.Generator().manual_seed(seed)
    off = offsets_of(sizes, first)
    rows = off[-1] + behind
    x = torch.randn(rows, K, generator=g).to(DT[ab])
    w = torch.randn(len(sizes), *((N, K) if major == "k" else (K, N)), generator=g).to(DT[ab])
    for r in list(range(first)) + list(range(off[-1], rows)):
        x[r] = float("nan")
    return off, rows, x, w, padded(x, 8, extra), padded(w, 8, extra)


def run(sizes, N, K, ab="bf16", major="k", d=None, accum=0, ew=None, seed=0, first=0, behind=0, extra=0, shared=False,
        stream=None):
    d = d or ab
    off, rows, x, w, xp, wp = case(sizes, N, K, ab, major, seed, first, behind, extra)
    G = len(sizes)
    ldd = up(N, 4 if d == "f32" else 8) + (8 if extra else 0)
    D0 = torch.randn(rows, ldd, generator=torch.Generator().manual_seed(seed + 1)).to(DT[d])
    xd, wd, D = xp.cuda(), wp.cuda(), D0.cuda()
    od = torch.tensor(off, dtype=torch.int32, device="cuda")
    say("grouped", sizes if G < 9 else (G, rows), N, K, ab, major, d, accum)
    bsm.bsm_gemm_grouped(rows, N, K, G, od, ab, xd, xd.stride(0), wd, wd.stride(1), major, 0 if shared else wd.stride(0), d, D,
                         ldd, accum, ew, stream)
    torch.cuda.synchronize()
    got = D.cpu()
    inside = torch.zeros(rows, dtype=torch.bool)
    for i in range(G):
        a, b = off[i], off[i + 1]
        inside[a:b] = True
        if a == b:
            continue
        wi = w[0 if shared else i].double()
        wi = wi.T if major == "k" else wi
        ref, mag = x[a:b].double() @ wi, x[a:b].double().abs() @ wi.abs()
        if accum:
            ref, mag = ref + D0[a:b, :N].double(), mag + D0[a:b, :N].double().abs()
        if ew is not None:
            # |d/dx silu| <= 1.1, silu itself within 4 ulp and the affine map's two roundings
            mag = 1.1 * abs(ew.scale) * mag + (abs(ew.scale) * ref.abs() + abs(ew.bias)) * 6 / (K + 2)
            ref = silu_affine(ref, ew.scale, ew.bias)
        check(got[a:b, :N], ref, mag, K, d, (sizes, i))
    same = lambda u, v: torch.equal(u.view(torch.int16 if d != "f32" else torch.int32), v.view(torch.int16 if d != "f32" else torch.int32))
    assert same(got[~inside].contiguous(), D0[~inside].contiguous()), "rows in no group were written"
    if ldd > N:
        assert same(got[:, N:].contiguous(), D0[:, N:].contiguous()), "columns past N were written"
    return got


SIZES = {
    "one row": [1],
    "one row each": [1] * 9,
    "empty first, last and between": [0, 3, 0, 0, 17, 0],
    "none at all": [0, 0, 0],
    "tile edges": [255, 256, 257],
    "uneven": [1, 70, 15, 16, 33, 129, 300],
    "over 64 groups": [(7 * i) % 5 for i in range(150)],
}


@pytest.mark.parametrize("ab", ["bf16", "f16"])
@pytest.mark.parametrize("major", ["k", "n"])
@pytest.mark.parametrize("sizes", SIZES.values(), ids=SIZES.keys())
def test_grouped_sizes(sizes, major, ab):
    run(sizes, 264, 136, ab, major, seed=len(sizes))


@pytest.mark.parametrize("major", ["k", "n"])
@pytest.mark.parametrize("N,K", [(1, 1), (7, 33), (16, 64), (63, 65), (257, 129), (1000, 520), (24, 2048), (130, 1003)])
def test_grouped_odd_sizes(N, K, major):
    run([3, 0, 18, 40], N, K, "bf16", major, seed=N + K, first=2, behind=3, extra=8)


@pytest.mark.parametrize("sizes", [[2, 9, 1], [40, 0, 90], [300, 20]])
@pytest.mark.parametrize("ab,d", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
def test_grouped_outputs_accumulate_and_epilogue(ab, d, sizes):
    for accum in (0, 1):
        run(sizes, 200, 96, ab, "k", d, accum, seed=3)
        run(sizes, 200, 96, ab, "n", d, accum, bsm.ewise_desc("silu_affine", 1.5, -0.25), seed=4)


def test_grouped_empty_k_and_rows():
    for major in "kn":
        run([3, 4], 40, 0, "bf16", major, "f32", 1)
        run([3, 4], 40, 0, "bf16", major, "bf16", 0)
    run([], 40, 8, "bf16")
    run([0], 40, 8, "bf16")


def test_grouped_shared_weight():
    run([5, 300, 2], 130, 72, "bf16", "k", shared=True)
    run([5, 300, 2], 130, 72, "bf16", "n", shared=True)


def test_grouped_offsets_outside_the_rows_stay_inside():
    """Offsets past the last row, negative ones and decreasing pairs are clamped: rows keep to their bounds."""
    rows, N, K = 20, 40, 24
    x, w = torch.randn(rows, K).bfloat16().cuda(), torch.randn(4, N, K).bfloat16().cuda()
    D = torch.zeros(rows + 30, N, dtype=torch.float32, device="cuda")
    off = torch.tensor([-5, 6, 2, 9, 4000], dtype=torch.int32, device="cuda")
    bsm.bsm_gemm_grouped(rows, N, K, 4, off, "bf16", x, K, w, K, "k", N * K, "f32", D, N)
    torch.cuda.synchronize()
    assert not D[rows:].any()
    ref, mag = x[9:].double() @ w[3].double().T, x[9:].double().abs() @ w[3].double().abs().T
    check(D[9:rows], ref.cpu(), mag.cpu(), K, "f32")


def test_grouped_large_offsets():
    """A weight whose start lies past 2^31 elements, and rows past 2^31 bytes."""
    N, K, G = 8, 64, 3
    stride = (1 << 30) + 64
    w = torch.zeros(2 * stride + N * K, dtype=torch.bfloat16, device="cuda")
    w[2 * stride:] = 1.0
    rows = (1 << 24) + 5          # rows * K * 2 bytes = 2 GiB
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    x[-5:] = torch.arange(1, 6, device="cuda")[:, None].bfloat16()
    D = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 2, 1 << 24, rows], dtype=torch.int32, device="cuda")
    say("grouped large")
    bsm.bsm_gemm_grouped(rows, N, K, G, off, "bf16", x, K, w, K, "k", stride, "bf16", D, N)
    torch.cuda.synchronize()
    assert torch.equal(D[-5:].float(), 64.0 * torch.arange(1, 6, device="cuda")[:, None].expand(5, N))
    assert not D[:-5].any()


def wgrad(sizes, M, N, ab="bf16", d="f32", accum=0, seed=0, first=0, behind=0, extra=0, pad=0):
    g = torch.Generator().manual_seed(seed)
    off, G = offsets_of(sizes, first), len(sizes)
    rows = off[-1] + behind
    y, x = (torch.randn(rows, n, generator=g).to(DT[ab]) for n in (M, N))
    for r in list(range(first)) + list(range(off[-1], rows)):
        y[r] = x[r] = float("nan")
    yd, xd = padded(y, 8, extra).cuda(), padded(x, 8, extra).cuda()
    ldd = up(N, 4 if d == "f32" else 8) + pad
    D0 = torch.randn(G, M, ldd, generator=g).to(DT[d])
    D = D0.cuda()
    say("wgrad", sizes if G < 9 else (G, rows), M, N, ab, d, accum)
    bsm.bsm_gemm_grouped_wgrad(rows, M, N, G, torch.tensor(off, dtype=torch.int32, device="cuda"), ab, yd, yd.stride(0), xd,
                               xd.stride(0), d, D, ldd, D.stride(0), accum)
    torch.cuda.synchronize()
    got = D.cpu()
    for i in range(G):
        a, b = off[i], off[i + 1]
        ref, mag = y[a:b].double().T @ x[a:b].double(), y[a:b].double().abs().T @ x[a:b].double().abs()
        if accum:
            ref, mag = ref + D0[i, :, :N].double(), mag + D0[i, :, :N].double().abs()
        check(got[i, :, :N], ref, mag, b - a, d, (sizes, i))
    assert torch.equal(got[:, :, N:], D0[:, :, N:]), "columns past N were written"


@pytest.mark.parametrize("ab,d", [("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("sizes", SIZES.values(), ids=SIZES.keys())
def test_wgrad_sizes(sizes, ab, d):
    wgrad(sizes, 136, 72, ab, d, seed=len(sizes))


@pytest.mark.parametrize("M,N", [(1, 1), (7, 33), (257, 129), (300, 520)])
@pytest.mark.parametrize("accum", [0, 1])
def test_wgrad_odd_sizes(M, N, accum):
    wgrad([5, 0, 64, 31, 130], M, N, "bf16", "f32", accum, seed=M, first=1, behind=2, extra=8, pad=8)
    wgrad([5, 0, 64, 31, 130], M, N, "f16", "f16", accum, seed=M, behind=2, pad=8)


def test_gradients_against_differences():
    """The gradients of L = sum(C * (X W_g^T)) in X and W against central differences of the forward call in
    float32 outputs (L is linear in each, so a difference of any step is exact up to rounding)."""
    sizes, N, K = [6, 0, 21], 48, 40
    off = offsets_of(sizes)
    rows = off[-1]
    g = torch.Generator().manual_seed(9)
    grid = lambda *s: (torch.randint(-8, 9, s, generator=g) / 8).bfloat16().cuda()
    x, w, c = grid(rows, K), grid(3, N, K), grid(rows, N)
    od = torch.tensor(off, dtype=torch.int32, device="cuda")
    dx = torch.empty(rows, K, dtype=torch.float32, device="cuda")
    dw = torch.empty(3, N, K, dtype=torch.float32, device="cuda")
    bsm.bsm_gemm_grouped(rows, K, N, 3, od, "bf16", c, N, w, K, "n", N * K, "f32", dx, K)
    bsm.bsm_gemm_grouped_wgrad(rows, N, K, 3, od, "bf16", c, N, x, K, "f32", dw, K, N * K)

    def loss(xx, ww):
        out = torch.empty(rows, N, dtype=torch.float32, device="cuda")
        bsm.bsm_gemm_grouped(rows, N, K, 3, od, "bf16", xx, K, ww, K, "k", N * K, "f32", out, N)
        return float((out.double() * c.double()).sum())

    for r, k in [(0, 0), (5, 39), (6, 7), (26, 21)]:
        p, m = x.clone(), x.clone()
        p[r, k] += 0.5
        m[r, k] -= 0.5
        assert abs(loss(p, w) - loss(m, w) - float(dx[r, k])) <= 1e-3
    for e, n, k in [(0, 0, 0), (0, 47, 39), (1, 3, 3), (2, 11, 30)]:
        p, m = w.clone(), w.clone()
        p[e, n, k] += 0.5
        m[e, n, k] -= 0.5
        assert abs(loss(x, p) - loss(x, m) - float(dw[e, n, k])) <= 1e-3
    assert not dw[1].any()


@pytest.mark.parametrize("sizes", [[1], [16], [17], [1] * 8, [64], [33, 0, 20], [90, 2, 3], [0, 150, 1, 2]])
@pytest.mark.parametrize("ab,d", [("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("K", [64, 72, 500, 512, 1099, 4160])
def test_few_rows_and_long_k(sizes, ab, d, K):
    """Few tiles and a long sum (the waves split K), with groups far above the average among them."""
    run(sizes, 50, K, ab, "k", d, seed=K, first=1, behind=1, extra=8)
    run(sizes, 50, K, ab, "k", d, 1, bsm.ewise_desc("silu_affine", 0.5, 0.25), seed=K)


@pytest.mark.parametrize("major", ["k", "n"])
@pytest.mark.parametrize("K", [32, 64, 100, 128, 192, 1000])
def test_fewer_tiles_than_compute_units(K, major):
    """Two sets of waves share a tile's sum: one, two, three and more K tiles and a partial one."""
    run([65, 0, 130, 90, 32], 260, K, "bf16", major, seed=K, behind=2)
    run([100, 200], 260, K, "f16", major, "f32", 1, bsm.ewise_desc("silu_affine", 1.0, 0.5), seed=K)


@pytest.mark.parametrize("sizes", [[1024], [1100], [1500, 0, 1663], [64, 1985]])
def test_wgrad_of_few_tiles(sizes):
    """Two sets of waves share a group's rows: an odd and an even number of K tiles, a partial one."""
    wgrad(sizes, 200, 140, "bf16", "f32", 1, seed=3, first=1, behind=2)
    wgrad(sizes, 200, 140, "f16", "f16", 0, seed=4, extra=8, pad=8)


def test_large_tiles():
    """Groups that the 256 x 256 tile takes (and their ragged ends), both orders of the weight, and long groups of a
    weight gradient."""
    for major in "kn":
        run([1300, 770, 3, 2047], 4100, 72, "bf16", major, seed=6)
        run([1300, 770, 3 * 256 + 193, 0, 2047 + 192], 3400, 200, "bf16", major, "f32", 1, seed=5, first=1, behind=3, extra=8)
    wgrad([700, 0, 1030], 520, 4200, "bf16", "f32", 1, seed=7)
    wgrad([700, 0, 1030], 4200, 520, "f16", "f16", 0, seed=8)
