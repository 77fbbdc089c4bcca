"""GPU parity: block-scaled products with a weight per group of rows, against 64 bits.

Bound with fast = 0: 1e-5 sum|ab| (the library's statement for exact products) and the output's half step.
With fast = 1 each 32-product block may further lose sum min(|p|, 2^-13 max|p|), at most 31 * 2^-13 of the
block's largest product; the same element's own other products stay exact. Padding scales are NaN codes."""
import pytest
import torch

import block_scaled_matrix_amd as bsm
from grouped_util import DT, HALF_STEP, offsets_of, up
from gpu_util import say

pytestmark = pytest.mark.gpu
BITS = {"e4m3": 8, "e2m1": 4}
E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def codes(g, lead, K, fmt, extra=0):
    """Random element codes without NaN in rows of a padded leading dimension, scale codes 123 .. 131 with NaN codes
    as padding, and the 64-bit values."""
    raw = torch.randint(0, 256, (*lead, K * BITS[fmt] // 8), generator=g, dtype=torch.uint8)
    if fmt == "e4m3":
        raw[(raw & 127) == 127] = 0x38
        v = raw.view(torch.float8_e4m3fn).double()
    else:
        v = E2M1[torch.stack((raw & 15, raw >> 4), -1).flatten(-2).long()]
    row = up(K * BITS[fmt] // 8, 16) + extra
    p = torch.full((*lead, row), 0x7F, dtype=torch.uint8)
    p[..., :raw.shape[-1]] = raw
    s = torch.full((*lead, up(K // 32, 4) + (4 if extra else 0)), 255, dtype=torch.uint8)
    s[..., :K // 32] = torch.randint(123, 132, (*lead, K // 32), generator=g, dtype=torch.uint8)
    return p, s, v * torch.exp2(s[..., :K // 32].double() - 127).repeat_interleave(32, -1)


def run(sizes, N, K, a="e4m3", b="e4m3", fast=0, d="bf16", accum=0, ew=None, seed=0, first=0, behind=0, extra=0):
    g = torch.Generator().manual_seed(seed)
    off, G = offsets_of(sizes, first), len(sizes)
    rows = off[-1] + behind
    x, xs, xv = codes(g, (rows,), K, a, extra)
    w, ws, wv = codes(g, (G, N), K, b, extra)
    for r in list(range(first)) + list(range(off[-1], rows)):
        xs[r] = 255
    ldd = up(N, 4 if d == "f32" else 8) + (8 if extra else 0)
    D0 = (K ** 0.5 * 10 * torch.randn(rows, ldd, generator=g)).to(DT[d])
    D = D0.cuda()
    xd, xsd, wd, wsd = x.cuda(), xs.cuda(), w.cuda(), ws.cuda()
    say("grouped mx", sizes if G < 9 else (G, rows), N, K, a, b, fast, d, accum)
    bsm.bsm_gemm_grouped_block_scale(rows, N, K, G, torch.tensor(off, dtype=torch.int32, device="cuda"), a, xd,
                                     xd.stride(0) * 8 // BITS[a], xsd, xsd.stride(0), b, wd, wd.stride(1) * 8 // BITS[b],
                                     wd.stride(0) * 8 // BITS[b], wsd, wsd.stride(1), wsd.stride(0), fast, d, D, ldd, accum, ew)
    torch.cuda.synchronize()
    got = D.cpu()
    inside = torch.zeros(rows, dtype=torch.bool)
    for i in range(G):
        lo, hi = off[i], off[i + 1]
        inside[lo:hi] = True
        ref, mag = xv[lo:hi] @ wv[i].T, xv[lo:hi].abs() @ wv[i].abs().T
        tol = 1e-5 * mag
        if fast:
            for k in range(0, K, 32):
                for r in range(lo, hi, 64):
                    p = (xv[r:min(r + 64, hi), None, k:k + 32] * wv[i][None, :, k:k + 32]).abs()
                    tol[r - lo:r - lo + 64] += torch.minimum(p, p.amax(-1, keepdim=True) * 2.0 ** -13).sum(-1)
        if accum:
            ref = ref + D0[lo:hi, :N].double()
            tol = tol + 2.0 ** -23 * (mag + D0[lo:hi, :N].double().abs())
        if ew is not None:   # as for the 16-bit products: slope below 1.1, a few ulp of silu, two roundings
            tol = 1.1 * abs(ew.scale) * tol + 6 * 2.0 ** -23 * (abs(ew.scale) * ref.abs() + abs(ew.bias))
            ref = ref / (1 + torch.exp(-ref)) * ew.scale + ew.bias
        tol = tol + HALF_STEP[d] * ref.abs() * (1 + 2.0 ** -7)
        bad = ~((got[lo:hi, :N].double() - ref).abs() <= tol)
        assert not bad.any(), (i, int(bad.sum()), bad.nonzero()[:4].tolist())
    same = lambda u, v: torch.equal(u.contiguous().view(torch.uint8), v.contiguous().view(torch.uint8))
    assert same(got[~inside], D0[~inside]), "rows in no group were written"
    assert same(got[:, N:], D0[:, N:]), "columns past N were written"
    return got


PAIRS = [("e4m3", "e4m3", 0), ("e4m3", "e4m3", 1), ("e4m3", "e2m1", 0), ("e4m3", "e2m1", 1), ("e2m1", "e2m1", 0), ("e2m1", "e2m1", 1)]
SIZES = [[1], [1] * 9, [0, 3, 0, 0, 17, 0], [0, 0], [255, 256, 1], [70, 15, 16, 33], [(5 * i) % 4 for i in range(130)]]


@pytest.mark.parametrize("a,b,fast", PAIRS)
@pytest.mark.parametrize("sizes", SIZES, ids=["one", "ones", "empty", "none", "edges", "uneven", "many"])
def test_sizes(sizes, a, b, fast):
    run(sizes, 72, 160, a, b, fast, seed=len(sizes))


@pytest.mark.parametrize("a,b,fast", PAIRS)
@pytest.mark.parametrize("N,K", [(1, 32), (7, 96), (16, 128), (33, 256), (257, 288), (130, 1024)])
def test_odd_sizes(N, K, a, b, fast):
    run([3, 0, 18, 40], N, K, a, b, fast, "f32", seed=N + K, first=2, behind=3, extra=16)


@pytest.mark.parametrize("sizes", [[2, 9, 1], [40, 0, 90], [200, 20]])
@pytest.mark.parametrize("a,b,fast", PAIRS)
def test_outputs_accumulate_and_epilogue(sizes, a, b, fast):
    for d in ("bf16", "f32"):
        run(sizes, 104, 192, a, b, fast, d, 1, None, 3)
        run(sizes, 104, 192, a, b, fast, d, 0, bsm.ewise_desc("silu_affine", 0.5, 0.25), 4)
    run(sizes, 40, 0, a, b, fast, "bf16", 1)
    run(sizes, 40, 0, a, b, fast, "f32", 0)


def test_a_scale_that_is_nan_stays_in_its_row():
    """Row 3 of the activations and one weight row carry a NaN scale in one block: their outputs are NaN, no others."""
    rows, N, K = 21, 24, 128
    g = torch.Generator().manual_seed(2)
    for a, b, fast in PAIRS:
        x, xs, _ = codes(g, (rows,), K, a)
        w, ws, _ = codes(g, (2, N), K, b)
        xs[3, 2] = 255
        ws[1, 5, 0] = 255
        D = torch.empty(rows, N, device="cuda")
        bsm.bsm_gemm_grouped_block_scale(rows, N, K, 2, torch.tensor([0, 9, rows], dtype=torch.int32, device="cuda"), a,
                                         x.cuda(), K, xs.cuda(), xs.stride(0), b, w.cuda(), K, N * K, ws.cuda(), ws.stride(1),
                                         ws.stride(0), fast, "f32", D, N)
        nan = torch.isnan(D).cpu()
        want = torch.zeros(rows, N, dtype=torch.bool)
        want[3] = True
        want[9:, 5] = True
        assert torch.equal(nan, want), (a, b, fast)


def test_matches_the_product_of_one_group():
    """One group of all rows is bsm_gemm_block_scale (exact products, float32 out) up to the order of the sum."""
    rows, N, K = 300, 264, 512
    g = torch.Generator().manual_seed(5)
    x, xs, xv = codes(g, (rows,), K, "e4m3")
    w, ws, wv = codes(g, (1, N), K, "e2m1")
    xd, xsd, wd, wsd = x.cuda(), xs.cuda(), w.cuda(), ws.cuda()
    D, E = torch.empty(rows, N, device="cuda"), torch.empty(rows, N, device="cuda")
    bsm.bsm_gemm_grouped_block_scale(rows, N, K, 1, torch.tensor([0, rows], dtype=torch.int32, device="cuda"), "e4m3", xd, K, xsd,
                                     xsd.stride(0), "e2m1", wd, K, 0, wsd, wsd.stride(1), 0, 0, "f32", D, N)
    bsm.bsm_gemm_block_scale(rows, N, K, "e4m3", xd, K, xsd, xsd.stride(0), "e2m1", wd, K, wsd, wsd.stride(1), E, N)
    assert ((D - E).abs().double().cpu() <= 2e-5 * (xv.abs() @ wv[0].abs().T)).all()


@pytest.mark.parametrize("a,b,fast", PAIRS)
@pytest.mark.parametrize("K", [32, 128, 160, 256, 384, 1184])
def test_fewer_tiles_than_compute_units(K, a, b, fast):
    """Two sets of waves share a tile's K: none, one and more whole K tiles each, an odd one, and a partial one."""
    run([65, 0, 130, 90, 32, 1], 260, K, a, b, fast, "f32", seed=K, behind=2, extra=16)


@pytest.mark.parametrize("a,b,fast", PAIRS)
def test_large_tiles(a, b, fast):
    """Groups that the 256 x 256 kernels take, and their ragged ends."""
    run([700, 300, 3, 520], 4100, 160, a, b, fast, "bf16", seed=6)


def test_many_groups_of_few_rows():
    """Exact E4M3 x E2M1 of up to 16 rows a group on average, single groups far above it, and tiles in plenty."""
    sizes = [(7 * i) % 9 for i in range(40)] + [70, 0, 33]
    for K in (96, 160, 1056):
        run(sizes, 1300, K, "e4m3", "e2m1", 0, "bf16", 1, None, K, first=1, behind=2, extra=16)
        run(sizes, 1300, K, "e4m3", "e2m1", 0, "f32", 0, bsm.ewise_desc("silu_affine", 0.5, 0.25), K)
