"""GPU parity: the weight gradient over groups of rows from activations kept in 8 bits, against 64 bits: the bound of
grouped_util, since a code times its scale is exact in the operands' formats inside their range. The codes here are drawn,
not saved from f16 values, so in f16 some lie below its normal numbers: a value below 2^-14 becomes a multiple of 2^-24, off
by at most 2^-25, and its product with y by 2^-25 |y|; a sum is off by 2^-25 sum|y| more."""
import pytest
import torch

import block_scaled_matrix_amd as bsm
from grouped_util import DT, check, offsets_of, padded, tolerance, up
from gpu_util import say
from test_gpu_checkpoint import F8, values
from test_gpu_grouped import SIZES

pytestmark = pytest.mark.gpu


def kept_rows(rows, N, fmt, g, spread):
    """Codes without NaN and infinities, and scale codes around 1."""
    c = torch.randint(0, 256, (rows, N), generator=g, dtype=torch.uint8)
    bad = ~torch.isfinite(c.view(F8[fmt]).float())
    c[bad] = 0x35
    s = torch.randint(127 - spread - (6 if fmt == "e4m3" else 12), 127 + spread - 4, (rows, (N + 31) // 32), generator=g).to(torch.uint8)
    return c, s


def wgrad(sizes, M, N, ab="bf16", fmt="e4m3", d="f32", accum=0, seed=0, first=0, behind=0, extra=0, pad=0, spread=5, stream=None, change=None):
    g = torch.Generator().manual_seed(seed)
    off, G = offsets_of(sizes, first), len(sizes)
    rows = off[-1] + behind
    y = torch.randn(rows, M, generator=g).to(DT[ab])
    c, s = kept_rows(rows, N, fmt, g, spread)
    for r in list(range(first)) + list(range(off[-1], rows)):
        y[r], c[r], s[r] = float("nan"), 0x7F, 255
    if change:
        change(y, c, s)
    yd = padded(y, 8, extra).cuda()
    cd = torch.full((rows, up(N, 16) + 2 * extra), 0x7F, dtype=torch.uint8)
    cd[:, :N] = c
    sd = torch.full((rows, up(s.shape[1], 4) + extra), 255, dtype=torch.uint8)
    sd[:, :s.shape[1]] = s
    cd, sd = cd.cuda(), sd.cuda()
    ldd = up(N, 4 if d == "f32" else 8) + pad
    D0 = torch.randn(G, M, ldd, generator=g).to(DT[d])
    D = D0.cuda()
    say("kept wgrad", sizes if G < 9 else (G, rows), M, N, ab, fmt, d, accum)
    bsm.bsm_gemm_grouped_wgrad_block_scale(rows, M, N, G, torch.tensor(off, dtype=torch.int32, device="cuda"), ab, yd, yd.stride(0),
                                           fmt, cd, cd.stride(0), sd, sd.stride(0), d, D, ldd, D.stride(0), accum, stream)
    torch.cuda.synchronize()
    got = D.cpu()
    x = values(c.view(F8[fmt]).double(), s, N)
    if not change:
        for i in range(G):
            a, b = off[i], off[i + 1]
            yy, xx = (y[a:b].double().cuda(), x[a:b].cuda()) if M * N * rows > 1 << 26 else (y[a:b].double(), x[a:b])
            ref, mag = (yy.T.contiguous() @ xx).cpu(), (yy.abs().T.contiguous() @ xx.abs()).cpu()
            if accum:
                ref, mag = ref + D0[i, :, :N].double(), mag + D0[i, :, :N].double().abs()
            if ab == "f16":
                # (check takes (terms + 2) 2^-23 of the magnitude: the same amount as a part of it)
                mag = mag + 2.0 ** -25 * y[a:b].double().abs().sum(0)[:, None] / ((b - a + 2) * 2.0 ** -23)
            here = got[i, :, :N]
            if d == "f16":
                # a sum that lies at 65520 or beyond, within its bound, is infinity in f16 (65504 and half its step)
                over = torch.isinf(here) & (here.sign() == ref.sign()) & (ref.abs() + tolerance(ref, mag, b - a, "f32") >= 65520)
                here = torch.where(over, ref.to(here.dtype).clamp(-65504, 65504), here)
                ref = torch.where(over, here.double(), ref)
            check(here, ref, mag, b - a, d, (sizes, i))
    assert torch.equal(got[:, :, N:], D0[:, :, N:]), "columns past N were written"
    return got, y, x


@pytest.mark.parametrize("ab,fmt,d", [("bf16", "e4m3", "f32"), ("bf16", "e5m2", "bf16"), ("f16", "e4m3", "f16"), ("f16", "e5m2", "f32")])
@pytest.mark.parametrize("sizes", SIZES.values(), ids=SIZES.keys())
def test_sizes(sizes, ab, fmt, d):
    wgrad(sizes, 136, 72, ab, fmt, d, seed=len(sizes))


@pytest.mark.parametrize("M,N", [(1, 1), (7, 33), (257, 129), (300, 520), (128, 136), (64, 1000)])
@pytest.mark.parametrize("accum", [0, 1])
def test_odd_sizes(M, N, accum):
    wgrad([5, 0, 64, 31, 130], M, N, "bf16", "e4m3", "f32", accum, seed=M, first=1, behind=2, extra=8, pad=8)
    wgrad([5, 0, 64, 31, 130], M, N, "f16", "e5m2", "f16", accum, seed=M, behind=2, pad=8)


@pytest.mark.parametrize("ab", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("sizes,M,N", [([200, 700, 33, 1000], 2100, 1500), ([96] * 3, 500, 300), ([1000, 3000], 512, 640), ([32, 64, 96, 128, 160], 130, 130)])
def test_tiles(sizes, M, N, ab, fmt):
    wgrad(sizes, M, N, ab, fmt, "f32", seed=M)
    wgrad(sizes, M, N, ab, fmt, ab, 1, seed=M)


@pytest.mark.parametrize("ab,fmt", [("bf16", "e4m3"), ("bf16", "e5m2"), ("f16", "e4m3"), ("f16", "e5m2")])
@pytest.mark.parametrize("sizes,M,N", [
    ([700, 0, 64, 1200, 1, 63, 3000, 1300], 1400, 1250),       # 256 x 256, groups of no row, one, a K tile and a long one
    ([640, 65, 2000], 2056, 2400), ([768], 4100, 3600),
    ([30, 0, 75], 300, 400), ([300], 520, 130),                # 64 x 64, two sets of waves
    ([2001], 200, 130), ([1000, 0, 2100], 260, 70),            # four
    ([3000, 1700], 1030, 600),                                 # 128 x 128, four sets
    ([33, 64, 0, 31, 100], 1030, 700)])                        # one
def test_every_tile(sizes, M, N, ab, fmt):
    wgrad(sizes, M, N, ab, fmt, "f32", seed=N, first=1, behind=1)
    wgrad(sizes, M, N, ab, fmt, "f32", 1, seed=N, first=1)
    wgrad(sizes, M, N, ab, fmt, ab, 1, seed=N, extra=16, pad=8)


def test_more_groups_than_are_ranked():
    """300 groups on 256 x 256 tiles come in their order; 256 are ranked."""
    for n in (256, 300):
        rows = [700 + (i * 37) % 100 for i in range(n)]
        off = offsets_of(rows)
        M, N = 8, 16
        y = torch.ones(off[-1], M, dtype=torch.bfloat16, device="cuda")
        c = torch.full((off[-1], N), 0x38, dtype=torch.uint8, device="cuda")
        s = torch.full((off[-1], 4), 127, dtype=torch.uint8, device="cuda")
        D = torch.full((n, M, N), float("nan"), device="cuda")
        bsm.bsm_gemm_grouped_wgrad_block_scale(off[-1], M, N, n, torch.tensor(off, dtype=torch.int32, device="cuda"), "bf16", y, M, "e4m3",
                                               c, N, s, 4, "f32", D, N, M * N)
        assert torch.equal(D, torch.tensor(rows, dtype=torch.float32, device="cuda")[:, None, None].expand(n, M, N))


def test_equals_the_gradient_of_restored_activations():
    """The same bits as bsm_gemm_grouped_wgrad where one K tile of 32 rows holds the group, whose products are then one sum."""
    g = torch.Generator().manual_seed(1)
    rows, M, N = 32, 128, 128
    y = torch.randn(rows, M, generator=g).bfloat16().cuda()
    x = torch.randn(rows, N, generator=g).bfloat16().cuda()
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    q, s = torch.empty(rows, N, dtype=torch.uint8, device="cuda"), torch.empty(rows, 4, dtype=torch.uint8, device="cuda")
    bsm.bsm_block_scale_save(rows, N, "bf16", x, N, "e4m3", q, N, s, 4)
    xr = torch.empty_like(x)
    bsm.bsm_block_scale_restore(rows, N, "e4m3", q, N, s, 4, "bf16", xr, N)
    a, b = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    bsm.bsm_gemm_grouped_wgrad_block_scale(rows, M, N, 1, off, "bf16", y, M, "e4m3", q, N, s, 4, "f32", a, N, 0)
    bsm.bsm_gemm_grouped_wgrad(rows, M, N, 1, off, "bf16", y, M, xr, N, "f32", b, N, 0)
    assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_nan_and_wide_scales(fmt):
    """A NaN code or scale shows in its column of its group and nowhere else; scales at the ends of bf16's range are exact."""
    def change(y, c, s):
        c[40, 3] = 0x7F if fmt == "e4m3" else 0x7E
        s[90, 1] = 255
    got, _, _ = wgrad([30, 40, 60], 70, 100, "bf16", fmt, change=change)
    nan = torch.isnan(got[:, :, :100])
    want = torch.zeros_like(nan)
    want[1, :, 3] = True
    want[2, :, 32:64] = True
    assert torch.equal(nan, want)
    top = 127 + 119 if fmt == "e4m3" else 127 + 110
    for code in (20, 60, 200, top):
        def change(y, c, s):
            y.zero_()
            y[::32] = 1.0       # one term a sum and 32 rows: exact
            s.fill_(code)
        got, y, x = wgrad([32, 32], 40, 96, "bf16", fmt, change=change)
        for i in range(2):
            want = x[32 * i].float()
            ok = torch.isfinite(want)
            assert torch.equal(got[i, 0, :96][ok], want[ok])


def test_f16_at_the_end_of_its_range():
    """65536 (65504 as kept) enters as 65504, not as infinity."""
    def change(y, c, s):
        y.zero_()
        y[0] = 0.5
        c.fill_(0x78)          # 256 in E4M3
        s.fill_(127 + 8)
    got, _, _ = wgrad([20], 16, 40, "f16", "e4m3", "f16", change=change)
    assert (got[0, :, :40] == 32752.0).all()


@pytest.mark.parametrize("rows,M,N", [(32, 128, 64), (800, 200, 200), (1600, 1032, 1200), (70, 1000, 2100), (800, 4096, 3600)])   # each tile
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("ab", ["bf16", "f16"])
def test_values_beyond_the_range(ab, fmt, rows, M, N):
    """Codes that stand for more than ab's range (2^128 and more in BF16) enter as its largest value, not as infinity, so that
    rows of zeros in dY leave no NaN; infinite codes stay so."""
    g = torch.Generator().manual_seed(rows)
    c, _ = kept_rows(rows, N, fmt, g, 1)
    s = torch.randint(236, 255, (rows, (N + 31) // 32), generator=g).to(torch.uint8)
    if fmt == "e5m2":
        c[5, 3] = 0xFC
    y = torch.zeros(rows, M, dtype=DT[ab])
    y[5::8, :M:3] = 2.0 ** -12                          # one term a sum and group: exact
    groups = -(-rows // 8)
    off = torch.tensor([min(8 * i, rows) for i in range(groups + 1)], dtype=torch.int32, device="cuda")
    sd = torch.full((rows, up(s.shape[1], 4)), 255, dtype=torch.uint8)
    sd[:, :s.shape[1]] = s
    cd = torch.zeros(rows, up(N, 16), dtype=torch.uint8)
    cd[:, :N] = c
    if rows >= 800:                                     # (one long group, one row of dY that is not 0)
        groups, off = 1, off[[0, -1]].contiguous()
        y[6:] = 0
    D = torch.full((groups, M, up(N, 4)), float("nan"), device="cuda")
    say("kept wgrad beyond the range", ab, fmt, rows, M, N)
    bsm.bsm_gemm_grouped_wgrad_block_scale(rows, M, N, groups, off, ab, y.cuda(), M, fmt, cd.cuda(), cd.stride(0), sd.cuda(),
                                           sd.stride(0), "f32", D, D.stride(1), D.stride(0))
    m = torch.finfo(DT[ab]).max
    x = values(c.view(F8[fmt]).double(), s, N)
    x = torch.where(torch.isfinite(x), x.clamp(-m, m), x).float()
    got = D[:, :, :N].cpu()
    for i in range(groups):
        r = 8 * i + 5
        want = x[r] * 2.0 ** -12 if r < rows else torch.zeros(N)
        inf = torch.isinf(x[8 * i:8 * i + 8]).any(0) if fmt == "e5m2" else torch.zeros(N, dtype=torch.bool)
        assert torch.equal(got[i, 0, ~inf], want[~inf])
        assert not got[i, 1][~inf].any() and torch.isnan(got[i, 1][inf]).all() and (got[i, 0][inf] == -float("inf")).all()


def test_offsets_outside_the_rows_stay_inside():
    rows, M, N = 20, 24, 40
    y = torch.randn(rows, M).bfloat16().cuda()
    c = torch.full((rows, 48), 0x38, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, 4), 127, dtype=torch.uint8, device="cuda")
    off = torch.tensor([-5, 6, 2, 9, 4000], dtype=torch.int32, device="cuda")
    D = torch.empty(4, M, N, device="cuda")
    bsm.bsm_gemm_grouped_wgrad_block_scale(rows, M, N, 4, off, "bf16", y, M, "e4m3", c, 48, s, 4, "f32", D, N, M * N)
    ref = torch.stack([y[:6].double().sum(0), y[:0].double().sum(0), y[2:9].double().sum(0), y[9:].double().sum(0)])
    check(D[:, :, 5], ref.cpu(), ref.abs().cpu() + 20, 20, "f32")


def test_rows_past_32_bits():
    """Codes past 2^31 bytes and rows of dY past 2^31 bytes."""
    M, N = 64, 128
    rows = (1 << 24) + 45
    y = torch.zeros(rows, M, dtype=torch.bfloat16, device="cuda")
    c = torch.zeros(rows, N, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, 4), 127, dtype=torch.uint8, device="cuda")
    y[-45:] = 1.0
    c[-45:] = 0x38             # 1.0
    off = torch.tensor([0, 1 << 24, rows], dtype=torch.int32, device="cuda")
    D = torch.empty(2, M, N, device="cuda")
    say("kept wgrad past 2^31")
    bsm.bsm_gemm_grouped_wgrad_block_scale(rows, M, N, 2, off, "bf16", y, M, "e4m3", c, N, s, 4, "f32", D, N, M * N)
    assert not D[0].any() and (D[1] == 45.0).all()


def test_same_bits_on_every_call():
    a = wgrad([300, 77, 500], 520, 260, seed=2)[0]
    for _ in range(3):
        assert torch.equal(a, wgrad([300, 77, 500], 520, 260, seed=2)[0])


@pytest.mark.parametrize("M,N", [(130, 200), (1030, 1200), (2056, 2400)])
def test_one_long_group_among_empty_ones(M, N):
    """The tile goes by the groups' mean length: one group with all of the rows on tiles for short ones."""
    wgrad([0] * 5 + [2500] + [0] * 10, M, N, seed=M, first=1)
    wgrad([0] * 3 + [2500, 1, 0, 0], M, N, "f16", "e5m2", "f16", 1, seed=M)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_large_tiles_beyond_the_range_added_to_in_16_bits(fmt):
    """256 x 256 tiles whose scales reach past bf16's range, onto a bf16 D with rows and columns behind the tile's; one
    group's scales are ordinary, and the bytes behind the scales hold wide ones."""
    rows, M, N, ldd = 1500, 2050, 3610, 3624
    g = torch.Generator().manual_seed(3)
    off = [0, 740, 1500]
    c, _ = kept_rows(rows, N, fmt, g, 1)
    s = torch.randint(236, 255, (rows, (N + 31) // 32), generator=g).to(torch.uint8)
    s[740:] = 127
    y = torch.zeros(rows, up(M, 8), dtype=torch.bfloat16)
    y[11, :M:3], y[745, 1:M:3] = 2.0 ** -12, 2.0 ** -12     # one term a sum: exact
    sd = torch.full((rows, up(s.shape[1], 4) + 4), 250, dtype=torch.uint8)
    sd[:, :s.shape[1]] = s
    cd = torch.full((rows, up(N, 16)), 0x70, dtype=torch.uint8)
    cd[:, :N] = c
    D0 = torch.randn(2, M, ldd, generator=g).bfloat16()
    D = D0.cuda()
    say("kept wgrad beyond the range, added to", fmt)
    bsm.bsm_gemm_grouped_wgrad_block_scale(rows, M, N, 2, torch.tensor(off, dtype=torch.int32, device="cuda"), "bf16", y.cuda(), y.shape[1],
                                           fmt, cd.cuda(), cd.stride(0), sd.cuda(), sd.stride(0), "bf16", D, ldd, M * ldd, 1)
    x = values(c.view(F8[fmt]).double(), s, N)
    m = torch.finfo(torch.bfloat16).max
    want = D0.clone()
    for i, r in ((0, 11), (1, 745)):
        want[i, i::3, :N] = (D0[i, i::3, :N].float() + x[r].clamp(-m, m).float() * 2.0 ** -12).bfloat16()
    assert torch.equal(D.cpu(), want)
