"""GPU parity: activations kept in 8 bits, restored, and the activation's gradient, against 64 bits.

Codes, scales and restored values are exact: x 2^-e has no rounding, so the code is the one rounding to nearest even of
the definition, and a code times its scale fits the outputs. The slope of silu is s (1 + x (1 - s)) with s = 1 / (1 + e^-x):
the exponential is off by at most 8 u (u = 2^-24), s and 1 - s by 20 u, the sum's two terms and the last products by
less than 48 u of s + |x| s (1 - s); then dY's product and the output's half step.
"""
import pytest
import torch

import block_scaled_matrix_amd as bsm
from grouped_util import DT, HALF_STEP, up
from gpu_util import say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FORMAT = {"e4m3": (3, -6, 448.0), "e5m2": (2, -14, 57344.0)}     # fraction bits, least exponent, largest value


def grid(y, fmt):
    """y (64-bit, inside the format's range) rounded to nearest even."""
    mb, low, _ = FORMAT[fmt]
    e = torch.frexp(y.abs().clamp_min(2.0 ** low)).exponent - 1
    step = torch.ldexp(torch.ones_like(y), e - mb)
    return torch.round(y / step) * step


def kept(x, fmt):
    """Values of the codes (64-bit, before the scale) and scale codes of x by the definition."""
    rows, K = x.shape
    b = torch.nn.functional.pad(x.double(), (0, -K % 32)).view(rows, -1, 32)
    top = torch.where(torch.isfinite(b), b.abs(), 0.0).amax(-1)
    m, e = torch.frexp(top / FORMAT[fmt][2])
    e = torch.where(m == 0.5, e - 1, e).clamp_min(-127)
    e = torch.where(top == 0, -127, e)
    y = b * torch.ldexp(torch.ones_like(b), -e[..., None])
    v = torch.where(torch.isfinite(y), grid(torch.where(torch.isfinite(y), y, 0.0), fmt), y)
    if fmt == "e4m3":
        v = torch.where(torch.isinf(v), torch.nan, v)
    return v.flatten(1)[:, :K], e + 127


def same(a, b):
    return torch.equal(torch.nan_to_num(a.double(), nan=1e300), torch.nan_to_num(b.double(), nan=1e300)) and \
        torch.equal(torch.isnan(a), torch.isnan(b))


def buffers(x, x_fmt, extra=0):
    rows, K = x.shape
    q = 4 if x_fmt == "f32" else 8
    X = torch.full((rows, up(K, q) + extra * q), float("nan"), dtype=DT[x_fmt])
    X[:, :K] = x
    Q = torch.full((rows, up(K, 16) + 16 * extra), 0xA5, dtype=torch.uint8)
    S = torch.full((rows, up((K + 31) // 32, 4) + 4 * extra), 0xA5, dtype=torch.uint8)
    return X.cuda(), Q.cuda(), S.cuda()


def save(x, x_fmt, fmt, extra=0, stream=None):
    rows, K = x.shape
    X, Q, S = buffers(x, x_fmt, extra)
    say("save", rows, K, x_fmt, fmt, extra)
    bsm.bsm_block_scale_save(rows, K, x_fmt, X, X.stride(0), fmt, Q, Q.stride(0), S, S.stride(0), stream)
    torch.cuda.synchronize()
    nb = (K + 31) // 32
    assert (Q[:, K:] == 0xA5).all() and (S[:, nb:] == 0xA5).all(), "padding was written"
    return Q, S, Q.cpu()[:, :K].contiguous().view(F8[fmt]).double(), S.cpu()[:, :nb]


def check_save(x, x_fmt, fmt, extra=0):
    Q, S, v, s = save(x, x_fmt, fmt, extra)
    rv, rs = kept(x, fmt)
    assert torch.equal(s.long(), rs.long())
    assert same(v, rv)
    return Q, S, rv, rs


def values(v, s, K):
    return v * torch.ldexp(torch.ones(s.shape, dtype=torch.float64), s.int() - 127).repeat_interleave(32, 1)[:, :K]


def rounded(v, d):
    m = torch.finfo(DT[d]).max
    v = torch.where(torch.isfinite(v), v.clamp(-m, m), v) if d == "f16" else v
    return v.float().to(DT[d]) if d != "f32" else v.float()


def check_restore(Q, S, v, s, fmt, d, ew=None):
    rows, K = v.shape
    D = torch.full((rows, up(K, 4 if d == "f32" else 8) + 8), 7.0, dtype=DT[d], device="cuda")
    say("restore", rows, K, fmt, d)
    bsm.bsm_block_scale_restore(rows, K, fmt, Q, Q.stride(0), S, S.stride(0), d, D, D.stride(0), ew)
    torch.cuda.synchronize()
    got = D.cpu()
    assert (got[:, K:] == 7.0).all()
    x = values(v, s, K)
    if ew is None:
        assert same(got[:, :K], rounded(x, d))
        return
    ref = x / (1 + torch.exp(-x)) * ew.scale + ew.bias
    # silu within 4 ulp (8 u), the affine map's rounding, the output's
    tol = (12 * U) * (abs(ew.scale) * (x / (1 + torch.exp(-x))).abs() + abs(ew.bias)) + HALF_STEP[d] * ref.abs() * 1.01 + 2.0 ** -25
    assert ((got[:, :K].double() - ref).abs() <= tol).all()


def check_grad(Q, S, v, s, fmt, d, scale=1.25, inplace=False, op="silu_affine", seed=0):
    rows, K = v.shape
    g = torch.Generator().manual_seed(seed)
    dy = torch.randn(rows, up(K, 4 if d == "f32" else 8), generator=g).to(DT[d])
    Y = dy.cuda()
    D = Y if inplace else torch.full((rows, Y.shape[1] + 8), 7.0, dtype=DT[d], device="cuda")
    say("ewise grad", rows, K, fmt, d, inplace)
    bsm.bsm_block_scale_ewise_grad(rows, K, fmt, Q, Q.stride(0), S, S.stride(0), d, Y, Y.stride(0), D, D.stride(0),
                                   bsm.ewise_desc(op, scale, 0.5))
    torch.cuda.synchronize()
    got = D.cpu()
    if not inplace:
        assert (got[:, K:] == 7.0).all()
    y, x = dy[:, :K].double(), values(v, s, K)
    if op == "none":
        assert torch.equal(got[:, :K].double(), y)
        return
    a, b = torch.sigmoid(x), torch.sigmoid(-x)
    xb = torch.where(torch.isinf(x), 0.0, x * a * b)
    ref = y * scale * (a + xb)
    tol = y.abs() * abs(scale) * (a + xb.abs()) * 52 * U + HALF_STEP[d] * ref.abs() * 1.01 + (2.0 ** -25 if d == "f16" else 2.0 ** -118)
    ok = ((got[:, :K].double() - ref).abs() <= tol) | (torch.isnan(ref) & torch.isnan(got[:, :K]))
    assert ok.all()


def spread(rows, K, x_fmt, seed):
    """Values over many powers of two, zero blocks among them."""
    g = torch.Generator().manual_seed(seed)
    e = {"f16": 8.0, "bf16": 60.0, "f32": 60.0}[x_fmt]
    x = torch.randn(rows, K, generator=g) * torch.exp2((torch.rand(rows, -(-K // 32), generator=g) * 2 - 1) * e).repeat_interleave(32, 1)[:, :K]
    x *= torch.exp2(-torch.rand(rows, K, generator=g) * 12)
    x[::3, 32:64] = 0
    return x.to(DT[x_fmt])


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("x_fmt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 32), (3, 31), (2, 33), (5, 36), (7, 100), (129, 96), (64, 1000), (33, 2048), (3, 8193)])
def test_round_trip(rows, K, x_fmt, fmt):
    Q, S, v, s = check_save(spread(rows, K, x_fmt, rows + K), x_fmt, fmt, extra=rows % 2)
    check_restore(Q, S, v, s, fmt, x_fmt)
    check_grad(Q, S, v, s, fmt, x_fmt, inplace=K % 2 == 0)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_every_f16_value(fmt):
    """Each finite and infinite f16 pattern and the NaN, in a block of its own sign and in one with the largest value."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.float16)
    check_save(bits.view(-1, 32), "f16", fmt)
    x = bits.view(-1, 1).repeat(1, 32)
    x[:, 1] = 448.0
    x[:, 2] = 1.0
    Q, S, v, s = check_save(x, "f16", fmt)
    for d in ("f16", "bf16", "f32"):
        check_restore(Q, S, v, s, fmt, d)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_scale_edges(fmt):
    """Blocks whose largest value lies at, below and above the format's largest times a power of two, and at float32's ends."""
    top = FORMAT[fmt][2]
    rows = []
    for e in list(range(-149, 120, 7)) + [118, 119, 112, 111]:
        for f in (1.0, 1 - 2.0 ** -23, 1 + 2.0 ** -23, 8 / 7, 0.5):
            a = torch.tensor(top * f, dtype=torch.float64) * 2.0 ** e
            if float(a) < 3.4e38:
                rows.append(torch.cat((a.view(1), a.view(1) * torch.rand(31, dtype=torch.float64))))
    tiny = torch.tensor([2.0 ** -149, 2.0 ** -140, 2.0 ** -126, 3.4028234663852886e38], dtype=torch.float64)
    rows += [torch.cat((t.view(1), torch.zeros(31, dtype=torch.float64))) for t in tiny]
    x = torch.stack(rows).float()
    Q, S, v, s = check_save(x, "f32", fmt)
    check_restore(Q, S, v, s, fmt, "f32")


@pytest.mark.parametrize("x_fmt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_not_finite(fmt, x_fmt):
    x = torch.randn(8, 96).to(DT[x_fmt])
    x[1, 3], x[2, 40], x[3, 70] = float("nan"), float("inf"), -float("inf")
    x[4] = float("inf")
    x[5] = float("nan")
    Q, S, v, s = check_save(x, x_fmt, fmt)
    check_restore(Q, S, v, s, fmt, x_fmt)
    check_grad(Q, S, v, s, fmt, x_fmt)


def test_scale_codes_read_from_elsewhere():
    """Codes of another maker: every scale code, 0xFF making its block NaN."""
    for fmt in ("e4m3", "e5m2"):
        codes = torch.arange(256, dtype=torch.uint8).view(8, 32).repeat(32, 1)     # every code under every scale
        s = torch.arange(256, dtype=torch.uint8).view(256, 1)
        S = torch.zeros(256, 4, dtype=torch.uint8)
        S[:, :1] = s
        v = codes.view(F8[fmt]).double()
        x = values(v, s, 32)
        x[255] = float("nan")
        D = torch.empty(256, 32, device="cuda")
        bsm.bsm_block_scale_restore(256, 32, fmt, codes.cuda(), 32, S.cuda(), 4, "f32", D, 32)
        assert same(D.cpu(), x.float())


@pytest.mark.parametrize("d", ["bf16", "f16", "f32"])
def test_activation_made_again(d):
    x = torch.randn(40, 200).to(DT[d]) * 3
    Q, S, v, s = check_save(x, d, "e4m3")
    check_restore(Q, S, v, s, "e4m3", d, bsm.ewise_desc("silu_affine", 1.5, -0.25))
    check_grad(Q, S, v, s, "e4m3", d, op="none")
    Q, S, v, s = check_save(x, d, "e5m2")
    check_restore(Q, S, v, s, "e5m2", d, bsm.ewise_desc("silu_affine", 1.5, -0.25))


def test_slope_over_its_range():
    x = torch.cat((torch.linspace(-120, 120, 4096), torch.linspace(-2, 2, 4096))).view(-1, 32)
    for d in ("f32", "bf16"):
        Q, S, v, s = check_save(x, "f32", "e4m3")
        check_grad(Q, S, v, s, "e4m3", d, scale=-0.5)


def test_gradient_against_differences():
    x = torch.linspace(-6, 6, 96).view(3, 32)
    Q, S, v, s = check_save(x, "f32", "e4m3")
    z = values(v, s, 32)
    dy = torch.ones(3, 32, device="cuda")
    D = torch.empty(3, 32, device="cuda")
    bsm.bsm_block_scale_ewise_grad(3, 32, "e4m3", Q, Q.stride(0), S, S.stride(0), "f32", dy, 32, D, 32, bsm.ewise_desc("silu_affine", 2.0, 1.0))
    f = lambda t: 2 * t / (1 + torch.exp(-t)) + 1
    h = 1e-5
    assert ((f(z + h) - f(z - h)) / (2 * h) - D.cpu().double()).abs().max() < 1e-6


def test_f16_at_the_end_of_its_range():
    """65504 is kept as 65536 and comes back as 65504, not as infinity."""
    x = torch.full((2, 32), 65504.0).half()
    Q, S, v, s = check_save(x, "f16", "e4m3")
    assert float(values(v, s, 32)[0, 0]) == 65536.0
    check_restore(Q, S, v, s, "e4m3", "f16")


def ends(v, s, K, d):
    """values() in the format d, finite ones beyond its range its largest (codes and scales of any maker)."""
    x = values(v, s, K)
    m = torch.finfo(DT[d]).max
    return torch.where(torch.isfinite(x), x.clamp(-m, m), x).to(DT[d])


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("d", ["bf16", "f16"])
def test_every_code_under_every_scale_in_16_bits(d, fmt):
    """Finite values beyond the range come back as its largest, infinite codes as infinity."""
    codes = torch.arange(256, dtype=torch.uint8).view(8, 32).repeat(256, 1)
    s = torch.arange(256, dtype=torch.uint8).repeat_interleave(8).view(-1, 1)
    S = torch.zeros(2048, 4, dtype=torch.uint8)
    S[:, :1] = s
    want = ends(codes.view(F8[fmt]).double(), s, 32, d)
    want[s[:, 0] == 255] = float("nan")
    D = torch.empty(2048, 32, dtype=DT[d], device="cuda")
    say("restore every code", d, fmt)
    bsm.bsm_block_scale_restore(2048, 32, fmt, codes.cuda(), 32, S.cuda(), 4, d, D, 32)
    assert same(D.cpu(), want)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("x_fmt", ["bf16", "f32"])
def test_lowest_value_of_the_type(x_fmt, fmt):
    """A mask's fill, kept as a code that stands for -2^128, comes back finite in 16 bits."""
    low = torch.finfo(DT[x_fmt]).min
    x = torch.randn(6, 64).to(DT[x_fmt])
    x[1:, 5:40] = low
    x[3] = low
    x[4, 50] = -low
    Q, S, v, s = check_save(x, x_fmt, fmt)
    assert float(values(v, s, 64).min()) == -2.0 ** 128
    for d in ("bf16", "f16"):
        D = torch.empty(6, 64, dtype=DT[d], device="cuda")
        bsm.bsm_block_scale_restore(6, 64, fmt, Q, Q.stride(0), S, S.stride(0), d, D, 64)
        assert same(D.cpu(), ends(v, s, 64, d)) and torch.isfinite(D).all()


@pytest.mark.parametrize("d", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_activation_of_values_beyond_float32(fmt, d):
    """f of a code that stands for +-2^128 or more: f's limit below, the largest value (float32: infinity) above."""
    big = 0x78                                          # 256 and 32768
    codes = torch.full((4, 32), big, dtype=torch.uint8)
    codes[1], codes[2], codes[3] = big | 0x80, 0x30, 0x7F
    S = torch.full((4, 4), 127 + (120 if fmt == "e4m3" else 113), dtype=torch.uint8)
    D = torch.empty(4, 32, dtype=DT[d], device="cuda")
    say("activation beyond float32", d, fmt)
    bsm.bsm_block_scale_restore(4, 32, fmt, codes.cuda(), 32, S.cuda(), 4, d, D, 32, bsm.ewise_desc("silu_affine", 1.5, -0.25))
    m = float("inf") if d == "f32" else torch.finfo(DT[d]).max
    got = D.cpu().float()
    mid = float(codes[2, 0].view(F8[fmt]).float()) * 2.0 ** (120 if fmt == "e4m3" else 113) * 1.5
    assert (got[0] == m).all() and (got[1] == -0.25).all() and torch.isnan(got[3]).all()
    assert (got[2] == (m if d == "f16" else mid)).all()
    bsm.bsm_block_scale_restore(4, 32, fmt, codes.cuda(), 32, S.cuda(), 4, d, D, 32, bsm.ewise_desc("silu_affine", 2.0 ** -10, 0.0))
    if d == "bf16":      # 2^128 counts as float32's largest: 2^-10 of it is 2^118 in bf16
        assert (D[0].float() == 2.0 ** 118).all() and not D[1].any()


def test_long_rows_and_many_rows():
    """More than 2^31 elements: past 32-bit offsets."""
    rows, K = 1 << 16, 32800
    X = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    X[-1, -40:] = torch.arange(40, device="cuda").bfloat16()
    Q = torch.empty(rows, K, dtype=torch.uint8, device="cuda")
    S = torch.empty(rows, 1028, dtype=torch.uint8, device="cuda")
    say("save past 2^31")
    bsm.bsm_block_scale_save(rows, K, "bf16", X, K, "e4m3", Q, K, S, 1028)
    X.fill_(3.0)
    bsm.bsm_block_scale_restore(rows, K, "e4m3", Q, K, S, 1028, "bf16", X, K)
    v, s = kept(torch.cat((torch.zeros(24), torch.arange(40).float())).view(1, 64), "e4m3")
    assert torch.equal(X[-1, -64:].cpu().double(), values(v, s, 64)[0]) and not X[:-1].any() and not X[-1, :-64].any()
