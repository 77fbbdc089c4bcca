"""GPU parity on sizes chosen for the kernel that they reach (route_cases.py): every kernel of the products over groups of
rows and of the adapters, in both types or every pairing, both outputs, with and without accumulation and epilogue.

Bounds as in the tests of each operator; for block-scaled calls with fast = 1 the window's loss is bounded without going
through the products: a block loses at most 31 * 2^-13 of its largest product, which is at most the block's largest
|a| times its largest |b|."""
import pytest
import torch

import block_scaled_matrix_amd as bsm
import route_cases as R
import test_gpu_grouped as dense
import test_gpu_lora as lora
from grouped_util import DT, HALF_STEP, offsets_of, up
from gpu_util import say
from test_gpu_grouped_mx import BITS, codes

pytestmark = pytest.mark.gpu
SILU = ("silu_affine", 0.5, 0.25)


def flat(table):
    return [pytest.param(name, *case, id=f"{name}-{case[-2]}-{case[-1]}") for name, cases in table.items() for case in cases]


@pytest.mark.parametrize("ab", ["bf16", "f16"])
@pytest.mark.parametrize("name,sizes,N,K,major", [pytest.param(*p.values, m, id=f"{p.id}-{m}") for p in flat(R.GROUPED)
                                                  for m in ("k" if p.values[0] in R.K_MAJOR_ONLY else "kn")])
def test_grouped(name, sizes, N, K, major, ab):
    rows = sum(sizes) + 3                            # (with the rows in no group)
    assert bsm.bsm_debug_grouped_route("g", rows, N, K, len(sizes), a_fmt=ab, b_major=major) == name
    dense.run(sizes, N, K, ab, major, ab, 0, None, 1, first=1, behind=2, extra=8)
    dense.run(sizes, N, K, ab, major, ab, 1, bsm.ewise_desc(*SILU), 2, first=1, behind=2)
    dense.run(sizes, N, K, ab, major, "f32", 1, None, 3, first=1, behind=2, extra=8)
    dense.run(sizes, N, K, ab, major, "f32", 0, bsm.ewise_desc(*SILU), 4, first=1, behind=2)


@pytest.mark.parametrize("ab", ["bf16", "f16"])
@pytest.mark.parametrize("name,sizes,M,N", flat(R.WGRAD))
def test_wgrad(name, sizes, M, N, ab):
    assert bsm.bsm_debug_grouped_route("w", sum(sizes) + 3, N, n=len(sizes), M=M, a_fmt=ab) == name
    for d, accum, extra in (("f32", 0, 0), ("f32", 1, 8), (ab, 0, 8), (ab, 1, 0)):
        dense.wgrad(sizes, M, N, ab, d, accum, 5, first=1, behind=2, extra=extra, pad=extra)


@pytest.mark.parametrize("name,a,b,fast,sizes,N,K", [pytest.param(name, *pair, *case, id=f"{name}-{'-'.join(map(str, pair))}-{case[2]}")
                                                     for name, (pairs, cases) in R.MX.items() for case in cases for pair in pairs])
def test_block_scaled(name, a, b, fast, sizes, N, K):
    g = torch.Generator().manual_seed(K + len(sizes))
    off, G = offsets_of(sizes, 1), len(sizes)
    rows = off[-1] + 2
    assert bsm.bsm_debug_grouped_route("m", rows, N, K, G, a_fmt=a, b_fmt=b, fast=fast) == name
    x, xs, xv = codes(g, (rows,), K, a, 16)
    w, ws, wv = codes(g, (G, N), K, b, 16)
    xs[0] = xs[off[-1]:] = 255
    ref, mag, lost = (torch.zeros(rows, N, dtype=torch.float64) for _ in range(3))
    top = lambda v: v.abs().unflatten(-1, (-1, 32)).amax(-1)
    for i in range(G):
        lo, hi = off[i], off[i + 1]
        ref[lo:hi], mag[lo:hi] = xv[lo:hi] @ wv[i].T, xv[lo:hi].abs() @ wv[i].abs().T
        if fast and (a, b) != ("e2m1", "e2m1"):
            lost[lo:hi] = 31 * 2.0 ** -13 * (top(xv[lo:hi]) @ top(wv[i]).T)
    dev = [t.cuda() for t in (x, xs, w, ws)]
    od = torch.tensor(off, dtype=torch.int32, device="cuda")
    inside = torch.zeros(rows, dtype=torch.bool)
    inside[off[0]:off[-1]] = True
    for d, accum, ew, extra in (("bf16", 0, None, 8), ("bf16", 1, SILU, 0), ("f32", 1, None, 8), ("f32", 0, SILU, 0), ("f32", 1, SILU, 4)):
        ldd = up(N, 4 if d == "f32" else 8) + extra
        D0 = (K ** 0.5 * 10 * torch.randn(rows, ldd, generator=g)).to(DT[d])
        D = D0.cuda()
        say("grouped mx", name, G, rows, N, K, a, b, fast, d, accum, ew)
        bsm.bsm_gemm_grouped_block_scale(rows, N, K, G, od, a, dev[0], dev[0].stride(0) * 8 // BITS[a], dev[1], dev[1].stride(0), b,
                                         dev[2], dev[2].stride(1) * 8 // BITS[b], dev[2].stride(0) * 8 // BITS[b], dev[3],
                                         dev[3].stride(1), dev[3].stride(0), fast, d, D, ldd, accum,
                                         bsm.ewise_desc(*ew) if ew else None)
        torch.cuda.synchronize()
        got = D.cpu()
        want, tol = ref, 1e-5 * mag + lost
        if accum:
            want = want + D0[:, :N].double()
            tol = tol + 2.0 ** -23 * (mag + D0[:, :N].double().abs())
        if ew:           # slope of silu below 1.1, a few ulp of silu, two roundings
            tol = 1.1 * abs(ew[1]) * tol + 6 * 2.0 ** -23 * (abs(ew[1]) * want.abs() + abs(ew[2]))
            want = want / (1 + torch.exp(-want)) * ew[1] + ew[2]
        tol = tol + HALF_STEP[d] * want.abs() * (1 + 2.0 ** -7)
        bad = ~((got[:, :N].double() - want).abs() <= tol)
        bad[~inside] = False
        assert not bad.any(), (d, accum, ew, int(bad.sum()), bad.nonzero()[:4].tolist())
        same = lambda u, v: torch.equal(u.contiguous().view(torch.uint8), v.contiguous().view(torch.uint8))
        assert same(got[~inside], D0[~inside]), "rows in no group were written"
        assert same(got[:, N:], D0[:, N:]), "columns past N were written"


@pytest.mark.parametrize("ab", ["bf16", "f16"])
@pytest.mark.parametrize("names,rows,N,K,rank,n", [pytest.param(names, *c, id=f"{names[0]}-{names[1]}-{c[0]}")
                                                   for names, cases in R.LORA.items() for c in cases])
def test_adapters(names, rows, N, K, rank, n, ab):
    route = lambda shrink: bsm.bsm_debug_grouped_route("a", rows, N, K, n, R=rank, a_fmt=ab, shrink=shrink)
    assert (route(0), route(1)) == names
    runs = [(t // 37) % (n + 1) - 1 for t in range(rows)]
    lora.run(lora.mixed(rows, n, 5), N, K, rank, n, ab, seed=rows, extra=8)
    lora.run(runs, N, K, rank, n, ab, "f32", 1, seed=K)
    lora.run(runs, N, K, rank, n, ab, ab, 0, bsm.ewise_desc(*SILU), seed=N)


@pytest.mark.parametrize("name,a,b,fast,sizes,N,K", [pytest.param(name, *pair, *cases[-1], id=f"{name}-{'-'.join(map(str, pair))}")
                                                     for name, (pairs, cases) in R.MX.items() for pair in pairs])
def test_block_scaled_wide_scales_and_nan(name, a, b, fast, sizes, N, K):
    """Scales over most of E8M0's range (an operand's large where the other's is small) keep the bound, and NaN element
    codes or scales in rows at the groups' ends and in one weight row make their own outputs NaN and no others."""
    g = torch.Generator().manual_seed(K)
    off, G = offsets_of(sizes), len(sizes)
    rows = off[-1]
    x, xs, xv = codes(g, (rows,), K, a)
    w, ws, wv = codes(g, (G, N), K, b)
    nb = K // 32
    unit = lambda v, s: v / torch.exp2(s[..., :nb].double() - 127).repeat_interleave(32, -1)
    xv, wv = unit(xv, xs), unit(wv, ws)
    shift = torch.randint(-95, 96, (nb,), generator=g)
    xs[:, :nb] = (torch.randint(125, 130, (rows, nb), generator=g) + shift).to(torch.uint8)
    ws[..., :nb] = (torch.randint(125, 130, (G, N, nb), generator=g) - shift).to(torch.uint8)
    # the reference without the shifts, which cancel in every product
    xv = xv * torch.exp2(xs[:, :nb].double() - shift - 127).repeat_interleave(32, -1)
    wv = wv * torch.exp2(ws[..., :nb].double() + shift - 127).repeat_interleave(32, -1)
    nan_rows, (ng, nn) = [off[1] - 1, off[-2]], (next(i for i in range(G) if sizes[i] > 1), N // 2)
    if a == "e4m3":
        x[nan_rows[0], 40], xs[nan_rows[1], nb - 1] = 0xFF, 255
    else:
        xs[nan_rows[0], 1], xs[nan_rows[1], nb - 1] = 255, 255
    if b == "e4m3":
        w[ng, nn, K - 1] = 0x7F
    else:
        ws[ng, nn, 3] = 255
    D = torch.empty(rows, up(N, 4), device="cuda")
    dev = [t.cuda() for t in (x, xs, w, ws)]
    say("grouped mx, wide scales", name, a, b, fast)
    assert bsm.bsm_debug_grouped_route("m", rows, N, K, G, a_fmt=a, b_fmt=b, fast=fast) == name
    bsm.bsm_gemm_grouped_block_scale(rows, N, K, G, torch.tensor(off, dtype=torch.int32, device="cuda"), a, dev[0],
                                     dev[0].stride(0) * 8 // BITS[a], dev[1], dev[1].stride(0), b, dev[2],
                                     dev[2].stride(1) * 8 // BITS[b], dev[2].stride(0) * 8 // BITS[b], dev[3], dev[3].stride(1),
                                     dev[3].stride(0), fast, "f32", D, D.stride(0))
    got = D.cpu()[:, :N].double()
    want = torch.zeros(rows, N, dtype=torch.bool)
    want[nan_rows] = True
    want[off[ng]:off[ng + 1], nn] = True
    assert torch.equal(torch.isnan(got), want)
    top = lambda v: v.abs().unflatten(-1, (-1, 32)).amax(-1)
    for i in range(G):
        lo, hi = off[i], off[i + 1]
        if lo == hi:
            continue
        tol = 1e-5 * (xv[lo:hi].abs() @ wv[i].abs().T)
        if fast and (a, b) != ("e2m1", "e2m1"):
            tol = tol + 31 * 2.0 ** -13 * (top(xv[lo:hi]) @ top(wv[i]).T)
        bad = ~((got[lo:hi] - xv[lo:hi] @ wv[i].T).abs() <= tol) & ~want[lo:hi]
        assert not bad.any(), (i, int(bad.sum()), bad.nonzero()[:4].tolist())


@pytest.mark.parametrize("name,sizes,N,K,major", [pytest.param(*p.values, m, id=f"{p.id}-{m}") for p in flat({n: c[-1:] for n, c in R.GROUPED.items()})
                                                  for m in ("k" if p.values[0] in R.K_MAJOR_ONLY else "kn")])
def test_grouped_nan_and_infinity_stay_in_place(name, sizes, N, K, major):
    """A NaN in a group's last row, an infinity in the next group's first and a NaN in one weight: their own outputs only."""
    g = torch.Generator().manual_seed(K)
    off, G = offsets_of(sizes), len(sizes)
    rows = off[-1]
    x, w = torch.randn(rows, K, generator=g).bfloat16(), torch.rand(G, N, K, generator=g).bfloat16() + 0.5
    at = next(i for i in range(G - 1) if sizes[i] and sizes[i + 1])
    x[off[at + 1] - 1, K - 1], x[off[at + 1], 0], w[G - 1, N // 2, K // 3] = float("nan"), float("inf"), float("nan")
    want_nan = torch.zeros(rows, N, dtype=torch.bool)
    want_nan[off[at + 1] - 1] = True
    want_nan[off[G - 1]:, N // 2] = True
    want_inf = torch.zeros(rows, N, dtype=torch.bool)
    want_inf[off[at + 1]] = True
    want_inf &= ~want_nan
    wm = w if major == "k" else w.transpose(1, 2).contiguous()
    xd, wd = dense.padded(x).cuda(), dense.padded(wm).cuda()
    D = torch.empty(rows, up(N, 4), device="cuda")
    assert bsm.bsm_debug_grouped_route("g", rows, N, K, G, b_major=major) == name
    say("grouped, NaN", name, N, K, major)
    bsm.bsm_gemm_grouped(rows, N, K, G, torch.tensor(off, dtype=torch.int32, device="cuda"), "bf16", xd, xd.stride(0), wd,
                         wd.stride(1), major, wd.stride(0), "f32", D, D.stride(0))
    got = D.cpu()[:, :N]
    assert torch.equal(torch.isnan(got), want_nan)
    assert torch.equal(got == float("inf"), want_inf) and not (got == -float("inf")).any()


@pytest.mark.parametrize("name,sizes,M,N", flat(R.WGRAD))
def test_wgrad_nan_and_infinity_stay_in_place(name, sizes, M, N):
    """The same for the weight gradient: a row's NaN and infinity reach its own group's row and column."""
    g = torch.Generator().manual_seed(M)
    off, G = offsets_of(sizes), len(sizes)
    rows = off[-1]
    y, x = torch.randn(rows, M, generator=g).bfloat16(), torch.rand(rows, N, generator=g).bfloat16() + 0.5
    last = max(i for i in range(G) if sizes[i])
    y[off[1] - 1, M - 1], x[off[last], 0], y[off[last], 0] = float("nan"), float("nan"), float("inf")
    want = torch.zeros(G, M, N, dtype=torch.bool)
    want[0, M - 1] = True
    want[last, :, 0] = True
    inf = torch.zeros_like(want)
    inf[last, 0, 1:] = True
    inf &= ~want
    yd, xd = dense.padded(y).cuda(), dense.padded(x).cuda()
    D = torch.empty(G, M, up(N, 4), device="cuda")
    assert bsm.bsm_debug_grouped_route("w", rows, N, n=G, M=M) == name
    say("wgrad, NaN", name, M, N)
    bsm.bsm_gemm_grouped_wgrad(rows, M, N, G, torch.tensor(off, dtype=torch.int32, device="cuda"), "bf16", yd, yd.stride(0), xd,
                               xd.stride(0), "f32", D, D.stride(1), D.stride(0))
    got = D.cpu()[..., :N]
    assert torch.equal(torch.isnan(got), want)
    assert torch.equal(got == float("inf"), inf) and not (got == -float("inf")).any()
