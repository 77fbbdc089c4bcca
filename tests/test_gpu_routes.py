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
