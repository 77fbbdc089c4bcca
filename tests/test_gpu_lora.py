"""GPU parity: a shared projection with a low-rank adapter chosen per row, against 64 bits.

Bound: the projection's sum of K terms and the adapter's of R terms are float32 sums as in grouped_util; U
carries the error of its own K-term sum and the rounding of its scaling, (K + 2) 2^-23 of sum|x a|, through
LB, so the adapter's part is off by at most (K + R + 4) 2^-23 of its sum of magnitudes."""
import pytest
import torch

import block_scaled_matrix_amd as bsm
from grouped_util import DT, check, padded, silu_affine, up
from gpu_util import say

pytestmark = pytest.mark.gpu


def run(ids, N, K, R, L, ab="bf16", d=None, accum=0, ew=None, seed=0, extra=0, bad=None):
    d = d or ab
    g = torch.Generator().manual_seed(seed)
    T = len(ids)
    mk = lambda *s: torch.randn(*s, generator=g).to(DT[ab])
    x, w, la, lb = mk(T, K), mk(N, K), mk(L, R, K), mk(L, N, R)
    scale = torch.rand(L, generator=g) + 0.5
    if bad is not None:                       # an adapter that no checked row may feel
        la[bad], lb[bad] = float("inf"), float("nan")
    ldd = up(N, 4 if d == "f32" else 8) + (8 if extra else 0)
    D0 = torch.randn(T + 2, ldd, generator=g).to(DT[d])
    xd, wd, lad, lbd = (padded(t, 8, extra).cuda() for t in (x, w, la, lb))
    D = D0.cuda()
    nbytes = bsm.bsm_gemm_lora_workspace(T, R)
    ws = torch.full((nbytes + 64,), 0xFF, dtype=torch.uint8, device="cuda")     # NaN, and a guard behind
    say("lora", T, N, K, R, L, ab, d, accum)
    bsm.bsm_gemm_lora(T, N, K, R, L, torch.tensor(ids, dtype=torch.int32, device="cuda"), ab, xd, xd.stride(0), wd, wd.stride(0),
                      lad, lad.stride(1), lad.stride(0), lbd, lbd.stride(1), lbd.stride(0), scale.cuda(), ws, d, D, ldd, accum, ew)
    torch.cuda.synchronize()
    assert (ws[nbytes:] == 0xFF).all(), "written past the workspace"
    X, W = x.double(), w.double()
    ref, mag = X @ W.T, X.abs() @ W.abs().T
    for t, a in enumerate(ids):
        if 0 <= a < L and a != bad:
            u, um = X[t] @ la[a].double().T, X[t].abs() @ la[a].double().abs().T
            ref[t] += scale[a].double() * (u @ lb[a].double().T)
            mag[t] += scale[a].double() * (um @ lb[a].double().abs().T)
    if accum:
        ref, mag = ref + D0[:T, :N].double(), mag + D0[:T, :N].double().abs()
    if ew is not None:
        mag = 1.1 * abs(ew.scale) * mag + (abs(ew.scale) * ref.abs() + abs(ew.bias)) * 6 / (K + R + 2)
        ref = silu_affine(ref, ew.scale, ew.bias)
    got = D.cpu()
    keep = [t for t in range(T) if bad is None or ids[t] != bad]
    check(got[:T, :N][keep], ref[keep], mag[keep], K + R + 4, d, (T, N, K, R))
    assert torch.equal(got[T:], D0[T:]) and torch.equal(got[:T, N:], D0[:T, N:]), "untouched memory was written"
    return got[:T, :N]


def mixed(T, L, seed=1, none=4):
    g = torch.Generator().manual_seed(seed)
    return [int(v) - 1 if int(v) % none else -1 for v in torch.randint(0, L + 1, (T,), generator=g)]


@pytest.mark.parametrize("ab", ["bf16", "f16"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 48, 64, 65, 130, 300])
def test_rows(T, ab):
    run(mixed(T, 7, T), 136, 200, 16, 7, ab, seed=T)


@pytest.mark.parametrize("ab", ["bf16", "f16"])
@pytest.mark.parametrize("R", [1, 4, 8, 15, 16, 17, 32, 40, 64, 100, 128, 256])
def test_ranks(R, ab):
    run(mixed(21, 3, R), 72, 96, R, 3, ab, "f32", seed=R)
    run([2] * 70 + [0] * 70, 72, 96, R, 3, ab, seed=R)


@pytest.mark.parametrize("N,K", [(1, 1), (7, 33), (63, 65), (257, 129), (1000, 520), (24, 2048), (130, 1003)])
@pytest.mark.parametrize("T", [3, 40, 150])
def test_odd_sizes(T, N, K):
    run(mixed(T, 5), N, K, 12, 5, "bf16", seed=N, extra=8)


@pytest.mark.parametrize("T", [5, 50, 200])
def test_outputs_accumulate_and_epilogue(T):
    for ab, d in (("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")):
        run(mixed(T, 4), 200, 96, 8, 4, ab, d, 1, None, 3)
        run(mixed(T, 4), 200, 96, 8, 4, ab, d, 0, bsm.ewise_desc("silu_affine", 1.5, -0.25), 4)


@pytest.mark.parametrize("T", [16, 64, 256])
def test_every_row_its_own_adapter(T):
    run(list(range(T)), 72, 64, 8, T)
    run(list(range(T))[::-1], 72, 64, 8, T)


def test_rows_without_an_adapter():
    run([-1] * 40, 72, 64, 8, 3)
    run([3, 100, -7, 2, 1 << 30], 72, 64, 8, 3)          # outside 0 .. 2: none
    run([0, 1, 2], 72, 64, 0, 3)                         # rank 0


def test_no_adapters_and_empty_k():
    run([-1] * 20, 72, 64, 0, 1)
    run([0, 1] * 10, 40, 0, 8, 2, "bf16", "f32", 1)


@pytest.mark.parametrize("T", [16, 60, 200])
def test_a_broken_adapter_stays_with_its_rows(T):
    """Infinities and NaN in one adapter's weights do not reach rows of other adapters, or of none, beside it."""
    got = run(mixed(T, 5, 3), 72, 64, 8, 5, bad=2)
    ids = mixed(T, 5, 3)
    assert all(bool(torch.isnan(got[t]).all()) for t in range(T) if ids[t] == 2)


def test_same_bits_every_time():
    a = run(mixed(100, 6), 264, 520, 24, 6, seed=8)
    for _ in range(3):
        assert torch.equal(run(mixed(100, 6), 264, 520, 24, 6, seed=8), a)


@pytest.mark.parametrize("T,N", [(70, 4200), (200, 1500), (3300, 1100), (260, 520)])
@pytest.mark.parametrize("K", [64, 100, 264])
def test_tile_shapes(T, N, K):
    """Few tiles (two sets of waves a tile) and many, requests of several rows each, ranks of one step and more."""
    ids = [(t // 37) % 4 - 1 for t in range(T)]
    run(ids, N, K, 24, 3, "bf16", seed=T)
    run(ids, N, K, 72, 3, "f16", "f32", seed=K)


@pytest.mark.parametrize("T,L,R", [(1100, 3, 24), (1100, 40, 24), (1300, 40, 130), (90, 3, 256)])
def test_shrink_by_rows_and_by_tiles(T, L, R):
    """Both forms of the shrink: few adapters and many, blocks of rows of one adapter and of many."""
    for N in (72, 1400):                    # (1400: too many workgroups of 16 columns)
        run(mixed(T, L, 2), N, 200, R, L, "bf16", seed=R)
        run([(t // 50) % L for t in range(T)], N, 200, R, L, "f16", "f32", seed=T)


def nonfinite_case(ids, N, ab, kind, bits, seed):
    """Operands with infinities and NaN in LB (`kind` "weight") or adapters of an infinite scale ("u", "both"), the values
    of U of few bits (small integers: its lower terms are zero, and so are some of its values) or of many, and the
    64-bit result by the definition, products one by one."""
    g = torch.Generator().manual_seed(seed)
    T, K, R, L = len(ids), 40, 12, 3
    few = lambda *s: torch.randint(-2, 3, s, generator=g).to(DT[ab])
    mk = few if bits == "few" else lambda *s: torch.randn(*s, generator=g).to(DT[ab])
    x, la, lb = mk(T, K), mk(L, R, K), mk(L, N, R)
    w = torch.randn(N, K, generator=g).to(DT[ab])
    scale = torch.tensor([1.0, 0.5, 2.0])
    if kind in ("weight", "both"):
        for a, n, r, v in ((0, 3, 0, "inf"), (0, 17, 11, "-inf"), (1, 0, 5, "-inf"), (1, N - 1, 3, "inf"), (1, 20, 2, "nan"),
                           (0, 30, 1, "inf"), (0, 30, 2, "-inf"), (2, 33, 7, "inf")):
            lb[a, n, r] = float(v)
    if kind in ("u", "both"):
        scale[1], scale[2] = float("inf"), float("-inf")
    if kind == "u":                                 # (sums of one sign: every output of adapters 1 and 2 infinite)
        x, la, lb = (t.abs().where(t != 0, torch.ones_like(t)) for t in (x, la, lb))
    u = scale[torch.tensor(ids).clamp_min(0), None].double() * torch.stack(
        [(x[t].double() * la[max(a, 0)].double()).sum(-1) for t, a in enumerate(ids)])
    ref, mag = torch.empty(T, N, dtype=torch.float64), torch.empty(T, N, dtype=torch.float64)
    for t, a in enumerate(ids):
        p = x[t].double() * w.double()
        q = u[t] * lb[max(a, 0)].double() if a >= 0 else torch.zeros(N, R, dtype=torch.float64)
        ref[t], mag[t] = p.sum(-1) + q.sum(-1), p.abs().sum(-1) + q.abs().sum(-1)
    if kind == "weight":                            # (U's own error reaches the finite outputs)
        um = torch.stack([(x[t].double() * la[max(a, 0)].double()).abs().sum(-1) * scale[max(a, 0)].double() for t, a in enumerate(ids)])
        for t, a in enumerate(ids):
            if a >= 0:
                mag[t] = (x[t].double() * w.double()).abs().sum(-1) + (um[t] * lb[a].double().abs()).sum(-1)
    return x, w, la, lb, scale, ref, mag, T, K, R, L


@pytest.mark.parametrize("ab", ["bf16", "f16"])
@pytest.mark.parametrize("kind", ["weight", "u", "both"])
@pytest.mark.parametrize("bits", ["few", "many"])
@pytest.mark.parametrize("T,N", [(16, 40), (64, 40), (200, 1500), (70, 4200), (3300, 1100)])
def test_infinities_follow_the_definition(T, N, bits, kind, ab):
    """An infinite weight or U gives what the formula gives, infinity or NaN, whichever kernel the sizes choose; the other
    outputs stay finite and within the bound."""
    ids = [(t // 37) % 4 - 1 if t % 5 else t % 3 for t in range(T)]
    x, w, la, lb, scale, ref, mag, T, K, R, L = nonfinite_case(ids, N, ab, kind, bits, T + N)
    xd, wd, lad, lbd = (padded(t).cuda() for t in (x, w, la, lb))
    D = torch.empty(T, up(N, 4), device="cuda")
    ws = torch.full((bsm.bsm_gemm_lora_workspace(T, R),), 0xFF, dtype=torch.uint8, device="cuda")
    say("lora, not finite", T, N, bits, kind, ab)
    bsm.bsm_gemm_lora(T, N, K, R, L, torch.tensor(ids, dtype=torch.int32, device="cuda"), ab, xd, xd.stride(0), wd, wd.stride(0),
                      lad, lad.stride(1), lad.stride(0), lbd, lbd.stride(1), lbd.stride(0), scale.cuda(), ws, "f32", D, D.stride(0))
    got = D.cpu()[:, :N].double()
    assert torch.isinf(ref).any() and torch.isfinite(ref).any()
    wrong = torch.isnan(got) != torch.isnan(ref)
    assert not wrong.any(), ("NaN", int(wrong.sum()), wrong.nonzero()[:4].tolist())
    wrong = torch.isinf(got) != torch.isinf(ref)
    wrong |= torch.isinf(ref) & (got != ref)
    assert not wrong.any(), ("infinity", int(wrong.sum()), wrong.nonzero()[:4].tolist())
    fine = torch.isfinite(ref)
    check(got[fine], ref[fine], mag[fine], K + R + 4, "f32", (T, N))
