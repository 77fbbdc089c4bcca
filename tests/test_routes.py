"""CPU tests: which kernel a call on groups of rows takes, and that the sizes of route_cases.py reach every one of them."""
import os
import re

import pytest

import block_scaled_matrix_amd as bsm
import route_cases as R

CSRC = os.path.join(os.path.dirname(bsm.__file__), "csrc")


@pytest.fixture(scope="module", autouse=True)
def L():
    if not os.path.exists(bsm.LIB_PATH):
        from block_scaled_matrix_amd import _build
        _build.build()
    return bsm.lib()


def test_every_case_takes_its_kernel():
    route = bsm.bsm_debug_grouped_route
    for name, cases in R.GROUPED.items():
        for sizes, N, K in cases:
            for major in "k" if name in R.K_MAJOR_ONLY else "kn":
                assert route("g", sum(sizes), N, K, len(sizes), b_major=major) == name, (sizes, N, K, major)
    for name, cases in R.WGRAD.items():
        for sizes, M, N in cases:
            assert route("w", sum(sizes), N, n=len(sizes), M=M) == name, (sizes, M, N)
    for name, (pairs, cases) in R.MX.items():
        for a, b, fast in pairs:
            for sizes, N, K in cases:
                assert route("m", sum(sizes), N, K, len(sizes), a_fmt=a, b_fmt=b, fast=fast) == name, (sizes, N, K, a, b, fast)
    for (name, shrink), cases in R.LORA.items():
        for rows, N, K, rank, n in cases:
            assert route("a", rows, N, K, n, R=rank) == name, (rows, N, K, rank, n)
            assert route("a", rows, N, K, n, R=rank, shrink=1) == shrink, (rows, N, K, rank, n)


def test_every_kernel_has_a_case():
    """Every kernel that the grouped and adapter sources launch, every tile of those that have several, and every pairing
    of each block-scaled kernel that takes several."""
    launched = set()
    for f in os.listdir(CSRC):
        if re.fullmatch(r"k_gemm_(grouped.*|lora)\.hip", f):
            launched |= set(re.findall(r"hipLaunchKernelGGL\(\(*(k_\w+)", open(os.path.join(CSRC, f)).read()))
    names = [*R.GROUPED, *R.WGRAD, *R.MX, *(n for pair in R.LORA for n in pair if n)]
    assert {n.split("<")[0] for n in names} == launched
    names_in_sources = set()
    for f in ("k_gemm_grouped.hip", "k_gemm_lora.hip", "k_gemm_grouped_mx.hip", "k_gemm_grouped_mx_mid.hip"):
        names_in_sources |= set(re.findall(r'"(k_[^"]+)"', open(os.path.join(CSRC, f)).read()))
    assert set(names) == names_in_sources
    for name, (pairs, _) in R.MX.items():
        if name in ("k_grouped_mx_split", "k_grouped_mx_mid"):
            assert pairs == R.PAIRS
    assert sorted(R.MX["k_gemm_mx"][0] + R.MX["k_gemm_mx_any"][0]) == sorted(R.PAIRS)


def test_refusals():
    for bad in (dict(rows=0), dict(rows=1 << 31), dict(N=0), dict(K=-1), dict(n=0), dict(n=65537), dict(call="w", M=0), dict(R=257)):
        with pytest.raises(bsm.BsmError) as e:
            bsm.bsm_debug_grouped_route(**{**dict(call="g", rows=10, N=10, K=10), **bad})
        assert e.value.status == "BSM_E_SHAPE", bad
    with pytest.raises(bsm.BsmError) as e:
        bsm.bsm_debug_grouped_route("x", 10, 10)
    assert e.value.status == "BSM_E_ARG"


def test_large_tiles_only_where_they_fill_the_chip():
    """The grouped products' 256 x 256 tiles need the best part of a round over 256 CUs, however long the groups. (An even
    group's last rows take a large tile from 193 of them on.)"""
    fewest = 1 << 30
    for n in (1, 2, 3, 8, 16):
        for rows in (768, 994, 1000, 1024, 1500, 2000, 3000, 5000, 8190, 16381, 100000):
            for N in (1, 16, 256, 257, 537, 1024, 1280, 2048, 4100, 8192):
                for major in "kn":
                    if bsm.bsm_debug_grouped_route("g", rows * n, N, 4096, n, b_major=major) == "k_grouped":
                        fewest = min(fewest, n * (rows // 256 + (rows % 256 >= 193)) * -(-N // 256))
    assert 0.85 * 256 <= fewest < 1 << 30


def test_the_shrink_goes_by_its_own_work():
    """Which kernel forms U depends on rows, rank and adapters, not on the width of the projection behind it."""
    seen = set()
    for rows in (1, 16, 65, 100, 300, 1000, 1024, 2000, 5000, 16384):
        for rank in (1, 16, 32, 64, 128, 256):
            for n in (1, 8, 31, 32, 64, 1000):
                kinds = {bsm.bsm_debug_grouped_route("a", rows, N, 4096, n, R=rank, shrink=1) for N in (1, 16, 256, 1024, 4096, 16384)}
                assert len(kinds) == 1, (rows, rank, n, kinds)
                seen |= kinds
    assert seen == {"k_lora_shrink", "k_lora_shrink_rows"}
