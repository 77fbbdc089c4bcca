"""CPU tests: what the products over groups of rows refuse, before any HIP call."""
import pytest
import torch

import block_scaled_matrix_amd as bsm

FAKE = 1 << 40          # a fake device address, never dereferenced (checks fail first)
A, B, D, OFF = FAKE, FAKE + (1 << 36), FAKE + (2 << 36), FAKE + (3 << 36)


@pytest.fixture(scope="module", autouse=True)
def L():
    import os
    if not os.path.exists(bsm.LIB_PATH):
        from block_scaled_matrix_amd import _build
        _build.build()
    return bsm.lib()


def expect(code, fn, **changed):
    with pytest.raises(bsm.BsmError) as e:
        fn(**changed)
    assert e.value.status == code, (changed, e.value.status, str(e.value))


def grouped(rows=100, N=64, K=64, n_groups=4, offsets=OFF, ab="bf16", a=A, lda=64, b=B, ldb=64, major="k", stride_b=4096,
            d_fmt="bf16", d=D, ldd=64, accum=0, ew=None):
    bsm.bsm_gemm_grouped(rows, N, K, n_groups, offsets, ab, a, lda, b, ldb, major, stride_b, d_fmt, d, ldd, accum, ew, 0)


def wgrad(rows=100, M=64, N=64, n_groups=4, offsets=OFF, ab="bf16", a=A, lda=64, b=B, ldb=64, d_fmt="bf16", d=D, ldd=64,
          stride_d=4096, accum=0):
    bsm.bsm_gemm_grouped_wgrad(rows, M, N, n_groups, offsets, ab, a, lda, b, ldb, d_fmt, d, ldd, stride_d, accum, 0)


@pytest.mark.parametrize("fn", [grouped, wgrad])
def test_common_refusals(fn):
    for name, bad in (("BSM_E_NULL", dict(offsets=0)), ("BSM_E_NULL", dict(a=0)), ("BSM_E_NULL", dict(b=0)),
                      ("BSM_E_NULL", dict(d=0)), ("BSM_E_ALIGN", dict(offsets=OFF + 2)), ("BSM_E_ALIGN", dict(a=A + 8)),
                      ("BSM_E_ALIGN", dict(b=B + 2)), ("BSM_E_ALIGN", dict(d=D + 8)), ("BSM_E_ALIGN", dict(lda=56)),
                      ("BSM_E_ALIGN", dict(lda=68)), ("BSM_E_ALIGN", dict(ldb=60)), ("BSM_E_ALIGN", dict(ldd=56)),
                      ("BSM_E_ALIGN", dict(ldd=68)), ("BSM_E_DTYPE", dict(ab="f32")), ("BSM_E_DTYPE", dict(ab="e4m3")),
                      ("BSM_E_DTYPE", dict(d_fmt="f16")), ("BSM_E_DTYPE", dict(d_fmt="u16")), ("BSM_E_SHAPE", dict(rows=-1)),
                      ("BSM_E_SHAPE", dict(rows=1 << 31)), ("BSM_E_SHAPE", dict(N=-1)), ("BSM_E_SHAPE", dict(N=1 << 31)),
                      ("BSM_E_SHAPE", dict(n_groups=-1)), ("BSM_E_SHAPE", dict(n_groups=65537)),
                      ("BSM_E_SHAPE", dict(lda=1 << 23)), ("BSM_E_SHAPE", dict(ldb=1 << 23)), ("BSM_E_ARG", dict(accum=2)),
                      ("BSM_E_ALIAS", dict(a=D + 1024)), ("BSM_E_ALIAS", dict(b=D + 64)), ("BSM_E_ALIAS", dict(offsets=D + 4))):
        expect(name, fn, **bad)
    assert bsm.bsm_last_error()


def test_grouped_refusals():
    expect("BSM_E_MAJOR", grouped, major="m")
    expect("BSM_E_SHAPE", grouped, K=-1)
    expect("BSM_E_SHAPE", grouped, stride_b=-8)
    expect("BSM_E_ALIGN", grouped, stride_b=4100)
    expect("BSM_E_ALIGN", grouped, N=65, ldd=72, major="n")              # ldb < N
    expect("BSM_E_ARG", grouped, ew=bsm.ewise_desc(7))
    expect("BSM_E_ALIAS", grouped, b=D - (1 << 20), stride_b=1 << 20)    # the last group's weight reaches D
    expect("BSM_E_ALIGN", grouped, d_fmt="f32", ldd=66)


def test_wgrad_refusals():
    expect("BSM_E_SHAPE", wgrad, M=-1)
    expect("BSM_E_ALIAS", wgrad, stride_d=4088)                          # the groups' outputs overlap
    expect("BSM_E_ALIAS", wgrad, stride_d=0)
    expect("BSM_E_ALIGN", wgrad, stride_d=4100)
    expect("BSM_E_SHAPE", wgrad, stride_d=-4096)
    expect("BSM_E_ALIAS", wgrad, a=D + 3 * 8192)                         # inside the last group's output


def test_nothing_to_do_needs_no_pointers():
    grouped(rows=0, offsets=OFF, a=0, b=0, d=0)
    grouped(N=0, a=0, b=0, d=0)
    grouped(n_groups=0, offsets=0, a=0, b=0, d=0)
    wgrad(M=0, a=0, b=0, d=0)
    wgrad(N=0, a=0, b=0, d=0)
    wgrad(n_groups=0, offsets=0, a=0, b=0, d=0)


def test_tensors_of_the_host_are_refused():
    t = torch.zeros(8192, dtype=torch.bfloat16)
    off = torch.zeros(5, dtype=torch.int32)
    for fn in (grouped, wgrad):
        expect("BSM_E_ARG", fn, a=t)
        expect("BSM_E_ARG", fn, offsets=off)
        expect("BSM_E_ARG", fn, d=t)
