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


SA, SB = FAKE + (4 << 36), FAKE + (5 << 36)


def mx(rows=100, N=64, K=128, n_groups=4, offsets=OFF, a_fmt="e4m3", a=A, lda=128, sa=SA, ld_sfa=4, b_fmt="e4m3", b=B, ldb=128,
       stride_b=8192, sb=SB, ld_sfb=4, stride_sfb=256, fast=0, d_fmt="bf16", d=D, ldd=64, accum=0, ew=None):
    bsm.bsm_gemm_grouped_block_scale(rows, N, K, n_groups, offsets, a_fmt, a, lda, sa, ld_sfa, b_fmt, b, ldb, stride_b, sb, ld_sfb,
                                     stride_sfb, fast, d_fmt, d, ldd, accum, ew, 0)


def test_block_scaled_refusals():
    for name, bad in (("BSM_E_NULL", dict(offsets=0)), ("BSM_E_NULL", dict(a=0)), ("BSM_E_NULL", dict(sa=0)),
                      ("BSM_E_NULL", dict(sb=0)), ("BSM_E_NULL", dict(d=0)), ("BSM_E_ALIGN", dict(a=A + 8)),
                      ("BSM_E_ALIGN", dict(sa=SA + 2)), ("BSM_E_ALIGN", dict(sb=SB + 1)), ("BSM_E_ALIGN", dict(lda=112)),
                      ("BSM_E_ALIGN", dict(lda=136)), ("BSM_E_ALIGN", dict(ldb=130)), ("BSM_E_ALIGN", dict(ld_sfa=6)),
                      ("BSM_E_ALIGN", dict(K=256, lda=256, ldb=256, ld_sfb=4)), ("BSM_E_ALIGN", dict(stride_b=8200)),
                      ("BSM_E_ALIGN", dict(stride_sfb=258)), ("BSM_E_SHAPE", dict(stride_b=-128)),
                      ("BSM_E_SHAPE", dict(stride_sfb=-4)), ("BSM_E_SHAPE", dict(K=100)), ("BSM_E_SHAPE", dict(rows=1 << 31)),
                      ("BSM_E_SHAPE", dict(n_groups=65537)), ("BSM_E_SHAPE", dict(lda=1 << 24)),
                      ("BSM_E_DTYPE", dict(a_fmt="e2m1")), ("BSM_E_DTYPE", dict(b_fmt="e5m2")), ("BSM_E_DTYPE", dict(a_fmt="bf16")),
                      ("BSM_E_DTYPE", dict(d_fmt="f16")), ("BSM_E_ARG", dict(fast=2)), ("BSM_E_ARG", dict(accum=-1)),
                      ("BSM_E_ALIAS", dict(a=D + 1024)), ("BSM_E_ALIAS", dict(sa=D + 64)), ("BSM_E_ALIAS", dict(b=D - 8192)),
                      ("BSM_E_ALIAS", dict(sb=D - 512)), ("BSM_E_ALIAS", dict(offsets=D + 4))):
        expect(name, mx, **bad)
    mx(rows=0, a=0, sa=0, b=0, sb=0, d=0)
    mx(N=0, a=0, sa=0, b=0, sb=0, d=0)
    mx(n_groups=0, offsets=0, a=0, d=0)
    expect("BSM_E_ARG", mx, a=torch.zeros(64, dtype=torch.uint8))


WS, AD, SC = FAKE + (6 << 36), FAKE + (7 << 36), FAKE + (8 << 36)


def lora(rows=100, N=64, K=64, R=16, n=4, adapter=AD, ab="bf16", x=A, ldx=64, w=B, ldw=64, la=SA, ld_la=64, stride_la=1024, lb=SB,
         ld_lb=16, stride_lb=1024, scale=SC, ws=WS, d_fmt="bf16", d=D, ldd=64, accum=0, ew=None):
    bsm.bsm_gemm_lora(rows, N, K, R, n, adapter, ab, x, ldx, w, ldw, la, ld_la, stride_la, lb, ld_lb, stride_lb, scale, ws, d_fmt, d,
                      ldd, accum, ew, 0)


def test_adapter_refusals():
    for name, bad in (("BSM_E_NULL", dict(x=0)), ("BSM_E_NULL", dict(w=0)), ("BSM_E_NULL", dict(la=0)), ("BSM_E_NULL", dict(lb=0)),
                      ("BSM_E_NULL", dict(adapter=0)), ("BSM_E_NULL", dict(scale=0)), ("BSM_E_NULL", dict(ws=0)),
                      ("BSM_E_NULL", dict(d=0)), ("BSM_E_ALIGN", dict(x=A + 2)), ("BSM_E_ALIGN", dict(la=SA + 8)),
                      ("BSM_E_ALIGN", dict(ws=WS + 4)), ("BSM_E_ALIGN", dict(adapter=AD + 1)), ("BSM_E_ALIGN", dict(scale=SC + 2)),
                      ("BSM_E_ALIGN", dict(ldx=60)), ("BSM_E_ALIGN", dict(ldw=56)), ("BSM_E_ALIGN", dict(ld_la=56)),
                      ("BSM_E_ALIGN", dict(ld_lb=8)), ("BSM_E_ALIGN", dict(ld_lb=20)), ("BSM_E_ALIGN", dict(stride_la=1028)),
                      ("BSM_E_ALIGN", dict(stride_lb=1020)), ("BSM_E_ALIGN", dict(ldd=60)), ("BSM_E_SHAPE", dict(R=257)),
                      ("BSM_E_SHAPE", dict(R=-1)), ("BSM_E_SHAPE", dict(rows=-1)), ("BSM_E_SHAPE", dict(n=-1)),
                      ("BSM_E_SHAPE", dict(stride_la=-8)), ("BSM_E_SHAPE", dict(ld_la=1 << 23)), ("BSM_E_DTYPE", dict(ab="e4m3")),
                      ("BSM_E_DTYPE", dict(d_fmt="f16")), ("BSM_E_ARG", dict(accum=2)), ("BSM_E_ARG", dict(ew=bsm.ewise_desc(9))),
                      ("BSM_E_ALIAS", dict(x=D + 64)), ("BSM_E_ALIAS", dict(ws=D + 64)), ("BSM_E_ALIAS", dict(ws=B)),
                      ("BSM_E_ALIAS", dict(adapter=WS + 4)), ("BSM_E_ALIAS", dict(lb=D - 2 * 3 * 1024))):
        expect(name, lora, **bad)
    lora(rows=0, x=0, w=0, d=0)
    lora(N=0, x=0, w=0, d=0)
    assert bsm.bsm_gemm_lora_workspace(100, 16) == 100 * 32 * 4
    assert bsm.bsm_gemm_lora_workspace(0, 16) == 0 == bsm.bsm_gemm_lora_workspace(7, 0)
    for rows, R in ((-1, 8), (8, 300), (1 << 31, 8)):
        expect("BSM_E_SHAPE", bsm.bsm_gemm_lora_workspace, rows=rows, R=R)
    expect("BSM_E_ARG", lora, scale=torch.ones(4))


def test_scales_of_another_type_are_refused():
    """The adapters' scales are read as float32, one after another: a tensor of another type or with gaps is refused, as
    the offsets and the rows' adapters are (before its device is looked at)."""
    for t in (torch.float64, torch.bfloat16, torch.float16, torch.int32):
        expect("BSM_E_DTYPE", lora, scale=torch.ones(4, dtype=t))
    expect("BSM_E_ALIGN", lora, scale=torch.ones(8)[::2])


def test_short_arrays_are_refused():
    """Arrays whose length a call fixes are refused where a tensor is too short: the kernels would read (and, in the
    workspace, write) past its end. Arguments that a call does not use may have any length."""
    ints = lambda n: torch.zeros(n, dtype=torch.int32)
    for fn in (grouped, wgrad, mx):
        expect("BSM_E_SHAPE", fn, offsets=ints(4))
        expect("BSM_E_ARG", fn, offsets=ints(5))                         # (long enough: on the host)
        fn(n_groups=0, offsets=0, a=0, d=0)
    expect("BSM_E_SHAPE", lora, adapter=ints(99))
    expect("BSM_E_SHAPE", lora, scale=torch.ones(3))
    need = bsm.bsm_gemm_lora_workspace(100, 16)
    expect("BSM_E_SHAPE", lora, ws=torch.zeros(need - 1, dtype=torch.uint8))
    expect("BSM_E_SHAPE", lora, ws=torch.zeros(need // 4 - 1))
    expect("BSM_E_ALIGN", lora, ws=torch.zeros(need, 2, dtype=torch.uint8)[:, 0])
    expect("BSM_E_ARG", lora, adapter=ints(100))
    expect("BSM_E_ARG", lora, ws=torch.zeros(need // 4))
    expect("BSM_E_ARG", grouped, rows=0, offsets=ints(1))
    expect("BSM_E_ARG", mx, N=0, offsets=ints(1))
    expect("BSM_E_SHAPE", wgrad, rows=0, offsets=ints(1))               # (empty groups' outputs are written)
    expect("BSM_E_ARG", wgrad, M=0, offsets=ints(1))
    for unused in (dict(n=0), dict(R=0), dict(K=0), dict(N=0)):
        expect("BSM_E_ARG", lora, adapter=ints(1), **unused)             # (refused for its device alone)
        expect("BSM_E_ARG", lora, scale=torch.ones(1), **unused)
        expect("BSM_E_ARG", lora, ws=torch.zeros(1), **unused)


def test_outputs_too_short_are_refused(monkeypatch):
    """D that ends before the call's last row does, a bf16 one for float32 results among them. (Where the tensors live is
    looked at before that.)"""
    monkeypatch.setattr(bsm, "_here", lambda stream, *tensors: 0)
    z = lambda n, t=torch.bfloat16: torch.zeros(n, dtype=t)
    for fn, extra, whole in ((grouped, {}, 99 * 64 + 64), (wgrad, {}, 3 * 4096 + 64 * 64), (mx, {}, 99 * 64 + 64),
                             (lora, {}, 99 * 64 + 64), (wgrad, dict(n_groups=1, stride_d=0), 64 * 64)):
        for bad in (dict(d=z(whole - 1)), dict(d_fmt="f32", d=z(2 * whole - 1)), dict(d_fmt="f32", d=z(whole - 1, torch.float32)),
                    dict(d=z(whole + 7)[8:]), dict(d=z(2 * whole - 2, torch.uint8))):
            expect("BSM_E_SHAPE", fn, **extra, **bad)
        # long enough: refused for what comes after it
        for good in (dict(d=z(whole)), dict(d_fmt="f32", d=z(2 * whole)), dict(d=z(2 * whole, torch.uint8)), dict(d=z(whole + 8)[8:])):
            expect("BSM_E_ARG", fn, accum=2, **extra, **good)
