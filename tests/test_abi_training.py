"""CPU tests: what the calls around the products of a training step refuse, before any HIP call."""
import pytest
import torch

import block_scaled_matrix_amd as bsm

FAKE = 1 << 40          # a fake device address, never dereferenced (checks fail first)
AT = [FAKE + (i << 36) for i in range(12)]


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


def balance(rows=1000, E=64, k=4, fmt="bf16", logits=AT[0], ldl=64, ids=AT[1], scale=1.0, counts=AT[2], offsets=AT[3], loss=AT[4],
            ws=AT[5]):
    bsm.bsm_router_balance(rows, E, k, fmt, logits, ldl, ids, scale, counts, offsets, loss, ws, 0)


def balance_grad(rows=1000, E=64, k=4, fmt="bf16", logits=AT[0], ldl=64, ids=AT[1], counts=AT[2], scale=1.0, dloss=AT[3],
                 d_fmt="f32", d=AT[4], ldd=64, accum=0):
    bsm.bsm_router_balance_grad(rows, E, k, fmt, logits, ldl, ids, counts, scale, dloss, d_fmt, d, ldd, accum, 0)


@pytest.mark.parametrize("fn", [balance, balance_grad])
def test_router_refusals(fn):
    for name, bad in (("BSM_E_DTYPE", dict(fmt="e4m3")), ("BSM_E_SHAPE", dict(E=0)), ("BSM_E_SHAPE", dict(E=1025, ldl=1032, ldd=1032)),
                      ("BSM_E_SHAPE", dict(k=0)), ("BSM_E_SHAPE", dict(k=1025)), ("BSM_E_SHAPE", dict(rows=-1)),
                      ("BSM_E_SHAPE", dict(rows=1 << 31)), ("BSM_E_SHAPE", dict(rows=1 << 30, k=4)), ("BSM_E_NULL", dict(logits=0)),
                      ("BSM_E_NULL", dict(ids=0)), ("BSM_E_NULL", dict(counts=0)), ("BSM_E_ALIGN", dict(logits=AT[0] + 1)),
                      ("BSM_E_ALIGN", dict(ids=AT[1] + 2)), ("BSM_E_ALIGN", dict(counts=AT[2] + 2)), ("BSM_E_ALIGN", dict(ldl=63)),
                      ("BSM_E_SHAPE", dict(ldl=1 << 32)),
                      ("BSM_E_ARG", dict(logits=torch.zeros(1000, 64, dtype=torch.bfloat16))),
                      ("BSM_E_DTYPE", dict(logits=torch.zeros(1000, 64))), ("BSM_E_DTYPE", dict(ids=torch.zeros(4000, dtype=torch.int64))),
                      ("BSM_E_SHAPE", dict(ids=torch.zeros(3999, dtype=torch.int32))),
                      ("BSM_E_SHAPE", dict(logits=torch.zeros(999, 64, dtype=torch.bfloat16))),
                      ("BSM_E_SHAPE", dict(counts=torch.zeros(64, dtype=torch.int32)))):
        bad = {k: v for k, v in bad.items() if not (k == "ldd" and fn is balance)}
        expect(name, fn, **bad)


def test_balance_refusals():
    for name, bad in (("BSM_E_NULL", dict(offsets=0)), ("BSM_E_NULL", dict(loss=0)), ("BSM_E_NULL", dict(ws=0)),
                      ("BSM_E_ALIGN", dict(offsets=AT[3] + 1)), ("BSM_E_ALIGN", dict(loss=AT[4] + 2)), ("BSM_E_ALIGN", dict(ws=AT[5] + 8)),
                      ("BSM_E_ALIAS", dict(counts=AT[3] + 256)), ("BSM_E_ALIAS", dict(loss=AT[2] + 256)),
                      ("BSM_E_ALIAS", dict(counts=AT[0] + 64)), ("BSM_E_ALIAS", dict(ws=AT[1])), ("BSM_E_ALIAS", dict(offsets=AT[1] + 15996)),
                      ("BSM_E_DTYPE", dict(loss=torch.zeros(1, dtype=torch.float64))),
                      ("BSM_E_SHAPE", dict(offsets=torch.zeros(64, dtype=torch.int32))),
                      ("BSM_E_SHAPE", dict(ws=torch.zeros(bsm.bsm_router_balance_workspace(1000, 64) - 1, dtype=torch.uint8)))):
        expect(name, balance, **bad)
    assert bsm.bsm_router_balance_workspace(8, 64) == 0 and bsm.bsm_router_balance_workspace(0, 1) == 0
    for rows, E in ((-1, 4), (1 << 31, 4), (4, 0), (4, 1025)):
        expect("BSM_E_SHAPE", bsm.bsm_router_balance_workspace, rows=rows, n_experts=E)


def test_balance_grad_refusals():
    for name, bad in (("BSM_E_NULL", dict(d=0)), ("BSM_E_ALIGN", dict(d=AT[4] + 2)), ("BSM_E_ALIGN", dict(dloss=AT[3] + 2)),
                      ("BSM_E_ALIGN", dict(ldd=63)), ("BSM_E_DTYPE", dict(d_fmt="f16")), ("BSM_E_DTYPE", dict(d_fmt="u8")),
                      ("BSM_E_ARG", dict(accum=2)), ("BSM_E_ALIAS", dict(d=AT[0] + 64)), ("BSM_E_ALIAS", dict(d=AT[2])),
                      ("BSM_E_ALIAS", dict(d=AT[3])), ("BSM_E_ALIAS", dict(d=AT[1] + 64)),
                      ("BSM_E_SHAPE", dict(d=torch.zeros(999, 64))), ("BSM_E_ARG", dict(d=torch.zeros(1000, 64)))):
        expect(name, balance_grad, **bad)
    balance_grad(rows=0, logits=0, ids=0, counts=0, d=0)


def save(rows=100, K=100, x_fmt="bf16", x=AT[0], ldx=104, fmt="e4m3", q=AT[1], ldq=112, sf=AT[2], ld_sf=4):
    bsm.bsm_block_scale_save(rows, K, x_fmt, x, ldx, fmt, q, ldq, sf, ld_sf, 0)


def restore(rows=100, K=100, fmt="e4m3", q=AT[1], ldq=112, sf=AT[2], ld_sf=4, d_fmt="bf16", d=AT[3], ldd=104, ew=None):
    bsm.bsm_block_scale_restore(rows, K, fmt, q, ldq, sf, ld_sf, d_fmt, d, ldd, ew, 0)


def ewise_grad(rows=100, K=100, fmt="e4m3", q=AT[1], ldq=112, sf=AT[2], ld_sf=4, dy_fmt="bf16", dy=AT[0], lddy=104, d=AT[3], ldd=104,
               ew=bsm.ewise_desc()):
    bsm.bsm_block_scale_ewise_grad(rows, K, fmt, q, ldq, sf, ld_sf, dy_fmt, dy, lddy, d, ldd, ew, 0)


@pytest.mark.parametrize("fn", [save, restore, ewise_grad])
def test_kept_refusals(fn):
    for name, bad in (("BSM_E_DTYPE", dict(fmt="e2m1")), ("BSM_E_DTYPE", dict(fmt="f16")), ("BSM_E_SHAPE", dict(rows=-1)),
                      ("BSM_E_SHAPE", dict(rows=1 << 31)), ("BSM_E_SHAPE", dict(K=-1)), ("BSM_E_SHAPE", dict(K=(1 << 24) + 1)),
                      ("BSM_E_NULL", dict(q=0)), ("BSM_E_NULL", dict(sf=0)), ("BSM_E_ALIGN", dict(q=AT[1] + 8)),
                      ("BSM_E_ALIGN", dict(sf=AT[2] + 2)), ("BSM_E_ALIGN", dict(ldq=96)), ("BSM_E_ALIGN", dict(ldq=120)),
                      ("BSM_E_ALIGN", dict(ld_sf=3)), ("BSM_E_ALIGN", dict(ld_sf=6)), ("BSM_E_ALIGN", dict(K=112, ld_sf=0)),
                      ("BSM_E_DTYPE", dict(q=torch.zeros(100, 112))), ("BSM_E_SHAPE", dict(q=torch.zeros(99, 112, dtype=torch.uint8))),
                      ("BSM_E_SHAPE", dict(sf=torch.zeros(99, 4, dtype=torch.uint8))),
                      ("BSM_E_ARG", dict(q=torch.zeros(100, 112, dtype=torch.uint8)))):
        expect(name, fn, **bad)
    for none in (dict(rows=0), dict(K=0)):
        fn(q=0, sf=0, **none)


def test_save_refusals():
    for name, bad in (("BSM_E_DTYPE", dict(x_fmt="e4m3")), ("BSM_E_NULL", dict(x=0)), ("BSM_E_ALIGN", dict(x=AT[0] + 8)),
                      ("BSM_E_ALIGN", dict(ldx=96)), ("BSM_E_ALIGN", dict(ldx=100)), ("BSM_E_ALIGN", dict(x_fmt="f32", ldx=102)),
                      ("BSM_E_ALIAS", dict(q=AT[0] + 16)), ("BSM_E_ALIAS", dict(sf=AT[0] + 16)), ("BSM_E_ALIAS", dict(sf=AT[1] + 16)),
                      ("BSM_E_SHAPE", dict(x=torch.zeros(99 * 104 + 100, dtype=torch.bfloat16))),
                      ("BSM_E_DTYPE", dict(x=torch.zeros(100, 104)))):
        expect(name, save, **bad)


def test_restore_and_gradient_refusals():
    for fn, f in ((restore, "d_fmt"), (ewise_grad, "dy_fmt")):
        for name, bad in (("BSM_E_DTYPE", {f: "u16"}), ("BSM_E_NULL", dict(d=0)), ("BSM_E_ALIGN", dict(d=AT[3] + 8)),
                          ("BSM_E_ALIGN", dict(ldd=96)), ("BSM_E_ALIGN", dict(ldd=100)), ("BSM_E_ALIAS", dict(d=AT[1] + 16)),
                          ("BSM_E_ALIAS", dict(d=AT[2] + 16)), ("BSM_E_ARG", dict(ew=bsm.ewise_desc(7))),
                          ("BSM_E_SHAPE", dict(d=torch.zeros(99, 104, dtype=torch.bfloat16)))):
            expect(name, fn, **bad)
    for name, bad in (("BSM_E_NULL", dict(dy=0)), ("BSM_E_ALIGN", dict(lddy=100)), ("BSM_E_ALIAS", dict(dy=AT[3] + 16)),
                      ("BSM_E_ALIAS", dict(dy=AT[3], lddy=112)), ("BSM_E_NULL", dict(ew=None))):
        expect(name, ewise_grad, **bad)


def xent(rows=100, N=1000, K=64, ab="bf16", x=AT[0], ldx=64, w=AT[1], ldw=64, labels=AT[2], loss=AT[3], lse=AT[4], ws=AT[5]):
    bsm.bsm_gemm_cross_entropy(rows, N, K, ab, x, ldx, w, ldw, labels, loss, lse, ws, 0)


def xent_grad(rows=100, N=1000, K=64, ab="bf16", x=AT[0], ldx=64, w=AT[1], ldw=64, labels=AT[2], lse=AT[4], dloss=AT[3], piece=0,
              ws=AT[5], dx_fmt="bf16", dx=AT[6], lddx=64, dw_fmt="f32", dw=AT[7], lddw=64, accum=0):
    bsm.bsm_gemm_cross_entropy_grad(rows, N, K, ab, x, ldx, w, ldw, labels, lse, dloss, piece, ws, dx_fmt, dx, lddx, dw_fmt, dw, lddw,
                                    accum, 0)


@pytest.mark.parametrize("fn", [xent, xent_grad])
def test_cross_entropy_refusals(fn):
    for name, bad in (("BSM_E_DTYPE", dict(ab="f32")), ("BSM_E_DTYPE", dict(ab="e4m3")), ("BSM_E_SHAPE", dict(rows=-1)),
                      ("BSM_E_SHAPE", dict(rows=1 << 31)), ("BSM_E_SHAPE", dict(N=0)), ("BSM_E_SHAPE", dict(N=1 << 31)),
                      ("BSM_E_SHAPE", dict(K=-1)), ("BSM_E_SHAPE", dict(K=(1 << 22) + 1)), ("BSM_E_SHAPE", dict(rows=1 << 30, N=1 << 30)),
                      ("BSM_E_SHAPE", dict(ldx=1 << 23)), ("BSM_E_SHAPE", dict(ldw=1 << 23)), ("BSM_E_NULL", dict(x=0)),
                      ("BSM_E_NULL", dict(w=0)), ("BSM_E_NULL", dict(labels=0)), ("BSM_E_NULL", dict(lse=0)), ("BSM_E_NULL", dict(ws=0)),
                      ("BSM_E_ALIGN", dict(x=AT[0] + 8)), ("BSM_E_ALIGN", dict(w=AT[1] + 2)), ("BSM_E_ALIGN", dict(labels=AT[2] + 2)),
                      ("BSM_E_ALIGN", dict(lse=AT[4] + 1)), ("BSM_E_ALIGN", dict(ws=AT[5] + 8)), ("BSM_E_ALIGN", dict(ldx=56)),
                      ("BSM_E_ALIGN", dict(ldw=68)), ("BSM_E_ALIAS", dict(ws=AT[1])), ("BSM_E_ALIAS", dict(ws=AT[0] + 64)),
                      ("BSM_E_ARG", dict(x=torch.zeros(100, 64, dtype=torch.bfloat16))), ("BSM_E_DTYPE", dict(x=torch.zeros(100, 64))),
                      ("BSM_E_SHAPE", dict(w=torch.zeros(999, 64, dtype=torch.bfloat16))),
                      ("BSM_E_SHAPE", dict(labels=torch.zeros(99, dtype=torch.int32))),
                      ("BSM_E_DTYPE", dict(labels=torch.zeros(100, dtype=torch.int64))),
                      ("BSM_E_DTYPE", dict(lse=torch.zeros(100, dtype=torch.float64))),
                      ("BSM_E_SHAPE", dict(ws=torch.zeros(64, dtype=torch.uint8)))):
        expect(name, fn, **bad)


def test_cross_entropy_loss_refusals():
    for name, bad in (("BSM_E_NULL", dict(loss=0)), ("BSM_E_ALIGN", dict(loss=AT[3] + 2)), ("BSM_E_ALIAS", dict(loss=AT[4] + 8)),
                      ("BSM_E_ALIAS", dict(loss=AT[0] + 4)), ("BSM_E_ALIAS", dict(lse=AT[2] + 4)), ("BSM_E_ALIAS", dict(lse=AT[5] + 4)),
                      ("BSM_E_SHAPE", dict(loss=torch.zeros(99)))):
        expect(name, xent, **bad)
    xent(rows=0, x=0, w=0, labels=0, loss=0, lse=0, ws=0)
    for rows, N in ((-1, 4), (1 << 31, 4), (4, 0), (4, 1 << 31)):
        expect("BSM_E_SHAPE", bsm.bsm_gemm_cross_entropy_workspace, rows=rows, N=N)
    assert bsm.bsm_gemm_cross_entropy_workspace(0, 5) == 0
    # rows to 2^25; fewer than 2^24 tiles of 128 x 128 logits and 2^23 of dX
    for rows, N in (((1 << 25) + 1, 4), (1 << 25, 64 * 128 + 1), (128, 0x7FFFFF81)):
        expect("BSM_E_SHAPE", bsm.bsm_gemm_cross_entropy_workspace, rows=rows, N=N)
    assert bsm.bsm_gemm_cross_entropy_workspace(1 << 25, 63 * 128) > 0 and bsm.bsm_gemm_cross_entropy_workspace(128, 0x7FFFFF80) > 0
    expect("BSM_E_SHAPE", bsm.bsm_gemm_cross_entropy_grad_workspace, rows=1 << 25, N=4, K=32 * 128, piece=0)
    assert bsm.bsm_gemm_cross_entropy_grad_workspace(1 << 25, 4, 31 * 128, 0) > 0


def test_cross_entropy_grad_refusals():
    for name, bad in (("BSM_E_NULL", dict(dloss=0)), ("BSM_E_ALIGN", dict(dloss=AT[3] + 2)), ("BSM_E_ARG", dict(accum=2)),
                      ("BSM_E_DTYPE", dict(dx_fmt="f16")), ("BSM_E_DTYPE", dict(dw_fmt="u8")), ("BSM_E_ALIGN", dict(dx=AT[6] + 8)),
                      ("BSM_E_ALIGN", dict(dw=AT[7] + 8)), ("BSM_E_ALIGN", dict(lddx=56)), ("BSM_E_ALIGN", dict(lddx=68)),
                      ("BSM_E_ALIGN", dict(lddw=60)), ("BSM_E_SHAPE", dict(piece=-1)), ("BSM_E_ALIAS", dict(dx=AT[0] + 1024)),
                      ("BSM_E_ALIAS", dict(dw=AT[1])), ("BSM_E_ALIAS", dict(dw=AT[6] + 1024)), ("BSM_E_ALIAS", dict(dx=AT[5])),
                      ("BSM_E_ALIAS", dict(dw=AT[3])), ("BSM_E_ALIAS", dict(dx=AT[4] - 64)),
                      ("BSM_E_SHAPE", dict(dx=torch.zeros(99, 64, dtype=torch.bfloat16))), ("BSM_E_SHAPE", dict(dw=torch.zeros(999, 64))),
                      ("BSM_E_DTYPE", dict(dw=torch.zeros(1000, 64, dtype=torch.bfloat16)))):
        expect(name, xent_grad, **bad)
    xent_grad(K=0, ldx=0, ldw=0, x=0, w=0)
    xent_grad(dx=None, dw=None)
    xent_grad(rows=0, dw=None, x=0, w=0, labels=0, lse=0, dloss=0, ws=0)
    for bad in (dict(rows=-1), dict(N=0), dict(K=-1), dict(piece=-1), dict(piece=1 << 31)):
        expect("BSM_E_SHAPE", bsm.bsm_gemm_cross_entropy_grad_workspace, **{**dict(rows=4, N=4, K=4, piece=0), **bad})


def kept_wgrad(rows=100, M=64, N=100, n_groups=4, offsets=AT[8], ab="bf16", a=AT[0], lda=64, b_fmt="e4m3", b=AT[1], ldb=112, sf=AT[2],
               ld_sf=4, d_fmt="f32", d=AT[3], ldd=104, stride_d=8192, accum=0):
    bsm.bsm_gemm_grouped_wgrad_block_scale(rows, M, N, n_groups, offsets, ab, a, lda, b_fmt, b, ldb, sf, ld_sf, d_fmt, d, ldd, stride_d,
                                           accum, 0)


def test_kept_weight_gradient_refusals():
    for name, bad in (("BSM_E_NULL", dict(offsets=0)), ("BSM_E_NULL", dict(a=0)), ("BSM_E_NULL", dict(b=0)), ("BSM_E_NULL", dict(sf=0)),
                      ("BSM_E_NULL", dict(d=0)), ("BSM_E_ALIGN", dict(a=AT[0] + 8)), ("BSM_E_ALIGN", dict(b=AT[1] + 8)),
                      ("BSM_E_ALIGN", dict(sf=AT[2] + 2)), ("BSM_E_ALIGN", dict(d=AT[3] + 4)), ("BSM_E_ALIGN", dict(lda=60)),
                      ("BSM_E_ALIGN", dict(lda=68)), ("BSM_E_ALIGN", dict(ldb=96)), ("BSM_E_ALIGN", dict(ldb=104)),
                      ("BSM_E_ALIGN", dict(ld_sf=3)), ("BSM_E_ALIGN", dict(N=129, ldb=144, ldd=132, stride_d=1 << 14, ld_sf=4)),
                      ("BSM_E_ALIGN", dict(ldd=96)), ("BSM_E_ALIGN", dict(stride_d=8194)), ("BSM_E_ALIAS", dict(stride_d=6400)),
                      ("BSM_E_SHAPE", dict(rows=-1)), ("BSM_E_SHAPE", dict(rows=1 << 31)), ("BSM_E_SHAPE", dict(M=-1)),
                      ("BSM_E_SHAPE", dict(N=1 << 31)), ("BSM_E_SHAPE", dict(n_groups=65537)), ("BSM_E_SHAPE", dict(lda=1 << 23)),
                      ("BSM_E_SHAPE", dict(ldb=1 << 24)), ("BSM_E_DTYPE", dict(ab="f32")), ("BSM_E_DTYPE", dict(b_fmt="e2m1")),
                      ("BSM_E_DTYPE", dict(d_fmt="f16")), ("BSM_E_ARG", dict(accum=2)), ("BSM_E_ALIAS", dict(a=AT[3] + 64)),
                      ("BSM_E_ALIAS", dict(b=AT[3] + 64)), ("BSM_E_ALIAS", dict(sf=AT[3] + 64)), ("BSM_E_ALIAS", dict(offsets=AT[3] + 8)),
                      ("BSM_E_DTYPE", dict(a=torch.zeros(100, 64))), ("BSM_E_SHAPE", dict(b=torch.zeros(99, 112, dtype=torch.uint8))),
                      ("BSM_E_SHAPE", dict(sf=torch.zeros(399, dtype=torch.uint8))), ("BSM_E_SHAPE", dict(offsets=torch.zeros(4, dtype=torch.int32))),
                      ("BSM_E_ARG", dict(a=torch.zeros(100, 64, dtype=torch.bfloat16)))):
        expect(name, kept_wgrad, **bad)
    for none in (dict(M=0), dict(N=0), dict(n_groups=0, offsets=0)):
        kept_wgrad(a=0, b=0, sf=0, d=0, **none)


def test_kept_weight_gradient_output_refusals():
    """D of another type than d_fmt says, and D that ends before the last group's last row does."""
    z = lambda n, t=torch.float32: torch.zeros(n, dtype=t)
    whole = 3 * 8192 + 63 * 104 + 100
    for name, bad in (("BSM_E_DTYPE", dict(d=z(4 * 8192, torch.bfloat16))), ("BSM_E_DTYPE", dict(d_fmt="bf16", d=z(4 * 8192))),
                      ("BSM_E_DTYPE", dict(d=z(4 * 8192, torch.int32))), ("BSM_E_DTYPE", dict(d_fmt="e4m3")),
                      ("BSM_E_SHAPE", dict(d=z(whole - 1))), ("BSM_E_SHAPE", dict(d=z(whole + 3)[4:])),
                      ("BSM_E_SHAPE", dict(n_groups=1, d=z(63 * 104 + 99))), ("BSM_E_SHAPE", dict(rows=0, d=z(whole - 1))),
                      ("BSM_E_ALIGN", dict(d=z(2 * whole).view(-1, 2)[:, 0])),
                      # long enough: refused for living on the host
                      ("BSM_E_ARG", dict(d=z(whole))), ("BSM_E_ARG", dict(n_groups=1, d=z(63 * 104 + 100))),
                      ("BSM_E_ARG", dict(d=z(whole + 4)[4:])), ("BSM_E_ARG", dict(d_fmt="bf16", d=z(whole, torch.bfloat16)))):
        expect(name, kept_wgrad, **bad)
