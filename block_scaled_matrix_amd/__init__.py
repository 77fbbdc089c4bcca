"""block_scaled_matrix_amd - Python binding of libbsm, the gfx950 HIP library.

Argument marshalling only: every entry point forwards to the C function of the same
name in libbsm.so (declared in include/bsm.h) and raises BsmError on a negative
status. Device buffers are torch tensors (or raw device addresses); the stream is
torch's current HIP stream unless one is given. There is no other implementation of
these operations: if libbsm.so has not been built, every call raises.
"""
from __future__ import annotations

import ctypes as C
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbsm.so")

DTYPE = {"u8": 0, "u16": 1, "u32": 2, "f16": 3, "bf16": 4, "f32": 5, "e4m3": 6, "e2m1": 7, "e8m0": 8, "e5m2": 9,
         "e2m3": 10, "e3m2": 11}
ESIZE = {"u8": 1, "u16": 2, "u32": 4, "f16": 2, "bf16": 2, "f32": 4, "e4m3": 1, "e8m0": 1, "e5m2": 1}
STATUS = {0: "BSM_OK", -1: "BSM_E_NULL", -2: "BSM_E_RANK", -3: "BSM_E_BOX", -4: "BSM_E_ESTRIDE",
          -5: "BSM_E_ALIGN", -6: "BSM_E_SWIZZLE", -7: "BSM_E_FILL", -8: "BSM_E_DTYPE", -9: "BSM_E_SHAPE",
          -10: "BSM_E_MAJOR", -11: "BSM_E_ALIAS", -12: "BSM_E_HIP", -13: "BSM_E_ARG"}
EWISE = {"none": 0, "silu_affine": 1}
EXPORTS = ("bsm_image_stride", "bsm_tile_box_load", "bsm_tile_box_store", "bsm_tile_box_copy",
           "bsm_tile_box_load_steps", "bsm_tile_box_store_steps", "bsm_tile_gather4", "bsm_tile_scatter4", "bsm_gemm",
           "bsm_gemm_block_scale", "bsm_gemm_ewise", "bsm_gemm_block_scale_ewise", "bsm_gemm_block_scale_major",
           "bsm_gemm_block_scale_fastacc", "bsm_gemm_grouped", "bsm_gemm_grouped_wgrad",
           "bsm_gemm_grouped_block_scale", "bsm_gemm_lora", "bsm_gemm_lora_workspace", "bsm_router_balance",
           "bsm_router_balance_workspace", "bsm_router_balance_grad", "bsm_block_scale_save", "bsm_block_scale_restore",
           "bsm_block_scale_ewise_grad", "bsm_gemm_grouped_wgrad_block_scale", "bsm_gemm_cross_entropy", "bsm_gemm_cross_entropy_workspace",
           "bsm_gemm_cross_entropy_grad", "bsm_gemm_cross_entropy_grad_workspace",
           "bsm_debug_grouped_route", "bsm_debug_stream_mix_bf16", "bsm_debug_mfma_loop", "bsm_tile_add_scalar_f32", "bsm_debug_fragments", "bsm_debug_fragment_shape", "bsm_last_error")


class BsmError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code
        self.status = STATUS.get(code, str(code))


class bsm_tensor(C.Structure):
    _fields_ = [("base", C.c_void_p), ("dtype", C.c_int32), ("rank", C.c_int32),
                ("dims", C.c_int64 * 5), ("strides", C.c_int64 * 5)]


class bsm_box(C.Structure):
    _fields_ = [("rank", C.c_int32), ("box", C.c_int32 * 5), ("element_strides", C.c_int32 * 5),
                ("swizzle", C.c_int32), ("oob_fill", C.c_int32)]


class bsm_ewise(C.Structure):
    _fields_ = [("op", C.c_int32), ("scale", C.c_float), ("bias", C.c_float)]


_lib = None


def lib():
    """The loaded libbsm.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "(python block_scaled_matrix_amd/_build.py)")
        L = C.CDLL(LIB_PATH)
        P, I64, I32 = C.c_void_p, C.c_int64, C.c_int32
        L.bsm_last_error.restype = C.c_char_p
        L.bsm_image_stride.restype = I64
        L.bsm_image_stride.argtypes = [C.POINTER(bsm_box), I32]
        L.bsm_tile_box_load.argtypes = [C.POINTER(bsm_tensor), C.POINTER(bsm_box), P, I64, P, P]
        L.bsm_tile_box_store.argtypes = [C.POINTER(bsm_tensor), C.POINTER(bsm_box), P, I64, P, C.c_int, P]
        L.bsm_tile_box_copy.argtypes = [C.POINTER(bsm_tensor), C.POINTER(bsm_tensor), C.POINTER(bsm_tensor),
                                        C.POINTER(bsm_box), P]
        L.bsm_tile_box_load_steps.argtypes = [C.POINTER(bsm_tensor), C.POINTER(bsm_box), P, I32, P, P, P, P]
        L.bsm_tile_box_store_steps.argtypes = [C.POINTER(bsm_tensor), C.POINTER(bsm_box), P, I32, P, P, P, C.c_int, P]
        L.bsm_tile_gather4.argtypes = [C.POINTER(bsm_tensor), C.POINTER(bsm_box), P, I64, P, P]
        L.bsm_tile_scatter4.argtypes = [C.POINTER(bsm_tensor), C.POINTER(bsm_box), P, I64, P, P]
        L.bsm_gemm.argtypes = [I64, I64, I64, I32, P, I64, C.c_char, P, I64, C.c_char, P, I64, C.c_int, C.c_int,
                               C.c_int, P]
        L.bsm_gemm_block_scale.argtypes = [I64, I64, I64, I32, P, I64, P, I64, I32, P, I64, P, I64, P, I64,
                                           C.c_int, C.c_int, C.c_int, P]
        L.bsm_gemm_ewise.argtypes = L.bsm_gemm.argtypes[:-1] + [C.POINTER(bsm_ewise), P]
        L.bsm_gemm_block_scale_ewise.argtypes = L.bsm_gemm_block_scale.argtypes[:-1] + [C.POINTER(bsm_ewise), P]
        L.bsm_gemm_block_scale_major.argtypes = [I64, I64, I64, I32, P, I64, C.c_char, P, I64, I32, P, I64, C.c_char,
                                                 P, I64, P, I64, C.c_int, C.c_int, C.c_int, C.POINTER(bsm_ewise), P]
        L.bsm_gemm_block_scale_fastacc.argtypes = L.bsm_gemm_block_scale_ewise.argtypes
        L.bsm_gemm_grouped.argtypes = [I64, I64, I64, I32, P, I32, P, I64, P, I64, C.c_char, I64, I32, P, I64, C.c_int,
                                       C.POINTER(bsm_ewise), P]
        L.bsm_gemm_grouped_wgrad.argtypes = [I64, I64, I64, I32, P, I32, P, I64, P, I64, I32, P, I64, I64, C.c_int, P]
        L.bsm_gemm_grouped_block_scale.argtypes = [I64, I64, I64, I32, P, I32, P, I64, P, I64, I32, P, I64, I64, P, I64, I64,
                                                   C.c_int, I32, P, I64, C.c_int, C.POINTER(bsm_ewise), P]
        L.bsm_gemm_lora_workspace.restype = I64
        L.bsm_gemm_lora_workspace.argtypes = [I64, I64]
        L.bsm_gemm_lora.argtypes = [I64, I64, I64, I64, I32, P, I32, P, I64, P, I64, P, I64, I64, P, I64, I64, P, P, I32, P,
                                    I64, C.c_int, C.POINTER(bsm_ewise), P]
        L.bsm_router_balance_workspace.restype = I64
        L.bsm_router_balance_workspace.argtypes = [I64, I32]
        L.bsm_router_balance.argtypes = [I64, I32, I32, I32, P, I64, P, C.c_float, P, P, P, P, P]
        L.bsm_router_balance_grad.argtypes = [I64, I32, I32, I32, P, I64, P, P, C.c_float, P, I32, P, I64, C.c_int, P]
        L.bsm_block_scale_save.argtypes = [I64, I64, I32, P, I64, I32, P, I64, P, I64, P]
        L.bsm_block_scale_restore.argtypes = [I64, I64, I32, P, I64, P, I64, I32, P, I64, C.POINTER(bsm_ewise), P]
        L.bsm_block_scale_ewise_grad.argtypes = [I64, I64, I32, P, I64, P, I64, I32, P, I64, P, I64, C.POINTER(bsm_ewise), P]
        L.bsm_gemm_grouped_wgrad_block_scale.argtypes = [I64, I64, I64, I32, P, I32, P, I64, I32, P, I64, P, I64, I32, P, I64, I64,
                                                         C.c_int, P]
        L.bsm_gemm_cross_entropy_workspace.restype = L.bsm_gemm_cross_entropy_grad_workspace.restype = I64
        L.bsm_gemm_cross_entropy_workspace.argtypes = [I64, I64]
        L.bsm_gemm_cross_entropy_grad_workspace.argtypes = [I64, I64, I64, I64]
        L.bsm_gemm_cross_entropy.argtypes = [I64, I64, I64, I32, P, I64, P, I64, P, P, P, P, P]
        L.bsm_gemm_cross_entropy_grad.argtypes = [I64, I64, I64, I32, P, I64, P, I64, P, P, P, I64, P, I32, P, I64, I32, P, I64,
                                                  C.c_int, P]
        L.bsm_tile_add_scalar_f32.argtypes = [P, P, I64, C.c_float, P]
        L.bsm_debug_stream_mix_bf16.argtypes = [P, P, P, I64, P]
        L.bsm_debug_grouped_route.restype = C.c_char_p
        L.bsm_debug_grouped_route.argtypes = [C.c_char, I64, I64, I64, I64, I64, I32, I32, I32, C.c_char, C.c_int, C.c_int]
        L.bsm_debug_mfma_loop.argtypes = [I32, I64, I32, P, P]
        L.bsm_debug_fragments.argtypes = [P, I64, I64, C.c_char, P, P]
        L.bsm_debug_fragment_shape.restype = None
        L.bsm_debug_fragment_shape.argtypes = [C.POINTER(I64), C.POINTER(I64)]
        for rc_fn in ("bsm_tile_box_load", "bsm_tile_box_store", "bsm_tile_box_copy", "bsm_tile_box_load_steps",
                      "bsm_tile_box_store_steps", "bsm_tile_gather4",
                      "bsm_tile_scatter4", "bsm_gemm",
                      "bsm_gemm_block_scale", "bsm_gemm_ewise", "bsm_gemm_block_scale_ewise",
                      "bsm_gemm_block_scale_major", "bsm_gemm_block_scale_fastacc", "bsm_gemm_grouped",
                      "bsm_gemm_grouped_wgrad", "bsm_gemm_grouped_block_scale", "bsm_gemm_lora", "bsm_router_balance", "bsm_router_balance_grad",
                      "bsm_block_scale_save", "bsm_block_scale_restore", "bsm_block_scale_ewise_grad",
                      "bsm_gemm_grouped_wgrad_block_scale", "bsm_gemm_cross_entropy", "bsm_gemm_cross_entropy_grad", "bsm_tile_add_scalar_f32",
                      "bsm_debug_fragments", "bsm_debug_stream_mix_bf16", "bsm_debug_mfma_loop"):
            getattr(L, rc_fn).restype = C.c_int
        _lib = L
    return _lib


def _ptr(x):
    """Device address of a torch tensor, an int address, or None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int):
    if rc < 0:
        raise BsmError(rc, bsm_last_error())
    return rc


def bsm_last_error() -> str:
    return lib().bsm_last_error().decode()


def tensor_desc(base, dtype: str, dims, strides_bytes) -> bsm_tensor:
    """A bsm_tensor view: dims and byte strides outer to inner."""
    t = bsm_tensor()
    t.base = _ptr(base)
    t.dtype = DTYPE[dtype]
    t.rank = len(dims)
    for i, (d, s) in enumerate(zip(dims, strides_bytes)):
        t.dims[i] = int(d)
        t.strides[i] = int(s)
    return t


def box_desc(box, element_strides=None, swizzle: int = 0, oob_fill: int = 0) -> bsm_box:
    b = bsm_box()
    b.rank = len(box)
    es = element_strides or (1,) * len(box)
    for i, (x, e) in enumerate(zip(box, es)):
        b.box[i] = int(x)
        b.element_strides[i] = int(e)
    b.swizzle = swizzle
    b.oob_fill = oob_fill
    return b


def bsm_image_stride(box: bsm_box, dtype: str) -> int:
    return _check(lib().bsm_image_stride(C.byref(box), DTYPE[dtype]))


def bsm_tile_box_load(src: bsm_tensor, box: bsm_box, coords, n_boxes: int, images, stream=None):
    _check(lib().bsm_tile_box_load(C.byref(src), C.byref(box), _ptr(coords), n_boxes, _ptr(images),
                                   _stream(stream)))


def bsm_tile_box_store(dst: bsm_tensor, box: bsm_box, coords, n_boxes: int, images, reduce_add: int = 0,
                       stream=None):
    _check(lib().bsm_tile_box_store(C.byref(dst), C.byref(box), _ptr(coords), n_boxes, _ptr(images),
                                    reduce_add, _stream(stream)))


def bsm_tile_box_copy(src: bsm_tensor, dst: bsm_tensor | None, dst_add: bsm_tensor | None, box: bsm_box,
                      stream=None):
    _check(lib().bsm_tile_box_copy(C.byref(src), C.byref(dst) if dst is not None else None,
                                   C.byref(dst_add) if dst_add is not None else None, C.byref(box),
                                   _stream(stream)))


def _host_i64(xs):
    a = (C.c_int64 * max(len(xs), 1))(*[int(x) for x in xs])
    return a


def _repeat_args(coords, repeats, steps):
    rank = len(coords)
    flat = [int(v) for st in steps for v in st]
    assert len(flat) == rank * len(repeats)
    return (_host_i64(coords), len(repeats), (C.c_int32 * max(len(repeats), 1))(*[int(r) for r in repeats]),
            _host_i64(flat))


def bsm_tile_box_load_steps(src: bsm_tensor, box: bsm_box, coords, repeats, steps, images, stream=None):
    """coords: rank ints; repeats: one extent per repeat axis; steps: one rank-length vector per axis."""
    c, n, r, s = _repeat_args(coords, repeats, steps)
    _check(lib().bsm_tile_box_load_steps(C.byref(src), C.byref(box), c, n, r, s, _ptr(images), _stream(stream)))


def bsm_tile_box_store_steps(dst: bsm_tensor, box: bsm_box, coords, repeats, steps, images, reduce_add: int = 0,
                             stream=None):
    c, n, r, s = _repeat_args(coords, repeats, steps)
    _check(lib().bsm_tile_box_store_steps(C.byref(dst), C.byref(box), c, n, r, s, _ptr(images), reduce_add,
                                          _stream(stream)))


def bsm_tile_gather4(src: bsm_tensor, box: bsm_box, coords, n_issues: int, images, stream=None):
    _check(lib().bsm_tile_gather4(C.byref(src), C.byref(box), _ptr(coords), n_issues, _ptr(images), _stream(stream)))


def bsm_tile_scatter4(dst: bsm_tensor, box: bsm_box, coords, n_issues: int, images, stream=None):
    _check(lib().bsm_tile_scatter4(C.byref(dst), C.byref(box), _ptr(coords), n_issues, _ptr(images),
                                   _stream(stream)))


def bsm_gemm(M, N, K, ab: str, A, lda, a_major: str, B, ldb, b_major: str, D, ldd, neg_a=0, neg_b=0,
             accum=0, stream=None):
    _check(lib().bsm_gemm(M, N, K, DTYPE[ab], _ptr(A), lda, a_major.encode(), _ptr(B), ldb, b_major.encode(),
                          _ptr(D), ldd, neg_a, neg_b, accum, _stream(stream)))


def bsm_gemm_block_scale(M, N, K, a_fmt: str, A, lda, SFA, ld_sfa, b_fmt: str, B, ldb, SFB, ld_sfb, D, ldd,
                         neg_a=0, neg_b=0, accum=0, stream=None):
    _check(lib().bsm_gemm_block_scale(M, N, K, DTYPE[a_fmt], _ptr(A), lda, _ptr(SFA), ld_sfa, DTYPE[b_fmt],
                                      _ptr(B), ldb, _ptr(SFB), ld_sfb, _ptr(D), ldd, neg_a, neg_b, accum,
                                      _stream(stream)))


def ewise_desc(op: str = "silu_affine", scale: float = 1.0, bias: float = 0.0) -> bsm_ewise:
    """A bsm_ewise epilogue: op "none" or "silu_affine" (y = x / (1 + exp(-x)); y * scale + bias)."""
    return bsm_ewise(EWISE[op] if isinstance(op, str) else int(op), scale, bias)


def bsm_gemm_ewise(M, N, K, ab: str, A, lda, a_major: str, B, ldb, b_major: str, D, ldd, neg_a=0, neg_b=0,
                   accum=0, ew: bsm_ewise | None = None, stream=None):
    _check(lib().bsm_gemm_ewise(M, N, K, DTYPE[ab], _ptr(A), lda, a_major.encode(), _ptr(B), ldb,
                                b_major.encode(), _ptr(D), ldd, neg_a, neg_b, accum,
                                C.byref(ew) if ew is not None else None, _stream(stream)))


def bsm_gemm_block_scale_ewise(M, N, K, a_fmt: str, A, lda, SFA, ld_sfa, b_fmt: str, B, ldb, SFB, ld_sfb, D, ldd,
                               neg_a=0, neg_b=0, accum=0, ew: bsm_ewise | None = None, stream=None):
    _check(lib().bsm_gemm_block_scale_ewise(M, N, K, DTYPE[a_fmt], _ptr(A), lda, _ptr(SFA), ld_sfa, DTYPE[b_fmt],
                                            _ptr(B), ldb, _ptr(SFB), ld_sfb, _ptr(D), ldd, neg_a, neg_b, accum,
                                            C.byref(ew) if ew is not None else None, _stream(stream)))


def bsm_gemm_block_scale_major(M, N, K, a_fmt: str, A, lda, a_major: str, SFA, ld_sfa, b_fmt: str, B, ldb,
                               b_major: str, SFB, ld_sfb, D, ldd, neg_a=0, neg_b=0, accum=0,
                               ew: bsm_ewise | None = None, stream=None):
    _check(lib().bsm_gemm_block_scale_major(M, N, K, DTYPE[a_fmt], _ptr(A), lda, a_major.encode(), _ptr(SFA), ld_sfa,
                                            DTYPE[b_fmt], _ptr(B), ldb, b_major.encode(), _ptr(SFB), ld_sfb, _ptr(D),
                                            ldd, neg_a, neg_b, accum, C.byref(ew) if ew is not None else None,
                                            _stream(stream)))


def bsm_gemm_block_scale_fastacc(M, N, K, a_fmt: str, A, lda, SFA, ld_sfa, b_fmt: str, B, ldb, SFB, ld_sfb, D, ldd,
                                 neg_a=0, neg_b=0, accum=0, ew: bsm_ewise | None = None, stream=None):
    _check(lib().bsm_gemm_block_scale_fastacc(M, N, K, DTYPE[a_fmt], _ptr(A), lda, _ptr(SFA), ld_sfa, DTYPE[b_fmt],
                                              _ptr(B), ldb, _ptr(SFB), ld_sfb, _ptr(D), ldd, neg_a, neg_b, accum,
                                              C.byref(ew) if ew is not None else None, _stream(stream)))


def _here(stream, *tensors):
    """The stream's handle, once every torch tensor given is known to live on the current device: the kernels
    take addresses, and one of the host or of another device would fault them. Work on another device goes
    under torch.cuda.device of that device."""
    at = -2
    for t in tensors:
        if t is None or type(t) is int:
            continue
        d = t.get_device()
        if d == at:
            continue
        if d < 0:
            raise BsmError(-13, f"a tensor on {t.device}: the library takes device memory")
        if _torch_c is None:
            _fill_torch_c()
        if d != _torch_c._cuda_getDevice():   # (current_device() without the check that CUDA is initialised: it holds t)
            raise BsmError(-13, f"a tensor on {t.device} while the current device is cuda:{_torch_c._cuda_getDevice()}")
        at = d
    if stream is None and at >= 0:
        return _torch_c._cuda_getCurrentRawStream(at)   # (current_stream() without the object around it)
    return _stream(stream)


_torch_c = None


def _fill_torch_c():
    global _torch_c
    import torch
    _torch_c = torch._C


_dtypes = {}


def _array(t, dtype: str, what, least):
    """Address of a DEVICE array of at least `least` elements, its type, order and length checked where it is a torch tensor."""
    if t is None or type(t) is int:
        return t
    if dtype not in _dtypes:
        import torch
        _dtypes[dtype] = getattr(torch, dtype)
    if t.dtype is _dtypes[dtype] and t.is_contiguous() and t.numel() >= least:
        return t.data_ptr()
    if t.dtype is not _dtypes[dtype]:
        raise BsmError(-8, f"{what} must be {dtype}, not {t.dtype}")
    if not t.is_contiguous():
        raise BsmError(-5, f"{what} must be contiguous")
    raise BsmError(-9, f"{what} holds {t.numel()} elements, the call takes {least}")


def _workspace(t, least):
    if t is None or type(t) is int:
        return t
    if not t.is_contiguous():
        raise BsmError(-5, "workspace must be contiguous")
    if t.numel() * t.element_size() < least:
        raise BsmError(-9, f"workspace holds {t.numel() * t.element_size()} bytes, the call takes {least}")
    return t.data_ptr()


_SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def _output(t, d_fmt: str, n, stride, rows, cols, ld):
    """Address of the output D of n matrices of rows x cols elements, `stride` apart, which a torch tensor (of any type) has
    to hold from its start on: the kernels write to its last row's end."""
    if t is None or type(t) is int or n <= 0 or rows <= 0 or cols <= 0:
        return _ptr(t)
    need = ((n - 1) * stride + (rows - 1) * ld + cols) * _SIZE.get(d_fmt, 0)
    size = t.element_size()
    if not (t.is_contiguous() and t.numel() * size >= need):   # (as nearly every call has it)
        have = t.untyped_storage().nbytes() - t.storage_offset() * size
        if have < need:
            raise BsmError(-9, f"D holds {have} bytes from its start on, the call writes to byte {need}")
    return _ptr(t)


def bsm_gemm_grouped(rows, N, K, n_groups, offsets, ab: str, A, lda, B, ldb, b_major: str, stride_b, d_fmt: str, D, ldd,
                     accum=0, ew: bsm_ewise | None = None, stream=None):
    # (a call without groups, rows or columns reads no offsets)
    off = _array(offsets, "int32", "offsets", n_groups + 1 if n_groups > 0 and rows > 0 and N > 0 else 0)
    s = _here(stream, offsets, A, B, D)
    d = _output(D, d_fmt, min(n_groups, 1), 0, rows, N, ldd)
    _check(lib().bsm_gemm_grouped(rows, N, K, n_groups, off, DTYPE[ab], _ptr(A), lda, _ptr(B), ldb,
                                  b_major.encode(), stride_b, DTYPE[d_fmt], d, ldd, accum,
                                  C.byref(ew) if ew is not None else None, s))


def bsm_gemm_grouped_wgrad(rows, M, N, n_groups, offsets, ab: str, A, lda, B, ldb, d_fmt: str, D, ldd, stride_d, accum=0,
                           stream=None):
    # (a call without groups, rows of D or columns reads no offsets)
    off = _array(offsets, "int32", "offsets", n_groups + 1 if n_groups > 0 and M > 0 and N > 0 else 0)
    s = _here(stream, offsets, A, B, D)
    d = _output(D, d_fmt, n_groups, stride_d, M, N, ldd)
    _check(lib().bsm_gemm_grouped_wgrad(rows, M, N, n_groups, off, DTYPE[ab], _ptr(A), lda, _ptr(B), ldb,
                                        DTYPE[d_fmt], d, ldd, stride_d, accum, s))


def bsm_gemm_grouped_block_scale(rows, N, K, n_groups, offsets, a_fmt: str, A, lda, SFA, ld_sfa, b_fmt: str, B, ldb, stride_b,
                                 SFB, ld_sfb, stride_sfb, fast, d_fmt: str, D, ldd, accum=0, ew: bsm_ewise | None = None,
                                 stream=None):
    # (a call without groups, rows or columns reads no offsets)
    off = _array(offsets, "int32", "offsets", n_groups + 1 if n_groups > 0 and rows > 0 and N > 0 else 0)
    s = _here(stream, offsets, A, SFA, B, SFB, D)
    d = _output(D, d_fmt, min(n_groups, 1), 0, rows, N, ldd)
    _check(lib().bsm_gemm_grouped_block_scale(rows, N, K, n_groups, off, DTYPE[a_fmt], _ptr(A), lda,
                                              _ptr(SFA), ld_sfa, DTYPE[b_fmt], _ptr(B), ldb, stride_b, _ptr(SFB), ld_sfb,
                                              stride_sfb, fast, DTYPE[d_fmt], d, ldd, accum,
                                              C.byref(ew) if ew is not None else None, s))


def bsm_gemm_lora_workspace(rows, R) -> int:
    return _check(lib().bsm_gemm_lora_workspace(rows, R))


def bsm_gemm_lora(rows, N, K, R, n_adapters, adapter, ab: str, X, ldx, W, ldw, LA, ld_la, stride_la, LB, ld_lb, stride_lb, scale,
                  workspace, d_fmt: str, D, ldd, accum=0, ew: bsm_ewise | None = None, stream=None):
    with_adapters = n_adapters > 0 and R > 0 and K > 0 and N > 0
    ids = _array(adapter, "int32", "adapter", rows if with_adapters else 0)
    scales = _array(scale, "float32", "scale", n_adapters if with_adapters else 0)
    work = _workspace(workspace, rows * ((R + 31) // 32 * 32) * 4 if with_adapters else 0)
    s = _here(stream, adapter, X, W, LA, LB, scale, workspace, D)
    d = _output(D, d_fmt, 1, 0, rows, N, ldd)
    _check(lib().bsm_gemm_lora(rows, N, K, R, n_adapters, ids, DTYPE[ab], _ptr(X), ldx, _ptr(W), ldw, _ptr(LA), ld_la, stride_la,
                               _ptr(LB), ld_lb, stride_lb, scales, work, DTYPE[d_fmt], d, ldd, accum,
                               C.byref(ew) if ew is not None else None, s))


def _rows(t, dtype: str, what, rows, n, ld, chunk=1):
    """Address of a DEVICE matrix of `rows` rows of n elements, ld apart; where it is a torch tensor, of the type that
    the call says ("u8", codes and scales: any of one byte), its rows contiguous, and reaching to the last row's end, in
    whole chunks where the kernels read it in such."""
    if type(t) is int or t is None:
        return t
    if not _torch_types:
        _fill_torch_types()
    same = t.dtype is _torch_types[dtype]
    if same and t.is_contiguous() and t.numel() >= rows * ld:   # (as nearly every call has it)
        return t.data_ptr()
    if not same and (dtype != "u8" or t.element_size() != 1):
        raise BsmError(-8, f"{what} must be {dtype}, not {t.dtype}")
    if rows > 0 and n > 0:
        if t.dim() and t.stride(-1) != 1 and t.shape[-1] > 1:
            raise BsmError(-5, f"{what}: a row's elements must lie one after another")
        need = (rows - 1) * ld + -(-n // chunk) * chunk
        have = t.untyped_storage().nbytes() // t.element_size() - t.storage_offset()
        if have < need:
            raise BsmError(-9, f"{what} holds {have} elements from its start on, the call takes {need}")
    return t.data_ptr()


_torch_types = {}


def _fill_torch_types():
    import torch
    _torch_types.update(f32=torch.float32, f16=torch.float16, bf16=torch.bfloat16, u8=torch.uint8)


def _float_fmt(fmt: str, what):
    if fmt not in ("f32", "bf16", "f16"):
        raise BsmError(-8, f"{what} = {fmt} is not f32, bf16 or f16")


def bsm_router_balance_workspace(rows, n_experts) -> int:
    return _check(lib().bsm_router_balance_workspace(rows, n_experts))


def bsm_router_balance(rows, n_experts, k, l_fmt: str, logits, ldl, ids, scale, counts, offsets, loss, workspace=None, stream=None):
    _float_fmt(l_fmt, "l_fmt")
    x = _rows(logits, l_fmt, "logits", rows, n_experts, ldl)
    i = _array(ids, "int32", "ids", rows * k)
    c, o = _array(counts, "int32", "counts", n_experts + 1), _array(offsets, "int32", "offsets", n_experts + 1)
    f = _array(loss, "float32", "loss", 1)
    work = _workspace(workspace, lib().bsm_router_balance_workspace(rows, n_experts))
    s = _here(stream, logits, ids, counts, offsets, loss, workspace)
    _check(lib().bsm_router_balance(rows, n_experts, k, DTYPE[l_fmt], x, ldl, i, scale, c, o, f, work, s))


def bsm_router_balance_grad(rows, n_experts, k, l_fmt: str, logits, ldl, ids, counts, scale, dloss, d_fmt: str, D, ldd, accum=0,
                            stream=None):
    _float_fmt(l_fmt, "l_fmt")
    _float_fmt(d_fmt, "d_fmt")
    x = _rows(logits, l_fmt, "logits", rows, n_experts, ldl)
    i = _array(ids, "int32", "ids", rows * k)
    c, g = _array(counts, "int32", "counts", n_experts + 1), _array(dloss, "float32", "dloss", 1)
    d = _rows(D, d_fmt, "D", rows, n_experts, ldd)
    s = _here(stream, logits, ids, counts, dloss, D)
    _check(lib().bsm_router_balance_grad(rows, n_experts, k, DTYPE[l_fmt], x, ldl, i, c, scale, g, DTYPE[d_fmt], d, ldd, accum, s))


def bsm_block_scale_save(rows, K, x_fmt: str, X, ldx, fmt: str, Q, ldq, SF, ld_sf, stream=None):
    _float_fmt(x_fmt, "x_fmt")
    x = _rows(X, x_fmt, "X", rows, K, ldx, 4 if x_fmt == "f32" else 8)
    q, f = _rows(Q, "u8", "Q", rows, K, ldq), _rows(SF, "u8", "SF", rows, (K + 31) // 32, ld_sf)
    s = _here(stream, X, Q, SF)
    _check(lib().bsm_block_scale_save(rows, K, DTYPE[x_fmt], x, ldx, DTYPE[fmt], q, ldq, f, ld_sf, s))


def bsm_block_scale_restore(rows, K, fmt: str, Q, ldq, SF, ld_sf, d_fmt: str, D, ldd, ew: bsm_ewise | None = None, stream=None):
    _float_fmt(d_fmt, "d_fmt")
    q, f = _rows(Q, "u8", "Q", rows, K, ldq, 8), _rows(SF, "u8", "SF", rows, (K + 31) // 32, ld_sf)
    d = _rows(D, d_fmt, "D", rows, K, ldd)
    s = _here(stream, Q, SF, D)
    _check(lib().bsm_block_scale_restore(rows, K, DTYPE[fmt], q, ldq, f, ld_sf, DTYPE[d_fmt], d, ldd,
                                         C.byref(ew) if ew is not None else None, s))


def bsm_block_scale_ewise_grad(rows, K, fmt: str, Q, ldq, SF, ld_sf, dy_fmt: str, dY, lddy, D, ldd, ew: bsm_ewise, stream=None):
    _float_fmt(dy_fmt, "dy_fmt")
    q, f = _rows(Q, "u8", "Q", rows, K, ldq, 8), _rows(SF, "u8", "SF", rows, (K + 31) // 32, ld_sf)
    y, d = _rows(dY, dy_fmt, "dY", rows, K, lddy, 4 if dy_fmt == "f32" else 8), _rows(D, dy_fmt, "D", rows, K, ldd)
    s = _here(stream, Q, SF, dY, D)
    _check(lib().bsm_block_scale_ewise_grad(rows, K, DTYPE[fmt], q, ldq, f, ld_sf, DTYPE[dy_fmt], y, lddy, d, ldd,
                                            C.byref(ew) if ew is not None else None, s))


def bsm_gemm_grouped_wgrad_block_scale(rows, M, N, n_groups, offsets, ab: str, A, lda, b_fmt: str, B, ldb, SFB, ld_sfb, d_fmt: str,
                                       D, ldd, stride_d, accum=0, stream=None):
    _operand_fmt(ab)
    _float_fmt(d_fmt, "d_fmt")
    # (a call without groups, rows of D or columns reads no offsets)
    some = n_groups > 0 and M > 0 and N > 0
    off = _array(offsets, "int32", "offsets", n_groups + 1 if some else 0)
    r = rows if some else 0
    x, c = _rows(A, ab, "A", r, M, lda, 8), _rows(B, "u8", "B", r, N, ldb, 16)
    f = _rows(SFB, "u8", "SFB", r, (N + 31) // 32, ld_sfb, 4)
    need = (n_groups - 1) * stride_d + (M - 1) * ldd + N
    d = _rows(D, d_fmt, "D", 1 if some else 0, need, need)
    s = _here(stream, offsets, A, B, SFB, D)
    _check(lib().bsm_gemm_grouped_wgrad_block_scale(rows, M, N, n_groups, off, DTYPE[ab], x, lda, DTYPE[b_fmt], c, ldb, f, ld_sfb,
                                                    DTYPE[d_fmt], d, ldd, stride_d, accum, s))


def bsm_gemm_cross_entropy_workspace(rows, N) -> int:
    return _check(lib().bsm_gemm_cross_entropy_workspace(rows, N))


def bsm_gemm_cross_entropy_grad_workspace(rows, N, K, piece=0) -> int:
    return _check(lib().bsm_gemm_cross_entropy_grad_workspace(rows, N, K, piece))


def _operand_fmt(ab: str):
    if ab not in ("bf16", "f16"):
        raise BsmError(-8, f"ab = {ab} is neither bf16 nor f16")


def bsm_gemm_cross_entropy(rows, N, K, ab: str, X, ldx, W, ldw, labels, loss, lse, workspace, stream=None):
    _operand_fmt(ab)
    x, v = _rows(X, ab, "X", rows, K, ldx, 8), _rows(W, ab, "W", N if rows > 0 else 0, K, ldw, 8)
    i = _array(labels, "int32", "labels", rows)
    f, g = _array(loss, "float32", "loss", rows), _array(lse, "float32", "lse", rows)
    work = _workspace(workspace, lib().bsm_gemm_cross_entropy_workspace(rows, N))
    s = _here(stream, X, W, labels, loss, lse, workspace)
    _check(lib().bsm_gemm_cross_entropy(rows, N, K, DTYPE[ab], x, ldx, v, ldw, i, f, g, work, s))


def bsm_gemm_cross_entropy_grad(rows, N, K, ab: str, X, ldx, W, ldw, labels, lse, dloss, piece, workspace, dx_fmt: str, dX, lddx,
                                dw_fmt: str, dW, lddw, accum=0, stream=None):
    _operand_fmt(ab)
    _float_fmt(dx_fmt, "dx_fmt")
    _float_fmt(dw_fmt, "dw_fmt")
    x, v = _rows(X, ab, "X", rows, K, ldx, 8), _rows(W, ab, "W", N if rows > 0 else 0, K, ldw, 8)
    i = _array(labels, "int32", "labels", rows)
    f, g = _array(lse, "float32", "lse", rows), _array(dloss, "float32", "dloss", rows)
    dx, dw = _rows(dX, dx_fmt, "dX", rows, K, lddx), _rows(dW, dw_fmt, "dW", N, K, lddw)
    work = _workspace(workspace, lib().bsm_gemm_cross_entropy_grad_workspace(rows, N, K, piece) if rows > 0 and K > 0 else 0)
    s = _here(stream, X, W, labels, lse, dloss, dX, dW, workspace)
    _check(lib().bsm_gemm_cross_entropy_grad(rows, N, K, DTYPE[ab], x, ldx, v, ldw, i, f, g, piece, work, DTYPE[dx_fmt], dx, lddx,
                                             DTYPE[dw_fmt], dw, lddw, accum, s))


def bsm_tile_add_scalar_f32(src, dst, n: int, s: float, stream=None):
    _check(lib().bsm_tile_add_scalar_f32(_ptr(src), _ptr(dst), n, s, _stream(stream)))


def bsm_debug_fragment_shape():
    r, k = C.c_int64(0), C.c_int64(0)
    lib().bsm_debug_fragment_shape(C.byref(r), C.byref(k))
    return r.value, k.value


def bsm_debug_fragments(src, rows: int, kdim: int, major: str, dump, stream=None):
    _check(lib().bsm_debug_fragments(_ptr(src), rows, kdim, major.encode(), _ptr(dump), _stream(stream)))


def bsm_debug_stream_mix_bf16(src, dst, add, n: int, stream=None):
    _check(lib().bsm_debug_stream_mix_bf16(_ptr(src), _ptr(dst), _ptr(add), n, _stream(stream)))


def bsm_debug_grouped_route(call: str, rows, N, K=0, n=1, M=0, R=0, a_fmt: str = "bf16", b_fmt: str = "bf16", b_major: str = "k",
                            fast=0, shrink=0) -> str:
    name = lib().bsm_debug_grouped_route(call.encode(), rows, M, N, K, R, n, DTYPE[a_fmt], DTYPE[b_fmt], b_major.encode(), fast,
                                         shrink)
    if name is None:
        raise BsmError(-13 if call not in "gwma" else -9, bsm_last_error())
    return name.decode()


def bsm_debug_mfma_loop(kind: str, workgroups: int, iters: int, out, stream=None):
    _check(lib().bsm_debug_mfma_loop(DTYPE[kind], workgroups, iters, _ptr(out), _stream(stream)))
