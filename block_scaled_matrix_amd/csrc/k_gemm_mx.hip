// k_gemm_mx.hip - block-scaled GEMM (MXFP8 E4M3 or E5M2 / MXFP4 E2M1 with E8M0 scales per 32
// K elements) D = s * A * B^T (+ D) on gfx950 v_mfma_scale_f32_32x32x64_f8f6f4, K-major
// operands. The other pairings (6-bit formats, mixed widths) and MN-major operands go to
// the general kernel (gemm_mx_any.hpp; k_gemm_mx_any.hip, k_gemm_mx_mn_*.hip).
//
// Semantics ("tcgen05.mma": Weight-stationary and block scaling, Call parameters;
// "Explicit CUDA tile patterns": tcgen05 MMA): operand value = element * 2^(scale-127)
// with one scale per 32 consecutive K elements of a row, float32 accumulation.
//
// gfx950 design (operand layouts probed on the device):
//  - the scaled MFMA takes per lane one 32-bit register of scales and selects a byte
//    with op_sel; for K = 64 per instruction the scale of row i, block b (32 K) is
//    taken from lane i + 32*b;
//  - fp8 operand (32 bytes per lane): lane l holds row l%32 with k in
//    [16(l/32), +16) and [32 + 16(l/32), +16) of the 64-K step;
//  - fp4 operand (16 bytes per lane, two elements per byte, low nibble first): lane l
//    holds row l%32 with k in [32(l/32), +32);
//  - the MFMA is issued with the operands swapped (B first, with B's scales), so a lane
//    holds four consecutive output columns per register group (16-byte epilogue);
//  - workgroup tile 256 x 256 x (128 bytes of K per row), four wave64s with 128 x 128
//    sub-tiles (4 x 4 accumulators of 16 fp32 in AGPRs); operand tiles (whole 128-byte
//    lines per row, the 128-byte-row XOR swizzle shared with the dense kernel) stream
//    HBM -> LDS with global_load_lds_dwordx4 into two stages;
//  - scale words reach LDS through a ring of two groups of 32 bytes per row (8 K tiles
//    of fp8, 4 of fp4), copied a slice per K tile with 8 rows per 4-byte-per-lane copy:
//    measured on the device, a copy whose 64 lanes touch 64 rows occupies the copy path
//    four times as long as a 1 KiB operand copy, one touching 8 rows 0.6 times as long;
//  - each wave reads a tile's fragments into registers early, so a stage is released
//    during the tile's first 64-K step and the copy of tile kt+2 starts while tile kt is
//    still being multiplied: two K tiles stay in flight;
//  - fragment reads, copies and barriers are placed one by one between the MFMAs: four
//    wave bursts of copies would block the issuing waves behind the shared copy path
//    while the matrix pipe idles, whereas one copy per 64-cycle fp8 MFMA (per two 32-cycle
//    fp4 MFMAs) keeps it fed in the background.
#include "gemm_mx_tile.hpp"

namespace bsm {

using namespace mxtile;

hipError_t launch_gemm_mx(const GemmArgs& a, hipStream_t st) {
  if (a.K == 0) return launch_empty_gemm(a.D, a.ldd, a.M, a.N, a.accum, a.ew_op, a.ew_scale, a.ew_bias, st);
  const bool byte_a = a.dtype == BSM_E4M3 || a.dtype == BSM_E5M2, byte_b = a.dtype_b == BSM_E4M3 || a.dtype_b == BSM_E5M2;
  if (!a.a_kmajor && !a.b_kmajor) return launch_gemm_mx_mn_ab(a, st);
  if (!a.a_kmajor) return launch_gemm_mx_mn_a(a, st);
  if (!a.b_kmajor) return launch_gemm_mx_mn_b(a, st);
  if (!(byte_a && byte_b) && !(a.dtype == BSM_E2M1 && a.dtype_b == BSM_E2M1)) return launch_gemm_mx_any(a, st);
  // 8-bit pairs sum exactly only through the general kernel's bf16 route; this kernel's
  // scaled fp8 MFMA serves calls that take its accumulation window
  if (byte_a && byte_b && !a.mx_window) return launch_gemm_mx_any(a, st);
  const int64_t tm64 = (a.M + BM - 1) / BM, tn64 = (a.N + BN - 1) / BN;
  if (tm64 * tn64 > 0x7FFFFFFF) return hipErrorInvalidValue;
  const int tiles_m = (int)tm64, tiles_n = (int)tn64;
  const dim3 grid(tiles_m * tiles_n);
  const gemm::WholeProduct where{tiles_m, tiles_n};
  // MFMA format codes: E4M3 0, E5M2 1, E2M1 4 (fp4 pairs only with fp4)
#define BSM_MX_LAUNCH(FMT, CA, CB)                                                                              \
  do {                                                                                                            \
    if (a.accum) hipLaunchKernelGGL((k_gemm_mx<FMT, CA, CB, true, gemm::WholeProduct, BSM_F32>), grid, dim3(256), 0, st, a, where);  \
    else hipLaunchKernelGGL((k_gemm_mx<FMT, CA, CB, false, gemm::WholeProduct, BSM_F32>), grid, dim3(256), 0, st, a, where);         \
  } while (0)
  const bool a5 = a.dtype == BSM_E5M2, b5 = a.dtype_b == BSM_E5M2;
  if (a.dtype == BSM_E2M1) BSM_MX_LAUNCH(4, 4, 4);
  else if (!a5 && !b5) BSM_MX_LAUNCH(0, 0, 0);
  else if (a5 && b5) BSM_MX_LAUNCH(0, 1, 1);
  else if (a5) BSM_MX_LAUNCH(0, 1, 0);
  else BSM_MX_LAUNCH(0, 0, 1);
#undef BSM_MX_LAUNCH
  return hipGetLastError();
}

}  // namespace bsm
