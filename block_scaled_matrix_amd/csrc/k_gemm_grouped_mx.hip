// k_gemm_grouped_mx.hip - block-scaled products with a weight per group of rows: E4M3 pairs on the
// scaled fp8 MFMA (fast accumulation) and E2M1 pairs, on the tuned kernel's tile (gemm_mx_tile.hpp).
#include "gemm_mx_tile.hpp"
#include "grouped_mx.hpp"

namespace bsm {

using namespace mxtile;

template <int FMT, int CA, int CB, int OUT>
static hipError_t launch_tuned(const GemmArgs& a, const GroupArgs& gr, hipStream_t st) {
  constexpr int BITS = FMT == 4 ? 4 : 8;
  typedef grouped::GroupProduct<BITS, BITS, OUT == BSM_F32 ? 4 : 2> Where;
  const int64_t tn = (a.N + BN - 1) / BN, n = (grouped::most_row_tiles(gr.rows, gr.n, BM) * tn + 7) / 8 * 8;
  if (n > 0x7FFFFFFF) return hipErrorInvalidValue;
  const Where where{gr, (int)tn};
  const dim3 grid((uint32_t)n);
  if (a.accum) hipLaunchKernelGGL((k_gemm_mx<FMT, CA, CB, true, Where, OUT>), grid, dim3(256), 0, st, a, where);
  else hipLaunchKernelGGL((k_gemm_mx<FMT, CA, CB, false, Where, OUT>), grid, dim3(256), 0, st, a, where);
  return hipGetLastError();
}

hipError_t launch_gemm_grouped_mx(const GemmArgs& a, const GroupArgs& gr, hipStream_t st) {
  // Few rows a group: 64 rows over 32 groups (E4M3 x E2M1, N 4096, K 4096) 65.6 us against 162 us on 256 x 256
  // tiles; at 512 and 2048 rows a group those are faster (MXFP8 317 against 448 us, MXFP4 329 against 590 us).
  if (gr.rows / gr.n < 192) return launch_gemm_grouped_mx_mid(a, gr, st);
  const bool f32 = a.d_fmt == BSM_F32;
  if (a.dtype == BSM_E2M1 && a.dtype_b == BSM_E2M1)
    return f32 ? launch_tuned<4, 4, 4, BSM_F32>(a, gr, st) : launch_tuned<4, 4, 4, BSM_BF16>(a, gr, st);
  if (a.dtype_b == BSM_E2M1 || !a.mx_window) return launch_gemm_grouped_mx_any(a, gr, st);
  return f32 ? launch_tuned<0, 0, 0, BSM_F32>(a, gr, st) : launch_tuned<0, 0, 0, BSM_BF16>(a, gr, st);
}

}  // namespace bsm
