// k_gemm_grouped_mx_any.hip - block-scaled products with a weight per group of rows on the general
// kernel's tile (gemm_mx_any.hpp): E4M3 x E4M3 with exact products, E4M3 x E2M1 on both routes.
#include "gemm_mx_any.hpp"
#include "grouped_mx.hpp"

namespace bsm {

using namespace mxany;

template <int CB, bool BF, int OUT>
static hipError_t launch_any(const GemmArgs& a, const GroupArgs& gr, hipStream_t st) {
  typedef grouped::GroupProduct<8, fmt_bits(CB), OUT == BSM_F32 ? 4 : 2> Where;
  const int64_t tn = (a.N + BN - 1) / BN, n = (grouped::most_row_tiles(gr.rows, gr.n, BM) * tn + 7) / 8 * 8;
  if (n > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL((k_gemm_mx_any<0, CB, false, false, BF, Where, OUT>), dim3((uint32_t)n), dim3(256), 0, st, a,
                     Where{gr, (int)tn});
  return hipGetLastError();
}

template <int OUT>
static hipError_t launch_out(const GemmArgs& a, const GroupArgs& gr, hipStream_t st) {
  if (a.dtype_b == BSM_E4M3) return launch_any<0, true, OUT>(a, gr, st);
  return a.mx_window ? launch_any<4, false, OUT>(a, gr, st) : launch_any<4, true, OUT>(a, gr, st);
}

hipError_t launch_gemm_grouped_mx_any(const GemmArgs& a, const GroupArgs& gr, hipStream_t st) {
  return a.d_fmt == BSM_F32 ? launch_out<BSM_F32>(a, gr, st) : launch_out<BSM_BF16>(a, gr, st);
}

}  // namespace bsm
