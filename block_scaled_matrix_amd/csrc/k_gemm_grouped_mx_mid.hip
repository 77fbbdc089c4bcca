// k_gemm_grouped_mx_mid.hip - block-scaled products with a weight per group of rows where groups have
// few rows: tiles of 128 rows, a group's last one of as few as hold its rows (gemm_mid_mx_tile.hpp).
#include "gemm_mid_mx_tile.hpp"
#include "grouped_mx.hpp"

namespace bsm {

template <int CA, int CB, bool BF>
static __global__ __launch_bounds__(256, 2) void k_grouped_mx_mid(GemmArgs a, GroupArgs gr, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[midmx::LDS_BYTES];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  grouped::Spot s;
  if (!grouped::find_tile<128, 4>(gr, blockIdx.x, tiles_n, lane, s)) return;
  grouped::group_product<mxany::fmt_bits(CA), mxany::fmt_bits(CB)>(a, gr, s, a.d_fmt == BSM_F32 ? 4 : 2);
  const int64_t m0 = 128 * (int64_t)s.tm, n0 = midmx::BN * (int64_t)s.tn;
  const int left = s.rows - 128 * s.tm;
  if (left <= 32) midmx::tile<CA, CB, BF, 32>(a, m0, n0, lds, lane, w);
  else if (left <= 64) midmx::tile<CA, CB, BF, 64>(a, m0, n0, lds, lane, w);
  else midmx::tile<CA, CB, BF, 128>(a, m0, n0, lds, lane, w);
}

template <int CA, int CB, bool BF>
static hipError_t launch_mid(const GemmArgs& a, const GroupArgs& gr, hipStream_t st) {
  const int64_t tn = (a.N + midmx::BN - 1) / midmx::BN, n = (grouped::most_row_tiles(gr.rows, gr.n, 128) * tn + 7) / 8 * 8;
  if (n > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL((k_grouped_mx_mid<CA, CB, BF>), dim3((uint32_t)n), dim3(256), 0, st, a, gr, (int)tn);
  return hipGetLastError();
}

hipError_t launch_gemm_grouped_mx_mid(const GemmArgs& a, const GroupArgs& gr, hipStream_t st) {
  if (a.dtype == BSM_E2M1) return launch_mid<4, 4, false>(a, gr, st);
  if (a.dtype_b == BSM_E2M1) return a.mx_window ? launch_mid<0, 4, false>(a, gr, st) : launch_mid<0, 4, true>(a, gr, st);
  return a.mx_window ? launch_mid<0, 0, false>(a, gr, st) : launch_mid<0, 0, true>(a, gr, st);
}

}  // namespace bsm
