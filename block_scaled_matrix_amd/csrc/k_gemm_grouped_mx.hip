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

// Whether a call takes the 256 x 256 tiles.
static bool large_tiles(const GemmArgs& a, const GroupArgs& gr) {
  // 256 x 256 tiles (in rounds over the 256 CUs) or 128 x 128 ones (512 slots, 0.6 of the large tile's
  // rate on even groups), with half a tile lost per group and half a round at the end on the small
  // ones: at 512 and 2048 rows a group the large are faster (8190 rows over 16 groups, N 8192, K 4096 in
  // MXFP8 317 against 448 us; 16381 over 8, N 4096, K 8192 in MXFP4 329 against 590 us); 64 rows over 32 groups
  // (E4M3 x E2M1, N = K = 4096) took 162 us on them, 57 us on the small ones, 1000 rows over 4 groups (N 2048,
  // K 1024) 30 us.
  auto row_tiles = [&](double bm) { return gr.n == 1 ? (double)((gr.rows + (int64_t)bm - 1) / (int64_t)bm) : gr.rows / bm + 0.5 * gr.n; };
  const double large = (double)(((int64_t)(row_tiles(BM) * ((a.N + BN - 1) / BN)) + 255) / 256) * 256 * BM * BN;
  const double small = (row_tiles(128) * ((a.N + 127) / 128) + 256) * 128 * 128 / 0.6;
  return gr.rows / gr.n >= 192 && small >= large;
}

// Of those, whether it runs on the general kernel (exact products of 8-bit operands, mixed pairs) or the tuned one.
static bool general_kernel(const GemmArgs& a) { return a.dtype != BSM_E2M1 && (a.dtype_b == BSM_E2M1 || !a.mx_window); }

const char* route_gemm_grouped_mx(const GemmArgs& a, const GroupArgs& gr) {
  if (!large_tiles(a, gr)) return route_gemm_grouped_mx_mid(a, gr);
  return general_kernel(a) ? "k_gemm_mx_any" : "k_gemm_mx";
}

hipError_t launch_gemm_grouped_mx(const GemmArgs& a, const GroupArgs& gr, hipStream_t st) {
  if (!large_tiles(a, gr)) return launch_gemm_grouped_mx_mid(a, gr, st);
  if (general_kernel(a)) return launch_gemm_grouped_mx_any(a, gr, st);
  const bool f32 = a.d_fmt == BSM_F32;
  if (a.dtype == BSM_E2M1) return f32 ? launch_tuned<4, 4, 4, BSM_F32>(a, gr, st) : launch_tuned<4, 4, 4, BSM_BF16>(a, gr, st);
  return f32 ? launch_tuned<0, 0, 0, BSM_F32>(a, gr, st) : launch_tuned<0, 0, 0, BSM_BF16>(a, gr, st);
}

}  // namespace bsm
