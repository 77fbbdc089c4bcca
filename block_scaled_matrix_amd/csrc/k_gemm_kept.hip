// k_gemm_kept.hip - the weight gradient of products over groups of rows from activations kept in 8 bits:
//
//   D_g[m, n] = (D_g[m, n] +) sum_{r in group g} Y[r, m] code[r, n] 2^(scale[r, n / 32] - 127)
//
// on the tiles of gemm_kept_tile.hpp; groups as in grouped.hpp.
#include "gemm_kept_tile.hpp"
#include "grouped.hpp"

namespace bsm {
namespace {

// Workgroup p runs on XCD p % 8. Every XCD gets a contiguous eighth of each group's tiles (groups in turn), so that the
// groups' row counts, which are the tiles' lengths here, do not unbalance the XCDs, while the tiles that share a group's
// panels still meet in one L2.
template <int DT, int FMT, int BM>
__global__ __launch_bounds__(256, 2) void k_kept_wgrad(GemmArgs a, GroupArgs gr, int tiles_m, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[keptmm::lds_bytes<BM>()];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = tiles_m * tiles_n, share = (per + 7) >> 3, pid = blockIdx.x, x = pid & 7, q = pid >> 3;
  const int g = q / share, in = x * share + (q - g * share);
  if (in >= per) return;
  int tm, tn, lo, hi;
  grouped::band_tile<4>(in, tiles_m, tiles_n, tm, tn);
  grouped::group_range(gr, g, lo, hi);
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi);
  GemmArgs t = a;
  t.K = hi - lo;
  t.A = (const uint16_t*)a.A + (int64_t)lo * a.lda;
  t.B = (const uint8_t*)a.B + (int64_t)lo * a.ldb;
  t.SFB = a.SFB + (int64_t)lo * a.ld_sfb;
  t.D = (float*)((uint8_t*)a.D + (int64_t)g * gr.stride_d * (a.d_fmt == BSM_F32 ? 4 : 2));
  keptmm::tile<DT, FMT, BM>(t, BM * (int64_t)tm, keptmm::BN * (int64_t)tn, lds, lane, w);
}

template <int DT, int FMT>
hipError_t launch(const GemmArgs& a, const GroupArgs& gr, hipStream_t st) {
  // 256 rows a tile where groups are long and the tiles fill the CUs (as bsm_gemm_grouped_wgrad's)
  const int64_t tn = (a.N + keptmm::BN - 1) / keptmm::BN;
  const bool tall = gr.rows / gr.n >= 192 && (a.M + 255) / 256 * tn * gr.n >= 512;
  const int64_t bm = tall ? 256 : 128, tm = (a.M + bm - 1) / bm, share = (tm * tn + 7) / 8;
  if (share > 0x7FFFFFFF / 8 / gr.n) return hipErrorInvalidValue;
  const dim3 grid((uint32_t)(share * 8 * gr.n));
  if (tall) hipLaunchKernelGGL((k_kept_wgrad<DT, FMT, 256>), grid, dim3(256), 0, st, a, gr, (int)tm, (int)tn);
  else hipLaunchKernelGGL((k_kept_wgrad<DT, FMT, 128>), grid, dim3(256), 0, st, a, gr, (int)tm, (int)tn);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(const GemmArgs& a, const GroupArgs& gr, hipStream_t st) {
  return a.dtype_b == BSM_E4M3 ? launch<DT, BSM_E4M3>(a, gr, st) : launch<DT, BSM_E5M2>(a, gr, st);
}

}  // namespace

hipError_t launch_gemm_kept_wgrad(const GemmArgs& a, const GroupArgs& gr, hipStream_t st) {
  return a.dtype == BSM_BF16 ? launch_dt<BSM_BF16>(a, gr, st) : launch_dt<BSM_F16>(a, gr, st);
}

}  // namespace bsm
