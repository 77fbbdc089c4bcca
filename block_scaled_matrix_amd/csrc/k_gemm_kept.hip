// k_gemm_kept.hip - the weight gradient of products over groups of rows from activations kept in 8 bits:
//
//   D_g[m, n] = (D_g[m, n] +) sum_{r in group g} Y[r, m] code[r, n] 2^(scale[r, n / 32] - 127)
//
// on the tiles of gemm_kept_tile.hpp; groups as in grouped.hpp.
#include "gemm_kept_tile.hpp"
#include "grouped.hpp"

namespace bsm {
namespace {

// The group with the q-th most rows (of as many, the first), by the whole workgroup of 256: a lane ranks a group. More
// groups than that come in their order.
constexpr int kRanked = 256;
__device__ __forceinline__ int ranked_group(const GroupArgs& gr, int q, int* lds) {
  if (gr.n > kRanked) return q;
  const int t = threadIdx.x;
  int lo = 0, hi = -1;
  if (t < gr.n) grouped::group_range(gr, t, lo, hi);
  lds[t] = hi - lo;   // (-1 past the last group)
  __syncthreads();
  int rank = 0;
  for (int i = 0; i < gr.n; i += 4) {
    const i32x4 v = *(const BSM_LDS i32x4*)(lds + i);
#pragma unroll
    for (int e = 0; e < 4; e++) rank += v[e] > hi - lo || (v[e] == hi - lo && i + e < t) ? 1 : 0;
  }
  __syncthreads();
  if (t < gr.n && rank == q) lds[0] = t;
  __syncthreads();
  const int g = __builtin_amdgcn_readfirstlane(lds[0]);
  __syncthreads();
  return g;
}

// Workgroup p runs on XCD p % 8. Every XCD gets a contiguous eighth of each group's tiles, groups in turn, so that the
// groups' row counts, which are the tiles' lengths here, do not unbalance the XCDs, while the tiles that share a group's
// panels still meet in one L2. Groups come in `order`(their turn). Makes `a` the group's product and gives the tile;
// false: the workgroup has none.
template <class ORDER>
__device__ __forceinline__ bool enter(GemmArgs& a, const GroupArgs& gr, int tiles_m, int tiles_n, ORDER order, int& tm, int& tn) {
  const int per = tiles_m * tiles_n, share = (per + 7) >> 3, pid = blockIdx.x, x = pid & 7, q = pid >> 3;
  const int turn = q / share, in = x * share + (q - turn * share);
  if (in >= per) return false;
  const int g = order(turn);
  int lo, hi;
  grouped::band_tile<4>(in, tiles_m, tiles_n, tm, tn);
  grouped::group_range(gr, g, lo, hi);
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi);
  a.K = hi - lo;
  a.A = (const uint16_t*)a.A + (int64_t)lo * a.lda;
  a.B = (const uint8_t*)a.B + (int64_t)lo * a.ldb;
  a.SFB += (int64_t)lo * a.ld_sfb;
  a.D = (float*)((uint8_t*)a.D + (int64_t)g * gr.stride_d * (a.d_fmt == BSM_F32 ? 4 : 2));
  return true;
}

template <int DT, int FMT, int BM>
__global__ __launch_bounds__(256, 2) void k_kept_wgrad(GemmArgs a, GroupArgs gr, int tiles_m, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[keptmm::lds_bytes<BM>()];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tm, tn;
  if (!enter(a, gr, tiles_m, tiles_n, [](int turn) { return turn; }, tm, tn)) return;
  keptmm::tile<DT, FMT, BM>(a, BM * (int64_t)tm, keptmm::BN * (int64_t)tn, lds, lane, w);
}

// Long groups first: a tile takes its group's rows, and a long one begun last keeps its CU while the others are done (16381
// rows over 8 groups, the longest 8082 and the seventh in order: 335 us in order).
template <int DT, int FMT, int OUT, bool ACC>
__global__ __launch_bounds__(256, 1) void k_kept_wgrad_large(GemmArgs a, GroupArgs gr, int tiles_m, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[keptmm::large::LDS_BYTES];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tm, tn;
  if (!enter(a, gr, tiles_m, tiles_n, [&](int turn) { return ranked_group(gr, turn, (int*)lds); }, tm, tn)) return;
  f32x4 acc[8][8];
  keptmm::large::product<DT, FMT>(a, 256 * (int64_t)tm, 256 * (int64_t)tn, lds, lane, w, acc);
  const int64_t row0 = 256 * (int64_t)tm + 128 * (w >> 1), col0 = 256 * (int64_t)tn + 128 * (w & 1);
  if constexpr (OUT == BSM_F32) dense::store_tile16(a.D, a.ldd, a.M, a.N, row0, col0, lane, 1.0f, acc, lds + 32768 * w, ACC, 0, 0.0f, 0.0f);
  else gemm::store_tile16_bits<OUT>((uint16_t*)a.D, a.ldd, a.M, a.N, row0, col0, lane, acc, lds + 32768 * w, ACC, 0, 0.0f, 0.0f);
}

template <int DT, int FMT>
hipError_t launch(const GemmArgs& a, const GroupArgs& gr, hipStream_t st) {
  const int64_t m256 = (a.M + 255) / 256, n256 = (a.N + 255) / 256;
  const bool large = gr.rows / gr.n >= 192 && m256 * n256 * gr.n >= 218;
  const int64_t bm = large ? 256 : 128, tm = (a.M + bm - 1) / bm, tn = (a.N + bm - 1) / bm, share = (tm * tn + 7) / 8;
  if (share > 0x7FFFFFFF / 8 / gr.n) return hipErrorInvalidValue;
  const dim3 grid((uint32_t)(share * 8 * gr.n));
  if (!large) {
    hipLaunchKernelGGL((k_kept_wgrad<DT, FMT, 128>), grid, dim3(256), 0, st, a, gr, (int)tm, (int)tn);
    return hipGetLastError();
  }
  auto go = [&](auto out, auto acc) {
    hipLaunchKernelGGL((k_kept_wgrad_large<DT, FMT, decltype(out)::value, decltype(acc)::value>), grid, dim3(256), 0, st, a, gr, (int)tm, (int)tn);
  };
  auto with = [&](auto out) {
    if (a.accum) go(out, std::true_type{});
    else go(out, std::false_type{});
  };
  if (a.d_fmt == BSM_F32) with(std::integral_constant<int, BSM_F32>{});
  else with(std::integral_constant<int, DT>{});
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
