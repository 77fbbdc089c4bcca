// k_gemm_kept.hip - the weight gradient of products over groups of rows from activations kept in 8 bits:
//
//   D_g[m, n] = (D_g[m, n] +) sum_{r in group g} Y[r, m] code[r, n] 2^(scale[r, n / 32] - 127)
//
// on the tiles of gemm_kept_tile.hpp; groups as in grouped.hpp.
#include "gemm_kept_tile.hpp"
#include "grouped.hpp"
#include "store_large.hpp"

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

template <int DT, int FMT, int SIZE, int R, int Q>
__global__ __launch_bounds__(256 * Q, 4) void k_kept_wgrad(GemmArgs a, GroupArgs gr, int tiles_m, int tiles_n) {
  constexpr int LDS = keptmm::mid2::lds_bytes<SIZE, R>();
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Q * LDS];
  const int lane = threadIdx.x & 63, wq = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wq & 3, q = wq >> 2;
  int tm, tn;
  if (!enter(a, gr, tiles_m, tiles_n, [](int turn) { return turn; }, tm, tn)) return;
  keptmm::mid2::tile<DT, FMT, SIZE, R, Q>(a, SIZE * (int64_t)tm, SIZE * (int64_t)tn, lds + q * LDS, lds, lane, w, q);
}

// The 128 x 128 tile at (m0, n0) of the product whose arguments lie in LDS, for a workgroup of the large tiles. A function, not
// inlined: the large tile's loop pays for what stands beside it in registers.
constexpr int kArgsAt = 128 * 1024;
static_assert(keptmm::mid2::lds_bytes<128, 2>() <= kArgsAt && kArgsAt + sizeof(GemmArgs) <= keptmm::large::LDS_BYTES, "the arguments in LDS");
template <int DT, int FMT>
__device__ __attribute__((noinline)) void small_tile(uint32_t lds0, int m0, int n0) {
  // (the same in every lane, which the compiler does not know of a function's arguments)
  auto same = [](auto x) {
    if constexpr (sizeof(x) == 4) return (decltype(x))__builtin_amdgcn_readfirstlane(x);
    else {
      const uint64_t b = __builtin_bit_cast(uint64_t, x);
      const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b), hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
      return __builtin_bit_cast(decltype(x), (uint64_t)hi << 32 | lo);
    }
  };
  lds0 = same(lds0);
  uint8_t* lds = (uint8_t*)(BSM_LDS uint8_t*)(uintptr_t)lds0;
  const BSM_LDS GemmArgs* v = (const BSM_LDS GemmArgs*)(uintptr_t)(lds0 + kArgsAt);
  GemmArgs a{};
  a.M = same(v->M); a.N = same(v->N); a.K = same(v->K);
  a.A = same(v->A); a.lda = same(v->lda); a.B = same(v->B); a.ldb = same(v->ldb);
  a.SFB = same(v->SFB); a.ld_sfb = same(v->ld_sfb);
  a.D = same(v->D); a.ldd = same(v->ldd); a.d_fmt = same(v->d_fmt); a.accum = same(v->accum);
  const int t = threadIdx.x;
  keptmm::mid2::tile<DT, FMT, 128, 2, 1>(a, same(m0), same(n0), lds, lds, t & 63, same(t >> 6), 0);
}

// Long groups first: a tile takes its group's rows, and a long one begun last keeps its CU while the others are done (16381
// rows over 8 groups, the longest 8082 and the seventh in order: 335 us in order).
template <int DT, int FMT, int OUT, dense::Add ADD>
__global__ __launch_bounds__(256, 1) void k_kept_wgrad_large(GemmArgs a, GroupArgs gr, int tiles_m, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[keptmm::large::LDS_BYTES];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tm, tn;
  if (!enter(a, gr, tiles_m, tiles_n, [&](int turn) { return ranked_group(gr, turn, (int*)lds); }, tm, tn)) return;
  f32x4 acc[8][8];
  const bool wide = keptmm::large::product<DT, FMT>(a, 256 * (int64_t)tm, 256 * (int64_t)tn, lds, lane, w, acc);
  if constexpr (DT == BSM_BF16) {
    // A scale so wide that a finite code may lie beyond bf16's range: the tile again as small ones, which bound what they
    // convert. (In the loop itself a bound in every conversion takes 16381 rows over 8 groups, 4096 x 2048 from 267 to 290 us, a
    // branch round it 287, one branch a K tile 311; this 1%.)
    ((int*)lds)[w] = __any(wide);   // (every wave is done with LDS)
    __syncthreads();
    const int4 met = *(const int4*)lds;
    __syncthreads();
    if (__builtin_expect(__builtin_amdgcn_readfirstlane(met.x | met.y | met.z | met.w), 0)) {
      BSM_LDS GemmArgs* v = (BSM_LDS GemmArgs*)(uintptr_t)(gemm::lds_addr(lds) + kArgsAt);
      if (threadIdx.x == 0) {   // (one by one: a copy of the whole kept the arguments in memory)
        v->M = a.M; v->N = a.N; v->K = a.K;
        v->A = a.A; v->lda = a.lda; v->B = a.B; v->ldb = a.ldb;
        v->SFB = a.SFB; v->ld_sfb = a.ld_sfb;
        v->D = a.D; v->ldd = a.ldd; v->d_fmt = a.d_fmt; v->accum = a.accum;
      }
      for (int i = 0; i < 4; i++) {
        const int64_t m = 256 * (int64_t)tm + 128 * (i >> 1), n = 256 * (int64_t)tn + 128 * (i & 1);
        __syncthreads();
        if (m < a.M && n < a.N) small_tile<DT, FMT>(gemm::lds_addr(lds), (int)m, (int)n);
      }
      return;
    }
  }
  const int64_t row0 = 256 * (int64_t)tm + 128 * (w >> 1), col0 = 256 * (int64_t)tn + 128 * (w & 1);
  dense::store_large<OUT, ADD>(a, row0, col0, lane, acc, lds + 32768 * w);
}

enum Tile { FEW_SHORT, FEW_LONG, SPLIT, MID, LARGE };

// Times in us, E4M3 codes, float32 sums, groups of one length:
//  - 256 x 256 from 700 rows a group on, where they fill the best part of a round: 500 / 1000 / 2000 rows, 4096 x 4096
//    35 / 47 / 72 against 33 / 52 / 89 on 128 x 128; 8 groups of 500 / 1000 rows, 2048 x 2048 64 / 88 against 55 / 107;
//  - up to 64 tiles of 128 x 128, a quarter of the CUs: 64 x 64, two sets of waves a tile, from 800 rows on four (200 / 500 /
//    1000 / 4000 rows, 1024 x 1024: two 7.5 / 8.9 / 13.5 / 41, four 7.6 / 9.2 / 12.6 / 34, 128 x 128 10.9 / 15.6 / 24 / 73);
//  - up to 192: long groups 128 x 128 with four sets of waves (4000 rows, 2048 x 1024 56 against 75 with one set, 57 on 64 x
//    64; 2 groups of 8000, 1024 x 1024 100, 138 and 103), others 64 x 64 with two (1000 rows, 2048 x 1024 19.5 against
//    24.7 on 128 x 128; 200 rows 9.3 and 11.0);
//  - 128 x 128, four workgroups a CU (1021 rows over 32 groups, 1024 x 512 16.2 against 17.4 on 64 x 64).
Tile tile_for(const GemmArgs& a, const GroupArgs& gr) {
  const int64_t n = gr.n, each = gr.rows / n, t128 = (a.M + 127) / 128 * ((a.N + 127) / 128) * n;
  if (each >= 700 && (a.M + 255) / 256 * ((a.N + 255) / 256) * n >= 218) return LARGE;
  if (t128 <= 64) return each >= 800 ? FEW_LONG : FEW_SHORT;
  if (t128 <= 192) return each >= 1500 ? SPLIT : FEW_SHORT;
  return MID;
}

template <int DT, int FMT>
hipError_t launch(const GemmArgs& a, const GroupArgs& gr, hipStream_t st) {
  const Tile tile = tile_for(a, gr);
  const int64_t size = tile == LARGE ? 256 : tile == MID || tile == SPLIT ? 128 : 64;
  const int64_t m = (a.M + size - 1) / size, n = (a.N + size - 1) / size, share = (m * n + 7) / 8;
  if (share > 0x7FFFFFFF / 8 / gr.n) return hipErrorInvalidValue;
  const dim3 grid((uint32_t)(share * 8 * gr.n));
  const int tm = (int)m, tn = (int)n;
  switch (tile) {
    case FEW_SHORT: hipLaunchKernelGGL((k_kept_wgrad<DT, FMT, 64, 3, 2>), grid, dim3(512), 0, st, a, gr, tm, tn); break;
    case FEW_LONG: hipLaunchKernelGGL((k_kept_wgrad<DT, FMT, 64, 3, 4>), grid, dim3(1024), 0, st, a, gr, tm, tn); break;
    case SPLIT: hipLaunchKernelGGL((k_kept_wgrad<DT, FMT, 128, 2, 4>), grid, dim3(1024), 0, st, a, gr, tm, tn); break;
    case MID: hipLaunchKernelGGL((k_kept_wgrad<DT, FMT, 128, 2, 1>), grid, dim3(256), 0, st, a, gr, tm, tn); break;
    case LARGE:
      if (a.d_fmt != BSM_F32) hipLaunchKernelGGL((k_kept_wgrad_large<DT, FMT, DT, dense::ASK>), grid, dim3(256), 0, st, a, gr, tm, tn);
      else if (a.accum) hipLaunchKernelGGL((k_kept_wgrad_large<DT, FMT, BSM_F32, dense::ALWAYS>), grid, dim3(256), 0, st, a, gr, tm, tn);
      else hipLaunchKernelGGL((k_kept_wgrad_large<DT, FMT, BSM_F32, dense::NEVER>), grid, dim3(256), 0, st, a, gr, tm, tn);
      break;
  }
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
