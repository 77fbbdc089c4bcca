// k_gemm_grouped.hip - fp16/bf16 products with a weight per group of rows, and their weight gradient.
//
//   grouped:  D[r, n] = f((D[r, n] +) sum_k A[r, k] B_g(n, k))      r in group g
//   wgrad:    D_g[m, n] = (D_g[m, n] +) sum_{r in group g} A[r, m] B[r, n]
//
// A tile works on one group's product: the operands' bases move to the group's first row and its
// weight, M (grouped) or K (wgrad) is the group's row count. Rows past a group's end are other groups'
// rows: they are clamped away on the load (grouped) or zeroed (wgrad, the partial last K tile) and
// never stored. Two tiles: the dense GEMM's 256 x 256 (gemm_dense_tile.hpp) and 32 / 64 / 128 x 128
// (gemm_mid_tile.hpp).
#include <algorithm>
#include "gemm_dense_tile.hpp"
#include "gemm_mid_tile.hpp"
#include "skinny.hpp"
#include "store16.hpp"
#include "grouped.hpp"

namespace bsm {
namespace {

using namespace dense;

template <int DT>
__device__ __forceinline__ void store_out(const GemmArgs& a, void* D, int64_t M, int64_t row0, int64_t col0, int lane,
                                          const f32x4 (&acc)[8][8], uint8_t* region) {
  if (a.d_fmt == BSM_F32) {
    if (a.accum) store_tile16((float*)D, a.ldd, M, a.N, row0, col0, lane, 1.0f, acc, region, true, a.ew_op, a.ew_scale, a.ew_bias);
    else store_tile16((float*)D, a.ldd, M, a.N, row0, col0, lane, 1.0f, acc, region, false, a.ew_op, a.ew_scale, a.ew_bias);
  } else {
    if (a.accum) gemm::store_tile16_bits<DT>((uint16_t*)D, a.ldd, M, a.N, row0, col0, lane, acc, region, true, a.ew_op, a.ew_scale, a.ew_bias);
    else gemm::store_tile16_bits<DT>((uint16_t*)D, a.ldd, M, a.N, row0, col0, lane, acc, region, false, a.ew_op, a.ew_scale, a.ew_bias);
  }
}

__device__ __forceinline__ void* row_ptr(const GemmArgs& a, int64_t elements) {
  return (uint8_t*)a.D + elements * (a.d_fmt == BSM_F32 ? 4 : 2);
}

// The product of one group of rows out of the call's: operands and output moved to it.
__device__ __forceinline__ GemmArgs group_product(const GemmArgs& a, const GroupArgs& gr, int g, int row0, int rows) {
  GemmArgs t = a;
  t.M = rows;
  t.A = (const uint16_t*)a.A + (int64_t)row0 * a.lda;
  t.B = (const uint16_t*)a.B + (int64_t)g * gr.stride_b;
  t.D = (float*)row_ptr(a, (int64_t)row0 * a.ldd);
  return t;
}

// Tiles of 256 x 256 for a group's whole 256 rows (kFull and more of the last ones count as whole), then, for the
// rows behind them, tiles of 128 (64, 32) x 128 in the same launch: they fill the last round.
constexpr int kFull = 193;
__device__ __forceinline__ int large_tiles(int rows) { return rows / 256 + (rows % 256 >= kFull ? 1 : 0); }
__device__ __forceinline__ int rest_tiles(int rows) { const int r = rows % 256; return r >= kFull ? 0 : (r + 127) / 128; }

template <int DT, bool BKM>
__global__ __launch_bounds__(256, 1) void k_grouped(GemmArgs a, GroupArgs gr, int large_n, int rest_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * STAGE_BYTES];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  grouped::Spot s;
  int used;
  if (grouped::find_tile_of<4>(gr, blockIdx.x, large_n, lane, large_tiles, s, used)) {
    const GemmArgs t = group_product(a, gr, s.g, s.row0, s.rows);
    f32x4 acc[8][8];
    tile_product<DT, true, BKM>(t, s.tm, s.tn, lds, lane, w, acc);
    store_out<DT>(t, t.D, s.rows, (int64_t)s.tm * BM + 128 * (w >> 1), (int64_t)s.tn * BN + 128 * (w & 1), lane, acc,
                  lds + 32768 * w);
    return;
  }
  const int pid = (int)blockIdx.x - used;
  if (pid < 0 || !grouped::find_tile_of<8>(gr, pid, rest_n, lane, rest_tiles, s, used)) return;
  const GemmArgs t = group_product(a, gr, s.g, s.row0, s.rows);
  const int64_t m0 = (int64_t)(s.rows / 256) * 256 + 128 * s.tm, n0 = mid::BN * (int64_t)s.tn;
  const int left = s.rows - (int)m0;
  constexpr int LDS = 2 * STAGE_BYTES;
  if (left <= 32) mid::tile<DT, 32, true, BKM, 64, mid::NoMore, LDS>(t, m0, n0, lds, lane, w);
  else if (left <= 64) mid::tile<DT, 64, true, BKM, 64, mid::NoMore, LDS>(t, m0, n0, lds, lane, w);
  else mid::tile<DT, 128, true, BKM, 64, mid::NoMore, LDS>(t, m0, n0, lds, lane, w);
}

// Workgroup p runs on XCD p % 8. Every XCD gets a contiguous eighth of each group's tiles (groups in
// turn), so that the groups' row counts, which are the tiles' lengths here, do not unbalance the XCDs,
// while the tiles that share a group's panels still meet in one L2.
struct WgradSpot { int g, tm, tn; };
__device__ __forceinline__ bool wgrad_tile(int pid, int n, int tiles_m, int tiles_n, WgradSpot& s) {
  const int per = tiles_m * tiles_n, share = (per + 7) >> 3;
  const int x = pid & 7, q = pid >> 3;
  s.g = q / share;
  const int in = x * share + (q - s.g * share);
  if (in >= per) return false;
  grouped::band_tile<4>(in, tiles_m, tiles_n, s.tm, s.tn);
  return true;
}

// One group's weight gradient out of the call's: K is its row count.
__device__ __forceinline__ GemmArgs wgrad_product(const GemmArgs& a, const GroupArgs& gr, int g) {
  int lo, hi;
  grouped::group_range(gr, g, lo, hi);
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi);
  GemmArgs t = a;
  t.K = hi - lo;
  t.A = (const uint16_t*)a.A + (int64_t)lo * a.lda;
  t.B = (const uint16_t*)a.B + (int64_t)lo * a.ldb;
  t.D = (float*)row_ptr(a, (int64_t)g * gr.stride_d);
  return t;
}

// PER_CU workgroups of Q times four waves share a CU; Q > 1: the waves' fours share a tile's rows.
template <int DT, int BM, int BK, int PER_CU, int Q = 1>
__global__ __launch_bounds__(256 * Q, PER_CU * Q) void k_grouped_wgrad(GemmArgs a, GroupArgs gr, int tiles_m, int tiles_n) {
  constexpr int LDS = 160 * 1024 / PER_CU / Q;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Q * LDS];
  const int lane = threadIdx.x & 63, wq = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wq & 3, q = wq >> 2;
  WgradSpot s;
  if (!wgrad_tile(blockIdx.x, gr.n, tiles_m, tiles_n, s)) return;
  mid::tile<DT, BM, false, false, BK, mid::NoMore, LDS, Q>(wgrad_product(a, gr, s.g), BM * (int64_t)s.tm,
                                                           mid::BN * (int64_t)s.tn, lds + q * LDS, lane, w,
                                                           mid::NoMore(), q);
}

// Tiles of 128 rows, a group's last one of as few as hold its rows. Bands of eight tile rows: an XCD's 64
// tiles at work then read 16 panels of A and B, not 20 as in bands of four (8192 rows over 8 groups,
// N 4096, K 8192: 545 against 567 us).
template <int DT, bool BKM>
__global__ __launch_bounds__(256, 2) void k_grouped_mid(GemmArgs a, GroupArgs gr, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[mid::LDS_BYTES];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  grouped::Spot s;
  if (!grouped::find_tile<128, 8>(gr, blockIdx.x, tiles_n, lane, s)) return;
  const GemmArgs t = group_product(a, gr, s.g, s.row0, s.rows);
  const int64_t m0 = 128 * (int64_t)s.tm, n0 = mid::BN * (int64_t)s.tn;
  const int left = s.rows - 128 * s.tm;
  if (left <= 32) mid::tile<DT, 32, true, BKM>(t, m0, n0, lds, lane, w);
  else if (left <= 64) mid::tile<DT, 64, true, BKM>(t, m0, n0, lds, lane, w);
  else mid::tile<DT, 128, true, BKM>(t, m0, n0, lds, lane, w);
}

// Fewer tiles than CUs: tiles of 64 (32) rows, and eight waves a tile, each four every other K tile.
template <int DT, bool BKM>
__global__ __launch_bounds__(512) void k_grouped_split(GemmArgs a, GroupArgs gr, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * mid::LDS_BYTES];
  const int lane = threadIdx.x & 63, w8 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = w8 & 3, q = w8 >> 2;
  grouped::Spot s;
  if (!grouped::find_tile<64, 8>(gr, blockIdx.x, tiles_n, lane, s)) return;
  const GemmArgs t = group_product(a, gr, s.g, s.row0, s.rows);
  const int64_t m0 = 64 * (int64_t)s.tm, n0 = mid::BN * (int64_t)s.tn;
  uint8_t* part = lds + q * mid::LDS_BYTES;
  if (s.rows - 64 * s.tm <= 32)
    mid::tile<DT, 32, true, BKM, 64, mid::NoMore, mid::LDS_BYTES, 2>(t, m0, n0, part, lane, w, mid::NoMore(), q);
  else
    mid::tile<DT, 64, true, BKM, 64, mid::NoMore, mid::LDS_BYTES, 2>(t, m0, n0, part, lane, w, mid::NoMore(), q);
}

// Few tiles: 16 MT rows x 16 columns a workgroup, its eight waves splitting K (skinny.hpp).
template <int DT, int MT>
__global__ __launch_bounds__(skinny::THREADS, MT == 1 ? 4 : 2) void k_grouped_skinny(GemmArgs a, GroupArgs gr, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[skinny::lds_bytes<MT>()];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  grouped::Spot s;
  if (!grouped::find_tile<16 * MT, 4>(gr, blockIdx.x, tiles_n, lane, s)) return;
  const GemmArgs t = group_product(a, gr, s.g, s.row0, s.rows);
  const int64_t m0 = 16 * MT * (int64_t)s.tm, n0 = skinny::BN * (int64_t)s.tn;
  f32x4 acc[MT];
  skinny::product<DT, MT>(t, m0, n0, lane, w, lds + w * (1 + MT) * 2048, acc, []() {});
  skinny::join<MT>(lds, lane, w, acc);
  if (w < MT) skinny::store4<DT>(t, m0 + 16 * w + (lane & 15), n0 + 4 * (lane >> 4), acc[0]);
}

// The kernels of a call, and the rules that choose among them.
enum GroupedTile { SKINNY_16, SKINNY_32, SKINNY_64, SPLIT, MID, LARGE };
constexpr const char* kGroupedNames[] = {"k_grouped_skinny<1>", "k_grouped_skinny<2>", "k_grouped_skinny<4>",
                                         "k_grouped_split", "k_grouped_mid", "k_grouped"};

GroupedTile grouped_tile(const GemmArgs& a, const GroupArgs& gr) {
  // Sixteen columns a workgroup where 128-column tiles would leave half the CUs without one: 16 rows of
  // one group, N = K = 4096 (32 such tiles) 21.8 -> 11.0 us, 64 rows 29.9 -> 15.2 us, 8 rows over 8 groups,
  // N 1024, K 2048 (64) 12.4 -> 9.3 us; even at 128 of them (32 rows over 8 groups, N = K = 2048: 18.0
  // and 18.2 us) and behind for more rows a group (500 rows, N = K = 2048: 21.8 and 27.1 us).
  const int64_t used = gr.n < gr.rows ? gr.n : gr.rows, each = (gr.rows + used - 1) / used;
  if (a.b_kmajor && each <= 64 && used * ((a.N + mid::BN - 1) / mid::BN) < 128)
    return each <= 16 ? SKINNY_16 : each <= 32 ? SKINNY_32 : SKINNY_64;
  // 256 x 256 tiles (and small ones for the rest of a group) where groups are long and the large tiles,
  // 0.45 a group fewer than the rows would fill, leave little of their last round over the 256 CUs empty.
  // Even groups, small tiles alone against both: 16381 rows over 16 groups (N 4096, K 8192) 1124 and 987 us, 8190 over
  // 8 (N 2048, K 8192) 290 and 227 us; groups of a router's split 1158 and 1163, 360 and 307 us. Short groups
  // (16384 rows over 64, N 4096, K 2048, uneven) 392 and 454 us; one and a half rounds (6000 rows, N = K =
  // 4096) 185 and 215 us; half a round (8190 over 8, N 1024, K 4096) 66 and 103 us; a twentieth (1000 rows, N = K =
  // 1024) 9.3 and 35 us, (994 rows, N 537, K 7577) 47 and 189 us: one round at least has to be begun.
  auto row_tiles = [&](double bm) { return gr.n == 1 ? (double)((gr.rows + (int64_t)bm - 1) / (int64_t)bm) : gr.rows / bm + 0.5 * gr.n; };
  const double whole = gr.n == 1 ? (double)(gr.rows / BM) : gr.rows / (double)BM - 0.45 * gr.n;
  const double rounds = whole * ((a.N + BN - 1) / BN) / 256, last = rounds - (int64_t)rounds;
  const double begun = (double)std::max<int64_t>((int64_t)rounds + (last > 0.05), 1);
  if (gr.rows / gr.n >= 768 && rounds >= 0.85 * begun) return LARGE;
  // Fewer 128-row tiles than CUs: half as many rows and eight waves a tile (1000 rows over 4 groups,
  // N = K = 1024, 78 tiles: 13.8 -> 9.7 us; 582 rows, N 1665, K 7227, 70: 69 -> 41 us; 1000 over 4, N 2048, K
  // 1024, 157: 14.3 -> 10.7 us; at 258 and 314 tiles it is behind, 46.7 to 44.2 and 18.8 to 15.9 us).
  return row_tiles(128) * ((a.N + mid::BN - 1) / mid::BN) < 192 ? SPLIT : MID;
}

template <int DT>
hipError_t launch_grouped_dt(const GemmArgs& a, const GroupArgs& gr, hipStream_t st) {
  const GroupedTile tile = grouped_tile(a, gr);
  const int bm = tile == SKINNY_16 ? 16 : tile == SKINNY_32 ? 32 : tile <= SPLIT ? 64 : tile == MID ? 128 : BM;
  const int bn = tile <= SKINNY_64 ? skinny::BN : tile == LARGE ? BN : mid::BN;
  const int64_t tn = (a.N + bn - 1) / bn, n = (grouped::most_row_tiles(gr.rows, gr.n, bm) * tn + 7) / 8 * 8;
  if (n > 0x7FFFFFFF) return hipErrorInvalidValue;
  const dim3 grid((uint32_t)n);
  switch (tile) {
    case SKINNY_16: hipLaunchKernelGGL((k_grouped_skinny<DT, 1>), grid, dim3(skinny::THREADS), 0, st, a, gr, (int)tn); break;
    case SKINNY_32: hipLaunchKernelGGL((k_grouped_skinny<DT, 2>), grid, dim3(skinny::THREADS), 0, st, a, gr, (int)tn); break;
    case SKINNY_64: hipLaunchKernelGGL((k_grouped_skinny<DT, 4>), grid, dim3(skinny::THREADS), 0, st, a, gr, (int)tn); break;
    case SPLIT:
      if (a.b_kmajor) hipLaunchKernelGGL((k_grouped_split<DT, true>), grid, dim3(512), 0, st, a, gr, (int)tn);
      else hipLaunchKernelGGL((k_grouped_split<DT, false>), grid, dim3(512), 0, st, a, gr, (int)tn);
      break;
    case MID:
      if (a.b_kmajor) hipLaunchKernelGGL((k_grouped_mid<DT, true>), grid, dim3(256), 0, st, a, gr, (int)tn);
      else hipLaunchKernelGGL((k_grouped_mid<DT, false>), grid, dim3(256), 0, st, a, gr, (int)tn);
      break;
    case LARGE: {
      const int64_t rest_n = (a.N + mid::BN - 1) / mid::BN, rest = 2 * (gr.n < gr.rows ? gr.n : gr.rows) * rest_n;
      if (n + rest > 0x7FFFFFF0) return hipErrorInvalidValue;
      const dim3 both((uint32_t)(n + (rest + 7) / 8 * 8));
      if (a.b_kmajor) hipLaunchKernelGGL((k_grouped<DT, true>), both, dim3(256), 0, st, a, gr, (int)tn, (int)rest_n);
      else hipLaunchKernelGGL((k_grouped<DT, false>), both, dim3(256), 0, st, a, gr, (int)tn, (int)rest_n);
      break;
    }
  }
  return hipGetLastError();
}

enum WgradTile { TALL, WGRAD_SPLIT, FEW_ROWS, SQUARE };
constexpr const char* kWgradNames[] = {"k_grouped_wgrad<256, 32, 2, 1>", "k_grouped_wgrad<128, 64, 1, 2>",
                                       "k_grouped_wgrad<128, 32, 4, 1>", "k_grouped_wgrad<128, 64, 2, 1>"};

WgradTile wgrad_tile_kind(const GemmArgs& a, const GroupArgs& gr) {
  const int64_t tn = (a.N + mid::BN - 1) / mid::BN, each = gr.rows / gr.n;
  // Tiles of 256 rows where groups have rows enough for a long loop and the tiles fill the CUs: 16381
  // rows over 8 groups (M 4096, N 2048) 306 us against 343 us on 128; 1021 over 32 (M 1000, N 520) 21.1
  // against 19.8 us. (The dense GEMM's 256 x 256 tile: 350 and 40 us.)
  if (each >= 192 && (a.M + 255) / 256 * tn * gr.n >= 512) return TALL;
  // Few tiles of long groups: eight waves a tile, each four every other 64 rows (16000 rows over 2 groups, M =
  // N = 1024 80 -> 68 us; 4000 in one, 43 -> 38 us; at 250 rows a group it is behind).
  if (each >= 1000 && (a.M + 127) / 128 * tn * gr.n < 192) return WGRAD_SPLIT;
  // Few rows a group: the loop is a step or two and loads, sums and stores of different tiles overlap, so
  // four workgroups share a CU (K tiles of 32, 40 KiB of LDS each): 1021 rows over 32 groups (M 1000,
  // N 520) 15.0 us against 18.5 us on two.
  return each < 64 ? FEW_ROWS : SQUARE;
}

}  // namespace

hipError_t launch_gemm_grouped(const GemmArgs& a, const GroupArgs& gr, hipStream_t st) {
  return a.dtype == BSM_BF16 ? launch_grouped_dt<BSM_BF16>(a, gr, st) : launch_grouped_dt<BSM_F16>(a, gr, st);
}

template <int DT>
static hipError_t launch_wgrad_dt(const GemmArgs& a, const GroupArgs& gr, hipStream_t st) {
  const WgradTile tile = wgrad_tile_kind(a, gr);
  const int64_t bm = tile == TALL ? 256 : 128, tn = (a.N + mid::BN - 1) / mid::BN, tm = (a.M + bm - 1) / bm;
  const int64_t share = (tm * tn + 7) / 8;
  if (share > 0x7FFFFFFF / 8 / gr.n) return hipErrorInvalidValue;
  const dim3 grid((uint32_t)(share * 8 * gr.n));
  switch (tile) {
    case TALL: hipLaunchKernelGGL((k_grouped_wgrad<DT, 256, 32, 2>), grid, dim3(256), 0, st, a, gr, (int)tm, (int)tn); break;
    case WGRAD_SPLIT: hipLaunchKernelGGL((k_grouped_wgrad<DT, 128, 64, 1, 2>), grid, dim3(512), 0, st, a, gr, (int)tm, (int)tn); break;
    case FEW_ROWS: hipLaunchKernelGGL((k_grouped_wgrad<DT, 128, 32, 4>), grid, dim3(256), 0, st, a, gr, (int)tm, (int)tn); break;
    case SQUARE: hipLaunchKernelGGL((k_grouped_wgrad<DT, 128, 64, 2>), grid, dim3(256), 0, st, a, gr, (int)tm, (int)tn); break;
  }
  return hipGetLastError();
}

hipError_t launch_gemm_grouped_wgrad(const GemmArgs& a, const GroupArgs& gr, hipStream_t st) {
  return a.dtype == BSM_BF16 ? launch_wgrad_dt<BSM_BF16>(a, gr, st) : launch_wgrad_dt<BSM_F16>(a, gr, st);
}

const char* route_gemm_grouped(const GemmArgs& a, const GroupArgs& gr) { return kGroupedNames[grouped_tile(a, gr)]; }
const char* route_gemm_grouped_wgrad(const GemmArgs& a, const GroupArgs& gr) { return kWgradNames[wgrad_tile_kind(a, gr)]; }

}  // namespace bsm
