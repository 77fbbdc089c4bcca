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
  if (left <= 32) midmx::tile<CA, CB, BF, 32>(a, a, m0, n0, lds, lane, w);
  else if (left <= 64) midmx::tile<CA, CB, BF, 64>(a, a, m0, n0, lds, lane, w);
  else midmx::tile<CA, CB, BF, 128>(a, a, m0, n0, lds, lane, w);
}

// Tiles of 32 rows alone, three workgroups a CU.
template <int CA, int CB, bool BF>
static __global__ __launch_bounds__(256, 3) void k_grouped_mx_rows32(GemmArgs a, GroupArgs gr, int tiles_n) {
  constexpr int LDS = 53 * 1024;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[LDS];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  grouped::Spot s;
  if (!grouped::find_tile<32, 4>(gr, blockIdx.x, tiles_n, lane, s)) return;
  grouped::group_product<mxany::fmt_bits(CA), mxany::fmt_bits(CB)>(a, gr, s, a.d_fmt == BSM_F32 ? 4 : 2);
  midmx::tile<CA, CB, BF, 32, 1, LDS>(a, a, 32 * (int64_t)s.tm, midmx::BN * (int64_t)s.tn, lds, lane, w);
}

// Fewer tiles than CUs: tiles of 64 (32) rows, and eight waves a tile, four for each half of K.
template <int CA, int CB, bool BF>
static __global__ __launch_bounds__(512) void k_grouped_mx_split(GemmArgs a, GroupArgs gr, int tiles_n) {
  constexpr int LDS = 72 * 1024;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * LDS];
  __shared__ GemmArgs late;
  const int lane = threadIdx.x & 63, w8 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = w8 & 3, q = w8 >> 2;
  grouped::Spot s;
  if (!grouped::find_tile<64, 4>(gr, blockIdx.x, tiles_n, lane, s)) return;
  grouped::group_product<mxany::fmt_bits(CA), mxany::fmt_bits(CB)>(a, gr, s, a.d_fmt == BSM_F32 ? 4 : 2);
  const int64_t m0 = 64 * (int64_t)s.tm, n0 = midmx::BN * (int64_t)s.tn;
  uint8_t* part = lds + q * LDS;
  if (threadIdx.x == 0) late = a;
  if (s.rows - 64 * s.tm <= 32) midmx::tile<CA, CB, BF, 32, 2, LDS>(a, late, m0, n0, part, lane, w, q);
  else midmx::tile<CA, CB, BF, 64, 2, LDS>(a, late, m0, n0, part, lane, w, q);
}

enum MidTile { ROWS32, SPLIT, MID };
static MidTile mid_tile(const GemmArgs& a, const GroupArgs& gr) {
  const int64_t tn = (a.N + midmx::BN - 1) / midmx::BN, used = gr.n < gr.rows ? gr.n : gr.rows;
  // (300 rows over 4 groups, N 1024, K 4096: E4M3 x E2M1 35.1 -> 22.1 us, E2M1 pairs 21.8 -> 15.5 us; 64 over 8,
  // N 2048, K 4096: 19.5 -> 17.8 us)
  if ((gr.rows / 128 + (used + 1) / 2) * tn < 192) return SPLIT;
  // Exact E4M3 x E2M1 of up to 16 rows a group: its conversions leave room for a third workgroup (64 rows over 32
  // groups, N = K = 4096 62 -> 56 us, 512 rows 83.8 -> 78.6 us; E4M3 pairs 101 -> 104 us, the others the same).
  const bool exact_mixed = a.dtype == BSM_E4M3 && a.dtype_b == BSM_E2M1 && !a.mx_window;
  return exact_mixed && gr.rows / gr.n <= 16 ? ROWS32 : MID;
}

const char* route_gemm_grouped_mx_mid(const GemmArgs& a, const GroupArgs& gr) {
  constexpr const char* names[] = {"k_grouped_mx_rows32", "k_grouped_mx_split", "k_grouped_mx_mid"};
  return names[mid_tile(a, gr)];
}

template <int CA, int CB, bool BF>
static hipError_t launch_mid(const GemmArgs& a, const GroupArgs& gr, hipStream_t st) {
  const MidTile tile = mid_tile(a, gr);
  const int64_t tn = (a.N + midmx::BN - 1) / midmx::BN, bm = tile == ROWS32 ? 32 : tile == SPLIT ? 64 : 128;
  const int64_t n = (grouped::most_row_tiles(gr.rows, gr.n, bm) * tn + 7) / 8 * 8;
  if (n > 0x7FFFFFFF) return hipErrorInvalidValue;
  const dim3 grid((uint32_t)n);
  if (tile == SPLIT) hipLaunchKernelGGL((k_grouped_mx_split<CA, CB, BF>), grid, dim3(512), 0, st, a, gr, (int)tn);
  else if (tile == MID) hipLaunchKernelGGL((k_grouped_mx_mid<CA, CB, BF>), grid, dim3(256), 0, st, a, gr, (int)tn);
  else if constexpr (BF && CB == 4) hipLaunchKernelGGL((k_grouped_mx_rows32<CA, CB, BF>), grid, dim3(256), 0, st, a, gr, (int)tn);
  return hipGetLastError();
}

hipError_t launch_gemm_grouped_mx_mid(const GemmArgs& a, const GroupArgs& gr, hipStream_t st) {
  if (a.dtype == BSM_E2M1) return launch_mid<4, 4, false>(a, gr, st);
  if (a.dtype_b == BSM_E2M1) return a.mx_window ? launch_mid<0, 4, false>(a, gr, st) : launch_mid<0, 4, true>(a, gr, st);
  return a.mx_window ? launch_mid<0, 0, false>(a, gr, st) : launch_mid<0, 0, true>(a, gr, st);
}

}  // namespace bsm
