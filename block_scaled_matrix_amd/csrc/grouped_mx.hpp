// grouped_mx.hpp - where a workgroup of the block-scaled kernels works when the rows are in groups.
#pragma once
#include "grouped.hpp"

namespace bsm {
namespace grouped {

// Makes `a` the product of group s.g's rows: operands, scales and output moved to the group's rows and
// weight. BA, BB: bits per element of A and B; db: bytes per element of D. A group's first row is any
// row, so its scale row starts 4-byte aligned and its element row 16-byte aligned, as the host's rules
// on the leading dimensions give them.
template <int BA, int BB>
__device__ __forceinline__ void group_product(GemmArgs& a, const GroupArgs& gr, const Spot& s, int db) {
  a.M = s.rows;
  a.A = (const uint8_t*)a.A + (int64_t)s.row0 * a.lda * BA / 8;
  a.SFA += (int64_t)s.row0 * a.ld_sfa;
  a.B = (const uint8_t*)a.B + (int64_t)s.g * gr.stride_b * BB / 8;
  a.SFB += (int64_t)s.g * gr.stride_sfb;
  a.D = (float*)((uint8_t*)a.D + (int64_t)s.row0 * a.ldd * db);
}

// Tile of one group's product for the 256 x 256 kernels (gemm::WholeProduct's counterpart).
template <int BA, int BB, int DB>
struct GroupProduct {
  GroupArgs gr;
  int tiles_n;
  __device__ __forceinline__ bool locate(GemmArgs& a, int lane, int& tm, int& tn) const {
    Spot s;
    if (!find_tile<256, 4>(gr, blockIdx.x, tiles_n, lane, s)) return false;
    group_product<BA, BB>(a, gr, s, DB);
    tm = s.tm;
    tn = s.tn;
    return true;
  }
};

}  // namespace grouped
}  // namespace bsm
