// store_large.hpp - the 256 x 256 tile's store in a chosen format, for kernels whose K loop must not see it.
//
// As dense::store_tile16 and gemm::store_tile16_bits, but every accumulator is copied to an ordinary register before it goes
// to LDS (an asm that claims to change the copy). Where the stores read the 256 accumulator registers themselves the compiler
// gave some accumulators other registers behind the K loop than in it and moved up to 480 of them in every turn of the loop:
// dX and dW of 8190 x 32001 x 4096 took 1867 and 2179 us, with the copies 1526 and 1824 us.
#pragma once
#include "gemm_dense_tile.hpp"
#include "store16.hpp"

namespace bsm {
namespace dense {

// Whether D is added to: known when compiled, or by the call's own flag. (A float32 store that asks needs registers for both
// ways and spills 60: 16381 rows over 8 groups, 4096 x 2048 330 us against 267.)
enum Add { NEVER, ALWAYS, ASK };

// D = round(acc (+ D)) for the wave's 128 x 128 sub-tile at (row0, col0), OUT BSM_F32, BSM_BF16 or BSM_F16, through
// 32 KiB of LDS in two halves of 64 rows (region row r keeps its 16-byte chunk c at c ^ (r & 15)).
template <int OUT, Add ADD>
__device__ __forceinline__ void store_large(const GemmArgs& a, int64_t row0, int64_t col0, int lane, const f32x4 (&acc)[8][8],
                                            uint8_t* region) {
  const bool add = ADD == ASK ? a.accum : ADD == ALWAYS;
#pragma unroll
  for (int half = 0; half < 2; half++) {
#pragma unroll
    for (int m4 = 0; m4 < 4; m4++) {
      const int r = 16 * m4 + (lane & 15);
#pragma unroll
      for (int nt = 0; nt < 8; nt++) {
        const int c = 4 * nt + (lane >> 4);
        f32x4 v = acc[4 * half + m4][nt];
        asm volatile("" : "+v"(v));
        lds_write_b128(region + 512 * r + 16 * (c ^ (r & 15)),
                       make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
      }
    }
    const int64_t rowh = row0 + 64 * half;
    if constexpr (OUT != BSM_F32) {
      gemm::store_half_bits16<OUT>((uint16_t*)a.D, a.ldd, a.M, a.N, rowh, col0, lane, region, add, 0, 0.0f, 0.0f);
    } else {
      const int c = lane & 31;
      const int64_t col = col0 + 4 * c;
      if (rowh + 64 <= a.M && col0 + 128 <= a.N) {   // wave-uniform
        gemm::store_half_whole<false>(a.D, a.ldd, rowh, col, lane, c, region, add, 0.0f, 0.0f);
      } else {
        for (int j = 0; j < 32; j++) {
          const int r = 2 * j + (lane >> 5);
          const uint4 x = lds_read_b128(region + 512 * r + 16 * (c ^ (r & 15)));
          const float xv[4] = {__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w)};
          if (rowh + r < a.M) {
            gemm::global_f32* p = (gemm::global_f32*)(a.D + (rowh + r) * a.ldd + col);
#pragma unroll
            for (int e = 0; e < 4; e++)
              if (col + e < a.N) p[e] = add ? xv[e] + p[e] : xv[e];
          }
        }
      }
    }
  }
}

}  // namespace dense
}  // namespace bsm
