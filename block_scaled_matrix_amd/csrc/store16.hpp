// store16.hpp - the GEMM tiles' epilogue for 16-bit outputs: the accumulators pass through LDS as
// in gemm_common.hpp's float32 epilogue and leave as whole 128-byte lines; and which product's
// which tile a workgroup of the block-scaled kernels computes.
#pragma once
#include "gemm_common.hpp"
#include "../../include/bsm.h"

namespace bsm {
namespace gemm {

// One value in a 16-bit output format (BSM_BF16 or BSM_F16), rounded to nearest even, and back.
template <int OUT>
__device__ __forceinline__ uint16_t to_bits16(float v) { return OUT == 4 ? f32_to_bf16_bits(v) : f32_to_f16_bits(v); }
template <int OUT>
__device__ __forceinline__ float from_bits16(uint16_t h) { return OUT == 4 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h); }

// The 64 staged rows of one half of a 128 x 128 sub-tile (region row r, chunk c at c ^ (r & 15),
// as store_tile_lines keeps them) as 16-bit outputs D = round(f(x (+ D))): lane l moves the
// eight columns 8(l%16) of rows 4j + l/16 as one 16-byte piece, so that one instruction writes
// four 256-byte row pieces (whole 128-byte lines). x is the float32 sum; the output is the only
// rounding to fewer bits. Rows past M and columns past N are not touched.
template <int OUT>
__device__ __forceinline__ void store_half_bits16(uint16_t* __restrict__ D, int64_t ldd, int64_t M, int64_t N,
                                                  int64_t rowh, int64_t col0, int lane, const uint8_t* region, bool add,
                                                  int ew_op, float es, float eb) {
  const bool whole = rowh + 64 <= M && col0 + 128 <= N;  // wave-uniform
  const int c = 2 * (lane & 15);
  const int64_t col = col0 + 4 * c;
#pragma unroll 4
  for (int j = 0; j < 16; j++) {
    const int r = 4 * j + (lane >> 4);
    const uint4 x0 = lds_read_b128(region + 512 * r + 16 * (c ^ (r & 15)));
    const uint4 x1 = lds_read_b128(region + 512 * r + 16 * ((c + 1) ^ (r & 15)));
    float v[8] = {__uint_as_float(x0.x), __uint_as_float(x0.y), __uint_as_float(x0.z), __uint_as_float(x0.w),
                  __uint_as_float(x1.x), __uint_as_float(x1.y), __uint_as_float(x1.z), __uint_as_float(x1.w)};
    const int64_t row = rowh + r;
    if (whole) {
      global_u32x4* p = (global_u32x4*)(D + row * ldd + col);
      if (add) {
        const u32x4 y = *p;
#pragma unroll
        for (int e = 0; e < 8; e++) v[e] += from_bits16<OUT>((uint16_t)(y[e >> 1] >> (16 * (e & 1))));
      }
      u32x4 o;
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const float lo = ew_op ? silu_affine(v[2 * e], es, eb) : v[2 * e];
        const float hi = ew_op ? silu_affine(v[2 * e + 1], es, eb) : v[2 * e + 1];
        o[e] = (uint32_t)to_bits16<OUT>(lo) | ((uint32_t)to_bits16<OUT>(hi) << 16);
      }
      *p = o;
    } else if (row < M) {
      uint16_t* p = D + row * ldd + col;
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (col + e < N) {
          float x = add ? v[e] + from_bits16<OUT>(p[e]) : v[e];
          if (ew_op) x = silu_affine(x, es, eb);
          p[e] = to_bits16<OUT>(x);
        }
    }
  }
}

// Whether every row piece of a 16-bit tile may be moved as 16-byte pieces follows from the
// host's rules (D 16-byte aligned, ldd a multiple of 8). This is store_tile_lines for them.
template <int OUT>
__device__ __forceinline__ void store_tile_lines16(uint16_t* __restrict__ D, int64_t ldd, int64_t M, int64_t N,
                                                   int64_t row0, int64_t col0, int lane, const f32x16 (&acc)[4][4],
                                                   uint8_t* region, bool add, int ew_op, float es, float eb) {
#pragma unroll
  for (int half = 0; half < 2; half++) {
#pragma unroll
    for (int m2 = 0; m2 < 2; m2++) {
      const int r = 32 * m2 + (lane & 31);
#pragma unroll
      for (int nt = 0; nt < 4; nt++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const int c = 8 * nt + 2 * q + (lane >> 5);
          const f32x16& v = acc[2 * half + m2][nt];
          lds_write_b128(region + 512 * r + 16 * (c ^ (r & 15)),
                         make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                                    __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3])));
        }
    }
    store_half_bits16<OUT>(D, ldd, M, N, row0 + 64 * half, col0, lane, region, add, ew_op, es, eb);
  }
}

// The same for a 128 x 128 sub-tile of 8 x 8 blocks of 16x16 accumulators (register e of block (mt, nt)
// is output row 16mt + l%16, column 16nt + 4(l/16) + e).
template <int OUT>
__device__ __forceinline__ void store_tile16_bits(uint16_t* __restrict__ D, int64_t ldd, int64_t M, int64_t N,
                                                  int64_t row0, int64_t col0, int lane, const f32x4 (&acc)[8][8],
                                                  uint8_t* region, bool add, int ew_op, float es, float eb) {
#pragma unroll
  for (int half = 0; half < 2; half++) {
#pragma unroll
    for (int m4 = 0; m4 < 4; m4++) {
      const int r = 16 * m4 + (lane & 15);
#pragma unroll
      for (int nt = 0; nt < 8; nt++) {
        const int c = 4 * nt + (lane >> 4);
        const f32x4& v = acc[4 * half + m4][nt];
        lds_write_b128(region + 512 * r + 16 * (c ^ (r & 15)),
                       make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                  __float_as_uint(v[3])));
      }
    }
    store_half_bits16<OUT>(D, ldd, M, N, row0 + 64 * half, col0, lane, region, add, ew_op, es, eb);
  }
}

// Which tile of which product a workgroup computes: the whole of one product (the calls on one
// matrix), or a tile of one group's (grouped.hpp). locate() makes `a` that product and gives its
// tile; false: the workgroup has none.
struct WholeProduct {
  int tiles_m, tiles_n;
  __device__ __forceinline__ bool locate(GemmArgs&, int, int& tm, int& tn) const {
    tile_coords(blockIdx.x, tiles_m, tiles_n, tm, tn);
    return true;
  }
};

// A tile's store in D's format: OUT is BSM_F32, BSM_BF16 or BSM_F16.
template <int OUT>
__device__ __forceinline__ void store_tile_as(const GemmArgs& a, int64_t row0, int64_t col0, int lane, float sgn,
                                              const f32x16 (&acc)[4][4], uint8_t* region, bool add) {
  if constexpr (OUT == BSM_F32)
    store_tile_lines(a.D, a.ldd, a.M, a.N, row0, col0, lane, sgn, acc, region, add, a.ew_op, a.ew_scale, a.ew_bias);
  else
    store_tile_lines16<OUT>((uint16_t*)a.D, a.ldd, a.M, a.N, row0, col0, lane, acc, region, add, a.ew_op, a.ew_scale,
                            a.ew_bias);
}

}  // namespace gemm
}  // namespace bsm
