// lora.hpp - low-rank adapters chosen per row: what the shrink and the expand share.
//
//   D[t, n] = f((D[t, n] +) sum_k X[t, k] W[n, k] + sum_r U[t, r] LB_a[n, r]),
//   U[t, r] = scale_a * sum_k X[t, k] LA_a[r, k],      a = adapter[t] (outside 0 .. n - 1: none)
//
// U is kept in float32 in the caller's workspace, rows of Rp = R rounded up to 32 values, those past
// R zero; rows without an adapter are not written and never read.
//
// A 16-row block of the matrix instruction may hold rows of up to 16 adapters. The block is worked
// off adapter by adapter with the other rows' operand zeroed, so a row's sum only ever sees its own
// adapter's weights: requests in any order need no sorting, and long requests cost one pass.
#pragma once
#include <type_traits>
#include "bsm_device.hpp"
#include "bsm_internal.hpp"
#include "../../include/bsm.h"

namespace bsm {
namespace lora {

__host__ __device__ inline int64_t padded_rank(int64_t R) { return (R + 31) / 32 * 32; }

// The adapter of row t (lane-wise), -1 for none and for rows past the last.
__device__ __forceinline__ int adapter_of(const LoraArgs& lo, int64_t t, int64_t rows) {
  const int a = lo.n > 0 && t < rows ? lo.adapter[t] : -1;
  return a < lo.n ? a : -1;
}

// 8 consecutive elements (16 bytes) of a 16-bit row, those at or past `left` elements zero.
__device__ __forceinline__ uint4 load8(const uint16_t* p, int64_t left) {
  if (left <= 0) return make_uint4(0, 0, 0, 0);
  uint4 v = *(const uint4*)p;
  if (left < 8) {
    uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int d = 0; d < 4; d++) {
      const int64_t n = left - 2 * d;
      wd[d] &= n >= 2 ? 0xFFFFFFFFu : (n == 1 ? 0xFFFFu : 0u);
    }
    v = make_uint4(wd[0], wd[1], wd[2], wd[3]);
  }
  return v;
}

template <int DT>
__device__ __forceinline__ f32x4 mfma16(uint4 b, uint4 a, f32x4 c) {
  if constexpr (DT == BSM_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a), c, 0, 0, 0);
}

// One 32-value step of a row's U: what the lane (row l%16, r 8(l/16) .. +7) holds.
struct UPart { float v[8]; };

__device__ __forceinline__ UPart load_u(const float* U, int64_t Rp, int64_t t, int r0, int lane, bool mine) {
  UPart u;
  if (mine) {
    const float4* p = (const float4*)(U + t * Rp + r0 + 8 * (lane >> 4));
    const float4 x = p[0], y = p[1];
    u.v[0] = x.x; u.v[1] = x.y; u.v[2] = x.z; u.v[3] = x.w;
    u.v[4] = y.x; u.v[5] = y.y; u.v[6] = y.z; u.v[7] = y.w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; e++) u.v[e] = 0.f;
  }
  return u;
}

// A float32 as a sum of bf16 terms cut off from the top (8 significant bits each, so three hold all
// 24 and nothing rounds or overflows): the upper half of the word, then the rest. An infinity has no
// rest; a NaN's rest is NaN.
__device__ __forceinline__ uint32_t top_bits(float v) { return __float_as_uint(v) & 0xFFFF0000u; }
__device__ __forceinline__ float rest_of(float v) {
  const float t = __uint_as_float(top_bits(v));
  return v == t ? 0.f : v - t;
}
// The top terms of eight values as an operand of the bf16 matrix instruction; v becomes the rests.
__device__ __forceinline__ uint4 cut_top(float (&v)[8]) {
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; e++) {
    o[e] = (top_bits(v[2 * e]) >> 16) | top_bits(v[2 * e + 1]);
    v[2 * e] = rest_of(v[2 * e]);
    v[2 * e + 1] = rest_of(v[2 * e + 1]);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// One 32-value step of U as three bf16 operands, U = t[0] + t[1] + t[2] (to float32's last bit, values
// near its subnormals aside).
struct USplit { uint4 t[3]; };
__device__ __forceinline__ USplit split_u(UPart u) {
  USplit s;
#pragma unroll
  for (int q = 0; q < 3; q++) s.t[q] = cut_top(u.v);
  return s;
}

// d + U (16 rows x 32) LB^T (32 x 16 columns) with U at float32 precision on the bf16 matrix instruction:
// three products with bf16 weights, six with f16 ones (11 bits: two bf16 terms), the small terms
// first. U rounded to 16 bits instead would cost one, and an error of 2^-9 (2^-12) of the adapter's
// part; the float32 matrix instruction takes 8 for the same 32 values at an eighth of the rate.
template <int DT>
__device__ __forceinline__ f32x4 expand_step(const USplit& u, uint4 b, f32x4 d) {
  if constexpr (DT == BSM_BF16) {
#pragma unroll
    for (int q = 2; q >= 0; q--) d = mfma16<BSM_BF16>(b, u.t[q], d);
  } else {
    const uint32_t wd[4] = {b.x, b.y, b.z, b.w};
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] = f16_bits_to_f32((uint16_t)(wd[e >> 1] >> (16 * (e & 1))));
    const uint4 hi = cut_top(v), lo = cut_top(v);
#pragma unroll
    for (int q = 2; q >= 0; q--) d = mfma16<BSM_BF16>(lo, u.t[q], d);
#pragma unroll
    for (int q = 2; q >= 0; q--) d = mfma16<BSM_BF16>(hi, u.t[q], d);
  }
  return d;
}

// Infinities and NaN do not go through expand_step: a term that is zero (the rests of a U of few bits, the low
// term of a weight of few bits) times an infinity would be NaN where the product is infinite. The steps that hold one
// (none does in earnest) take those products apart: with o(v) = v where it is not finite, else 0, and c(v) = NaN, 0 or
// v's sign,
//   sum_r o(U) c(LB) + c(U) o(LB)
// has every such product's value (an infinity times an infinity in both, with one sign) and zeros for the finite ones,
// and expand_step gets finite operands, the others zero. Every step is looked at: zero times a value is NaN where
// it is not finite, summed in one instruction a value of U and one a pair of weights (8190 rows of rank 64, N 8192,
// K 4096: 595 us without it, 600 with it; integer tests of the exponents take twice the instructions and cost 1.3%).
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ float zeros_of(const UPart& u, float z) {
#pragma unroll
  for (int e = 0; e < 8; e++) z = __builtin_fmaf(u.v[e], 0.f, z);
  return z;
}
template <int DT>
__device__ __forceinline__ float zeros_of(uint4 b, float z) {
  const uint32_t wd[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int d = 0; d < 4; d++) {
    if constexpr (DT == BSM_BF16) z = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, wd[d]), bf16x2{}, z, false);
    else z = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, wd[d]), f16x2{}, z, false);
  }
  return z;
}
// o(v) and c(v) of eight values as bf16 operands; v's own become finite. (Masks in vector registers by shifts of a sign:
// comparisons' masks, eight at a time, made the compiler spill SGPRs.)
struct Apart { uint4 o, c; };
__device__ __forceinline__ Apart take_apart(float (&v)[8]) {
  uint32_t o[4] = {0, 0, 0, 0}, c[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; e++) {
    const uint32_t x = __float_as_uint(v[e]), a = x & 0x7FFFFFFFu, s = (x >> 16) & 0x8000u;
    const uint32_t odd = (uint32_t)((int32_t)(a + 0x00800000u) >> 31), nan = (uint32_t)((int32_t)(0x7F800000u - a) >> 31);
    const uint32_t some = (uint32_t)((int32_t)(0u - a) >> 31);   // not zero
    o[e >> 1] |= ((s | 0x7F80u | (nan & 0x40u)) & odd) << (16 * (e & 1));
    c[e >> 1] |= (((s | 0x3F80u) & some & ~nan) | (0x7FC0u & nan)) << (16 * (e & 1));
    v[e] = __uint_as_float(x & ~odd);
  }
  return {make_uint4(o[0], o[1], o[2], o[3]), make_uint4(c[0], c[1], c[2], c[3])};
}
template <int DT>
__device__ __forceinline__ Apart take_apart(uint4& b) {
  uint32_t wd[4] = {b.x, b.y, b.z, b.w};
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; e++) {
    const uint16_t h = (uint16_t)(wd[e >> 1] >> (16 * (e & 1)));
    v[e] = DT == BSM_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h);
  }
  const Apart p = take_apart(v);
  const uint32_t od[4] = {p.o.x, p.o.y, p.o.z, p.o.w};
#pragma unroll
  for (int d = 0; d < 4; d++) {   // (o's bit 14 is set where the value is not finite)
    const uint32_t full = (od[d] >> 14) & 0x10001u;
    wd[d] &= ~((full << 16) - full);
  }
  b = make_uint4(wd[0], wd[1], wd[2], wd[3]);
  return p;
}

// Smallest adapter above `after` among the rows whose adapters the lanes hold in id[] (lane l: row
// l%16 of each 16-row block), INT_MAX if there is none. Wave-uniform.
template <int MI>
__device__ __forceinline__ int next_adapter(const int (&id)[MI], int after) {
  int v = 0x7FFFFFFF;
#pragma unroll
  for (int m = 0; m < MI; m++) v = id[m] > after ? min(v, id[m]) : v;
#pragma unroll
  for (int d = 8; d; d >>= 1) v = min(v, __shfl_xor(v, d));
  return __builtin_amdgcn_readfirstlane(v);
}

// Adds the adapters' part U LB^T to a wave's MI x NI blocks of 16x16 accumulators (operands swapped:
// lane l holds row row0 + 16 m + l%16, columns col0 + 16 n + 4(l/16) .. +3), adapter by adapter in
// ascending order, 32 of the rank at a time: all of U's and LB's loads of a step go out together, and LB
// is read once for all the rows. A block whose 16 rows are all the adapter's accumulates in place; in
// a mixed one the product is a sum of its own, added where the row is the adapter's (another row's
// zeros times an infinity of this adapter are not zero).
template <int DT, int MI, int NI>
__device__ __forceinline__ void expand(const LoraArgs& lo, int64_t Rp, int64_t M, int64_t N, int64_t row0, int64_t col0,
                                       int lane, f32x4 (&acc)[MI][NI]) {
  const int i = lane & 15, G = lane >> 4, R = __builtin_amdgcn_readfirstlane(lo.R);
  int id[MI];
#pragma unroll
  for (int m = 0; m < MI; m++) id[m] = adapter_of(lo, row0 + 16 * m + i, M);
  for (int ad = next_adapter(id, -1); ad != 0x7FFFFFFF; ad = next_adapter(id, ad)) {
    const uint16_t* lb = (const uint16_t*)lo.LB + (int64_t)ad * lo.stride_lb + 8 * G;
    for (int r0 = 0; r0 < R; r0 += 32) {
      UPart u[MI];
      uint4 b[NI];
#pragma unroll
      for (int n = 0; n < NI; n++) b[n] = load8(lb + min(col0 + 16 * n + i, N - 1) * lo.ld_lb + r0, R - r0 - 8 * G);
#pragma unroll
      for (int m = 0; m < MI; m++) u[m] = load_u(lo.U, Rp, row0 + 16 * m + i, r0, lane, id[m] == ad);
      float z = 0.f;
#pragma unroll
      for (int n = 0; n < NI; n++) z = zeros_of<DT>(b[n], z);
#pragma unroll
      for (int m = 0; m < MI; m++) z = zeros_of(u[m], z);
      if (__any(z != 0.f)) {   // (NaN)
        Apart up[MI];
#pragma unroll
        for (int m = 0; m < MI; m++) {
          up[m] = take_apart(u[m].v);
          __builtin_amdgcn_sched_barrier(0);   // (one at a time: few registers)
        }
#pragma unroll
        for (int n = 0; n < NI; n++) {
          const Apart bp = take_apart<DT>(b[n]);
#pragma unroll
          for (int m = 0; m < MI; m++) {
            const f32x4 d = mfma16<BSM_BF16>(bp.o, up[m].c, mfma16<BSM_BF16>(bp.c, up[m].o, f32x4{0.f, 0.f, 0.f, 0.f}));
            if (id[m] == ad) acc[m][n] += d;
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int m = 0; m < MI; m++) {
        const uint32_t rows = (uint32_t)__ballot(id[m] == ad) & 0xFFFFu;
        if (!rows) continue;
        const USplit us = split_u(u[m]);
        if (rows == 0xFFFFu) {
#pragma unroll
          for (int n = 0; n < NI; n++) acc[m][n] = expand_step<DT>(us, b[n], acc[m][n]);
        } else {
#pragma unroll
          for (int n = 0; n < NI; n++) {
            const f32x4 d = expand_step<DT>(us, b[n], f32x4{0.f, 0.f, 0.f, 0.f});
            if (id[m] == ad) acc[m][n] += d;
          }
        }
      }
    }
  }
}

}  // namespace lora
}  // namespace bsm
