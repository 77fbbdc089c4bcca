// skinny.hpp - fp16/bf16 products of a few rows (up to 64) with K-major weights: the weights' stream
// bounds them, so each workgroup takes 16 columns (N / 16 workgroups: 256 at N 4096) and its eight waves
// split K, in interleaved pieces of 64.
//
// Weights go straight to registers: lane l holds row l%16, k 16(l/16) .. +15 of a piece (two 16-byte
// loads, so a row's piece is one whole 128-byte line) as two 16x16x32 matrix operands; the rows of X
// take the same order of k, so no value moves between lanes. No LDS and no barrier until the waves' sums
// meet, in a fixed order. Several pieces' loads are in flight per wave.
#pragma once
#include "lora.hpp"
#include "store16.hpp"

namespace bsm {
namespace skinny {

constexpr int WAVES = 8, BN = 16, THREADS = 64 * WAVES;

// The sums of this wave's pieces for rows m0 .. + 16 MT - 1 and columns n0 .. + 15: acc[mt] holds row
// 16 mt + l%16, columns 4(l/16) .. +3. Rows past M and columns past N repeat the last ones.
// The weights of eight pieces (a wave's whole share of K 4096) are asked for before anything else is,
// then `meanwhile` runs once, then the rows of X arrive two pieces at a time from the L2.
template <int DT, int MT, typename F>
__device__ __forceinline__ void product(const GemmArgs& a, int64_t m0, int64_t n0, int lane, int w, f32x4 (&acc)[MT],
                                        F meanwhile) {
  constexpr int U = 8;   // pieces whose weights are in flight
  const int i = lane & 15, G = lane >> 4;
  const uint16_t* b = (const uint16_t*)a.B + min(n0 + i, a.N - 1) * a.ldb + 16 * G;
  const uint16_t* x[MT];
#pragma unroll
  for (int m = 0; m < MT; m++) {
    x[m] = (const uint16_t*)a.A + min(m0 + 16 * m + i, a.M - 1) * a.lda + 16 * G;
    acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  const int full = (int)(a.K / 64);
  auto load_w = [&](int p, uint4 (&fb)[U][2]) {
#pragma unroll
    for (int u = 0; u < U; u++)
      if (p + u * WAVES < full) {
#pragma unroll
        for (int h = 0; h < 2; h++) fb[u][h] = *(const uint4*)(b + 64 * (int64_t)(p + u * WAVES) + 8 * h);
      }
  };
  uint4 fb[U][2];
  load_w(w, fb);
  asm volatile("" ::: "memory");   // (the loads stay ahead of what follows)
  meanwhile();
  for (int p = w; p < full; p += U * WAVES) {
    if (p != w) load_w(p, fb);
#pragma unroll
    for (int u0 = 0; u0 < U; u0 += 2) {
      uint4 fx[2][MT][2];
#pragma unroll
      for (int u = 0; u < 2; u++)
        if (p + (u0 + u) * WAVES < full) {
#pragma unroll
          for (int m = 0; m < MT; m++)
#pragma unroll
            for (int h = 0; h < 2; h++) fx[u][m][h] = *(const uint4*)(x[m] + 64 * (int64_t)(p + (u0 + u) * WAVES) + 8 * h);
        }
#pragma unroll
      for (int u = 0; u < 2; u++)
        if (p + (u0 + u) * WAVES < full) {
#pragma unroll
          for (int h = 0; h < 2; h++)
#pragma unroll
            for (int m = 0; m < MT; m++) acc[m] = lora::mfma16<DT>(fb[u0 + u][h], fx[u][m][h], acc[m]);
        }
    }
  }
  if (a.K % 64 && full % WAVES == w) {
    // the partial last piece, elements at or past K zero on both sides
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int64_t k = 64 * (int64_t)full + 8 * h, left = a.K - k - 16 * G;
      const uint4 bv = lora::load8(b + k, left);
#pragma unroll
      for (int m = 0; m < MT; m++) acc[m] = lora::mfma16<DT>(bv, lora::load8(x[m] + k, left), acc[m]);
    }
  }
}

// One lane's four outputs D = round(f(v (+ D))) at (row, col), masked at D's edges.
template <int DT>
__device__ __forceinline__ void store4(const GemmArgs& a, int64_t row, int64_t col, f32x4 v) {
  if (row >= a.M || col >= a.N) return;
  const bool whole = col + 4 <= a.N;
  if (a.d_fmt == BSM_F32) {
    float* p = a.D + row * a.ldd + col;
#pragma unroll
    for (int e = 0; e < 4; e++)
      if (whole || col + e < a.N) {
        if (a.accum) v[e] += p[e];
        if (a.ew_op) v[e] = silu_affine(v[e], a.ew_scale, a.ew_bias);
        if (!whole) p[e] = v[e];
      }
    if (whole) *(f32x4*)p = v;
    return;
  }
  uint16_t* p = (uint16_t*)a.D + row * a.ldd + col;
#pragma unroll
  for (int e = 0; e < 4; e++)
    if (whole || col + e < a.N) {
      if (a.accum) v[e] += gemm::from_bits16<DT>(p[e]);
      if (a.ew_op) v[e] = silu_affine(v[e], a.ew_scale, a.ew_bias);
      if (!whole) p[e] = gemm::to_bits16<DT>(v[e]);
    }
  if (whole) {
    const uint32_t lo = (uint32_t)gemm::to_bits16<DT>(v[0]) | ((uint32_t)gemm::to_bits16<DT>(v[1]) << 16);
    const uint32_t hi = (uint32_t)gemm::to_bits16<DT>(v[2]) | ((uint32_t)gemm::to_bits16<DT>(v[3]) << 16);
    *(uint2*)p = make_uint2(lo, hi);
  }
}

}  // namespace skinny
}  // namespace bsm
