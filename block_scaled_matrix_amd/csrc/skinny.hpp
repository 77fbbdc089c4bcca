// skinny.hpp - fp16/bf16 products of a few rows (up to 64) with K-major weights: the weights' stream
// bounds them, so each workgroup takes 16 columns (N / 16 workgroups: 256 at N 4096) and its eight waves
// split K, in interleaved pieces of 64.
//
// A piece of 16 rows x 64 K (weights, or 16 rows of X) is loaded as eight lanes a 128-byte row, written
// to LDS in the K-major tile layout of gemm_common.hpp and read back as the two 16x16x32 operands, all by
// one wave in a buffer of its own: no barrier until the waves' sums meet, in a fixed order. Loading the
// operands' own layout (sixteen lanes, sixteen rows) without LDS was bound by the address path, which
// takes four neighbouring lanes a clock only if they share a line: 48 rows, N = K = 4096 took 22.9 us.
#pragma once
#include "lora.hpp"
#include "store16.hpp"

namespace bsm {
namespace skinny {

// (Up to 16 rows two workgroups share a CU, 128 registers a lane.)
constexpr int WAVES = 8, BN = 16, THREADS = 64 * WAVES;

// LDS a workgroup needs: each wave a piece of the weights and MT of X.
template <int MT>
constexpr int lds_bytes() { return WAVES * (1 + MT) * 2048; }

// The sums of this wave's pieces for rows m0 .. + 16 MT - 1 and columns n0 .. + 15: acc[mt] holds row
// 16 mt + l%16, columns 4(l/16) .. +3. Rows past M and columns past N repeat the last ones.
// P pieces of the weights and of X are in flight per wave, asked for before anything else is; then
// `meanwhile` runs once.
template <int DT, int MT, typename F>
__device__ __forceinline__ void product(const GemmArgs& a, int64_t m0, int64_t n0, int lane, int w, uint8_t* buf,
                                        f32x4 (&acc)[MT], F meanwhile) {
  constexpr int P = MT <= 2 ? 4 : MT == 3 ? 3 : 2;   // (what the registers hold)
  const int i = lane & 15, G = lane >> 4, lr = lane >> 3, lc = lane & 7;
  // this lane's rows (8h + lr of a 16-row block) at its chunk lc of a piece, and where they go in LDS
  const uint16_t* b[2];
  const uint16_t* x[MT][2];
  uint32_t at[2];
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const int r = 8 * h + lr;
    b[h] = (const uint16_t*)a.B + min(n0 + r, a.N - 1) * a.ldb + 8 * lc;
    at[h] = (uint32_t)(r * 128 + ((lc ^ ((r >> 1) & 7)) << 4));
#pragma unroll
    for (int m = 0; m < MT; m++) x[m][h] = (const uint16_t*)a.A + min(m0 + 16 * m + r, a.M - 1) * a.lda + 8 * lc;
  }
#pragma unroll
  for (int m = 0; m < MT; m++) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int full = (int)(a.K / 64);
  uint4 fb[P][2], fx[P][MT][2];
  auto load = [&](int p, uint4 (&wv)[2], uint4 (&xv)[MT][2]) {
    if (p < full) {
#pragma unroll
      for (int h = 0; h < 2; h++) {
        wv[h] = *(const uint4*)(b[h] + 64 * (int64_t)p);
#pragma unroll
        for (int m = 0; m < MT; m++) xv[m][h] = *(const uint4*)(x[m][h] + 64 * (int64_t)p);
      }
    }
  };
  auto multiply = [&](const uint4 (&wv)[2], const uint4 (&xv)[MT][2]) {
#pragma unroll
    for (int h = 0; h < 2; h++) {
      lds_write_b128(buf + at[h], wv[h]);
#pragma unroll
      for (int m = 0; m < MT; m++) lds_write_b128(buf + 2048 * (m + 1) + at[h], xv[m][h]);
    }
#pragma unroll
    for (int s = 0; s < 2; s++) {
      const uint32_t o = (uint32_t)(i * 128 + (((4 * s + G) ^ ((i >> 1) & 7)) << 4));
      const uint4 bv = lds_read_b128(buf + o);
#pragma unroll
      for (int m = 0; m < MT; m++) acc[m] = lora::mfma16<DT>(bv, lds_read_b128(buf + 2048 * (m + 1) + o), acc[m]);
    }
  };
#pragma unroll
  for (int u = 0; u < P; u++) load(w + u * WAVES, fb[u], fx[u]);
  asm volatile("" ::: "memory");   // (the loads stay ahead of what follows)
  meanwhile();
  for (int p = w; p < full; p += P * WAVES) {
#pragma unroll
    for (int u = 0; u < P; u++) {
      const int q = p + u * WAVES;
      if (q < full) multiply(fb[u], fx[u]);
      load(q + P * WAVES, fb[u], fx[u]);
    }
  }
  if (a.K % 64 && full % WAVES == w) {
    // the partial last piece, elements at or past K zero on both sides
    const int64_t k = 64 * (int64_t)full, left = a.K - k - 8 * lc;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      fb[0][h] = lora::load8(b[h] + k, left);
#pragma unroll
      for (int m = 0; m < MT; m++) fx[0][m][h] = lora::load8(x[m][h] + k, left);
    }
    multiply(fb[0], fx[0]);
  }
}

// Joins the waves' sums in wave order: on return acc[0] of wave m < MT is the sum for the 16 rows 16 m ..
template <int MT>
__device__ __forceinline__ void join(uint8_t* lds, int lane, int w, f32x4 (&acc)[MT]) {
  uint8_t* buf = lds + w * (1 + MT) * 2048;   // the wave's own, free after its product
#pragma unroll
  for (int m = 0; m < MT; m++) *(BSM_LDS f32x4*)(buf + 1024 * m + 16 * lane) = acc[m];
  __syncthreads();
  if (w < MT) {
    acc[0] = *(const BSM_LDS f32x4*)(lds + 1024 * w + 16 * lane);
#pragma unroll
    for (int q = 1; q < WAVES; q++) acc[0] += *(const BSM_LDS f32x4*)(lds + q * (1 + MT) * 2048 + 1024 * w + 16 * lane);
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
