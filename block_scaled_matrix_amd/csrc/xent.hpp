// xent.hpp - cross entropy of a projection (k_gemm_xent.hip): the calls' arguments, and what a tile of logits becomes
// while it is still in the accumulators.
#pragma once
#include <type_traits>
#include "bsm_internal.hpp"
#include "store16.hpp"

namespace bsm {

struct XentArgs {
  int64_t rows, N, K;                       // N: columns of the vocabulary
  int32_t dtype;                            // of X and W: BSM_BF16 or BSM_F16
  const void* X; int64_t ldx;
  const void* W; int64_t ldw;
  const int32_t* labels;                    // DEVICE, rows; outside 0 .. N - 1: none
  float* lse;                               // written by the loss, read by the gradient
  float* loss;
};
struct XentGradArgs {
  const float* dloss;                       // DEVICE, rows
  int64_t piece;                            // columns at once (0: the library's choice)
  void* dX; int64_t lddx; int32_t dx_fmt;   // NULL: not wanted
  void* dW; int64_t lddw; int32_t dw_fmt, accum;
};
int64_t xent_workspace(int64_t rows, int64_t N);
hipError_t launch_xent(const XentArgs& a, void* workspace, hipStream_t st);
int64_t xent_grad_workspace(int64_t rows, int64_t N, int64_t K, int64_t piece);
hipError_t launch_xent_grad(const XentArgs& a, const XentGradArgs& g, void* workspace, hipStream_t st);

namespace xent {

constexpr float kLog2e = 0x1.715476p+0f;    // log2 e as float; what it lacks is made up for where the sums meet

// A wave's block of logits, MI x NJ blocks of 16 x 16 at (row0, col0): acc[m][n][e] is row row0 + 16m + l%16, column
// col0 + 16n + 4(l/16) + e. Columns at or past N do not exist.

// One row of blocks in registers of its own: what follows changes copies. (Accumulators that a branch behind the K loop
// changes made the compiler move up to 480 of them about in every turn of the 256 x 256 tile's loop: 2123 us for
// 8190 x 32001 x 4096 against 1603 us.)
template <int NJ>
__device__ __forceinline__ void take(const f32x4 (&row)[NJ], f32x4 (&v)[NJ]) {
#pragma unroll
  for (int n = 0; n < NJ; n++) {
    v[n] = row[n];
    asm volatile("" : "+v"(v[n]));
  }
}

// Its rows' part of the log-sum-exp: base b, the largest logit times log2 e, and s = sum 2^(z log2 e - b), to slot
// col0 / width; and the logit of the rows' labels that lie in it. b is a float that the join takes as it is, so its
// rounding cancels; the exponent's own fma rounds once. (A logit whose b overflows counts as infinite.)
struct Stats {
  static constexpr bool kStores = true;
  const int32_t* labels;
  float2* part;      // slots of `rows` pairs
  float* at;         // rows
  int64_t rows, N;
  int width;
  template <int MI, int NJ>
  __device__ __forceinline__ void operator()(int64_t row0, int64_t col0, f32x4 (&acc)[MI][NJ]) const {
    if (col0 >= N) return;
    const int lane = threadIdx.x & 63, G = lane >> 4;
    const bool edge = col0 + 16 * NJ > N;   // wave-uniform
    float2* to = part + (col0 / width) * rows;
#pragma unroll
    for (int m = 0; m < MI; m++) {
      f32x4 v[NJ];
      take(acc[m], v);
      const int64_t row = row0 + 16 * m + (lane & 15);
      if (edge) {
        const int left = (int)(N - col0) - 4 * G;
#pragma unroll
        for (int n = 0; n < NJ; n++)
#pragma unroll
          for (int e = 0; e < 4; e++) v[n][e] = 16 * n + e < left ? v[n][e] : -INFINITY;
      }
      float top = -INFINITY;
#pragma unroll
      for (int n = 0; n < NJ; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) top = fmaxf(top, v[n][e]);
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float b = top * kLog2e, from = b == -INFINITY ? 0.0f : b;
      float s = 0.0f;
#pragma unroll
      for (int n = 0; n < NJ; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) s += __builtin_amdgcn_exp2f(__builtin_fmaf(v[n][e], kLog2e, -from));
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      const bool in = row < rows;
      if (in && G == 0) to[row] = make_float2(b, s);
      const int64_t off = (in ? (int64_t)labels[row] : -1) - col0;
      const bool mine = off >= 0 && off < 16 * NJ && ((off >> 2) & 3) == G;
      if (__any(mine)) {
        const int o = (int)off - 4 * G;
        float z = 0.0f;
#pragma unroll
        for (int n = 0; n < NJ; n++)
#pragma unroll
          for (int e = 0; e < 4; e++) z = 16 * n + e == o ? v[n][e] : z;
        if (mine) at[row] = z;
      }
    }
  }
};

// The gradient in the logits, (softmax - onehot) times the row's weight. Column 0 of the block is column `first` of the
// vocabulary. Rows without a label give 0 whatever their logits.
struct Weights {
  const int32_t* labels;
  const float* lse;
  const float* dloss;
  const float* by;     // a power of two on the weights (f16), or NULL
  int64_t rows, vocabulary, first;
  // One row of blocks, logits in, gradients out.
  template <int NJ>
  __device__ __forceinline__ void turn(int64_t row, int64_t col0, int G, float f, f32x4 (&v)[NJ]) const {
    const bool in = row < rows;
    const int64_t lab = in ? labels[row] : -1;
    const bool has = lab >= 0 && lab < vocabulary;
    const float d = has ? dloss[row] * f : 0.0f, l = has ? lse[row] : 0.0f;
    // 2^(z log2 e - l log2 e), the second product in two floats
    const float hi = l * kLog2e, lo = __builtin_fmaf(l, kLog2e, -hi);
#pragma unroll
    for (int n = 0; n < NJ; n++)
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(v[n][e], kLog2e, -hi) - lo);
        v[n][e] = has ? p * d : 0.0f;
      }
    const int64_t off = lab - first - col0;
    const bool mine = has && off >= 0 && off < 16 * NJ && ((off >> 2) & 3) == G;
    if (__any(mine)) {
      // p d - d, not (p - 1) d: one rounding more, half a float step of d
      const int o = mine ? (int)off - 4 * G : -1;
#pragma unroll
      for (int n = 0; n < NJ; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) v[n][e] -= 16 * n + e == o ? d : 0.0f;
    }
  }
};

// In place, for the tile's own 16-bit store.
struct Grad : Weights {
  static constexpr bool kStores = false;
  template <int MI, int NJ>
  __device__ __forceinline__ void operator()(int64_t row0, int64_t col0, f32x4 (&acc)[MI][NJ]) const {
    const int lane = threadIdx.x & 63;
    const float f = by ? *by : 1.0f;
#pragma unroll
    for (int m = 0; m < MI; m++) {
      f32x4 v[NJ];
      take(acc[m], v);
      turn(row0 + 16 * m + (lane & 15), col0, lane >> 4, f, v);
#pragma unroll
      for (int n = 0; n < NJ; n++) acc[m][n] = v[n];
    }
  }
};

// As the sum of T 16-bit terms, rounded and again what the rounding dropped, for gradients kept in float32: term t at `to` +
// t * second. Three terms are all of a float's bits in bf16 (24, eight a term); two leave at most 2^-23 of the value in f16.
template <int DT, int T>
struct GradTerms : Weights {
  static constexpr bool kStores = true;
  uint16_t* to;
  int64_t ld, second, cols;
  template <int MI, int NJ>
  __device__ __forceinline__ void operator()(int64_t row0, int64_t col0, f32x4 (&acc)[MI][NJ]) const {
    const int lane = threadIdx.x & 63, G = lane >> 4;
    const float f = by ? *by : 1.0f;
    if (col0 >= cols) return;
    const bool whole = col0 + 16 * NJ <= cols;   // wave-uniform
#pragma unroll
    for (int m = 0; m < MI; m++) {
      const int64_t row = row0 + 16 * m + (lane & 15);
      f32x4 v[NJ];
      take(acc[m], v);
      turn(row, col0, G, f, v);
      // (taken anew for each row of blocks: kept, the comparisons' masks spilled scalar registers)
      int left = (int)min(cols - col0, (int64_t)(16 * NJ)) - 4 * G;
      asm volatile("" : "+v"(left));
      uint16_t* q = to + row * ld + col0 + 4 * G;
      auto store = [&](auto all) {
#pragma unroll
        for (int n = 0; n < NJ; n++) {
          uint16_t* p = q + 16 * n;
#pragma unroll
          for (int t = 0; t < T; t++) {
            uint16_t h[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
              h[e] = gemm::to_bits16<DT>(v[n][e]);
              v[n][e] -= gemm::from_bits16<DT>(h[e]);
            }
            if (decltype(all)::value || 16 * n + 4 <= left) {
              *(uint2*)p = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
            } else {
#pragma unroll
              for (int e = 0; e < 4; e++)
                if (16 * n + e < left) p[e] = h[e];
            }
            p += second;
          }
        }
      };
      if (row < rows) {
        if (whole) store(std::true_type{});
        else store(std::false_type{});
      }
    }
  }
};

// Sums as they are, or times a power of two on the device (f16; NULL where there are no rows, whose sums are 0).
template <bool BY>
struct Times {
  static constexpr bool kStores = false;
  const float* by;
  template <int MI, int NJ>
  __device__ __forceinline__ void operator()(int64_t, int64_t, f32x4 (&acc)[MI][NJ]) const {
    if constexpr (BY) {
      const float f = by ? *by : 1.0f;
#pragma unroll
      for (int m = 0; m < MI; m++)
#pragma unroll
        for (int n = 0; n < NJ; n++) acc[m][n] *= f;
    }
  }
};

}  // namespace xent
}  // namespace bsm
