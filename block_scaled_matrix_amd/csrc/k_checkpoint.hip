// k_checkpoint.hip - activations kept in 8 bits for the backward pass, and their element-wise use there.
//
//   save:    per 32 values of a row, e the smallest exponent with amax <= max_fmt 2^e (amax over the finite values, e in
//            -127 .. 127), code = round(x 2^-e) to nearest even, scale code e + 127
//   restore: D = f(code 2^e)        ewise_grad: dX = dY f'(code 2^e)
//
// The scale is rounded up, not down to the exponent of amax: no value saturates (rounding down clips values between
// 448 and 512 times the scale by up to an eighth), at the cost of one bit of range at the bottom. x 2^-e is exact, so
// a code is x's only rounding.
// Bound by the bytes: eight values a lane (16 bytes of 16-bit rows, 8 bytes of codes), four lanes a scale block, two
// blocks' loads in flight a lane. The blocks of all rows are numbered through, so short rows fill the lanes as long
// ones do; the row of a number comes from a multiplication (Divide).
#include <algorithm>
#include <type_traits>
#include "bsm_device.hpp"
#include "kept.hpp"
#include "../../include/bsm.h"

namespace bsm {
namespace {

using kept::Divide;

constexpr int UNROLL = 2, PER_GROUP = 64;   // a workgroup of 256 lanes takes UNROLL * PER_GROUP scale blocks

// Eight values from element i on; those at or past `left` are 0. Rows are whole 16-byte chunks.
template <int F>
__device__ __forceinline__ void load8(const void* p, int64_t i, int left, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e++) v[e] = 0.0f;
  if (left <= 0) return;
  if constexpr (F == BSM_F32) {
    const float* q = (const float*)p + i;
    const f32x4 x = __builtin_nontemporal_load((const f32x4*)q);
#pragma unroll
    for (int e = 0; e < 4; e++) v[e] = e < left ? x[e] : 0.0f;
    if (left > 4) {
      const f32x4 y = __builtin_nontemporal_load((const f32x4*)(q + 4));
#pragma unroll
      for (int e = 0; e < 4; e++) v[4 + e] = 4 + e < left ? y[e] : 0.0f;
    }
  } else {
    const u32x4 x = __builtin_nontemporal_load((const u32x4*)((const uint16_t*)p + i));
#pragma unroll
    for (int e = 0; e < 8; e++) {
      const uint16_t h = (uint16_t)(x[e >> 1] >> (16 * (e & 1)));
      const float f = F == BSM_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h);
      v[e] = e < left ? f : 0.0f;
    }
  }
}

// Rounded to the format; finite values beyond f16's range become its largest (a value that fits f16 may be kept as a
// code just past it: 65504 as 65536), and where BOUND says so those beyond bf16's (its own last ones are kept as 2^128).
template <int F, bool BOUND>
__device__ __forceinline__ uint16_t bits16(float v) {
  if constexpr (F == BSM_BF16) return f32_to_bf16_bits(BOUND ? kept::clamp_bf16(v) : v);
  else return f32_to_f16_bits(kept::clamp_f16(v));
}

template <int F, bool BOUND>
__device__ __forceinline__ void store8(void* p, int64_t i, int left, const float (&v)[8]) {
  if constexpr (F == BSM_F32) {
    float* q = (float*)p + i;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      if (left >= 4 * h + 4) {
        const f32x4 x = {v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
        __builtin_nontemporal_store(x, (f32x4*)(q + 4 * h));
      } else {
#pragma unroll
        for (int e = 4 * h; e < 4 * h + 4; e++)
          if (e < left) q[e] = v[e];
      }
    }
  } else {
    uint16_t* q = (uint16_t*)p + i;
    if (left >= 8) {
      u32x4 x;
#pragma unroll
      for (int e = 0; e < 4; e++) x[e] = bits16<F, BOUND>(v[2 * e]) | (uint32_t)bits16<F, BOUND>(v[2 * e + 1]) << 16;
      __builtin_nontemporal_store(x, (u32x4*)q);
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (e < left) q[e] = bits16<F, BOUND>(v[e]);
    }
  }
}

// Eight codes at byte i of a row (a multiple of 8), `left` of them wanted; rows are whole 16-byte chunks.
__device__ __forceinline__ void load_codes(const uint8_t* p, int64_t at, int left, uint32_t (&c)[2]) {
  c[0] = c[1] = 0;
  if (left > 0) {
    const uint2 x = *(const uint2*)(p + at);
    c[0] = x.x; c[1] = x.y;
  }
}

// Number `q` of the launch's scale blocks, as row and first element; this lane's eight of its 32 start at `col`.
struct Place { int64_t row; int col, left; bool in; };
__device__ __forceinline__ Place place(const KeptArgs& a, const Divide& per_row, uint32_t blocks, int u) {
  const uint32_t q = (blockIdx.x * UNROLL + u) * PER_GROUP + (threadIdx.x >> 2);
  Place p;
  p.in = q < blocks;
  const uint32_t row = per_row.quotient(q);
  p.row = row;
  p.col = (int)(q - row * per_row.d) * 32 + 8 * (threadIdx.x & 3);
  p.left = p.in ? (int)min(a.K - p.col, (int64_t)8) : 0;
  return p;
}

template <int F, int FMT>
__global__ __launch_bounds__(256) void k_save(KeptArgs a, Divide per_row, uint32_t blocks) {
  float v[UNROLL][8];
  Place p[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; u++) {
    p[u] = place(a, per_row, blocks, u);
    load8<F>(a.X, p[u].row * a.ldx + p[u].col, p[u].left, v[u]);
  }
#pragma unroll
  for (int u = 0; u < UNROLL; u++) {
    float top = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      const float m = __builtin_fabsf(v[u][e]);
      top = fmaxf(top, m < INFINITY ? m : 0.0f);
    }
    top = fmaxf(top, __shfl_xor(top, 1));
    top = fmaxf(top, __shfl_xor(top, 2));
    const int code = kept::scale_code<FMT>(top);
    const float by = kept::inverse_scale(code);
    uint32_t c[2];
#pragma unroll
    for (int h = 0; h < 2; h++) c[h] = kept::encode4<FMT>(v[u][4 * h] * by, v[u][4 * h + 1] * by, v[u][4 * h + 2] * by, v[u][4 * h + 3] * by);
    uint8_t* q = a.Q + p[u].row * a.ldq + p[u].col;
    if (p[u].left >= 8) {
      *(uint2*)q = make_uint2(c[0], c[1]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (e < p[u].left) q[e] = (uint8_t)(c[e >> 2] >> (8 * (e & 3)));
    }
    if (p[u].in && (threadIdx.x & 3) == 0) a.SF[p[u].row * a.ld_sf + p[u].col / 32] = (uint8_t)code;
  }
}

// EW 0: D = x, 1: D = f(x), 2: D = dY f'(x).
template <int F, int FMT, int EW>
__global__ __launch_bounds__(256) void k_use(KeptArgs a, Divide per_row, uint32_t blocks) {
  uint32_t c[UNROLL][2];
  float dy[UNROLL][8], s[UNROLL];
  Place p[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; u++) {
    p[u] = place(a, per_row, blocks, u);
    load_codes(a.Q, p[u].row * a.ldq + p[u].col, p[u].left, c[u]);
    s[u] = kept::scale(p[u].in ? a.SF[p[u].row * a.ld_sf + p[u].col / 32] : 127);
    if constexpr (EW == 2) load8<F>(a.X, p[u].row * a.ldx + p[u].col, p[u].left, dy[u]);
  }
#pragma unroll
  for (int u = 0; u < UNROLL; u++) {
    float v[8];
    // A finite value is made a finite one in 16 bits, and f of it (-2^128, a mask's fill as it is kept, gives f's limit and
    // not NaN). In float32 without f it is the value rounded: infinity from 2^128 on. The slope has the same limits at both.
    constexpr bool BOUND = EW == 1 || (EW == 0 && F != BSM_F32);
#pragma unroll
    for (int h = 0; h < 2; h++) kept::decode4<FMT, BOUND>(c[u][h], s[u], v + 4 * h);
#pragma unroll
    for (int e = 0; e < 8; e++) {
      if constexpr (EW == 1) {
        const float x = v[e];
        v[e] = silu_affine(x, a.ew_scale, a.ew_bias);
        if constexpr (F != BSM_F32)   // (times a scale above 1 it may leave float32)
          if (__builtin_fabsf(v[e]) == INFINITY && __builtin_fabsf(x) < INFINITY && __builtin_fabsf(a.ew_scale) < INFINITY &&
              __builtin_fabsf(a.ew_bias) < INFINITY)
            v[e] = __builtin_copysignf(kept::kMaxF32, v[e]);
      }
      if constexpr (EW == 2) v[e] = dy[u][e] * (a.ew_op ? a.ew_scale * kept::silu_slope(v[e]) : 1.0f);
    }
    store8<F, EW != 2>(a.D, p[u].row * a.ldd + p[u].col, p[u].left, v);
  }
}

// The rows in slices of fewer than 2^31 scale blocks: launch(slice, Divide, blocks).
template <class FN>
hipError_t in_slices(const KeptArgs& a, int xsize, FN launch) {
  const int64_t per_row = (a.K + 31) / 32, most = std::max<int64_t>((int64_t(1) << 30) / per_row, 1);
  for (int64_t r = 0; r < a.rows; r += most) {
    KeptArgs t = a;
    t.rows = std::min(most, a.rows - r);
    t.Q = a.Q + r * a.ldq;
    t.SF = a.SF + r * a.ld_sf;
    if (a.X) t.X = (const uint8_t*)a.X + r * a.ldx * xsize;
    if (a.D) t.D = (uint8_t*)a.D + r * a.ldd * xsize;
    const uint32_t blocks = (uint32_t)(t.rows * per_row);
    launch(t, Divide((uint32_t)per_row), blocks, dim3((blocks + UNROLL * PER_GROUP - 1) / (UNROLL * PER_GROUP)));
  }
  return hipGetLastError();
}

// f(format of X and D, format of the codes).
template <class FN>
hipError_t with_formats(const KeptArgs& a, FN f) {
  using std::integral_constant;
  auto second = [&](auto x) {
    return a.fmt == BSM_E4M3 ? f(x, integral_constant<int, BSM_E4M3>{}) : f(x, integral_constant<int, BSM_E5M2>{});
  };
  if (a.x_fmt == BSM_F32) return second(integral_constant<int, BSM_F32>{});
  if (a.x_fmt == BSM_BF16) return second(integral_constant<int, BSM_BF16>{});
  return second(integral_constant<int, BSM_F16>{});
}

template <int EW>
hipError_t launch_use(const KeptArgs& a, hipStream_t st) {
  return with_formats(a, [&](auto x, auto fmt) {
    constexpr int F = decltype(x)::value, FMT = decltype(fmt)::value;
    return in_slices(a, F == BSM_F32 ? 4 : 2, [&](const KeptArgs& t, Divide d, uint32_t blocks, dim3 grid) {
      hipLaunchKernelGGL((k_use<F, FMT, EW>), grid, dim3(256), 0, st, t, d, blocks);
    });
  });
}

}  // namespace

hipError_t launch_block_scale_save(const KeptArgs& a, hipStream_t st) {
  return with_formats(a, [&](auto x, auto fmt) {
    constexpr int F = decltype(x)::value, FMT = decltype(fmt)::value;
    return in_slices(a, F == BSM_F32 ? 4 : 2, [&](const KeptArgs& t, Divide d, uint32_t blocks, dim3 grid) {
      hipLaunchKernelGGL((k_save<F, FMT>), grid, dim3(256), 0, st, t, d, blocks);
    });
  });
}

hipError_t launch_block_scale_restore(const KeptArgs& a, hipStream_t st) {
  return a.ew_op ? launch_use<1>(a, st) : launch_use<0>(a, st);
}

hipError_t launch_block_scale_ewise_grad(const KeptArgs& a, hipStream_t st) { return launch_use<2>(a, st); }

}  // namespace bsm
