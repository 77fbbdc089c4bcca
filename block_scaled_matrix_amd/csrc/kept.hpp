// kept.hpp - activations kept as 8-bit codes with E8M0 scales: the calls' arguments, encoding, decoding, and the numbering
// of scale blocks.
#pragma once
#include <stdint.h>
#include "bsm_device.hpp"
#include "bsm_internal.hpp"
#include "../../include/bsm.h"

namespace bsm {

// Kept activations (k_checkpoint.hip): rows of K values as 8-bit codes (fmt BSM_E4M3 or BSM_E5M2) with an E8M0 scale per
// 32 of them.
struct KeptArgs {
  int64_t rows, K;
  int32_t fmt;
  uint8_t* Q; int64_t ldq;
  uint8_t* SF; int64_t ld_sf;
  int32_t x_fmt;                       // format of X and D: BSM_F32, BSM_BF16 or BSM_F16
  const void* X; int64_t ldx;          // what is saved, or dY of the gradient
  void* D; int64_t ldd;                // what is restored, or dX
  int32_t ew_op; float ew_scale, ew_bias;
};
hipError_t launch_block_scale_save(const KeptArgs& a, hipStream_t st);
hipError_t launch_block_scale_restore(const KeptArgs& a, hipStream_t st);
hipError_t launch_block_scale_ewise_grad(const KeptArgs& a, hipStream_t st);
// As launch_gemm_grouped_wgrad, B the codes (dtype_b BSM_E4M3 or BSM_E5M2) and SFB their scales.
hipError_t launch_gemm_kept_wgrad(const GemmArgs& a, const GroupArgs& gr, hipStream_t st);

namespace kept {

constexpr float kMaxF32 = 0x1.fffffep127f, kMaxBf16 = 0x1.fep127f;

// n / d for n < 2^31: the top of n times 2^(31+s) / d rounded up, 2^(s-1) < d <= 2^s. The excess of the
// multiplier, less than d, moves the quotient by less than 1 / d.
struct Divide {
  uint32_t d, mul, shift;
  explicit Divide(uint32_t by) : d(by), mul(0), shift(0) {
    while ((uint64_t(1) << shift) < by) shift++;
    mul = (uint32_t)(((uint64_t(1) << (31 + shift)) + by - 1) / by);
  }
  __device__ __forceinline__ uint32_t quotient(uint32_t n) const { return shift == 0 ? n : __umulhi(n, mul) >> (shift - 1); }
};

// Scale code of a block whose largest finite magnitude is `top`: the largest finite code of both formats is
// 1.75 * 2^EMAX, so with top = 1.f 2^(E-127) the exponent is E - 127 - EMAX, one more if 1.f > 1.75. (A subnormal or
// zero top clamps to code 0, as do all below 2^(EMAX - 126).)
template <int FMT>
__device__ __forceinline__ int scale_code(float top) {
  constexpr int EMAX = FMT == BSM_E4M3 ? 8 : 15;
  const uint32_t b = __float_as_uint(top);
  return max((int)(b >> 23) - EMAX + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0), 0);
}
// 2^(127 - code) and 2^(code - 127). A saved code is at most 247, so the first is a normal number; code 255 is NaN.
__device__ __forceinline__ float inverse_scale(int code) { return __uint_as_float((uint32_t)(254 - code) << 23); }
__device__ __forceinline__ float scale(int code) {
  return __uint_as_float(code == 0 ? 0x00400000u : code == 255 ? 0x7FC00000u : (uint32_t)code << 23);
}

// Four values inside the format's range to codes, rounded to nearest even; E4M3 has no infinity and takes NaN for it.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  int r = 0;
  if constexpr (FMT == BSM_E4M3) {
    r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  } else {
    r = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, r, false);
    r = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, r, true);
  }
  return (uint32_t)r;
}

// scale() for values that are taken in f16, where it need not be larger than 2^119 (2^112 for E5M2: from there on every code
// but 0 lies past f16's range, and none past float32's yet) nor smaller than 2^-126.
template <int FMT>
__device__ __forceinline__ float scale_f16(int code) {
  constexpr int TOP = FMT == BSM_E4M3 ? 246 : 239;
  return __uint_as_float(code == 255 ? 0x7FC00000u : (uint32_t)min(max(code, 1), TOP) << 23);
}

// From this scale code on a finite code may stand for 2^128 or more.
template <int FMT>
constexpr uint32_t kWideScale = FMT == BSM_E4M3 ? 247 : 240;

typedef float f32x2 __attribute__((ext_vector_type(2)));
// Four codes times the scale (exact: at most four significant bits). BOUND: finite codes beyond float32's range give its
// largest value, not infinity.
template <int FMT, bool BOUND = false>
__device__ __forceinline__ void decode4(uint32_t c, float s, float* v) {
  f32x2 lo, hi;
  if constexpr (FMT == BSM_E4M3) {
    lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false);
    hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
  } else {
    lo = __builtin_amdgcn_cvt_pk_f32_bf8((int)c, false);
    hi = __builtin_amdgcn_cvt_pk_f32_bf8((int)c, true);
  }
  const float u[4] = {lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
  for (int e = 0; e < 4; e++) {
    v[e] = u[e] * s;
    if constexpr (BOUND) v[e] = __builtin_fabsf(v[e]) == INFINITY && __builtin_fabsf(u[e]) < INFINITY ? __builtin_copysignf(kMaxF32, u[e]) : v[e];
  }
}

// Finite values to f16's and bf16's range; infinities and NaN as they are.
__device__ __forceinline__ float clamp_f16(float v) {
  return __builtin_fabsf(v) < INFINITY ? __builtin_amdgcn_fmed3f(v, -65504.0f, 65504.0f) : v;
}
__device__ __forceinline__ float clamp_bf16(float v) {
  return __builtin_fabsf(v) < INFINITY ? __builtin_amdgcn_fmed3f(v, -kMaxBf16, kMaxBf16) : v;
}

// d/dx x / (1 + e^-x) = s (1 + x (1 - s)), s = 1 / (1 + e^-x). With t = e^-|x| both s and 1 - s are quotients of
// 1 + t without cancellation: 1 / (1 + t) on x's side, t / (1 + t) on the other. The slope of +-infinity is the
// limit, 1 and 0.
__device__ __forceinline__ float silu_slope(float x) {
  constexpr float kLog2e = 0x1.715476p+0f, kLog2eRest = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
  const float z = x != x ? x : -fminf(__builtin_fabsf(x), 128.0f);   // (e^-128 x is below every float sum here)
  const float p = z * kLog2e;
  const float r = __builtin_fmaf(z, kLog2eRest, __builtin_fmaf(z, kLog2e, -p));
  const float e0 = __builtin_amdgcn_exp2f(p), t = __builtin_fmaf(e0, r * kLn2, e0);
  const float q = __builtin_amdgcn_rcpf(1.0f + t), near = q, far = t * q;
  // x >= 0: s = near, 1 - s = far; x < 0: s = far, 1 - s = near. |x| far is what the product adds on either side.
  return x < 0.0f ? far * __builtin_fmaf(z, near, 1.0f) : near * __builtin_fmaf(-z, far, 1.0f);
}

}  // namespace kept
}  // namespace bsm
