// router.hpp - the router's balance loss (k_router.hip): its arguments, and the exponential it shares with the
// cross entropy.
#pragma once
#include <algorithm>
#include <cmath>
#include <type_traits>
#include "bsm_device.hpp"

namespace bsm {

// A router's choices (k_router.hip): E experts (1 .. 1024), k ids a row.
struct RouterArgs {
  int64_t rows;
  int32_t E, k, l_fmt;      // l_fmt: BSM_F32, BSM_BF16 or BSM_F16
  int32_t vec;              // rows of logits start aligned to four elements
  const void* logits; int64_t ldl;
  const int32_t* ids;       // DEVICE, rows * k; outside 0 .. E - 1: no expert
  int32_t* counts;          // E, then the rows kept (read by the gradient)
  int32_t* offsets;         // E + 1
  float* loss;
  float scale;
};
struct RouterGradArgs {
  const float* dloss;       // DEVICE or NULL (1)
  void* D; int64_t ldd;
  int32_t d_fmt, vec, accum;
};
int64_t balance_workspace(int64_t rows, int E);
hipError_t launch_router_balance(const RouterArgs& a, void* workspace, hipStream_t st);
hipError_t launch_router_balance_grad(const RouterArgs& a, const RouterGradArgs& g, hipStream_t st);

// e^x for x <= 0 (softmax terms, exp(x - max)): the base-2 exponential of the rounded product x log2 e, times the
// first-order factor for what the rounding dropped, so the error stays a few ulp down to the underflow
// (without it |x| 2^-24: 50 ulp at x = -50). -infinity gives 0, NaN stays NaN.
__device__ __forceinline__ float exp_f32(float x) {
  constexpr float kLog2e = 0x1.715476p+0f, kLog2eRest = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
  const float p = x * kLog2e;
  const float r = __builtin_fmaf(x, kLog2eRest, __builtin_fmaf(x, kLog2e, -p));
  const float e = __builtin_amdgcn_exp2f(p);
  return x > -104.0f ? __builtin_fmaf(e, r * kLn2, e) : e;
}

}  // namespace bsm
