// k_gemm_lora.hip - a shared projection with a low-rank adapter chosen per row (lora.hpp has the
// formula). Two launches: the shrink writes U, the projection adds U LB^T to its accumulators before
// its only store, so D is written once and never read back.
#include "gemm_dense_tile.hpp"
#include "lora.hpp"
#include "store16.hpp"

namespace bsm {
namespace {

using namespace dense;

// Shrink: workgroup (b, z, j) computes U[16b .. 16b + 15][16z .. 16z + 15] for the rows of the j-th
// distinct adapter of those 16 rows (none: it ends). Its four waves split K in interleaved pieces of
// 64 and are summed through LDS in a fixed order. Lane group G of a wave holds the contiguous k
// 16G .. 16G + 15 of a piece on both sides (two matrix instructions of 32), so a row's piece is one
// whole 128-byte line.
template <int DT>
__global__ __launch_bounds__(256) void k_lora_shrink(GemmArgs a, LoraArgs lo, int64_t Rp) {
  __shared__ f32x4 part[4][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, i = lane & 15, G = lane >> 4;
  const int64_t t = 16 * (int64_t)blockIdx.x + i;
  const int id = lora::adapter_of(lo, t, a.M);
  uint32_t firsts = lora::first_rows(id, lane);
  for (int j = blockIdx.z; j > 0 && firsts; j--) firsts &= firsts - 1;
  if (!firsts) return;
  const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(firsts));
  const bool mine = id == ad;
  const int r = 16 * blockIdx.y + i;
  const uint16_t* x = (const uint16_t*)a.A + t * a.lda + 16 * G;
  const uint16_t* la = (const uint16_t*)lo.LA + (int64_t)ad * lo.stride_la + (int64_t)r * lo.ld_la + 16 * G;
  const bool row = r < lo.R;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int64_t k0 = 64 * w; k0 < a.K; k0 += 256) {
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int64_t left = a.K - k0 - 16 * G - 8 * h;
      const uint4 av = lora::load8(x + k0 + 8 * h, mine ? left : 0);
      const uint4 bv = lora::load8(la + k0 + 8 * h, row ? left : 0);
      acc = lora::mfma16<DT>(bv, av, acc);
    }
  }
  part[w][lane] = acc;
  __syncthreads();
  if (w == 0 && mine) {
    f32x4 s = part[0][lane];
#pragma unroll
    for (int q = 1; q < 4; q++) s += part[q][lane];
    s *= lo.scale[ad];
    *(f32x4*)(lo.U + t * Rp + 16 * blockIdx.y + 4 * G) = s;
  }
}

template <int DT>
__global__ __launch_bounds__(256, 1) void k_lora(GemmArgs a, LoraArgs args, int64_t Rp, int tiles_m, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * STAGE_BYTES];
  // The adapters' arguments wait in LDS until the projection's K loop is over: held in SGPRs
  // through it they made the compiler spill some.
  __shared__ LoraArgs late;
  if (threadIdx.x == 0) late = args;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tm, tn;
  gemm::tile_coords(blockIdx.x, tiles_m, tiles_n, tm, tn);
  f32x4 acc[8][8];
  tile_product<DT, true, true>(a, tm, tn, lds, lane, w, acc);
  const int64_t row0 = (int64_t)tm * BM + 128 * (w >> 1), col0 = (int64_t)tn * BN + 128 * (w & 1);
  const int i = lane & 15, G = lane >> 4;
  const LoraArgs lo = late;
  const int R = __builtin_amdgcn_readfirstlane(lo.R);
#pragma unroll
  for (int mt = 0; mt < 8; mt++) {
    const int64_t t = row0 + 16 * mt + i;
    const int id = lora::adapter_of(lo, t, a.M);
    for (uint32_t firsts = lora::first_rows(id, lane); firsts; firsts &= firsts - 1) {
      const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(firsts));
      const bool mine = id == ad;
      const uint16_t* lb = (const uint16_t*)lo.LB + (int64_t)ad * lo.stride_lb + 8 * G;
      for (int r0 = 0; r0 < R; r0 += 32) {
        const lora::USplit u = lora::split_u(lora::load_u(lo.U, Rp, t, r0, lane, mine));
#pragma unroll
        for (int nt = 0; nt < 8; nt++) {
          const int64_t n = min(col0 + 16 * nt + i, a.N - 1);
          const uint4 b = lora::load8(lb + n * lo.ld_lb + r0, R - r0 - 8 * G);
          // (a sum of its own: another row's zeros times an infinity of this adapter are not zero)
          const f32x4 d = lora::expand_step<DT>(u, b);
          if (mine) acc[mt][nt] += d;
        }
      }
    }
  }
  uint8_t* region = lds + 32768 * w;
  if (a.d_fmt == BSM_F32)
    store_tile16(a.D, a.ldd, a.M, a.N, row0, col0, lane, 1.0f, acc, region, a.accum, a.ew_op, a.ew_scale, a.ew_bias);
  else
    gemm::store_tile16_bits<DT>((uint16_t*)a.D, a.ldd, a.M, a.N, row0, col0, lane, acc, region, a.accum, a.ew_op,
                                a.ew_scale, a.ew_bias);
}

template <int DT>
hipError_t launch(const GemmArgs& a, const LoraArgs& lo, hipStream_t st) {
  const int64_t Rp = lora::padded_rank(lo.R);
  const int64_t tm = (a.M + BM - 1) / BM, tn = (a.N + BN - 1) / BN;
  if (tm * tn > 0x7FFFFFFF) return hipErrorInvalidValue;
  if (lo.R > 0 && lo.n > 0) {
    const dim3 grid((uint32_t)((a.M + 15) / 16), (uint32_t)(Rp / 16), (uint32_t)(lo.n < 16 ? lo.n : 16));
    hipLaunchKernelGGL(k_lora_shrink<DT>, grid, dim3(256), 0, st, a, lo, Rp);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(k_lora<DT>, dim3((uint32_t)(tm * tn)), dim3(256), 0, st, a, lo, Rp, (int)tm, (int)tn);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_lora(const GemmArgs& a, const LoraArgs& lo, hipStream_t st) {
  return a.dtype == BSM_BF16 ? launch<BSM_BF16>(a, lo, st) : launch<BSM_F16>(a, lo, st);
}

}  // namespace bsm
