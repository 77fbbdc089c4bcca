// k_gemm_lora.hip - a shared projection with a low-rank adapter chosen per row (lora.hpp has the
// formula). Two launches: the shrink writes U, the projection adds U LB^T to its accumulators before
// its only store, so D is written once and never read back. For decode batches both adapters' parts work
// row by row on the vector units, beside the weights' stream; beyond, on the matrix units.
#include "gemm_mid_tile.hpp"
#include "grouped.hpp"
#include "lora.hpp"
#include "skinny.hpp"
#include "store16.hpp"

namespace bsm {
namespace {

// Shrink: workgroup (b, y, z) computes U[32b .. 32b + 31][128y .. 128y + 127] for the z-th, (z + Z)-th, ..
// distinct adapter of those 32 rows in ascending order, on gemm_mid_tile.hpp's 32 x 128 tile with the
// adapter's LA as the weights. Rows of other adapters are multiplied along and not stored; values past R
// are zero. Bound by the copies into LDS (LA again for every 32 rows).
template <int DT>
struct StoreU {
  static constexpr bool kStores = true;
  const LoraArgs* late;
  int64_t Rp, M;
  int ad, lane;
  template <int MI>
  __device__ __forceinline__ void operator()(int64_t row0, int64_t col0, f32x4 (&acc)[MI][4]) const {
    const LoraArgs lo = *late;
    const int i = lane & 15, G = lane >> 4;
    const float scale = lo.scale[ad];
#pragma unroll
    for (int m = 0; m < MI; m++) {
      const int64_t t = row0 + 16 * m + i;
      if (lora::adapter_of(lo, t, M) != ad) continue;
#pragma unroll
      for (int n = 0; n < 4; n++) {
        const int r = (int)col0 + 16 * n + 4 * G;
        if (r >= Rp) continue;
        f32x4 u;
#pragma unroll
        for (int e = 0; e < 4; e++) u[e] = r + e < lo.R ? acc[m][n][e] * scale : 0.f;
        *(f32x4*)(lo.U + t * Rp + r) = u;
      }
    }
  }
};

template <int DT>
__global__ __launch_bounds__(256, 2) void k_lora_shrink(GemmArgs a, LoraArgs lo, int64_t Rp) {
  // The arguments that only the store needs wait in LDS, beside the tile's three stages (two
  // workgroups a CU still fit): held in SGPRs through the tile's loop they made the compiler spill some.
  constexpr int TILE = 60 * 1024;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[TILE];
  __shared__ LoraArgs late;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = 32 * (int64_t)blockIdx.x;
  int id[2];
#pragma unroll
  for (int m = 0; m < 2; m++) id[m] = lora::adapter_of(lo, m0 + 16 * m + (lane & 15), a.M);
  int ad = lora::next_adapter(id, -1);
  for (int z = 0; z < (int)blockIdx.z && ad != 0x7FFFFFFF; z++) ad = lora::next_adapter(id, ad);
  if (threadIdx.x == 0) late = lo;
  __syncthreads();
  while (ad != 0x7FFFFFFF) {
    GemmArgs p = a;
    p.B = (const uint16_t*)lo.LA + (int64_t)ad * lo.stride_la;
    p.ldb = lo.ld_la;
    p.N = lo.R;
    mid::tile<DT, 32, true, true, 64, StoreU<DT>, TILE>(p, m0, 128 * (int64_t)blockIdx.y, lds, lane, w,
                                                        StoreU<DT>{&late, Rp, a.M, ad, lane});
    for (int z = 0; z < (int)gridDim.z && ad != 0x7FFFFFFF; z++) ad = lora::next_adapter(id, ad);
    __syncthreads();   // every wave is done with LDS
  }
}

// Projection and expand on tiles of 32, 64 or 128 x 128 (the last rows take the smallest that holds
// them), two workgroups a CU. (On the 256 x 256 tile, whose accumulators leave the expand few
// registers, 8190 rows with rank 64, N 8192, K 4096 took 714 us.)
template <int DT>
struct Expand {
  static constexpr bool kStores = false;
  const LoraArgs& lo;
  int64_t Rp, M, N;
  int lane;
  template <int MI>
  __device__ __forceinline__ void operator()(int64_t row0, int64_t col0, f32x4 (&acc)[MI][4]) const {
    lora::expand<DT>(lo, Rp, M, N, row0, col0, lane, acc);
  }
};

// Q waves' fours a tile (gemm_mid_tile.hpp): 1, or 2 with tiles of 64 rows where there are few.
template <int DT, int Q>
__global__ __launch_bounds__(256 * Q, 3 - Q) void k_lora(GemmArgs a, LoraArgs lo, int64_t Rp, int tiles_m, int tiles_n) {
  constexpr int ROWS = Q == 1 ? 128 : 64;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Q * mid::LDS_BYTES];
  const int lane = threadIdx.x & 63, wq = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wq & 3, q = wq >> 2;
  // (an XCD's workgroups take a contiguous eighth of the tiles, in bands of eight tile rows)
  const int total = tiles_m * tiles_n, share = (total + 7) >> 3, lid = ((int)blockIdx.x & 7) * share + ((int)blockIdx.x >> 3);
  if (lid >= total) return;
  int tm, tn;
  grouped::band_tile<8>(lid, tiles_m, tiles_n, tm, tn);
  const Expand<DT> expand{lo, Rp, a.M, a.N, lane};
  const int64_t m0 = ROWS * (int64_t)tm, n0 = mid::BN * (int64_t)tn;
  const int64_t left = a.M - m0;
  uint8_t* part = lds + q * mid::LDS_BYTES;
  if (left <= 32) mid::tile<DT, 32, true, true, 64, Expand<DT>, mid::LDS_BYTES, Q>(a, m0, n0, part, lane, w, expand, q);
  else if (ROWS == 64 || left <= 64) mid::tile<DT, 64, true, true, 64, Expand<DT>, mid::LDS_BYTES, Q>(a, m0, n0, part, lane, w, expand, q);
  else if constexpr (ROWS == 128) mid::tile<DT, 128, true, true, 64, Expand<DT>, mid::LDS_BYTES, Q>(a, m0, n0, part, lane, w, expand, q);
}

// Eight consecutive 16-bit values as float32.
template <int DT>
__device__ __forceinline__ void widen8(uint4 x, float (&v)[8]) {
  const uint32_t wd[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int e = 0; e < 8; e++) {
    const uint16_t h = (uint16_t)(wd[e >> 1] >> (16 * (e & 1)));
    v[e] = DT == BSM_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h);
  }
}

// Shrink of few rows: workgroup (t, z) computes U[t][32z .. 32z + 31], wave w of sixteen its values
// 32z + w and + 16: lane l sums the products of k 8l .. 8l + 7 of every 512 (one line of each operand
// per eight lanes, eight pieces of 512 asked for at once), the lanes in a fixed tree. Values past R
// are zero.
template <int DT>
__global__ __launch_bounds__(1024) void k_lora_shrink_rows(GemmArgs a, LoraArgs lo, int64_t Rp) {
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.x;
  const int id = __builtin_amdgcn_readfirstlane(lora::adapter_of(lo, t, a.M));
  if (id < 0) return;
  const uint16_t* x = (const uint16_t*)a.A + t * a.lda + 8 * lane;
  for (int r = 32 * blockIdx.y + w; r < 32 * (int)blockIdx.y + 32; r += 16) {
    float s = 0.f;
    if (r < lo.R) {
      const uint16_t* la = (const uint16_t*)lo.LA + (int64_t)id * lo.stride_la + (int64_t)r * lo.ld_la + 8 * lane;
      auto dot = [&](uint4 p, uint4 q) {
        float pf[8], qf[8];
        widen8<DT>(p, pf);
        widen8<DT>(q, qf);
#pragma unroll
        for (int e = 0; e < 8; e++) s = __builtin_fmaf(pf[e], qf[e], s);
      };
      int64_t k = 0;
      for (; k + 8 * 512 <= a.K; k += 8 * 512) {
        uint4 xv[8], v[8];
#pragma unroll
        for (int q = 0; q < 8; q++) {
          xv[q] = *(const uint4*)(x + k + 512 * q);
          v[q] = *(const uint4*)(la + k + 512 * q);
        }
#pragma unroll
        for (int q = 0; q < 8; q++) dot(xv[q], v[q]);
      }
#pragma unroll 2
      for (; k < a.K; k += 512) {
        const int64_t left = a.K - k - 8 * lane;
        dot(lora::load8(x + k, left), lora::load8(la + k, left));
      }
#pragma unroll
      for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
      s *= lo.scale[id];
    }
    if (lane == 0) lo.U[t * Rp + r] = s;
  }
}

// Projection and expand of few rows: skinny.hpp's product for 16 MT rows and, while its weights are on
// their way, the adapters' part, row by row: wave w takes rows w, w + 8, ..; lane l sums r 8(l/16) .. +7 of every 32 for column l%16, in
// float32, the four lanes of a column in a fixed tree. A row reads its own adapter only.
template <int DT, int MT>
__global__ __launch_bounds__(skinny::THREADS, MT == 1 ? 4 : 2) void k_lora_skinny(GemmArgs a, LoraArgs lo, int64_t Rp, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[skinny::lds_bytes<MT>()];
  __shared__ float adapted[16 * MT][17];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i = lane & 15, G = lane >> 4;
  const int64_t m0 = 16 * MT * (int64_t)(blockIdx.x / tiles_n), n0 = skinny::BN * (int64_t)(blockIdx.x % tiles_n);
  f32x4 acc[MT];
  skinny::product<DT, MT>(a, m0, n0, lane, w, lds + w * (1 + MT) * 2048, acc, [&]() {
    // (no branch on a row's adapter: every row's loads go out together; a row without one reads
    // adapter 0's weights and its own unwritten U, and its sum is dropped)
    constexpr int ROWS = 2 * MT;
    int64_t t[ROWS];
    int id[ROWS];
    const uint16_t* lb[ROWS];
    float s[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; j++) {
      t[j] = min(m0 + w + 8 * j, a.M - 1);
      id[j] = __builtin_amdgcn_readfirstlane(lora::adapter_of(lo, m0 + w + 8 * j, a.M));
      lb[j] = (const uint16_t*)lo.LB + (int64_t)max(id[j], 0) * lo.stride_lb + min(n0 + i, a.N - 1) * lo.ld_lb + 8 * G;
      s[j] = 0.f;
    }
    for (int r = 0; r < lo.R; r += 32) {
      lora::UPart u[ROWS];
      uint4 b[ROWS];
#pragma unroll
      for (int j = 0; j < ROWS; j++) {
        b[j] = lora::load8(lb[j] + r, lo.R - r - 8 * G);
        u[j] = lora::load_u(lo.U, Rp, t[j], r, lane, true);
      }
#pragma unroll
      for (int j = 0; j < ROWS; j++) {
        float v[8];
        widen8<DT>(b[j], v);
#pragma unroll
        for (int e = 0; e < 8; e++) s[j] = __builtin_fmaf(u[j].v[e], v[e], s[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < ROWS; j++) {
      s[j] += __shfl_xor(s[j], 16);
      s[j] += __shfl_xor(s[j], 32);
      if (G == 0) adapted[w + 8 * j][i] = id[j] >= 0 ? s[j] : 0.f;
    }
  });
  skinny::join<MT>(lds, lane, w, acc);
  if (w < MT) {
#pragma unroll
    for (int e = 0; e < 4; e++) acc[0][e] += adapted[16 * w + i][4 * G + e];
    skinny::store4<DT>(a, m0 + 16 * w + i, n0 + 4 * G, acc[0]);
  }
}

// The projection's kernel, and the shrink's before it.
enum Projection { SKINNY_16, SKINNY_32, SKINNY_48, SKINNY_64, SPLIT, TILES };
enum Shrink { NO_SHRINK, ROWS, SHRINK_TILES };

Projection projection_of(const GemmArgs& a, const LoraArgs& lo) {
  if (a.M <= 64) return a.M <= 16 ? SKINNY_16 : a.M <= 32 ? SKINNY_32 : a.M <= 48 ? SKINNY_48 : SKINNY_64;
  // Beyond 64 rows still in one round of workgroups: 100 rows, N 2048, K 4096 (256) 31.1 -> 20.5 us on tiles and
  // here; at 512 (128 rows, N 4096) 31.5 and 34.9 us. With many adapters, which a tile's expand takes one after
  // another, further: 100 rows of 64 adapters 61.2 -> 20.2 us, 200 (512) 61.1 -> 33.2 us.
  const int64_t wgs = (a.M + 63) / 64 * ((a.N + skinny::BN - 1) / skinny::BN);
  if (wgs <= 256 || (lo.n >= 32 && wgs <= 768)) return SKINNY_64;
  // (fewer 128-row tiles than CUs: bsm_gemm_grouped's rule and figures)
  return (a.M + 127) / 128 * ((a.N + mid::BN - 1) / mid::BN) < 192 ? SPLIT : TILES;
}

Shrink shrink_of(const GemmArgs& a, const LoraArgs& lo) {
  if (lo.R == 0 || lo.n == 0) return NO_SHRINK;
  // Row by row while that is little work (U values / 32), tiles beyond, whichever projection follows. A row reads its
  // whole adapter, a tile its 32 rows' adapters one after another, so with many adapters rows go further. Rows
  // against tiles, whole calls (N 256, K 8192, requests of many rows): 400 rows of rank 64 (800) 61 and 62 us, 1000 of
  // rank 64 (2000) 92 and 67, of rank 128 (4000) 150 and 72; every row an adapter of its own choice, 8 adapters 1000
  // of rank 64 102 and 104, of rank 128 176 and 107; 40 adapters 1000 of rank 64 135 and 273, of rank 128 251 and
  // 280 (requests of many rows 157 and 71), 3000 of rank 128 (12000) 758 and 679 (420 and 133). Where they cross hardly
  // moves with K (512 to 8192): over 3 K, 4 ranks, 70 to 3000 rows, 1 to 40 adapters and N 256 and 2048 this choice
  // takes 2% longer than the better form of each (1.6 times at worst).
  const int64_t work = a.M * (lora::padded_rank(lo.R) / 32);
  return work <= (lo.n >= 32 ? 3000 : 1024) ? ROWS : SHRINK_TILES;
}

template <int DT>
hipError_t launch(const GemmArgs& a, const LoraArgs& lo, hipStream_t st) {
  const Projection kind = projection_of(a, lo);
  const Shrink shrink = shrink_of(a, lo);
  const int64_t Rp = lora::padded_rank(lo.R);
  const int64_t bm = kind <= SKINNY_64 ? 16 * (kind + 1) : kind == SPLIT ? 64 : 128;
  const int64_t bn = kind <= SKINNY_64 ? skinny::BN : mid::BN;
  const int64_t tm = (a.M + bm - 1) / bm, tn = (a.N + bn - 1) / bn;
  if (tm * tn > 0x7FFFFFF0) return hipErrorInvalidValue;
  if (shrink == ROWS) {
    hipLaunchKernelGGL(k_lora_shrink_rows<DT>, dim3((uint32_t)a.M, (uint32_t)(Rp / 32)), dim3(1024), 0, st, a, lo, Rp);
  } else if (shrink == SHRINK_TILES) {
    const dim3 grid((uint32_t)((a.M + 31) / 32), (uint32_t)((lo.R + 127) / 128), (uint32_t)(lo.n < 4 ? lo.n : 4));
    hipLaunchKernelGGL(k_lora_shrink<DT>, grid, dim3(256), 0, st, a, lo, Rp);
  }
  if (shrink != NO_SHRINK) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 few((uint32_t)(tm * tn)), grid((uint32_t)((tm * tn + 7) / 8 * 8));
  switch (kind) {
    case SKINNY_16: hipLaunchKernelGGL((k_lora_skinny<DT, 1>), few, dim3(skinny::THREADS), 0, st, a, lo, Rp, (int)tn); break;
    case SKINNY_32: hipLaunchKernelGGL((k_lora_skinny<DT, 2>), few, dim3(skinny::THREADS), 0, st, a, lo, Rp, (int)tn); break;
    case SKINNY_48: hipLaunchKernelGGL((k_lora_skinny<DT, 3>), few, dim3(skinny::THREADS), 0, st, a, lo, Rp, (int)tn); break;
    case SKINNY_64: hipLaunchKernelGGL((k_lora_skinny<DT, 4>), few, dim3(skinny::THREADS), 0, st, a, lo, Rp, (int)tn); break;
    case SPLIT: hipLaunchKernelGGL((k_lora<DT, 2>), grid, dim3(512), 0, st, a, lo, Rp, (int)tm, (int)tn); break;
    case TILES: hipLaunchKernelGGL((k_lora<DT, 1>), grid, dim3(256), 0, st, a, lo, Rp, (int)tm, (int)tn); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_lora(const GemmArgs& a, const LoraArgs& lo, hipStream_t st) {
  return a.dtype == BSM_BF16 ? launch<BSM_BF16>(a, lo, st) : launch<BSM_F16>(a, lo, st);
}

const char* route_gemm_lora(const GemmArgs& a, const LoraArgs& lo) {
  constexpr const char* names[] = {"k_lora_skinny<1>", "k_lora_skinny<2>", "k_lora_skinny<3>", "k_lora_skinny<4>", "k_lora<2>", "k_lora<1>"};
  return names[projection_of(a, lo)];
}
const char* route_gemm_lora_shrink(const GemmArgs& a, const LoraArgs& lo) {
  constexpr const char* names[] = {"", "k_lora_shrink_rows", "k_lora_shrink"};
  return names[shrink_of(a, lo)];
}

}  // namespace bsm
