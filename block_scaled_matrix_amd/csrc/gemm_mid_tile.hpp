// gemm_mid_tile.hpp - fp16/bf16 output tiles of 32, 64, 128 or 256 rows x 128 columns on gfx950 MFMA, for
// products with too few rows, or too few tiles, for the 256 x 256 tile of gemm_dense_tile.hpp.
//
//  - four waves in a 2 x 2 grid, each BM/2 x 64 of the tile as 16x16x32 blocks (operands swapped, so a
//    lane holds four consecutive columns of one row);
//  - K tiles of BK 64 (128-byte rows, or k-rows of 256 bytes where M or N is the contiguous axis) stream
//    HBM -> LDS by direct copies into a ring of NST stages sized so that two workgroups share a CU
//    (at most 80 KiB each): the copies of NST - 1 tiles are in flight while one is multiplied, and
//    one workgroup multiplies while the other waits;
//  - one barrier per K tile: it tells that the tile's copies have landed for every wave and that every
//    wave is done with the stage that the next copies overwrite;
//  - 256 rows need BK 32 to fit: fewer bytes through LDS and copy path per product, but K-major rows then
//    move in half lines, which cost more than that saves (16381 rows over 16 groups, N 4096, K 8192:
//    1259 us against 1188 us on 128 rows); with both operands MN-major it pays (the weight gradient of
//    16381 rows over 8 groups, M 4096, N 2048: 306 against 343 us). Raising the waves' priority
//    around the matrix instructions, or issuing the copies after the first fragment reads, was 2-6%
//    slower;
//  - LDS layouts: K-major as in gemm_common.hpp; MN-major rows of 256 bytes with chunk c of k-row kr
//    at c ^ 4(kr & 3) ^ 2((kr >> 3) & 1): the eight 32-byte pieces that a half-wave's transposing read
//    touches lie in the eight different eighths of a row, all 64 banks.
#pragma once
#include <type_traits>
#include "store16.hpp"
#include "../../include/bsm.h"

namespace bsm {
namespace mid {

constexpr int BN = 128;
constexpr int LDS_BYTES = 80 * 1024;

// An operand tile of ROWS rows (M or N) x BK K elements (64 or 32).
template <int ROWS, bool KMAJ, int BK>
struct Tile {
  static constexpr int BYTES = ROWS * BK * 2;
  static constexpr int CPR = BK / 8;            // 16-byte chunks of a row (K-major)
  static constexpr int COPIES = BYTES / 4096;   // per wave
  static constexpr int KROW = ROWS * 2;         // bytes of a k-row (MN-major)
  static constexpr int CPK = KROW / 16;         // its chunks
  static_assert(KMAJ || ROWS >= 128, "MN-major tiles are at least 128 wide");

  // chunk c of K-major row r sits at c ^ rswz(r): the 16 rows that one 16-lane group reads lie in all banks
  __device__ static int rswz(int r) { return CPR == 8 ? (r >> 1) & 7 : (r >> 2) & 3; }
  __device__ static uint32_t swz(int kr) { return (uint32_t)(4 * (kr & 3) ^ 2 * ((kr >> 3) & 1)); }

  // Per-lane byte offsets of this wave's copies from the tile's base; rows (K-major) or chunks
  // (MN-major) past the operand re-read its last ones, whose results are not stored.
  __device__ static void offsets(int64_t ld, int64_t row0, int64_t rows, int w, int lane, uint32_t (&off)[COPIES]) {
#pragma unroll
    for (int j = 0; j < COPIES; j++) {
      const int p = 64 * (w + 4 * j) + lane;    // 16-byte chunk of the tile
      if (KMAJ) {
        const int r = p / CPR, c = (p % CPR) ^ rswz(r);
        off[j] = (uint32_t)((min(row0 + r, rows - 1) - row0) * ld * 2 + 16 * c);
      } else {
        const int kr = p / CPK, c = (p % CPK) ^ (int)swz(kr);
        off[j] = (uint32_t)((kr * ld + min(row0 + 8 * c, (rows - 1) & ~int64_t(7)) - row0) * 2);
      }
    }
  }
  __device__ static const uint16_t* base(const uint16_t* p, int64_t ld, int64_t row0, int64_t k0) {
    return KMAJ ? p + row0 * ld + k0 : p + k0 * ld + row0;
  }
  // A partial K tile through registers, elements at or past `left` K elements zero.
  __device__ static void fill(const uint16_t* b, const uint32_t (&off)[COPIES], int left, uint8_t* tile, int w, int lane) {
#pragma unroll
    for (int j = 0; j < COPIES; j++) {
      const int p = 64 * (w + 4 * j) + lane;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (KMAJ) {
        const int r = p / CPR, c = (p % CPR) ^ rswz(r), n = left - 8 * c;
        if (n > 0) {
          v = *(const uint4*)((const uint8_t*)b + off[j]);
          if (n < 8) {
            uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int d = 0; d < 4; d++) wd[d] &= n >= 2 * d + 2 ? 0xFFFFFFFFu : (n == 2 * d + 1 ? 0xFFFFu : 0u);
            v = make_uint4(wd[0], wd[1], wd[2], wd[3]);
          }
        }
      } else if (p / CPK < left) {
        v = *(const uint4*)((const uint8_t*)b + off[j]);
      }
      lds_write_b128(tile + 16 * p, v);
    }
  }
  // Fragment of 16-row block at row r0 for 32-K step s: lane l holds row r0 + l%16, k 32s + 8(l/16) .. +7.
  __device__ static uint4 frag(const uint8_t* tile, int lane, int r0, int s) {
    const int G = lane >> 4, i = lane & 15;
    if (KMAJ) {
      const int r = r0 + i, c = 4 * s + G;
      return lds_read_b128(tile + r * 2 * BK + ((c ^ rswz(r)) << 4));
    }
    uint2 h[2];
#pragma unroll
    for (int q = 0; q < 2; q++) {
      const int kr = 32 * s + 8 * G + 4 * q + (i >> 2), o = 2 * r0 + 8 * (i & 3);
      h[q] = __builtin_bit_cast(uint2, lds_read_tr16(tile + kr * KROW + (((o >> 4) ^ swz(kr)) << 4) + (o & 15)));
    }
    return make_uint4(h[0].x, h[0].y, h[1].x, h[1].y);
  }
};

template <int DT>
__device__ __forceinline__ f32x4 mfma(uint4 b, uint4 a, f32x4 c) {
  if constexpr (DT == BSM_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a), c, 0, 0, 0);
}

// Stores one wave's MI x 4 blocks (rows row0 .. + 16 MI - 1, columns col0 .. + 63 of D) in D's format,
// through `region` (MI * 4 KiB of LDS): rows of 256 bytes, chunk c of row r at c ^ (r & 15), then
// whole row pieces: D = round(f(acc (+ D))), masked at D's edges. A is GemmArgs with M, N, D the product's.
template <int DT, int ALL, int M0, int MI>
__device__ __forceinline__ void store(const GemmArgs& a, int64_t row0, int64_t col0, int lane, const f32x4 (&acc)[ALL][4],
                                      uint8_t* region) {
  const int i = lane & 15, G = lane >> 4;
#pragma unroll
  for (int m = 0; m < MI; m++)
#pragma unroll
    for (int n = 0; n < 4; n++) {
      const int r = 16 * m + i, c = 4 * n + G;
      const f32x4& v = acc[M0 + m][n];
      lds_write_b128(region + 256 * r + 16 * (c ^ (r & 15)),
                     make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
    }
  if (a.d_fmt == BSM_F32) {
    // four rows of 256 bytes per step, 16 bytes a lane
#pragma unroll 4
    for (int j = 0; j < 4 * MI; j++) {
      const int r = 4 * j + G;
      const uint4 x = lds_read_b128(region + 256 * r + 16 * (i ^ (r & 15)));
      float v[4] = {__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w)};
      const int64_t row = row0 + r, col = col0 + 4 * i;
      if (row >= a.M || col >= a.N) continue;
      gemm::global_f32* p = (gemm::global_f32*)(a.D + row * a.ldd + col);
      if (col + 4 <= a.N) {
        if (a.accum) {
          const u32x4 y = *(gemm::global_u32x4*)p;
#pragma unroll
          for (int e = 0; e < 4; e++) v[e] += __uint_as_float(y[e]);
        }
        u32x4 o;
#pragma unroll
        for (int e = 0; e < 4; e++) o[e] = __float_as_uint(a.ew_op ? silu_affine(v[e], a.ew_scale, a.ew_bias) : v[e]);
        *(gemm::global_u32x4*)p = o;
      } else {
#pragma unroll
        for (int e = 0; e < 4; e++)
          if (col + e < a.N) {
            const float y = a.accum ? v[e] + p[e] : v[e];
            p[e] = a.ew_op ? silu_affine(y, a.ew_scale, a.ew_bias) : y;
          }
      }
    }
    return;
  }
  // eight rows of 128 bytes per step, 16 bytes (8 columns) a lane
#pragma unroll 2
  for (int j = 0; j < 2 * MI; j++) {
    const int r = 8 * j + (lane >> 3), c = 2 * (lane & 7);
    const uint4 x0 = lds_read_b128(region + 256 * r + 16 * (c ^ (r & 15)));
    const uint4 x1 = lds_read_b128(region + 256 * r + 16 * ((c + 1) ^ (r & 15)));
    float v[8] = {__uint_as_float(x0.x), __uint_as_float(x0.y), __uint_as_float(x0.z), __uint_as_float(x0.w),
                  __uint_as_float(x1.x), __uint_as_float(x1.y), __uint_as_float(x1.z), __uint_as_float(x1.w)};
    const int64_t row = row0 + r, col = col0 + 4 * c;
    if (row >= a.M || col >= a.N) continue;
    uint16_t* p = (uint16_t*)a.D + row * a.ldd + col;
    if (col + 8 <= a.N) {
      if (a.accum) {
        const u32x4 y = *(gemm::global_u32x4*)p;
#pragma unroll
        for (int e = 0; e < 8; e++) v[e] += gemm::from_bits16<DT>((uint16_t)(y[e >> 1] >> (16 * (e & 1))));
      }
      if (a.ew_op)
#pragma unroll
        for (int e = 0; e < 8; e++) v[e] = silu_affine(v[e], a.ew_scale, a.ew_bias);
      u32x4 o;
#pragma unroll
      for (int e = 0; e < 4; e++)
        o[e] = (uint32_t)gemm::to_bits16<DT>(v[2 * e]) | ((uint32_t)gemm::to_bits16<DT>(v[2 * e + 1]) << 16);
      *(gemm::global_u32x4*)p = o;
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (col + e < a.N) {
          float y = a.accum ? v[e] + gemm::from_bits16<DT>(p[e]) : v[e];
          if (a.ew_op) y = silu_affine(y, a.ew_scale, a.ew_bias);
          p[e] = gemm::to_bits16<DT>(y);
        }
    }
  }
}

// Nothing to add to a tile's sums before they are stored. (kStores: `more` stores them itself.)
struct NoMore {
  static constexpr bool kStores = false;
  template <int MI>
  __device__ __forceinline__ void operator()(int64_t, int64_t, f32x4 (&)[MI][4]) const {}
};

// One BM x 128 tile at (m0, n0) of the product that `a` describes (M, N, K, A, B, D its own), by four
// waves with LDS bytes of LDS. more(row0, col0, acc) may add to a wave's sums before the store.
// Q > 1: Q times four waves share the tile, wave w of part q taking every Q-th K tile from the q-th on in
// LDS of its own (part q's starts at part 0's + q * LDS); part 0 adds the sums in part order and
// stores. All waves of the workgroup come here together.
// first < the whole K tiles: the sum begins at that tile and wraps (the same for every call of the tile, so the bits stay).
// TERMS > 1: A is the sum of so many operands, each `second` elements behind the one before; their products make one sum.
template <int DT, int BM, bool AK, bool BKM, int BK = 64, class MORE = NoMore, int LDS = LDS_BYTES, int Q = 1, int TERMS = 1>
__device__ __forceinline__ void tile(const GemmArgs& a, int64_t m0, int64_t n0, uint8_t* lds, int lane, int w,
                                     const MORE& more = MORE(), int q = 0, int first = 0, int64_t second = 0) {
  typedef Tile<BM, AK, BK> TA;
  typedef Tile<BN, BKM, BK> TB;
  constexpr int MI = BM / 32, STAGE = TA::BYTES + TB::BYTES, NST = LDS / STAGE, PER = TA::COPIES + TB::COPIES;
  static_assert(NST >= 2, "stages");
  const int wa = (BM / 2) * (w >> 1), wb = 64 * (w & 1);
  const uint16_t* A = (const uint16_t*)a.A;
  const uint16_t* B = (const uint16_t*)a.B;
  uint32_t ao[TA::COPIES], bo[TB::COPIES];
  TA::offsets(a.lda, m0, a.M, w, lane, ao);
  TB::offsets(a.ldb, n0, a.N, w, lane, bo);
  f32x4 acc[MI][4];
#pragma unroll
  for (int m = 0; m < MI; m++)
#pragma unroll
    for (int n = 0; n < 4; n++) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int nfull = (int)(a.K / BK), tail = (int)(a.K % BK);
  const uint32_t lds0 = gemm::lds_addr(lds);
  // The copies of this part's it-th K tile; past the last one they re-read it into a stage that nobody
  // reads again, so that the counts waited for stay fixed.
  auto issue = [&](int it, int stage) {
    int kt = min(it * Q + q, nfull - 1) + first;
    if (kt >= nfull) kt -= nfull;
    const int64_t k0 = (int64_t)kt * BK;
    uint64_t ga, gb;
    gemm::sgpr_base2(TA::base(A, a.lda, m0, k0), TB::base(B, a.ldb, n0, k0), ga, gb);
    const uint32_t at = lds0 + stage * STAGE;
#pragma unroll
    for (int j = 0; j < TA::COPIES; j++) gemm::dma16u(ga, ao[j], at + 1024 * (w + 4 * j));
#pragma unroll
    for (int j = 0; j < TB::COPIES; j++) gemm::dma16u(gb, bo[j], at + TA::BYTES + 1024 * (w + 4 * j));
  };
  auto multiply = [&](const uint8_t* st, auto steps) {
#pragma unroll
    for (int s = 0; s < decltype(steps)::value; s++) {
      uint4 fa[MI], fb[4];
#pragma unroll
      for (int n = 0; n < 4; n++) fb[n] = TB::frag(st + TA::BYTES, lane, wb + 16 * n, s);
#pragma unroll
      for (int m = 0; m < MI; m++) fa[m] = TA::frag(st, lane, wa + 16 * m, s);
#pragma unroll
      for (int m = 0; m < MI; m++)
#pragma unroll
        for (int n = 0; n < 4; n++) acc[m][n] = mfma<DT>(fb[n], fa[m], acc[m][n]);
    }
  };
  for (int term = 0; term < TERMS; term++) {
    if (term > 0) A += second;   // (every wave is done with LDS)
    if (nfull > 0) {
#pragma unroll
      for (int i = 0; i < NST - 1; i++) issue(i, i);
      int cur = 0;
      for (int it = 0; it < (nfull + Q - 1) / Q; it++) {
        gemm::stage_barrier<(NST - 2) * PER>();
        issue(it + NST - 1, cur == 0 ? NST - 1 : cur - 1);
        if (Q == 1 || it * Q + q < nfull) multiply(lds + cur * STAGE, std::integral_constant<int, BK / 32>{});
        cur = cur + 1 == NST ? 0 : cur + 1;
      }
    }
    // every copy has landed and every wave is done with LDS (before it is refilled, before the
    // accumulators pass through it, and before the workgroup can end)
    gemm::stage_barrier<0>();
    if (tail) {
      const int64_t k0 = (int64_t)nfull * BK;
      if (q == 0) {
        TA::fill(TA::base(A, a.lda, m0, k0), ao, tail, lds, w, lane);
        TB::fill(TB::base(B, a.ldb, n0, k0), bo, tail, lds + TA::BYTES, w, lane);
      }
      __syncthreads();
      if (q == 0) {
        if (BK == 32 || tail <= 32) multiply(lds, std::integral_constant<int, 1>{});
        else multiply(lds, std::integral_constant<int, 2>{});
      }
      __syncthreads();
    }
  }
  if constexpr (Q > 1) {
    static_assert(MI * 16384 <= LDS, "joined sums");
    uint8_t* mine = lds + MI * 4096 * w + 16 * lane;
    if (q > 0) {
#pragma unroll
      for (int m = 0; m < MI; m++)
#pragma unroll
        for (int n = 0; n < 4; n++) *(BSM_LDS f32x4*)(mine + 1024 * (4 * m + n)) = acc[m][n];
    }
    __syncthreads();
    if (q > 0) return;
#pragma unroll
    for (int p = 1; p < Q; p++)
#pragma unroll
      for (int m = 0; m < MI; m++)
#pragma unroll
        for (int n = 0; n < 4; n++) acc[m][n] += *(const BSM_LDS f32x4*)(mine + p * LDS + 1024 * (4 * m + n));
  }
  more(m0 + wa, n0 + wb, acc);
  // the sums leave through LDS in parts of MC blocks of 16 rows a wave
  if constexpr (!MORE::kStores) {
    constexpr int FIT = LDS / 16384, MC = MI < FIT ? MI : (FIT >= 4 ? 4 : 2);
    static_assert(MI % MC == 0 && MC * 16384 <= LDS, "store parts");
    auto part = [&](auto m) {
      constexpr int M0 = decltype(m)::value * MC;
      if constexpr (M0 < MI) store<DT, MI, M0, MC>(a, m0 + wa + 16 * M0, n0 + wb, lane, acc, lds + MC * 4096 * w);
    };
    part(std::integral_constant<int, 0>{});
    part(std::integral_constant<int, 1>{});
  }
}

}  // namespace mid
}  // namespace bsm
