// gemm_dense_tile.hpp - the 256 x 256 tile of the fp16/bf16 GEMM on gfx950 MFMA, shared by the dense
// GEMM (k_gemm_dense.hip, whose header states its design) and the products over groups of rows
// (k_gemm_grouped.hip, k_gemm_lora.hip).
#pragma once
#include "gemm_common.hpp"
#include "../../include/bsm.h"

namespace bsm {
namespace dense {

constexpr int BM = 256, BN = 256, BK = 64;
constexpr int TILE_BYTES = 256 * BK * 2;  // one operand tile: 32 KiB
constexpr int STAGE_BYTES = 2 * TILE_BYTES;
constexpr int DMA_PER_TILE = 16;          // copies per wave per K tile (8 A + 8 B)
static_assert(TILE_BYTES == gemm::kKTileBytes, "K-major tile geometry");

template <int DT>
struct Frag;
template <>
struct Frag<BSM_BF16> { typedef bf16x8 T; };
template <>
struct Frag<BSM_F16> { typedef f16x8 T; };

constexpr int STEPS = 2;     // 32-K MFMA steps per K tile

// MN-major tiles: 16-byte chunk c of k-row kr stored at c ^ mn_swz(kr).
__device__ __forceinline__ uint32_t mn_swz(int kr) { return (uint32_t)(4 * (kr & 3) ^ 2 * ((kr >> 3) & 1)); }

// LDS read addresses of the v_mfma_f32_16x16x32 operand fragments. Lane l (G = l/16, i = l%16)
// must hold operand (row wbase + 16t + i, k 32s + 8G + e), e = 0..7.
//  K-major: one ds_read_b128 of row wbase + 16t + i, logical chunk 4s + G;
//  MN-major: two ds_read_b64_tr_b16 (h = 0, 1): lane i of group G addresses k-row
//   32s + 8G + 4h + i/4, columns 16t + 4(i%4)..+3, and receives column i, k-rows +0..3.
template <bool KMAJ>
__device__ __forceinline__ uint32_t frag_addr(int lane, int wbase, int s, int t, int h) {
  const int G = lane >> 4, i = lane & 15;
  if (KMAJ) {
    const int r = wbase + 16 * t + i;
    const int c = 4 * s + G;
    return (uint32_t)(r * 128 + ((c ^ ((r >> 1) & 7)) << 4));
  } else {
    const int kr = 32 * s + 8 * G + 4 * h + (i >> 2);
    const int colb = 2 * wbase + 32 * t + 8 * (i & 3);
    const int c = colb >> 4;
    return (uint32_t)(kr * 512 + ((c ^ mn_swz(kr)) << 4) + (colb & 15));
  }
}

template <bool KMAJ>
__device__ __forceinline__ uint4 read_frag(const uint8_t* tile, int lane, int wbase, int s, int t) {
  if (KMAJ) {
    return lds_read_b128(tile + frag_addr<true>(lane, wbase, s, t, 0));
  } else {
    const uint2 lo = __builtin_bit_cast(uint2, lds_read_tr16(tile + frag_addr<false>(lane, wbase, s, t, 0)));
    const uint2 hi = __builtin_bit_cast(uint2, lds_read_tr16(tile + frag_addr<false>(lane, wbase, s, t, 1)));
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
}

// One 16x16x32 MFMA with the B fragment as the first source: lane l holds output row
// m = l%16 and, in registers 0..3, columns n = 4(l/16) + 0..3 of the block.
template <int DT>
__device__ __forceinline__ f32x4 mfma(uint4 b, uint4 a, f32x4 c) {
  typedef typename Frag<DT>::T T;
  const T bv = __builtin_bit_cast(T, b), av = __builtin_bit_cast(T, a);
  if constexpr (DT == BSM_BF16) return __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv, av, c, 0, 0, 0);
  else return __builtin_amdgcn_mfma_f32_16x16x32_f16(bv, av, c, 0, 0, 0);
}

struct Frags { uint4 a[8], b[8]; };

__device__ __forceinline__ void pin_frags(Frags& f) {
#pragma unroll
  for (int t = 0; t < 8; t++) {
    gemm::pin_frag(f.a[t]);
    gemm::pin_frag(f.b[t]);
  }
}

// Read r (0..15) of a step's fragments, in the order the step's MFMAs (row-block-major) first
// need them: A block 0, B blocks 0..7, A blocks 1..7.
template <bool AK, bool BKM>
__device__ __forceinline__ void read_one(const uint8_t* ta, const uint8_t* tb, int lane, int wa, int wb, int s, int r,
                                         Frags& f) {
  if (r >= 1 && r <= 8) f.b[r - 1] = read_frag<BKM>(tb, lane, wb, s, r - 1);
  else {
    const int t = r == 0 ? 0 : r - 8;
    f.a[t] = read_frag<AK>(ta, lane, wa, s, t);
  }
}

// The 64 MFMAs of one 32-K step, row-block-major; side(i) runs after MFMA i, so that LDS
// reads, copies and barriers issue while the matrix pipe is busy. Empty asm "rewrites" of
// each accumulator before and after its MFMA fix the order of the MFMAs and the side
// operations (all volatile) without any hardware wait.
template <int DT, typename Side>
__device__ __forceinline__ void mfma_step_il(const Frags& f, f32x4 (&acc)[8][8], Side side) {
#pragma unroll
  for (int i = 0; i < 64; i++) {
    const int mt = i >> 3, nt = i & 7;
    asm volatile("" : "+a"(acc[mt][nt])::"memory");
    acc[mt][nt] = mfma<DT>(f.b[nt], f.a[mt], acc[mt][nt]);
    asm volatile("" : "+a"(acc[mt][nt])::"memory");
    side(i);
  }
}

// Per-lane byte offsets (relative to the tile's global base) of the 8 direct LDS copies
// a wave issues for one operand tile; copy j of wave w fills LDS bytes
// [1024 (w + 4j), +1024).
//  K-major: the shared 128-byte-row layout (gemm::kmajor_dma_offsets);
//  MN-major: LDS k-row kr = 2(w+4j) + l/32 holds global k-row k0 + kr, its physical
//           chunk l%32 holds logical chunk (l%32) ^ mn_swz(kr) (columns clamped to
//           the last 8-aligned chunk).
template <bool KMAJ>
__device__ __forceinline__ void dma_offsets(int64_t ld, int64_t row0, int64_t rows, int w, int lane,
                                            uint32_t (&off)[8]) {
  if (KMAJ) {
    gemm::kmajor_dma_offsets(2 * ld, row0, rows, w, lane, off);
  } else {
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const int kr = 2 * (w + 4 * j) + (lane >> 5);
      const int c = (lane & 31) ^ (int)mn_swz(kr);
      const int64_t col = min(row0 + 8 * c, (rows - 1) & ~int64_t(7));
      off[j] = (uint32_t)((kr * ld + (col - row0)) * 2);
    }
  }
}

// Global base (wave-uniform) of the operand tile whose K range starts at k0.
template <bool KMAJ>
__device__ __forceinline__ const uint16_t* tile_base(const uint16_t* p, int64_t ld, int64_t row0, int64_t k0) {
  return KMAJ ? p + row0 * ld + k0 : p + k0 * ld + row0;
}

// The same tile for a partial K tile: through registers, elements with k >= K zeroed.
template <bool KMAJ>
__device__ __forceinline__ void fill_tile_masked(const uint16_t* __restrict__ p, int64_t ld, int64_t row0,
                                                 int64_t rows, int64_t k0, int64_t K, uint8_t* tile, int w, int lane) {
  if (KMAJ) {
    gemm::kmajor_fill_masked((const uint8_t*)p, 2 * ld, row0, rows, 2 * k0, 2 * K, tile, w, lane);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; j++) {
    const int i = w + 4 * j;
    const int kr = 2 * i + (lane >> 5);
    const int c = (lane & 31) ^ (int)mn_swz(kr);
    const int64_t col = min(row0 + 8 * c, (rows - 1) & ~int64_t(7));
    uint4 v = make_uint4(0, 0, 0, 0);
    if (k0 + kr < K) v = *(const uint4*)(p + (k0 + kr) * ld + col);
    lds_write_b128(tile + 1024 * i + 16 * lane, v);
  }
}

template <bool AK, bool BKM>
__device__ __forceinline__ void issue_stage(const uint16_t* A, int64_t lda, int64_t m0, const uint16_t* B,
                                            int64_t ldb, int64_t n0, int kt, const uint32_t (&aoff)[8],
                                            const uint32_t (&boff)[8], uint32_t stage, int w) {
  const int64_t k0 = (int64_t)kt * BK;
  gemm::issue_tile8(tile_base<AK>(A, lda, m0, k0), aoff, stage, w);
  gemm::issue_tile8(tile_base<BKM>(B, ldb, n0, k0), boff, stage + TILE_BYTES, w);
}

// D = f(s * acc (+ D)) for a 128 x 128 wave sub-tile held as 8 x 8 blocks of 16x16
// accumulators (register e of block (mt, nt) is output row 16mt + l%16, column
// 16nt + 4(l/16) + e), staged through the wave's 32 KiB LDS region in two halves of 64 rows
// (region row r keeps its 16-byte chunk c at c ^ (r & 15)) and stored as whole lines.
__device__ __forceinline__ void store_tile16(float* __restrict__ D, int64_t ldd, int64_t M, int64_t N, int64_t row0,
                                             int64_t col0, int lane, float sgn, const f32x4 (&acc)[8][8],
                                             uint8_t* region, bool add, int ew_op, float es, float eb) {
  const bool whole = row0 + 128 <= M && col0 + 128 <= N;
#pragma unroll
  for (int half = 0; half < 2; half++) {
#pragma unroll
    for (int m4 = 0; m4 < 4; m4++) {
      const int r = 16 * m4 + (lane & 15);
#pragma unroll
      for (int nt = 0; nt < 8; nt++) {
        const int c = 4 * nt + (lane >> 4);
        const f32x4& v = acc[4 * half + m4][nt];
        const uint4 x = make_uint4(__float_as_uint(sgn * v[0]), __float_as_uint(sgn * v[1]),
                                   __float_as_uint(sgn * v[2]), __float_as_uint(sgn * v[3]));
        lds_write_b128(region + 512 * r + 16 * (c ^ (r & 15)), x);
      }
    }
    const int c = lane & 31;
    const int64_t col = col0 + 4 * c;
    if (whole) {
      if (ew_op) gemm::store_half_whole<true>(D, ldd, row0 + 64 * half, col, lane, c, region, add, es, eb);
      else gemm::store_half_whole<false>(D, ldd, row0 + 64 * half, col, lane, c, region, add, es, eb);
    } else {
      for (int j = 0; j < 32; j++) {
        const int r = 2 * j + (lane >> 5);
        const uint4 x = lds_read_b128(region + 512 * r + 16 * (c ^ (r & 15)));
        const int64_t row = row0 + 64 * half + r;
        if (row < M) {
          gemm::global_f32* p = (gemm::global_f32*)(D + row * ldd + col);
          const float xv[4] = {__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w)};
#pragma unroll
          for (int e = 0; e < 4; e++)
            if (col + e < N) {
              float v = add ? xv[e] + p[e] : xv[e];
              if (ew_op) v = silu_affine(v, es, eb);
              p[e] = v;
            }
        }
      }
    }
  }
}

// The accumulators of output tile (tm, tn) of the product that `a` describes, by the whole
// workgroup (four waves, 2 * STAGE_BYTES of LDS); every wave is done with LDS on return.
template <int DT, bool AK, bool BKM>
__device__ __forceinline__ void tile_product(const GemmArgs& a, int tm, int tn, uint8_t* lds, int lane, int w,
                                             f32x4 (&acc)[8][8]) {
  const int wm = w >> 1, wn = w & 1;
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const uint16_t* A = (const uint16_t*)a.A;
  const uint16_t* B = (const uint16_t*)a.B;
  const int wa = 128 * wm, wb = 128 * wn;
#pragma unroll
  for (int i = 0; i < 8; i++)
#pragma unroll
    for (int j = 0; j < 8; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  uint32_t aoff[8], boff[8];
  dma_offsets<AK>(a.lda, m0, a.M, w, lane, aoff);
  dma_offsets<BKM>(a.ldb, n0, a.N, w, lane, boff);

  const int nfull = (int)(a.K / BK);
  const int tail = (int)(a.K % BK);
  const uint32_t lds0 = gemm::lds_addr(lds);
  Frags f0, f1;
  if (nfull > 0) {
    issue_stage<AK, BKM>(A, a.lda, m0, B, a.ldb, n0, 0, aoff, boff, lds0, w);
    issue_stage<AK, BKM>(A, a.lda, m0, B, a.ldb, n0, min(1, nfull - 1), aoff, boff, lds0 + STAGE_BYTES, w);
    gemm::stage_barrier<DMA_PER_TILE>();
#pragma unroll
    for (int r = 0; r < 16; r++) read_one<AK, BKM>(lds, lds + TILE_BYTES, lane, wa, wb, 0, r, f0);
  }
  // K tile kt lives in stage kt & 1; f0 holds its step-0 fragments when iteration kt starts.
  for (int kt = 0; kt < nfull; kt++) {
    const uint8_t* ta = lds + (kt & 1) * STAGE_BYTES;
    const uint8_t* tb = ta + TILE_BYTES;
    const uint8_t* na = lds + ((kt + 1) & 1) * STAGE_BYTES;
    const uint32_t stage = lds0 + (kt & 1) * STAGE_BYTES;
    const int64_t k2 = (int64_t)min(kt + 2, nfull - 1) * BK;
    uint64_t ga, gb;
    gemm::sgpr_base2(tile_base<AK>(A, a.lda, m0, k2), tile_base<BKM>(B, a.ldb, n0, k2), ga, gb);
    auto copy = [&](int d) {
      if (d < 8) gemm::dma16u(ga, aoff[d], stage + 1024 * (w + 4 * d));
      else gemm::dma16u(gb, boff[d - 8], stage + TILE_BYTES + 1024 * (w + 4 * (d - 8)));
    };
    // Side work by MFMA slot g (0..63 step 0, 64..127 step 1): step 1's 16 fragment reads at
    // every second slot from 0; barrier once every wave has read the stage; the 16 copies of
    // tile kt + 2, one every fifth slot; barrier once this wave's copies of tile kt + 1 have
    // landed; the next tile's step-0 reads in step 1's last slots.
    constexpr int R1S = 2, CPS = 5;
    constexpr int C0 = 16 * R1S, B2 = C0 + 15 * CPS, G2 = B2 + 1 > 64 ? B2 + 1 : 64, RS2 = (128 - G2) / 16;
    static_assert(RS2 >= 1 && G2 >= 64 && C0 <= 64, "side-work schedule");
    auto side = [&](int g) {
      if (g < C0 && g % R1S == 0) read_one<AK, BKM>(ta, tb, lane, wa, wb, 1, g / R1S, f1);
      if (g == C0 - 1) gemm::lds_barrier();
      if (g >= C0 && g <= B2 && (g - C0) % CPS == 0) copy((g - C0) / CPS);
      if (g == B2) gemm::stage_barrier<DMA_PER_TILE>();
      if (g >= G2 && (g - G2) % RS2 == 0 && (g - G2) / RS2 < 16)
        read_one<AK, BKM>(na, na + TILE_BYTES, lane, wa, wb, 0, (g - G2) / RS2, f0);
    };
    pin_frags(f0);
    mfma_step_il<DT>(f0, acc, [&](int i) { side(i); });
    pin_frags(f1);
    mfma_step_il<DT>(f1, acc, [&](int i) { side(64 + i); });
  }
  // Every copy has landed and every wave is done with LDS before the stage is refilled
  // (and before the workgroup can end with copies in flight).
  gemm::stage_barrier<0>();
  if (tail) {
    const int64_t k0 = (int64_t)nfull * BK;
    fill_tile_masked<AK>(A, a.lda, m0, a.M, k0, a.K, lds, w, lane);
    fill_tile_masked<BKM>(B, a.ldb, n0, a.N, k0, a.K, lds + TILE_BYTES, w, lane);
    __syncthreads();
    for (int s = 0; s < (tail + 31) / 32; s++) {
#pragma unroll
      for (int r = 0; r < 16; r++) read_one<AK, BKM>(lds, lds + TILE_BYTES, lane, wa, wb, s, r, f0);
      mfma_step_il<DT>(f0, acc, [](int) {});
    }
  }
  __syncthreads();
}

}  // namespace dense
}  // namespace bsm
