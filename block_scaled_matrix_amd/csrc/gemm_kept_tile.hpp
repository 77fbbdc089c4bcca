// gemm_kept_tile.hpp - output tiles of the weight gradient D = Y^T X whose X is kept as 8-bit codes with E8M0 scales
// (kept.hpp), on gfx950 16-bit MFMA: BM rows (Y's columns) x 128 columns (X's), four waves in a 2 x 2 grid.
//
// The scales run along X's columns, the sum along its rows, so no scale can leave the sum: every code is multiplied by its
// own scale before the product. A code times its scale has at most four significant bits: as bf16 (as f16 inside that
// format's range) it is exact, and the product and its sums are those of bsm_gemm_grouped_wgrad on the restored X.
//
//  - Y streams HBM -> LDS by direct copies into a ring of three stages, as in gemm_mid_tile.hpp. X's codes and scale words
//    stream the same way into a ring of their own, one K tile ahead of Y's: half the bytes of 16-bit rows through
//    HBM, the copy path and the ring;
//  - while the MFMAs work on K tile t, each wave takes the rows of codes that it copied itself for tile t + 1 out of LDS,
//    converts them (eight codes a lane: four conversions with the scale in bf16) and writes the 16-bit k-rows that the
//    fragments are read from, into the second of two buffers. Each code is converted once a workgroup, where
//    conversion at the fragment would be once a wave and need a scale per element; one barrier a K tile, as without it;
//  - K tiles of 32 rows: 256 rows x 128 columns take 79 KiB of LDS, two workgroups a CU.
#pragma once
#include "gemm_mid_tile.hpp"
#include "kept.hpp"

namespace bsm {
namespace keptmm {

constexpr int BN = 128, BK = 32;
constexpr int RAW = BK * BN, SCALES = 4 * 256;       // codes of a K tile; its scale words, 256 bytes a wave
constexpr int WIDE = BK * BN * 2;                    // the same as 16-bit k-rows
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef mid::Tile<BN, false, BK> TB;                 // their layout

template <int BM>
constexpr int a_bytes() { return BM * BK * 2; }
template <int BM>
constexpr int lds_bytes() { return 3 * (a_bytes<BM>() + RAW + SCALES) + 2 * WIDE; }

// Eight codes times 2^(code - 127) as the operand's 16-bit format.
template <int DT, int FMT>
__device__ __forceinline__ uint4 widen8(uint32_t c0, uint32_t c1, uint32_t code) {
  if constexpr (DT == BSM_BF16) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const float s = __uint_as_float(code << 23);   // (the conversion takes the exponent field: 0 is 2^-127, 255 NaN)
    auto two = [&](uint32_t c, auto hi) {
      bf16x2 v;
      if constexpr (FMT == BSM_E4M3) v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, s, decltype(hi)::value);
      else v = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c, s, decltype(hi)::value);
      return __builtin_bit_cast(uint32_t, v);
    };
    return make_uint4(two(c0, std::false_type{}), two(c0, std::true_type{}), two(c1, std::false_type{}), two(c1, std::true_type{}));
  } else {
    float v[8];
    const float s = kept::scale((int)code);
    kept::decode4<FMT>(c0, s, v);
    kept::decode4<FMT>(c1, s, v + 4);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; e++)
      w[e] = f32_to_f16_bits(kept::clamp_f16(v[2 * e])) | (uint32_t)f32_to_f16_bits(kept::clamp_f16(v[2 * e + 1])) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The tile at (m0, n0) of the product that `a` describes: A is Y (K rows of M), B the codes (K rows of N bytes), SFB the
// scales (ld_sfb bytes a row); K the group's rows. All four waves of the workgroup come here.
template <int DT, int FMT, int BM>
__device__ __forceinline__ void tile(const GemmArgs& a, int64_t m0, int64_t n0, uint8_t* lds, int lane, int w) {
  typedef mid::Tile<BM, false, BK> TA;
  constexpr int MI = BM / 32, PER = TA::COPIES + 2, RING = 3;
  uint8_t* raw = lds + RING * TA::BYTES;
  uint8_t* words = raw + RING * RAW;
  uint8_t* wide = words + RING * SCALES;
  const int wa = (BM / 2) * (w >> 1), wb = 64 * (w & 1);
  const uint16_t* A = (const uint16_t*)a.A;
  const uint8_t* B = (const uint8_t*)a.B;
  uint32_t ao[TA::COPIES];
  TA::offsets(a.lda, m0, a.M, w, lane, ao);
  // this wave copies rows 8w .. 8w + 7 of codes, 16 a lane, and their scale words (chunks past the operand re-read
  // its last one; their results are not stored), and converts them: rows 8w + l/16 and + 4, eight codes a lane
  const int cr = 8 * w + (lane >> 3);
  const uint32_t bo = (uint32_t)(cr * a.ldb + min(n0 + 16 * (lane & 7), (a.N - 1) & ~int64_t(15)) - n0);
  const uint32_t so = (uint32_t)((8 * w + (lane & 7)) * a.ld_sfb);
  const int vr = 8 * w + (lane >> 4), vc = lane & 15;
  f32x4 acc[MI][4];
#pragma unroll
  for (int m = 0; m < MI; m++)
#pragma unroll
    for (int n = 0; n < 4; n++) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int nfull = (int)(a.K / BK), tail = (int)(a.K % BK);
  const uint32_t lds0 = gemm::lds_addr(lds), raw0 = gemm::lds_addr(raw), words0 = gemm::lds_addr(words);
  // Copies of codes and scales of tile t, and of Y; past the last tile they re-read it into a stage that nobody reads
  // again, so that the counts waited for stay fixed.
  auto issue_codes = [&](int t, int slot) {
    const int64_t k0 = (int64_t)min(t, nfull - 1) * BK;
    uint64_t gb, gs;
    gemm::sgpr_base2(B + k0 * a.ldb + n0, a.SFB + k0 * a.ld_sfb + n0 / 32, gb, gs);
    gemm::dma16u(gb, bo, raw0 + slot * RAW + 1024 * w);
    gemm::dma4u(gs, so, words0 + slot * SCALES + 256 * w);
  };
  auto issue_a = [&](int t, int slot) {
    const int64_t k0 = (int64_t)min(t, nfull - 1) * BK;
    const uint64_t ga = gemm::sgpr_base(TA::base(A, a.lda, m0, k0));
#pragma unroll
    for (int j = 0; j < TA::COPIES; j++) gemm::dma16u(ga, ao[j], lds0 + slot * TA::BYTES + 1024 * (w + 4 * j));
  };
  auto put = [&](int h, uint32_t c0, uint32_t c1, uint32_t word, uint8_t* to) {
    const int kr = vr + 4 * h;
    lds_write_b128(to + kr * 256 + ((vc ^ (int)TB::swz(kr)) << 4), widen8<DT, FMT>(c0, c1, (word >> (8 * (vc >> 2))) & 255));
  };
  auto convert = [&](int slot, uint8_t* to) {
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const u32x2 c = *(const BSM_LDS u32x2*)(raw + slot * RAW + 128 * (vr + 4 * h) + 8 * vc);
      const uint32_t word = *(const BSM_LDS uint32_t*)(words + slot * SCALES + 256 * w + 4 * ((lane >> 4) + 4 * h));
      put(h, c[0], c[1], word, to);
    }
  };
  auto multiply = [&](const uint8_t* ta, const uint8_t* tb) {
    uint4 fa[MI], fb[4];
#pragma unroll
    for (int n = 0; n < 4; n++) fb[n] = TB::frag(tb, lane, wb + 16 * n, 0);
#pragma unroll
    for (int m = 0; m < MI; m++) fa[m] = TA::frag(ta, lane, wa + 16 * m, 0);
#pragma unroll
    for (int m = 0; m < MI; m++)
#pragma unroll
      for (int n = 0; n < 4; n++) acc[m][n] = mid::mfma<DT>(fb[n], fa[m], acc[m][n]);
  };
  if (nfull > 0) {
    issue_codes(0, 0);
    issue_a(0, 0);
    issue_codes(1, 1);
    issue_a(1, 1);
    issue_codes(2, 2);
    gemm::stage_barrier<2 * PER>();   // tile 0's codes
    convert(0, wide);
    int cur = 0;
    for (int t = 0; t < nfull; t++) {
      // Y of tile t and the codes of t + 1 have landed, tile t's k-rows are written, and nobody reads t - 1 any more
      gemm::stage_barrier<PER>();
      const int last = cur == 0 ? 2 : cur - 1, next = cur == 2 ? 0 : cur + 1;
      issue_a(t + 2, last);
      issue_codes(t + 3, cur);
      if (t + 1 < nfull) convert(next, wide + ((t + 1) & 1) * WIDE);
      multiply(lds + cur * TA::BYTES, wide + (t & 1) * WIDE);
      cur = next;
    }
  }
  // every copy has landed and every wave is done with LDS
  gemm::stage_barrier<0>();
  if (tail) {
    const int64_t k0 = (int64_t)nfull * BK;
    TA::fill(TA::base(A, a.lda, m0, k0), ao, tail, lds, w, lane);
    const int64_t col = min(n0 + 8 * vc, (a.N - 1) & ~int64_t(7));
#pragma unroll
    for (int h = 0; h < 2; h++) {
      uint2 c = make_uint2(0, 0);
      uint32_t word = 0;
      if (vr + 4 * h < tail) {
        const int64_t row = k0 + vr + 4 * h;
        c = *(const uint2*)(B + row * a.ldb + col);
        word = *(const uint32_t*)(a.SFB + row * a.ld_sfb + n0 / 32);
      }
      put(h, c.x, c.y, word, wide);
    }
    __syncthreads();
    multiply(lds, wide);
    __syncthreads();
  }
  // the sums leave through LDS in two parts
  constexpr int MC = MI / 2;
  static_assert(MC * 16384 <= lds_bytes<BM>(), "store parts");
  mid::store<DT, MI, 0, MC>(a, m0 + wa, n0 + wb, lane, acc, lds + MC * 4096 * w);
  mid::store<DT, MI, MC, MC>(a, m0 + wa + 16 * MC, n0 + wb, lane, acc, lds + MC * 4096 * w);
}

}  // namespace keptmm
}  // namespace bsm
