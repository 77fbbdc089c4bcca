// gemm_kept_tile.hpp - output tiles of the weight gradient D = Y^T X whose X is kept as 8-bit codes with E8M0 scales
// (kept.hpp), on gfx950 16-bit MFMA.
//
// The scales run along X's columns, the sum along its rows, so no scale can leave the sum: every code is multiplied by its
// own scale before the product. A code times its scale has at most four significant bits: as bf16 (as f16 inside that
// format's range) it is exact, and the product and its sums are those of bsm_gemm_grouped_wgrad on the restored X.
//
// Y streams HBM -> LDS by direct copies, as in the other tiles. X's codes and scale words stream the same way: half the
// bytes of 16-bit rows. Each wave takes the rows of codes that it copied itself out of LDS, converts them (eight codes a lane:
// four conversions with the scale in bf16) and writes the 16-bit k-rows that the fragments are read from. So a code
// is converted once a workgroup, where conversion at the fragment would be once a wave and need a scale per element. (Loads
// into registers instead of copies would make the compiler wait for all copies in flight: it does not count them.)
// A group's rows seldom are a multiple of a K tile. The first tile is the short one, filled through registers with zeros
// past its rows, and the others follow by copies.
#pragma once
#include <utility>
#include "gemm_dense_tile.hpp"
#include "gemm_mid_tile.hpp"
#include "kept.hpp"

namespace bsm {
namespace keptmm {

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

// Eight codes times 2^(code - 127) as the operand's 16-bit format. Finite ones beyond its range are its largest value: in f16
// by the scale, in bf16 where BOUND says so. (In bf16 that takes more operations than the conversion, and seldom a scale
// asks for it: the small tiles convert again where a wave has met one; of the 256 x 256 tile see k_gemm_kept.hip.)
template <int DT, int FMT, bool BOUND>
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
    uint32_t w[4] = {two(c0, std::false_type{}), two(c0, std::true_type{}), two(c1, std::false_type{}), two(c1, std::true_type{})};
    if constexpr (BOUND) {
      // infinities that are not the code's own: one less in their bits
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const uint32_t byte = (e < 4 ? c0 : c1) >> (8 * (e & 3)), half = w[e >> 1] >> (16 * (e & 1));
        if ((half & 0x7FFFu) == 0x7F80u && !(FMT == BSM_E5M2 && (byte & 0x7Fu) == 0x7Cu)) w[e >> 1] -= 1u << (16 * (e & 1));
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float v[8];
    const float s = kept::scale_f16<FMT>((int)code);
    kept::decode4<FMT>(c0, s, v);
    kept::decode4<FMT>(c1, s, v + 4);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; e++)
      w[e] = f32_to_f16_bits(kept::clamp_f16(v[2 * e])) | (uint32_t)f32_to_f16_bits(kept::clamp_f16(v[2 * e + 1])) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ---- 128 x 128 and 64 x 64 tiles ---------------------------------------------------------------------------------------
// Four waves, K tiles of 32 in two stages, 34 KiB of LDS (64 x 64: three, 31 KiB): four workgroups share a CU, and one converts or
// stores while another multiplies. With few tiles and long groups Q sets of four waves share a tile instead, each every Q-th K
// tile in LDS of its own; their sums meet in a fixed order.
namespace mid2 {

constexpr int BK = 32;

// BK k-rows of ROWS 16-bit values: chunk c of k-row kr at c ^ swz(kr), so that the eight 32-byte pieces that a half-wave's
// transposing read touches (k-rows 0 .. 3 and 8 .. 11 of 16) lie in all 64 banks.
template <int ROWS>
struct Tile {
  static constexpr int KROW = ROWS * 2, CPK = KROW / 16, BYTES = BK * KROW, COPIES = BYTES / 4096;
  __device__ static int swz(int kr) { return ROWS == 128 ? 4 * (kr & 3) ^ 2 * ((kr >> 3) & 1) : 2 * ((kr >> 1) & 1) + 4 * ((kr >> 3) & 1); }
  // chunk p of the tile as its k-row and column
  __device__ static int kr(int p) { return p / CPK; }
  __device__ static int col(int p) { return 8 * ((p % CPK) ^ swz(p / CPK)); }
  __device__ static uint4 frag(const uint8_t* tile, int lane, int r0) {
    const int G = lane >> 4, i = lane & 15;
    uint2 h[2];
#pragma unroll
    for (int q = 0; q < 2; q++) {
      const int k = 8 * G + 4 * q + (i >> 2), o = 2 * r0 + 8 * (i & 3);
      h[q] = __builtin_bit_cast(uint2, lds_read_tr16(tile + k * KROW + (((o >> 4) ^ swz(k)) << 4) + (o & 15)));
    }
    return make_uint4(h[0].x, h[0].y, h[1].x, h[1].y);
  }
};

constexpr int RAW = 4096, SCALES = 4 * 256;          // a K tile's codes and scale words: 1024 and 256 bytes a wave
template <int SIZE, int R>
constexpr int lds_bytes() { return R * (Tile<SIZE>::BYTES + RAW + SCALES) + Tile<SIZE>::BYTES; }
static_assert(4 * lds_bytes<128, 2>() <= 160 * 1024 && 4 * lds_bytes<64, 3>() <= 160 * 1024, "four workgroups, or four sets of waves, a CU");

// The SIZE x SIZE tile at (m0, n0) of the product that `a` describes: A is Y (K rows of M), B the codes (K rows of N bytes),
// SFB the scales (ld_sfb bytes a row); K the group's rows. All 4 Q waves of the workgroup come here; lds is the set's own,
// all the workgroup's.
template <int DT, int FMT, int SIZE, int R, int Q>
__device__ __forceinline__ void tile(const GemmArgs& a, int64_t m0, int64_t n0, uint8_t* lds, uint8_t* all, int lane, int w, int q) {
  typedef Tile<SIZE> T;
  constexpr int MI = SIZE == 128 ? 4 : 1, UNITS = SIZE / 64, GROUPS = SIZE / 8;   // a lane's units of eight codes; units a k-row
  constexpr int RAW_AT = R * T::BYTES, SCALES_AT = RAW_AT + R * RAW, WIDE_AT = SCALES_AT + R * SCALES, LDS = lds_bytes<SIZE, R>();
  const int wa = SIZE == 128 ? 64 * (w >> 1) : 16 * w, wb = SIZE == 128 ? 64 * (w & 1) : 0;
  const uint16_t* A = (const uint16_t*)a.A;
  const uint8_t* B = (const uint8_t*)a.B;
  uint32_t ao[T::COPIES];
#pragma unroll
  for (int j = 0; j < T::COPIES; j++) {
    const int p = 64 * (w + 4 * j) + lane;
    ao[j] = (uint32_t)((T::kr(p) * a.lda + min(m0 + T::col(p), (a.M - 1) & ~int64_t(7)) - m0) * 2);
  }
  // this wave copies rows 8w .. 8w + 7 of codes, 16 a lane (64 columns: the upper lanes the same again), and their scale
  // words (chunks past the operand re-read its last one; their results are not stored), and converts them: unit h of lane
  // l is row 8w + l / GROUPS + h * 64 / GROUPS, codes 8(l % GROUPS) .. + 7
  constexpr int CHUNKS = SIZE / 16;
  const uint32_t bo = (uint32_t)((8 * w + ((lane / CHUNKS) & 7)) * a.ldb + min(n0 + 16 * (lane % CHUNKS), (a.N - 1) & ~int64_t(15)) - n0);
  const uint32_t so = (uint32_t)((8 * w + (lane & 7)) * a.ld_sfb);
  const int ur = lane / GROUPS, uc = lane % GROUPS;
  const int64_t word0 = n0 / 128 * 4;                                   // the scale word of the tile's columns,
  const int byte = (int)(n0 / 32 - word0) + (uc >> 2);                  // this lane's byte of it
  f32x4 acc[MI][4];
#pragma unroll
  for (int m = 0; m < MI; m++)
#pragma unroll
    for (int n = 0; n < 4; n++) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int nt = (int)((a.K + BK - 1) / BK), head = (int)a.K - BK * (nt - 1);
  const uint32_t lds0 = gemm::lds_addr(lds);
  // (A stage number that alternates with the loop count is known to the compiler; one kept in a variable cost the
  // two-stage kernel a seventh of its time.)
  // The copies of this set's i-th tile. With two stages it is waited for whole, and there are none of the first tile nor past
  // the last; with three the counts waited for stay fixed: past the last the last again, for the first the one behind it
  // into a stage not yet used, and none where the first is the only one.
  auto issue = [&](int i, int stage) {
    int t = i * Q + q;
    if (R == 2 ? t < 1 || t >= nt : nt < 2) return;
    if (R > 2) t = min(max(t, 1), nt - 1);
    const int64_t k0 = BK * (int64_t)(t - 1) + head;
    uint64_t ga, gb;
    gemm::sgpr_base2(A + k0 * a.lda + m0, B + k0 * a.ldb + n0, ga, gb);
    const uint64_t gs = gemm::sgpr_base(a.SFB + k0 * a.ld_sfb + word0);
#pragma unroll
    for (int j = 0; j < T::COPIES; j++) gemm::dma16u(ga, ao[j], lds0 + stage * T::BYTES + 1024 * (w + 4 * j));
    gemm::dma16u(gb, bo, lds0 + RAW_AT + stage * RAW + 1024 * w);
    gemm::dma4u(gs, so, lds0 + SCALES_AT + stage * SCALES + 256 * w);
  };
  const uint32_t wide = n0 + 8 * uc < a.N ? kept::kWideScale<FMT> : 256;   // (past N the scales may be anything)
  auto put = [&](int h, uint32_t c0, uint32_t c1, uint32_t code, auto bound) {
    const int kr = 8 * w + ur + h * (64 / GROUPS);
    lds_write_b128(lds + WIDE_AT + kr * T::KROW + ((uc ^ T::swz(kr)) << 4), widen8<DT, FMT, decltype(bound)::value>(c0, c1, code));
  };
  if (q == 0 && nt > 0) {
    const int64_t col = min(n0 + 8 * uc, (a.N - 1) & ~int64_t(7));
#pragma unroll
    for (int h = 0; h < UNITS; h++) {
      const int row = 8 * w + ur + h * (64 / GROUPS);
      uint2 c = make_uint2(0, 0);
      uint32_t word = 0;
      if (row < head) {
        c = *(const uint2*)(B + row * a.ldb + col);
        word = *(const uint32_t*)(a.SFB + row * a.ld_sfb + word0);
      }
      put(h, c.x, c.y, (word >> (8 * byte)) & 255, std::true_type{});
    }
#pragma unroll
    for (int j = 0; j < T::COPIES; j++) {
      const int p = 64 * (w + 4 * j) + lane;
      lds_write_b128(lds + 16 * p, T::kr(p) < head ? *(const uint4*)((const uint8_t*)(A + m0) + ao[j]) : make_uint4(0, 0, 0, 0));
    }
  }
  issue(0, q == 0 ? R - 1 : 0);
#pragma unroll
  for (int i = 1; i < R - 1; i++) issue(i, i);
  int ring = 0;
  for (int it = 0; it < (nt + Q - 1) / Q; it++) {
    const int t = it * Q + q, st = R == 2 ? it & 1 : ring;
    // tile t has landed (the first is written), and nobody reads the one before any more
    gemm::stage_barrier<(R - 2) * (T::COPIES + 2)>();
    issue(it + R - 1, R == 2 ? st ^ 1 : ring == 0 ? R - 1 : ring - 1);
    if (t > 0 && t < nt) {
      u32x2 c[UNITS];
      uint32_t code[UNITS], top = 0;
#pragma unroll
      for (int h = 0; h < UNITS; h++) {
        const int row = ur + h * (64 / GROUPS);   // of the wave's eight
        c[h] = *(const BSM_LDS u32x2*)(lds + RAW_AT + st * RAW + 1024 * w + SIZE * row + 8 * uc);
        code[h] = (*(const BSM_LDS uint32_t*)(lds + SCALES_AT + st * SCALES + 256 * w + 4 * row) >> (8 * byte)) & 255;
        put(h, c[h][0], c[h][1], code[h], std::false_type{});
        top = max(top, code[h]);
      }
      if constexpr (DT == BSM_BF16)
        if (__builtin_expect(__any(top >= wide), 0))
#pragma unroll
          for (int h = 0; h < UNITS; h++) put(h, c[h][0], c[h][1], code[h], std::true_type{});
    }
    gemm::lds_barrier();
    if (t < nt) {
      uint4 fa[MI], fb[4];
#pragma unroll
      for (int n = 0; n < 4; n++) fb[n] = T::frag(lds + WIDE_AT, lane, wb + 16 * n);
#pragma unroll
      for (int m = 0; m < MI; m++) fa[m] = T::frag(lds + st * T::BYTES, lane, wa + 16 * m);
#pragma unroll
      for (int m = 0; m < MI; m++)
#pragma unroll
        for (int n = 0; n < 4; n++) acc[m][n] = mid::mfma<DT>(fb[n], fa[m], acc[m][n]);
    }
    ring = ring + 1 == R ? 0 : ring + 1;
  }
  gemm::stage_barrier<0>();
  if constexpr (Q > 1) {
    static_assert(MI * 16384 <= Q * LDS, "joined sums");
    uint8_t* mine = all + MI * 4096 * w + 16 * lane;
    for (int p = 1; p < Q; p++) {
      if (q == p)
#pragma unroll
        for (int m = 0; m < MI; m++)
#pragma unroll
          for (int n = 0; n < 4; n++) *(BSM_LDS f32x4*)(mine + 1024 * (4 * m + n)) = acc[m][n];
      __syncthreads();
      if (q == 0)
#pragma unroll
        for (int m = 0; m < MI; m++)
#pragma unroll
          for (int n = 0; n < 4; n++) acc[m][n] += *(const BSM_LDS f32x4*)(mine + 1024 * (4 * m + n));
      __syncthreads();
    }
    if (q > 0) return;
  }
  // the sums leave through LDS, of 128 rows in two parts
  constexpr int MC = MI == 4 ? 2 : 1;
  static_assert(MC * 16384 <= LDS, "store parts");
  mid::store<DT, MI, 0, MC>(a, m0 + wa, n0 + wb, lane, acc, lds + MC * 4096 * w);
  if constexpr (MI > MC) mid::store<DT, MI, MC, MC>(a, m0 + wa + 16 * MC, n0 + wb, lane, acc, lds + MC * 4096 * w);
}

}  // namespace mid2

// ---- 256 x 256 tiles: the dense GEMM's (gemm_dense_tile.hpp) with X's k-rows made in LDS ---------------------------------
// Four waves of 128 x 128, K tiles of 64: 112 KiB through LDS for 256 x 256 x 32 products where 256 x 128 tiles take 164 (they
// ran at 372 us where these take 335, in the same order of groups).
// Y's two stages are the dense tile's. One buffer holds X's 16-bit k-rows: its fragments are in registers by the middle of a
// K tile's first 32-K step, so between that step's barrier and the next tile's first reads the waves convert the next
// tile's codes into it, a unit of eight codes a lane every ninth MFMA slot, each wave its own copies' rows. The codes come
// through a ring of three stages, a K tile further ahead than Y, so that they are there when the conversion begins.
namespace large {

// LDS by its byte address.
template <class T>
__device__ __forceinline__ BSM_LDS T* at_lds(uint32_t address) { return (BSM_LDS T*)(uintptr_t)address; }

constexpr int BM = 256, BK = 64, COPIES = 13;               // a K tile's copies: 8 of Y, 4 of codes, 1 of scale words
constexpr int A_STAGE = BM * BK * 2, X_WIDE = BK * 256 * 2, X_RAW = BK * 256, X_SCALES = 4 * 256;
constexpr int WIDE_AT = 2 * A_STAGE, RAW_AT = WIDE_AT + X_WIDE, SCALES_AT = RAW_AT + 3 * X_RAW;
constexpr int LDS_BYTES = SCALES_AT + 3 * X_SCALES;
static_assert(LDS_BYTES >= 4 * 32768 && LDS_BYTES <= 160 * 1024, "the stores' regions");

// The 64 MFMAs of a 32-K step with their side work, as dense::mfma_step_il, the slots as constants (a loop over this much
// side work is not unrolled any more).
template <int DT, int FROM, class SIDE, int... I>
__device__ __forceinline__ void mfma_steps(const dense::Frags& f, f32x4 (&acc)[8][8], SIDE side, std::integer_sequence<int, I...>) {
  auto one = [&](auto i) {
    constexpr int mt = decltype(i)::value >> 3, nt = decltype(i)::value & 7;
    asm volatile("" : "+a"(acc[mt][nt])::"memory");
    acc[mt][nt] = dense::mfma<DT>(f.b[nt], f.a[mt], acc[mt][nt]);
    asm volatile("" : "+a"(acc[mt][nt])::"memory");
    side(std::integral_constant<int, FROM + decltype(i)::value>{});
  };
  (one(std::integral_constant<int, I>{}), ...);
}

// The lane's result: whether it has met a scale of kept::kWideScale or more (bf16 values beyond the range are infinite then).
template <int DT, int FMT>
__device__ __forceinline__ bool product(const GemmArgs& a, int64_t m0, int64_t n0, uint8_t* lds, int lane, int w, f32x4 (&acc)[8][8]) {
  using namespace dense;
  const int wa = 128 * (w >> 1), wb = 128 * (w & 1);
  const uint16_t* A = (const uint16_t*)a.A;
  const uint8_t* B = (const uint8_t*)a.B;
#pragma unroll
  for (int i = 0; i < 8; i++)
#pragma unroll
    for (int j = 0; j < 8; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // Y: copy j of wave w holds k-rows 2w + 8j and the one behind (dense::dma_offsets); the swizzle differs between even
  // and odd j alone, so two offsets and a scalar step of 16 rows make all eight. Codes: copy j holds k-rows 4(w + 4j) ..
  // + 3, 16 codes a lane. Scale words: lane l the word l%2 of the wave's row l/2 (a row's second word may lie past N's
  // scales: the first again).
  uint32_t ao[2];
  // The short tile first: behind the loop, more matrix instructions on the same accumulators made the compiler move up to
  // 700 accumulators about in every turn of it. With one tile alone the copies, whose counts stay, read the first row
  // over and over.
  const int nt = (int)((a.K + BK - 1) / BK), head = (int)a.K - BK * (nt - 1);
  const int64_t lda = nt > 1 ? a.lda : 0, ldb = nt > 1 ? a.ldb : 0, lds_row = nt > 1 ? a.ld_sfb : 0;
#pragma unroll
  for (int j = 0; j < 2; j++) {
    const int kr = 2 * (w + 4 * j) + (lane >> 5), c = (lane & 31) ^ (int)mn_swz(kr);
    ao[j] = (uint32_t)((kr * lda + min(m0 + 8 * c, (a.M - 1) & ~int64_t(7)) - m0) * 2);
  }
  const uint32_t bo = (uint32_t)((4 * w + (lane >> 4)) * ldb + min(n0 + 16 * (lane & 15), (a.N - 1) & ~int64_t(15)) - n0);
  const int r16 = (lane >> 1) & 15;
  const uint32_t so = (uint32_t)((4 * (w + 4 * (r16 >> 2)) + (r16 & 3)) * lds_row + (n0 + 128 < a.N ? 4 * (lane & 1) : 0));
  const uint32_t lds0 = gemm::lds_addr(lds);
  auto copy_a = [&](uint64_t base, int stage, int j) {
    gemm::dma16u(base + (uint64_t)((j >> 1) * 32 * lda), ao[j & 1], lds0 + stage * A_STAGE + 1024 * (w + 4 * j));
  };
  auto copy_codes = [&](uint64_t base, int slot, int j) {
    gemm::dma16u(base + (uint64_t)(16 * j * ldb), bo, lds0 + RAW_AT + slot * X_RAW + 1024 * (w + 4 * j));
  };
  auto copy_scales = [&](uint64_t base, int slot) { gemm::dma4u(base, so, lds0 + SCALES_AT + slot * X_SCALES + 256 * w); };
  // bases of tile t >= 1 (past the last: the last again, into a stage that nobody reads)
  auto row_of = [&](int t) { return (int64_t)max(BK * (min(t, nt - 1) - 1) + head, 0); };
  auto at_a = [&](int t) { return A + row_of(t) * lda + m0; };
  auto at_codes = [&](int t) { return B + row_of(t) * ldb + n0; };
  auto at_scales = [&](int t) { return a.SFB + row_of(t) * lds_row + n0 / 32; };
  // unit u = 2j + h: eight codes of k-row 4(w + 4j) + 2h + l/32 at column 8(l%32). The k-row's swizzle does not depend on
  // j, so two addresses and constant steps make all eight stores; loads are one address a stage.
  uint32_t to[2];
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const int kr = 4 * w + 2 * h + (lane >> 5);
    to[h] = lds0 + WIDE_AT + (uint32_t)(kr * 512 + (((lane & 31) ^ (int)mn_swz(kr)) << 4));
  }
  const uint32_t from = lds0 + RAW_AT + 1024 * w + 8 * lane;
  const uint32_t from_scale = lds0 + SCALES_AT + 256 * w + 8 * (lane >> 5) + ((lane & 31) >> 2);
  auto put = [&](int u, uint32_t c0, uint32_t c1, uint32_t code) {
    const uint4 x = widen8<DT, FMT, false>(c0, c1, code);
    *at_lds<u32x4>(to[u & 1] + 8192 * (u >> 1)) = u32x4{x.x, x.y, x.z, x.w};
  };
  u32x2 c;
  uint32_t code, top = 0;
  auto take = [&](int u, int slot) {
    c = *at_lds<u32x2>(from + slot * X_RAW + 4096 * (u >> 1) + 512 * (u & 1));
    code = *at_lds<uint8_t>(from_scale + slot * X_SCALES + 32 * (u >> 1) + 16 * (u & 1));
  };
  // Fragment addresses (dense::frag_addr): the swizzle depends on the lane alone and block t flips bits 5 .. 7, so one address
  // an operand makes all of them; step s and half h are constants. Taken anew every K tile (an asm that claims to change
  // it): otherwise the compiler keeps every address of both stages in registers and the accumulators move about for them.
  const int G = lane >> 4, i4 = lane & 15;
  const uint32_t sw = (uint32_t)(4 * (i4 >> 2) ^ 2 * (G & 1));
  auto frag_base = [&](int wbase) {
    return (uint32_t)((8 * G + (i4 >> 2)) * 512 + ((((wbase >> 3) + ((i4 & 3) >> 1)) ^ sw) << 4) + 8 * (i4 & 1));
  };
  const uint32_t fa = lds0 + frag_base(wa), fb = lds0 + WIDE_AT + frag_base(wb);
  auto frag = [&](uint32_t base, int s, int t) {
    uint2 h[2];
#pragma unroll
    for (int q = 0; q < 2; q++)
      h[q] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(at_lds<i16x4>((base ^ (32u * t)) + 16384 * s + 2048 * q)));
    return make_uint4(h[0].x, h[0].y, h[1].x, h[1].y);
  };
  // read r of a step's fragments, in the order of dense::read_one
  auto read = [&](uint32_t ba, uint32_t bb, int s, int r, Frags& f) {
    if (r >= 1 && r <= 8) f.b[r - 1] = frag(bb, s, r - 1);
    else f.a[r == 0 ? 0 : r - 8] = frag(ba, s, r == 0 ? 0 : r - 8);
  };
  Frags f0, f1;
  if (nt > 0) {
    auto issue_codes = [&](int t, int slot) {
      uint64_t gb, gs;
      gemm::sgpr_base2(at_codes(t), at_scales(t), gb, gs);
#pragma unroll
      for (int j = 0; j < 4; j++) copy_codes(gb, slot, j);
      copy_scales(gs, slot);
    };
    // the first tile: this wave's rows of codes and of Y
    const int64_t col = min(n0 + 8 * (lane & 31), (a.N - 1) & ~int64_t(7));
#pragma unroll
    for (int u = 0; u < 8; u++) {
      const int row = 4 * (w + 4 * (u >> 1)) + 2 * (u & 1) + (lane >> 5);
      uint2 x = make_uint2(0, 0);
      uint32_t sc = 0;
      if (row < head) {
        x = *(const uint2*)(B + row * a.ldb + col);
        sc = a.SFB[row * a.ld_sfb + col / 32];
      }
      put(u, x.x, x.y, sc);
      top = max(top, sc);
    }
    fill_tile_masked<false>(A, a.lda, m0, a.M, 0, head, lds, w, lane);
    issue_codes(1, 1);
    const uint64_t base = gemm::sgpr_base(at_a(1));
#pragma unroll
    for (int j = 0; j < 8; j++) copy_a(base, 1, j);
    issue_codes(2, 2);
    gemm::stage_barrier<COPIES>();   // the first tile is written, the codes of the next have landed
#pragma unroll
    for (int r = 0; r < 16; r++) read(fa, fb, 0, r, f0);
  }
  int slot = 0;   // tile kt's codes
  for (int kt = 0; kt < nt; kt++) {
    const int st = kt & 1, next = slot == 2 ? 0 : slot + 1;
    uint32_t ta = fa + st * A_STAGE, na = fa + (st ^ 1) * A_STAGE, tb = fb;
    asm volatile("" : "+v"(ta), "+v"(na), "+v"(tb));
    uint64_t ga, gb;
    gemm::sgpr_base2(at_a(kt + 2), at_codes(kt + 3), ga, gb);
    const uint64_t gs = gemm::sgpr_base(at_scales(kt + 3));
    auto copy = [&](int d) {
      if (d < 8) copy_a(ga, st, d);
      else if (d < 12) copy_codes(gb, slot, d - 8);
      else copy_scales(gs, slot);
    };
    // Side work by MFMA slot g, as in dense::tile_product: the second step's fragments; barrier, nobody reads this tile any
    // more; the copies of Y's tile kt + 2 and the codes of kt + 3; the codes of kt + 1 into the k-rows; barrier, Y's tile
    // kt + 1 has landed (and the codes of kt + 2); the next tile's first fragments.
    constexpr int C0 = 32, CPS = 5, V0 = 34, VPS = 9, LATER = 6, B2 = 107, G2 = 108;
    static_assert(C0 + CPS * (COPIES - 1) < B2 && V0 + 7 * VPS + LATER < B2 && G2 + 16 <= 128, "side-work schedule");
    auto side = [&](auto slot_no) {
      constexpr int g = decltype(slot_no)::value;
      if constexpr (g < C0 && g % 2 == 0) read(ta, tb, 1, g / 2, f1);
      if constexpr (g == C0 - 1) gemm::lds_barrier();
      if constexpr (g >= C0 && (g - C0) % CPS == 0 && (g - C0) / CPS < COPIES) copy((g - C0) / CPS);
      if constexpr (g >= V0 && (g - V0) % VPS == 0 && (g - V0) / VPS < 8) take((g - V0) / VPS, next);
      if constexpr (g >= V0 + LATER && (g - V0 - LATER) % VPS == 0 && (g - V0 - LATER) / VPS < 8) {
        put((g - V0 - LATER) / VPS, c[0], c[1], code);
        top = max(top, code);
      }
      if constexpr (g == B2) gemm::stage_barrier<COPIES>();
      if constexpr (g >= G2 && g - G2 < 16) read(na, tb, 0, g - G2, f0);
    };
    pin_frags(f0);
    mfma_steps<DT, 0>(f0, acc, side, std::make_integer_sequence<int, 64>{});
    pin_frags(f1);
    mfma_steps<DT, 64>(f1, acc, side, std::make_integer_sequence<int, 64>{});
    slot = next;
  }
  gemm::stage_barrier<0>();
  return top >= (n0 + 8 * (lane & 31) < a.N ? kept::kWideScale<FMT> : 256);   // (past N the scales may be anything)
}

}  // namespace large

}  // namespace keptmm
}  // namespace bsm
