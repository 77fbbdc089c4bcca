// gemm_mid_mx_tile.hpp - block-scaled output tiles of 32, 64 or 128 rows x 128 columns on gfx950 MFMA, the
// counterpart of gemm_mid_tile.hpp (ring of direct copies, two workgroups a CU, one barrier per K tile)
// for products with few rows.
//
//  - K tiles of 128 elements (128 or 64 bytes of a row; one 32-bit scale word per row: the tile's four
//    32-K blocks); operand layouts, fragment reads and conversions are the general kernel's
//    (gemm_mx_any.hpp);
//  - 32x32 accumulators with the operands swapped, waves 2 x 2 of BM/2 x 64 (BM 32: 1 x 4 of 32 x 32);
//  - BF: exact products on the bf16 MFMA (elements times their scale converted in registers), else the
//    scaled f8f6f4 MFMA. Which one a call takes is gemm_mx_any.hpp's rule;
//  - scale words come through a ring of three groups of four K tiles (16 bytes of a row), a quarter of a
//    group with every K tile's operands, 16 rows a copy: copies of 64 rows, one word of each per K tile,
//    held the copy path for longer than the operands did (E4M3 x E2M1, 64 rows over 32 groups,
//    N = K = 4096: 65 us).
#pragma once
#include "gemm_mx_any.hpp"

namespace bsm {
namespace midmx {

constexpr int BN = 128, KT = 128;
constexpr int LDS_BYTES = 80 * 1024;

// An operand tile of ROWS rows x 128 elements of format code C.
template <int C, int ROWS>
struct Tile {
  typedef mxany::Op<C, false> P;
  static constexpr int BYTES = ROWS * P::ROW;
  static constexpr int ALL = BYTES / 1024;                  // 1 KiB copies
  static constexpr int COPIES = ALL < 4 ? 1 : ALL / 4;      // per wave (fewer than four: repeated)
  __device__ static int copy_of(int w, int j) { return (w + 4 * j) % ALL; }
  __device__ static void offsets(int64_t ld_bytes, int64_t rows, int w, int lane, uint32_t (&off)[COPIES]) {
#pragma unroll
    for (int j = 0; j < COPIES; j++) {
      const int p = 64 * copy_of(w, j) + lane, r = p / P::CPR, c = P::logical(p % P::CPR, r);
      off[j] = (uint32_t)(min((int64_t)r, rows - 1) * ld_bytes + 16 * c);
    }
  }
  // The partial last K tile, `left` bytes of each row (whole chunks), zero past them.
  __device__ static void fill(const uint8_t* base, const uint32_t (&off)[COPIES], int left, uint8_t* tile, int w, int lane) {
#pragma unroll
    for (int j = 0; j < COPIES; j++) {
      const int p = 64 * copy_of(w, j) + lane, r = p / P::CPR, c = P::logical(p % P::CPR, r);
      lds_write_b128(tile + 16 * p, 16 * c < left ? *(const uint4*)(base + off[j]) : make_uint4(0, 0, 0, 0));
    }
  }
};

// A BM x 128 tile staged in LDS as float32 (rows of 512 bytes, chunk c of row r at c ^ (r & 15)) to D
// in its format, D = round(f(x (+ D))), whole row pieces, masked at D's edges: wave w of four takes rows
// w BM/4 ...
template <int BM>
__device__ __forceinline__ void store_rows(const GemmArgs& a, int64_t m0, int64_t n0, const uint8_t* lds, int lane, int w) {
  if (a.d_fmt == BSM_F32) {
#pragma unroll 4
    for (int j = 0; j < BM / 8; j++) {
      const int r = w * (BM / 4) + 2 * j + (lane >> 5), c = lane & 31;
      const uint4 x = lds_read_b128(lds + 512 * r + 16 * (c ^ (r & 15)));
      float v[4] = {__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w)};
      const int64_t row = m0 + r, col = n0 + 4 * c;
      if (row >= a.M || col >= a.N) continue;
      gemm::global_f32* p = (gemm::global_f32*)(a.D + row * a.ldd + col);
      const bool whole = col + 4 <= a.N;
#pragma unroll
      for (int e = 0; e < 4; e++)
        if (whole || col + e < a.N) {
          if (a.accum) v[e] += p[e];
          if (a.ew_op) v[e] = silu_affine(v[e], a.ew_scale, a.ew_bias);
          if (!whole) p[e] = v[e];
        }
      if (whole) *(gemm::global_u32x4*)p = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    }
    return;
  }
#pragma unroll 2
  for (int j = 0; j < BM / 16; j++) {
    const int r = w * (BM / 4) + 4 * j + (lane >> 4), c = 2 * (lane & 15);
    const uint4 x0 = lds_read_b128(lds + 512 * r + 16 * (c ^ (r & 15)));
    const uint4 x1 = lds_read_b128(lds + 512 * r + 16 * ((c + 1) ^ (r & 15)));
    float v[8] = {__uint_as_float(x0.x), __uint_as_float(x0.y), __uint_as_float(x0.z), __uint_as_float(x0.w),
                  __uint_as_float(x1.x), __uint_as_float(x1.y), __uint_as_float(x1.z), __uint_as_float(x1.w)};
    const int64_t row = m0 + r, col = n0 + 4 * c;
    if (row >= a.M || col >= a.N) continue;
    uint16_t* p = (uint16_t*)a.D + row * a.ldd + col;
    const bool whole = col + 8 <= a.N;
#pragma unroll
    for (int e = 0; e < 8; e++)
      if (whole || col + e < a.N) {
        if (a.accum) v[e] += bf16_bits_to_f32(p[e]);
        if (a.ew_op) v[e] = silu_affine(v[e], a.ew_scale, a.ew_bias);
        if (!whole) p[e] = f32_to_bf16_bits(v[e]);
      }
    if (whole) {
      u32x4 o;
#pragma unroll
      for (int e = 0; e < 4; e++) o[e] = (uint32_t)f32_to_bf16_bits(v[2 * e]) | ((uint32_t)f32_to_bf16_bits(v[2 * e + 1]) << 16);
      *(gemm::global_u32x4*)p = o;
    }
  }
}

// One BM x 128 tile at (m0, n0) of the product that `a` describes, by four waves with LDS_BYTES of LDS.
// Q 2: eight waves share it, part q's four (LDS of their own, part 1's LDS bytes behind part 0's) taking
// the q-th half of the whole K tiles; part 0 adds the sums and stores. All waves come here together.
// `out` is `a` once more, for the store (a copy in LDS leaves the loop more SGPRs).
template <int CA, int CB, bool BF, int BM, int Q = 1, int LDS = LDS_BYTES>
__device__ __forceinline__ void tile(const GemmArgs& a, const GemmArgs& out, int64_t m0, int64_t n0, uint8_t* lds, int lane,
                                     int w, int q = 0) {
  typedef Tile<CA, BM> TA;
  typedef Tile<CB, BN> TB;
  // three scale buffers of A's 128 rows and B's 128, 16 bytes a row, then the stages
  constexpr int GROUP = 4096, RING = 3 * GROUP, STAGE = TA::BYTES + TB::BYTES;
  constexpr int FIT = (LDS - RING) / STAGE, NST = FIT < 6 ? FIT : 6, PER = TA::COPIES + TB::COPIES + 1;
  constexpr int MI = BM == 128 ? 2 : 1, NI = BM == 32 ? 1 : 2;
  static_assert(NST >= 2 && NST <= 6 && BM * 512 <= LDS, "stages");
  const int wa = BM == 32 ? 0 : (BM / 2) * (w >> 1), wb = BM == 32 ? 32 * w : 64 * (w & 1);
  const int sh = 8 * (lane >> 5);
  const int64_t lda = a.lda * TA::P::BITS / 8, ldb = a.ldb * TB::P::BITS / 8;
  // this part's whole K tiles: nfull of them from tile t0 on (none: it goes through the motions on tile 0)
  const int all = (int)(a.K / KT), share = (all + Q - 1) / Q, tail = (int)(a.K % KT);
  const int nfull = Q == 1 ? all : max(min(all - q * share, share), 0), t0 = nfull > 0 ? q * share : 0, last = max(nfull - 1, 0);
  const uint8_t* A = (const uint8_t*)a.A + m0 * lda + (int64_t)t0 * TA::P::ROW;
  const uint8_t* B = (const uint8_t*)a.B + n0 * ldb + (int64_t)t0 * TB::P::ROW;
  uint32_t ao[TA::COPIES], bo[TB::COPIES];
  TA::offsets(lda, a.M - m0, w, lane, ao);
  TB::offsets(ldb, a.N - n0, w, lane, bo);
  uint64_t sfa, sfb;
  gemm::sgpr_base2(a.SFA + m0 * a.ld_sfa + 4 * (int64_t)t0, a.SFB + n0 * a.ld_sfb + 4 * (int64_t)t0, sfa, sfb);
  f32x16 acc[MI][NI];
#pragma unroll
  for (int m = 0; m < MI; m++)
#pragma unroll
    for (int n = 0; n < NI; n++)
#pragma unroll
      for (int e = 0; e < 16; e++) acc[m][n][e] = 0.f;
  const uint32_t lds0 = gemm::lds_addr(lds);
  // Quarter q of scale group g (K tiles 4g ..), this wave's 16 rows of its 64: rows 64q + 16w .. of A's
  // 128 and B's 128, lane l moving the word at place l%4 of row l/4 (mxany::ring_word_offset). Words
  // past the last whole tile and rows past the operand repeat the last ones (unused values).
  auto quarter = [&](int g, int q) {
    const int op = q >> 1, R = 64 * (q & 1) + 16 * w + (lane >> 2);
    const int word = (lane & 3) ^ ((R >> 4) & 3) ^ ((R >> 6) & 1) ^ (op ? 2 : 0);
    const int64_t rows = op ? a.N - n0 : a.M - m0;
    const uint32_t off = (uint32_t)(min((int64_t)R, rows - 1) * (op ? a.ld_sfb : a.ld_sfa)) + 4u * (uint32_t)min(4 * g + word, last);
    gemm::dma4u(op ? sfb : sfa, off, lds0 + (g % 3) * GROUP + 2048 * op + 16 * (64 * (q & 1) + 16 * w));
  };
  // Tile kt's copies, and with them quarter (kt + 3) % 4 of scale group (kt + 3) / 4: group g comes with
  // tiles 4g - 3 .. 4g, so waiting for tile 4g's operands waits for it; its buffer was last read for tile
  // 4g - 9, before the copies of tile 4g - 3 go out (at tile 4g - 2 - NST or later, NST <= 6).
  // Past the last tile the copies repeat the last one's into a stage that nobody reads again, so
  // that the counts waited for stay fixed.
  auto issue = [&](int kt, int stage) {
    const int64_t k = min(kt, last);
    uint64_t ga, gb;
    gemm::sgpr_base2(A + k * TA::P::ROW, B + k * TB::P::ROW, ga, gb);
    const uint32_t at = lds0 + RING + stage * STAGE;
    quarter((kt + 3) >> 2, (kt + 3) & 3);
#pragma unroll
    for (int j = 0; j < TA::COPIES; j++) gemm::dma16u(ga, ao[j], at + 1024 * TA::copy_of(w, j));
#pragma unroll
    for (int j = 0; j < TB::COPIES; j++) gemm::dma16u(gb, bo[j], at + TA::BYTES + 1024 * TB::copy_of(w, j));
  };
  auto multiply = [&](int st, const uint32_t (&sa)[MI], const uint32_t (&sb)[NI]) {
    const uint8_t* ta = lds + RING + st * STAGE;
    const uint8_t* tb = ta + TA::BYTES;
    auto step = [&](auto sc) {
      constexpr int S = decltype(sc)::value;
      i32x8 fa[MI], fb[NI];
#pragma unroll
      for (int n = 0; n < NI; n++) fb[n] = mxany::read_frag<CB, false, BF>(tb, wb, n, S, lane);
#pragma unroll
      for (int m = 0; m < MI; m++) fa[m] = mxany::read_frag<CA, false, BF>(ta, wa, m, S, lane);
      if constexpr (BF) {
        const uint32_t rot = (uint32_t)(16 * S + 9 + sh) & 31u;
        uint4 pb[NI][4];
#pragma unroll
        for (int n = 0; n < NI; n++) mxany::cvt_whole<CB>(fb[n], __builtin_amdgcn_alignbit(sb[n], sb[n], rot), pb[n]);
#pragma unroll
        for (int m = 0; m < MI; m++) {
          uint4 pa[4];
          mxany::cvt_whole<CA>(fa[m], __builtin_amdgcn_alignbit(sa[m], sa[m], rot), pa);
#pragma unroll
          for (int j = 0; j < 4; j++)
#pragma unroll
            for (int n = 0; n < NI; n++) acc[m][n] = mxany::mfma_bf16(pb[n][j], pa[j], acc[m][n]);
        }
      } else {
#pragma unroll
        for (int m = 0; m < MI; m++)
#pragma unroll
          for (int n = 0; n < NI; n++)
            acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[n], fa[m], acc[m][n], CB, CA, 2 * S,
                                                                        (int)(sb[n] >> sh), 2 * S, (int)(sa[m] >> sh));
      }
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
  };
  uint32_t sa[MI], sb[NI];
  if (share > 0) {
#pragma unroll
    for (int j = 0; j < 3; j++) quarter(0, j);
#pragma unroll
    for (int i = 0; i < NST - 1; i++) issue(i, i);
    int cur = 0;
    for (int kt = 0; kt < share; kt++) {
      gemm::stage_barrier<(NST - 2) * PER>();
      issue(kt + NST - 1, cur == 0 ? NST - 1 : cur - 1);
      if (Q > 1 && kt >= nfull) continue;   // (the other part has one more; its barriers are joined)
      const uint8_t* sc = lds + ((kt >> 2) % 3) * GROUP;
#pragma unroll
      for (int m = 0; m < MI; m++) sa[m] = *(const BSM_LDS uint32_t*)(sc + mxany::ring_word_offset(0, wa + 32 * m + (lane & 31), kt & 3));
#pragma unroll
      for (int n = 0; n < NI; n++) sb[n] = *(const BSM_LDS uint32_t*)(sc + 2048 + mxany::ring_word_offset(1, wb + 32 * n + (lane & 31), kt & 3));
      multiply(cur, sa, sb);
      cur = cur + 1 == NST ? 0 : cur + 1;
    }
  }
  gemm::stage_barrier<0>();
  if (tail) {
    const int64_t kt = all - t0;            // (from this part's bases)
    if (q == 0) {
      TA::fill(A + kt * TA::P::ROW, ao, tail * TA::P::BITS / 8, lds + RING, w, lane);
      TB::fill(B + kt * TB::P::ROW, bo, tail * TB::P::BITS / 8, lds + RING + TA::BYTES, w, lane);
      // (each lane reads its rows' words itself: once per tile)
#pragma unroll
      for (int m = 0; m < MI; m++)
        sa[m] = mxany::mask_scale_word(mxany::load_scale_word(a.SFA, a.ld_sfa, m0, a.M, wa + 32 * m + (lane & 31), all), all, a.K / 32);
#pragma unroll
      for (int n = 0; n < NI; n++)
        sb[n] = mxany::mask_scale_word(mxany::load_scale_word(a.SFB, a.ld_sfb, n0, a.N, wb + 32 * n + (lane & 31), all), all, a.K / 32);
    }
    __syncthreads();
    if (q == 0) multiply(0, sa, sb);
    __syncthreads();
  }
  if constexpr (Q > 1) {
    uint8_t* mine = lds + MI * NI * 4096 * w + 16 * lane;
    static_assert(MI * NI * 16384 <= LDS, "joined sums");
    if (q > 0) {
#pragma unroll
      for (int m = 0; m < MI; m++)
#pragma unroll
        for (int n = 0; n < NI; n++)
#pragma unroll
          for (int e = 0; e < 4; e++)
            *(BSM_LDS f32x4*)(mine + 1024 * (4 * (NI * m + n) + e)) =
                f32x4{acc[m][n][4 * e], acc[m][n][4 * e + 1], acc[m][n][4 * e + 2], acc[m][n][4 * e + 3]};
    }
    __syncthreads();
    if (q == 0) {
#pragma unroll
      for (int m = 0; m < MI; m++)
#pragma unroll
        for (int n = 0; n < NI; n++)
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const f32x4 v = *(const BSM_LDS f32x4*)(mine + LDS + 1024 * (4 * (NI * m + n) + e));
#pragma unroll
            for (int u = 0; u < 4; u++) acc[m][n][4 * e + u] += v[u];
          }
    }
  }
  // register 4e + u of a block is row l%32, column 8e + 4(l/32) + u
  if (q == 0) {
#pragma unroll
    for (int m = 0; m < MI; m++)
#pragma unroll
      for (int n = 0; n < NI; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
        const int r = wa + 32 * m + (lane & 31), c = wb / 4 + 8 * n + 2 * e + (lane >> 5);
        const f32x16& v = acc[m][n];
        lds_write_b128(lds + 512 * r + 16 * (c ^ (r & 15)),
                       make_uint4(__float_as_uint(v[4 * e]), __float_as_uint(v[4 * e + 1]), __float_as_uint(v[4 * e + 2]),
                                  __float_as_uint(v[4 * e + 3])));
      }
  }
  __syncthreads();
  if (q == 0) store_rows<BM>(out, m0, n0, lds, lane, w);
}

}  // namespace midmx
}  // namespace bsm
