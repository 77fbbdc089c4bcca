// k_gemm_xent.hip - softmax cross entropy of a projection onto a large vocabulary, without keeping the logits.
//
//   z = X W^T (rows x N),  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t,label
//   G_tv = (exp(z_tv - lse_t) - [v = label_t]) dloss_t,  dX = G W,  dW = G^T X
//
// Loss: the GEMM tiles' accumulators hold the logits; each wave reduces its block to a pair per row (xent.hpp) and the
// logits end there: rows x N / 64 pairs leave the chip instead of rows x N logits. A second launch joins a row's
// pairs in a fixed order.
// Gradient: the vocabulary is cut into pieces. A piece's logits are made again (2 rows N K operations more than an
// implementation that had kept them), become G in the accumulators and leave as 16-bit values, which two products then read:
// dX += G W_piece and dW_piece = G^T X. So nothing of rows x N lives between the two calls, and how much lives in the second
// is the piece's choice: of the default piece no less than float32 logits would be (8190 x 32001: 1.32 GB with room for every
// format, the logits 1.05 GB), of one of 4096 columns an eighth.
// G is rounded to the operands' format because the matrix unit takes it so: half a step (2^-8 in bf16, 2^-11 in f16) of
// each term, independent from term to term, like the rounding of a 16-bit gradient. A gradient kept in float32 takes G as a
// sum of such values, three in bf16, which are all of a float's bits, and two in f16 (2^-23 left), and as often the product's
// operations. (Two in bf16 leave 2^-17: 2.5e-6 of dW's norm where float32 products have 3e-7.) In f16 the weights are
// brought to 2^15 at most by a power of two found on the device, so a probability keeps all its bits down to 2^-29 of the
// largest weight, and the products' sums are scaled back in float32.
// Tiles: gemm_dense_tile.hpp (256 x 256) where they fill the chip, gemm_mid_tile.hpp (32 / 64 / 128 x 128) otherwise, and
// for the loss of few rows skinny.hpp. dX with few tiles is cut along the vocabulary into parts that are summed in a
// fixed order; with few rows both gradients share a launch (k_xent_both).
#include <algorithm>
#include "gemm_dense_tile.hpp"
#include "gemm_mid_tile.hpp"
#include "skinny.hpp"
#include "store_large.hpp"
#include "xent.hpp"

namespace bsm {
namespace {

using namespace dense;

// A product's K cut into n parts side by side: part p takes K elements p * per .. and writes its own sums, stride_d
// elements behind part p - 1's. With several terms of A, `second` elements apart, the first n / terms parts take the first, and
// so on. Makes `a` the part's product and pid the tile's number in it.
struct Parts {
  int n, terms;
  int64_t per, stride_d, second;
  template <bool AK, bool BKM>
  __device__ __forceinline__ void enter(GemmArgs& a, int tiles, int& pid) const {
    if (n == 1) return;
    int p = pid / tiles;
    pid -= p * tiles;
    a.D += p * stride_d;
    if (terms > 1) {
      const int of = n / terms, t = p / of;
      a.A = (const uint16_t*)a.A + t * second;
      p -= t * of;
    }
    const int64_t k0 = p * per;
    a.A = (const uint16_t*)a.A + (AK ? k0 : k0 * a.lda);
    a.B = (const uint16_t*)a.B + (BKM ? k0 : k0 * a.ldb);
    a.K = min(per, a.K - k0);
  }
};

// One 256 x 256 tile: the product, what EP makes of the sums, and their store in OUT unless EP keeps none.
template <int DT, bool AK, bool BKM, int OUT, Add ADD, class EP>
__global__ __launch_bounds__(256, 1) void k_xent_large(GemmArgs a, EP ep, int tiles_m, int tiles_n, Parts parts) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * STAGE_BYTES];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tm, tn, pid = blockIdx.x;
  parts.enter<AK, BKM>(a, tiles_m * tiles_n, pid);
  gemm::tile_coords(pid, tiles_m, tiles_n, tm, tn);
  f32x4 acc[8][8];
  tile_product<DT, AK, BKM>(a, tm, tn, lds, lane, w, acc);
  const int64_t row0 = (int64_t)tm * BM + 128 * (w >> 1), col0 = (int64_t)tn * BN + 128 * (w & 1);
  ep(row0, col0, acc);
  if constexpr (!EP::kStores) store_large<OUT, ADD>(a, row0, col0, lane, acc, lds + 32768 * w);
}

// Tiles of BM x 128 (128-row ones with a K-major A: of as few rows as hold the last ones). TERMS > 1: A's terms in one sum.
template <int DT, bool AK, bool BKM, class EP, int BM = 128, int BK = 64, int PER_CU = 2, int Q = 1, int TERMS = 1>
__global__ __launch_bounds__(256 * Q, PER_CU * Q) void k_xent_mid(GemmArgs a, EP ep, int tiles_m, int tiles_n, Parts parts) {
  constexpr int LDS = 160 * 1024 / PER_CU / Q;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Q * LDS];
  const int lane = threadIdx.x & 63, wq = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wq & 3, q = wq >> 2;
  int tm, tn, pid = blockIdx.x;
  parts.enter<AK, BKM>(a, tiles_m * tiles_n, pid);
  gemm::tile_coords(pid, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = BM * (int64_t)tm, n0 = mid::BN * (int64_t)tn;
  uint8_t* mine = lds + q * LDS;
  // Rows of W a power of two apart: workgroups that all begin at K 0 read the same few memory channels. Each column tile
  // begins its sum elsewhere (24 rows x 50021 columns, K 4096: 99 -> 79 us, 64 x 32768: 66 -> 50 us).
  int first = 0;
  if constexpr (BKM) {
    const uint32_t full = (uint32_t)(a.K / BK);
    if (full > 0) first = (int)((uint32_t)(3 * tn) % full);
  }
  if constexpr (AK && BM == 128) {
    const int64_t left = a.M - m0;
    if (left <= 32) return mid::tile<DT, 32, AK, BKM, BK, EP, LDS, Q>(a, m0, n0, mine, lane, w, ep, q, first);
    if (left <= 64) return mid::tile<DT, 64, AK, BKM, BK, EP, LDS, Q>(a, m0, n0, mine, lane, w, ep, q, first);
  }
  mid::tile<DT, BM, AK, BKM, BK, EP, LDS, Q, TERMS>(a, m0, n0, mine, lane, w, ep, q, first, parts.second);
}

// Both gradients of a piece in one launch, for few rows: dX's tiles and parts, then dW's, all of 128 x 128 with K tiles of 32,
// four workgroups a CU. Neither fills the chip for long, and they need nothing of one another (one after the other and
// together, float32 dW: 200 rows x 10007, K 1000 39 and 27 us, 800 rows 79 and 77; 200 x 32000, K 2048 154 and 139; 16-bit dW:
// 1500 x 4000, K 512 44 and 29 us, 500 x 20000, K 1024 69 and 61).
template <int DT, int W_TERMS, class EP>
__global__ __launch_bounds__(256, 4) void k_xent_both(GemmArgs x, GemmArgs y, EP ep, Parts parts, int x_m, int x_n, int y_m, int y_n, int x_grid,
                                                      int64_t y_second) {
  constexpr int LDS = 40 * 1024;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[LDS];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tm, tn, pid = blockIdx.x;
  if (pid < x_grid) {
    if (pid >= x_m * x_n * parts.n) return;   // (x_grid is a multiple of 8, so that dW's tiles keep their XCDs)
    parts.enter<true, false>(x, x_m * x_n, pid);
    gemm::tile_coords(pid, x_m, x_n, tm, tn);
    mid::tile<DT, 128, true, false, 32, EP, LDS>(x, 128 * (int64_t)tm, mid::BN * (int64_t)tn, lds, lane, w, ep);
  } else {
    gemm::tile_coords(pid - x_grid, y_m, y_n, tm, tn);
    mid::tile<DT, 128, false, false, 32, EP, LDS, 1, W_TERMS>(y, 128 * (int64_t)tm, mid::BN * (int64_t)tn, lds, lane, w, ep, 0, 0, y_second);
  }
}

// The loss of up to 64 rows: 16 columns a workgroup, its eight waves splitting K (skinny.hpp).
template <int DT, int MT>
__global__ __launch_bounds__(skinny::THREADS, MT == 1 ? 4 : 2) void k_xent_skinny(GemmArgs a, xent::Stats ep) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[skinny::lds_bytes<MT>()];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = skinny::BN * (int64_t)blockIdx.x;
  f32x4 acc[MT];
  skinny::product<DT, MT>(a, 0, n0, lane, w, lds + w * (1 + MT) * 2048, acc, []() {});
  skinny::join<MT>(lds, lane, w, acc);
  if (w < MT) {
    f32x4 one[1][1] = {{acc[0]}};
    ep(16 * w, n0, one);
  }
}

// A row's pairs (b, s) joined: lse = log sum s 2^b. 16 rows a workgroup, 64 lanes a row, each every 64th slot; then the
// lanes meet in a fixed order. Everything is relative to exponents of base 2^(1/log2 e as float), so the last step, in
// double, divides by that float.
__global__ __launch_bounds__(1024) void k_xent_join(XentArgs a, const float2* part, const float* at, int slots) {
  __shared__ float2 meet[16][16];
  const int t = threadIdx.x, r = t & 15, q = t >> 4;
  const int64_t row = 16 * (int64_t)blockIdx.x + r;
  float m = -INFINITY, s = 0.0f;
  auto add = [&](float b, float v) {
    const float top = fmaxf(m, b);
    const float z = top == -INFINITY ? 0.0f : top;   // (nothing but -infinity so far; NaN comes with its s)
    s = s * __builtin_amdgcn_exp2f(m - z) + v * __builtin_amdgcn_exp2f(b - z);
    m = top;
  };
  if (row < a.rows) {
#pragma unroll 4
    for (int i = q; i < slots; i += 64) {
      const float2 p = part[i * a.rows + row];
      add(p.x, p.y);
    }
  }
#pragma unroll
  for (int d = 16; d < 64; d *= 2) {
    const float b = __shfl_xor(m, d), v = __shfl_xor(s, d);
    add(b, v);
  }
  if ((t & 63) < 16) meet[t >> 6][r] = make_float2(m, s);
  __syncthreads();
  if (t < 16 && row < a.rows) {
    m = -INFINITY;
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; w++) add(meet[w][r].x, meet[w][r].y);
    const double lse = ((double)m + (double)__builtin_amdgcn_logf(s)) / (double)xent::kLog2e;
    const int64_t lab = a.labels[row];
    a.lse[row] = (float)lse;
    a.loss[row] = lab >= 0 && lab < a.N ? (float)(lse - (double)at[row]) : 0.0f;
  }
}

// f16: by[0] = 2^15 / s on the weights before they are rounded, by[1] = s / 2^15 on the sums, s the smallest power of two
// that no finite weight of a row with a label exceeds.
__global__ __launch_bounds__(1024) void k_xent_range(XentArgs a, const float* dloss, float* by) {
  __shared__ float meet[16];
  float top = 0.0f;
  for (int64_t i = threadIdx.x; i < a.rows; i += 1024) {
    const float d = __builtin_fabsf(dloss[i]);
    const int32_t lab = a.labels[i];
    if (lab >= 0 && lab < a.N && d < INFINITY) top = fmaxf(top, d);
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
  if ((threadIdx.x & 63) == 0) meet[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 16; w++) top = fmaxf(top, meet[w]);
    const uint32_t bits = __float_as_uint(top);
    // exponent of s: top <= 2^e; kept where 2^15 / s and s / 2^15 are normal
    int e = (int)(bits >> 23) - 127 + ((bits & 0x7FFFFFu) ? 1 : 0);
    e = top == 0.0f ? 0 : max(e, -110);
    by[0] = __uint_as_float((uint32_t)(127 + 15 - e) << 23);
    by[1] = __uint_as_float((uint32_t)(127 - 15 + e) << 23);
  }
}

// dX from its float32 parts: four columns a lane, the parts dealt to four lanes (64 apart) that meet in a fixed order.
template <int OUT>
__global__ __launch_bounds__(256) void k_xent_sum(const float* F, int parts, int64_t stride, int64_t ldf, int64_t rows, int64_t K,
                                                  void* D, int64_t ldd) {
  __shared__ f32x4 meet[256];
  const int t = threadIdx.x, s = t >> 6;
  const int64_t per = (K + 3) / 4, i = blockIdx.x * (int64_t)64 + (t & 63);
  const bool in = i < rows * per;
  const int64_t row = in ? i / per : 0, col = in ? 4 * (i - row * per) : 0;
  const float* p = F + row * ldf + col;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int q = s; q < parts; q += 4) v += *(const f32x4*)(p + q * stride);
  meet[t] = v;
  __syncthreads();
  if (s > 0 || !in) return;
  v += meet[t + 64];
  v += meet[t + 128];
  v += meet[t + 192];
#pragma unroll
  for (int e = 0; e < 4; e++)
    if (col + e < K) {
      if constexpr (OUT == BSM_F32) ((float*)D)[row * ldd + col + e] = v[e];
      else ((uint16_t*)D)[row * ldd + col + e] = gemm::to_bits16<OUT>(v[e]);
    }
}

// Share of the chip's time that the product's own operations take, with tm x tn tiles of `area` elements, `slots` of them
// at a time.
double filled(int64_t M, int64_t N, int64_t tm, int64_t tn, int64_t area, int64_t slots) {
  const int64_t rounds = (tm * tn + slots - 1) / slots;
  return (double)M * N / ((double)rounds * slots * area);
}

enum Tile { SKINNY, FEW, SPLIT, MID, LARGE };

// The tiles of M x N logits. Losses, K 1000 / 2048 / 4096, in us:
//  - sixteen columns a workgroup (loss only) for up to 64 rows while 128-column tiles leave half the CUs without one;
//  - 64-row tiles whose K two sets of four waves share, while they fit the CUs at once: 100 x 4000 13.4 / 18.0 / 25.3
//    against 19.1 / 26.4 / 43.0 on 128-row tiles; in a second round (200 x 10007) 31.4 / 37.6 / 66.4 against 23.1 / 28.3 /
//    47.6;
//  - up to 32 rows 32-row tiles, three workgroups a CU: 24 x 50021 28.2 / 44.0 / 74.8 against 29.8 / 47.8 / 78.9 on two;
//  - 256 x 256 where their rounds over the CUs are as full as those of the smaller tiles, which run at 0.85 of their rate.
Tile tile_for(int64_t M, int64_t N) {
  const int64_t m128 = (M + 127) / 128, n128 = (N + 127) / 128, m256 = (M + 255) / 256, n256 = (N + 255) / 256;
  if (M <= 64 && n128 < 128) return SKINNY;
  if ((M + 63) / 64 * n128 <= 256) return SPLIT;
  if (M <= 32) return FEW;
  return filled(M, N, m256, n256, 65536, 256) >= 0.85 * filled(M, N, m128, n128, 16384, 512) ? LARGE : MID;
}

int slot_width(Tile t) { return t == SKINNY ? 16 : t == LARGE ? 128 : 64; }
int64_t slots_of(int64_t rows, int64_t N) {
  const int w = slot_width(tile_for(rows, N));
  return (N + w - 1) / w;
}

// z = X W_piece^T for `cols` columns from `first` on, into EP.
template <int DT, class EP>
void launch_logits(const GemmArgs& g, Tile tile, const EP& ep, hipStream_t st) {
  const int64_t t = tile == LARGE ? 256 : 128, tm = (g.M + t - 1) / t, tn = (g.N + t - 1) / t;   // (FEW: one row of tiles)
  const dim3 grid((uint32_t)(tm * tn));
  const Parts one{1, 1, 0, 0, 0};
  if (tile == LARGE) hipLaunchKernelGGL((k_xent_large<DT, true, true, DT, NEVER, EP>), grid, dim3(256), 0, st, g, ep, (int)tm, (int)tn, one);
  else if (tile == FEW) hipLaunchKernelGGL((k_xent_mid<DT, true, true, EP, 32, 64, 3>), grid, dim3(256), 0, st, g, ep, (int)tm, (int)tn, one);
  else if (tile == MID) hipLaunchKernelGGL((k_xent_mid<DT, true, true, EP>), grid, dim3(256), 0, st, g, ep, (int)tm, (int)tn, one);
  else {
    const int64_t m64 = (g.M + 63) / 64;
    hipLaunchKernelGGL((k_xent_mid<DT, true, true, EP, 64, 64, 1, 2>), dim3((uint32_t)(m64 * tn)), dim3(512), 0, st, g, ep, (int)m64,
                       (int)tn, one);
  }
}

// A gradient's product on 256 x 256 tiles, B's rows along K, stored in the format of `g`.
template <int DT, bool AK, class EP>
void launch_large(const GemmArgs& g, const EP& ep, const Parts& parts, hipStream_t st) {
  const int64_t tm = (g.M + 255) / 256, tn = (g.N + 255) / 256;
  auto go = [&](auto out, auto add) {
    hipLaunchKernelGGL((k_xent_large<DT, AK, false, decltype(out)::value, decltype(add)::value, EP>), dim3((uint32_t)(tm * tn * parts.n)),
                       dim3(256), 0, st, g, ep, (int)tm, (int)tn, parts);
  };
  using std::integral_constant;
  // (a 16-bit dX is never added to)
  if (g.d_fmt != BSM_F32) go(integral_constant<int, DT>{}, integral_constant<Add, AK ? NEVER : ASK>{});
  else if (g.accum) go(integral_constant<int, BSM_F32>{}, integral_constant<Add, ALWAYS>{});
  else go(integral_constant<int, BSM_F32>{}, integral_constant<Add, NEVER>{});
}

GemmArgs logits_of(const XentArgs& a) {
  GemmArgs g{};
  g.M = a.rows; g.N = a.N; g.K = a.K; g.dtype = a.dtype;
  g.A = a.X; g.lda = a.ldx; g.B = a.W; g.ldb = a.ldw;
  return g;
}

template <int DT>
hipError_t launch_loss(const XentArgs& a, float2* part, float* at, hipStream_t st) {
  const Tile tile = tile_for(a.rows, a.N);
  const GemmArgs g = logits_of(a);
  const xent::Stats ep{a.labels, part, at, a.rows, a.N, slot_width(tile)};
  if (tile == SKINNY) {
    const dim3 grid((uint32_t)((a.N + skinny::BN - 1) / skinny::BN));
    if (a.rows <= 16) hipLaunchKernelGGL((k_xent_skinny<DT, 1>), grid, dim3(skinny::THREADS), 0, st, g, ep);
    else if (a.rows <= 32) hipLaunchKernelGGL((k_xent_skinny<DT, 2>), grid, dim3(skinny::THREADS), 0, st, g, ep);
    else hipLaunchKernelGGL((k_xent_skinny<DT, 4>), grid, dim3(skinny::THREADS), 0, st, g, ep);
  } else {
    launch_logits<DT>(g, tile, ep, st);
  }
  hipLaunchKernelGGL(k_xent_join, dim3((uint32_t)((a.rows + 15) / 16)), dim3(1024), 0, st, a, part, at, (int)slots_of(a.rows, a.N));
  return hipGetLastError();
}

// How a gradient is made: `piece` columns at a time, dX on `large` tiles or 128-row ones, in `parts` parts of a piece's
// columns.
struct Plan {
  int64_t piece, pieces, ldg, ldf;
  bool large;
  int parts;
  int64_t per;      // columns of a part
  int64_t g_second;             // elements from a term of G to the next
  int64_t g_bytes, f_bytes, bytes;
};

// Terms of G for gradients kept in float32.
constexpr int f32_terms(int dt) { return dt == BSM_BF16 ? 3 : 2; }

// One piece takes what 1 GiB of G holds (two terms: 2 GiB; three: 1 GiB of them all, so that the workspace need not be larger
// for them): more pieces cost dX its sums' way through memory once a piece.
constexpr int64_t kPieceBytes = int64_t(1) << 30;

// dX has rows x K outputs and a sum over the whole piece: few tiles, long sums. Its tiles and parts are those of the least
// expected time: rounds over the chip, each a part's products at the tile's rate (5.0 TFLOP/s a workgroup of 256 x 256, one a
// CU; 1.86 of 128 x 128, two a CU) and a tile's fixed time (5 and 4 us: first loads, the sums' store), and the float32
// parts' way through memory, at 5 TB/s, and their sum's launch. (3000 rows x 32000, K 2048: one part of 128-row tiles, 496
// us, fills 384 of 512 places.)
void plan_dx(int64_t rows, int64_t K, Plan& p) {
  double best = 0.0;
  for (int large = 0; large < 2; large++) {
    const int64_t t = large ? 256 : 128, tiles = ((rows + t - 1) / t) * ((K + t - 1) / t), slots = large ? 256 : 512;
    const double rate = large ? 5.0e6 : 1.86e6, fixed = large ? 5.0 : 4.0;   // (operations a us)
    for (int64_t parts = 1; parts <= 32 && (parts == 1 || p.piece / parts >= 256); parts++) {
      const int64_t per = ((p.piece + parts - 1) / parts + 63) / 64 * 64, n = (p.piece + per - 1) / per;
      const double rounds = (double)((tiles * n + slots - 1) / slots);
      double us = p.pieces * rounds * (2.0 * t * t * per / rate + fixed);
      if (n > 1 || p.pieces > 1) us += 4.0 + 8.0 * n * p.pieces * rows * K / 5.0e6;
      if (best == 0.0 || us < best) {
        best = us;
        p.large = large;
        p.parts = (int)n;
        p.per = per;
      }
    }
  }
}

Plan plan_of(int64_t rows, int64_t N, int64_t K, int64_t piece, int terms) {
  Plan p{};
  if (piece <= 0) piece = std::max<int64_t>(kPieceBytes / ((terms == 3 ? 6 : 2) * std::max<int64_t>(rows, 1)), 4096);
  piece = std::min(piece, int64_t(1) << 21);   // (G's rows: 32-bit offsets in a tile)
  p.pieces = (N + piece - 1) / piece;
  const int64_t even = (N + p.pieces - 1) / p.pieces;            // pieces of one length
  p.piece = std::min<int64_t>((even + 255) / 256 * 256, N);
  p.pieces = (N + p.piece - 1) / p.piece;
  p.ldg = (p.piece + 63) / 64 * 64;
  plan_dx(std::max<int64_t>(rows, 1), std::max<int64_t>(K, 1), p);
  p.ldf = (K + 3) / 4 * 4;
  p.g_second = (rows * p.ldg + 127) / 128 * 128;
  p.g_bytes = terms * p.g_second * 2;
  p.f_bytes = (terms * p.parts * rows * p.ldf * 4 + 255) / 256 * 256;
  p.bytes = 256 + p.g_bytes + p.f_bytes;
  return p;
}

int terms_of(const XentGradArgs& g, int dt) {
  return (g.dX && g.dx_fmt == BSM_F32) || (g.dW && g.dw_fmt == BSM_F32) ? f32_terms(dt) : 1;
}

template <int DT>
hipError_t launch_grad(const XentArgs& a, const XentGradArgs& g, const Plan& p, uint8_t* workspace, hipStream_t st) {
  float* by = (float*)workspace;
  uint16_t* G = (uint16_t*)(workspace + 256);
  float* F = (float*)(workspace + 256 + p.g_bytes);
  const float* up = nullptr;
  const float* down = nullptr;
  if (DT == BSM_F16 && a.rows > 0) {
    hipLaunchKernelGGL(k_xent_range, dim3(1), dim3(1024), 0, st, a, g.dloss, by);
    up = by;
    down = by + 1;
  }
  using Times = xent::Times<DT == BSM_F16>;
  const Parts one{1, 1, 0, 0, 0};
  // float32 gradients take G as several terms: dX in as many times the parts, dW's in one sum
  constexpr int TERMS = f32_terms(DT);
  const bool more = terms_of(g, DT) > 1;
  const int dx_terms = g.dx_fmt == BSM_F32 ? TERMS : 1;
  const bool direct = dx_terms == 1 && p.parts == 1 && p.pieces == 1;
  for (int64_t c0 = 0, at = 0; c0 < a.N; c0 += p.piece, at++) {
    const int64_t cols = std::min(p.piece, a.N - c0);
    const uint16_t* W = (const uint16_t*)a.W + c0 * a.ldw;
    if (a.rows > 0) {
      GemmArgs z = logits_of(a);
      z.N = cols; z.B = W;
      z.D = (float*)G; z.ldd = p.ldg; z.d_fmt = DT;
      Tile tile = tile_for(a.rows, cols);
      if (tile == SKINNY) tile = SPLIT;   // (fewer than 128 tiles)
      const xent::Weights weights{a.labels, a.lse, g.dloss, up, a.rows, a.N, c0};
      if (more) launch_logits<DT>(z, tile, xent::GradTerms<DT, TERMS>{weights, G, p.ldg, p.g_second, cols}, st);
      else launch_logits<DT>(z, tile, xent::Grad{weights}, st);
    }
    GemmArgs x{}, w{};
    const Times ep{down};
    // (the last piece may be short: parts past its columns have nothing to add)
    const Parts parts{dx_terms * (int)((cols + p.per - 1) / p.per), dx_terms, p.per, a.rows * p.ldf, p.g_second};
    const bool dw_large = a.rows >= 1600 && tile_for(cols, a.K) == LARGE, dw_more = g.dw_fmt == BSM_F32;
    if (g.dX && a.rows > 0) {
      x.M = a.rows; x.N = a.K; x.K = cols; x.dtype = DT;
      x.A = G; x.lda = p.ldg; x.B = W; x.ldb = a.ldw;
      x.accum = at > 0;
      if (direct) { x.D = (float*)g.dX; x.ldd = g.lddx; x.d_fmt = DT; }
      else { x.D = F; x.ldd = p.ldf; x.d_fmt = BSM_F32; }
    }
    if (g.dW) {
      w.M = cols; w.N = a.K; w.K = a.rows; w.dtype = DT;
      w.A = G; w.lda = p.ldg; w.B = a.X; w.ldb = a.ldx;
      w.D = (float*)((uint8_t*)g.dW + c0 * g.lddw * (g.dw_fmt == BSM_F32 ? 4 : 2)); w.ldd = g.lddw; w.d_fmt = g.dw_fmt; w.accum = g.accum;
    }
    if (g.dX && g.dW && a.rows > 0 && !p.large && !dw_large) {
      const int xm = (int)((x.M + 127) / 128), xn = (int)((x.N + 127) / 128), ym = (int)((w.M + 127) / 128), yn = (int)((w.N + 127) / 128);
      const int xg = (xm * xn * parts.n + 7) / 8 * 8;
      const dim3 grid((uint32_t)(xg + ym * yn));
      if (dw_more) hipLaunchKernelGGL((k_xent_both<DT, TERMS, Times>), grid, dim3(256), 0, st, x, w, ep, parts, xm, xn, ym, yn, xg, p.g_second);
      else hipLaunchKernelGGL((k_xent_both<DT, 1, Times>), grid, dim3(256), 0, st, x, w, ep, parts, xm, xn, ym, yn, xg, int64_t(0));
      continue;
    }
    if (g.dX && a.rows > 0) {
      const int64_t m128 = (a.rows + 127) / 128, n128 = (a.K + 127) / 128;
      if (p.large) launch_large<DT, true>(x, ep, parts, st);
      else
        hipLaunchKernelGGL((k_xent_mid<DT, true, false, Times>), dim3((uint32_t)(m128 * n128 * parts.n)), dim3(256), 0, st, x, ep, (int)m128,
                           (int)n128, parts);
    }
    if (g.dW) {
      const int64_t m128 = (cols + 127) / 128, n128 = (a.K + 127) / 128;
      // Short sums and many tiles: four workgroups a CU, K tiles of 32, so that one's loads and stores run beside
      // another's products (10007 columns, K 1000, float32: 200 rows 16 us against 24 on 256 x 256 and 20 on 128 x 128 at
      // two a CU, 800 rows 27 against 38 and 34; 32000, K 2048: 800 rows 136 and 141, 1600 rows 205 and 201, 3000 rows 378
      // and 363 us).
      const dim3 grid((uint32_t)(m128 * n128));
      if (dw_large) {
        launch_large<DT, false>(w, ep, one, st);
        // (the other terms as products of their own onto the first: their sums' way through memory is short beside 1600 rows)
        for (int t = 1; t < TERMS && dw_more; t++) {
          w.A = G + t * p.g_second;
          w.accum = 1;
          launch_large<DT, false>(w, ep, one, st);
        }
      } else if (dw_more) {
        hipLaunchKernelGGL((k_xent_mid<DT, false, false, Times, 128, 32, 4, 1, TERMS>), grid, dim3(256), 0, st, w, ep, (int)m128, (int)n128,
                           Parts{1, 1, 0, 0, p.g_second});
      } else {
        hipLaunchKernelGGL((k_xent_mid<DT, false, false, Times, 128, 32, 4>), grid, dim3(256), 0, st, w, ep, (int)m128, (int)n128, one);
      }
    }
  }
  if (g.dX && a.rows > 0 && !direct) {
    // (slices of rows: a launch has fewer than 2^32 lanes)
    const int64_t per = (a.K + 3) / 4, most = std::max<int64_t>((int64_t(1) << 26) / per, 1);
    auto sum = [&](auto out) {
      constexpr int OUT = decltype(out)::value;
      for (int64_t r = 0; r < a.rows; r += most) {
        const int64_t rows = std::min(most, a.rows - r);
        hipLaunchKernelGGL((k_xent_sum<OUT>), dim3((uint32_t)((rows * per + 63) / 64)), dim3(256), 0, st, F + r * p.ldf, dx_terms * p.parts,
                           a.rows * p.ldf, p.ldf, rows, a.K, (uint8_t*)g.dX + r * g.lddx * (OUT == BSM_F32 ? 4 : 2), g.lddx);
      }
    };
    if (g.dx_fmt == BSM_F32) sum(std::integral_constant<int, BSM_F32>{});
    else sum(std::integral_constant<int, DT>{});
  }
  return hipGetLastError();
}

}  // namespace

int64_t xent_workspace(int64_t rows, int64_t N) { return (slots_of(rows, N) * rows * 8 + 15) / 16 * 16 + rows * 4; }

hipError_t launch_xent(const XentArgs& a, void* workspace, hipStream_t st) {
  float2* part = (float2*)workspace;
  float* at = (float*)((uint8_t*)workspace + (slots_of(a.rows, a.N) * a.rows * 8 + 15) / 16 * 16);
  return a.dtype == BSM_BF16 ? launch_loss<BSM_BF16>(a, part, at, st) : launch_loss<BSM_F16>(a, part, at, st);
}

// (What the gradients' formats will be is not known here.)
int64_t xent_grad_workspace(int64_t rows, int64_t N, int64_t K, int64_t piece) {
  int64_t most = 0;
  for (int terms = 1; terms <= 3; terms++) most = std::max(most, plan_of(rows, N, K, piece, terms).bytes);
  return most;
}

hipError_t launch_xent_grad(const XentArgs& a, const XentGradArgs& g, void* workspace, hipStream_t st) {
  const Plan p = plan_of(a.rows, a.N, a.K, g.piece, terms_of(g, a.dtype));
  return a.dtype == BSM_BF16 ? launch_grad<BSM_BF16>(a, g, p, (uint8_t*)workspace, st)
                             : launch_grad<BSM_F16>(a, g, p, (uint8_t*)workspace, st);
}

}  // namespace bsm
