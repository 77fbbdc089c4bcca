// k_router.hip - counts, offsets and balance loss of a router's choices, and the loss's gradient.
//
//   p_t = softmax(l_t), c_e = assignments of expert e, n = rows kept (those with an expert among their ids),
//   f_e = c_e / (k n), P_e = sum_t p_te / n over the rows kept
//   loss = s E sum_e f_e P_e,   dl_te = g s E / n p_te (f_e - sum_j f_j p_tj)
//
// The gradient needs the counts but not P, so each direction reads the logits once and nothing but the
// counts passes between them. LPR lanes share a row (4 to 16, beyond 256 experts 64; four experts a lane and
// vector, J vectors: lanes of 16 reduce without LDS, and more values a lane are more loads in flight), so a lane keeps
// the same experts for every row it sees: f stays in its registers, and P's column sums are register sums, joined at the
// end across the wave's rows, the workgroup's waves (LDS) and the workgroups (a second launch over at most 256 of them),
// all in a fixed order. A lane adds at most 64 rows in float32, then into a double; a workgroup's sums go to the join as
// float32, 2^-24 of each, and meet in double: the error does not grow with the rows. Counts are integers, so the LDS atomics that make them cannot change a result by their order.
// Bound: for many rows the latency of a few loads and reductions behind one another, sixteen waves a CU in turn (32768
// rows, 128 experts, bf16: 9 us for 8 MB, 4-8 us for the join, the gradient 9.5 us for 17 MB); for few rows launches, so
// up to kOneGroup logits a single workgroup does everything in one (16 rows, 64 experts: 3.7 us).
#include "grouped.hpp"
#include "router.hpp"
#include "../../include/bsm.h"

namespace bsm {
namespace {

constexpr int THREADS = 1024, WAVES = THREADS / 64, JOIN = 1024;
constexpr int kMaxGroups = 256;
constexpr int64_t kOneGroup = 32768;

template <int F>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (F == BSM_F32) return ((const float*)p)[i];
  else if constexpr (F == BSM_BF16) return bf16_bits_to_f32(((const uint16_t*)p)[i]);
  else return f16_bits_to_f32(((const uint16_t*)p)[i]);
}
// Four consecutive values from element i on, those at or past `left` -infinity.
template <int F>
__device__ __forceinline__ void load4(const void* p, int64_t i, int left, bool vec, float (&v)[4]) {
  if (vec && left >= 4) {
    if constexpr (F == BSM_F32) {
      const f32x4 x = *(const f32x4*)((const float*)p + i);
#pragma unroll
      for (int e = 0; e < 4; e++) v[e] = x[e];
    } else {
      const uint2 x = *(const uint2*)((const uint16_t*)p + i);
      const uint32_t w[2] = {x.x, x.y};
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const uint16_t h = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        v[e] = F == BSM_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h);
      }
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; e++) v[e] = e < left ? load1<F>(p, i + e) : -INFINITY;
}

// The row's reduction to all of its lanes: pairs, quads, halves and rows of 16 by the vector unit's own lane
// permutations, beyond that through the LDS crossbar.
template <int CTRL>
__device__ __forceinline__ float lane_swap(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
template <int LPR, class OP>
__device__ __forceinline__ float row_reduce(float v, OP op) {
  v = op(v, lane_swap<0xB1>(v));                             // quad_perm 1 0 3 2
  v = op(v, lane_swap<0x4E>(v));                             // quad_perm 2 3 0 1
  if constexpr (LPR >= 8) v = op(v, lane_swap<0x141>(v));    // row_half_mirror
  if constexpr (LPR >= 16) v = op(v, lane_swap<0x140>(v));   // row_mirror
#pragma unroll
  for (int d = 16; d < LPR; d *= 2) v = op(v, __shfl_xor(v, d));
  return v;
}
template <int LPR>
__device__ __forceinline__ float row_max(float v) { return row_reduce<LPR>(v, [](float a, float b) { return fmaxf(a, b); }); }
template <int LPR>
__device__ __forceinline__ float row_sum(float v) { return row_reduce<LPR>(v, [](float a, float b) { return a + b; }); }

// One row's softmax in this lane's registers: in the logits, out exp(l - max) and the factor 1 / sum. A
// row without a finite logit above -infinity has no softmax: every probability is 0. NaN and +infinity
// make the row NaN, as the formula does.
template <int LPR, int J>
__device__ __forceinline__ float row_softmax(float (&v)[J][4]) {
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < J; j++)
#pragma unroll
    for (int e = 0; e < 4; e++) m = fmaxf(m, v[j][e]);
  m = row_max<LPR>(m);
  // (fmaxf passes over NaN; a row of NaN and -infinity has max -infinity and must stay NaN)
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < J; j++)
#pragma unroll
    for (int e = 0; e < 4; e++) {
      v[j][e] = v[j][e] == -INFINITY ? 0.0f : exp_f32(v[j][e] - m);
      s += v[j][e];
    }
  s = row_sum<LPR>(s);
  return s == 0.0f ? 0.0f : 1.0f / s;
}

// The row's id of this lane's place, -1 where it has none, and, once it is there: whether the row has an expert among
// its ids, for every lane of the row; with `count`, counts them. (Ids past the first LPR are loaded where they are
// looked at.)
__device__ __forceinline__ int first_id(const RouterArgs& a, int64_t row, bool in, int lr) {
  return in && lr < a.k ? a.ids[row * a.k + lr] : -1;
}
template <int LPR>
__device__ __forceinline__ bool row_kept(const RouterArgs& a, int64_t row, bool in, int lr, int lane, int id, int* count) {
  bool any = false;
  for (int j0 = 0;;) {
    const bool ok = id >= 0 && id < a.E;
    if (ok && count) atomicAdd(count + id, 1);
    any |= ok;
    j0 += LPR;
    if (j0 >= a.k) break;
    id = in && j0 + lr < a.k ? a.ids[row * a.k + j0 + lr] : -1;
  }
  const uint64_t mine = (LPR == 64 ? ~0ull : ((1ull << LPR) - 1)) << (lane & ~(LPR - 1));
  return (__ballot(any) & mine) != 0;
}

// Sum over the wave, in lane 63: as grouped::wave_inclusive_scan moves it, a double's halves apart.
template <int CTRL, int ROWS>
__device__ __forceinline__ double shifted(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum(double v) {
  v += shifted<0x111, 0xF>(v);   // row_shr:1, 2, 4, 8
  v += shifted<0x112, 0xF>(v);
  v += shifted<0x114, 0xF>(v);
  v += shifted<0x118, 0xF>(v);
  v += shifted<0x142, 0xA>(v);   // row_bcast:15, 31
  v += shifted<0x143, 0xC>(v);
  return v;
}

// Exclusive sums, the loss and the outputs, by the whole workgroup of NT lanes: cnt[0 .. E - 1], kept and the column sums
// psum in LDS; E <= 1024, two experts a lane. wscan and wred: LDS of one value a wave.
template <int NT>
__device__ __forceinline__ void finish(const RouterArgs& a, const int* cnt, int kept, const double* psum, int* wscan, double* wred) {
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const bool h0 = 2 * t < a.E, h1 = 2 * t + 1 < a.E;
  const int c0 = h0 ? cnt[2 * t] : 0, c1 = h1 ? cnt[2 * t + 1] : 0;
  double part = (h0 ? (double)c0 * psum[2 * t] : 0.0) + (h1 ? (double)c1 * psum[2 * t + 1] : 0.0);
  const int incl = grouped::wave_inclusive_scan(c0 + c1);
  part = wave_sum(part);
  if (lane == 63) { wscan[w] = incl; wred[w] = part; }
  __syncthreads();
  int before = incl - c0 - c1, all = 0;
  double sum = 0.0;
#pragma unroll
  for (int q = 0; q < NT / 64; q++) {
    if (q < w) before += wscan[q];
    all += wscan[q];
    sum += wred[q];
  }
  if (h0) { a.counts[2 * t] = c0; a.offsets[2 * t] = before; }
  if (h1) { a.counts[2 * t + 1] = c1; a.offsets[2 * t + 1] = before + c0; }
  if (t == 0) {
    a.counts[a.E] = kept;
    a.offsets[a.E] = all;
    const double n = kept;
    a.loss[0] = kept ? (float)(a.scale * (a.E * sum / (n * n * a.k))) : 0.0f;
  }
}

// Where a workgroup's sums go: two experts' column sums and counts in 16 bytes, `pairs` of them a workgroup (the
// column sums rounded to float32 once more: 2^-24 of each), and its kept rows.
struct Pair { float s0, s1; int c0, c1; };
struct Parts { Pair* sums; int* kept; int pairs; };

// ONE: the only workgroup, which finishes too. Otherwise workgroup b's sums go to row b of `parts`.
template <int F, int LPR, int J, bool ONE>
__global__ __launch_bounds__(THREADS) void k_balance(RouterArgs a, Parts parts) {
  constexpr int RPW = 64 / LPR, E4 = 4 * LPR * J, U = 2;
  __shared__ double total[E4];
  __shared__ double sums[E4 > 256 ? 1 : WAVES][E4];
  __shared__ int cnt[E4];
  __shared__ int kept_all;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, lr = lane & (LPR - 1), sub = lane / LPR;
  for (int i = t; i < E4; i += THREADS) { cnt[i] = 0; total[i] = 0.0; }
  if (t == 0) kept_all = 0;
  __syncthreads();
  double dsum[J][4] = {};
  float fsum[J][4] = {};
  int kept = 0, since = 0;
  const int64_t step = (int64_t)gridDim.x * WAVES * RPW;
  for (int64_t r0 = ((int64_t)blockIdx.x * WAVES + w) * RPW; r0 < a.rows; r0 += U * step) {
    // U rows of logits are asked for before the first is worked on
    float v[U][J][4];
    int id[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int64_t row = r0 + u * step + sub;
      id[u] = first_id(a, row, row < a.rows, lr);
#pragma unroll
      for (int j = 0; j < J; j++) {
        const int e0 = 4 * (LPR * j + lr);
        load4<F>(a.logits, row * a.ldl + e0, row < a.rows ? a.E - e0 : 0, a.vec, v[u][j]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int64_t row = r0 + u * step + sub;
      const bool keep = row_kept<LPR>(a, row, row < a.rows, lr, lane, id[u], cnt);
      const float inv = row_softmax<LPR, J>(v[u]);
      kept += keep && lr == 0;
#pragma unroll
      for (int j = 0; j < J; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) fsum[j][e] += keep ? v[u][j][e] * inv : 0.0f;
    }
    if (++since == 64 / U) {
      since = 0;
#pragma unroll
      for (int j = 0; j < J; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) { dsum[j][e] += fsum[j][e]; fsum[j][e] = 0.0f; }
    }
  }
  if (kept) atomicAdd(&kept_all, kept);
#pragma unroll
  for (int j = 0; j < J; j++)
#pragma unroll
    for (int e = 0; e < 4; e++) {
      double d = dsum[j][e] + fsum[j][e];
#pragma unroll
      for (int s = LPR; s < 64; s *= 2) d += __shfl_xor(d, s);
      dsum[j][e] = d;
    }
  if constexpr (E4 <= 256) {
    if (sub == 0)
#pragma unroll
      for (int j = 0; j < J; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) sums[w][4 * (LPR * j + lr) + e] = dsum[j][e];
    __syncthreads();
    for (int i = t; i < E4; i += THREADS) {
      double d = 0.0;
#pragma unroll
      for (int q = 0; q < WAVES; q++) d += sums[q][i];
      total[i] = d;
    }
  } else {
    // (one wave after another: a wave's lanes hold different experts)
    for (int q = 0; q < WAVES; q++) {
      if (w == q)
#pragma unroll
        for (int j = 0; j < J; j++)
#pragma unroll
          for (int e = 0; e < 4; e++) total[4 * (LPR * j + lr) + e] += dsum[j][e];
      __syncthreads();
    }
  }
  __syncthreads();
  if constexpr (ONE) {
    __shared__ int wscan[WAVES];
    __shared__ double wred[WAVES];
    finish<THREADS>(a, cnt, kept_all, total, wscan, wred);
  } else {
    // (experts past E have sums and counts of 0: their logits are taken as -infinity)
    for (int i = t; i < parts.pairs; i += THREADS)
      *(uint4*)(parts.sums + (int64_t)blockIdx.x * parts.pairs + i) =
          make_uint4(__float_as_uint((float)total[2 * i]), __float_as_uint((float)total[2 * i + 1]), (uint32_t)cnt[2 * i],
                     (uint32_t)cnt[2 * i + 1]);
    if (t == 0) parts.kept[blockIdx.x] = kept_all;
  }
}

// Joins the workgroups' sums: a lane adds a pair of every slices-th workgroup (with 128 experts 16 of 256, all in flight
// at once), then the slices meet in LDS.
__global__ __launch_bounds__(JOIN) void k_balance_join(RouterArgs a, Parts parts, int groups) {
  __shared__ double red[2 * JOIN];
  __shared__ int num[2 * JOIN];
  __shared__ double total[1024];
  __shared__ int cnt[1024];
  __shared__ int kept_all;
  __shared__ int wscan[JOIN / 64];
  __shared__ double wred[JOIN / 64];
  const int t = threadIdx.x;
  int cols = 1;
  while (cols < parts.pairs) cols *= 2;   // at most 512
  const int slices = JOIN / cols, s = t / cols, c = t & (cols - 1);
  double d0 = 0.0, d1 = 0.0;
  int n0 = 0, n1 = 0, kept = 0;
  if (t < 64)
#pragma unroll 4
    for (int b = t; b < groups; b += 64) kept += parts.kept[b];
  if (c < parts.pairs) {
    constexpr int AT_ONCE = 16;
    for (int b0 = s; b0 < groups; b0 += AT_ONCE * slices) {
      uint4 x[AT_ONCE];
#pragma unroll
      for (int i = 0; i < AT_ONCE; i++) {
        const int b = b0 + i * slices;
        x[i] = b < groups ? *(const uint4*)(parts.sums + (int64_t)b * parts.pairs + c) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < AT_ONCE; i++) {
        d0 += __uint_as_float(x[i].x); d1 += __uint_as_float(x[i].y);
        n0 += (int)x[i].z; n1 += (int)x[i].w;
      }
    }
  }
  red[2 * t] = d0; red[2 * t + 1] = d1;
  num[2 * t] = n0; num[2 * t + 1] = n1;
  if (t < 64) {
    kept = grouped::wave_inclusive_scan(kept);
    if (t == 63) kept_all = kept;
  }
  __syncthreads();
  for (int i = t; i < 2 * cols; i += JOIN) {
    double d = 0.0;
    int n = 0;
#pragma unroll 8
    for (int q = 0; q < slices; q++) { d += red[2 * q * cols + i]; n += num[2 * q * cols + i]; }
    total[i] = d;
    cnt[i] = n;
  }
  __syncthreads();
  finish<JOIN>(a, cnt, kept_all, total, wscan, wred);
}

// The gradient: one pass, each row's probabilities made again from its logits.
template <int F, int LPR, int J>
__global__ __launch_bounds__(256) void k_balance_grad(RouterArgs a, RouterGradArgs g) {
  constexpr int RPW = 64 / LPR;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, lr = lane & (LPR - 1), sub = lane / LPR;
  const int64_t step = (int64_t)gridDim.x * 4 * RPW;
  int64_t r0 = ((int64_t)blockIdx.x * 4 + w) * RPW;
  // a row's logits and id are asked for before the row ahead of them (the first: before the counts) is worked on
  float v[J][4];
  int id;
  auto load = [&](int64_t row) {
    const bool in = row < a.rows;
    id = first_id(a, row, in, lr);
#pragma unroll
    for (int j = 0; j < J; j++) {
      const int e0 = 4 * (LPR * j + lr);
      load4<F>(a.logits, row * a.ldl + e0, in ? a.E - e0 : 0, a.vec, v[j]);
    }
  };
  load(r0 + sub);
  float f[J][4];
  int c[J][4];
  const int n = a.counts[a.E];
  const float dl = g.dloss ? *g.dloss : 1.0f;
#pragma unroll
  for (int j = 0; j < J; j++)
#pragma unroll
    for (int e = 0; e < 4; e++) c[j][e] = a.counts[min(4 * (LPR * j + lr) + e, a.E)];
  const float over = n > 0 ? 1.0f / ((float)a.k * (float)n) : 0.0f;
  const float coef = n > 0 ? dl * a.scale * (float)a.E / (float)n : 0.0f;
#pragma unroll
  for (int j = 0; j < J; j++)
#pragma unroll
    for (int e = 0; e < 4; e++) f[j][e] = 4 * (LPR * j + lr) + e < a.E ? (float)c[j][e] * over : 0.0f;
  for (; r0 < a.rows; r0 += step) {
    const int64_t row = r0 + sub;
    const bool in = row < a.rows;
    float p[J][4];
#pragma unroll
    for (int j = 0; j < J; j++)
#pragma unroll
      for (int e = 0; e < 4; e++) p[j][e] = v[j][e];
    const int now = id;
    if (r0 + step < a.rows) load(row + step);
    const bool keep = row_kept<LPR>(a, row, in, lr, lane, now, nullptr);
    const float inv = row_softmax<LPR, J>(p);
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < J; j++)
#pragma unroll
      for (int e = 0; e < 4; e++) {
        p[j][e] *= inv;
        dot += f[j][e] * p[j][e];
      }
    dot = row_sum<LPR>(dot);
    if (!in) continue;
#pragma unroll
    for (int j = 0; j < J; j++) {
      const int e0 = 4 * (LPR * j + lr), left = a.E - e0;
      if (left <= 0) continue;
      float o[4];
#pragma unroll
      for (int e = 0; e < 4; e++) o[e] = keep ? coef * p[j][e] * (f[j][e] - dot) : 0.0f;
      const int64_t at = row * g.ldd + e0;
      if (g.d_fmt == BSM_F32) {
        float* q = (float*)g.D + at;
        if (g.vec && left >= 4) {
          f32x4 x = {o[0], o[1], o[2], o[3]};
          if (g.accum) x += *(const f32x4*)q;
          *(f32x4*)q = x;
        } else {
#pragma unroll
          for (int e = 0; e < 4; e++)
            if (e < left) q[e] = g.accum ? q[e] + o[e] : o[e];
        }
      } else if constexpr (F != BSM_F32) {
        uint16_t* q = (uint16_t*)g.D + at;
        auto bits = [](float x) { return F == BSM_BF16 ? f32_to_bf16_bits(x) : f32_to_f16_bits(x); };
        auto val = [](uint16_t h) { return F == BSM_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h); };
        if (g.vec && left >= 4) {
          if (g.accum) {
            const uint2 y = *(const uint2*)q;
            o[0] += val((uint16_t)y.x); o[1] += val((uint16_t)(y.x >> 16));
            o[2] += val((uint16_t)y.y); o[3] += val((uint16_t)(y.y >> 16));
          }
          *(uint2*)q = make_uint2(bits(o[0]) | (uint32_t)bits(o[1]) << 16, bits(o[2]) | (uint32_t)bits(o[3]) << 16);
        } else {
#pragma unroll
          for (int e = 0; e < 4; e++)
            if (e < left) q[e] = bits(g.accum ? val(q[e]) + o[e] : o[e]);
        }
      }
    }
  }
}

int lanes_per_row(int E) { return E <= 16 ? 4 : E <= 32 ? 8 : E <= 256 ? 16 : 64; }

int64_t groups_of(int64_t rows, int E) {
  if (rows * E <= kOneGroup) return 1;
  // (two rows a lane at least: half as many sums to join)
  const int64_t per = 2 * WAVES * (64 / lanes_per_row(E));
  return std::min<int64_t>((rows + per - 1) / per, kMaxGroups);
}

// f with the row layout for E experts: f(LPR, J).
template <class FN>
void with_layout(int E, FN f) {
  using std::integral_constant;
  if (E <= 16) f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  else if (E <= 32) f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  else if (E <= 64) f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (E <= 128) f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  else if (E <= 256) f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  else if (E <= 512) f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else f(integral_constant<int, 64>{}, integral_constant<int, 4>{});
}

template <int F>
void launch_balance(const RouterArgs& a, const Parts& parts, int64_t groups, hipStream_t st) {
  with_layout(a.E, [&](auto lpr, auto j) {
    constexpr int LPR = decltype(lpr)::value, J = decltype(j)::value;
    if (groups == 1) hipLaunchKernelGGL((k_balance<F, LPR, J, true>), dim3(1), dim3(THREADS), 0, st, a, parts);
    else hipLaunchKernelGGL((k_balance<F, LPR, J, false>), dim3((uint32_t)groups), dim3(THREADS), 0, st, a, parts);
  });
}

template <int F>
void launch_grad(const RouterArgs& a, const RouterGradArgs& g, hipStream_t st) {
  const int64_t per = 4 * (64 / lanes_per_row(a.E));
  const dim3 grid((uint32_t)std::min<int64_t>((a.rows + per - 1) / per, 2048));
  with_layout(a.E, [&](auto lpr, auto j) {
    hipLaunchKernelGGL((k_balance_grad<F, decltype(lpr)::value, decltype(j)::value>), grid, dim3(256), 0, st, a, g);
  });
}

}  // namespace

int64_t balance_workspace(int64_t rows, int E) {
  const int64_t n = groups_of(rows, E);
  return n == 1 ? 0 : n * ((E + 1) / 2 * (int64_t)sizeof(Pair) + (int64_t)sizeof(int));
}

hipError_t launch_router_balance(const RouterArgs& a, void* workspace, hipStream_t st) {
  const int64_t n = groups_of(a.rows, a.E);
  Parts parts{};
  parts.pairs = (a.E + 1) / 2;
  if (n > 1) {
    parts.sums = (Pair*)workspace;
    parts.kept = (int*)(parts.sums + n * parts.pairs);
  }
  if (a.l_fmt == BSM_F32) launch_balance<BSM_F32>(a, parts, n, st);
  else if (a.l_fmt == BSM_BF16) launch_balance<BSM_BF16>(a, parts, n, st);
  else launch_balance<BSM_F16>(a, parts, n, st);
  if (n > 1) hipLaunchKernelGGL(k_balance_join, dim3(1), dim3(JOIN), 0, st, a, parts, (int)n);
  return hipGetLastError();
}

hipError_t launch_router_balance_grad(const RouterArgs& a, const RouterGradArgs& g, hipStream_t st) {
  if (a.l_fmt == BSM_F32) launch_grad<BSM_F32>(a, g, st);
  else if (a.l_fmt == BSM_BF16) launch_grad<BSM_BF16>(a, g, st);
  else launch_grad<BSM_F16>(a, g, st);
  return hipGetLastError();
}

}  // namespace bsm
