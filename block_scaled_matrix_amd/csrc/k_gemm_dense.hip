// k_gemm_dense.hip - fp16/bf16 GEMM D = s * A * B^T (+ D) on gfx950 MFMA.
//
// Semantics ("tcgen05.mma": Call parameters, Operand specification, Code generation,
// Example: four K16 issues; "Explicit CUDA tile patterns": Warp MMA): B is the
// (N,K) operand, the product is A times B transposed, float32 accumulation; the
// first K step starts from D when accumulating and from zero otherwise.
//
// gfx950 design:
//  - workgroup tile 256 x 256, K tile 64, four wave64s in a 2 x 2 grid, each owning a
//    128 x 128 sub-tile as 8 x 8 v_mfma_f32_16x16x32 accumulators (256 fp32 per lane,
//    held in AGPRs). Under sustained load the chip's power limit sets the clock, and the
//    16x16x32 shape moves fewer accumulator bytes per product than 32x32x16 (4 registers
//    read and written per 8192 products instead of 16 per 16384): a pure MFMA loop of it
//    sustains about 7% more than the 32x32x16 loop, and this kernel runs 4-6% faster with
//    it. The MFMA is issued with the operands swapped (B fragment first), so a lane ends up
//    holding four consecutive output columns per block and the epilogue moves D in 16-byte
//    pieces;
//  - operand tiles stream HBM -> LDS with global_load_lds_dwordx4 (no register
//    staging) in whole 128-byte lines: an SGPR tile base plus per-lane 32-bit offsets
//    that stay fixed over the whole K loop; two LDS stages of 64 KiB;
//  - a K tile is two 32-K steps of 64 MFMAs; each wave reads step 1's fragments during
//    step 0, so the stage is released in the middle of step 0 and the copy of tile kt+2
//    starts while tile kt is still being multiplied: two K tiles stay in flight;
//  - LDS reads and copies are interleaved one by one with the MFMAs (a copy every fifth
//    16-cycle MFMA: denser copies held the issuing waves behind the shared copy path), so
//    they issue while the matrix pipe is busy rather than in bursts that stall it;
//  - K-major tiles: 128-byte rows, 16-byte chunk c of row r stored at chunk
//    c ^ ((r >> 1) & 7), so the 16 rows one 16-lane group reads with ds_read_b128
//    cover all 64 LDS banks;
//  - MN-major tiles (the transposed storage): 512-byte k-rows, chunk c of k-row kr
//    stored at c ^ 4(kr & 3) ^ 2((kr >> 3) & 1); fragments come from ds_read_b64_tr_b16,
//    the LDS transpose read (the analog of ldmatrix .trans in "ldmatrix / stmatrix",
//    Transpose and stores): the two 16-lane groups of a half-wave read k-rows 8 apart, and
//    the swizzle puts their eight 32-byte row pieces in distinct banks (checked on the CPU);
//  - M/N edges clamp the rows that are loaded and mask the stores; a ragged last K
//    tile is loaded through registers with the elements past K zeroed.
#include "gemm_dense_tile.hpp"

namespace bsm {
namespace {

using namespace dense;

template <int DT, bool AK, bool BKM, bool ACC>
__global__ __launch_bounds__(256, 1) void k_gemm_dense(GemmArgs a, int tiles_m, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * STAGE_BYTES];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tm, tn;
  gemm::tile_coords(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const float sgn = a.negate ? -1.0f : 1.0f;
  f32x4 acc[8][8];
  tile_product<DT, AK, BKM>(a, tm, tn, lds, lane, w, acc);
  store_tile16(a.D, a.ldd, a.M, a.N, (int64_t)tm * BM + 128 * (w >> 1), (int64_t)tn * BN + 128 * (w & 1), lane, sgn,
               acc, lds + 32768 * w, ACC, a.ew_op, a.ew_scale, a.ew_bias);
}

template <int DT, bool AK, bool BKM>
hipError_t launch_one(const GemmArgs& a, hipStream_t st) {
  const int64_t tm64 = (a.M + BM - 1) / BM, tn64 = (a.N + BN - 1) / BN;
  if (tm64 * tn64 > 0x7FFFFFFF) return hipErrorInvalidValue;
  const int tiles_m = (int)tm64, tiles_n = (int)tn64;
  if (a.accum)
    hipLaunchKernelGGL((k_gemm_dense<DT, AK, BKM, true>), dim3(tiles_m * tiles_n), dim3(256), 0, st, a, tiles_m, tiles_n);
  else
    hipLaunchKernelGGL((k_gemm_dense<DT, AK, BKM, false>), dim3(tiles_m * tiles_n), dim3(256), 0, st, a, tiles_m, tiles_n);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(const GemmArgs& a, hipStream_t st) {
  if (a.a_kmajor && a.b_kmajor) return launch_one<DT, true, true>(a, st);
  if (a.a_kmajor) return launch_one<DT, true, false>(a, st);
  if (a.b_kmajor) return launch_one<DT, false, true>(a, st);
  return launch_one<DT, false, false>(a, st);
}

// Debug: one operand tile through the GEMM's loader and fragment reads. The dump holds, for
// 16-row block b (0..15) and 32-K step s (0..1), each lane's 8 elements: dump[((b * 2 + s) * 64
// + lane) * 8 + e] = operand (16b + lane % 16, 32s + 8 (lane / 16) + e).
template <bool KMAJ>
__global__ __launch_bounds__(256) void k_debug_fragments(const uint16_t* __restrict__ src, uint16_t* dump) {
  __shared__ __attribute__((aligned(1024))) uint8_t tile[TILE_BYTES];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t off[8];
  dma_offsets<KMAJ>(KMAJ ? BK : BM, 0, BM, w, lane, off);
  gemm::issue_tile8(src, off, gemm::lds_addr(tile), w);
  gemm::stage_barrier<0>();
  for (int b = 4 * w; b < 4 * w + 4; b++) {
    for (int s = 0; s < STEPS; s++) {
      // rows 16b ..: wave base 128 (b / 8), 16-row block b % 8
      const uint4 v = read_frag<KMAJ>(tile, lane, 128 * (b >> 3), s, b & 7);
      *(uint4*)(dump + ((b * STEPS + s) * 64 + lane) * 8) = v;
    }
  }
}

}  // namespace

hipError_t launch_gemm_dense(const GemmArgs& a, hipStream_t st) {
  // Empty sum: D = f(accum ? D : 0) (the sign of an empty sum is irrelevant).
  if (a.K == 0) return launch_empty_gemm(a.D, a.ldd, a.M, a.N, a.accum, a.ew_op, a.ew_scale, a.ew_bias, st);
  return a.dtype == BSM_BF16 ? launch_dt<BSM_BF16>(a, st) : launch_dt<BSM_F16>(a, st);
}

hipError_t launch_debug_fragments(const uint16_t* src, int kmajor, uint16_t* dump, hipStream_t st) {
  if (kmajor) hipLaunchKernelGGL(k_debug_fragments<true>, dim3(1), dim3(256), 0, st, src, dump);
  else hipLaunchKernelGGL(k_debug_fragments<false>, dim3(1), dim3(256), 0, st, src, dump);
  return hipGetLastError();
}

}  // namespace bsm
