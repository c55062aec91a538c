// Rows to 8 bits: residual addition with root-mean-square norm, and the plain
// e4m3 rounding of rows.
//
//   v = x + residual,  r = 1 / sqrt(mean(v^2) + eps),  y = (v r) weight
//
// and from the fp32 y: the row in another type, q8_1 blocks of 32, e4m3 with a
// scale for each 128.  Every element is read once and written once, with about
// ten operations in between: HBM bounds long batches, latency short ones (one
// read, the join of the row's sums, one write, and the launch).  Measured, in a
// captured graph: 21000 x 4096 bf16 with residual, y and e4m3 139 to 142 us
// (777 MB, 5.5 TB/s; a large copy reaches 5.1), 5268 x 4096 fp32 with residual and q8_1
// 31 us, 4 x 4096 3.3 us; e4m3 rounding alone of 21000 x 4096 bf16 43 us
// (6.1 TB/s), of 333 x 2000 fp16 2.1 us.
#include "block_fp8.h"

namespace latmoe {
namespace {

// Sum over a 64-lane wave, in every lane.
__device__ __forceinline__ double wave_sum(double s) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) s += __shfl_xor(s, m);
  return s;
}

// 1 / sqrt(a), a > 0, rounded to fp32: the hardware's 64-bit estimate (at least
// 20 bits) and two steps of y += y (1 - a y^2) / 2, each of which doubles them.
__device__ __forceinline__ float inverse_root(double a) {
  double y = __builtin_amdgcn_rsq(a);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const double e = __builtin_fma(-a * y, y, 1.0);
    y = __builtin_fma(0.5 * y, e, y);
  }
  return (float)y;
}

// Adds CH chunks of residual (TYPE) to v.
template <int TYPE, int TPR, int CH>
__device__ __forceinline__ void add_rows(const void* p, int64_t row, int lane, int C, float (*v)[8]) {
  Raw8<TYPE> raw[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = (i * TPR + lane) * 8;
    if (c < C) raw[i].load(p, row + c);
    else raw[i].zero();
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    float f[8];
    raw[i].values(f);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] += f[j];
  }
}

// TPR threads hold one row in registers, 8 contiguous values a chunk and CH
// chunks a thread, chunk i of thread `lane` at column 8 (i TPR + lane): a
// q8_1 block is 4 neighbouring lanes, an e4m3 block 16, so both roundings stay
// inside a wave.  TPR = 64 needs no barrier (four rows to a workgroup).
template <int XT, int TPR, int CH>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_rmsnorm(const NormArgs a) {
  // every product is rounded to fp32 on its own (the q8_1 rule has no FMA)
#pragma clang fp contract(off)
  constexpr int kWaves = TPR / 64;
  const int lane = TPR == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t group = workgroup_number();
  const int64_t t = TPR == 64 ? group * 4 + (threadIdx.x >> 6) : group;
  if (t >= a.T) return;  // whole waves, and with TPR > 64 whole workgroups
  const int C = a.C;
  const int64_t row = t * C;
  float v[CH][8];
  // the weights are on their way during the sum, where the registers allow it
  constexpr bool kEarly = CH <= 2;
  Raw8<LAT_MOE_F32> weight[kEarly ? CH : 1];
  {
    Raw8<XT> raw[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = (i * TPR + lane) * 8;
      if (c < C) raw[i].load(a.x, row + c);
      else raw[i].zero();
    }
    if constexpr (kEarly) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = (i * TPR + lane) * 8;
        if (c < C) weight[i].load(a.weight, c);
        else weight[i].zero();
      }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) raw[i].values(v[i]);
  }
  if (a.residual) {
    if (a.residual_type == LAT_MOE_F32) add_rows<LAT_MOE_F32, TPR, CH>(a.residual, row, lane, C, v);
    else if (a.residual_type == LAT_MOE_BF16) add_rows<LAT_MOE_BF16, TPR, CH>(a.residual, row, lane, C, v);
    else add_rows<LAT_MOE_F16, TPR, CH>(a.residual, row, lane, C, v);
  }
  // Squares of fp32 values are exact in 64 bits, and 2^15 of them add up with a
  // relative error below 2^-38 in any order: r is the formula's, rounded once.
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = __builtin_fma((double)v[i][j], (double)v[i][j], ss);
  ss = wave_sum(ss);
  if constexpr (kWaves > 1) {
    __shared__ double part[kWaves];
    if ((lane & 63) == 0) part[lane >> 6] = ss;
    __syncthreads();
    ss = 0.0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) ss += part[w];
  }
  const float r = inverse_root(ss * a.inv_c + (double)a.eps);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = (i * TPR + lane) * 8;
    const bool in = c < C;
    if (a.residual_out && in) store8(a.residual_out, a.residual_type, row + c, v[i]);
    float y[8];
    if (in) {
      float g[8];
      if constexpr (kEarly) {
        weight[i].values(g);
      } else {
        Raw8<LAT_MOE_F32> w;
        w.load(a.weight, c);
        w.values(g);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = v[i][j] * r * g[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = 0.f;
    }
    if (a.y && in) store8(a.y, a.y_type, row + c, y);
    if (a.y_fp8) {
      float scale;
      const uint2 codes = e4m3_block(y, scale);
      if (in) {
        *reinterpret_cast<uint2*>(a.y_fp8 + row + c) = codes;
        if ((lane & 15) == 0) a.y_scales[t * ((C + kFp8Block - 1) / kFp8Block) + c / kFp8Block] = scale;
      }
    }
    if (a.y_q8) {
      const float d = group_max<4>(amax8(y)) / 127.0f;
      const float id = d != 0.0f ? 1.0f / d : 0.0f;
      uint32_t pk[2];
      int sum = 0;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        pk[q] = pack_codes(round_half_away(y[4 * q] * id), round_half_away(y[4 * q + 1] * id),
                           round_half_away(y[4 * q + 2] * id), round_half_away(y[4 * q + 3] * id));
        sum = __builtin_amdgcn_sdot4((int)pk[q], 0x01010101, sum, false);
      }
      sum += __shfl_xor(sum, 1);
      sum += __shfl_xor(sum, 2);
      if (in) {
        uint32_t* blk = reinterpret_cast<uint32_t*>(a.y_q8 + (t * (C / 32) + c / 32) * kQ81Bytes);
        blk[1 + 2 * (lane & 3)] = pk[0];
        blk[2 + 2 * (lane & 3)] = pk[1];
        if ((lane & 3) == 0)
          blk[0] = float_to_half_bits(d) | (float_to_half_bits(fp32_barrier(d * (float)sum)) << 16);
      }
    }
  }
}

// 16 lanes to a block of 128 values; a workgroup takes 16 blocks of the
// [rows][blocks] order.
template <int XT>
__global__ __launch_bounds__(256) void k_quantize_fp8(const void* __restrict__ x, uint32_t nblocks, int blocks_per_row,
                                                      int cols, uint8_t* __restrict__ codes,
                                                      float* __restrict__ scales) {
#pragma clang fp contract(off)
  const uint64_t at16 = (uint64_t)workgroup_number() * 16 + (threadIdx.x >> 4);
  if (at16 >= nblocks) return;  // whole 16-lane groups
  const uint32_t b = (uint32_t)at16;
  const uint32_t row = b / (uint32_t)blocks_per_row;
  const int c = (int)(b - row * blocks_per_row) * kFp8Block + (threadIdx.x & 15) * 8;
  const int64_t at = (int64_t)row * cols + c;
  Raw8<XT> raw;
  if (c < cols) raw.load(x, at);
  else raw.zero();
  float v[8], scale;
  raw.values(v);
  const uint2 w = e4m3_block(v, scale);
  if (c < cols) *reinterpret_cast<uint2*>(codes + at) = w;
  if ((threadIdx.x & 15) == 0) scales[b] = scale;
}

template <int TPR, int CH>
void run_rmsnorm(const NormArgs& a, hipStream_t st) {
  const dim3 grid = grid_of(TPR == 64 ? (a.T + 3) / 4 : a.T), block(TPR < 256 ? 256 : TPR);
  if (a.x_type == LAT_MOE_F32) hipLaunchKernelGGL((k_rmsnorm<LAT_MOE_F32, TPR, CH>), grid, block, 0, st, a);
  else if (a.x_type == LAT_MOE_BF16) hipLaunchKernelGGL((k_rmsnorm<LAT_MOE_BF16, TPR, CH>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_rmsnorm<LAT_MOE_F16, TPR, CH>), grid, block, 0, st, a);
}

}  // namespace

// Rows of bf16 with residual, y and e4m3 (us, TB/s): 21000 x 512 18.7 (5.2),
// x 528 29 (3.4: 66 of 256 threads have data), x 1024 34 (5.8), x 2048 71 (5.5),
// x 4096 140 (5.5), x 7168 250 (5.4), x 8192 286 (5.4), 10000 x 16384 279 (5.3),
// 5000 x 32768 294 (5.0).
hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t st) {
  if (a.C <= 512) run_rmsnorm<64, 1>(a, st);
  else if (a.C <= 2048) run_rmsnorm<256, 1>(a, st);
  else if (a.C <= 4096) run_rmsnorm<256, 2>(a, st);
  else if (a.C <= 8192) run_rmsnorm<256, 4>(a, st);
  else run_rmsnorm<1024, 4>(a, st);
  return hipGetLastError();
}

hipError_t launch_quantize_fp8(const void* x, int x_type, int64_t rows, int cols, uint8_t* codes, float* scales,
                               hipStream_t st) {
  const int bpr = (cols + kFp8Block - 1) / kFp8Block;
  const uint32_t nb = (uint32_t)(rows * bpr);
  const dim3 grid = grid_of(((int64_t)nb + 15) / 16), block(256);
  if (x_type == LAT_MOE_F32)
    hipLaunchKernelGGL(k_quantize_fp8<LAT_MOE_F32>, grid, block, 0, st, x, nb, bpr, cols, codes, scales);
  else if (x_type == LAT_MOE_BF16)
    hipLaunchKernelGGL(k_quantize_fp8<LAT_MOE_BF16>, grid, block, 0, st, x, nb, bpr, cols, codes, scales);
  else
    hipLaunchKernelGGL(k_quantize_fp8<LAT_MOE_F16>, grid, block, 0, st, x, nb, bpr, cols, codes, scales);
  return hipGetLastError();
}

}  // namespace latmoe
