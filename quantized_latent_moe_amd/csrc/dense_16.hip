// Products of 16-bit rows with 16-bit weights: the dense projection with bias,
// activation and residual, and the gated pair.
//
//   y[t][n] = act(sum over k of x[t][k] w[n][k] + bias[n]) + residual[t][n]
//   h[t][f] = act(gate) * up
//
// A workgroup of four waves takes 64 weight rows (gated: 32 gate rows and the
// same columns' up rows) x 64 tokens, in steps of 64 values of K.
#include "epilogue16.h"

namespace latmoe {
namespace {

constexpr int kStep = 64;          // K per step
constexpr int kRowBytes = 2 * kStep;

typedef _Float16 v8h __attribute__((ext_vector_type(8)));

template <int TYPE>
__device__ __forceinline__ v4f mfma16(v4i a, v4i b, v4f c) {
  if constexpr (TYPE == LAT_MOE_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

template <int TYPE, bool GATED>
__global__ __launch_bounds__(256) void k_dense_16(const Dense16Args a) {
  __shared__ __align__(16) uint8_t As[64 * kRowBytes], Bs[64 * kRowBytes];
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t number = workgroup_number();
  if (number >= (uint32_t)a.n_nt * (uint32_t)a.n_tt) return;
  constexpr int COLS = GATED ? 32 : 64;
  const int n0 = (int)(number % a.n_nt) * COLS;
  const int64_t t0 = (int64_t)(number / a.n_nt) * 64;
  const uint16_t* xp = static_cast<const uint16_t*>(a.x);
  const uint16_t* wp = static_cast<const uint16_t*>(a.w);
  v4f acc[4] = {};
  for (int k0 = 0; k0 < a.K; k0 += kStep) {
    for (int p = tid; p < 64 * 8; p += 256) {
      const int row = p >> 3, k = k0 + (p & 7) * 8;
      uint4 va = {0, 0, 0, 0}, vb = {0, 0, 0, 0};
      const int n = n0 + (GATED ? row & 31 : row);
      if (n < a.N && k < a.K)
        va = *reinterpret_cast<const uint4*>(wp + ((int64_t)n + (GATED && row >= 32 ? a.N : 0)) * a.K + k);
      if (t0 + row < a.T && k < a.K) vb = *reinterpret_cast<const uint4*>(xp + (t0 + row) * a.x_stride + k);
      *reinterpret_cast<uint4*>(As + row * kRowBytes + (p & 7) * 16) = va;
      *reinterpret_cast<uint4*>(Bs + row * kRowBytes + (p & 7) * 16) = vb;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const v4i b = *reinterpret_cast<const v4i*>(Bs + (16 * wave + r) * kRowBytes + (4 * h + g) * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const v4i w = *reinterpret_cast<const v4i*>(As + (16 * i + r) * kRowBytes + (4 * h + g) * 16);
        acc[i] = mfma16<TYPE>(w, b, acc[i]);
      }
    }
    __syncthreads();
  }
  // transposed among the lane groups: lane (r, g) then holds fragment g's 16 columns of token r
  float v[16];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = __builtin_bit_cast(uint32_t, (float)acc[i][e]);
    transpose4(q);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * i + e] = __builtin_bit_cast(float, q[i]);
  }
  const int64_t t = t0 + 16 * wave + r;
  float b[16];
  if constexpr (GATED) {
    const int n = n0 + 16 * (g & 1);
    load_bias16(a.e.bias ? a.e.bias + (g < 2 ? 0 : a.N) : nullptr, n, a.N, b);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += b[i];
    if (g < 2) activate<16>(v, a.e.act);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= __shfl_xor(v[i], 32);
    if (g < 2 && t < a.T && n < a.N) finish16(a.e, t, n, v);
  } else {
    const int n = n0 + 16 * g;
    const bool live = t < a.T && n < a.N;
    load_bias16(a.e.bias, n, a.N, b);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += b[i];
    activate<16>(v, a.e.act);
    if (live) finish16(a.e, t, n, v);
    if (a.e.y_q8) store_q8(a.e.y_q8 + (t * (a.N / 32) + n / 32) * kQ81Bytes, v, !(g & 1), 16, live);
  }
}

}  // namespace

hipError_t launch_dense_16(Dense16Args a, int type, bool gated, int num_cus, hipStream_t st) {
  const int cols = gated ? 32 : 64;
  a.n_nt = (a.N + cols - 1) / cols;
  a.n_tt = (int)((a.T + 63) / 64);
  const dim3 grid = grid_of((int64_t)a.n_nt * a.n_tt), block(256);
  if (type == LAT_MOE_BF16) {
    if (gated) hipLaunchKernelGGL((k_dense_16<LAT_MOE_BF16, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_dense_16<LAT_MOE_BF16, false>), grid, block, 0, st, a);
  } else {
    if (gated) hipLaunchKernelGGL((k_dense_16<LAT_MOE_F16, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_dense_16<LAT_MOE_F16, false>), grid, block, 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace latmoe
