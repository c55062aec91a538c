// What follows a 16-bit product in registers: bias, activation, residual, and
// the stores of y and of its q8_1 blocks.
#pragma once

#include "block_fp8.h"

namespace latmoe {

// erfc by Abramowitz and Stegun's 7.1.26: with t = 1 / (1 + p x), x >= 0,
// (a1 t + ... + a5 t^5) exp(-x^2) is within 1.5e-7 of it, so that the
// activation is within 0.75e-7 |v|: as near as an fp32 v is to a sum of
// products, for a third of the operations of erff.
__device__ __forceinline__ float gelu(float v) {
  const float x = fabsf(v) * 0.70710678f;
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.3275911f * x);
  const float p = t * (0.254829592f + t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
  const float q = 0.5f * p * __expf(-x * x);
  return v * (v < 0.f ? q : 1.0f - q);
}

// (1 + tanh z) / 2 = 1 / (1 + exp(-2 z)).
__device__ __forceinline__ float gelu_tanh(float v) {
  const float z2 = v * (1.59576912f + 0.07135481f * v * v);
  return v / (1.0f + __expf(-z2));
}

// n values; the activation is the same for a whole launch.
template <int n>
__device__ __forceinline__ void activate(float* v, int act) {
  if (act == LAT_MOE_ACT_NONE) return;
  if (act == LAT_MOE_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = silu(v[i]);
  } else if (act == LAT_MOE_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];
  } else if (act == LAT_MOE_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = gelu(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = gelu_tanh(v[i]);
  }
}

__device__ __forceinline__ float load1(const void* base, int type, int64_t elem) {
  if (type == LAT_MOE_F32) return static_cast<const float*>(base)[elem];
  const uint32_t b = static_cast<const uint16_t*>(base)[elem];
  return type == LAT_MOE_BF16 ? __builtin_bit_cast(float, b << 16) : half_bits_to_float(b);
}
__device__ __forceinline__ void store1(void* base, int type, int64_t elem, float v) {
  if (type == LAT_MOE_F32) static_cast<float*>(base)[elem] = v;
  else static_cast<uint16_t*>(base)[elem] = (uint16_t)(type == LAT_MOE_BF16 ? pack_bf16(v, v) : pack_f16(v, v));
}
__device__ __forceinline__ void load8(const void* base, int type, int64_t elem, float* v) {
  if (type == LAT_MOE_F32) {
    Raw8<LAT_MOE_F32> r;
    r.load(base, elem);
    r.values(v);
  } else if (type == LAT_MOE_BF16) {
    Raw8<LAT_MOE_BF16> r;
    r.load(base, elem);
    r.values(v);
  } else {
    Raw8<LAT_MOE_F16> r;
    r.load(base, elem);
    r.values(v);
  }
}

typedef float v4f_unaligned __attribute__((ext_vector_type(4), aligned(4)));

// Bias of the 16 columns from n on, a multiple of 16 (columns past `count` have none).
__device__ __forceinline__ void load_bias16(const float* bias, int n, int count, float* b) {
  const int live = bias ? count - n : 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) b[i] = 0.f;
  if (live >= 16) {
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const v4f_unaligned p = *reinterpret_cast<const v4f_unaligned*>(bias + n + i);
      b[i] = p[0];
      b[i + 1] = p[1];
      b[i + 2] = p[2];
      b[i + 3] = p[3];
    }
  } else if (live > 0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) b[i] = i < live ? bias[n + min(i, live - 1)] : 0.f;
  }
}

// Residual and y of row t's 16 columns from n on, a multiple of 16: v is what
// the activation left, and becomes what is rounded.  n < e.N.  `lds`: 16 floats
// of the lane's own, where rows that are not whole pieces take their values
// from one by one (unrolled, that path would be most of a kernel's code).
__device__ __forceinline__ void finish16(const Epilogue16& e, int64_t t, int n, float* v, float* lds) {
  if (e.vec) {
#pragma unroll
    for (int h = 0; h < 16; h += 8) {
      if (n + h < e.N) {
        if (e.residual) {
          float r[8];
          load8(e.residual, e.residual_type, t * e.residual_stride + n + h, r);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[h + i] += r[i];
        }
        if (e.y) store8(e.y, e.y_type, t * e.y_stride + n + h, v + h);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) lds[i] = v[i];
    const int live = min(16, e.N - n);
#pragma unroll 1
    for (int i = 0; i < live; ++i) {
      float u = lds[i];
      if (e.residual) u += load1(e.residual, e.residual_type, t * e.residual_stride + n + i);
      if (e.y) store1(e.y, e.y_type, t * e.y_stride + n + i, u);
      lds[i] = u;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = lds[i];
  }
}
constexpr int kFinishPitch = 17;  // floats of a lane's part: no two lanes of a piece in one bank

// q8_1 block of a row of 32 columns that two lanes hold, 16 each (`first`: the
// block's first 16); `other` is the distance between the two lanes.
__device__ __forceinline__ void store_q8(uint8_t* block, const float* v, bool first, int other, bool live) {
#pragma clang fp contract(off)
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = max_or_nan(amax, fabsf(v[i]));
  amax = max_or_nan(amax, __shfl_xor(amax, other));
  const float d = amax / 127.0f;
  const float id = d != 0.0f ? 1.0f / d : 0.0f;
  uint32_t pk[4];
  int sum = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    pk[q] = pack_codes(round_half_away(v[4 * q] * id), round_half_away(v[4 * q + 1] * id),
                       round_half_away(v[4 * q + 2] * id), round_half_away(v[4 * q + 3] * id));
    sum = __builtin_amdgcn_sdot4((int)pk[q], 0x01010101, sum, false);
  }
  sum += __shfl_xor(sum, other);
  if (!live) return;
  uint32_t* w = reinterpret_cast<uint32_t*>(block) + (first ? 1 : 5);
#pragma unroll
  for (int q = 0; q < 4; ++q) w[q] = pk[q];
  if (first)
    *reinterpret_cast<uint32_t*>(block) =
        float_to_half_bits(d) | (float_to_half_bits(fp32_barrier(d * (float)sum)) << 16);
}

}  // namespace latmoe
