// Device helpers of the e4m3 formats: rows with a scale for each 128 values,
// and loads and stores of eight fp32, bf16 or fp16 values.
#pragma once

#include "lat_moe_internal.h"

namespace latmoe {

constexpr int kFp8Block = LAT_MOE_FP8_BLOCK;
constexpr float kE4m3Max = 448.0f;
constexpr float kFp8AmaxMin = kE4m3Max * 0x1p-126f;  // keeps 448 / amax finite, also for a block of zeros

typedef float v2f __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef int v8i __attribute__((ext_vector_type(8)));

// A launch has fewer than 2^32 threads along a dimension: more than 2^20
// workgroups come in rows of 2^20, and those past the last one return at once.
inline dim3 grid_of(int64_t workgroups) {
  constexpr int64_t kRow = 1 << 20;
  return workgroups <= kRow ? dim3((unsigned)workgroups) : dim3(kRow, (unsigned)((workgroups + kRow - 1) / kRow));
}
__device__ __forceinline__ uint32_t workgroup_number() { return blockIdx.y * gridDim.x + blockIdx.x; }

// Scale of a block whose largest magnitude is amax, and what its values are
// multiplied by to get the codes: two quotients of amax, each rounded once.
__device__ __forceinline__ float fp8_scale(float amax, float& inverse) {
  const float a = fmaxf(amax, kFp8AmaxMin);
  inverse = kE4m3Max / a;
  return a / kE4m3Max;
}

// Four values within +-448 to e4m3, byte i = value i (nearest, ties to even).
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// Eight e4m3 codes to bf16, exactly (NaN stays NaN).
__device__ __forceinline__ v8bf widen(int lo, int hi) {
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Eight values of type TYPE as they lie in memory (16 bytes each for the
// 16-bit types, 32 for fp32), and their fp32 values.
template <int TYPE>
struct Raw8 {
  uint4 a, b;  // b: fp32 only
  __device__ __forceinline__ void load(const void* base, int64_t elem) {
    if constexpr (TYPE == LAT_MOE_F32) {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + elem);
      a = p[0];
      b = p[1];
    } else {
      a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + elem);
    }
  }
  __device__ __forceinline__ void zero() { a = b = uint4{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ void values(float* v) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
    if constexpr (TYPE == LAT_MOE_F32) {
      const uint32_t u[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = __builtin_bit_cast(float, w[i]);
        v[4 + i] = __builtin_bit_cast(float, u[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (TYPE == LAT_MOE_BF16) {
          v[2 * i] = __builtin_bit_cast(float, w[i] << 16);
          v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
        } else {
          v[2 * i] = half_bits_to_float(w[i] & 0xffffu);
          v[2 * i + 1] = half_bits_to_float(w[i] >> 16);
        }
      }
    }
  }
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f){a, b}, v2bf));
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f){a, b}, v2h));
}

// Eight values rounded to `type` (nearest, ties to even) and stored.
__device__ __forceinline__ void store8(void* base, int type, int64_t elem, const float* v) {
  if (type == LAT_MOE_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + elem);
    p[0] = float4{v[0], v[1], v[2], v[3]};
    p[1] = float4{v[4], v[5], v[6], v[7]};
  } else {
    uint4 w;
    if (type == LAT_MOE_BF16)
      w = uint4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
    else
      w = uint4{pack_f16(v[0], v[1]), pack_f16(v[2], v[3]), pack_f16(v[4], v[5]), pack_f16(v[6], v[7])};
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + elem) = w;
  }
}

__device__ __forceinline__ float amax8(const float* v) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

// The larger value, or a NaN if one is (v_maximum3_f32): what a q8_1 block's
// scale is made of, since its codes cannot hold a NaN.
__device__ __forceinline__ float max_or_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// Largest value of each aligned group of 4 or 16 lanes, in all of its lanes.
template <int LANES>
__device__ __forceinline__ float group_max(float m) {
#pragma unroll
  for (int s = 1; s < LANES; s <<= 1) m = fmaxf(m, __shfl_xor(m, s));
  return m;
}

// A 16-lane group's 128 values (8 a lane, zeros past the row's end) to e4m3:
// the lane's 8 codes, and the block's scale.
__device__ __forceinline__ uint2 e4m3_block(const float* v, float& scale) {
  float id;
  scale = fp8_scale(group_max<16>(amax8(v)), id);
  return uint2{pack_e4m3(v[0] * id, v[1] * id, v[2] * id, v[3] * id),
               pack_e4m3(v[4] * id, v[5] * id, v[6] * id, v[7] * id)};
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + __expf(-g)); }

}  // namespace latmoe
