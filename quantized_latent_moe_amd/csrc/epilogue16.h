// The 16-bit products' MFMA, and what follows a product in registers: bias, activation, residual, and
// the stores of y and of its q8_1 blocks.
#pragma once

#include "block_fp8.h"

namespace latmoe {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));

template <int TYPE>
__device__ __forceinline__ v4f mfma16(v4i a, v4i b, v4f c) {
  if constexpr (TYPE == LAT_MOE_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}


// v Phi(v), Phi the normal distribution: the tail Phi(-x), x = |v|, is half of
// 2^(-x P(x)).  P is of degree 9, fitted by reweighted least squares to
// -log2(2 Phi(-x)) / x on 0 <= x <= 6 so that the tail is within 4e-9 and within
// 5e-6 of itself; beyond, x P(x) grows faster than the true exponent, and the
// tail is below 1e-9.  Rounding adds most where the tail is one half: with the
// hardware's exp2 (1 ulp) the activation is within 1e-7 |v| (computed over 6e6
// values: 0.99e-7; a rational formula for erfc, 0.75e-7 by itself, was off by
// 3e-7 in fp32, from terms of either sign that add up to one).  Small x leaves
// the exponent near 0, where nothing is lost, and v - v tail is one operation.
__device__ __forceinline__ float gelu(float v) {
  const float x = fabsf(v);
  float p = 0x1.871d9p-26f;
  p = fmaf(p, x, -0x1.7d8edcp-21f);
  p = fmaf(p, x, 0x1.3dbb42p-17f);
  p = fmaf(p, x, -0x1.1e8916p-14f);
  p = fmaf(p, x, 0x1.0a2c64p-12f);
  p = fmaf(p, x, 0x1.98799ep-15f);
  p = fmaf(p, x, -0x1.cac5f2p-8f);
  p = fmaf(p, x, 0x1.addc56p-5f);
  p = fmaf(p, x, 0x1.d63b9cp-2f);
  p = fmaf(p, x, 0x1.26aed2p+0f);
  // the largest finite half: infinity times a tail of 0 would be a NaN
  const float e = __builtin_amdgcn_exp2f(-(x * p)), half = fminf(0.5f * v, 0x1.fffffep+127f);
  return v < 0.f ? half * e : fmaf(-half, e, v);
}

// v / (1 + exp(-z)), with the hardware's reciprocal (1 ulp; a correctly rounded
// quotient is ten operations, and a gated tile has 64 of them a lane).  In
// units of 2^-23: 1 for exp2 and 0.63 z for its argument, which count 1 - s, s
// the quotient, 1 for the reciprocal, 1/2 each for the sum and the product; z of
// the tanh is off by up to 2.75 z.  The reciprocal of sums past 2^126, z < -87.3, is 0.
__device__ __forceinline__ float logistic_times(float v, float z) {
  return v * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}
// (1 + tanh z) / 2 = 1 / (1 + exp(-2 z)).
__device__ __forceinline__ float gelu_tanh(float v) {
  return logistic_times(v, v * (1.59576912f + 0.07135481f * v * v));
}

// n values; the activation is the same for a whole launch.
template <int n>
__device__ __forceinline__ void activate(float* v, int act) {
  if (act == LAT_MOE_ACT_NONE) return;
  if (act == LAT_MOE_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = logistic_times(v[i], v[i]);
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
// Pieces of rows that begin anywhere (rows of an odd length): the memory takes
// 16 bytes at any address of the element's alignment.
typedef float v4f_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t v4u_any __attribute__((ext_vector_type(4), aligned(2)));

// The 8 columns from n on of a row of `count` columns (those past it: zeros).
__device__ __forceinline__ void load_bias8(const float* bias, int n, int count, float* b) {
  const int live = bias ? count - n : 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = 0.f;
  if (live >= 8) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const v4f_any p = *reinterpret_cast<const v4f_any*>(bias + n + i);
      b[i] = p[0];
      b[i + 1] = p[1];
      b[i + 2] = p[2];
      b[i + 3] = p[3];
    }
  } else if (live > 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = i < live ? bias[n + min(i, live - 1)] : 0.f;
  }
}

// Eight values of a type known at run time, as they lie in memory.
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
struct Piece8 {
  v4u a, b;  // b: fp32 only
  __device__ __forceinline__ void load(const void* base, int type, int64_t elem) {
    if (type == LAT_MOE_F32) {
      const v4u_any* p = reinterpret_cast<const v4u_any*>(static_cast<const float*>(base) + elem);
      a = p[0];
      b = p[1];
    } else {
      a = *reinterpret_cast<const v4u_any*>(static_cast<const uint16_t*>(base) + elem);
    }
  }
  __device__ __forceinline__ void add_to(int type, float* v) const {
    if (type == LAT_MOE_F32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] += __builtin_bit_cast(float, (uint32_t)a[i]);
        v[4 + i] += __builtin_bit_cast(float, (uint32_t)b[i]);
      }
    } else if (type == LAT_MOE_BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] += __builtin_bit_cast(float, (uint32_t)a[i] << 16);
        v[2 * i + 1] += __builtin_bit_cast(float, (uint32_t)a[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] += half_bits_to_float(a[i] & 0xffffu);
        v[2 * i + 1] += half_bits_to_float(a[i] >> 16);
      }
    }
  }
};
__device__ __forceinline__ void store8_any(void* base, int type, int64_t elem, const float* v) {
  if (type == LAT_MOE_F32) {
    v4f_any* p = reinterpret_cast<v4f_any*>(static_cast<float*>(base) + elem);
    p[0] = v4f_any{v[0], v[1], v[2], v[3]};
    p[1] = v4f_any{v[4], v[5], v[6], v[7]};
  } else {
    const bool bf = type == LAT_MOE_BF16;
    v4u_any w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf ? pack_bf16(v[2 * i], v[2 * i + 1]) : pack_f16(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<v4u_any*>(static_cast<uint16_t*>(base) + elem) = w;
  }
}

// q8_1 block of a row of 32 columns that four neighbouring lanes hold, 8 each.
__device__ __forceinline__ void store_q8(uint8_t* block, const float* v, int part, bool live) {
#pragma clang fp contract(off)
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max_or_nan(amax, fabsf(v[i]));
  amax = max_or_nan(amax, __shfl_xor(amax, 1));
  amax = max_or_nan(amax, __shfl_xor(amax, 2));
  const float d = amax / 127.0f;
  const float id = d != 0.0f ? 1.0f / d : 0.0f;
  uint32_t pk[2];
  int sum = 0;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    pk[q] = pack_codes(round_half_away(v[4 * q] * id), round_half_away(v[4 * q + 1] * id),
                       round_half_away(v[4 * q + 2] * id), round_half_away(v[4 * q + 3] * id));
    sum = __builtin_amdgcn_sdot4((int)pk[q], 0x01010101, sum, false);
  }
  sum += __shfl_xor(sum, 1);
  sum += __shfl_xor(sum, 2);
  if (!live) return;
  uint32_t* w = reinterpret_cast<uint32_t*>(block);
  w[1 + 2 * part] = pk[0];
  w[2 + 2 * part] = pk[1];
  if (part == 0) w[0] = float_to_half_bits(d) | (float_to_half_bits(fp32_barrier(d * (float)sum)) << 16);
}

// What follows a wave's 16 FA weight rows x 16 FB tokens of a product.  The
// results pass through LDS, 16 tokens at a time, so that a row's columns lie in
// neighbouring lanes (whole lines are stored, 8 columns a lane) and so that the
// code is there once and not for each register: unrolled it took 6 us a tile to
// fetch.  A wave uses its own part of LDS, whose accesses are in order.
//   first  bias, activation and the gated product, where there are any
//   then   residual and stores; the residual's loads run ahead by 16 tokens
template <int FA, int FB, bool GATED>
struct TileEpilogue {
  static constexpr int OUT = GATED ? 8 * FA : 16 * FA;  // columns of the wave
  static constexpr int kLanes = OUT / 8;                // of a row
  static constexpr int kRows = 64 / kLanes;             // at a time
  static constexpr int kPasses = 16 / kRows;            // of 16 tokens
  static constexpr int kPitch = 16 * FA + 4;            // floats between rows: no two lanes of a store in one bank
  static constexpr int kBytes = 16 * kPitch * 4;        // of LDS for a wave
  static_assert(64 % kLanes == 0 && 16 % kRows == 0, "whole rows");

  // Bias, activation and the gated product of the 16 tokens in LDS, in place.
  static __device__ __forceinline__ void shape(const Epilogue16& e, float* lds, int n, int lane) {
    const int c = (lane % kLanes) * 8, row = lane / kLanes;
    float b[8], bu[8];
    load_bias8(e.bias, n, e.N, b);
    if (GATED) load_bias8(e.bias ? e.bias + e.N : nullptr, n, e.N, bu);
#pragma unroll 1
    for (int p = 0; p < kPasses; ++p) {
      v4f* at = reinterpret_cast<v4f*>(lds + (kRows * p + row) * kPitch + c);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = at[i / 4][i % 4] + b[i];
      activate<8>(v, e.act);
      if constexpr (GATED) {
        const v4f* up = reinterpret_cast<const v4f*>(lds + (kRows * p + row) * kPitch + OUT + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= up[i / 4][i % 4] + bu[i];
      }
      at[0] = v4f{v[0], v[1], v[2], v[3]};
      at[1] = v4f{v[4], v[5], v[6], v[7]};
    }
  }
  static __device__ __forceinline__ bool shapes(const Epilogue16& e) {
    return GATED || e.bias || e.act != LAT_MOE_ACT_NONE;
  }

  // A wave's part that lies inside the matrix whole, with y of type YT (none:
  // q8_1 alone) and a residual of type RT (or none): types and places are known
  // here, and pointers go from row to row.  The general form below takes 50 VALU
  // operations for each 8 columns, 4 us for a tile of 256 x 256; this one 15.
  // Calls that have to take the general one (us, by 4096 x 4096 with 21000
  // tokens): fp32 y with a 16-bit residual 624 (fp32 residual, here: 615), y or
  // residual of the other 16-bit type 551 to 595 (of the same: 543 to 564),
  // q8_1 with a residual 596 to 602 or beside an fp32 y 612 (alone: 545).
  static constexpr int kNone = -1;
  template <int YT, int RT>
  static __device__ __forceinline__ void run_whole(const Epilogue16& e, const v4f (&acc)[FA][FB], float* lds, int n0,
                                                   int64_t t0, int lane) {
    const int r = lane & 15, g = lane >> 4;
    const int c = (lane % kLanes) * 8, row = lane / kLanes, n = n0 + c;
    constexpr int kDepth = RT == LAT_MOE_F32 ? 1 : 3;  // 16 tokens' residual on their way
    constexpr int kSizeY = YT == LAT_MOE_F32 ? 4 : 2, kSizeR = RT == LAT_MOE_F32 ? 4 : 2;
    Piece8 ahead[kDepth][kPasses];
    const int64_t step_y = kRows * e.y_stride * kSizeY, step_r = kRows * e.residual_stride * kSizeR;
    char* y = YT == kNone ? nullptr : static_cast<char*>(e.y) + ((t0 + row) * e.y_stride + n) * kSizeY;
    const char* res = nullptr;
    if (RT != kNone) res = static_cast<const char*>(e.residual) + ((t0 + row) * e.residual_stride + n) * kSizeR;
    auto fetch = [&](int j) {
      if constexpr (RT != kNone) {
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
          ahead[j % kDepth][p].load(res, RT, 0);
          res += step_r;
        }
      }
    };
#pragma unroll
    for (int j = 0; j < kDepth && j < FB; ++j) fetch(j);
#pragma unroll 1
    for (int j = 0; j < FB; ++j) {
      Piece8 now[kPasses];
#pragma unroll
      for (int q = 0; q < FB; ++q)
        if (q == j) {
#pragma unroll
          for (int i = 0; i < FA; ++i) *reinterpret_cast<v4f*>(lds + r * kPitch + 16 * i + 4 * g) = acc[i][q];
          // keeps the branches apart: merged, they would need registers with an index
          asm volatile("; turn %0" ::"n"(q));
          if constexpr (RT != kNone) {
#pragma unroll
            for (int p = 0; p < kPasses; ++p) now[p] = ahead[q % kDepth][p];
          }
          if (q + kDepth < FB) fetch(q + kDepth);
        }
      if (shapes(e)) shape(e, lds, n, lane);
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const v4f* at = reinterpret_cast<const v4f*>(lds + (kRows * p + row) * kPitch + c);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = at[i / 4][i % 4];
        if constexpr (RT != kNone) now[p].add_to(RT, v);
        if constexpr (YT != kNone) {
          store8_any(y, YT, 0, v);
          y += step_y;
        } else if constexpr (!GATED) {
          const int64_t t = t0 + 16 * j + kRows * p + row;
          store_q8(e.y_q8 + (t * (e.N / 32) + n / 32) * kQ81Bytes, v, lane & 3, true);
        }
      }
    }
  }

  // n0: the wave's first column; t0: its first token; live: its tokens inside
  // the matrix; TYPE: the operands' type.
  template <int TYPE>
  static __device__ __forceinline__ void run(const Epilogue16& e, const v4f (&acc)[FA][FB], float* lds, int n0,
                                             int64_t t0, int live, int lane) {
    if (live >= 16 * FB && n0 + OUT <= e.N) {
      if (GATED || !e.y_q8) {
        if (GATED || !e.residual) {
          if (e.y_type == TYPE) return run_whole<TYPE, kNone>(e, acc, lds, n0, t0, lane);
          if (e.y_type == LAT_MOE_F32) return run_whole<LAT_MOE_F32, kNone>(e, acc, lds, n0, t0, lane);
        } else if constexpr (!GATED) {
          if (e.y_type == TYPE && e.residual_type == TYPE) return run_whole<TYPE, TYPE>(e, acc, lds, n0, t0, lane);
          if (e.y_type == TYPE && e.residual_type == LAT_MOE_F32)
            return run_whole<TYPE, LAT_MOE_F32>(e, acc, lds, n0, t0, lane);
          if (e.y_type == LAT_MOE_F32 && e.residual_type == LAT_MOE_F32)
            return run_whole<LAT_MOE_F32, LAT_MOE_F32>(e, acc, lds, n0, t0, lane);
        }
      } else if constexpr (!GATED) {
        if (!e.y && !e.residual) return run_whole<kNone, kNone>(e, acc, lds, n0, t0, lane);
      }
    }
    run_any(e, acc, lds, n0, t0, live, lane);
  }

  // Any other part: at the matrix's ends, q8_1 beside y, mixed types.
  static __device__ __forceinline__ void run_any(const Epilogue16& e, const v4f (&acc)[FA][FB], float* lds, int n0,
                                                 int64_t t0, int live, int lane) {
    const int r = lane & 15, g = lane >> 4;
    const int c = (lane % kLanes) * 8, row = lane / kLanes, n = n0 + c;
    const bool inside = n < e.N, whole = n + 8 <= e.N;
    Piece8 ahead[kPasses];
    auto fetch = [&](int j, int p) {
      const int tl = 16 * j + kRows * p + row;
      if (e.residual && whole && tl < live) ahead[p].load(e.residual, e.residual_type, (t0 + tl) * e.residual_stride + n);
    };
#pragma unroll
    for (int p = 0; p < kPasses; ++p) fetch(0, p);
#pragma unroll 1
    for (int j = 0; j < FB; ++j) {
      if (16 * j >= live) break;  // the whole wave
#pragma unroll
      for (int q = 0; q < FB; ++q)
        if (q == j) {
#pragma unroll
          for (int i = 0; i < FA; ++i) *reinterpret_cast<v4f*>(lds + r * kPitch + 16 * i + 4 * g) = acc[i][q];
          // keeps the branches apart: merged, they would need registers with an index
          asm volatile("; turn %0" ::"n"(q));
        }
      if (shapes(e)) shape(e, lds, n, lane);
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int tl = 16 * j + kRows * p + row;
        const int64_t t = t0 + tl;
        const bool stored = inside && tl < live;
        float* at = lds + (kRows * p + row) * kPitch + c;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = reinterpret_cast<v4f*>(at)[i / 4][i % 4];
        if (stored) {
          if (whole) {
            if (e.residual) ahead[p].add_to(e.residual_type, v);
            if (e.y) store8_any(e.y, e.y_type, t * e.y_stride + n, v);
          } else {
            const int count = e.N - n;
#pragma unroll 1
            for (int i = 0; i < count; ++i) {
              float u = at[i];
              if (e.residual) u += load1(e.residual, e.residual_type, t * e.residual_stride + n + i);
              if (e.y) store1(e.y, e.y_type, t * e.y_stride + n + i, u);
              at[i] = u;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = reinterpret_cast<v4f*>(at)[i / 4][i % 4];
          }
        }
        if (j + 1 < FB) fetch(j + 1, p);
        if (!GATED && e.y_q8)
          store_q8(e.y_q8 + (t * (e.N / 32) + n / 32) * kQ81Bytes, v, lane & 3, stored);
      }
    }
  }
};

}  // namespace latmoe
