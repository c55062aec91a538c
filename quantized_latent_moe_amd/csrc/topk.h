// Largest values and their indices across lanes.
#pragma once

#include "lat_moe_internal.h"

namespace latmoe {

// (value, index) of the better of two candidates: larger value, then lower index.
__device__ __forceinline__ void better(float& v, int& i, float ov, int oi) {
  if (ov > v || (ov == v && oi < i)) {
    v = ov;
    i = oi;
  }
}

// One DPP step of the wave reduction: combine with the lane the control word
// selects (rows outside row_mask keep their own pair).
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ void dpp_step(float& v, int& i) {
  const int vb = __builtin_bit_cast(int, v);
  const float ov = __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(vb, vb, CTRL, ROW_MASK, 0xF, false));
  const int oi = __builtin_amdgcn_update_dpp(i, i, CTRL, ROW_MASK, 0xF, false);
  better(v, i, ov, oi);
}

// Wave-wide best (value, index), returned to every lane: DPP within the VALU
// (quad swaps, half-row and row mirrors, row broadcasts 15 and 31) leaves the
// result in lane 63, read back as a scalar.
__device__ __forceinline__ void wave_best(float& v, int& i) {
  dpp_step<0xB1, 0xF>(v, i);   // quad_perm [1,0,3,2]
  dpp_step<0x4E, 0xF>(v, i);   // quad_perm [2,3,0,1]
  dpp_step<0x141, 0xF>(v, i);  // row_half_mirror
  dpp_step<0x140, 0xF>(v, i);  // row_mirror
  dpp_step<0x142, 0xA>(v, i);  // row_bcast:15 into rows 1 and 3
  dpp_step<0x143, 0xC>(v, i);  // row_bcast:31 into rows 2 and 3
  v = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
  i = __builtin_amdgcn_readlane(i, 63);
}

// One DPP step that takes the larger value.
template <int CTRL>
__device__ __forceinline__ float dpp_max(float v) {
  const int b = __builtin_bit_cast(int, v);
  return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(b, b, CTRL, 0xF, 0xF, false)));
}
template <int CTRL>
__device__ __forceinline__ int dpp_min(int v) {
  return min(v, __builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ double dpp_add(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const int lo = (int)(uint32_t)b, hi = (int)(uint32_t)(b >> 32);
  const uint32_t l = (uint32_t)__builtin_amdgcn_update_dpp(lo, lo, CTRL, 0xF, 0xF, false);
  const uint32_t h = (uint32_t)__builtin_amdgcn_update_dpp(hi, hi, CTRL, 0xF, 0xF, false);
  return v + __builtin_bit_cast(double, (uint64_t)h << 32 | l);
}
// Across each row of 16 lanes, in all of them.
__device__ __forceinline__ float row_max(float v) {
  return dpp_max<0x140>(dpp_max<0x141>(dpp_max<0x4E>(dpp_max<0xB1>(v))));
}
__device__ __forceinline__ int row_min(int v) {
  return dpp_min<0x140>(dpp_min<0x141>(dpp_min<0x4E>(dpp_min<0xB1>(v))));
}
__device__ __forceinline__ double row_sum(double v) {
  return dpp_add<0x140>(dpp_add<0x141>(dpp_add<0x4E>(dpp_add<0xB1>(v))));
}

}  // namespace latmoe
