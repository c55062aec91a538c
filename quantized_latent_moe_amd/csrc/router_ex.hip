// Routing by scores with a bias, in groups:
//
//   s = softmax or sigmoid of the logits (64 bits, rounded once to fp32)
//   c = s + bias; groups by their largest c, or the sum of their two largest;
//   the k largest c of the best groups; w = scale s (/ the sum of the picks' s)
//
// The scores are in 64 bits because their order decides: among 21000 rows of
// 256 scores a few neighbours lie within an fp32 rounding of each other.
//
// One wave a token.  Lane l holds experts l, l + 64, ...; a lane for each group
// ranks the groups, and each of k rounds takes the best candidate left.
#include "block_fp8.h"

namespace latmoe {
namespace {

constexpr int kWaves = 4;
constexpr float kLowest = -3.402823466e38f;

// P: experts a lane (E <= 64 P).
template <int P>
__global__ __launch_bounds__(64 * kWaves) void k_router_ex(const RouterExArgs a) {
  __shared__ float cs[kWaves][64 * P];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)workgroup_number() * kWaves + wave;
  if (t >= a.T) return;  // whole waves; a wave uses its own part of cs alone
  const float* row = a.logits + t * a.E;
  float l[P], c[P], s[P];
  float top = kLowest;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + 64 * i;
    const float v = e < a.E ? row[e] : -INFINITY;
    l[i] = v > -INFINITY ? fminf(v, -kLowest) : -INFINITY;  // NaN: closed
    top = fmaxf(top, l[i]);
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) top = fmaxf(top, __shfl_xor(top, m));
  double p[P], sum = 0.0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const double v = l[i];
    p[i] = l[i] == -INFINITY ? 0.0 : a.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - (double)top);
    sum += p[i];
  }
  if (!a.sigmoid) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
#pragma unroll
    for (int i = 0; i < P; ++i) p[i] = sum > 0.0 ? p[i] / sum : 0.0;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + 64 * i;
    s[i] = (float)p[i];
    const float b = a.bias && e < a.E ? a.bias[e] : 0.f;
    const float v = fminf(s[i] + b, -kLowest);
    const bool open = l[i] > -INFINITY && b > -INFINITY;
    c[i] = open ? fmaxf(v, kLowest) : kLowest;
    if (!open) s[i] = 0.f;
    cs[wave][e] = c[i];
  }
  uint64_t kept = ~0ull;
  if (a.top_groups < a.groups) {
    const int size = a.E / a.groups;
    float score = -INFINITY;
    if (lane < a.groups) {
      float m1 = -INFINITY, m2 = -INFINITY;
      for (int i = 0; i < size; ++i) {
        const float v = cs[wave][lane * size + i];
        m2 = fmaxf(m2, fminf(m1, v));
        m1 = fmaxf(m1, v);
      }
      score = a.top2 ? m1 + (m2 > kLowest ? m2 : 0.f) : m1;
    }
    int better = 0;
    for (int g = 0; g < a.groups; ++g) {
      const float v = __shfl(score, g);
      better += v > score || (v == score && g < lane);
    }
    kept = __ballot(lane < a.groups && better < a.top_groups);
    const int sz = size;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = lane + 64 * i;
      if (e < a.E && !((kept >> (e / sz)) & 1)) c[i] = -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (lane + 64 * i >= a.E) c[i] = -INFINITY;
  int my_idx = 0;
  float my_s = 0.f;
  for (int j = 0; j < a.k; ++j) {
    float bv = -INFINITY, bs = 0.f;
    int bi = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (c[i] > bv) {
        bv = c[i];
        bs = s[i];
        bi = lane + 64 * i;
      }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const float ov = __shfl_xor(bv, m), os = __shfl_xor(bs, m);
      const int oi = __shfl_xor(bi, m);
      if (ov > bv || (ov == bv && oi < bi)) {
        bv = ov;
        bs = os;
        bi = oi;
      }
    }
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (lane + 64 * i == bi) c[i] = -INFINITY;
    if (lane == j) {
      my_idx = bi;
      my_s = bs;
    }
  }
  double w = lane < a.k ? (double)my_s : 0.0, total = w;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) total += __shfl_xor(total, m);
  if (a.renormalise) w = total > 0.0 ? w / total : 0.0;
  if (lane < a.k) {
    a.idx[t * a.k + lane] = my_idx;
    a.w[t * a.k + lane] = (float)(w * (double)a.scale);
  }
}

}  // namespace

hipError_t launch_router_ex(const RouterExArgs& a, hipStream_t st) {
  const dim3 grid = grid_of((a.T + kWaves - 1) / kWaves), block(64 * kWaves);
  if (a.E <= 64) hipLaunchKernelGGL(k_router_ex<1>, grid, block, 0, st, a);
  else if (a.E <= 128) hipLaunchKernelGGL(k_router_ex<2>, grid, block, 0, st, a);
  else if (a.E <= 256) hipLaunchKernelGGL(k_router_ex<4>, grid, block, 0, st, a);
  else if (a.E <= 512) hipLaunchKernelGGL(k_router_ex<8>, grid, block, 0, st, a);
  else hipLaunchKernelGGL(k_router_ex<16>, grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace latmoe
