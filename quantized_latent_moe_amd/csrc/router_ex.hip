// Routing by scores with a bias, in groups:
//
//   s = softmax or sigmoid of the logits (64 bits, rounded once to fp32)
//   c = s + bias; groups by their largest c, or the sum of their two largest;
//   the k largest c of the best groups; w = scale s (/ the sum of the picks' s)
//
// The scores are in 64 bits because their order decides: among 21000 rows of
// 256 scores a few neighbours lie within an fp32 rounding of each other, and a
// pick would depend on how exp rounds.
#include "block_fp8.h"
#include "topk.h"

namespace latmoe {
namespace {

constexpr int kWaves = 4;
constexpr float kLowest = -3.402823466e38f;

// exp(x), |x| <= 700, within 2^-51: x = n ln 2 + r, and the polynomial of degree
// 10 through exp at the Chebyshev points of |r| <= ln 2 / 2 (the library's exp
// takes twice the operations, for its last bit and its ends).
__device__ __forceinline__ double exp64(double x) {
  const double n = __builtin_rint(x * 0x1.71547652b82fep+0);
  const double r = __builtin_fma(n, -0x1.62e42fefa39efp-1, x);
  double p = 2.7626357241447223e-07;
  p = __builtin_fma(p, r, 2.764018079620985e-06);
  p = __builtin_fma(p, r, 2.4801504346997686e-05);
  p = __builtin_fma(p, r, 0.00019841170270440067);
  p = __builtin_fma(p, r, 0.0013888888932488599);
  p = __builtin_fma(p, r, 0.008333333385667782);
  p = __builtin_fma(p, r, 0.04166666666657314);
  p = __builtin_fma(p, r, 0.16666666666554406);
  p = __builtin_fma(p, r, 0.5000000000000006);
  p = __builtin_fma(p, r, 1.0000000000000067);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_amdgcn_ldexp(p, (int)n);
}
// 1 / d, 0 < d <= e^700: the hardware's estimate (at least 20 bits) and two steps that double them.
__device__ __forceinline__ double inverse64(double d) {
  double q = __builtin_amdgcn_rcp(d);
#pragma unroll
  for (int i = 0; i < 2; ++i) q = __builtin_fma(q, __builtin_fma(-d, q, 1.0), q);
  return q;
}

// A logit as it counts: the largest finite number for +inf, -inf for NaN.
__device__ __forceinline__ float counted(float l) { return l > -INFINITY ? fminf(l, -kLowest) : -INFINITY; }

// What is left of the score once the row's statistics are known: exp(l - top)
// and 1 / sum for the softmax, l and 1 for the sigmoid.  Beyond |x| = 700 a
// score is 0 or 1 in fp32.
__device__ __forceinline__ double unscaled(float l, float top, bool sigmoid) {
  if (l == -INFINITY) return 0.0;
  if (sigmoid) return inverse64(1.0 + exp64(fmin(fmax(-(double)l, -700.0), 700.0)));
  return exp64(fmax((double)l - (double)top, -700.0));
}

// Candidate of a score; closed experts have the lowest.
__device__ __forceinline__ float candidate(float l, float s, float bias) {
  const bool open = l > -INFINITY && bias > -INFINITY;
  return open ? fmaxf(fminf(s + bias, -kLowest), kLowest) : kLowest;
}

// What the other lanes of the wave have written to LDS is read after this.
__device__ __forceinline__ void wave_lds() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// Up to 256 experts, 16 picks and 16 groups: a row of 16 lanes takes a token,
// four tokens a wave.  Lane l holds experts 64 j + 4 l .. + 3 for each of Q
// quads j, so that a row's loads are whole lines.  The candidates are in LDS,
// where a lane finds a group's members and the quad that it has to look at;
// registers hold each quad's largest.  In each of k rounds the row's largest
// quad maximum comes by four DPP steps, each lane that holds it looks for the
// member in its quad, the lowest id among them is picked (four more steps), and
// its lane takes it out of its quad.
template <int Q>
__global__ __launch_bounds__(64 * kWaves) void k_router_ex16(const RouterExArgs a) {
  __shared__ __align__(16) float lds[kWaves][4][64 * Q];
  __shared__ __align__(16) float group_lds[kWaves][4][16];
  const int lane = threadIdx.x & 63, l = lane & 15, wave = threadIdx.x >> 6;
  const int64_t t = ((int64_t)workgroup_number() * kWaves + wave) * 4 + (lane >> 4);
  if (__builtin_amdgcn_ballot_w64(t < a.T) == 0) return;  // whole waves; a wave uses its own LDS alone
  const bool live = t < a.T;
  const float* row = a.logits + (live ? t : a.T - 1) * a.E;
  float* c = lds[wave][lane >> 4];
  const int E = a.E;
  const bool fours = E % 4 == 0;

  float x[Q][4], bias[Q][4];
#pragma unroll
  for (int j = 0; j < Q; ++j) {
    const int e = 64 * j + 4 * l;
    if (fours) {
      v4f v = {0.f, 0.f, 0.f, 0.f}, b = v;
      if (e < E) {
        v = *reinterpret_cast<const v4f*>(row + e);
        if (a.bias) b = *reinterpret_cast<const v4f*>(a.bias + e);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[j][i] = v[i];
        bias[j][i] = b[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[j][i] = e + i < E ? row[e + i] : 0.f;
        bias[j][i] = a.bias && e + i < E ? a.bias[e + i] : 0.f;
      }
    }
  }
  float top = kLowest;
  double scale = 1.0;
#pragma unroll
  for (int j = 0; j < Q; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[j][i] = 64 * j + 4 * l + i < E ? counted(x[j][i]) : -INFINITY;
      top = fmaxf(top, x[j][i]);
    }
  float quad[Q];
  auto place = [&](int j, const double* p) {
    float m = -INFINITY;
    v4f v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = 64 * j + 4 * l + i < E ? candidate(x[j][i], (float)(p[i] * scale), bias[j][i]) : -INFINITY;
      m = fmaxf(m, v[i]);
    }
    *reinterpret_cast<v4f*>(c + 64 * j + 4 * l) = v;
    quad[j] = m;
  };
  if (a.sigmoid) {
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      double p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = unscaled(x[j][i], 0.f, true);
      place(j, p);
    }
  } else {
    top = row_max(top);
    double p[Q][4], sum = 0.0;
#pragma unroll
    for (int j = 0; j < Q; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[j][i] = unscaled(x[j][i], top, false);
        sum += p[j][i];
      }
    sum = row_sum(sum);
    scale = sum > 0.0 ? inverse64(sum) : 0.0;
#pragma unroll
    for (int j = 0; j < Q; ++j) place(j, p[j]);
  }
  wave_lds();

  if (a.top_groups < a.groups) {
    // a few lanes to a group, each with every share-th member
    const int G = a.groups, size = E / G;
    const int share = G > 8 ? 1 : G > 4 ? 2 : G > 2 ? 4 : 8;
    const int g = l / share;
    float m1 = -INFINITY, m2 = -INFINITY;
    if (g < G)
      for (int i = l % share; i < size; i += share) {
        const float v = c[g * size + i];
        m2 = fmaxf(m2, fminf(m1, v));
        m1 = fmaxf(m1, v);
      }
    auto merge = [&](float o1, float o2) {
      m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
      m1 = fmaxf(m1, o1);
    };
    if (share > 1) merge(__shfl_xor(m1, 1), __shfl_xor(m2, 1));
    if (share > 2) merge(__shfl_xor(m1, 2), __shfl_xor(m2, 2));
    if (share > 4) merge(__shfl_xor(m1, 4), __shfl_xor(m2, 4));
    const float score = a.top2 ? m1 + (m2 > kLowest ? m2 : 0.f) : m1;
    float* gs = group_lds[wave][lane >> 4];
    if (l % share == 0 && g < G) gs[g] = score;
    wave_lds();
    int better = 0;
    for (int q = 0; q < G; ++q) {
      const float v = gs[q];
      better += v > score || (v == score && q < g);
    }
    // bit share * g of the row's sixteen: whether group g is kept
    const uint64_t all = __builtin_amdgcn_ballot_w64(better < a.top_groups);
    const uint32_t kept = (uint32_t)(all >> (lane & 48)) & 0xffffu;
    const float inverse = 1.0f / (float)size;  // (e + 1/2) / size is never near a whole number
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const int e = 64 * j + 4 * l;
      v4f v = *reinterpret_cast<const v4f*>(c + e);
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int of = (int)(((float)(e + i) + 0.5f) * inverse);
        v[i] = kept >> (of * share) & 1u ? v[i] : -INFINITY;
        m = fmaxf(m, v[i]);
      }
      *reinterpret_cast<v4f*>(c + e) = v;
      quad[j] = m;
    }
    wave_lds();
  }

  int pick = 0;
  for (int r = 0; r < a.k; ++r) {
    float best = quad[0];
#pragma unroll
    for (int j = 1; j < Q; ++j) best = fmaxf(best, quad[j]);
    const float most = row_max(best);
    int e = 4 * l;  // the lane's first quad that holds its best
#pragma unroll
    for (int j = Q - 1; j >= 0; --j) e = quad[j] == best ? 64 * j + 4 * l : e;
    const v4f v = *reinterpret_cast<const v4f*>(c + e);
    const int i = v[0] == best ? 0 : v[1] == best ? 1 : v[2] == best ? 2 : 3;
    const int id = row_min(best == most ? e + i : 0x7fffffff);
    if (id == e + i) {
      c[id] = -INFINITY;
      const float m = fmaxf(fmaxf(i == 0 ? -INFINITY : v[0], i == 1 ? -INFINITY : v[1]),
                            fmaxf(i == 2 ? -INFINITY : v[2], i == 3 ? -INFINITY : v[3]));
#pragma unroll
      for (int j = 0; j < Q; ++j) quad[j] = e >> 6 == j ? m : quad[j];
    }
    if (l == r) pick = id;
  }
  // the picks' scores once more, a lane for each
  const bool mine = l < a.k;
  const float xl = mine ? counted(row[pick]) : -INFINITY;
  const float xb = a.bias && mine ? a.bias[pick] : 0.f;
  const float s = (float)(unscaled(xl, top, a.sigmoid) * scale);
  double w = xb > -INFINITY ? (double)s : 0.0;
  if (a.renormalise) {
    const double total = row_sum(w);
    w = total > 0.0 ? w / total : 0.0;
  }
  if (live && mine) {
    a.idx[t * a.k + l] = pick;
    a.w[t * a.k + l] = (float)(w * (double)a.scale);
  }
}

// Any other call: a wave takes a token, lane l experts l, l + 64, ...; a lane
// for each group.  P: experts a lane (E <= 64 P).
template <int P>
__global__ __launch_bounds__(64 * kWaves) void k_router_ex(const RouterExArgs a) {
  __shared__ float lds[kWaves][64 * P];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)workgroup_number() * kWaves + wave;
  if (t >= a.T) return;  // whole waves; a wave uses its own part of LDS alone
  const float* row = a.logits + t * a.E;
  float x[P], c[P];
  float top = kLowest;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + 64 * i;
    x[i] = e < a.E ? counted(row[e]) : -INFINITY;
    top = fmaxf(top, x[i]);
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) top = fmaxf(top, __shfl_xor(top, m));
  double scale = 1.0;
  if (!a.sigmoid) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < P; ++i) sum += unscaled(x[i], top, false);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
    scale = sum > 0.0 ? inverse64(sum) : 0.0;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + 64 * i;
    const float b = a.bias && e < a.E ? a.bias[e] : 0.f;
    c[i] = e < a.E ? candidate(x[i], (float)(unscaled(x[i], top, a.sigmoid) * scale), b) : -INFINITY;
    lds[wave][e] = c[i];
  }
  wave_lds();
  if (a.top_groups < a.groups) {
    const int size = a.E / a.groups;
    float score = -INFINITY;
    if (lane < a.groups) {
      float m1 = -INFINITY, m2 = -INFINITY;
      for (int i = 0; i < size; ++i) {
        const float v = lds[wave][lane * size + i];
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
    const uint64_t kept = __ballot(lane < a.groups && better < a.top_groups);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = lane + 64 * i;
      if (e < a.E && !((kept >> (e / size)) & 1)) c[i] = -INFINITY;
    }
  }
  int pick = 0;
  for (int j = 0; j < a.k; ++j) {
    float bv = -INFINITY;
    int bi = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (c[i] > bv) {
        bv = c[i];
        bi = lane + 64 * i;
      }
    wave_best(bv, bi);
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (lane + 64 * i == bi) c[i] = -INFINITY;
    if (lane == j) pick = bi;
  }
  const bool mine = lane < a.k;
  const float xl = mine ? counted(row[pick]) : -INFINITY;
  const float xb = a.bias && mine ? a.bias[pick] : 0.f;
  const float s = (float)(unscaled(xl, top, a.sigmoid) * scale);
  double w = xb > -INFINITY ? (double)s : 0.0, total = w;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) total += __shfl_xor(total, m);
  if (a.renormalise) w = total > 0.0 ? w / total : 0.0;
  if (mine) {
    a.idx[t * a.k + lane] = pick;
    a.w[t * a.k + lane] = (float)(w * (double)a.scale);
  }
}

}  // namespace

hipError_t launch_router_ex(const RouterExArgs& a, hipStream_t st) {
  const dim3 block(64 * kWaves);
  const bool groups = a.top_groups < a.groups;
  if (a.E <= 256 && a.k <= 16 && (!groups || a.groups <= 16)) {
    const dim3 grid = grid_of((a.T + 4 * kWaves - 1) / (4 * kWaves));
    if (a.E <= 64) hipLaunchKernelGGL(k_router_ex16<1>, grid, block, 0, st, a);
    else if (a.E <= 128) hipLaunchKernelGGL(k_router_ex16<2>, grid, block, 0, st, a);
    else if (a.E <= 192) hipLaunchKernelGGL(k_router_ex16<3>, grid, block, 0, st, a);
    else hipLaunchKernelGGL(k_router_ex16<4>, grid, block, 0, st, a);
    return hipGetLastError();
  }
  const dim3 grid = grid_of((a.T + kWaves - 1) / kWaves);
  if (a.E <= 64) hipLaunchKernelGGL(k_router_ex<1>, grid, block, 0, st, a);
  else if (a.E <= 128) hipLaunchKernelGGL(k_router_ex<2>, grid, block, 0, st, a);
  else if (a.E <= 256) hipLaunchKernelGGL(k_router_ex<4>, grid, block, 0, st, a);
  else if (a.E <= 512) hipLaunchKernelGGL(k_router_ex<8>, grid, block, 0, st, a);
  else hipLaunchKernelGGL(k_router_ex<16>, grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace latmoe
