// Routing by scores with a bias, in groups:
//
//   s = softmax or sigmoid of the logits (64 bits, rounded once to fp32)
//   c = s + bias; groups by their largest c, or the sum of their two largest;
//   the k largest c of the best groups; w = scale s (/ the sum of the picks' s)
//
// The scores are in 64 bits because their order decides: among 21000 rows of
// 256 scores a few neighbours lie within an fp32 rounding of each other, and a
// pick would depend on how exp rounds.
//
// Up to 256 experts, 16 picks and 16 groups, 16 lanes take a token, so that a
// wave's VALU works on four and a maximum is four DPP steps.  What bounds it:
// many tokens the VALU (21000 x 256 in 8 groups, 8 picks: 1420 operations for
// four tokens, of them 37 for a score of each lane and 43 for a round of
// picking; 19.8 us, without groups 16, 5268 x 128 without groups 5.6), few
// tokens the rounds, one behind the other (4 x 128 5.1 us, without groups 4.2).
// A wave for each token takes 36 to 44 us for 21000 x 256, and 5.8 for 4 x 128.
#include "block_fp8.h"
#include "exp64.h"

namespace latmoe {
namespace {

constexpr int kWaves = 4;
constexpr float kLowest = -3.402823466e38f;

// Across each row of 16 lanes, in all of them (quad swaps, half-row and row
// mirrors; every lane has a source, so that the step is part of the operation).
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}
__device__ __forceinline__ int row_max(int v) {
  v = max(v, dpp<0xB1>(v));
  v = max(v, dpp<0x4E>(v));
  v = max(v, dpp<0x141>(v));
  return max(v, dpp<0x140>(v));
}
__device__ __forceinline__ int row_min(int v) {
  v = min(v, dpp<0xB1>(v));
  v = min(v, dpp<0x4E>(v));
  v = min(v, dpp<0x141>(v));
  return min(v, dpp<0x140>(v));
}
template <int CTRL>
__device__ __forceinline__ double dpp_add(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)dpp<CTRL>((int)(uint32_t)b), hi = (uint32_t)dpp<CTRL>((int)(uint32_t)(b >> 32));
  return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double row_sum(double v) {
  return dpp_add<0x140>(dpp_add<0x141>(dpp_add<0x4E>(dpp_add<0xB1>(v))));
}

// Whole numbers in the order of the floats (no NaN, no -0), and back.
__device__ __forceinline__ int ordered(float f) {
  const int b = __builtin_bit_cast(int, f);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int k) {
  return __builtin_bit_cast(float, k ^ ((k >> 31) & 0x7fffffff));
}

// exp(x), |x| <= 700.  The coefficients are kept in scalar registers, which a
// multiply-add can read; as constants the compiler moves each of them, twice 32
// bits, before each use.
struct Exp64 {
  double c[kExp64Coefficients];
  __device__ __forceinline__ Exp64() {
#pragma unroll
    for (int i = 0; i < kExp64Coefficients; ++i) {
      c[i] = kExp64[i];
      asm("" : "+s"(c[i]));
    }
  }
  __device__ __forceinline__ double operator()(double x) const {
    const double n = exp64_power(x);
    return __builtin_amdgcn_ldexp(exp64_series(c, exp64_rest(x, n)), (int)n);
  }
};
// 1 / d, 0 < d <= e^700: the hardware's estimate (at least 20 bits) and two steps that double them.
__device__ __forceinline__ double inverse64(double d) {
  double q = __builtin_amdgcn_rcp(d);
#pragma unroll
  for (int i = 0; i < 2; ++i) q = __builtin_fma(q, __builtin_fma(-d, q, 1.0), q);
  return q;
}

// A logit as it counts: the largest finite number for +inf, -inf for NaN.
__device__ __forceinline__ float counted(float l) { return l > -INFINITY ? fminf(l, -kLowest) : -INFINITY; }

// What is left of the score once the row's statistics are known: exp(l - top),
// to be divided by the row's sum, for the softmax, the score itself for the
// sigmoid.  Beyond |x| = 700 both are 0 or 1 in fp32, for -inf too.
__device__ __forceinline__ double sigmoid64(const Exp64& e, float l) {
  return inverse64(1.0 + e((double)__builtin_amdgcn_fmed3f(-l, -700.0f, 700.0f)));
}
__device__ __forceinline__ double softmax64(const Exp64& e, float l, float top) {
  return e(fmax((double)l - (double)top, -700.0));
}

// Candidate of a score as an ordered whole number; closed experts have the
// lowest finite one: -inf enters the sum and is cut.
__device__ __forceinline__ int candidate(float l, float s, float bias) {
  const float b = bias > -INFINITY ? bias : -INFINITY;  // NaN: closed
  return ordered(__builtin_amdgcn_fmed3f(s + (l > -INFINITY ? b : -INFINITY), kLowest, -kLowest));
}
// Below every candidate: an expert that cannot be picked.
constexpr int kNone = (int)0x80000000u;
// The fp32 sum of a group's two largest; a second at the lowest value (closed, or
// a bias of that value) counts as 0.
__device__ __forceinline__ int group_score(int m1, int m2, int lowest, bool top2) {
  return top2 && m2 > lowest ? ordered(unordered(m1) + unordered(m2)) : m1;
}

// What the other lanes of the wave have written to LDS is read after this.
__device__ __forceinline__ void wave_lds() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// Weight of a pick: its score once more (a lane for each pick).
template <bool SIGMOID>
__device__ __forceinline__ double picked(const RouterExArgs& a, const Exp64& e, const float* row, int pick, float top,
                                         double scale) {
  const float l = counted(row[pick]), b = a.bias ? a.bias[pick] : 0.f;
  const float s = (float)(SIGMOID ? sigmoid64(e, l) : softmax64(e, l, top) * scale);
  return l > -INFINITY && b > -INFINITY ? (double)s : 0.0;
}

// Up to 256 experts, 16 picks and 16 groups: a row of 16 lanes takes a token,
// four tokens a wave.  Lane l holds experts 64 j + 4 l .. + 3 for each of Q
// quads j, so that a row's loads are whole lines.  The candidates are in LDS,
// where a lane finds a group's members and the quad that it has to look at;
// registers hold each quad's largest.  In each of k rounds the row's largest
// quad maximum comes by four DPP steps, each lane that holds it looks for the
// member in its quad, the lowest id among them is picked (four more steps), and
// its lane takes it out of its quad.
template <int Q, bool SIGMOID>
__global__ __launch_bounds__(64 * kWaves) void k_router_ex16(const RouterExArgs a) {
  __shared__ __align__(16) int lds[kWaves][4][64 * Q];
  __shared__ __align__(16) int group_lds[kWaves][4][16];
  const int lane = threadIdx.x & 63, l = lane & 15, wave = threadIdx.x >> 6;
  const int64_t t = ((int64_t)workgroup_number() * kWaves + wave) * 4 + (lane >> 4);
  const bool live = t < a.T;
  if (__builtin_amdgcn_ballot_w64(live) == 0) return;  // whole waves; a wave uses its own LDS alone
  const float* row = a.logits + (live ? t : a.T - 1) * a.E;
  int* c = lds[wave][lane >> 4] + 4 * l;
  const int E = a.E;
  const Exp64 exp64;

  float x[Q][4], bias[Q][4];
  if (E % 4 == 0) {
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const int e = 64 * j + 4 * l;
      v4f v = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, b = {0.f, 0.f, 0.f, 0.f};
      if (e < E) {
        v = *reinterpret_cast<const v4f*>(row + e);
        if (a.bias) b = *reinterpret_cast<const v4f*>(a.bias + e);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[j][i] = v[i];
        bias[j][i] = b[i];
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < Q; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 64 * j + 4 * l + i;
        x[j][i] = e < E ? row[e] : -INFINITY;
        bias[j][i] = a.bias && e < E ? a.bias[e] : 0.f;
      }
  }
#pragma unroll
  for (int j = 0; j < Q; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) x[j][i] = counted(x[j][i]);
  const int lowest = ordered(kLowest);
  float top = kLowest;
  double scale = 1.0;
  int quad[Q];
  auto place = [&](int j, const float* s) {
    v4i v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = candidate(x[j][i], s[i], bias[j][i]);
    if (64 * Q > E) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = 64 * j + 4 * l + i < E ? v[i] : kNone;
    }
    *reinterpret_cast<v4i*>(c + 64 * j) = v;
    quad[j] = max(max(v[0], v[1]), max(v[2], v[3]));
  };
  if constexpr (SIGMOID) {
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      float s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = (float)sigmoid64(exp64, x[j][i]);
      place(j, s);
    }
  } else {
#pragma unroll
    for (int j = 0; j < Q; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, x[j][i]);
    top = unordered(row_max(ordered(top)));
    double p[Q][4], sum = 0.0;
#pragma unroll
    for (int j = 0; j < Q; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[j][i] = softmax64(exp64, x[j][i], top);
        sum += p[j][i];
      }
    scale = inverse64(row_sum(sum));
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      float s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = (float)(p[j][i] * scale);
      place(j, s);
    }
  }
  wave_lds();

  if (a.top_groups < a.groups) {
    // a few lanes to a group, each with every share-th member
    const int G = a.groups, size = E / G;
    const int share = G > 8 ? 1 : G > 4 ? 2 : G > 2 ? 4 : 8;
    const int g = l / share;
    int m1 = kNone, m2 = kNone;
    auto merge = [&](int o1, int o2) {
      m2 = max(min(m1, o1), max(m2, o2));
      m1 = max(m1, o1);
    };
    if (g < G) {
      const int* member = lds[wave][lane >> 4] + g * size;
#pragma unroll 4
      for (int i = l % share; i < size; i += share) {
        const int v = member[i];
        m2 = max(m2, min(m1, v));
        m1 = max(m1, v);
      }
    }
    if (share > 1) merge(dpp<0xB1>(m1), dpp<0xB1>(m2));
    if (share > 2) merge(dpp<0x4E>(m1), dpp<0x4E>(m2));
    if (share > 4) merge(dpp<0x141>(m1), dpp<0x141>(m2));
    const int score = group_score(m1, m2, lowest, a.top2);
    int* gs = group_lds[wave][lane >> 4];
    if (l % share == 0 && g < G) gs[g] = score;
    wave_lds();
    int better = 0;
#pragma unroll 4
    for (int q = 0; q < G; ++q) {
      const int v = gs[q];
      better += v > score || (v == score && q < g);
    }
    // bit share * g of the row's sixteen: whether group g is kept
    const uint64_t all = __builtin_amdgcn_ballot_w64(better < a.top_groups);
    const uint32_t kept = (uint32_t)(all >> (lane & 48)) & 0xffffu;
    const float inverse = 1.0f / (float)size;
    // (e + 1/2) / size is never near a whole number; ids past the last, which stay
    // out whatever this says, are in groups past the last and shift by any number
    auto is_kept = [&](int e) { return (kept >> (((int)(((float)e + 0.5f) * inverse) * share) & 31) & 1u) != 0; };
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const int e = 64 * j + 4 * l;
      v4i v = *reinterpret_cast<const v4i*>(c + 64 * j);
      if (size % 4 == 0) {  // a quad lies in one group
        if (!is_kept(e)) v = v4i{kNone, kNone, kNone, kNone};
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = is_kept(e + i) ? v[i] : kNone;
      }
      *reinterpret_cast<v4i*>(c + 64 * j) = v;
      quad[j] = max(max(v[0], v[1]), max(v[2], v[3]));
    }
    wave_lds();
  }

  int pick = 0;
  for (int r = 0; r < a.k; ++r) {
    int best = quad[0];
#pragma unroll
    for (int j = 1; j < Q; ++j) best = max(best, quad[j]);
    const int most = row_max(best);
    int at = 0;  // the lane's first quad that holds its best
#pragma unroll
    for (int j = Q - 1; j > 0; --j) at = quad[j] == best ? 64 * j : at;
    at = quad[0] == best ? 0 : at;
    const v4i v = *reinterpret_cast<const v4i*>(c + at);
    const int i = v[0] == best ? 0 : v[1] == best ? 1 : v[2] == best ? 2 : 3;
    const int e = at + 4 * l + i;
    const int id = row_min(best == most ? e : 0x7fffffff);
    if (id == e) {
      c[at + i] = kNone;
      const int m = max(max(i == 0 ? kNone : v[0], i == 1 ? kNone : v[1]),
                        max(i == 2 ? kNone : v[2], i == 3 ? kNone : v[3]));
#pragma unroll
      for (int j = 0; j < Q; ++j) quad[j] = at == 64 * j ? m : quad[j];
    }
    pick = l == r ? id : pick;
  }
  const bool mine = l < a.k;
  double w = mine ? picked<SIGMOID>(a, exp64, row, pick, top, scale) : 0.0;
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
// for each group.  P: experts a lane (E <= 64 P).  In 8 groups, 8 picks:
// 512 experts take 9.6 us for 4 tokens, 21 for 5268 and 57 for 21000, 1024
// experts 15, 33 and 100 (their bytes: 17), bound by the rounds' reductions
// over 64 lanes.
template <int P>
__global__ __launch_bounds__(64 * kWaves) void k_router_ex(const RouterExArgs a) {
  __shared__ int lds[kWaves][64 * P];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)workgroup_number() * kWaves + wave;
  if (t >= a.T) return;  // whole waves; a wave uses its own part of LDS alone
  const float* row = a.logits + t * a.E;
  const Exp64 exp64;
  float x[P];
  int c[P];
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
    for (int i = 0; i < P; ++i) sum += softmax64(exp64, x[i], top);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
    scale = inverse64(sum);
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + 64 * i;
    const float b = a.bias && e < a.E ? a.bias[e] : 0.f;
    const double p = a.sigmoid ? sigmoid64(exp64, x[i]) : softmax64(exp64, x[i], top);
    c[i] = e < a.E ? candidate(x[i], (float)(p * scale), b) : kNone;
    lds[wave][e] = c[i];
  }
  wave_lds();
  if (a.top_groups < a.groups) {
    const int size = a.E / a.groups;
    int score = kNone;
    if (lane < a.groups) {
      int m1 = kNone, m2 = kNone;
      for (int i = 0; i < size; ++i) {
        const int v = lds[wave][lane * size + i];
        m2 = max(m2, min(m1, v));
        m1 = max(m1, v);
      }
      score = group_score(m1, m2, ordered(kLowest), a.top2);
    }
    int better = 0;
    for (int g = 0; g < a.groups; ++g) {
      const int v = __shfl(score, g);
      better += v > score || (v == score && g < lane);
    }
    const uint64_t kept = __builtin_amdgcn_ballot_w64(lane < a.groups && better < a.top_groups);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = lane + 64 * i;
      if (e < a.E && !((kept >> (e / size)) & 1)) c[i] = kNone;
    }
  }
  int pick = 0;
  for (int j = 0; j < a.k; ++j) {
    int bv = kNone, bi = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (c[i] > bv) {
        bv = c[i];
        bi = lane + 64 * i;
      }
    // the wave's largest, then the lowest id that has it
    int most = row_max(bv);
    most = max(most, __shfl_xor(most, 16));
    most = max(most, __shfl_xor(most, 32));
    int id = row_min(bv == most ? bi : 0x7fffffff);
    id = min(id, __shfl_xor(id, 16));
    id = min(id, __shfl_xor(id, 32));
#pragma unroll
    for (int i = 0; i < P; ++i) c[i] = lane + 64 * i == id ? kNone : c[i];
    pick = lane == j ? id : pick;
  }
  const bool mine = lane < a.k;
  double w = 0.0;
  if (mine) w = a.sigmoid ? picked<true>(a, exp64, row, pick, top, scale) : picked<false>(a, exp64, row, pick, top, scale);
  double total = w;
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
    auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, st, a); };
    if (a.E <= 64) run(a.sigmoid ? k_router_ex16<1, true> : k_router_ex16<1, false>);
    else if (a.E <= 128) run(a.sigmoid ? k_router_ex16<2, true> : k_router_ex16<2, false>);
    else if (a.E <= 192) run(a.sigmoid ? k_router_ex16<3, true> : k_router_ex16<3, false>);
    else run(a.sigmoid ? k_router_ex16<4, true> : k_router_ex16<4, false>);
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
