// Products of 16-bit rows with 16-bit weights for few tokens (decode): the
// formulas of the tile kernel, arranged to stream the weights.
//
// A workgroup takes its weight rows whole: 16 waves deal K among themselves,
// load fragments straight from memory into registers, and add their partial
// sums in LDS at the end, in wave order, so that the result does not depend on
// timing.
//
// The 16 places of an MFMA operand are four weight rows (four tokens on the
// other side) times four slices of K, and only the products of equal slices, on
// the diagonal, count: a quarter of the matrix unit's work, which is idle here
// anyway.  In return four rows make a workgroup, so that few weight rows still
// fill the chip, and four neighbouring lanes load 64 neighbouring bytes of a
// row.  (With 16 rows to an operand neighbouring lanes are in different rows,
// and a CU was seen to load 16 bytes a cycle, 35 GB/s: 4 x 4096 by 128 took
// 7.3 us.)
//
// What bounds it: launch, the latency of one read and the join; then the
// weights' rate.  In a captured graph 4 x 4096 by 128 takes 2.9 us, by 1024
// 3.2, by 4096 4.8 (weights from the last-level cache; 6.9 with the residual and
// whatever else ran between), 4 x 8192 by 8192 21 us (134 MB, 6.4 TB/s),
// 16 x 4096 by 4096 6.9 us, the gated pair 4 x 4096 by 2 x 2048 4.9 us.
#include "dense16_tiles.h"
#include "epilogue16.h"

namespace latmoe {
namespace {

constexpr int kWaves = 16;
constexpr int kStep = 128;  // K of an MFMA: 4 slices of 32

// Sum over each four neighbouring lanes, in all of them.
__device__ __forceinline__ float quad_sum(float v) {
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xF, 0xF, true));
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x4E, 0xF, 0xF, true));
  return v;
}

// FR fragments of four weight rows (gated: half of them gate rows, half the
// same columns' up rows) and TF of four tokens; U steps of K in flight.
template <int TYPE, int FR, int TF, bool GATED, int U>
__global__ __launch_bounds__(64 * kWaves) void k_dense_16_small(const Dense16Args a) {
  constexpr int COLS = GATED ? 2 * FR : 4 * FR, TOKENS = 4 * TF;  // of the workgroup
  __shared__ float red[kWaves][FR * TF * 16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = (lane >> 2) & 3;  // the lane's row within a fragment
  const int n0 = (int)blockIdx.x * COLS, cols = min(COLS, a.N - n0);
  const int64_t t0 = (int64_t)blockIdx.y * TOKENS;
  const int tokens = (int)min((int64_t)TOKENS, a.T - t0);
  const int row_w = 2 * a.K, row_x = 2 * (int)a.x_stride;
  const uint16_t* w = static_cast<const uint16_t*>(a.w) + (int64_t)n0 * a.K;
  const rsrc_t rw = make_rsrc(w, (uint32_t)cols * row_w);
  const rsrc_t ru = GATED ? make_rsrc(w + (int64_t)a.N * a.K, (uint32_t)cols * row_w) : rw;
  const rsrc_t rx = make_rsrc(static_cast<const uint16_t*>(a.x) + t0 * a.x_stride,
                              (uint32_t)(tokens - 1) * row_x + 2 * a.K);
  const int chunk = (4 * (lane >> 4) + (lane & 3)) * 16;  // the lane's bytes within a step

  v4f acc[FR][TF] = {};
  for (int k0 = wave * U; k0 * kStep < a.K; k0 += kWaves * U) {
    v4i wa[U][FR], xa[U][TF];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = (k0 + u) * (2 * kStep) + chunk;
      const bool in = c < row_w;
      // rows past the last and chunks past a row's end are read as zeros
#pragma unroll
      for (int f = 0; f < FR; ++f) {
        const int row = 4 * (GATED ? f % (FR / 2) : f) + i;
        const uint4 v = buf_u128(GATED && f >= FR / 2 ? ru : rw, in && row < cols ? row * row_w + c : kOutOfRange, 0);
        wa[u][f] = v4i{(int)v.x, (int)v.y, (int)v.z, (int)v.w};
      }
#pragma unroll
      for (int f = 0; f < TF; ++f) {
        const int t = 4 * f + i;
        const uint4 v = buf_u128(rx, in && t < tokens ? t * row_x + c : kOutOfRange, 0);
        xa[u][f] = v4i{(int)v.x, (int)v.y, (int)v.z, (int)v.w};
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int f = 0; f < FR; ++f)
#pragma unroll
        for (int j = 0; j < TF; ++j) acc[f][j] = mfma16<TYPE>(wa[u][f], xa[u][j], acc[f][j]);
  }
  // Lane 16 i + 4 j + s holds row i's products with token j in its element s.
#pragma unroll
  for (int f = 0; f < FR; ++f)
#pragma unroll
    for (int j = 0; j < TF; ++j) {
      const v4f d = acc[f][j];
      const int s = lane & 3;
      const float v = quad_sum(s == 0 ? d[0] : s == 1 ? d[1] : s == 2 ? d[2] : d[3]);
      if (s == 0) red[wave][(f * TF + j) * 16 + (lane >> 2)] = v;
    }
  __syncthreads();

  // row n of token t, within the workgroup
  auto total = [&](int n, int t) {
    const int at = ((n >> 2) * TF + (t >> 2)) * 16 + 4 * (n & 3) + (t & 3);
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < kWaves; ++q) v += red[q][at];
    return v;
  };
  for (int o = tid; o < COLS * TOKENS; o += 64 * kWaves) {
    const int t = o / COLS, c = o % COLS, n = n0 + c;
    const bool live = t < tokens && c < cols;  // a whole q8_1 block of a token, or none of it
    const Epilogue16& e = a.e;
    float v = total(c, t);
    if (e.bias && live) v += e.bias[n];
    activate<1>(&v, e.act);
    if constexpr (GATED) {
      float u = total(COLS + c, t);
      if (e.bias && live) u += e.bias[a.N + n];
      v *= u;
    }
    const int64_t row = t0 + t;
    if (live) {
      if (e.residual) v += load1(e.residual, e.residual_type, row * e.residual_stride + n);
      if (e.y) store1(e.y, e.y_type, row * e.y_stride + n, v);
    }
    if constexpr (!GATED && COLS == 32) {
#pragma clang fp contract(off)
      if (e.y_q8) {
        // 32 lanes hold one q8_1 block
        float amax = fabsf(v);
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) amax = max_or_nan(amax, __shfl_xor(amax, s));
        const float d = amax / 127.0f;
        const float id = d != 0.0f ? 1.0f / d : 0.0f;
        const int q = round_half_away(v * id);
        int sum = q;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) sum += __shfl_xor(sum, s);
        if (live) {
          uint8_t* blk = e.y_q8 + (row * (a.N / 32) + n / 32) * kQ81Bytes;
          blk[4 + c] = (uint8_t)q;
          if (c == 0)
            *reinterpret_cast<uint32_t*>(blk) =
                float_to_half_bits(d) | (float_to_half_bits(fp32_barrier(d * (float)sum)) << 16);
        }
      }
    }
  }
}

template <int TYPE, int FR, int TF, bool GATED>
hipError_t run(const Dense16Args& a, hipStream_t st) {
  constexpr int COLS = GATED ? 2 * FR : 4 * FR, kTwo = FR * TF * 4 + 2 * (FR + TF) * 4 <= 96;
  const dim3 grid((unsigned)((a.N + COLS - 1) / COLS), (unsigned)((a.T + 4 * TF - 1) / (4 * TF)));
  const dim3 block(64 * kWaves);
  // two steps in flight where a wave has as many and the registers hold them
  if constexpr (kTwo) {
    if (a.K > kWaves * kStep) {
      hipLaunchKernelGGL((k_dense_16_small<TYPE, FR, TF, GATED, 2>), grid, block, 0, st, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((k_dense_16_small<TYPE, FR, TF, GATED, 1>), grid, block, 0, st, a);
  return hipGetLastError();
}

template <int TYPE, bool GATED, int TF>
hipError_t launch_rows(const Dense16Args& a, int num_cus, hipStream_t st) {
  if constexpr (!GATED && TF <= 2)
    if (a.e.y_q8) return run<TYPE, 8, TF, false>(a, st);  // a q8_1 block is 32 columns
  const int fr = dense16_small_rows(a.T, GATED ? 2 * (int64_t)a.N : a.N, num_cus) / 4;
  if constexpr (!GATED)
    if (fr == 1) return run<TYPE, 1, TF, false>(a, st);
  if constexpr (TF == 4)
    if (fr == 4) return run<TYPE, 4, TF, GATED>(a, st);
  return run<TYPE, 2, TF, GATED>(a, st);
}

template <int TYPE, bool GATED>
hipError_t launch(const Dense16Args& a, int num_cus, hipStream_t st) {
  if (a.T <= 4) return launch_rows<TYPE, GATED, 1>(a, num_cus, st);
  if (a.T <= 8 || a.e.y_q8) return launch_rows<TYPE, GATED, 2>(a, num_cus, st);
  return launch_rows<TYPE, GATED, 4>(a, num_cus, st);
}

}  // namespace

hipError_t launch_dense_16_small(const Dense16Args& a, int type, bool gated, int num_cus, hipStream_t st) {
  if (type == LAT_MOE_BF16)
    return gated ? launch<LAT_MOE_BF16, true>(a, num_cus, st) : launch<LAT_MOE_BF16, false>(a, num_cus, st);
  return gated ? launch<LAT_MOE_F16, true>(a, num_cus, st) : launch<LAT_MOE_F16, false>(a, num_cus, st);
}

}  // namespace latmoe
