// Products of e4m3 rows with e4m3 weights for few tokens (decode), and exact
// ones for few weight rows: the formulas of the tile kernel, arranged to stream
// the weights.
//
// Each weight is used for a few tokens only, so the time is that of reading
// the weights once, and the products are exact: codes are widened to bf16 for
// the bf16 MFMA, whatever the output type.  A workgroup takes 16 FR weight rows
// whole: its waves deal the blocks of K = 128 among themselves, load fragments
// straight from memory into registers (no LDS on the way in; a lane's two
// 16-byte pieces lie 64 bytes apart, so each load covers 64 contiguous bytes of
// a row), and add their partial sums in LDS at the end, in wave order: the
// result does not depend on timing.
//
// What bounds it: launch, the latency of one or two reads in a row, and the
// adding of partial sums; then the weights' rate.  In a captured graph a
// product of 4 tokens takes 2.9 us for 4096 x 1024 weights, 4.8 us for
// 1024 x 4096 (64 workgroups, two blocks of K a wave), 5.3 us for 4096 x 4096
// (16 MB, 3.2 TB/s), 14 us for 8192 x 8192 and 25 us for 16384 x 8192 (5.4 TB/s).
// With a q8_1 output, whose blocks are 32 columns, a workgroup takes 32 weight
// rows: 7.6 us for 1024 x 4096.
//
// Against the tiles (us, 16 | 17 .. 32 tokens here and in tiles):
//   4096 x 4096:  7.0 | 7.8 .. 9.6, bf16 tiles 8.7, fp32 (exact) tiles 13.4
//   8192 x 2048:  6.7 | 7.3 .. 9.4, bf16 tiles 6.0, fp32 (exact) tiles 8.4
// so a call for rounded outputs comes here up to 16 tokens, one for the fp32 y
// up to 32.  Larger batches come in groups of 32 tokens, one a workgroup; with a
// CU for each workgroup that beats the exact tiles, whose step of K is as long
// on one CU as on all (us here | tiles):
//   64 tokens, 1024 x 4096:  9.1 | 13.5, 128 tokens  9.6 | 13.8 (256 workgroups)
//   512 tokens, 256 x 8192: 17.3 | 24.4, 33 tokens, 2048 x 2048  5.7 | 8.2
// and with two on a CU it does not: 256 tokens, 1024 x 4096  16.5 | 13.8.
#include "block_fp8.h"

namespace latmoe {
namespace {

struct SmallArgs {
  const uint8_t* x;  // [T][K] e4m3, or null: the rows are h32
  const float* xs;
  const float* h32;  // [T][K] fp32 rows to be rounded to e4m3 here
  const uint8_t* w;
  const float* ws;
  float* y_f32;
  uint16_t* y_bf16;
  uint8_t* y_q8;
  int T, N, K, nb;
};

// Two 16-byte pieces of codes to four bf16 operands.
__device__ __forceinline__ void widen16(const uint4* p, v8bf* o) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    o[2 * h] = widen((int)p[h].x, (int)p[h].y);
    o[2 * h + 1] = widen((int)p[h].z, (int)p[h].w);
  }
}

// What a kernel computes: a projection of e4m3 rows; the gated pair (its 16
// weight rows are 8 gate rows and the same columns' 8 up rows, so that one
// fragment holds both and twice as many workgroups share the weights); a
// projection of fp32 rows that it rounds to e4m3 itself (every workgroup
// rounds them again, which for few tokens costs less than a launch between).
enum SmallMode : int { kRows = 0, kGatedPair = 1, kRound = 2 };

// Waves of a workgroup, each with TF blocks in flight.  For 16 tokens 16 waves
// with one block each take 3.0 us for 4096 x 1024 weights and 4.8 us for
// 8192 x 2048, eight with four each 3.6 and 5.7 us (the wave's own chain of
// blocks is as long, and few blocks leave it waiting for the last).
constexpr int small_waves(int tf) { return tf == 1 ? 16 : 8; }

// Token columns past T and weight rows past N hold zeros or a clamped row;
// they meet only results that are not stored.
template <int FR, int TF, int MODE>
__global__ __launch_bounds__(64 * small_waves(TF)) void k_dense_fp8_small(SmallArgs a) {
  constexpr bool GATED = MODE == kGatedPair;
  constexpr int kWaves = small_waves(TF), U = TF;  // U blocks in flight per wave
  constexpr int NF = GATED ? 8 : 16 * FR;          // output columns
  static_assert(!GATED || FR == 1, "one fragment of gate and up rows");
  static_assert(MODE != kRound || TF == 1, "rounding for 16 tokens");
  __shared__ __align__(16) float red[kWaves][FR * TF][64][4];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n0 = (int)blockIdx.x * NF;
  if (TF == 2) {  // the workgroup's 32 tokens
    const int64_t t0 = (int64_t)blockIdx.y * 32;
    a.x += t0 * a.K;
    a.xs += t0 * a.nb;
    a.T = min(a.T - (int)t0, 32);
    if (a.y_f32) a.y_f32 += t0 * a.N;
    if (a.y_bf16) a.y_bf16 += t0 * a.N;
    if (a.y_q8) a.y_q8 += t0 * (a.N / 32) * kQ81Bytes;
  }
  const int K = a.K, nb = a.nb;
  const int nbn = (a.N + kFp8Block - 1) / kFp8Block;

  rsrc_t rw[FR];
  int wrow[FR], wblk[FR];  // byte offset of the lane's weight row; of the scales of the lane's result rows
#pragma unroll
  for (int i = 0; i < FR; ++i) {
    const int base = min(n0 + 16 * i, a.N - 1);  // of the fragment's rows
    if (GATED) {
      const int live = min(8, a.N - base);
      rw[i] = make_rsrc(a.w + (int64_t)base * K, (uint32_t)(a.N + live) * (uint32_t)K);
      wrow[i] = (min(r & 7, live - 1) + (r < 8 ? 0 : a.N)) * K;
      wblk[i] = (base / kFp8Block + (g < 2 ? 0 : nbn)) * nb;
    } else {
      const int live = min(16, a.N - base);
      rw[i] = make_rsrc(a.w + (int64_t)base * K, (uint32_t)live * K);
      wrow[i] = min(r, live - 1) * K;
      wblk[i] = base / kFp8Block * nb;
    }
  }
  const rsrc_t rx = MODE == kRound ? make_rsrc(a.h32, (uint32_t)a.T * K * 4) : make_rsrc(a.x, (uint32_t)a.T * K);
  const rsrc_t rs = MODE == kRound ? rx : make_rsrc(a.xs, (uint32_t)a.T * nb * 4);
  const rsrc_t rws = make_rsrc(a.ws, (uint32_t)((GATED ? 2 : 1) * nbn * nb) * 4u);

  v4f acc[FR][TF] = {};
  for (int k0 = wave; k0 < nb; k0 += U * kWaves) {
    uint4 wa[U][FR][2], xa[U][TF][2], xh[U][MODE == kRound ? 8 : 1];
    float sx[U][TF], sw[U][FR];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = k0 + u * kWaves;
      const int c0 = kb * kFp8Block + 16 * g, c1 = c0 + 64;
      const bool in0 = c0 < K, in1 = c1 < K;  // false past the row's end, and so for every block past the last
#pragma unroll
      for (int i = 0; i < FR; ++i) {
        wa[u][i][0] = buf_u128(rw[i], in0 ? wrow[i] + c0 : kOutOfRange, 0);
        wa[u][i][1] = buf_u128(rw[i], in1 ? wrow[i] + c1 : kOutOfRange, 0);
        sw[u][i] = __builtin_bit_cast(float, buf_u32(rws, kb < nb ? (wblk[i] + kb) * 4 : kOutOfRange, 0));
      }
      if constexpr (MODE == kRound) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          xh[u][e] = buf_u128(rx, in0 && r < a.T ? (r * K + c0 + 4 * e) * 4 : kOutOfRange, 0);
          xh[u][4 + e] = buf_u128(rx, in1 && r < a.T ? (r * K + c1 + 4 * e) * 4 : kOutOfRange, 0);
        }
      } else {
#pragma unroll
        for (int j = 0; j < TF; ++j) {
          const int t = 16 * j + r;
          xa[u][j][0] = buf_u128(rx, in0 && t < a.T ? t * K + c0 : kOutOfRange, 0);
          xa[u][j][1] = buf_u128(rx, in1 && t < a.T ? t * K + c1 : kOutOfRange, 0);
          sx[u][j] = __builtin_bit_cast(float, buf_u32(rs, kb < nb && t < a.T ? (t * nb + kb) * 4 : kOutOfRange, 0));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (MODE == kRound) {
#pragma clang fp contract(off)
        // the four lanes of token r hold its block of 128 values
        float v[32], id;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t w[4] = {xh[u][e].x, xh[u][e].y, xh[u][e].z, xh[u][e].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) v[4 * e + i] = __builtin_bit_cast(float, w[i]);
        }
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(v[i]));
        amax = fmaxf(amax, __shfl_xor(amax, 16));
        amax = fmaxf(amax, __shfl_xor(amax, 32));
        sx[u][0] = fp8_scale(amax, id);
        uint32_t pk[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          pk[e] = pack_e4m3(v[4 * e] * id, v[4 * e + 1] * id, v[4 * e + 2] * id, v[4 * e + 3] * id);
        xa[u][0][0] = uint4{pk[0], pk[1], pk[2], pk[3]};
        xa[u][0][1] = uint4{pk[4], pk[5], pk[6], pk[7]};
      }
#pragma unroll
      for (int i = 0; i < FR; ++i) {
        v8bf fa[4];
        widen16(wa[u][i], fa);
#pragma unroll
        for (int j = 0; j < TF; ++j) {
          v8bf fb[4];
          widen16(xa[u][j], fb);
          v4f d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < 4; ++q) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[q], fb[q], d, 0, 0, 0);
          const float s = sx[u][j] * sw[u][i];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(s, d[e], acc[i][j][e]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < FR; ++i)
#pragma unroll
    for (int j = 0; j < TF; ++j) *reinterpret_cast<v4f*>(red[wave][i * TF + j][lane]) = acc[i][j];
  __syncthreads();

  // column c of token t: fragment (c / 16, t / 16), lane 16 (c % 16 / 4) + t % 16, element c % 4
  auto total = [&](int c, int t) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      s += red[w][(c >> 4) * TF + (t >> 4)][((c & 15) >> 2) * 16 + (t & 15)][c & 3];
    return s;
  };
  for (int o = tid; o < NF * 16 * TF; o += 64 * kWaves) {
    const int t = o / NF, c = o % NF, n = n0 + c;
    const bool live = t < a.T && n < a.N;  // a whole 32-column block of a token, or none of it, where N % 32 == 0
    float v = total(c, t);
    if constexpr (GATED) {
      const float u = total(8 + c, t);
      v = silu(v) * u;
    }
    if (live && a.y_f32) a.y_f32[(int64_t)t * a.N + n] = v;
    if (live && a.y_bf16) a.y_bf16[(int64_t)t * a.N + n] = (uint16_t)pack_bf16(v, v);
    if constexpr (!GATED && FR == 2) {
#pragma clang fp contract(off)
      if (a.y_q8) {
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
          uint8_t* blk = a.y_q8 + ((int64_t)t * (a.N / 32) + n / 32) * kQ81Bytes;
          blk[4 + c] = (uint8_t)q;
          if (c == 0)
            *reinterpret_cast<uint32_t*>(blk) =
                float_to_half_bits(d) | (float_to_half_bits(fp32_barrier(d * (float)sum)) << 16);
        }
      }
    }
  }
}

template <int FR, int MODE>
void run(const SmallArgs& a, hipStream_t st) {
  const int nf = MODE == kGatedPair ? 8 : 16 * FR;
  const dim3 grid((unsigned)((a.N + nf - 1) / nf));
  if constexpr (MODE == kRows) {
    if (a.T > 16) {
      const dim3 grid2(grid.x, (unsigned)((a.T + 31) / 32));
      hipLaunchKernelGGL((k_dense_fp8_small<FR, 2, MODE>), grid2, dim3(64 * small_waves(2)), 0, st, a);
      return;
    }
  }
  hipLaunchKernelGGL((k_dense_fp8_small<FR, 1, MODE>), grid, dim3(64 * small_waves(1)), 0, st, a);
}

}  // namespace

hipError_t launch_dense_fp8_small(const uint8_t* x, const float* xs, const uint8_t* w, const float* ws, int T, int N,
                                  int K, float* y_f32, uint16_t* y_bf16, uint8_t* y_q8, hipStream_t st) {
  const SmallArgs a{x, xs, nullptr, w, ws, y_f32, y_bf16, y_q8, T, N, K, (K + kFp8Block - 1) / kFp8Block};
  if (y_q8) run<2, kRows>(a, st);  // a q8_1 block is 32 columns
  else run<1, kRows>(a, st);
  return hipGetLastError();
}

hipError_t launch_dense_fp8_round(const float* h, const uint8_t* w, const float* ws, int T, int N, int K, float* y_f32,
                                  uint16_t* y_bf16, hipStream_t st) {
  run<1, kRound>(SmallArgs{nullptr, nullptr, h, w, ws, y_f32, y_bf16, nullptr, T, N, K,
                           (K + kFp8Block - 1) / kFp8Block}, st);
  return hipGetLastError();
}

hipError_t launch_gateup_fp8_small(const uint8_t* x, const float* xs, const uint8_t* gu, const float* gus, int T,
                                   int F, int C, float* h, hipStream_t st) {
  run<1, kGatedPair>(SmallArgs{x, xs, nullptr, gu, gus, h, nullptr, nullptr, T, F, C,
                               (C + kFp8Block - 1) / kFp8Block}, st);
  return hipGetLastError();
}

}  // namespace latmoe
