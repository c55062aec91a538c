// Products of e4m3 rows with e4m3 weights, for batches of whole token tiles:
// the dense projection, and the gated feed-forward block's gate/up projections
// with the activation and the rounding of H to e4m3 rows.
//
//   P[t][n][b] = sum over k in block b of xc[t][k] wc[n][k]      (v_mfma_f32_16x16x128_f8f6f4)
//   y[t][n]    = sum over blocks b of (xs[t][b] ws[n/128][b]) P[t][n][b]
//
// One MFMA covers exactly one block of K = 128, so its result with a zero
// accumulator input is P, and one fp32 FMA an element folds it into y: four
// VALU operations for each 16-pass MFMA, which run beside the next MFMAs.
//
// The e4m3 MFMA adds products in groups of eight neighbours in K, each cut
// (toward zero) to a multiple of 2^-13 of the power of two of the group's
// largest exponent, and the groups in fp32 (found by feeding it pairs of
// products of known size).  On Gaussian data that is 1.5e-5 of y's norm: 100
// times below the rounding of a bf16 y (1.7e-3), and further below those of
// q8_1 and e4m3, so these outputs take it.  A call that asks for the fp32 y
// gets exact products instead: the codes are widened to bf16 in registers
// (two a VALU operation), and four bf16 MFMAs a block (error 1e-8) take twice
// the matrix time.
//
// One workgroup computes TN = 16 FA WN weight rows x TT = 16 FB WT tokens.
// Weights are the MFMA's row operand: a lane then holds four neighbouring
// weight rows of one token, one scale for a whole MFMA result, and stores
// four neighbouring outputs at once.  Per K step of 128 both tiles go to LDS
// by direct loads (16 bytes a lane, no registers), double-buffered; a row is
// 128 bytes, its 16-byte chunks XOR-swizzled by the row so that a fragment
// read touches every bank once (the swizzle is applied to the global address
// of a lane, since the LDS side of a direct load is linear).
#include <type_traits>

#include "block_fp8.h"

namespace latmoe {
namespace {

typedef __attribute__((address_space(3))) void lds_void;

constexpr int kXcds = 8;
constexpr int kStep = kFp8Block;  // K per step: one MFMA, one scale
constexpr int kScaleSteps = 4;    // steps whose scales are staged together

__device__ __forceinline__ int swz(int row) { return (row >> 1) & 7; }

// Wait for this wave's outstanding loads, then for the workgroup.
__device__ __forceinline__ void loads_done_barrier() {
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
  __syncthreads();
}

struct DenseArgs {
  const uint8_t* x;   // [T][K] e4m3
  const float* xs;    // [T][nb]
  const uint8_t* w;   // [N][K] e4m3; gated: [2N][K], gate rows then up rows
  const float* ws;    // [ceil(N/128)][nb]; gated: twice that
  float* y_f32;
  uint16_t* y_bf16;
  uint8_t* y_q8;
  uint8_t* h;         // gated: [T][N] e4m3
  float* hs;          // gated: [T][ceil(N/128)]
  int64_t T;
  int N, K, nb;
  int n_nt, n_tt;     // weight and token tiles
};

// Tile order: groups of kGroup weight tiles sweep the token tiles, and each
// XCD takes a contiguous piece of that order, so that the tiles an XCD works
// on at one time share rows in its L2.
constexpr int kGroup = 4;
__device__ __forceinline__ void tile_of(const DenseArgs& a, int& nt, int& tt) {
  const int items = a.n_nt * a.n_tt;
  const int xcd = (int)blockIdx.x % kXcds, idx = (int)blockIdx.x / kXcds;
  const int q = items / kXcds, r = items % kXcds;
  const int item = xcd * q + min(xcd, r) + idx;
  const int group = item / (kGroup * a.n_tt);
  const int within = item - group * kGroup * a.n_tt;
  const int g = min(kGroup, a.n_nt - group * kGroup);
  tt = within / g;
  nt = group * kGroup + (within - tt * g);
}

// What a tile kernel computes: the projection with e4m3 products, the
// projection with bf16 products, or the gated pair of projections.
enum Mode : int { kFast = 0, kExact = 1, kGated = 2 };

template <int FA, int FB, int WN, int WT, int MODE>
struct Tile {
  static constexpr bool GATED = MODE == kGated;
  static constexpr int kThreads = 64 * WN * WT;
  static constexpr int TN = 16 * FA * WN, TT = 16 * FB * WT;
  static constexpr int kWaves = WN * WT;
  static constexpr int kLoadsA = TN / 8 / kWaves, kLoadsB = TT / 8 / kWaves;  // 1 KB each
  // a tile's weight rows lie in kSets scale blocks (gated: the gate's and the up's)
  static constexpr int kSets = GATED ? 2 : TN <= kFp8Block ? 1 : TN / kFp8Block;
  static constexpr int kScalesPerThread = kScaleSteps * TT / kThreads;
  static_assert(kScalesPerThread >= 1 && kScaleSteps % kScalesPerThread == 0, "whole runs of scales");
  static_assert(kFp8Block % (16 * FA) == 0, "a wave's weight rows lie in one scale block");
  static_assert(TN % (8 * kWaves) == 0 && TT % (8 * kWaves) == 0, "whole loads");
  static_assert(!GATED || TN == 256, "a gated tile holds one e4m3 block of H");

  // H column (within the tile) of LDS row r of the weight tile, gated tiles:
  // each wave's 16 FA rows are FA/2 gate fragments and the same columns' up
  // fragments.
  static __device__ __forceinline__ int gated_col(int r) {
    const int wave_rows = 16 * FA;
    return (r / wave_rows) * (wave_rows / 2) + (r % (wave_rows / 2));
  }
  static __device__ __forceinline__ bool gated_up(int r) { return (r % (16 * FA)) >= 8 * FA; }

  // Direct loads of one K step into LDS.
  static __device__ __forceinline__ void load_tiles(rsrc_t ra, rsrc_t ru, rsrc_t rb, uint8_t* __restrict__ As,
                                                    uint8_t* __restrict__ Bs, const int* va, const int* vb, int k0,
                                                    int wave) {
#pragma unroll
    for (int j = 0; j < kLoadsA; ++j) {
      const int piece = wave * kLoadsA + j;  // rows 8 piece .. +7
      const bool up = GATED && gated_up(8 * piece);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(up ? ru : ra, (lds_void*)(As + piece * 1024), 16, va[j], k0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kLoadsB; ++j) {
      const int piece = wave * kLoadsB + j;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(Bs + piece * 1024), 16, vb[j], k0, 0, 0);
    }
  }

  static __device__ __forceinline__ v8i fragment(const uint8_t* s, int row, int g) {
    // chunks 2g, 2g + 1 of the row: the same K order in both operands
    const v4i lo = *reinterpret_cast<const v4i*>(s + row * kStep + (((2 * g) ^ swz(row)) << 4));
    const v4i hi = *reinterpret_cast<const v4i*>(s + row * kStep + (((2 * g + 1) ^ swz(row)) << 4));
    return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  }

  // An MFMA operand of 16 rows and K = 128: the e4m3 codes, or (kExact) the
  // same values in bf16 (e4m3 is a subset of bf16).
  struct Codes { v8i v; };
  struct Wide { v8bf v[4]; };
  using Operand = std::conditional_t<MODE == kExact, Wide, Codes>;
  static __device__ __forceinline__ Operand operand(const uint8_t* s, int row, int g) {
    const v8i f = fragment(s, row, g);
    if constexpr (MODE == kExact) {
      Wide o;
#pragma unroll
      for (int q = 0; q < 4; ++q) o.v[q] = widen(f[2 * q], f[2 * q + 1]);
      return o;
    } else {
      return Codes{f};
    }
  }
  static __device__ __forceinline__ v4f product(const Operand& a, const Operand& b) {
    v4f p = {0.f, 0.f, 0.f, 0.f};
    if constexpr (MODE == kExact) {
#pragma unroll
      for (int q = 0; q < 4; ++q) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[q], b.v[q], p, 0, 0, 0);
    } else {
      p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, p, 0, 0, 0, 0, 0, 0);
    }
    return p;
  }

  // The step's products.  The MFMA of fragment pair q is issued before the
  // fold of pair q - kLag, whose result is then complete, and the weight
  // fragment of the next row of pairs is read meanwhile.
  static constexpr int kLag = 2;
  static __device__ __forceinline__ void multiply(const uint8_t* __restrict__ As, const uint8_t* __restrict__ Bs,
                                                  const float* __restrict__ sx, v4f (*acc)[FB], int wn, int wt,
                                                  int lane) {
    const int r = lane & 15, g = lane >> 4;
    const int a_row = wn * 16 * FA + r, b_row = wt * 16 * FB + r;
    const int set = kSets == 1 || GATED ? 0 : wn * 16 * FA / kFp8Block;
    Operand b[FB], a[2];
    float s[GATED ? 2 : 1][FB];
    a[0] = operand(As, a_row, g);
#pragma unroll
    for (int j = 0; j < FB; ++j) b[j] = operand(Bs, b_row + 16 * j, g);
#pragma unroll
    for (int j = 0; j < FB; ++j) {
      s[0][j] = sx[set * TT + b_row + 16 * j];
      if (GATED) s[GATED][j] = sx[TT + b_row + 16 * j];
    }
    v4f p[kLag + 1];
#pragma unroll
    for (int q = 0; q < FA * FB + kLag; ++q) {
      if (q < FA * FB) {
        const int i = q / FB, j = q % FB;
        if (j == 0 && i + 1 < FA) a[(i + 1) & 1] = operand(As, a_row + 16 * (i + 1), g);
        p[q % (kLag + 1)] = product(a[i & 1], b[j]);
      }
      if (q >= kLag) {
        const int i = (q - kLag) / FB, j = (q - kLag) % FB;
        const float f = s[GATED && i >= FA / 2][j];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(f, p[(q - kLag) % (kLag + 1)][e], acc[i][j][e]);
      }
    }
    // the folds stay in this step (the compiler would sink them past the next branch)
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) asm volatile("" : "+v"(acc[i][j]));
    if constexpr (MODE != kExact) {
      // the order above, as the scheduler is to keep it
#pragma unroll
      for (int q = 0; q < FA * FB + kLag; ++q) {
        if (q < FA * FB) {
          if (q % FB == 0 && q / FB + 1 < FA) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);  // LDS reads
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                                      // MFMA
        }
        if (q >= kLag) __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);  // VALU
      }
    }
  }

  // One step: the next step's loads into the other buffers, then this step's products.
  static __device__ __forceinline__ void step(bool more, rsrc_t ra, rsrc_t ru, rsrc_t rb,
                                              const uint8_t* __restrict__ As, const uint8_t* __restrict__ Bs,
                                              uint8_t* __restrict__ An, uint8_t* __restrict__ Bn,
                                              const float* __restrict__ sx, const int* va, const int* vb, int k_next,
                                              v4f (*acc)[FB], int wave, int wn, int wt, int lane) {
    if (more) load_tiles(ra, ru, rb, An, Bn, va, vb, k_next, wave);
    multiply(As, Bs, sx, acc, wn, wt, lane);
  }
};

template <int FA, int FB, int WN, int WT, int MODE>
__global__ __launch_bounds__(64 * WN * WT) void k_dense_fp8(const DenseArgs a) {
  using D = Tile<FA, FB, WN, WT, MODE>;
  constexpr int TN = D::TN, TT = D::TT;
  constexpr bool GATED = D::GATED;
  __shared__ __align__(16) uint8_t As0[TN * kStep], As1[TN * kStep];
  __shared__ __align__(16) uint8_t Bs0[TT * kStep], Bs1[TT * kStep];
  __shared__ __align__(16) float sxs[2][kScaleSteps][D::kSets * TT];  // xs * ws

  int nt, tt;
  tile_of(a, nt, tt);
  const int K = a.K, nb = a.nb;
  const int n0 = nt * (GATED ? TN / 2 : TN);  // first weight row (gated: first H column)
  const int64_t t0 = (int64_t)tt * TT;
  const int n_live = min(GATED ? TN / 2 : TN, a.N - n0);
  const int t_live = (int)min((int64_t)TT, a.T - t0);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave % WN, wt = wave / WN;

  // Rows past the end lie past num_records: their loads return zeros.
  const rsrc_t ra = make_rsrc(a.w + (int64_t)n0 * K, (uint32_t)n_live * K);
  const rsrc_t ru = GATED ? make_rsrc(a.w + ((int64_t)a.N + n0) * K, (uint32_t)n_live * K) : ra;
  const rsrc_t rb = make_rsrc(a.x + t0 * K, (uint32_t)t_live * K);
  const rsrc_t rs = make_rsrc(a.xs + t0 * nb, (uint32_t)t_live * nb * 4);

  // byte offsets of this lane's 16-byte pieces, K step 0; chunk: its logical position in the row
  int va[D::kLoadsA], vb[D::kLoadsB], ca[D::kLoadsA], cb[D::kLoadsB];
#pragma unroll
  for (int j = 0; j < D::kLoadsA; ++j) {
    const int r = 8 * (wave * D::kLoadsA + j) + (lane >> 3);
    const int row = GATED ? D::gated_col(r) : r;
    ca[j] = ((lane & 7) ^ swz(r)) << 4;
    va[j] = row < n_live ? row * K + ca[j] : kOutOfRange;
  }
#pragma unroll
  for (int j = 0; j < D::kLoadsB; ++j) {
    const int r = 8 * (wave * D::kLoadsB + j) + (lane >> 3);
    cb[j] = ((lane & 7) ^ swz(r)) << 4;
    vb[j] = r < t_live ? r * K + cb[j] : kOutOfRange;
  }
  // the last step of a ragged K: chunks past the row's end read as zeros
  const int tail = K % kStep ? K % kStep : kStep;
  auto cut = [&](int step) {
    if (step == nb - 1 && tail < kStep) {
#pragma unroll
      for (int j = 0; j < D::kLoadsA; ++j)
        if (ca[j] >= tail) va[j] = kOutOfRange;
#pragma unroll
      for (int j = 0; j < D::kLoadsB; ++j)
        if (cb[j] >= tail) vb[j] = kOutOfRange;
    }
  };

  // Scales: the products xs ws of kScaleSteps steps are staged at a time.
  // Thread -> (token, run of steps), and the kSets weight blocks of each step.
  constexpr int V = D::kScalesPerThread, S = D::kSets;
  const int s_tok = tid % TT, s_step = tid / TT * V;
  const int nbn = (a.N + kFp8Block - 1) / kFp8Block;
  const int w_blk = n0 / kFp8Block;
  const rsrc_t rw = make_rsrc(a.ws, (uint32_t)((GATED ? 2 : 1) * nbn * nb) * 4u);
  float sreg[V], wreg[S][V];
  auto scales_load = [&](int kb) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int b = kb + s_step + i;
      sreg[i] = __builtin_bit_cast(float, buf_u32(rs, b < nb ? (s_tok * nb + b) * 4 : kOutOfRange, 0));
#pragma unroll
      for (int q = 0; q < S; ++q) {
        const int blk = GATED ? w_blk + q * nbn : min(w_blk + q, nbn - 1);
        wreg[q][i] = __builtin_bit_cast(float, buf_u32(rw, b < nb ? (blk * nb + b) * 4 : kOutOfRange, 0));
      }
    }
  };
  auto scales_store = [&](int buf) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int q = 0; q < S; ++q) sxs[buf][s_step + i][q * TT + s_tok] = sreg[i] * wreg[q][i];
  };

  v4f acc[FA][FB] = {};
  scales_load(0);
  cut(0);
  D::load_tiles(ra, ru, rb, As0, Bs0, va, vb, 0, wave);
  scales_store(0);
  for (int s = 0; s < nb; s += 2) {
    const int sbuf = (s / kScaleSteps) & 1, srow = s % kScaleSteps;
    loads_done_barrier();
    // the next run's scales: loaded in a run's first step, stored in its second
    if (srow == 0) scales_load(s + kScaleSteps);
    cut(s + 1);
    D::step(s + 1 < nb, ra, ru, rb, As0, Bs0, As1, Bs1, sxs[sbuf][srow], va, vb, (s + 1) * kStep, acc, wave, wn, wt,
            lane);
    if (s + 1 == nb) break;
    loads_done_barrier();
    if (srow == 0) scales_store(sbuf ^ 1);
    cut(s + 2);
    D::step(s + 2 < nb, ra, ru, rb, As1, Bs1, As0, Bs0, sxs[sbuf][srow + 1], va, vb, (s + 2) * kStep, acc, wave, wn, wt,
            lane);
  }

  const int r = lane & 15, g = lane >> 4;
  if constexpr (!GATED) {
    const bool vec = a.N % 4 == 0;
#pragma unroll
    for (int j = 0; j < FB; ++j) {
      const int tl = wt * 16 * FB + 16 * j + r;
      const bool live = tl < t_live;
      const int64_t t = t0 + tl;
#pragma unroll
      for (int i = 0; i < FA; ++i) {
        const int n = n0 + wn * 16 * FA + 16 * i + 4 * g;
        const v4f v = acc[i][j];
        if (live && n < a.N) {
          if (a.y_f32) {
            float* dst = a.y_f32 + t * a.N + n;
            if (vec) *reinterpret_cast<v4f*>(dst) = v;
            else
              for (int e = 0; e < 4; ++e)
                if (n + e < a.N) dst[e] = v[e];
          }
          if (a.y_bf16) {
            uint16_t* dst = a.y_bf16 + t * a.N + n;
            const uint2 pk = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
            if (vec) *reinterpret_cast<uint2*>(dst) = pk;
            else
              for (int e = 0; e < 4; ++e)
                if (n + e < a.N) dst[e] = (uint16_t)((e < 2 ? pk.x : pk.y) >> (16 * (e & 1)));
          }
        }
      }
      if (a.y_q8) {
#pragma clang fp contract(off)
        // fragments 2q and 2q + 1 are one q8_1 block of the token
#pragma unroll
        for (int q = 0; q < FA / 2; ++q) {
          const int n = n0 + wn * 16 * FA + 32 * q;
          float amax = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            amax = fmaxf(amax, fmaxf(fabsf(acc[2 * q][j][e]), fabsf(acc[2 * q + 1][j][e])));
          amax = fmaxf(amax, __shfl_xor(amax, 16));
          amax = fmaxf(amax, __shfl_xor(amax, 32));
          const float d = amax / 127.0f;
          const float id = d != 0.0f ? 1.0f / d : 0.0f;
          uint32_t pk[2];
          int sum = 0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const v4f v = acc[2 * q + h][j];
            pk[h] = pack_codes(round_half_away(v[0] * id), round_half_away(v[1] * id), round_half_away(v[2] * id),
                               round_half_away(v[3] * id));
            sum = __builtin_amdgcn_sdot4((int)pk[h], 0x01010101, sum, false);
          }
          sum += __shfl_xor(sum, 16);
          sum += __shfl_xor(sum, 32);
          if (live && n < a.N) {
            uint32_t* blk = reinterpret_cast<uint32_t*>(a.y_q8 + (t * (a.N / 32) + n / 32) * kQ81Bytes);
            blk[1 + g] = pk[0];
            blk[5 + g] = pk[1];
            if (g == 0) blk[0] = float_to_half_bits(d) | (float_to_half_bits(fp32_barrier(d * (float)sum)) << 16);
          }
        }
      }
    }
  } else {
    // H = silu(G) U in place of the gate accumulators; a token's 128 columns
    // of the tile are one e4m3 block, held by WN waves
    __shared__ float part[WN][TT];
#pragma unroll
    for (int j = 0; j < FB; ++j) {
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < FA / 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float gv = acc[i][j][e];
          const float h = gv / (1.0f + __expf(-gv)) * acc[i + FA / 2][j][e];
          acc[i][j][e] = h;
          amax = fmaxf(amax, fabsf(h));
        }
      amax = fmaxf(amax, __shfl_xor(amax, 16));
      amax = fmaxf(amax, __shfl_xor(amax, 32));
      if (g == 0) part[wn][wt * 16 * FB + 16 * j + r] = amax;
    }
    __syncthreads();
    const int hb = (a.N + kFp8Block - 1) / kFp8Block;
#pragma unroll
    for (int j = 0; j < FB; ++j) {
#pragma clang fp contract(off)
      const int tl = wt * 16 * FB + 16 * j + r;
      float amax = part[0][tl];
#pragma unroll
      for (int w = 1; w < WN; ++w) amax = fmaxf(amax, part[w][tl]);
      float id;
      const float scale = fp8_scale(amax, id);
      const int64_t t = t0 + tl;
      if (tl < t_live) {
        if (wn == 0 && g == 0) a.hs[t * hb + n0 / kFp8Block] = scale;
#pragma unroll
        for (int i = 0; i < FA / 2; ++i) {
          const int n = wn * 8 * FA + 16 * i + 4 * g;
          const v4f v = acc[i][j];
          if (n < n_live)
            *reinterpret_cast<uint32_t*>(a.h + t * a.N + n0 + n) = pack_e4m3(v[0] * id, v[1] * id, v[2] * id, v[3] * id);
        }
      }
    }
  }
}

template <int FA, int FB, int WN, int WT, int MODE>
hipError_t run(DenseArgs a, hipStream_t st) {
  using D = Tile<FA, FB, WN, WT, MODE>;
  const int tn = MODE == kGated ? D::TN / 2 : D::TN;
  a.n_nt = (a.N + tn - 1) / tn;
  a.n_tt = (int)((a.T + D::TT - 1) / D::TT);
  hipLaunchKernelGGL((k_dense_fp8<FA, FB, WN, WT, MODE>), dim3((unsigned)(a.n_nt * a.n_tt)), dim3(D::kThreads), 0, st,
                     a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dense_fp8(const uint8_t* x, const float* xs, const uint8_t* w, const float* ws, int64_t T, int N,
                            int K, float* y_f32, uint16_t* y_bf16, uint8_t* y_q8, int num_cus, hipStream_t st) {
  const DenseArgs a{x, xs, w, ws, y_f32, y_bf16, y_q8, nullptr, nullptr, T, N, K, (K + kStep - 1) / kStep, 0, 0};
  // fp32 outputs take the bf16 products (see the head of the file)
  if (y_f32) return run<4, 4, 2, 2, kExact>(a, st);
  return run<4, 4, 2, 2, kFast>(a, st);
}

hipError_t launch_gateup_fp8(const uint8_t* x, const float* xs, const uint8_t* gu, const float* gus, int64_t T, int F,
                             int C, uint8_t* h, float* hs, int num_cus, hipStream_t st) {
  const DenseArgs a{x, xs, gu, gus, nullptr, nullptr, nullptr, h, hs, T, F, C, (C + kStep - 1) / kStep, 0, 0};
  return run<8, 4, 2, 1, kGated>(a, st);
}

}  // namespace latmoe
