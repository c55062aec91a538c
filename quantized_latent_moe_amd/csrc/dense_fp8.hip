// Products of e4m3 rows with e4m3 weights, for batches of whole token tiles:
// the dense projection, and the gated feed-forward block's gate/up projections
// with the activation and the rounding of H to e4m3 rows.
//
//   P[t][n][b] = sum over k in block b of xc[t][k] wc[n][k]      (v_mfma_f32_16x16x128_f8f6f4)
//   y[t][n]    = sum over blocks b of (xs[t][b] ws[n/128][b]) P[t][n][b]
//
// One MFMA covers exactly one block of K = 128, so its result with a zero
// accumulator input is P, and one fp32 FMA an element folds it into y: four
// VALU operations for each MFMA of 8 passes (32 cycles), beside the next MFMAs.
//
// The e4m3 MFMA adds products in groups of eight neighbours in K, each cut
// (toward zero) to a multiple of 2^-13 of the power of two of the group's
// largest exponent, and the groups in fp32 (found by feeding it pairs of
// products of known size).  On Gaussian data that is 1.5e-5 of y's norm: 100
// times below the rounding of a bf16 y (1.7e-3), so calls for rounded outputs
// take it unless they ask for exact products.  It is more where large products
// cancel and small ones beside them are what is left, and where a rounding to
// few bits follows: in the gated block 0.24% of H's codes become their
// neighbours, which are as near, and that moves y by 1.2e-3 of its norm (H's
// rounding itself by 2.3e-2, with either products).  Exact products, which the
// fp32 y of a projection takes unless the call says otherwise (y is then off by
// 1e-7 of its norm at K = 4096): the codes are widened to bf16 in registers (two
// a VALU operation), and four bf16 MFMAs a block take twice the matrix time.
//
// One workgroup computes TN = 16 FA WN weight rows x TT = 16 FB WT tokens.
// Weights are the MFMA's row operand: a lane then holds four neighbouring
// weight rows of one token, one scale for a whole MFMA result.  NP waves only
// load: per K step of 128 both tiles go to LDS by direct loads (16 bytes a
// lane, no registers), STAGES steps ahead; a row is 128 bytes, its 16-byte
// chunks XOR-swizzled by the row so that fragment reads have no bank conflicts
// (none counted; the swizzle is applied to the global address of a lane, since
// the LDS side of a direct load is linear).  Scale reads, whose lanes are 16
// bytes apart, have eight conflict cycles a wave and step, a tenth of LDS's.  WN x WT waves multiply: each reads its
// fragments a step ahead into the registers that their last MFMA has left, so
// that no LDS latency stands between two steps, and one barrier a step joins
// all waves.  (A wave that loads and multiplies waits for the memory pipe to
// take each load, 20 cycles for each of all the waves' loads, and its MFMAs
// with it: 128 x 128 tiles took 0.7 us a step that way and take 0.47 us now.)
//
// What bounds it: a step of 256 x 128 takes 1700 cycles of a CU, 0.86 to 1 us as
// the clock falls to 1.7 to 2 GHz under it, and no unit is busy all of them: the
// MFMAs need 1024 (the matrix pipe is counted busy 60% of the cycles), the LDS
// reads 640 (38%; fragment reads alone run at 244 bytes a cycle, 128 KB in
// 0.26 us), and the direct loads alone take 0.36 us (132 GB/s a CU where L2 has
// the rows), 0.39 together with the reads.  So neither LDS nor loads are the
// bound; what is left stands at the step's barrier, where all waves of the CU
// wait for the slowest.  A small tile's step is its loads: 0.20 us for the 16 KB
// of 64 x 64 on one CU, and 8 stages instead of 4, a barrier for two steps or a
// second set of fragment registers leave it there.  21000 x 4096 rows by 4096
// weights take 330 to 360 us (2000 to 2130 TF; with exact products 620 to
// 690 us, 1020 to 1130 TF), the range of several runs.
#include <algorithm>
#include <type_traits>

#include "block_fp8.h"

namespace latmoe {
namespace {

typedef __attribute__((address_space(3))) void lds_void;

constexpr int kXcds = 8;
constexpr int kStep = kFp8Block;  // K per step: one MFMA, one scale
constexpr int kScaleSteps = 4;  // a run: steps whose scales are staged together
constexpr int kRunBuffers = 4;

__device__ __forceinline__ int swz(int row) { return (row >> 1) & 7; }

// 4 x 4 transpose between four registers and the four 16-lane groups of a
// wave: register k of group g becomes register g of group k.
__device__ __forceinline__ void transpose4(uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto v = __builtin_amdgcn_permlane32_swap(r[i], r[i + 2], false, false);
    r[i] = v[0];
    r[i + 2] = v[1];
  }
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const auto v = __builtin_amdgcn_permlane16_swap(r[i], r[i + 1], false, false);
    r[i] = v[0];
    r[i + 1] = v[1];
  }
}

// Wait until at most N of this wave's loads and none of its LDS accesses are
// outstanding, then for the workgroup.  (__syncthreads waits for every load,
// those of later steps too.)
template <int N>
__device__ __forceinline__ void loads_done_barrier() {
  static_assert(N < 64, "vmcnt has 6 bits");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The workgroup's barrier for LDS alone: stores to memory go on.
__device__ __forceinline__ void lds_barrier() { loads_done_barrier<63>(); }

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
__device__ __forceinline__ void tile_of(const DenseArgs& a, int number, int& nt, int& tt) {
  const int items = a.n_nt * a.n_tt;
  const int xcd = number % kXcds, idx = number / kXcds;
  const int q = items / kXcds, r = items % kXcds;
  const int item = xcd * q + min(xcd, r) + idx;
  const int group = item / (kGroup * a.n_tt);
  const int within = item - group * kGroup * a.n_tt;
  const int g = min(kGroup, a.n_nt - group * kGroup);
  tt = within / g;
  nt = group * kGroup + (within - tt * g);
}

// What a tile kernel computes: the projection with e4m3 products, the
// projection with bf16 products, or the gated pair of projections with H
// rounded to e4m3 (a tile then holds 128 columns of H, one scale's) or in fp32,
// each of them with e4m3 or (Exact) bf16 products.
enum Mode : int { kFast = 0, kExact = 1, kGated = 2, kGatedRaw = 3, kGatedExact = 4, kGatedRawExact = 5 };
constexpr bool is_exact(int mode) { return mode == kExact || mode == kGatedExact || mode == kGatedRawExact; }
// H is rounded where it is made.
constexpr bool is_rounded(int mode) { return mode == kGated || mode == kGatedExact; }
constexpr Fp8Product product_of(int mode) {
  if (mode >= kGated) return is_exact(mode) ? kFp8GatedPairExact : kFp8GatedPair;
  return is_exact(mode) ? kFp8DenseExact : kFp8Dense;
}

template <int FA, int FB, int WN, int WT, int MODE, int STAGES, int NP>
struct Tile {
  static constexpr bool GATED = MODE >= kGated, EXACT = is_exact(MODE);
  static constexpr int kWaves = WN * WT;                // that multiply; NP more load
  static constexpr int kThreads = 64 * (kWaves + NP);
  static constexpr int TN = 16 * FA * WN, TT = 16 * FB * WT;
  // Whether the workgroups stay and take one tile after the other.
  static constexpr bool kPersistent = Fp8Tile{TN, TT, GATED}.stays();
  static constexpr int kLoadsA = TN / 8 / NP, kLoadsB = TT / 8 / NP;  // 1 KB each
  static_assert(kFp8Block % (16 * FA) == 0, "a wave's weight rows lie in one scale block");
  static_assert(TN % (8 * NP) == 0 && TT % (8 * NP) == 0, "whole loads");
  static_assert(TT % 64 == 0, "a load takes 64 tokens' scales");
  static_assert(STAGES >= 2, "at least a step ahead");
  static_assert(!is_rounded(MODE) || TN == 256, "a gated tile holds one e4m3 block of H");

  // H column (within the tile) of LDS row r of the weight tile, gated tiles:
  // each wave's 16 FA rows are FA/2 gate fragments and the same columns' up
  // fragments.
  static __device__ __forceinline__ int gated_col(int r) {
    const int wave_rows = 16 * FA;
    return (r / wave_rows) * (wave_rows / 2) + (r % (wave_rows / 2));
  }
  static __device__ __forceinline__ bool gated_up(int r) { return (r % (16 * FA)) >= 8 * FA; }

  // Where a tile lies: first weight row (gated: first H column) and token, and
  // how many of them are inside the matrices.
  struct Place {
    int n0, n_live, t_live;
    int64_t t0;
  };
  static __device__ __forceinline__ Place place(const DenseArgs& a, int number) {
    constexpr int COLS = GATED ? TN / 2 : TN;
    int nt, tt;
    tile_of(a, number, nt, tt);
    Place p;
    p.n0 = nt * COLS;
    p.t0 = (int64_t)tt * TT;
    p.n_live = min(COLS, a.N - p.n0);
    p.t_live = (int)min((int64_t)TT, a.T - p.t0);
    return p;
  }

  // What a wave loads: the tile's buffers (weight rows, gated: the up rows,
  // tokens, scales; rows past the end lie past the buffer's records: their
  // loads return zeros), and the lane's byte offset in each of its pieces at
  // K step 0.  Only the step's start, in the scalar offset, changes.
  struct Source {
    rsrc_t w, up, x;
    int vw[kLoadsA], vx[kLoadsB];
  };
  // The place of a lane's piece j within the step.
  static __device__ __forceinline__ int row_in_tile(int piece, int lane) { return 8 * piece + (lane >> 3); }
  static __device__ __forceinline__ int chunk_in_step(int row, int lane) { return ((lane & 7) ^ swz(row)) << 4; }
  static __device__ __forceinline__ void open(Source& src, const DenseArgs& a, const Place& at, int wave, int lane) {
    const int K = a.K;
    src.w = make_rsrc(a.w + (int64_t)at.n0 * K, (uint32_t)at.n_live * K);
    src.up = GATED ? make_rsrc(a.w + ((int64_t)a.N + at.n0) * K, (uint32_t)at.n_live * K) : src.w;
    src.x = make_rsrc(a.x + at.t0 * K, (uint32_t)at.t_live * K);
#pragma unroll
    for (int j = 0; j < kLoadsA; ++j) {
      const int r = row_in_tile(wave * kLoadsA + j, lane), row = GATED ? gated_col(r) : r;
      src.vw[j] = row < at.n_live ? row * K + chunk_in_step(r, lane) : kOutOfRange;
    }
#pragma unroll
    for (int j = 0; j < kLoadsB; ++j) {
      const int r = row_in_tile(wave * kLoadsB + j, lane);
      src.vx[j] = r < at.t_live ? r * K + chunk_in_step(r, lane) : kOutOfRange;
    }
  }
  // Chunks at or past `end` of the coming step read as zeros, and so do all later ones.
  static __device__ __forceinline__ void cut(Source& src, int end, int wave, int lane) {
#pragma unroll
    for (int j = 0; j < kLoadsA; ++j)
      if (chunk_in_step(row_in_tile(wave * kLoadsA + j, lane), lane) >= end) src.vw[j] = kOutOfRange;
#pragma unroll
    for (int j = 0; j < kLoadsB; ++j)
      if (chunk_in_step(row_in_tile(wave * kLoadsB + j, lane), lane) >= end) src.vx[j] = kOutOfRange;
  }
  // The wave's j-th direct load of a K step into LDS: weight rows, then tokens.
  static constexpr int kLoads = kLoadsA + kLoadsB;
  static __device__ __forceinline__ void load_piece(int j, const Source& src, uint8_t* As, uint8_t* Bs, int k0,
                                                    int wave) {
    if (j < kLoadsA) {
      const int piece = wave * kLoadsA + j;  // rows 8 piece .. +7
      const rsrc_t r = GATED && gated_up(8 * piece) ? src.up : src.w;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(As + piece * 1024), 16, src.vw[j], k0, 0, 0);
    } else {
      const int piece = wave * kLoadsB + j - kLoadsA;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(src.x, (lds_void*)(Bs + piece * 1024), 16, src.vx[j - kLoadsA], k0, 0,
                                               0);
    }
  }

  // The scales of a run of steps: one load for 64 tokens, a lane takes its
  // token's 16 bytes (values past a row's end are not used).
  static __device__ __forceinline__ rsrc_t open_scales(const DenseArgs& a, const Place& at) {
    return make_rsrc(a.xs + at.t0 * a.nb, (uint32_t)at.t_live * a.nb * 4);
  }
  static __device__ __forceinline__ void load_scales(rsrc_t xs, int nb, int run, float* to, int wave, int lane) {
#pragma unroll
    for (int q = 0; q < TT / 64; ++q)
      if (q % NP == wave)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(xs, (lds_void*)(to + q * 64 * kScaleSteps), 16,
                                                 ((q * 64 + lane) * nb + run * kScaleSteps) * 4, 0, 0, 0);
  }

  // LDS offset of chunk g of lane (r, g)'s row in a tile's first fragment.
  // Chunks g and g + 4 make the operand (64 bytes apart, whatever the swizzle):
  // the same K order on both sides, and no two of the lanes that LDS serves
  // together meet in a bank (chunks 2g and 2g + 1 with this swizzle do, at
  // half the read rate).
  static __device__ __forceinline__ int lane_offset(int row, int g) { return row * kStep + ((g ^ swz(row)) << 4); }
  // Fragment i from the lane's two chunk addresses (16 rows are 2 KB).
  static __device__ __forceinline__ v8i fragment(const uint8_t* lo, const uint8_t* hi, int i) {
    const v4i l = *reinterpret_cast<const v4i*>(lo + i * 16 * kStep);
    const v4i h = *reinterpret_cast<const v4i*>(hi + i * 16 * kStep);
    return v8i{l[0], l[1], l[2], l[3], h[0], h[1], h[2], h[3]};
  }

  // An MFMA operand of 16 rows and K = 128: the e4m3 codes, or (EXACT) the
  // same values in bf16 (e4m3 is a subset of bf16).
  struct Codes { v8i v; };
  struct Wide { v8bf v[4]; };
  using Operand = std::conditional_t<EXACT, Wide, Codes>;
  static __device__ __forceinline__ Operand operand(v8i f) {
    if constexpr (EXACT) {
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
    if constexpr (EXACT) {
#pragma unroll
      for (int q = 0; q < 4; ++q) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[q], b.v[q], p, 0, 0, 0);
    } else {
      p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, p, 0, 0, 0, 0, 0, 0);
    }
    return p;
  }

  // What a multiplying wave carries from step to step: the fragments and
  // scales of the step in hand, and the results that are not folded yet.
  // A product is folded kLag products later.  Where two multiplying waves of a
  // SIMD cover each other's waits and bf16 operands fill the registers, one is
  // enough; a wave alone (128 x 128 exact) takes 44 us with 1 and 37 with 3 for
  // 2048 x 2048 x 4096.
  static constexpr int kLag = EXACT && kWaves == 8 ? 1 : 3;
  static constexpr int kSides = GATED ? 2 : 1;
  static_assert(FA * FB % (kLag + 1) == 0, "the results' registers come round with the step");
  struct State {
    v8i a[FA], b[FB];
    float s[kSides][FB], s_last[kSides][FB];  // of this step, and of the one before
    v4f p[kLag + 1];
  };
  static __device__ __forceinline__ void start(State& st) {
#pragma unroll
    for (int q = 0; q <= kLag; ++q) st.p[q] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kSides; ++k)
#pragma unroll
      for (int j = 0; j < FB; ++j) st.s[k][j] = st.s_last[k][j] = 0.f;
  }
  static __device__ __forceinline__ void scales(State& st, const float* sx, float sw0, float sw1) {
#pragma unroll
    for (int j = 0; j < FB; ++j) {
      const float x = sx[16 * j * kScaleSteps];
      st.s[0][j] = x * sw0;
      if (GATED) st.s[kSides - 1][j] = x * sw1;
    }
  }
  // A step's products.  Each fragment's registers are filled with the next
  // step's fragment as soon as their last MFMA has been issued.
  static __device__ __forceinline__ void multiply(State& st, const uint8_t* Al, const uint8_t* Ah, const uint8_t* Bl,
                                                  const uint8_t* Bh, v4f (*acc)[FB]) {
    Operand ao, b[FB];
#pragma unroll
    for (int j = 0; j < FB; ++j) b[j] = operand(st.b[j]);
#pragma unroll
    for (int q = 0; q < FA * FB; ++q) {
      const int i = q / FB, j = q % FB;
      if (j == 0) ao = operand(st.a[i]);
      const int o = (q + FA * FB - kLag) % (FA * FB), oi = o / FB, oj = o % FB;
      const v4f done = st.p[o % (kLag + 1)];
      st.p[q % (kLag + 1)] = product(ao, b[j]);
      if (j == FB - 1) st.a[i] = fragment(Al, Ah, i);
      if (i == FA - 1) st.b[j] = fragment(Bl, Bh, j);
      const int side = GATED && oi >= FA / 2 ? 1 : 0;
      const float f = q >= kLag ? st.s[side][oj] : st.s_last[side][oj];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[oi][oj][e] = __builtin_fmaf(f, done[e], acc[oi][oj][e]);
      __builtin_amdgcn_sched_barrier(0);  // the scheduler keeps this order
    }
#pragma unroll
    for (int k = 0; k < kSides; ++k)
#pragma unroll
      for (int j = 0; j < FB; ++j) st.s_last[k][j] = st.s[k][j];
    // the folds stay in this step (the compiler would sink them past the next branch)
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) asm volatile("" : "+v"(acc[i][j]));
  }
  // The results that the last step has left.
  static __device__ __forceinline__ void finish(State& st, v4f (*acc)[FB]) {
#pragma unroll
    for (int o = FA * FB - kLag; o < FA * FB; ++o) {
      const int oi = o / FB, oj = o % FB, side = GATED && oi >= FA / 2 ? 1 : 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc[oi][oj][e] = __builtin_fmaf(st.s_last[side][oj], st.p[o % (kLag + 1)][e], acc[oi][oj][e]);
    }
  }
};

template <int FA, int FB, int WN, int WT, int MODE, int STAGES, int NP>
__global__ __launch_bounds__(64 * (WN * WT + NP)) void k_dense_fp8(const DenseArgs a) {
  using D = Tile<FA, FB, WN, WT, MODE, STAGES, NP>;
  constexpr int TN = D::TN, TT = D::TT;
  constexpr bool GATED = D::GATED;
  __shared__ __align__(16) uint8_t As[STAGES * TN * kStep], Bs[STAGES * TT * kStep];
  __shared__ __align__(16) float sxs[kRunBuffers * TT * kScaleSteps];  // runs of [token][step]
  constexpr int PARTS = is_rounded(MODE) ? WN : 1;
  __shared__ float part[PARTS][is_rounded(MODE) ? TT : 1];  // largest |H| of a token in a wave's columns

  const int K = a.K, nb = a.nb;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int first = (int)workgroup_number();
  if (!D::kPersistent && first >= a.n_nt * a.n_tt) return;  // the whole workgroup
  const int stride = D::kPersistent ? (int)gridDim.x : 1, items = D::kPersistent ? a.n_nt * a.n_tt : first + 1;

  if (wave >= D::kWaves) {
    // ---- loads: the steps of all the workgroup's tiles in a row ----
    const int p = wave - D::kWaves;
    const int tail = K % kStep ? K % kStep : kStep, runs = (nb + kScaleSteps - 1) / kScaleSteps;
    typename D::Source src;
    int tile = first, step = 0, buf = 0;  // what is loaded next
    const typename D::Place at = D::place(a, tile);
    D::open(src, a, at, p, lane);
    // past the last tile nothing is read (the zeros go to buffers no step uses)
    auto prepare = [&]() {
      if constexpr (D::kPersistent) {
        if (step == nb) {
          step = 0;
          tile = tile < items ? tile + stride : tile;
          if (tile < items) D::open(src, a, D::place(a, tile), p, lane);
        }
      }
      const int end = tile >= items || step >= nb ? 0 : step == nb - 1 ? tail : kStep;
      if (end < kStep) D::cut(src, end, p, lane);
    };
    auto load_next = [&]() {
#pragma unroll
      for (int j = 0; j < D::kLoads; ++j)
        D::load_piece(j, src, As + buf * TN * kStep, Bs + buf * TT * kStep, step * kStep, p);
      ++step;
      buf = buf + 1 == STAGES ? 0 : buf + 1;
    };
    int run_tile = first, run = 0, run_buf = 0;
    rsrc_t xs = D::open_scales(a, at);
    auto load_next_run = [&]() {
      if constexpr (D::kPersistent) {
        if (run == runs) {
          run = 0;
          run_tile = run_tile < items ? run_tile + stride : run_tile;
          if (run_tile < items) xs = D::open_scales(a, D::place(a, run_tile));
        }
      }
      if (run_tile < items && run < runs) D::load_scales(xs, nb, run, sxs + run_buf * TT * kScaleSteps, p, lane);
      ++run;
      run_buf = run_buf + 1 == kRunBuffers ? 0 : run_buf + 1;
    };
    // Fragments are read a step ahead: at barrier s step s + 1 has landed and
    // the buffers of step s are free.  A run's scales are loaded when the third
    // run before it begins: whatever the runs' lengths, three barriers or more
    // lie between, which wait for all but the loads of the last steps, and the
    // buffer's last reader is done.
#pragma unroll
    for (int r = 0; r < kRunBuffers - 1; ++r) load_next_run();
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
      prepare();
      load_next();
    }
    loads_done_barrier<(STAGES - 1) * D::kLoads>();
#pragma unroll 1
    for (int i = first; i < items; i += stride) {
#pragma unroll 1
      for (int s = 0; s < nb; ++s) {
        prepare();
        asm volatile("" : "+s"(step), "+s"(buf));  // before the barrier, where these waves wait
        loads_done_barrier<(STAGES - 2) * D::kLoads>();
        if ((s & (kScaleSteps - 1)) == 0) load_next_run();
        load_next();
      }
      if (is_rounded(MODE)) lds_barrier();
    }
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): no load may still write LDS when the workgroup ends
    return;
  }
  // ---- products ----
  const int wn = wave % WN, wt = wave / WN;
  // weight scales: one for the wave's rows and step (gated: one of the gate
  // rows, one of the up rows), a step ahead in scalar registers
  const int nbn = (a.N + kFp8Block - 1) / kFp8Block;
  typedef const __attribute__((address_space(4))) float* const_floats;
  auto weight_scales = [&](int n0) {
    const int block = GATED ? n0 / kFp8Block : min((n0 + wn * 16 * FA) / kFp8Block, nbn - 1);
    return (const_floats)(a.ws + (int64_t)block * nb);
  };
  const int64_t up = GATED ? (int64_t)nbn * nb : 0;
  typename D::State st;
  const int a_off = D::lane_offset(wn * 16 * FA + (lane & 15), lane >> 4);
  const int b_off = D::lane_offset(wt * 16 * FB + (lane & 15), lane >> 4);
  const float* sx = sxs + (wt * 16 * FB + (lane & 15)) * kScaleSteps;
  typename D::Place at = D::place(a, first);
  const_floats ws = weight_scales(at.n0);
  const_floats ws1 = ws + up;
  float sw0 = ws[0], sw1 = ws1[0];
  loads_done_barrier<63>();  // step 0 has landed
#pragma unroll
  for (int i = 0; i < FA; ++i) st.a[i] = D::fragment(As + a_off, As + (a_off ^ 64), i);
#pragma unroll
  for (int j = 0; j < FB; ++j) st.b[j] = D::fragment(Bs + b_off, Bs + (b_off ^ 64), j);
  int cur = 1;           // the coming step's buffers
  uint32_t in_runs = 0;  // and its place in the runs of scales, each of which starts at a multiple of kScaleSteps
#pragma unroll 1
  for (int tile = first; tile < items; tile += stride) {
    v4f acc[FA][FB] = {};
    D::start(st);
#pragma unroll 1
    for (int s = 0; s < nb;) {
      loads_done_barrier<63>();
      D::scales(st, sx + (in_runs / kScaleSteps % kRunBuffers * (TT * kScaleSteps) + in_runs % kScaleSteps), sw0, sw1);
      const int al = cur * TN * kStep + a_off, bl = cur * TT * kStep + b_off;
      D::multiply(st, As + al, As + (al ^ 64), Bs + bl, Bs + (bl ^ 64), acc);
      ++s;
      const uint32_t ahead = (uint32_t)min(s, nb - 1);
      sw0 = ws[ahead];
      if (GATED) sw1 = ws1[ahead];
      cur = cur + 1 == STAGES ? 0 : cur + 1;
      ++in_runs;
      if (D::kPersistent && s == nb) in_runs = (in_runs + kScaleSteps - 1) / kScaleSteps * kScaleSteps;
    }
    D::finish(st, acc);
    const int n0 = at.n0, n_live = at.n_live, t_live = at.t_live;
    const int64_t t0 = at.t0;
    if (tile + stride < items) {
      at = D::place(a, tile + stride);
      ws = weight_scales(at.n0);
      ws1 = ws + up;
      sw0 = ws[0];
      sw1 = ws1[0];
    }

    const int r = lane & 15, g = lane >> 4;
    if constexpr (MODE == kGatedRaw || MODE == kGatedRawExact) {
#pragma unroll
      for (int j = 0; j < FB; ++j)
#pragma unroll
        for (int i = 0; i < FA / 2; ++i) {
          const int tl = wt * 16 * FB + 16 * j + r, n = wn * 8 * FA + 16 * i + 4 * g;
          v4f h;
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = silu(acc[i][j][e]) * acc[i + FA / 2][j][e];
          if (tl < t_live && n < n_live) *reinterpret_cast<v4f*>(a.y_f32 + (t0 + tl) * a.N + n0 + n) = h;
        }
    } else if constexpr (!GATED) {
      const bool vec4 = a.N % 4 == 0, vec8 = a.N % 8 == 0;
#pragma unroll
      for (int j = 0; j < FB; ++j) {
        const int tl = wt * 16 * FB + 16 * j + r;
        const bool live = tl < t_live;
        const int64_t t = t0 + tl;
        if (a.y_f32) {
#pragma unroll
          for (int i = 0; i < FA; ++i) {
            const int n = n0 + wn * 16 * FA + 16 * i + 4 * g;
            const v4f v = acc[i][j];
            if (live && n < a.N) {
              float* dst = a.y_f32 + t * a.N + n;
              if (vec4) *reinterpret_cast<v4f*>(dst) = v;
              else
                for (int e = 0; e < 4; ++e)
                  if (n + e < a.N) dst[e] = v[e];
            }
          }
        }
        if (a.y_bf16) {
          // four fragments at a time (a narrow tile has two, and the other half
          // of the lanes nothing to store), transposed among the lane groups: a
          // lane then stores 16 neighbouring columns
#pragma unroll
          for (int q = 0; q < FA; q += 4) {
            uint32_t lo[4], hi[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const v4f v = acc[q + i < FA ? q + i : q][j];
              lo[i] = pack_bf16(v[0], v[1]);
              hi[i] = pack_bf16(v[2], v[3]);
            }
            transpose4(lo);
            transpose4(hi);
            const int n = n0 + wn * 16 * FA + 16 * (q + g);
            uint16_t* dst = a.y_bf16 + t * a.N + n;
            if (!live || q + g >= FA) continue;
            if (vec8) {
              if (n < a.N) *reinterpret_cast<uint4*>(dst) = uint4{lo[0], hi[0], lo[1], hi[1]};
              if (n + 8 < a.N) *reinterpret_cast<uint4*>(dst + 8) = uint4{lo[2], hi[2], lo[3], hi[3]};
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (vec4) {
                  if (n + 4 * i < a.N) *reinterpret_cast<uint2*>(dst + 4 * i) = uint2{lo[i], hi[i]};
                } else {
                  for (int e = 0; e < 4; ++e)
                    if (n + 4 * i + e < a.N)
                      dst[4 * i + e] = (uint16_t)((e < 2 ? lo[i] : hi[i]) >> (16 * (e & 1)));
                }
              }
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
              amax = max_or_nan(amax, max_or_nan(fabsf(acc[2 * q][j][e]), fabsf(acc[2 * q + 1][j][e])));
            amax = max_or_nan(amax, __shfl_xor(amax, 16));
            amax = max_or_nan(amax, __shfl_xor(amax, 32));
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
#pragma unroll
      for (int j = 0; j < FB; ++j) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < FA / 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float h = silu(acc[i][j][e]) * acc[i + FA / 2][j][e];
            acc[i][j][e] = h;
            amax = fmaxf(amax, fabsf(h));
          }
        amax = fmaxf(amax, __shfl_xor(amax, 16));
        amax = fmaxf(amax, __shfl_xor(amax, 32));
        if (g == 0) part[wn][wt * 16 * FB + 16 * j + r] = amax;
      }
      lds_barrier();
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
        if (tl < t_live && wn == 0 && g == 0) a.hs[t * hb + n0 / kFp8Block] = scale;
        uint32_t pk[FA / 2];
#pragma unroll
        for (int i = 0; i < FA / 2; ++i) {
          const v4f v = acc[i][j];
          pk[i] = pack_e4m3(v[0] * id, v[1] * id, v[2] * id, v[3] * id);
        }
        if constexpr (FA == 8) {  // a lane stores 16 neighbouring columns
          transpose4(pk);
          const int n = wn * 64 + 16 * g;
          if (tl < t_live && n < n_live)
            *reinterpret_cast<uint4*>(a.h + t * a.N + n0 + n) = uint4{pk[0], pk[1], pk[2], pk[3]};
        } else {
#pragma unroll
          for (int i = 0; i < FA / 2; ++i) {
            const int n = wn * 8 * FA + 16 * i + 4 * g;
            if (tl < t_live && n < n_live) *reinterpret_cast<uint32_t*>(a.h + t * a.N + n0 + n) = pk[i];
          }
        }
      }
    }
  }
}

// V: the variant's place among its product's.
template <int V, int FA, int FB, int WN, int WT, int MODE, int STAGES, int NP>
hipError_t run(DenseArgs a, int num_cus, hipStream_t st) {
  using D = Tile<FA, FB, WN, WT, MODE, STAGES, NP>;
  constexpr Fp8Tile tile = kFp8Tiles[product_of(MODE)][V];
  static_assert(tile.rows == D::TN && tile.tokens == D::TT && tile.gated == D::GATED, "the tile that the choice knows");
  a.n_nt = (a.N + tile.cols() - 1) / tile.cols();
  a.n_tt = (int)((a.T + D::TT - 1) / D::TT);
  const int items = a.n_nt * a.n_tt;
  const dim3 grid = grid_of(D::kPersistent ? std::min(items, num_cus) : items);
  hipLaunchKernelGGL((k_dense_fp8<FA, FB, WN, WT, MODE, STAGES, NP>), grid, dim3(D::kThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dense_fp8(const uint8_t* x, const float* xs, const uint8_t* w, const float* ws, int64_t T, int N,
                            int K, bool exact, float* y_f32, uint16_t* y_bf16, uint8_t* y_q8, int num_cus,
                            hipStream_t st) {
  const DenseArgs a{x, xs, w, ws, y_f32, y_bf16, y_q8, nullptr, nullptr, T, N, K, (K + kStep - 1) / kStep, 0, 0};
  if (exact) {
    switch (fp8_pick_tile(kFp8DenseExact, T, N, a.nb, num_cus)) {
      case 0: return run<0, 4, 3, 2, 4, kExact, 3, 4>(a, num_cus, st);
      case 1: return run<1, 4, 4, 2, 2, kExact, 3, 2>(a, num_cus, st);
      default: return run<2, 2, 2, 2, 2, kExact, 4, 4>(a, num_cus, st);
    }
  }
  switch (fp8_pick_tile(kFp8Dense, T, N, a.nb, num_cus)) {
    case 0: return run<0, 4, 4, 4, 2, kFast, 3, 4>(a, num_cus, st);
    case 1: return run<1, 4, 4, 2, 2, kFast, 3, 4>(a, num_cus, st);
    case 2: return run<2, 4, 2, 2, 2, kFast, 3, 2>(a, num_cus, st);
    default: return run<3, 2, 2, 2, 2, kFast, 4, 4>(a, num_cus, st);
  }
}

hipError_t launch_gateup_fp8(const uint8_t* x, const float* xs, const uint8_t* gu, const float* gus, int64_t T, int F,
                             int C, bool exact, float* h32, uint8_t* h, float* hs, int num_cus, hipStream_t st) {
  const DenseArgs a{x, xs, gu, gus, h32, nullptr, nullptr, h, hs, T, F, C, (C + kStep - 1) / kStep, 0, 0};
  const int variant = fp8_pick_tile(exact ? kFp8GatedPairExact : kFp8GatedPair, T, F, a.nb, num_cus);
  hipError_t e;
  if (exact) {
    if (variant == 0) return run<0, 4, 2, 4, 2, kGatedExact, 3, 4>(a, num_cus, st);
    e = run<1, 2, 2, 2, 2, kGatedRawExact, 4, 4>(a, num_cus, st);
  } else {
    if (variant == 0) return run<0, 4, 4, 4, 2, kGated, 3, 4>(a, num_cus, st);
    if (variant == 1) return run<1, 8, 2, 2, 2, kGated, 3, 4>(a, num_cus, st);
    e = variant == 2 ? run<2, 4, 2, 2, 2, kGatedRaw, 3, 2>(a, num_cus, st)
                     : run<3, 2, 2, 2, 2, kGatedRaw, 4, 4>(a, num_cus, st);
  }
  return e == hipSuccess ? launch_quantize_fp8(h32, LAT_MOE_F32, T, F, h, hs, st) : e;
}

}  // namespace latmoe
