// Products of 16-bit rows with 16-bit weights, for batches of whole token
// tiles: the dense projection with bias, activation and residual, and the gated
// pair.
//
//   y[t][n] = act(sum over k of x[t][k] w[n][k] + bias[n]) + residual[t][n]
//   h[t][f] = act(gate) * up
//
// One workgroup computes TN = 16 FA WN weight rows x TT = 16 FB WT tokens;
// gated tiles hold gate rows and the same columns' up rows, so that one lane
// has both.  Weights are the MFMA's row operand: a lane then holds four
// neighbouring weight rows of one token.  Products are exact and added in fp32
// by the MFMA.
//
// Per K step of 64 both tiles go to LDS by direct loads (16 bytes a lane, no
// registers), STAGES steps ahead; a row is 128 bytes, its 16-byte chunks
// XOR-swizzled by the row so that fragment reads have no bank conflicts (none
// counted; the swizzle is applied to the global address of a lane, since the
// LDS side of a direct load is linear).  Fragments are read a step ahead into
// the registers that their last MFMA has left, and the step's one barrier comes
// after its first MFMAs, when the reads are long done: nothing waits for LDS.
// The loads come at every third MFMA of a step's first half: they have to land
// within a step (8192^3 takes 767 us; with a load at every fourth MFMA 788, at
// every sixth 810, and at every second 2% more too: the memory pipe then makes
// the waves wait).
// Steps of 32 with twice the stages take 10% longer (a barrier for half the
// work), two workgroups of half the tile on a CU 25% (more bytes for a product),
// and four waves of 128 x 128 in twice the registers as long.
//
// Where few tiles would have all of K to go, WK slices of waves deal the steps
// among themselves, each with stages of its own, and add their sums in LDS at
// the end, in their order: a step of one slice is a chain of barrier, reads and
// MFMAs of 0.19 us, whatever it multiplies.
//
// What bounds it: large products the power that the chip may draw.  Under
// 21000 x 4096 by 4096 the clock falls to 1.8 GHz with the matrix pipes busy 65
// to 73% of the cycles; the loop alone, without the loads, runs at 1700 TF.
// 21000 x 4096 by 4096 with residual takes 565 to 590 us (1190 to 1250 TF; a
// library product without it 570 to 615 on the same machines), the gated pair
// 5268 x 4096 by 2 x 8192 495 to 610 us (1160 to 1430 TF), 8192^3 765 to 790 us
// (1390 to 1430 TF; the library 675 to 750).  Mid-sized ones are bound by what a CU
// loads, 75 to 100 GB/s with all of them at it: 5268 x 4096 by 1024 takes 50 us
// (870 TF), 517 x 2056 by 4100 25 us, 5268 x 4096 by 128 15 us.
#include "dense16_tiles.h"
#include "epilogue16.h"

namespace latmoe {
namespace {


constexpr int kXcds = 8;
constexpr int kStep = 64;              // K per step
constexpr int kRowBytes = 2 * kStep;   // of a step's row in LDS

// A buffer's descriptor in scalar registers (raw, stride 0).
__device__ __forceinline__ v4i descriptor(const void* base, uint32_t bytes) {
  const uint64_t p = (uint64_t)base;
  return v4i{(int)(uint32_t)p, (int)(uint32_t)(p >> 32) & 0xffff, (int)bytes, 0x00020000};
}
// Direct load into LDS: 16 bytes a lane, from voff + soff of the buffer to
// `lds` + 16 lane (an offset past the buffer's records brings zeros).  As
// assembly, which the compiler does not count: it would wait for every load on
// its way before any LDS read, since it cannot tell the stages apart.  The
// waits are those of loads_done_barrier.  No register is written.
__device__ __forceinline__ void load_lds(v4i buffer, uint32_t lds, int voff, int soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(buffer), "s"(soff)
               : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

__device__ __forceinline__ int swz(int row) { return (row >> 1) & 7; }

// Wait until at most N of this wave's accesses to memory and none of its LDS
// accesses are outstanding, then for the workgroup.
template <int N>
__device__ __forceinline__ void loads_done_barrier() {
  static_assert(N < 64, "vmcnt has 6 bits");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Tile order: groups of kGroup weight tiles sweep the token tiles, and each
// XCD takes a contiguous piece of that order, so that the tiles an XCD works
// on at one time share rows in its L2.  Groups of 8 take as long (and with few
// token tiles read a quarter more), of 16 2 to 10% longer.
constexpr int kGroup = 4;
__device__ __forceinline__ void tile_of(const Dense16Args& a, int number, int& nt, int& tt) {
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

template <int TYPE, int FA, int FB, int WN, int WT, int WK, bool GATED, int STAGES>
struct Tile {
  static constexpr int kWaves = WN * WT, kThreads = 64 * kWaves * WK;  // waves of a slice of K
  static constexpr int TN = 16 * FA * WN, TT = 16 * FB * WT;
  static constexpr int COLS = GATED ? TN / 2 : TN;  // columns of the output
  static constexpr int kLoadsA = TN / 8 / kWaves, kLoadsB = TT / 8 / kWaves, kLoads = kLoadsA + kLoadsB;  // 1 KB each
  static_assert(TN % (8 * kWaves) == 0 && TT % (8 * kWaves) == 0, "whole loads");
  static_assert(!GATED || FA % 2 == 0, "as many gate fragments as up fragments");
  static_assert(STAGES >= 2, "a step ahead");
  static constexpr int kA = TN * kRowBytes, kStage = kA + TT * kRowBytes;  // bytes of a stage: weights, then tokens

  // Output column (within the tile) of LDS row r of the weight tile, gated
  // tiles: each wave's 16 FA rows are FA/2 gate fragments and the same columns'
  // up fragments.
  static __device__ __forceinline__ int gated_col(int r) {
    const int wave_rows = 16 * FA;
    return (r / wave_rows) * (wave_rows / 2) + (r % (wave_rows / 2));
  }
  static __device__ __forceinline__ bool gated_up(int r) { return (r % (16 * FA)) >= 8 * FA; }

  struct Place {
    int n0, n_live, t_live;
    int64_t t0;
  };
  static __device__ __forceinline__ Place place(const Dense16Args& a, int number) {
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
  // tokens), and the lane's byte offset in each of its pieces at K step 0.
  // Only the step's start, in the scalar offset, changes.  Rows past the
  // tile's last, and what lies past a row's end, have an offset past the
  // buffer's records: their loads return zeros.
  struct Source {
    v4i w, up, x;
    int vw[kLoadsA], vx[kLoadsB];
  };
  static __device__ __forceinline__ int row_in_tile(int piece, int lane) { return 8 * piece + (lane >> 3); }
  static __device__ __forceinline__ int chunk_in_step(int row, int lane) { return ((lane & 7) ^ swz(row)) << 4; }
  static __device__ __forceinline__ void open(Source& src, const Dense16Args& a, const Place& at, int wave, int lane) {
    const uint16_t* w = static_cast<const uint16_t*>(a.w);
    const int row_w = 2 * a.K, row_x = 2 * (int)a.x_stride;
    const uint32_t bytes_w = (uint32_t)at.n_live * row_w;
    src.w = descriptor(w + (int64_t)at.n0 * a.K, bytes_w);
    src.up = GATED ? descriptor(w + ((int64_t)a.N + at.n0) * a.K, bytes_w) : src.w;
    src.x = descriptor(static_cast<const uint16_t*>(a.x) + at.t0 * a.x_stride,
                      (uint32_t)(at.t_live - 1) * row_x + 2 * a.K);
#pragma unroll
    for (int j = 0; j < kLoadsA; ++j) {
      const int r = row_in_tile(wave * kLoadsA + j, lane), row = GATED ? gated_col(r) : r;
      src.vw[j] = row < at.n_live ? row * row_w + chunk_in_step(r, lane) : kOutOfRange;
    }
#pragma unroll
    for (int j = 0; j < kLoadsB; ++j) {
      const int r = row_in_tile(wave * kLoadsB + j, lane);
      src.vx[j] = r < at.t_live ? r * row_x + chunk_in_step(r, lane) : kOutOfRange;
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
  static __device__ __forceinline__ void load_piece(int j, const Source& src, uint32_t stage, int k0, int wave) {
    if (j < kLoadsA) {
      const int piece = wave * kLoadsA + j;  // rows 8 piece .. +7
      load_lds(GATED && gated_up(8 * piece) ? src.up : src.w, stage + piece * 1024, src.vw[j], k0);
    } else {
      const int piece = wave * kLoadsB + j - kLoadsA;
      load_lds(src.x, stage + kA + piece * 1024, src.vx[j - kLoadsA], k0);
    }
  }

  static __device__ __forceinline__ v4i fragment(const uint8_t* at, int i) {
    return *reinterpret_cast<const v4i*>(at + i * 16 * kRowBytes);
  }
};

template <int TYPE, int FA, int FB, int WN, int WT, int WK, bool GATED, int STAGES>
__global__ __launch_bounds__(64 * WN * WT * WK) void k_dense_16(const Dense16Args a) {
  using D = Tile<TYPE, FA, FB, WN, WT, WK, GATED, STAGES>;
  __shared__ __align__(16) uint8_t stages[WK * STAGES * D::kStage];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) % D::kWaves;
  const int wk = __builtin_amdgcn_readfirstlane(tid >> 6) / D::kWaves;
  const int first = (int)workgroup_number();
  if (first >= a.n_nt * a.n_tt) return;  // the whole workgroup
  const int wn = wave % WN, wt = wave / WN;
  const int steps = (a.K + kStep - 1) / kStep;
  const int tail = a.K % kStep ? 2 * (a.K % kStep) : kRowBytes;
  const typename D::Place at = D::place(a, first);
  typename D::Source src;
  D::open(src, a, at, wave, lane);
  int step = wk;  // loaded next
  auto prepare = [&]() {
    const int end = step >= steps ? 0 : step == steps - 1 ? tail : kRowBytes;
    if (end < kRowBytes) D::cut(src, end, wave, lane);
  };

  const int row = lane & 15, g = lane >> 4;
  const int off0 = row * kRowBytes + ((g ^ swz(row)) << 4);
  const int a_off = wn * 16 * FA * kRowBytes + off0, b_off = D::kA + wt * 16 * FB * kRowBytes + off0;
  v4i fa[FA][2], fb[FB][2];
  v4f acc[FA][FB] = {};

  uint8_t* const own = stages + wk * STAGES * D::kStage;  // the slice's stages
  const uint32_t base = lds_address(own);
  int buf = 0;
#pragma unroll
  for (int s = 0; s < STAGES; ++s) {
    prepare();
#pragma unroll
    for (int j = 0; j < D::kLoads; ++j)
      D::load_piece(j, src, base + s * D::kStage, step * kRowBytes, wave);
    step += WK;
  }
  loads_done_barrier<(STAGES - 1) * D::kLoads>();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < FA; ++i) fa[i][h] = D::fragment(own + (a_off ^ (64 * h)), i);
#pragma unroll
    for (int j = 0; j < FB; ++j) fb[j][h] = D::fragment(own + (b_off ^ (64 * h)), j);
  }
  constexpr int M = 2 * FA * FB;  // MFMAs of a step
  constexpr int Q = FB;           // of which so many come before the step's barrier
#pragma unroll 1
  for (int s = 0; s < steps; s += WK) {
    // The step's fragments are in registers.  At its barrier the next step has
    // landed, and every wave has read this step's buffers, which then take step
    // s + STAGES; each fragment's registers take the next step's as soon as
    // their last MFMA has been issued.
    const int next = buf + 1 == STAGES ? 0 : buf + 1;
    const uint8_t* ahead = own + next * D::kStage;
    prepare();
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int h = m / (FA * FB), i = m / FB % FA, j = m % FB;
      acc[i][j] = mfma16<TYPE>(fa[i][h], fb[j][h], acc[i][j]);
      if (m == Q - 1) loads_done_barrier<(STAGES - 2) * D::kLoads>();
      if (m >= Q - 1) {
        // loads, spread over the first half of what is left
        constexpr int kSpan = (M - Q) / 2 / D::kLoads < 1 ? 1 : (M - Q) / 2 / D::kLoads;
        const int p = m - (Q - 1);
        if (p % kSpan == 0 && p / kSpan < D::kLoads)
          D::load_piece(p / kSpan, src, base + buf * D::kStage, step * kRowBytes, wave);
        if (j == FB - 1) fa[i][h] = D::fragment(ahead + (a_off ^ (64 * h)), i);
        if (i == FA - 1) fb[j][h] = D::fragment(ahead + (b_off ^ (64 * h)), j);
      }
      __builtin_amdgcn_sched_barrier(0);  // the scheduler keeps this order
    }
    step += WK;
    buf = next;
  }
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): no load may still write LDS when the workgroup ends

  using E = TileEpilogue<FA, FB, GATED>;
  static_assert(D::kWaves * E::kBytes <= WK * STAGES * D::kStage, "a part of the stages for each wave");
  __syncthreads();  // the stages are free
  if constexpr (WK > 1) {
    // the slices' sums, added in their order by the first slice's waves
    static_assert((WK - 1) * D::kWaves * FA * FB * 1024 <= WK * STAGES * D::kStage, "a part of the stages for each wave");
    v4f* sums = reinterpret_cast<v4f*>(stages) + wave * FA * FB * 64 + lane;
    constexpr int kSlice = D::kWaves * FA * FB * 64;
    if (wk > 0) {
#pragma unroll
      for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j) sums[(wk - 1) * kSlice + (i * FB + j) * 64] = acc[i][j];
    }
    __syncthreads();
    if (wk == 0) {
#pragma unroll
      for (int q = 0; q < WK - 1; ++q)
#pragma unroll
        for (int i = 0; i < FA; ++i)
#pragma unroll
          for (int j = 0; j < FB; ++j) acc[i][j] += sums[q * kSlice + (i * FB + j) * 64];
    }
    __syncthreads();  // the epilogue takes other parts
    if (wk > 0) return;
  }
  E::template run<TYPE>(a.e, acc, reinterpret_cast<float*>(stages + wave * E::kBytes), at.n0 + wn * E::OUT, at.t0 + wt * 16 * FB,
         at.t_live - wt * 16 * FB, lane);
}

// V: the variant's place in the table.
template <int V, int TYPE, int FA, int FB, int WN, int WT, int WK, bool GATED, int STAGES>
hipError_t run(Dense16Args a, hipStream_t st) {
  using D = Tile<TYPE, FA, FB, WN, WT, WK, GATED, STAGES>;
  static_assert(kDense16Tiles[V].rows == D::TN && kDense16Tiles[V].tokens == D::TT, "the tile that the choice knows");
  static_assert(kDense16Tiles[V].per_cu * WK * STAGES * D::kStage <= 160 * 1024, "LDS of a CU");
  a.n_nt = (a.N + D::COLS - 1) / D::COLS;
  a.n_tt = (int)((a.T + D::TT - 1) / D::TT);
  const dim3 grid = grid_of((int64_t)a.n_nt * a.n_tt);
  hipLaunchKernelGGL((k_dense_16<TYPE, FA, FB, WN, WT, WK, GATED, STAGES>), grid, dim3(D::kThreads), 0, st, a);
  return hipGetLastError();
}

template <int TYPE, bool GATED>
hipError_t run_variant(int variant, const Dense16Args& a, hipStream_t st) {
  switch (variant) {
    case 0: return run<0, TYPE, 8, 4, 2, 4, 1, GATED, 2>(a, st);
    case 1: return run<1, TYPE, 8, 3, 2, 4, 1, GATED, 2>(a, st);
    case 2: return run<2, TYPE, 8, 2, 2, 4, 1, GATED, 3>(a, st);
    case 3: return run<3, TYPE, 4, 2, 2, 4, 1, GATED, 4>(a, st);
    case 4: return run<4, TYPE, 4, 1, 2, 4, 1, GATED, 3>(a, st);
    case 5: return run<5, TYPE, 4, 1, 1, 4, 1, GATED, 4>(a, st);
    default: return run<6, TYPE, 4, 1, 1, 2, 4, GATED, 3>(a, st);
  }
}

// `p` of `type` at a row.
const char* row_of(const void* p, int type, int64_t row, int64_t stride) {
  return static_cast<const char*>(p) + row * stride * (type == LAT_MOE_F32 ? 4 : 2);
}

template <int TYPE, bool GATED>
hipError_t launch(Dense16Args a, int num_cus, hipStream_t st) {
  const int64_t weight_rows = (GATED ? 2 : 1) * (int64_t)a.N;
  const int steps = (a.K + kStep - 1) / kStep;
  int64_t left = a.T;
  while (left) {
    a.T = left;
    if (dense16_small(left, weight_rows, num_cus)) return launch_dense_16_small(a, TYPE, GATED, num_cus, st);
    const Dense16Launch plan = dense16_plan(left, weight_rows, steps, num_cus);
    a.T = plan.tokens;
    const hipError_t rc = run_variant<TYPE, GATED>(plan.variant, a, st);
    if (rc != hipSuccess) return rc;
    left -= plan.tokens;
    a.x = row_of(a.x, TYPE, plan.tokens, a.x_stride);
    if (a.e.residual) a.e.residual = row_of(a.e.residual, a.e.residual_type, plan.tokens, a.e.residual_stride);
    if (a.e.y) a.e.y = const_cast<char*>(row_of(a.e.y, a.e.y_type, plan.tokens, a.e.y_stride));
    if (a.e.y_q8) a.e.y_q8 += plan.tokens * (a.N / 32) * kQ81Bytes;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_dense_16(const Dense16Args& a, int type, bool gated, int num_cus, hipStream_t st) {
  if (type == LAT_MOE_BF16)
    return gated ? launch<LAT_MOE_BF16, true>(a, num_cus, st) : launch<LAT_MOE_BF16, false>(a, num_cus, st);
  return gated ? launch<LAT_MOE_F16, true>(a, num_cus, st) : launch<LAT_MOE_F16, false>(a, num_cus, st);
}

}  // namespace latmoe
