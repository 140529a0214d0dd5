// The gated linear recurrence, streamed: inputs go through shared memory in
// bulk copies, and the tiles that follow one another in time belong to the
// CTAs of one cluster.
//
// A cluster takes 64 channels of one batch entry from the first step to the
// last.  Its C CTAs take the tiles in turn (tile n C + rank in wave n).  Every
// CTA sends the map of its tile to all of them, into their shared memory, and
// each then runs the same chain of states over all maps in their order.  So no
// tile waits for another's result, only for maps that all depend on nothing
// but the inputs, and a wave's maps arrive while the next wave is composed.
// Nothing goes through global memory but inputs and outputs, and the result
// does not depend on timing.  (A look-back through global memory, in place of
// the cluster, took 231 us for 8 x 4096 x 2048 with fp32 gates and 1034 us for
// 65536 x 2048: a tile held its shared memory for the three to five L2 round
// trips that a look-back takes.)  These take 85 and 186 us (6.3 and 5.8 TB/s),
// the packed backward pass over 32768 x 2048 with fp32 gates 253 (6.4 TB/s):
// HBM bounds them.
//
// Warps of a CTA: one copies inputs (bulk tensor copies) into a ring of stages;
// two groups of four take the waves in turn, each warp a quarter of the tile's
// steps: a group composes its steps to maps, and once the start state has come
// runs its steps again from shared memory and stores, while the other group
// does the other part of its wave; one warp composes the four maps to the
// tile's and sends it; one runs the chain of states.  Clusters take columns
// (64 channels of a batch entry) in turn, without a pause between them.
//
// A warp may compose its next wave while another of its group still reads the
// maps of this one, so the warps' maps have two slots for each group, too.
//
// The map slots are two for each group: a CTA composes wave n after it finished
// wave n - 2, which took all maps of wave n - 2, and so every CTA had composed
// wave n - 2 by then and finished wave n - 4, whose slot is the one to
// overwrite.
//
// Rows of a multiple of 8 channels (EIGHT) are copied by their three
// coordinates, 64 channels x the tile's steps at once, and a lane has the
// channels 2 l and 2 l + 1.  Other rows do not start on the 16-byte boundaries
// that a copy needs, but eight of them together do: all rows of all entries are
// one matrix of eight rows a line, and a tile's rows of one remainder mod 8 are
// a box of it, from the 16-byte boundary at or before their first channel.  So
// a tile takes eight copies a tensor, its rows have a piece of 16 bytes more in
// shared memory, and a lane has the channels l and l + 32.  (Keeping pairs of
// channels where rows have an even length, with half the loads and stores,
// gained 1 % at 3 x 37651 x 494.)  The last rows, if not a whole line, are in no
// box; the warps fetch them.
#pragma once

#include <atomic>
#include <cstring>
#include <type_traits>

#include "cluster.cuh"
#include "linear_scan.cuh"
#include "linear_scan_call.h"

namespace kdn {

constexpr int kLsGroups = 2;   // groups of four warps
constexpr int kLsStreamWarps = 4 * kLsGroups + 3;
constexpr int kLsStreamThreads = 32 * kLsStreamWarps;
constexpr int kLsCluster = 8;  // CTAs of a cluster, at most

// Everything a call has; the forward uses a, b, x -> y, hT, the backward
// a, b, x, y, dy -> da, db, dx, dh0 (h0 as the forward, end_in = dh_T).
struct LsArgs {
  const float* h0;               // initial states or null
  const float* end_in;           // backward: dh_T or null
  void *out0, *out1, *out2;      // y | da, dx, db
  float* end_out;                // h_T | dh0
  const int32_t* cu;             // packed: offsets
  int N, T, D, groups;           // sequences, steps, channels, channel groups
  int chunks;                    // tiles along the steps
  int64_t cols;                  // columns: batch entries x channel groups
  int64_t lines8;                // not EIGHT: rows of all entries that are in whole lines of 8
  const void* in[5];             // not EIGHT: the tensors of the maps, for the rows behind them
  uint32_t* error;
  int64_t skip;                  // (LsCall)
};

template <bool BWD, typename GT, typename XT, bool HAS_B, bool EIGHT>
struct LsStage {
  // bytes of a step and channel over all inputs
  static constexpr int G = sizeof(GT), X = sizeof(XT);
  static constexpr int PER = BWD ? G + 2 * X + (HAS_B ? G + X : 0) : G + X + (HAS_B ? G : 0);
  // Steps of a warp, so that a CTA of two an SM has three stages at least.
  // Without EIGHT a tile of 16 steps is mostly copies of two rows each, so there
  // it is 32 steps, with one CTA an SM where that needs more room (8 x 6597 x 45,
  // backward with fp32 gates: 47 us in place of 87; 8 x 4096 x 2047 434 and 444).
  static constexpr int WIDE = EIGHT ? 64 : 72;  // (at most)
  static constexpr int LW = PER * WIDE * 64 <= 30000 ? 16 : PER * WIDE * 32 <= 30000 || !EIGHT ? 8 : 4;
  static constexpr int STEPS = 4 * LW;
  // channels of a row as copied, and elements of a box: a tensor's whole tile,
  // or every eighth row of it (boxes start on 128 bytes)
  static constexpr int WG = EIGHT ? kLsChannels : kLsChannels + 16 / G;
  static constexpr int WX = EIGHT ? kLsChannels : kLsChannels + 16 / X;
  static constexpr int BOXES = EIGHT ? 1 : 8, BOX_ROWS = STEPS / BOXES;
  static constexpr int BG = (BOX_ROWS * WG * G + 127) / 128 * 128 / G;
  static constexpr int BX = (BOX_ROWS * WX * X + 127) / 128 * 128 / X;
  static constexpr uint32_t GS = BOXES * BG * G, XS = BOXES * BX * X;  // bytes of a tensor
  // a | x or dy | y (backward) | b | x (backward with b)
  static constexpr uint32_t A = 0, X0 = GS, Y = X0 + XS, B = BWD ? Y + XS : Y, X1 = B + GS;
  static constexpr uint32_t BYTES = X1 + (HAS_B && BWD ? XS : 0) - (HAS_B ? 0 : GS);
  // bytes that the copies bring
  static constexpr uint32_t SENT =
      STEPS * (WG * G * (HAS_B ? 2 : 1) + WX * X * (BWD ? HAS_B ? 3 : 2 : 1));
  // element of channel 0 (or l) of the tile's row i, `e` being the row's
  // offset from a 16-byte boundary
  static constexpr __device__ int at_g(int i, uint32_t e) {
    return EIGHT ? i * WG : (i & 7) * BG + (i >> 3) * WG + (int)(e & (16 / G - 1));
  }
  static constexpr __device__ int at_x(int i, uint32_t e) {
    return EIGHT ? i * WX : (i & 7) * BX + (i >> 3) * WX + (int)(e & (16 / X - 1));
  }
  static constexpr int CTAS = BYTES > 29400 ? 1 : 2;  // of an SM
  // (the static arrays take less than 26.5 KB, the system 1 KB a CTA)
  static constexpr int ROOM = (233472 / CTAS - 1024 - 27136 - 128) / (int)BYTES;
  static constexpr int STAGES = ROOM < 6 ? ROOM : 6;
  static constexpr uint32_t SMEM = STAGES * BYTES + 128;
  static_assert(STAGES >= 3, "a stage for each group and one that loads");
};

__device__ __forceinline__ void ls_tma_load(void* dst, const void* tmap, uint64_t* bar, int c, int t,
                                            int b) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(tmap), "r"(smem_u32(bar)), "r"(c), "r"(t), "r"(b)
      : "memory");
}
__device__ __forceinline__ void ls_tma_load(void* dst, const void* tmap, uint64_t* bar, int c, int t) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(tmap), "r"(smem_u32(bar)), "r"(c), "r"(t)
      : "memory");
}
// A tensor's tile from global row R, channel c0 (steps t of entry bi), by lane 0,
// or each box by a lane of its own (a thread that issues all of a tile's 24 to
// 40 copies holds the ring up: 8 x 6597 x 45, backward with fp32 gates, 98 us in place of
// 87).
// es: bytes of an element; box: bytes of a box.
template <bool EIGHT>
__device__ __forceinline__ void ls_copy(uint8_t* dst, const void* tmap, uint64_t* bar, int c0, int t,
                                        int bi, int64_t R, int D, int es, uint32_t box, int lane) {
  if constexpr (EIGHT) {
    if (lane == 0) ls_tma_load(dst, tmap, bar, c0, t, bi);
  } else if (lane < 8) {
    const int64_t row = R + lane;
    const int x = ((int)(row & 7) * D + c0) & ~(16 / es - 1);
    ls_tma_load(dst + lane * box, tmap, bar, x, (int)(row >> 3));
  }
}
__device__ __forceinline__ float2 ls_sh2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 ls_sh2(const __nv_bfloat16* p) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ float2 ls_sh1(const float* p) { return make_float2(p[0], p[32]); }
__device__ __forceinline__ float2 ls_sh1(const __nv_bfloat16* p) {
  return make_float2(__bfloat162float(p[0]), __bfloat162float(p[32]));
}
__device__ __forceinline__ void ls_put(float* p, float v) { *p = v; }
__device__ __forceinline__ void ls_put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// The sequence of token t (as ls_sequence_of), by the whole warp: each round
// narrows the range 32-fold.
__device__ __forceinline__ int ls_sequence_warp(const int32_t* cu, int N, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = N;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int at = lo + lane * step;
    const bool le = lane * step < n && __ldg(cu + at) <= t;
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    // the last true of the leading ones (offsets that are in order give
    // nothing else)
    const int k = m ? 31 - __clz(m) : 0;
    n = min(step, n - k * step);
    lo += k * step;
  }
  return lo;
}
// Bits i of steps t0 + i that begin / end a sequence, for `len` steps.
__device__ __forceinline__ void ls_boundaries(const int32_t* cu, int N, int t0, int len,
                                              uint32_t& first, uint32_t& fin) {
  const int lane = threadIdx.x & 31;
  uint32_t f = 0, e = 0;
  int s = ls_sequence_warp(cu, N, t0);
  for (;; s += 32) {
    const int x = s + lane <= N ? __ldg(cu + s + lane) : 0x7fffffff;
    const int64_t d = (int64_t)x - t0;
    if (d >= 0 && d < len) f |= 1u << (int)d;
    if (d >= 1 && d <= len) e |= 1u << (int)(d - 1);
    // (any offset past the range ends the search)
    if (s + 32 > N || __any_sync(0xffffffffu, d > len)) break;
  }
  first = __reduce_or_sync(0xffffffffu, f);
  fin = __reduce_or_sync(0xffffffffu, e);
}

// 16 bytes into the same place of CTA `rank`'s shared memory, counted by its
// barrier
__device__ __forceinline__ void ls_send(const void* at, uint64_t* bar, uint32_t rank, float4 v) {
  asm volatile(
      "{\n\t.reg .b32 a, m;\n\t"
      "mapa.shared::cluster.u32 a, %0, %2;\n\t"
      "mapa.shared::cluster.u32 m, %1, %2;\n\t"
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [a], {%3, %4, %5, %6}, [m];"
      "\n\t}" ::"r"(smem_u32(at)),
      "r"(smem_u32(bar)), "r"(rank), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
      : "memory");
}

template <bool BWD, typename GT, typename XT, bool HAS_B, bool PACKED, bool EIGHT>
__global__ void __launch_bounds__(kLsStreamThreads, LsStage<BWD, GT, XT, HAS_B, EIGHT>::CTAS)
linear_scan_stream_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mx,
                          const __grid_constant__ CUtensorMap my, const __grid_constant__ CUtensorMap mb,
                          const __grid_constant__ CUtensorMap mx1, const LsArgs p) {
  using S = LsStage<BWD, GT, XT, HAS_B, EIGHT>;
  constexpr int LW = S::LW;
  constexpr int NS = S::STAGES;
  extern __shared__ __align__(128) uint8_t stream_raw[];
  constexpr int G = kLsGroups, W = 2 * G;
  __shared__ float4 warp_map[W][4][32];           // [wave % W][warp][lane]
  __shared__ float4 tile_map[W][kLsCluster][32];  // [wave % W][rank][lane]
  __shared__ float2 start[G][32];
  __shared__ uint64_t full[NS], empty[NS], mapped[G], maps_full[W], carried[G];
  __shared__ uint32_t abort_word;
  uint8_t* sm = stream_raw + ((128u - (smem_u32(stream_raw) & 127u)) & 127u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank(), C = (int)cluster_size();
  // this cluster's columns: col0, col0 + ncl, ...; a wave is C tiles of one
  const int ncl = (int)gridDim.x / C, col0 = (int)blockIdx.x / C;
  const int waves = (p.chunks + C - 1) / C;
  const int64_t total = (p.cols - col0 + ncl - 1) / ncl * waves;
  struct Pos {  // the column and wave of n
    int64_t col;
    int wave;
  };
  auto next = [&](Pos& q, int by) {
    for (q.wave += by; q.wave >= waves; q.wave -= waves) q.col += ncl;
  };
  volatile uint32_t* abort_flag = &abort_word;
  auto fail = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (*abort_flag) return true;
    if (mbar_wait(bar, parity)) return false;
    *abort_flag = 1u;
    atomicOr(p.error, DEV_TIMEOUT);
    return true;
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    for (int i = 0; i < G; ++i) {
      mbar_init(&mapped[i], 4);
      mbar_init(&carried[i], 1);
    }
    for (int i = 0; i < W; ++i) mbar_init(&maps_full[i], 1);
    abort_word = 0u;
    // (only this block reports bad offsets, and no wait gives up before it has
    // begun)
    if (blockIdx.x == 0) *p.error = DEV_OK;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  cluster_sync_all();

  // (at least 0, so that no difference with a step overflows)
  const int end = PACKED ? max(0, min(p.T, __ldg(p.cu + p.N))) : p.T;
  // first step of a tile (the backward counts tiles from the end)
  // a lane's two channels in a column's 64, and a state's two values
  const int l0 = EIGHT ? 2 * lane : lane, l1 = EIGHT ? 2 * lane + 1 : lane + 32;
  auto get2 = [&](const float* v, size_t at, int c0) -> float2 {  // row `at` of [.., D]
    const float* r = v + at * p.D + c0;
    if (EIGHT) return c0 + l0 < p.D ? *reinterpret_cast<const float2*>(r + l0) : make_float2(0.f, 0.f);
    return make_float2(c0 + l0 < p.D ? r[l0] : 0.f, c0 + l1 < p.D ? r[l1] : 0.f);
  };
  auto set2 = [&](float* v, size_t at, int c0, float2 x) {
    float* r = v + at * p.D + c0;
    if (EIGHT) {
      if (c0 + l0 < p.D) *reinterpret_cast<float2*>(r + l0) = x;
    } else {
      if (c0 + l0 < p.D) r[l0] = x.x;
      if (c0 + l1 < p.D) r[l1] = x.y;
    }
  };
  auto tile_start = [&](int j) -> int {
    return (BWD ? p.chunks - 1 - j : j) * S::STEPS;
  };

  if (warp == 4 * G) {
    // ------------------------------------------------------------- copies
    int64_t n = 0;
    int st = 0;
    uint32_t phase = 1;
    Pos q{col0, 0};
    const int64_t skip = blockIdx.x == 0 ? p.skip : -1;
    // (one lane where it issues alone: a vote of the warp each time costs 6 %)
    for (; n < total && (!EIGHT || lane == 0); ++n, next(q, 1)) {
      const bool bad = n >= NS && lane == 0 && fail(&empty[st], phase);
      if (EIGHT ? bad : __any_sync(0xffffffffu, bad) != 0) break;
      const int j = q.wave * C + rank;
      if (j < p.chunks) {
        const int bi = (int)(q.col / p.groups), t = tile_start(j);
        const int c0 = (int)(q.col - (int64_t)bi * p.groups) * kLsChannels;
        uint8_t* d = sm + (uint32_t)st * S::BYTES;
        const int64_t R = (int64_t)bi * p.T + t;
        if (lane == 0) mbar_expect_tx(&full[st], S::SENT);
        if (!EIGHT) __syncwarp();
        auto copy = [&](uint32_t at, const CUtensorMap& m, int back, int es, uint32_t box) {
          if (n != skip)
            ls_copy<EIGHT>(d + at, &m, &full[st], c0, t - back, bi, R - back, p.D, es, box, lane);
        };
        copy(S::A, ma, 0, S::G, S::BG * S::G);
        copy(S::X0, mx, 0, S::X, S::BX * S::X);
        if (BWD) copy(S::Y, my, 1, S::X, S::BX * S::X);
        if (HAS_B) copy(S::B, mb, 0, S::G, S::BG * S::G);
        if (BWD && HAS_B) copy(S::X1, mx1, 0, S::X, S::BX * S::X);
      } else if (lane == 0) {
        mbar_arrive(&full[st]);
      }
      if (++st == NS) {
        st = 0;
        phase ^= 1u;
      }
    }
    // copies in flight land before the CTA's memory goes, whatever became of
    // the other warps (bounded)
    if (lane == 0)
      for (int64_t i = n > NS ? n - NS : 0; i < n; ++i)
        mbar_wait(&full[i % NS], (uint32_t)(i / NS) & 1u);
  } else if (warp == 4 * G + 1) {
    // --------------------------------------------------- the tile's map, sent
    Pos q{col0, 0};
    for (int64_t n = 0; n < total; ++n, next(q, 1)) {
      const int g = (int)(n % G), sl = (int)(n % W);
      float4 m = make_float4(1.f, 0.f, 1.f, 0.f);  // (no tile: the identity)
      const bool bad = fail(&mapped[g], (uint32_t)(n / G) & 1u);
      if (__any_sync(0xffffffffu, bad)) break;
      if (q.wave * C + rank < p.chunks) {
        m = warp_map[sl][BWD ? 3 : 0][lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) {
          const float4 l = warp_map[sl][BWD ? 3 - w : w][lane];
          ls_compose<PACKED>(m.x, m.y, l.x, l.y);
          ls_compose<PACKED>(m.z, m.w, l.z, l.w);
        }
      }
      if (lane == 0) mbar_expect_tx(&maps_full[sl], (uint32_t)C * 512u);
      __syncwarp();
      for (int r = 0; r < C; ++r) ls_send(&tile_map[sl][rank][lane], &maps_full[sl], r, m);
    }
  } else if (warp == 4 * G + 2) {
    // ---------------------------------------------------- the chain of states
    // the state before a column's first tile
    auto enter = [&](int64_t col) -> float2 {
      const float* e = BWD ? p.end_in : p.h0;
      if (PACKED || !e || col >= p.cols) return make_float2(0.f, 0.f);
      const int bi = (int)(col / p.groups);
      return get2(e, bi, (int)(col - (int64_t)bi * p.groups) * kLsChannels);
    };
    Pos q{col0, 0};
    float2 state = make_float2(0.f, 0.f), later = enter(col0);
    int64_t n = 0;
    for (; n < total; ++n, next(q, 1)) {
      const int g = (int)(n % G), sl = (int)(n % W);
      if (q.wave == 0) {
        state = later;
        later = enter(q.col + ncl);
      }
      const bool bad = fail(&maps_full[sl], (uint32_t)(n / W) & 1u);
      if (__any_sync(0xffffffffu, bad)) break;
      float4 m[kLsCluster];
#pragma unroll
      for (int r = 0; r < kLsCluster; ++r)
        if (r < C) m[r] = tile_map[sl][r][lane];
#pragma unroll
      for (int r = 0; r < kLsCluster; ++r)
        if (r < C) {
          if (r == rank) start[g][lane] = state;
          state.x = ls_apply<PACKED>(m[r].x, m[r].y, state.x);
          state.y = ls_apply<PACKED>(m[r].z, m[r].w, state.y);
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&carried[g]);
    }
    // Where this gave up, maps that the other CTAs have sent land before the CTA's
    // memory goes (bounded; they cannot send more than the slots hold).
    if (lane == 0)
      for (int64_t i = n; i < total && i < n + W; ++i)
        if (!mbar_wait(&maps_full[i % W], (uint32_t)(i / W) & 1u)) break;
  } else {
    // ------------------------------------------------------------- steps
    const int g = warp >> 2, w4 = warp & 3;
    Pos q{col0, 0};
    next(q, g);
    uint32_t first = 0, fin = 0;  // steps that begin and that end a sequence
    // packed: what these steps need, if there is one of each at most
    struct Edge {
      int begins, ends;  // the sequences
      float2 in, h0;     // the state that enters (backward: at the end), and h0
    };
    Edge edge{};
    auto look = [&](uint32_t f, uint32_t e, int t, int c0) -> Edge {
      Edge x{};
      x.in = x.h0 = make_float2(0.f, 0.f);
      if (__popc(f) > 1 || __popc(e) > 1) return x;
      if (f) x.begins = ls_sequence_warp(p.cu, p.N, t + __ffs(f) - 1);
      if (e) x.ends = ls_sequence_warp(p.cu, p.N, t + __ffs(e) - 1);
      if (f && p.h0) x.h0 = get2(p.h0, x.begins, c0);
      if (!BWD) x.in = x.h0;
      else if (e && p.end_in) x.in = get2(p.end_in, x.ends, c0);
      return x;
    };
    for (int64_t n = g; n < total; n += G, next(q, G)) {
      const int st = (int)(n % NS), sl = (int)(n % W);
      const int bi = (int)(q.col / p.groups), grp = (int)(q.col - (int64_t)bi * p.groups);
      const int c0 = grp * kLsChannels;
      const bool in0 = c0 + l0 < p.D, in1 = c0 + l1 < p.D;
      const int j = q.wave * C + rank;
      // this warp's first step, and how many it has
      const int t0 = tile_start(min(j, p.chunks - 1)) + w4 * LW;
      const int len = j < p.chunks ? max(0, min(LW, end - t0)) : 0;
      if (!PACKED) {
        first = len > 0 && t0 == 0 ? 1u : 0u;
        fin = len > 0 && p.T - 1 - t0 < LW ? 1u << (p.T - 1 - t0) : 0u;
      } else if (n == g && len > 0) {
        ls_boundaries(p.cu, p.N, t0, len, first, fin);
        edge = look(first, fin, t0, c0);
      }
      const bool plain = len == LW && (!PACKED || (first | fin) == 0u);
      const bool single = PACKED && len == LW && __popc(first) <= 1 && __popc(fin) <= 1;
      const uint8_t* d = sm + (uint32_t)st * S::BYTES;
      // inputs of the warp's step i (hp: the state before it, in y)
      const int i0 = w4 * LW;
      // (only its remainders mod 8 are used)
      const uint32_t e0 = EIGHT ? 0u : (uint32_t)(((int64_t)bi * p.T + t0) * p.D);
      auto get_g = [&](uint32_t at, int i) -> float2 {
        const GT* v = reinterpret_cast<const GT*>(d + at) + S::at_g(i0 + i, e0 + (uint32_t)(i * p.D)) + l0;
        return EIGHT ? ls_sh2(v) : ls_sh1(v);
      };
      auto get_x = [&](uint32_t at, int i, int back) -> float2 {
        const XT* v =
            reinterpret_cast<const XT*>(d + at) + S::at_x(i0 + i, e0 + (uint32_t)((i - back) * p.D)) + l0;
        return EIGHT ? ls_sh2(v) : ls_sh1(v);
      };
      auto in_a = [&](int i) { return get_g(S::A, i); };
      auto in_x = [&](int i) { return get_x(S::X0, i, 0); };
      auto in_hp = [&](int i) { return get_x(S::Y, i, 1); };
      auto in_b = [&](int i) { return get_g(S::B, i); };
      auto in_x1 = [&](int i) { return get_x(S::X1, i, 0); };
      // outputs of step i: `o` is the lane's place in step 0
      const size_t out0 = ((size_t)bi * p.T + t0) * p.D + c0 + l0;
      auto put = [&](auto* o, int i, float2 v) {
        o += (size_t)i * p.D;
        if (EIGHT) {
          if (in0) ls_store2<true>(o, 0, 1, v);
        } else {
          if (in0) ls_put(o, v.x);
          if (in1) ls_put(o + 32, v.y);
        }
      };
      bool bad = fail(&full[st], (uint32_t)(n / NS) & 1u);
      if (__any_sync(0xffffffffu, bad)) break;
      if constexpr (!EIGHT) {
        // rows in no box (backward: its y is the row before)
        const int64_t R = (int64_t)bi * p.T + t0;
        if (len > 0 && R + len > p.lines8) {
          auto fetch_row = [&](auto* to, const void* from, int64_t row) {
            using V = std::remove_reference_t<decltype(*to)>;
            const V* src = static_cast<const V*>(from) + row * p.D + c0;
            if (in0) to[l0] = src[l0];
            if (in1) to[l1] = src[l1];
          };
          uint8_t* w = sm + (uint32_t)st * S::BYTES;
          for (int i = 0; i < len; ++i) {
            const int eg = S::at_g(i0 + i, e0 + (uint32_t)(i * p.D)), ex = S::at_x(i0 + i, e0 + (uint32_t)(i * p.D));
            if (R + i >= p.lines8) {
              fetch_row(reinterpret_cast<GT*>(w + S::A) + eg, p.in[0], R + i);
              fetch_row(reinterpret_cast<XT*>(w + S::X0) + ex, p.in[1], R + i);
              if (HAS_B) fetch_row(reinterpret_cast<GT*>(w + S::B) + eg, p.in[3], R + i);
              if (BWD && HAS_B) fetch_row(reinterpret_cast<XT*>(w + S::X1) + ex, p.in[4], R + i);
            }
            if (BWD && R + i > p.lines8)
              fetch_row(reinterpret_cast<XT*>(w + S::Y) + S::at_x(i0 + i, e0 + (uint32_t)((i - 1) * p.D)),
                        p.in[2], R + i - 1);
          }
          // (before a later copy into the stage)
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
      }
      // -------------------------------------------------------- compose
      // steps at which this direction starts afresh
      const uint32_t fresh = PACKED ? (BWD ? fin : first) : 0u;
      float2 A = make_float2(1.f, 1.f), H = make_float2(0.f, 0.f);
      if (len == LW && fresh == 0u) {
#pragma unroll
        for (int k = 0; k < LW; ++k) {
          const int i = BWD ? LW - 1 - k : k;
          const float2 a = in_a(i);
          float2 u = in_x(i);
          if (BWD) {
            H = __fmul2_rn(a, __fadd2_rn(H, u));
          } else {
            if (HAS_B) u = __fmul2_rn(u, in_b(i));
            H = __ffma2_rn(a, H, u);
          }
          A = __fmul2_rn(A, a);
        }
        if (PACKED) {  // never the mark
          A.x += 0.f;
          A.y += 0.f;
        }
      } else if (single) {
        // the state is selected at the one step that starts afresh; the map
        // is constant from there on
#pragma unroll
        for (int k = 0; k < LW; ++k) {
          const int i = BWD ? LW - 1 - k : k;
          const float2 a = in_a(i);
          float2 u = in_x(i);
          if ((fresh >> i) & 1u) H = edge.in;
          if (BWD) {
            H = __fmul2_rn(a, __fadd2_rn(H, u));
          } else {
            if (HAS_B) u = __fmul2_rn(u, in_b(i));
            H = __ffma2_rn(a, H, u);
          }
        }
        A.x = A.y = ls_const_mark();
      } else {
        for (int k = 0; k < len; ++k) {
          const int i = BWD ? len - 1 - k : k;
          float2 a = in_a(i), u = in_x(i);
          const bool f = (fresh >> i) & 1u;
          float2 e = make_float2(0.f, 0.f);
          const float* ends = BWD ? p.end_in : p.h0;
          if (f && ends) {
            const int s = ls_sequence_warp(p.cu, p.N, t0 + i);
            e = get2(ends, s, c0);
          }
          if (BWD) {
            u = __fmul2_rn(a, __fadd2_rn(u, e));
          } else {
            if (HAS_B) u = __fmul2_rn(u, in_b(i));
            if (f) u = __ffma2_rn(a, e, u);
          }
          ls_compose<PACKED>(A.x, H.x, f ? ls_const_mark() : a.x + 0.f, u.x);
          ls_compose<PACKED>(A.y, H.y, f ? ls_const_mark() : a.y + 0.f, u.y);
        }
      }
      warp_map[sl][w4][lane] = make_float4(A.x, H.x, A.y, H.y);
      __syncwarp();
      if (lane == 0) mbar_arrive(&mapped[g]);

      // the boundaries of this group's next tile, while the state is on its way
      uint32_t next_first = 0, next_fin = 0;
      Edge next_edge{};
      if (PACKED && n + G < total) {
        Pos qn = q;
        next(qn, G);
        const int tile = qn.wave * C + rank, tn = tile_start(min(tile, p.chunks - 1)) + w4 * LW;
        const int ln = tile < p.chunks ? max(0, min(LW, end - tn)) : 0;
        if (ln > 0) {
          ls_boundaries(p.cu, p.N, tn, ln, next_first, next_fin);
          if (next_first | next_fin)
            next_edge = look(next_first, next_fin, tn, (int)(qn.col % p.groups) * kLsChannels);
        }
      }

      // --------------------------------------------------------- finish
      float2 enter = make_float2(0.f, 0.f);  // backward, dense: the state before step 0
      if (BWD && !PACKED && first && p.h0) enter = get2(p.h0, bi, c0);
      // (mapped: the other warps' maps)
      bad = fail(&mapped[g], (uint32_t)(n / G) & 1u) || fail(&carried[g], (uint32_t)(n / G) & 1u);
      if (__any_sync(0xffffffffu, bad)) break;
      float2 h = start[g][lane];
      for (int w = 0; w < (BWD ? 3 - w4 : w4); ++w) {
        const float4 m = warp_map[sl][BWD ? 3 - w : w][lane];
        h.x = ls_apply<PACKED>(m.x, m.y, h.x);
        h.y = ls_apply<PACKED>(m.z, m.w, h.y);
      }
      if constexpr (!BWD) {
        XT* Y = static_cast<XT*>(p.out0) + out0;
        if (plain) {
#pragma unroll
          for (int i = 0; i < LW; ++i) {
            float2 u = in_x(i);
            if (HAS_B) u = __fmul2_rn(u, in_b(i));
            h = __ffma2_rn(in_a(i), h, u);
            put(Y, i, h);
          }
          if (!PACKED && fin) set2(p.end_out, bi, c0, h);
        } else if (single) {
          float2 leaves = h;
#pragma unroll
          for (int i = 0; i < LW; ++i) {
            float2 u = in_x(i);
            if (HAS_B) u = __fmul2_rn(u, in_b(i));
            if ((first >> i) & 1u) h = edge.in;
            h = __ffma2_rn(in_a(i), h, u);
            put(Y, i, h);
            if ((fin >> i) & 1u) leaves = h;
          }
          if (fin) set2(p.end_out, edge.ends, c0, leaves);
        } else {
          for (int i = 0; i < len; ++i) {
            float2 u = in_x(i);
            if (HAS_B) u = __fmul2_rn(u, in_b(i));
            const bool f = PACKED && ((first >> i) & 1u), e = (fin >> i) & 1u;
            int s = bi;
            if (PACKED && (f || e)) s = ls_sequence_warp(p.cu, p.N, t0 + i);
            if (f) {
              h = make_float2(0.f, 0.f);
              if (p.h0) h = get2(p.h0, s, c0);
            }
            h = __ffma2_rn(in_a(i), h, u);
            put(Y, i, h);
            if (e) set2(p.end_out, s, c0, h);
          }
        }
      } else {
        GT* dA = static_cast<GT*>(p.out0) + out0;
        XT* dX = static_cast<XT*>(p.out1) + out0;
        GT* dB = static_cast<GT*>(p.out2) + (HAS_B ? out0 : 0);
        auto step = [&](int i, float2 hp) {
          const float2 gr = __fadd2_rn(in_x(i), h);
          put(dA, i, __fmul2_rn(gr, hp));
          if (HAS_B) {
            put(dX, i, __fmul2_rn(gr, in_b(i)));
            put(dB, i, __fmul2_rn(gr, in_x1(i)));
          } else {
            put(dX, i, gr);
          }
          h = __fmul2_rn(in_a(i), gr);
        };
        if (plain) {
#pragma unroll
          for (int k = 0; k < LW; ++k) {
            const int i = LW - 1 - k;
            float2 hp = in_hp(i);
            if (!PACKED && i == 0 && first) hp = enter;
            step(i, hp);
          }
          if (!PACKED && first) set2(p.end_out, bi, c0, h);
        } else if (single) {
          float2 leaves = h;
#pragma unroll
          for (int k = 0; k < LW; ++k) {
            const int i = LW - 1 - k;
            if ((fin >> i) & 1u) h = edge.in;
            float2 hp = in_hp(i);
            if ((first >> i) & 1u) hp = edge.h0;
            step(i, hp);
            if ((first >> i) & 1u) leaves = h;
          }
          if (first) set2(p.end_out, edge.begins, c0, leaves);
        } else {
          for (int i = len - 1; i >= 0; --i) {
            const bool f = (first >> i) & 1u, e = PACKED && ((fin >> i) & 1u);
            int s = bi;
            if (PACKED && (f || e)) s = ls_sequence_warp(p.cu, p.N, t0 + i);
            if (e) {
              h = make_float2(0.f, 0.f);
              if (p.end_in) h = get2(p.end_in, s, c0);
            }
            float2 hp = in_hp(i);
            if (f) {
              hp = make_float2(0.f, 0.f);
              if (p.h0) hp = get2(p.h0, s, c0);
            }
            step(i, hp);
            if (f) set2(p.end_out, s, c0, h);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
      if (PACKED && j == 0) {
        // sequences without steps hand their state (or its gradient) through
        const float* ends = BWD ? p.end_in : p.h0;
        for (int s = w4; s < p.N; s += 4)
          if (__ldg(p.cu + s) >= __ldg(p.cu + s + 1))
            set2(p.end_out, s, c0, ends ? get2(ends, s, c0) : make_float2(0.f, 0.f));
        if (grp == 0 && w4 == 0) {
          bool odd = false;
          for (int i = lane; i <= p.N; i += 32) {
            const int x = __ldg(p.cu + i);
            odd |= x < 0 || x > p.T || (i == 0 && x != 0) || (i > 0 && x < __ldg(p.cu + i - 1));
          }
          if (odd) atomicOr(p.error, DEV_BAD_ARG);
        }
      }
      if (PACKED) {
        first = next_first;
        fin = next_fin;
        edge = next_edge;
      }
    }
  }
  // no CTA's shared memory goes while another may still write to it
  __syncwarp();
  cluster_sync_all();
}

// ------------------------------------------------------------------- host
// EIGHT: [entries, T, D] of 2- or 4-byte elements, boxes of 64 channels x the
// tile's steps; else lines of eight rows of D, boxes of one row a line.
template <bool EIGHT>
bool ls_map(CUtensorMap* m, const void* base, int es, int64_t entries, int64_t T, int64_t D,
            int wide, int box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)T, (cuuint64_t)entries};
  cuuint64_t strides[2] = {(cuuint64_t)(D * es), (cuuint64_t)(T * D * es)};
  if (!EIGHT) {
    dims[0] = (cuuint64_t)(8 * D);
    dims[1] = (cuuint64_t)(entries * T / 8);
    strides[0] = (cuuint64_t)(8 * D * es);
  }
  cuuint32_t box[3] = {(cuuint32_t)wide, (cuuint32_t)box_rows, 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  return enc(m, es == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
             EIGHT ? 3 : 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// a, x (forward x, backward dy), y, b, x1 (backward x): the tensors in the
// order of the kernel's maps.  same: the states that enter and that leave are
// the same memory; then a CTA may only store a column's last state when all of
// its cluster have read the first, which three waves give.
template <bool BWD, typename GT, typename XT, bool HAS_B, bool PACKED, bool EIGHT>
kdn_status ls_stream_go(const void* a, const void* x, const void* y, const void* b, const void* x1,
                        LsArgs p, int entries, bool same, void* workspace, cudaStream_t s) {
  using S = LsStage<BWD, GT, XT, HAS_B, EIGHT>;
  p.groups = (p.D + kLsChannels - 1) / kLsChannels;
  p.chunks = (int)(((int64_t)p.T + S::STEPS - 1) / S::STEPS);
  p.cols = (int64_t)entries * p.groups;
  p.error = ls_ws(workspace, LsPlan{}).error;
  CUtensorMap m[5];
  memset(m, 0, sizeof(m));
  const int64_t T = p.T;
  const void* t[5] = {a, x, BWD ? y : nullptr, HAS_B ? b : nullptr, BWD && HAS_B ? x1 : nullptr};
  for (int i = 0; i < 5; ++i) {
    const bool gate = i == 0 || i == 3;
    p.in[i] = t[i];
    if (t[i] && !ls_map<EIGHT>(&m[i], t[i], gate ? S::G : S::X, entries, T, p.D,
                               gate ? S::WG : S::WX, S::BOX_ROWS))
      return KDN_ERR_CUDA;
  }
  p.lines8 = (int64_t)entries * T / 8 * 8;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kLsStreamThreads);
  cfg.dynamicSmemBytes = S::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  // Clusters of 1, 2, 4 and 8 CTAs that a device holds at once (of eight fewer
  // than its SMs would give: they do not span its parts), asked for once.
  auto kernel = linear_scan_stream_kernel<BWD, GT, XT, HAS_B, PACKED, EIGHT>;
  static std::atomic<int> known[64][4];
  int dev = 0, room[4];
  if (cudaGetDevice(&dev) != cudaSuccess) return KDN_ERR_CUDA;
  for (int i = 0; i < 4; ++i) room[i] = dev < 64 ? known[dev][i].load(std::memory_order_acquire) : 0;
  if (!room[0] || !room[1] || !room[2] || !room[3]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::SMEM) !=
        cudaSuccess)
      return KDN_ERR_CUDA;
    for (int i = 0; i < 4; ++i) {
      at[0].val.clusterDim.x = 1u << i;
      cfg.gridDim = dim3(1u << i);
      if (cudaOccupancyMaxActiveClusters(&room[i], kernel, &cfg) != cudaSuccess || room[i] < 1)
        return KDN_ERR_CUDA;
      if (dev < 64) known[dev][i].store(room[i], std::memory_order_release);
    }
  }
  // Tiles that a CTA works through one after another, for each cluster size;
  // a wave of maps costs a little more the more CTAs it comes from.
  int C = 0, clusters = 0;
  int64_t least = 0;
  for (int i = 0, c = 1; c <= kLsCluster; ++i, c *= 2) {
    const int64_t k = p.cols < room[i] ? p.cols : room[i];
    const int64_t waves = (p.chunks + c - 1) / c;
    if (c > 1 && same && waves < 3) continue;
    const int64_t cost = (p.cols + k - 1) / k * waves * (16 + c);
    if (!C || cost < least) {
      C = c;
      clusters = (int)k;
      least = cost;
    }
  }
  cfg.gridDim = dim3((unsigned)(clusters * C));
  at[0].val.clusterDim.x = (unsigned)C;
  return enqueued(cudaLaunchKernelEx(&cfg, kernel, m[0], m[1], m[2], m[3], m[4], p));
}

// Whether a call streams.  With packed sequences the second pass reads the
// states that enter a sequence again, when another tile may have stored what
// leaves it, so the two must be different memory.  One or two columns over
// many tiles leave most of the device idle, where the look-back uses all of it:
// at 16384 steps and 128 channels, fp32 gates, 32 us instead of 56 (forward)
// and 37 instead of 62 (backward), both with a write gate; at 256 channels 43
// and 56 (forward), 60 and 67 (backward), at 4096 steps and 256 channels 16.0
// and 16.4, 18.7 and 18.0.
template <bool BWD, typename GT, typename XT, bool HAS_B, bool EIGHT>
bool ls_streams(const float* enter, const float* leave, bool packed, int64_t entries, int64_t T,
                int64_t D) {
  using S = LsStage<BWD, GT, XT, HAS_B, EIGHT>;
  if (T == 0 || (packed && enter == leave)) return false;
  // (whole lines of eight rows, and 32-bit coordinates)
  if (!EIGHT && (entries * T < 8 || entries * T >= int64_t(1) << 33 || D >= 1 << 27)) return false;
  const int64_t cols = entries * ((D + kLsChannels - 1) / kLsChannels);
  return cols > 2 || T < 128 * S::STEPS;
}

template <bool BWD, bool EIGHT, typename GT, typename XT, bool HAS_B>
bool ls_stream_types(const LsCall& k, kdn_status* st) {
  const float *enter = BWD ? k.end_in : k.h0, *leave = k.end_out;
  const bool packed = k.cu != nullptr, same = enter == leave;
  if (!ls_streams<BWD, GT, XT, HAS_B, EIGHT>(enter, leave, packed, k.B, k.T, k.D)) return false;
  LsArgs p{};
  p.h0 = k.h0;
  p.end_in = k.end_in;
  p.out0 = BWD ? k.da : k.y_out;
  p.out1 = k.dx;
  p.out2 = k.db;
  p.end_out = k.end_out;
  p.cu = k.cu;
  p.N = k.N;
  p.T = k.T;
  p.D = k.D;
  p.skip = k.skip;
  const void *x = BWD ? k.dy : k.x, *x1 = BWD ? k.x : nullptr;
  *st = packed ? ls_stream_go<BWD, GT, XT, HAS_B, true, EIGHT>(k.a, x, k.y, k.b, x1, p, k.B, same,
                                                               k.workspace, k.stream)
               : ls_stream_go<BWD, GT, XT, HAS_B, false, EIGHT>(k.a, x, k.y, k.b, x1, p, k.B, same,
                                                                k.workspace, k.stream);
  return true;
}

template <bool BWD, bool EIGHT>
bool ls_stream_call(const LsCall& k, kdn_status* st) {
  using bf = __nv_bfloat16;
  switch ((k.gate_dtype == KDN_BF16 ? 4 : 0) + (k.in_dtype == KDN_BF16 ? 2 : 0) + (k.b ? 1 : 0)) {
    case 0: return ls_stream_types<BWD, EIGHT, float, float, false>(k, st);
    case 1: return ls_stream_types<BWD, EIGHT, float, float, true>(k, st);
    case 2: return ls_stream_types<BWD, EIGHT, float, bf, false>(k, st);
    case 3: return ls_stream_types<BWD, EIGHT, float, bf, true>(k, st);
    case 4: return ls_stream_types<BWD, EIGHT, bf, float, false>(k, st);
    case 5: return ls_stream_types<BWD, EIGHT, bf, float, true>(k, st);
    case 6: return ls_stream_types<BWD, EIGHT, bf, bf, false>(k, st);
    default: return ls_stream_types<BWD, EIGHT, bf, bf, true>(k, st);
  }
}

}  // namespace kdn
