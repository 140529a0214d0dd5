// Shared parts of the gated linear recurrence kernels (kdn_linear_scan_*).
//
// Per channel the recurrence h_t = a_t h_{t-1} + u_t is a composition of
// affine maps: (A, H) stands for h -> A h + H, and a later map after an
// earlier one is (A_l A_e, A_l H_e + H_l).  The backward pass is the same
// recurrence run from the last step to the first on other inputs, so both
// directions share the tile, the look-back across tiles and this map.
//
// Most calls run in the streaming form (linear_scan_stream.cuh).  The form below
// is for one or two columns of 64 channels over many steps, where its tiles
// spread over the whole device, and for packed sequences whose states are
// updated in place, since a tile here reads its inputs once.
//
// Tile: 8 warps, 64 channels, 8 * L steps.  Warp w takes the L consecutive
// steps w L ... of the tile's order, lane l the channels 2 l and 2 l + 1, and
// all inputs of a step range sit in registers: one read of every input, and a
// warp's loads (128 bytes of bf16 or 256 of fp32 a row) are all in flight
// before the first is used.  A warp composes its L steps, the tile's eight
// maps meet in shared memory, and warp 0 finds the state at the tile's start
// by look-back while the others wait: it publishes the tile's map when the
// predecessor's state is not there yet, and applies the maps behind the
// nearest published state.  Tiles are handed out by a
// counter, all channel groups' first step ranges first, so whoever is waited
// for has been handed out before; every wait is bounded.
//
// Packed sequences run as one long sequence whose maps forget: at a
// sequence's first step the map is constant (its own initial state goes into
// H).  A constant map is marked by A = -0.0 and drops what came before it by
// selection, not by multiplication, so that an infinity or NaN in one
// sequence stays out of the next (products that are zero get the sign +).
#pragma once

#include "enqueue.h"
#include "kdn_common.cuh"

namespace kdn {

constexpr int kLsWarps = 8;
constexpr int kLsThreads = kLsWarps * 32;
constexpr int kLsChannels = 64;  // channels of a tile
constexpr int kLsFwdSteps = 8;   // steps of a warp, forward (16 spill)
constexpr int kLsBwdSteps = 8;   // steps of a warp, backward (the workspace is sized by it)

struct LsWs {
  uint32_t* error;    // device error word
  uint32_t* counter;  // next tile to hand out
  uint32_t* flag;     // per tile: 0 none, 1 map published, 2 state published
  float4* map;        // per tile and lane: (A, H) of its two channels
  float2* state;      // per tile and lane: the state after the tile
};

struct LsShared {
  float4 warp_map[kLsWarps][32];
  float2 start[32];  // the state at the tile's start
  uint32_t tile;
};

__device__ __forceinline__ bool ls_const(float A) { return __float_as_uint(A) == 0x80000000u; }
__device__ __forceinline__ float ls_const_mark() { return __uint_as_float(0x80000000u); }

// (Al, Hl) after (Ae, He)
template <bool PACKED>
__device__ __forceinline__ void ls_compose(float& A, float& H, float Al, float Hl) {
  if (PACKED && ls_const(Al)) {
    A = Al;
    H = Hl;
    return;
  }
  H = fmaf(Al, H, Hl);
  if (!PACKED) A = Al * A;
  else if (!ls_const(A)) A = fmaf(Al, A, 0.f);  // never -0.0
}
// the map applied to a state
template <bool PACKED>
__device__ __forceinline__ float ls_apply(float A, float H, float h) {
  return (PACKED && ls_const(A)) ? H : fmaf(A, h, H);
}

// Two neighbouring channels at element offset `at`; channels that do not
// exist read as `fill`.  EVEN: rows have an even number of channels, so the
// pair exists or not as one, and is aligned.
template <bool EVEN>
__device__ __forceinline__ float2 ls_load2(const float* p, size_t at, int have, float fill) {
  if (EVEN) {
    if (have) return __ldg(reinterpret_cast<const float2*>(p + at));
    return make_float2(fill, fill);
  }
  return make_float2(have > 0 ? __ldg(p + at) : fill, have > 1 ? __ldg(p + at + 1) : fill);
}
template <bool EVEN>
__device__ __forceinline__ float2 ls_load2(const __nv_bfloat16* p, size_t at, int have,
                                           float fill) {
  if (EVEN) {
    if (have)
      return __bfloat1622float2(__ldg(reinterpret_cast<const __nv_bfloat162*>(p + at)));
    return make_float2(fill, fill);
  }
  return make_float2(have > 0 ? __bfloat162float(p[at]) : fill,
                     have > 1 ? __bfloat162float(p[at + 1]) : fill);
}
template <bool EVEN>
__device__ __forceinline__ void ls_store2(float* p, size_t at, int have, float2 v) {
  if (EVEN) {
    if (have) *reinterpret_cast<float2*>(p + at) = v;
    return;
  }
  if (have > 0) p[at] = v.x;
  if (have > 1) p[at + 1] = v.y;
}
template <bool EVEN>
__device__ __forceinline__ void ls_store2(__nv_bfloat16* p, size_t at, int have, float2 v) {
  if (EVEN) {
    if (have) *reinterpret_cast<__nv_bfloat162*>(p + at) = __floats2bfloat162_rn(v.x, v.y);
    return;
  }
  if (have > 0) p[at] = __float2bfloat16_rn(v.x);
  if (have > 1) p[at + 1] = __float2bfloat16_rn(v.y);
}

// The sequence of token t: the largest s in [0, N) with cu[s] <= t (0 if
// none).  Any contents of cu give an s in range.
__device__ __forceinline__ int ls_sequence_of(const int32_t* cu, int N, int t) {
  int lo = 0, hi = N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Reports offsets that are out of order or out of range (all threads of one
// block).
__device__ __forceinline__ void ls_check_offsets(const int32_t* cu, int N, int total,
                                                 uint32_t* error) {
  bool bad = false;
  for (int i = threadIdx.x; i <= N; i += kLsThreads) {
    const int x = __ldg(cu + i);
    bad |= x < 0 || x > total || (i == 0 && x != 0) || (i > 0 && x < __ldg(cu + i - 1));
  }
  if (bad) atomicOr(error, DEV_BAD_ARG);
}

// The state at the start of tile (j, col) of `cols` columns, in warp 0: m is
// the tile's map (per lane: A, H of two channels), `init` the state before the
// first tile.  Publishes what later tiles need unless this is the last one.
// Lane i watches the tile i + 1 before this one; from the nearest published
// state the maps behind it are applied one by one, exactly as their own tiles
// do, so the result does not depend on which state was found.
template <bool PACKED>
__device__ __forceinline__ float2 ls_look_back(const LsWs& ws, int64_t j, int64_t col,
                                               int64_t cols, bool last, float4 m, float2 init) {
  const int lane = threadIdx.x & 31;
  const int64_t tile = j * cols + col;
  // (the warp barrier puts every lane's stores before lane 0's release)
  auto publish = [&](uint32_t what) {
    __syncwarp();
    if (lane == 0) st_release_u32(ws.flag + tile, what);
  };
  float2 s = init;
  if (j > 0) {
    const bool there = lane < j;
    const uint32_t* watched = ws.flag + (there ? tile - (lane + 1) * cols : tile);
    uint64_t t0 = 0;
    bool published = last;
    int back = 0;  // tiles between the published state and this one
    for (;;) {
      const uint32_t f = there ? ld_acquire_u32(watched) : 0u;
      __syncwarp();
      const uint32_t states = __ballot_sync(0xffffffffu, f == 2u);
      const uint32_t maps = __ballot_sync(0xffffffffu, f != 0u);
      if (states) {
        back = __ffs(states) - 1;
        const uint32_t between = (1u << back) - 1u;
        if ((maps & between) == between) break;
      }
      if (!published) {
        ws.map[tile * 32 + lane] = m;
        publish(1u);
        published = true;
        t0 = globaltimer_ns();
        continue;
      }
      if (t0 == 0) t0 = globaltimer_ns();
      const int late = globaltimer_ns() - t0 > kWaitLimitNs;
      if (__shfl_sync(0xffffffffu, late, 0)) {  // one decision for the warp
        if (lane == 0) atomicOr(ws.error, DEV_TIMEOUT);
        back = -1;
        break;
      }
      __nanosleep(20);
    }
    if (back >= 0) {
      s = __ldcg(ws.state + (tile - (back + 1) * cols) * 32 + lane);
      for (int k = back; k > 0; k -= 4) {
        float4 e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (k - i > 0) e[i] = __ldcg(ws.map + (tile - (k - i) * cols) * 32 + lane);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (k - i > 0) {
            s.x = ls_apply<PACKED>(e[i].x, e[i].y, s.x);
            s.y = ls_apply<PACKED>(e[i].z, e[i].w, s.y);
          }
      }
    }
  }
  if (!last) {
    ws.state[tile * 32 + lane] = make_float2(ls_apply<PACKED>(m.x, m.y, s.x),
                                             ls_apply<PACKED>(m.z, m.w, s.y));
    publish(2u);
  }
  return s;
}

// Host side: tiles of a call and the workspace they need.
struct LsPlan {
  int64_t chunks, cols;  // step ranges, (batch entry, channel group) columns
  size_t flag, map, state, bytes;
};
inline LsPlan ls_plan(int64_t B, int64_t T, int64_t D, int64_t per /* steps of a tile */) {
  LsPlan p{};
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  p.chunks = T > 0 ? (T + per - 1) / per : 1;
  p.cols = B * ((D + kLsChannels - 1) / kLsChannels);
  const size_t tiles = (size_t)(p.chunks * p.cols);
  p.flag = 256;
  p.map = p.flag + up(tiles * 4);
  p.state = p.map + tiles * 512;
  p.bytes = p.state + tiles * 256;
  if (p.chunks == 1) p.bytes = 256;  // nothing crosses tiles
  return p;
}
inline LsWs ls_ws(void* ws, const LsPlan& p) {
  char* c = static_cast<char*>(ws);
  LsWs w;
  w.error = reinterpret_cast<uint32_t*>(c);
  w.counter = reinterpret_cast<uint32_t*>(c) + 1;
  w.flag = reinterpret_cast<uint32_t*>(c + p.flag);
  w.map = reinterpret_cast<float4*>(c + p.map);
  w.state = reinterpret_cast<float2*>(c + p.state);
  return w;
}

}  // namespace kdn
