// kdn_fp8_quantize: a matrix into e4m3 codes with one fp32 scale for each 128
// of a row (activations) or each 128 x 128 tile (weights), as it lies or
// transposed (the operands of a projection's gradients: dX = dY W needs W's
// transpose, dW = dY^T X both factors').  fp8_common.cuh has the scale.
//
// Rows as they lie: eight threads a block of 128, sixteen elements a thread (a
// thread's two divisions are a good part of its instructions: with eight
// elements a third more time), one read and one write: 32768 x 2048 takes 49 us in
// fp32 (6.9 TB/s) and 36 in bf16 (5.7 TB/s).  Rows that are not a multiple of 8 do
// not start on 16-byte boundaries and are loaded one element at a time; there
// eight elements a thread keep more loads in flight (30000 x 1001, bf16: 27 us,
// with sixteen 40 % more).
//
// Tiles and transposes: one block of 256 threads a 128 x 128 tile; a thread
// holds an 8 x 8 piece, so eight codes of a column are one 8-byte word of the
// transposed tile.  The words go through shared memory with their position in
// the row XORed by the piece's column, which keeps the column-wise stores free
// of bank conflicts, and leave as 16-byte stores.  32749 x 1000 in bf16, turned:
// 19.5 us (5.0 TB/s); neither HBM (40 % of its peak) nor the issue slots (55 %)
// are full, as a block loads, meets its barriers, converts and stores with
// nothing of another tile under way.  32768 x 2048 in tiles: 56 us fp32, 33 bf16.
#include "enqueue.h"
#include "fp8_common.cuh"

namespace kdn {
namespace {

// The codes of `n` values `step` apart, those near a middle decided in fp64: 448
// |v| and a middle times `top` are exact there.  It reads the values again, so
// that nothing but its arguments is kept for it: calls are rare, some three for a
// million quotients (decided in place, 32768 x 2048 took 10 to 30 % longer).
__device__ __noinline__ void fp8_codes_decided(const float* x, int64_t step, int n,
                                               const Fp8Block<float> b, uint8_t* codes) {
  for (int i0 = 0; i0 < n; i0 += 8) {
    uint32_t which = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i0 + i < n && fp8_near_lifted<2>(x[(i0 + i) * step] * b.inv)) which |= 1u << i;
    for (; which; which &= which - 1) {
      const int i = i0 + __ffs(which) - 1;
      const float v = x[i * step];
      float q = v * b.inv;
      q = fp8_side(q, 448.0 * (double)fabsf(v) - (double)fp8_middle(q) * (double)b.top);
      codes[i] = (uint8_t)__nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
    }
  }
}
__device__ __forceinline__ void fp8_codes_decided(const __nv_bfloat16*, int64_t, int,
                                                  const Fp8Block<__nv_bfloat16>&, uint8_t*) {}

// Codes are stored in pieces of 8 or 16 bytes, into the room that a row of Q has
// up to its next 16-byte boundary.  Behind the last row there need be no such
// room.  Its end is always the last block's, which runs a copy of the code that
// stores those codes one by one (LAST): the question asked in every block cost
// 4 %.
__device__ __forceinline__ void store_last(uint8_t* to, uint32_t lo, uint32_t hi, int n) {
  for (int i = 0; i < n; ++i) to[i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
}

template <typename XT, bool LAST>
__device__ __forceinline__ void rows_block(const XT* __restrict__ X, uint8_t* __restrict__ Q,
                                           float* __restrict__ S, int64_t rows, int C, int64_t ldq,
                                           int kb) {
  // unit: 16 elements of the row padded to whole blocks
  const int64_t unit = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (unit / 8 >= rows * kb) return;  // (whole groups of eight threads; no barrier below)
  const int64_t row = unit / (8 * kb);
  const int e = (int)(unit - row * 8 * kb) * 16;
  const XT* x = X + row * C + e;
  float v[2][8];
  load8(x, max(0, min(8, C - e)), true, v[0]);
  load8(x + 8, max(0, min(8, C - e - 8)), true, v[1]);
  const uint32_t mask = 0xffu << (threadIdx.x & 24);
  float m = max_nan(amax8(v[0]), amax8(v[1]));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(mask, m, o));
  const Fp8Block<XT> block(m);
  if (e < C) {
    uint4 c;
    float q[8];
    bool close = block.quotients(v[0], q);
    c.x = fp8_pack4(q[0], q[1], q[2], q[3]);
    c.y = fp8_pack4(q[4], q[5], q[6], q[7]);
    close |= block.quotients(v[1], q);
    c.z = fp8_pack4(q[0], q[1], q[2], q[3]);
    c.w = fp8_pack4(q[4], q[5], q[6], q[7]);
    uint8_t* to = Q + row * ldq + e;
    if (LAST && e + 16 > C && row + 1 == rows) *reinterpret_cast<uint2*>(to) = make_uint2(c.x, c.y);
    else *reinterpret_cast<uint4*>(to) = c;
    if (close) fp8_codes_decided(x, 1, min(16, C - e), block, to);
  }
  if ((threadIdx.x & 7) == 0) S[row * kb + e / 128] = fp8_scale(m);
}
// ENDS: rows end inside a piece.  (128 threads a block: with 256 fewer blocks are
// under way when one ends.)
template <typename XT, bool ENDS>
__global__ void __launch_bounds__(128, 12)
fp8_rows_kernel(const XT* __restrict__ X, uint8_t* __restrict__ Q, float* __restrict__ S,
                int64_t rows, int C, int64_t ldq, int kb) {
  if (!ENDS || blockIdx.x + 1 < gridDim.x) rows_block<XT, false>(X, Q, S, rows, C, ldq, kb);
  else rows_block<XT, true>(X, Q, S, rows, C, ldq, kb);
}

template <typename XT, bool LAST>
__device__ __forceinline__ void rows_any_block(const XT* __restrict__ X, uint8_t* __restrict__ Q,
                                               float* __restrict__ S, int64_t rows, int C,
                                               int64_t ldq, int kb) {
  // unit: 8 elements of the row padded to whole blocks
  const int64_t unit = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (unit / 16 >= rows * kb) return;  // (whole half warps; no barrier below)
  const int64_t row = unit / (16 * kb);
  const int e = (int)(unit - row * 16 * kb) * 8;
  const int n = max(0, min(8, C - e));
  float v[8];
  load8(X + row * C + e, n, false, v);
  const uint32_t mask = 0xffffu << (threadIdx.x & 16);
  float m = amax8(v);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(mask, m, o));
  const Fp8Block<XT> block(m);
  if (n > 0) {
    uint2 c;
    float q[8];
    const bool close = block.quotients(v, q);
    c.x = fp8_pack4(q[0], q[1], q[2], q[3]);
    c.y = fp8_pack4(q[4], q[5], q[6], q[7]);
    uint8_t* to = Q + row * ldq + e;
    if (LAST && n < 8 && row + 1 == rows) store_last(to, c.x, c.y, n);
    else *reinterpret_cast<uint2*>(to) = c;
    if (close) fp8_codes_decided(X + row * C + e, 1, n, block, to);
  }
  if ((threadIdx.x & 15) == 0) S[row * kb + e / 128] = fp8_scale(m);
}
template <typename XT>
__global__ void __launch_bounds__(256)
fp8_rows_any_kernel(const XT* __restrict__ X, uint8_t* __restrict__ Q, float* __restrict__ S,
                    int64_t rows, int C, int64_t ldq, int kb) {
  if (blockIdx.x + 1 < gridDim.x) rows_any_block<XT, false>(X, Q, S, rows, C, ldq, kb);
  else rows_any_block<XT, true>(X, Q, S, rows, C, ldq, kb);
}

// A thread's eight elements of a row, as they were loaded: bf16 pairs stay
// packed, which halves a thread's registers and doubles the blocks of an SM.
template <typename XT>
struct Eight {
  float v[8];
  __device__ __forceinline__ void load(const XT* p, int n, bool vec) { load8(p, n, vec, v); }
  __device__ __forceinline__ float at(int e) const { return v[e]; }
};
template <>
struct Eight<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int n, bool vec) {
    if (vec) {
      uint4 a = make_uint4(0u, 0u, 0u, 0u);
      if (n > 0) a = __ldg(reinterpret_cast<const uint4*>(p));
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    } else {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = (2 * i < n ? (uint32_t)__ldg(q + 2 * i) : 0u) |
               (2 * i + 1 < n ? (uint32_t)__ldg(q + 2 * i + 1) << 16 : 0u);
    }
  }
  __device__ __forceinline__ float at(int e) const {
    return __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
  }
};

// The largest magnitudes of pairs of bf16 numbers: as integers they are in order,
// NaN above infinity.
__device__ __forceinline__ uint32_t max_pairs(uint32_t most, uint32_t a, uint32_t b) {
  return __vimax3_u16x2(most, a & 0x7fff7fffu, b & 0x7fff7fffu);
}

// TILE: one scale a tile, else one for each 128 along the output's rows.
// (TR = false is only used with TILE.)
template <typename XT, bool TILE, bool TR>
struct TileShared {
  alignas(16) float top[TILE ? 1 : 16][128];
  alignas(16) float column[2][TILE ? 1 : 128];  // the columns' Fp8Blocks
  uint2 turned[TR ? 128 : 1][16];
};
template <typename XT, bool TILE, bool TR, bool LAST>
__device__ __forceinline__ void tile_block(TileShared<XT, TILE, TR>& sh, const XT* __restrict__ X,
                                           uint8_t* __restrict__ Q, float* __restrict__ S,
                                           int64_t R, int64_t C, int64_t ldq, int64_t rblocks,
                                           int64_t cblocks, int vec) {
  auto& top = sh.top;
  const int rr = threadIdx.x >> 4, cv = threadIdx.x & 15;
  const int64_t rb = blockIdx.x / cblocks, cb = blockIdx.x - rb * cblocks;
  const int64_t r0 = rb * 128 + rr * 8, c0 = cb * 128 + cv * 8;
  const int nc = (int)max((int64_t)0, min((int64_t)8, C - c0));
  Eight<XT> v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool in = r0 + i < R;
    v[i].load(X + (in ? (r0 + i) * C + c0 : 0), in ? nc : 0, vec);
  }
  Fp8Block<XT> all;
  if constexpr (TILE) {
    float m = 0.f;
    if constexpr (sizeof(XT) == 2 && !TR) {
      uint32_t both = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; e += 2) both = max_pairs(both, v[i].w[e], v[i].w[e + 1]);
      m = max_nan(__uint_as_float(both << 16), __uint_as_float(both & 0xffff0000u));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(v[i].at(e)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) top[0][threadIdx.x >> 5] = m;
    __syncthreads();
    m = top[0][0];
#pragma unroll
    for (int w = 1; w < 8; ++w) m = max_nan(m, top[0][w]);
    if (threadIdx.x == 0) S[TR ? cb * rblocks + rb : rb * cblocks + cb] = fp8_scale(m);
    all = Fp8Block<XT>(m);
  } else {
    // the largest of each column over the tile's 128 rows
    float most[8];
    if constexpr (sizeof(XT) == 2) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t both = 0u;
#pragma unroll
        for (int i = 0; i < 8; i += 2) both = max_pairs(both, v[i].w[e], v[i + 1].w[e]);
        most[2 * e] = __uint_as_float(both << 16);
        most[2 * e + 1] = __uint_as_float(both & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        most[e] = fabsf(v[0].at(e));
#pragma unroll
        for (int i = 1; i < 8; ++i) most[e] = max_nan(most[e], fabsf(v[i].at(e)));
      }
    }
    reinterpret_cast<float4*>(&top[rr][cv * 8])[0] = make_float4(most[0], most[1], most[2], most[3]);
    reinterpret_cast<float4*>(&top[rr][cv * 8])[1] = make_float4(most[4], most[5], most[6], most[7]);
    __syncthreads();
    if (threadIdx.x < 128) {
      float m = top[0][threadIdx.x];
#pragma unroll
      for (int k = 1; k < 16; ++k) m = max_nan(m, top[k][threadIdx.x]);
      const int64_t c = cb * 128 + threadIdx.x;
      if (c < C) S[c * rblocks + rb] = fp8_scale(m);
      const Fp8Block<XT> b(m);
      sh.column[0][threadIdx.x] = b.first();
      sh.column[1][threadIdx.x] = b.second();
    }
    __syncthreads();
  }
  if constexpr (!TR) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (r0 + i < R && nc > 0) {
        uint2 c;
        float x[8], q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = v[i].at(e);
        const bool close = all.quotients(x, q);
        c.x = fp8_pack4(q[0], q[1], q[2], q[3]);
        c.y = fp8_pack4(q[4], q[5], q[6], q[7]);
        uint8_t* to = Q + (r0 + i) * ldq + c0;
        if (LAST && nc < 8 && r0 + i + 1 == R) store_last(to, c.x, c.y, nc);
        else *reinterpret_cast<uint2*>(to) = c;
        if (close) fp8_codes_decided(X + (r0 + i) * C + c0, 1, nc, all, to);
      }
    }
  } else {
    auto& turned = sh.turned;
    auto column = [&](int e) {
      return Fp8Block<XT>(sh.column[0][cv * 8 + e], sh.column[1][cv * 8 + e]);
    };
    // (fp32: all eight at once, in four loads; bf16 has no registers for them)
    float b0[8], b1[8];
    if constexpr (!TILE && sizeof(XT) == 4) {
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        *reinterpret_cast<float4*>(b0 + e) =
            *reinterpret_cast<const float4*>(&sh.column[0][cv * 8 + e]);
        *reinterpret_cast<float4*>(b1 + e) =
            *reinterpret_cast<const float4*>(&sh.column[1][cv * 8 + e]);
      }
    }
    uint32_t close = 0;  // columns of this thread with codes to decide
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint2 c;
      float x[8], q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = v[i].at(e);
      const Fp8Block<XT> b =
          TILE ? all : sizeof(XT) == 4 ? Fp8Block<XT>(b0[e], b1[e]) : column(e);
      if (b.quotients(x, q)) close |= 1u << e;
      c.x = fp8_pack4(q[0], q[1], q[2], q[3]);
      c.y = fp8_pack4(q[4], q[5], q[6], q[7]);
      turned[cv * 8 + e][rr ^ cv] = c;
    }
    for (; close; close &= close - 1) {
      const int e = __ffs(close) - 1;
      if (c0 + e < C && r0 < R)
        fp8_codes_decided(X + r0 * C + c0 + e, C, (int)min((int64_t)8, R - r0),
                          TILE ? all : column(e),
                          reinterpret_cast<uint8_t*>(&turned[cv * 8 + e][rr ^ cv]));
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int unit = k * 256 + threadIdx.x;
      const int c = unit >> 3, part = (unit & 7) * 2, x = c >> 3;
      const int64_t oc = cb * 128 + c, orow = rb * 128 + part * 8;
      if (oc < C && orow < R) {
        const uint2 a = turned[c][part ^ x], b = turned[c][(part + 1) ^ x];
        uint8_t* to = Q + oc * ldq + orow;
        if (LAST && oc + 1 == C && orow + 16 > R) {
          const int n = (int)(R - orow);
          store_last(to, a.x, a.y, min(8, n));
          store_last(to + 8, b.x, b.y, n - 8);
        } else {
          *reinterpret_cast<uint4*>(to) = make_uint4(a.x, a.y, b.x, b.y);
        }
      }
    }
  }
}
// Blocks of an SM, bf16: four, or three for turned tiles (32749 x 1000: rows
// turned 21.3 us with three and 19.8 with four, tiles 20.9 and 22.6); fp32: three
// where the tile is turned (34.2 with two and 31.0), else two (31.4 and 33.5 with
// three).
template <typename XT, bool TILE, bool TR>
__global__ void __launch_bounds__(256, sizeof(XT) == 2 ? (TILE && TR ? 3 : 4) : TR ? 3 : 2)
fp8_tile_kernel(const XT* __restrict__ X, uint8_t* __restrict__ Q, float* __restrict__ S,
                int64_t R, int64_t C, int64_t ldq, int64_t rblocks, int64_t cblocks, int vec) {
  __shared__ TileShared<XT, TILE, TR> sh;
  if (blockIdx.x + 1 < gridDim.x)
    tile_block<XT, TILE, TR, false>(sh, X, Q, S, R, C, ldq, rblocks, cblocks, vec);
  else
    tile_block<XT, TILE, TR, true>(sh, X, Q, S, R, C, ldq, rblocks, cblocks, vec);
}

template <typename XT>
kdn_status quantize_types(const void* x, void* q, float* scale, int64_t R, int64_t C, int64_t ldq,
                          bool tile, bool tr, cudaStream_t s) {
  const XT* X = static_cast<const XT*>(x);
  uint8_t* Q = static_cast<uint8_t*>(q);
  const int64_t rb = (R + 127) / 128, cb = (C + 127) / 128;
  const int vec = C % 8 == 0;
  if (!tile && !tr && vec)
    return launch(C % 16 == 0 ? fp8_rows_kernel<XT, false> : fp8_rows_kernel<XT, true>,
                  (R * cb * 8 + 127) / 128, 128, 0, s, X, Q, scale, R, (int)C, ldq, (int)cb);
  if (!tile && !tr)
    return launch(fp8_rows_any_kernel<XT>, (R * cb * 16 + 255) / 256, 256, 0, s, X, Q, scale, R,
                  (int)C, ldq, (int)cb);
  return launch(!tile ? fp8_tile_kernel<XT, false, true>
                      : tr ? fp8_tile_kernel<XT, true, true> : fp8_tile_kernel<XT, true, false>,
                rb * cb, 256, 0, s, X, Q, scale, R, C, ldq, rb, cb, vec);
}

}  // namespace

kdn_status fp8_quantize_launch(const void* x, kdn_dtype xt, void* q, int64_t ldq, float* scale,
                               int64_t rows, int64_t cols, bool tile, bool transpose,
                               cudaStream_t s) {
  return xt == KDN_F32 ? quantize_types<float>(x, q, scale, rows, cols, ldq, tile, transpose, s)
                       : quantize_types<__nv_bfloat16>(x, q, scale, rows, cols, ldq, tile,
                                                       transpose, s);
}

}  // namespace kdn
