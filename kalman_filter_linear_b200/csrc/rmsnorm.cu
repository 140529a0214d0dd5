// kdn_rmsnorm_forward / kdn_rmsnorm_backward: the residual addition and root-
// mean-square norm around a mixing layer.
//   h = x + residual (rounded to the residual's type),
//   y = h * rs * w,  rs = 1 / sqrt(mean(h^2) + eps),
// y in bf16, fp32 or e4m3 with one scale for each 128 of a row (fp8_common.cuh).
// Backward, with dy = dL/dy (for e4m3 the gradient of the value code * scale
// stands for) and dh what reaches h from elsewhere:
//   d = dh + rs (dy w - h rs^2 mean(dy w h)),  dx = dresidual = d,
//   dw = sum over rows of dy h rs.
//
// One read of every input and one write of every output: a row stays in
// registers between its reduction and its use, and the next row's loads are
// under way meanwhile.  Rows are taken in turn by as many blocks as stay on the
// device at once, eight elements a thread up to rows of 4096: 32768 rows of
// 2048, fp32 with a bf16 stream to e4m3, take 94 us (6.4 TB/s), backward 131
// (6.2 TB/s); a warp a row with 64 elements a lane, loaded as its turn came,
// took 268 and 309.  A row has G threads.
// VEC (rows of a multiple of 8): thread t holds the elements [8 (t + G v),
// 8 (t + G v) + 8), so loads are 16 bytes a thread and a block of 128 is a half
// warp's.  Otherwise rows do not start on 16-byte boundaries: a warp holds 256
// elements, lane l those at l, l + 32, ..., so that loads of single elements are
// consecutive, and a block of 128 is a warp's.
#include <atomic>

#include "enqueue.h"
#include "fp8_common.cuh"

namespace kdn {
namespace {

enum class Out { F32, BF16, E4M3 };

// A thread's eight elements of a row, as they were loaded.
template <typename T, bool VEC>
struct Held {
  float v[8];
  template <int G>
  __device__ __forceinline__ void load(const T* row, int t, int vth, int D) {
    if constexpr (VEC) {
      const int e = 8 * (t + G * vth);
      load8(row + e, D - e, true, v);
    } else {
      const int e = 256 * ((t >> 5) + G / 32 * vth) + (t & 31);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = e + 32 * i < D ? to_f32<T>(row[e + 32 * i]) : 0.f;
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v[i];
  }
};
template <>
struct Held<__nv_bfloat16, true> {
  uint4 w;
  template <int G>
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int t, int vth, int D) {
    const int e = 8 * (t + G * vth);
    w = e < D ? __ldg(reinterpret_cast<const uint4*>(row + e)) : make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const { unpack_bf16x8(w, x); }
};
__device__ __forceinline__ void put1(float* p, float v) { *p = v; }
__device__ __forceinline__ void put1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
template <int G, bool VEC, typename T>
__device__ __forceinline__ void put(T* row, int t, int vth, int D, const float (&x)[8]) {
  if constexpr (VEC) {
    const int e = 8 * (t + G * vth);
    store8(row + e, D - e, true, x);
  } else {
    const int e = 256 * ((t >> 5) + G / 32 * vth) + (t & 31);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e + 32 * i < D) put1(row + e + 32 * i, x[i]);
  }
}

// Threads of a block, rows of a block at once, and the blocks of an SM that
// registers allow, forward and backward.
template <int G, int NV, bool VEC>
struct Shape {
  enum : int {
    THREADS = G < 256 ? 256 : G,
    ROWS = THREADS / G,
    BLOCKS = (NV > 2 || (NV == 2 && VEC) ? 512 : 1024) / THREADS,
    BWD_BLOCKS = (G == 1024 ? 1024 : NV > 1 ? 512 : 768) / THREADS
  };
};

// Sums over a row's G threads, in all of them.  Two buffers in turn: a slow
// warp may still read the last row's sums.
template <int G, int N>
__device__ __forceinline__ void row_sums(float (&x)[N], float (*sh)[N], int turn, int warps) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = warp_sum(x[i]);
  if constexpr (G > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) sh[turn * warps + warp][i] = x[i];
    __syncthreads();
    const int w0 = turn * warps + (warp & ~(G / 32 - 1));
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = 0.f;
#pragma unroll
    for (int w = 0; w < G / 32; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] += sh[w0 + w][i];
  }
}

// The quotients of a block's codes from y = h rs w and its largest magnitude
// `top` (the block: N elements of each of LANES threads).  The factor rs is the
// same in all of them, so a quotient is 448 h w / max |h w|; where the six
// roundings of q (two each of y and top, one of the inverse and one of the
// product: less than six units in the last place) could decide a code, the warp
// decides it so, in fp64.  (One row of 2048 in forty has such a place.)
template <int N, int LANES>
__device__ __noinline__ void norm_decide(const float* h, const float* w, float* q) {
  double most = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) most = fmax(most, fabs((double)h[i] * (double)w[i]));
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) most = fmax(most, __shfl_xor_sync(0xffffffffu, most, o));
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (fp8_near_lifted<6>(q[i]))
      q[i] = fp8_side(q[i], 448.0 * fabs((double)h[i] * (double)w[i]) - (double)fp8_middle(q[i]) * most);
}
template <int N, int LANES>
__device__ __forceinline__ void norm_quotients(const float (&y)[N], const float (&h)[N],
                                               const float (&w)[N], float top, float (&q)[N]) {
  const float inv = fp8_inverse(top);
#pragma unroll
  for (int i = 0; i < N; ++i) q[i] = y[i] * inv;
  if (!__any_sync(0xffffffffu, fp8_any_near<6>(q))) return;
  float a[N], b[N], c[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    a[i] = h[i];
    b[i] = w[i];
    c[i] = q[i];
  }
  norm_decide<N, LANES>(a, b, c);
  // (a block below the floor, or one that is not finite, keeps what it has)
  if (top > kAmaxFloor && top <= 3.0e38f) {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = c[i];
  }
}

template <typename XT, typename RT, bool RES, Out OUT, int G, int NV, bool VEC>
__global__ void __launch_bounds__(Shape<G, NV, VEC>::THREADS, Shape<G, NV, VEC>::BLOCKS)
rmsnorm_forward_kernel(const XT* __restrict__ X, const RT* Res, const float* __restrict__ W,
                       RT* Hout, void* __restrict__ Yv, float* __restrict__ Scale, int64_t rows,
                       int D, int64_t ldy, float eps) {
  using S = Shape<G, NV, VEC>;
  constexpr int WARPS = S::THREADS / 32;
  __shared__ float sh[2 * WARPS][1];
  const int t = threadIdx.x % G;
  const int64_t step = (int64_t)gridDim.x * S::ROWS;
  int64_t row = (int64_t)blockIdx.x * S::ROWS + threadIdx.x / G;
  Held<XT, VEC> x[NV];
  Held<RT, VEC> r[NV];
  auto fetch = [&](int64_t from) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      x[v].template load<G>(X + from * D, t, v, D);
      if (RES) r[v].template load<G>(Res + from * D, t, v, D);
    }
  };
  constexpr bool AHEAD = VEC;
  if (AHEAD && row < rows) fetch(row);
  float w[NV][8];
  if (NV < 4) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      Held<float, VEC> h;
      h.template load<G>(W, t, v, D);
      h.get(w[v]);
    }
  }
  int turn = 0;
  // (all threads of a block go round together: a row's sums meet at a barrier)
  for (int64_t first = (int64_t)blockIdx.x * S::ROWS; first < rows;
       first += step, row += step, turn ^= 1) {
    const bool have = row < rows;
    if (!AHEAD && have) fetch(row);
    float h[NV][8], ss[1] = {0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      x[v].get(h[v]);
      if (RES) {
        float q[8];
        r[v].get(q);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h[v][i] += q[i];
          if (sizeof(RT) == 2) h[v][i] = __bfloat162float(__float2bfloat16_rn(h[v][i]));
        }
        if (have) put<G, VEC>(Hout + row * D, t, v, D, h[v]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss[0] = fmaf(h[v][i], h[v][i], ss[0]);
    }
    if (AHEAD && row + step < rows) fetch(row + step);
    row_sums<G>(ss, sh, turn, WARPS);
    const float rs = rsqrtf(ss[0] / (float)D + eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (NV >= 4) {
        Held<float, VEC> hw;
        hw.template load<G>(W, t, v, D);
        hw.get(w[v]);
      }
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = h[v][i] * rs * w[v][i];
      if (OUT == Out::F32) {
        if (have) put<G, VEC>(static_cast<float*>(Yv) + row * D, t, v, D, y);
      } else if (OUT == Out::BF16) {
        if (have) put<G, VEC>(static_cast<__nv_bfloat16*>(Yv) + row * D, t, v, D, y);
      } else if constexpr (VEC) {
        // elements behind the row's end are zeros here: they do not raise the
        // maximum
        const int e = 8 * (t + G * v);
        const float top = half_warp_max(amax8(y));
        float q[8];
        norm_quotients<8, 16>(y, h[v], w[v], top, q);
        if (have && e < D) {
          uint2 c;
          c.x = fp8_pack4(q[0], q[1], q[2], q[3]);
          c.y = fp8_pack4(q[4], q[5], q[6], q[7]);
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(Yv) + row * ldy + e) = c;
          if ((t & 15) == 0) Scale[row * ((D + 127) / 128) + e / 128] = fp8_scale(top);
        }
      } else {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int e = 256 * ((t >> 5) + G / 32 * v) + 128 * half + (t & 31);
          float z[4], hz[4], wz[4], q[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            z[i] = y[4 * half + i];
            hz[i] = h[v][4 * half + i];
            wz[i] = w[v][4 * half + i];
          }
          float top = fabsf(z[0]);
#pragma unroll
          for (int i = 1; i < 4; ++i) top = max_nan(top, fabsf(z[i]));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1)
            top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
          norm_quotients<4, 32>(z, hz, wz, top, q);
          const uint32_t c = fp8_pack4(q[0], q[1], q[2], q[3]);
          uint8_t* to = static_cast<uint8_t*>(Yv) + row * ldy + e;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (have && e + 32 * i < D) to[32 * i] = (uint8_t)(c >> (8 * i));
          if (have && (t & 31) == 0 && e < D)
            Scale[row * ((D + 127) / 128) + e / 128] = fp8_scale(top);
        }
      }
    }
  }
}

constexpr int kNormBwdBlocks = 592;  // most that write a part of dw

// A thread holds its elements as they were loaded, through the reduction, and
// with VEC, up to rows of 8192, the next row's too.
template <typename HT, typename YT, typename XT, int G, int NV, bool VEC>
__global__ void __launch_bounds__(Shape<G, NV, VEC>::THREADS, Shape<G, NV, VEC>::BWD_BLOCKS)
rmsnorm_backward_kernel(const HT* __restrict__ Hin, const float* __restrict__ W,
                        const YT* __restrict__ dY, const HT* dH, XT* __restrict__ dX, HT* dRes,
                        float* __restrict__ part, int64_t rows, int D, float eps) {
  using S = Shape<G, NV, VEC>;
  constexpr int WARPS = S::THREADS / 32;
  constexpr bool AHEAD = G < 1024 && VEC, KEEP = G < 1024;  // KEEP: the weights
  __shared__ float sh[2 * WARPS][2];
  extern __shared__ float acc_sh[];  // several rows a block: [row][D] sums
  const int t = threadIdx.x % G;
  const int64_t step = (int64_t)gridDim.x * S::ROWS;
  int64_t row = (int64_t)blockIdx.x * S::ROWS + threadIdx.x / G;
  struct Row {
    Held<HT, VEC> h, d;
    Held<YT, VEC> g;
  };
  Row now[NV], ahead[AHEAD ? NV : 1];
  float acc[NV][8], w[KEEP ? NV : 1][8];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[v][i] = 0.f;
  auto weights = [&](int v, float (&x)[8]) {
    Held<float, VEC> h;
    h.template load<G>(W, t, v, D);
    h.get(x);
  };
  auto fetch = [&](Row& r, int64_t from, int v) {
    r.h.template load<G>(Hin + from * D, t, v, D);
    r.g.template load<G>(dY + from * D, t, v, D);
    if (dH) r.d.template load<G>(dH + from * D, t, v, D);
  };
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (KEEP) weights(v, w[KEEP ? v : 0]);
    if (AHEAD && row < rows) fetch(ahead[AHEAD ? v : 0], row, v);
  }
  int turn = 0;
  for (int64_t first = (int64_t)blockIdx.x * S::ROWS; first < rows;
       first += step, row += step, turn ^= 1) {
    const bool have = row < rows;
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (AHEAD) {
        now[v] = ahead[AHEAD ? v : 0];
        if (row + step < rows) fetch(ahead[AHEAD ? v : 0], row + step, v);
      } else if (have) {
        fetch(now[v], row, v);
      }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float h[8], g[8];
      now[v].h.get(h);
      now[v].g.get(g);
      if (!KEEP) weights(v, w[0]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum[0] = fmaf(h[i], h[i], sum[0]);
        sum[1] = fmaf(g[i] * w[KEEP ? v : 0][i], h[i], sum[1]);
      }
    }
    row_sums<G>(sum, sh, turn, WARPS);
    const float rs = rsqrtf(sum[0] / (float)D + eps);
    const float k = rs * rs * (sum[1] / (float)D);
    if (have) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (!KEEP) weights(v, w[0]);
        float h[8], g[8], d[8];
        now[v].h.get(h);
        now[v].g.get(g);
        if (dH) {
          now[v].d.get(d);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          acc[v][i] = fmaf(g[i], h[i] * rs, acc[v][i]);
          d[i] += rs * (g[i] * w[KEEP ? v : 0][i] - h[i] * k);
        }
        put<G, VEC>(dX + row * D, t, v, D, d);
        if (dRes) put<G, VEC>(dRes + row * D, t, v, D, d);
      }
    }
  }
  // this block's part of dw
  float* out = part + (int64_t)blockIdx.x * D;
  if constexpr (S::ROWS == 1) {
#pragma unroll
    for (int v = 0; v < NV; ++v) put<G, VEC>(out, t, v, D, acc[v]);
  } else {
    float* mine = acc_sh + threadIdx.x / G * D;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = VEC ? 8 * (t + G * v) + i : 256 * ((t >> 5) + G / 32 * v) + (t & 31) + 32 * i;
        if (e < D) mine[e] = acc[v][i];
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < D; e += S::THREADS) {
      float s = 0.f;
#pragma unroll
      for (int r = 0; r < S::ROWS; ++r) s += acc_sh[r * D + e];
      out[e] = s;
    }
  }
}

// dw = the sum of the blocks' parts, in a fixed order: 32 columns a block, 32
// threads a column, each with every 32nd part
__global__ void __launch_bounds__(1024)
rmsnorm_dweight_kernel(const float* __restrict__ part, float* __restrict__ dw, int parts, int D) {
  __shared__ float sh[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < D) {
    for (int p = r; p < parts; p += 128) {
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = p + 32 * i < parts ? __ldg(part + (int64_t)(p + 32 * i) * D + c) : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += x[i];
    }
  }
  sh[r][threadIdx.x & 31] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  // warp r adds column r's 32 sums
  const float total = warp_sum(sh[threadIdx.x & 31][r]);
  if ((threadIdx.x & 31) == 0 && blockIdx.x * 32 + r < D) dw[blockIdx.x * 32 + r] = total;
}

struct FwdArgs {
  const void *x, *res;
  const float* w;
  void *h, *y;
  float* scale;
  int64_t rows;
  int D;
  int64_t ldy;
  float eps;
};

// blocks that the current device holds at once (0: an error)
inline int64_t resident(int per_sm) {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  int sms = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (!sms) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  }
  return (int64_t)sms * per_sm;
}

template <typename XT, typename RT, bool RES, Out OUT, int G, int NV, bool VEC>
kdn_status fwd_go(const FwdArgs& a, cudaStream_t s) {
  using S = Shape<G, NV, VEC>;
  const int64_t want = (a.rows + S::ROWS - 1) / S::ROWS, most = resident(S::BLOCKS);
  if (most == 0) return KDN_ERR_CUDA;
  return launch(rmsnorm_forward_kernel<XT, RT, RES, OUT, G, NV, VEC>, want < most ? want : most,
                S::THREADS, 0, s, static_cast<const XT*>(a.x), static_cast<const RT*>(a.res), a.w,
                static_cast<RT*>(a.h), a.y, a.scale, a.rows, a.D, a.ldy, a.eps);
}
template <typename XT, typename RT, bool RES, Out OUT, bool VEC>
kdn_status fwd_size(const FwdArgs& a, cudaStream_t s) {
  if (a.D <= 256) return fwd_go<XT, RT, RES, OUT, 32, 1, VEC>(a, s);
  if (a.D <= 512) return fwd_go<XT, RT, RES, OUT, 64, 1, VEC>(a, s);
  if (a.D <= 1024) return fwd_go<XT, RT, RES, OUT, 128, 1, VEC>(a, s);
  if (a.D <= 2048) return fwd_go<XT, RT, RES, OUT, 256, 1, VEC>(a, s);
  if (a.D <= 4096) return fwd_go<XT, RT, RES, OUT, 512, 1, VEC>(a, s);
  if (a.D <= 8192) return fwd_go<XT, RT, RES, OUT, 512, 2, VEC>(a, s);
  return fwd_go<XT, RT, RES, OUT, 512, 4, VEC>(a, s);
}
template <typename XT, typename RT, bool RES, bool VEC>
kdn_status fwd_out(const FwdArgs& a, kdn_dtype out, cudaStream_t s) {
  if (out == KDN_F32) return fwd_size<XT, RT, RES, Out::F32, VEC>(a, s);
  if (out == KDN_BF16) return fwd_size<XT, RT, RES, Out::BF16, VEC>(a, s);
  return fwd_size<XT, RT, RES, Out::E4M3, VEC>(a, s);
}
template <typename XT, typename RT, bool RES>
kdn_status fwd_vec(const FwdArgs& a, kdn_dtype out, cudaStream_t s) {
  return a.D % 8 == 0 ? fwd_out<XT, RT, RES, true>(a, out, s)
                      : fwd_out<XT, RT, RES, false>(a, out, s);
}
struct BwdArgs {
  const void* h;
  const float* w;
  const void *dy, *dh;
  void *dx, *dres;
  float *dw, *part;
  int64_t rows;
  int D;
  float eps;
};

template <typename HT, typename YT, typename XT, int G, int NV, bool VEC>
kdn_status bwd_go(const BwdArgs& a, cudaStream_t s) {
  using S = Shape<G, NV, VEC>;
  const int64_t want = (a.rows + S::ROWS - 1) / S::ROWS;
  int64_t most = resident(S::BWD_BLOCKS);
  if (most == 0) return KDN_ERR_CUDA;
  if (most > kNormBwdBlocks) most = kNormBwdBlocks;
  const int blocks = (int)(want < most ? want : most);
  const size_t smem = S::ROWS > 1 ? (size_t)S::ROWS * a.D * 4 : 0;
  if (blocks > 0) {
    const kdn_status st = launch(
        rmsnorm_backward_kernel<HT, YT, XT, G, NV, VEC>, blocks, S::THREADS, smem, s,
        static_cast<const HT*>(a.h), a.w, static_cast<const YT*>(a.dy),
        static_cast<const HT*>(a.dh), static_cast<XT*>(a.dx), static_cast<HT*>(a.dres), a.part,
        a.rows, a.D, a.eps);
    if (st != KDN_OK) return st;
  }
  return launch(rmsnorm_dweight_kernel, (a.D + 31) / 32, 1024, 0, s, a.part, a.dw, blocks, a.D);
}
template <typename HT, typename YT, typename XT, bool VEC>
kdn_status bwd_size(const BwdArgs& a, cudaStream_t s) {
  if (a.D <= 256) return bwd_go<HT, YT, XT, 32, 1, VEC>(a, s);
  if (a.D <= 512) return bwd_go<HT, YT, XT, 64, 1, VEC>(a, s);
  if (a.D <= 1024) return bwd_go<HT, YT, XT, 128, 1, VEC>(a, s);
  if (a.D <= 2048) return bwd_go<HT, YT, XT, 256, 1, VEC>(a, s);
  if (a.D <= 4096) return bwd_go<HT, YT, XT, 256, 2, VEC>(a, s);
  if (a.D <= 8192) return bwd_go<HT, YT, XT, 512, 2, VEC>(a, s);
  return bwd_go<HT, YT, XT, 1024, 2, VEC>(a, s);
}
template <typename HT, typename YT, typename XT>
kdn_status bwd_vec(const BwdArgs& a, cudaStream_t s) {
  return a.D % 8 == 0 ? bwd_size<HT, YT, XT, true>(a, s) : bwd_size<HT, YT, XT, false>(a, s);
}
template <typename HT, typename YT>
kdn_status bwd_x(const BwdArgs& a, kdn_dtype x, cudaStream_t s) {
  return x == KDN_F32 ? bwd_vec<HT, YT, float>(a, s) : bwd_vec<HT, YT, __nv_bfloat16>(a, s);
}

}  // namespace

size_t rmsnorm_backward_workspace_size(int64_t rows, int D) {
  const int64_t blocks = rows < kNormBwdBlocks ? rows : kNormBwdBlocks;
  return ((size_t)blocks * D * 4 + 255) / 256 * 256;
}

kdn_status rmsnorm_forward_launch(const void* x, kdn_dtype xt, const void* res, kdn_dtype rt,
                                  const float* w, void* h, void* y, kdn_dtype yt, int64_t ldy,
                                  float* scale, int64_t rows, int D, float eps, cudaStream_t s) {
  const FwdArgs a{x, res, w, h, y, scale, rows, D, ldy, eps};
  using bf = __nv_bfloat16;
  if (!res)  // (its type is not used)
    return xt == KDN_F32 ? fwd_vec<float, float, false>(a, yt, s)
                         : fwd_vec<bf, float, false>(a, yt, s);
  if (xt == KDN_F32)
    return rt == KDN_F32 ? fwd_vec<float, float, true>(a, yt, s)
                         : fwd_vec<float, bf, true>(a, yt, s);
  return rt == KDN_F32 ? fwd_vec<bf, float, true>(a, yt, s) : fwd_vec<bf, bf, true>(a, yt, s);
}

kdn_status rmsnorm_backward_launch(const void* h, kdn_dtype ht, const float* w, const void* dy,
                                   kdn_dtype yt, const void* dh, void* dx, kdn_dtype xt,
                                   void* dres, float* dw, int64_t rows, int D, float eps,
                                   void* workspace, cudaStream_t s) {
  const BwdArgs a{h, w, dy, dh, dx, dres, dw, static_cast<float*>(workspace), rows, D, eps};
  using bf = __nv_bfloat16;
  if (ht == KDN_F32)
    return yt == KDN_F32 ? bwd_x<float, float>(a, xt, s) : bwd_x<float, bf>(a, xt, s);
  return yt == KDN_F32 ? bwd_x<bf, float>(a, xt, s) : bwd_x<bf, bf>(a, xt, s);
}

}  // namespace kdn
