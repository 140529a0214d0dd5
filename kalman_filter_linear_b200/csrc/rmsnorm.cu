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
// registers between its reduction and its use.  Thread t of a row's G threads
// holds elements [8 (t + G v), 8 (t + G v) + 8), so loads are 16 bytes a
// thread and a block of 128 is a half warp's.
#include "fp8_common.cuh"

namespace kdn {
namespace {

enum class Out { F32, BF16, E4M3 };

// Sums of `x` over a row's G threads, in all of them (G = 32: a warp).
template <int G>
__device__ __forceinline__ float row_sum(float x, float* sh) {
  x = warp_sum(x);
  if constexpr (G > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) sh[warp] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int w = 0; w < G / 32; ++w) x += sh[w];
  }
  return x;
}

template <typename XT, typename RT, Out OUT, int G, int NV>
__global__ void __launch_bounds__(256)
rmsnorm_forward_kernel(const XT* __restrict__ X, const RT* __restrict__ Res,
                       const float* __restrict__ W, RT* __restrict__ Hout,
                       void* __restrict__ Yv, float* __restrict__ Scale, int64_t rows, int D,
                       int64_t ldy, float eps, int vec) {
  __shared__ float sh[8];
  const int t = threadIdx.x % G;
  const int64_t row = G == 32 ? (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32
                              : (int64_t)blockIdx.x;
  if (row >= rows) return;  // (whole warps or the whole block)
  float h[NV][8];
  const XT* x = X + row * D;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = 8 * (t + G * v);
    load8(x + e, min(8, D - e), vec, h[v]);
  }
  if (Res) {
    const RT* r = Res + row * D;
    float q[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = 8 * (t + G * v);
      load8(r + e, min(8, D - e), vec, q[v]);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = 8 * (t + G * v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[v][i] += q[v][i];
        if (sizeof(RT) == 2) h[v][i] = __bfloat162float(__float2bfloat16_rn(h[v][i]));
      }
      if (Hout) store8(Hout + row * D + e, min(8, D - e), vec, h[v]);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(h[v][i], h[v][i], ss);
  ss = row_sum<G>(ss, sh);
  const float rs = rsqrtf(ss / (float)D + eps);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = 8 * (t + G * v);
    const int n = min(8, D - e);
    float w[8];
    load8(W + e, n, vec, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[v][i] = h[v][i] * rs * w[i];
    if (OUT == Out::F32) {
      store8(static_cast<float*>(Yv) + row * D + e, n, vec, h[v]);
    } else if (OUT == Out::BF16) {
      store8(static_cast<__nv_bfloat16*>(Yv) + row * D + e, n, vec, h[v]);
    } else {
      // elements behind the row's end are zeros here: they do not raise the
      // maximum, and their codes fall into the row's padding
      const float top = half_warp_max(amax8(h[v]));
      const float inv = fp8_inverse(top);
      if (n > 0) {
        uint2 c;
        c.x = fp8_pack4(h[v][0], h[v][1], h[v][2], h[v][3], inv);
        c.y = fp8_pack4(h[v][4], h[v][5], h[v][6], h[v][7], inv);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(Yv) + row * ldy + e) = c;
        if ((t & 15) == 0) Scale[row * ((D + 127) / 128) + e / 128] = fp8_scale(top);
      }
    }
  }
}

constexpr int kNormBwdBlocks = 592;  // 4 a SM: rows are taken in turn

template <typename HT, typename YT, typename XT, int G, int NV>
__global__ void __launch_bounds__(256)
rmsnorm_backward_kernel(const HT* __restrict__ Hin, const float* __restrict__ W,
                        const YT* __restrict__ dY, const HT* __restrict__ dH,
                        XT* __restrict__ dX, HT* __restrict__ dRes, float* __restrict__ part,
                        int64_t rows, int D, float eps, int vec) {
  __shared__ float sh[2][16];
  extern __shared__ float acc_sh[];  // G = 32: one row of sums a warp
  const int t = threadIdx.x % G, warp = threadIdx.x >> 5;
  constexpr int kRowsPerBlock = 256 / G;
  float acc[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[v][i] = 0.f;
  const int64_t step = (int64_t)gridDim.x * kRowsPerBlock;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * kRowsPerBlock + (G == 32 ? warp : 0); row < rows;
       row += step, turn ^= 1) {
    float h[NV][8], g[NV][8];
    float ss = 0.f, sg = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = 8 * (t + G * v);
      load8(Hin + row * D + e, min(8, D - e), vec, h[v]);
      load8(dY + row * D + e, min(8, D - e), vec, g[v]);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = 8 * (t + G * v);
      float w[8];
      load8(W + e, min(8, D - e), vec, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(h[v][i], h[v][i], ss);
        sg = fmaf(g[v][i] * w[i], h[v][i], sg);
      }
    }
    ss = warp_sum(ss);
    sg = warp_sum(sg);
    if constexpr (G > 32) {
      // two buffers in turn: a slow warp may still read the last row's sums
      if ((threadIdx.x & 31) == 0) {
        sh[turn][2 * warp] = ss;
        sh[turn][2 * warp + 1] = sg;
      }
      __syncthreads();
      ss = sg = 0.f;
#pragma unroll
      for (int w = 0; w < G / 32; ++w) {
        ss += sh[turn][2 * w];
        sg += sh[turn][2 * w + 1];
      }
    }
    const float rs = rsqrtf(ss / (float)D + eps);
    const float k = rs * rs * (sg / (float)D);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = 8 * (t + G * v);
      const int n = min(8, D - e);
      float w[8], d[8];
      load8(W + e, n, vec, w);
      if (dH) {
        load8(dH + row * D + e, n, vec, d);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[v][i] = fmaf(g[v][i], h[v][i] * rs, acc[v][i]);
        d[i] += rs * (g[v][i] * w[i] - h[v][i] * k);
      }
      store8(dX + row * D + e, n, vec, d);
      if (dRes) store8(dRes + row * D + e, n, vec, d);
    }
  }
  // this block's part of dw
  float* out = part + (int64_t)blockIdx.x * D;
  if constexpr (G > 32) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = 8 * (t + G * v);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i < D) out[e + i] = acc[v][i];
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = 8 * (t + G * v);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i < D) acc_sh[warp * D + e + i] = acc[v][i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < D; e += 256) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) s += acc_sh[w * D + e];
      out[e] = s;
    }
  }
}

// dw = the sum of the blocks' parts, in a fixed order: 32 columns a block, 8
// threads a column
__global__ void __launch_bounds__(256)
rmsnorm_dweight_kernel(const float* __restrict__ part, float* __restrict__ dw, int parts, int D) {
  __shared__ float sh[8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;
  float s = 0.f;
  if (c < D)
    for (int p = r; p < parts; p += 8) s += part[(int64_t)p * D + c];
  sh[r][threadIdx.x & 31] = s;
  __syncthreads();
  if (r == 0 && c < D) {
#pragma unroll
    for (int k = 1; k < 8; ++k) s += sh[k][threadIdx.x & 31];
    dw[c] = s;
  }
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

template <typename XT, typename RT, Out OUT, int G, int NV>
kdn_status fwd_go(const FwdArgs& a, cudaStream_t s) {
  // a warp's row: as many warps a block as still give every SM a block
  int warps = 8;
  if (G == 32)
    while (warps > 1 && (a.rows + warps - 1) / warps < 148) warps >>= 1;
  const int threads = G == 32 ? 32 * warps : G;
  const int64_t blocks = G == 32 ? (a.rows + warps - 1) / warps : a.rows;
  rmsnorm_forward_kernel<XT, RT, OUT, G, NV><<<(unsigned)blocks, threads, 0, s>>>(
      static_cast<const XT*>(a.x), static_cast<const RT*>(a.res), a.w, static_cast<RT*>(a.h), a.y,
      a.scale, a.rows, a.D, a.ldy, a.eps, a.D % 8 == 0);
  return cudaGetLastError() == cudaSuccess ? KDN_OK : KDN_ERR_CUDA;
}
// A row of up to 2048 goes to one warp (no barrier), a longer one to 256
// threads.
template <typename XT, typename RT, Out OUT>
kdn_status fwd_size(const FwdArgs& a, cudaStream_t s) {
  if (a.D <= 256) return fwd_go<XT, RT, OUT, 32, 1>(a, s);
  if (a.D <= 512) return fwd_go<XT, RT, OUT, 32, 2>(a, s);
  if (a.D <= 1024) return fwd_go<XT, RT, OUT, 32, 4>(a, s);
  if (a.D <= 2048) return fwd_go<XT, RT, OUT, 32, 8>(a, s);
  if (a.D <= 4096) return fwd_go<XT, RT, OUT, 256, 2>(a, s);
  if (a.D <= 8192) return fwd_go<XT, RT, OUT, 256, 4>(a, s);
  return fwd_go<XT, RT, OUT, 256, 8>(a, s);
}
template <typename XT, typename RT>
kdn_status fwd_out(const FwdArgs& a, kdn_dtype out, cudaStream_t s) {
  if (out == KDN_F32) return fwd_size<XT, RT, Out::F32>(a, s);
  if (out == KDN_BF16) return fwd_size<XT, RT, Out::BF16>(a, s);
  return fwd_size<XT, RT, Out::E4M3>(a, s);
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

template <typename HT, typename YT, typename XT, int G, int NV>
kdn_status bwd_go(const BwdArgs& a, cudaStream_t s) {
  const int64_t per = 256 / G;
  const int64_t want = (a.rows + per - 1) / per;
  const int blocks = (int)(want < kNormBwdBlocks ? want : kNormBwdBlocks);
  const size_t smem = G == 32 ? (size_t)8 * a.D * 4 : 0;
  if (blocks > 0) {
    rmsnorm_backward_kernel<HT, YT, XT, G, NV><<<blocks, 256, smem, s>>>(
        static_cast<const HT*>(a.h), a.w, static_cast<const YT*>(a.dy),
        static_cast<const HT*>(a.dh), static_cast<XT*>(a.dx), static_cast<HT*>(a.dres), a.part,
        a.rows, a.D, a.eps, a.D % 8 == 0);
    if (cudaGetLastError() != cudaSuccess) return KDN_ERR_CUDA;
  }
  rmsnorm_dweight_kernel<<<(a.D + 31) / 32, 256, 0, s>>>(a.part, a.dw, blocks, a.D);
  return cudaGetLastError() == cudaSuccess ? KDN_OK : KDN_ERR_CUDA;
}
template <typename HT, typename YT, typename XT>
kdn_status bwd_size(const BwdArgs& a, cudaStream_t s) {
  if (a.D <= 256) return bwd_go<HT, YT, XT, 32, 1>(a, s);
  if (a.D <= 512) return bwd_go<HT, YT, XT, 32, 2>(a, s);
  if (a.D <= 1024) return bwd_go<HT, YT, XT, 32, 4>(a, s);
  if (a.D <= 2048) return bwd_go<HT, YT, XT, 256, 1>(a, s);
  if (a.D <= 4096) return bwd_go<HT, YT, XT, 256, 2>(a, s);
  if (a.D <= 8192) return bwd_go<HT, YT, XT, 256, 4>(a, s);
  return bwd_go<HT, YT, XT, 256, 8>(a, s);
}
template <typename HT, typename YT>
kdn_status bwd_x(const BwdArgs& a, kdn_dtype x, cudaStream_t s) {
  return x == KDN_F32 ? bwd_size<HT, YT, float>(a, s) : bwd_size<HT, YT, __nv_bfloat16>(a, s);
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
  if (!res) rt = KDN_F32;  // not read
  if (xt == KDN_F32)
    return rt == KDN_F32 ? fwd_out<float, float>(a, yt, s) : fwd_out<float, bf>(a, yt, s);
  return rt == KDN_F32 ? fwd_out<bf, float>(a, yt, s) : fwd_out<bf, bf>(a, yt, s);
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
