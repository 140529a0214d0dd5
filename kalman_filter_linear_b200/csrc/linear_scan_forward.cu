// kdn_linear_scan_forward and kdn_linear_scan_step: the gated linear
// recurrence h_t = a_t h_{t-1} + b_t x_t per channel (linear_scan.cuh has the
// tile and the look-back).
#include "linear_scan.cuh"
#include "linear_scan_call.h"

namespace kdn {
namespace {

template <typename GT, typename XT, bool HAS_B, bool PACKED, bool EVEN>
__global__ void __launch_bounds__(kLsThreads, 2)
linear_scan_forward_kernel(const GT* __restrict__ Ag, const GT* __restrict__ Bg,
                           const XT* __restrict__ X, const float* h0, XT* __restrict__ Y,
                           float* h_out, const int32_t* __restrict__ cu, int N, int T, int D,
                           int groups, int64_t chunks, int64_t cols, LsWs ws) {
  constexpr int L = kLsFwdSteps;
  __shared__ LsShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t tile = blockIdx.x;
  if (chunks > 1) {
    if (threadIdx.x == 0) sh.tile = atomicAdd(ws.counter, 1u);
    __syncthreads();
    tile = sh.tile;
  }
  const int64_t j = tile / cols, col = tile - j * cols;
  const int bi = (int)(col / groups), grp = (int)(col - (int64_t)bi * groups);
  const int c = grp * kLsChannels + 2 * lane;
  const int have = max(0, min(2, D - c));
  const int t0 = (int)(j * (L * kLsWarps)) + warp * L;
  const int end = PACKED ? min(T, __ldg(cu + N)) : T;
  const size_t base = (size_t)bi * T * D + c;

  float2 a[L], u[L];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int hv = t0 + i < end ? have : 0;
    const size_t at = base + (size_t)(t0 + i) * D;
    a[i] = ls_load2<EVEN>(Ag, at, hv, 1.f);
    u[i] = ls_load2<EVEN>(X, at, hv, 0.f);
    if (HAS_B) {
      const float2 b = ls_load2<EVEN>(Bg, at, hv, 0.f);
      u[i].x *= b.x;
      u[i].y *= b.y;
    }
  }
  // packed: the sequence of this warp's first step, and which steps begin one
  int seq = 0, next = 0;
  uint32_t first = 0;
  if (PACKED && t0 < end) {
    seq = ls_sequence_of(cu, N, t0);
    next = __ldg(cu + seq + 1);
    int s = seq, nx = next;
    if (__ldg(cu + s) == t0) first |= 1u;
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int t = t0 + i;
      if (i > 0 && t < end && t >= nx) {
        while (s + 1 < N && t >= nx) nx = __ldg(cu + ++s + 1);
        first |= 1u << i;
      }
      if ((first >> i) & 1u) {
        const float2 s0 = h0 ? ls_load2<false>(h0, (size_t)s * D + c, have, 0.f)
                             : make_float2(0.f, 0.f);
        u[i].x = fmaf(a[i].x, s0.x, u[i].x);
        u[i].y = fmaf(a[i].y, s0.y, u[i].y);
      }
    }
  }

  // this warp's map
  float A0 = 1.f, H0 = 0.f, A1 = 1.f, H1 = 0.f;
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const bool f = PACKED && ((first >> i) & 1u);
    ls_compose<PACKED>(A0, H0, f ? ls_const_mark() : (PACKED ? a[i].x + 0.f : a[i].x), u[i].x);
    ls_compose<PACKED>(A1, H1, f ? ls_const_mark() : (PACKED ? a[i].y + 0.f : a[i].y), u[i].y);
  }
  sh.warp_map[warp][lane] = make_float4(A0, H0, A1, H1);
  __syncthreads();
  if (warp == 0) {
    float4 m = sh.warp_map[0][lane];
#pragma unroll
    for (int w = 1; w < kLsWarps; ++w) {
      const float4 l = sh.warp_map[w][lane];
      ls_compose<PACKED>(m.x, m.y, l.x, l.y);
      ls_compose<PACKED>(m.z, m.w, l.z, l.w);
    }
    float2 init = make_float2(0.f, 0.f);
    if (!PACKED && h0 && j == 0) init = ls_load2<false>(h0, (size_t)bi * D + c, have, 0.f);
    sh.start[lane] = ls_look_back<PACKED>(ws, j, col, cols, j == chunks - 1, m, init);
  }
  __syncthreads();

  float2 h = sh.start[lane];
  for (int w = 0; w < warp; ++w) {
    const float4 m = sh.warp_map[w][lane];
    h.x = ls_apply<PACKED>(m.x, m.y, h.x);
    h.y = ls_apply<PACKED>(m.z, m.w, h.y);
  }
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int t = t0 + i;
    if (PACKED && ((first >> i) & 1u)) {
      h = u[i];
    } else {
      h.x = fmaf(a[i].x, h.x, u[i].x);
      h.y = fmaf(a[i].y, h.y, u[i].y);
    }
    if (t < end) {
      ls_store2<EVEN>(Y, base + (size_t)t * D, have, h);
      if (!PACKED) {
        if (t == T - 1) ls_store2<false>(h_out, (size_t)bi * D + c, have, h);
      } else {
        while (t >= next && seq + 1 < N) next = __ldg(cu + ++seq + 1);
        if (t + 1 == next) ls_store2<false>(h_out, (size_t)seq * D + c, have, h);
      }
    }
  }
  if (!PACKED && chunks == 1 && tile == 0 && threadIdx.x == 0) *ws.error = DEV_OK;
  // sequences without steps hand their initial state through
  if (!PACKED) {
    if (T == 0 && warp == 0)
      ls_store2<false>(h_out, (size_t)bi * D + c, have,
                       h0 ? ls_load2<false>(h0, (size_t)bi * D + c, have, 0.f)
                          : make_float2(0.f, 0.f));
  } else if (j == 0) {
    for (int s = warp; s < N; s += kLsWarps)
      if (__ldg(cu + s) >= __ldg(cu + s + 1))
        ls_store2<false>(h_out, (size_t)s * D + c, have,
                         h0 ? ls_load2<false>(h0, (size_t)s * D + c, have, 0.f)
                            : make_float2(0.f, 0.f));
    if (grp == 0) {
      if (chunks == 1) {
        // (with one step range nothing has cleared the word)
        if (threadIdx.x == 0) *ws.error = DEV_OK;
        __syncthreads();
      }
      ls_check_offsets(cu, N, T, ws.error);
    }
  }
}

// One token: the state and the gates are read once, four elements a thread
// (the arrays are flat, so only the last thread may have fewer).
template <typename GT, typename XT, bool HAS_B>
__global__ void __launch_bounds__(128)
linear_scan_step_kernel(const GT* __restrict__ Ag, const GT* __restrict__ Bg,
                        const XT* __restrict__ X, float* __restrict__ Hs, XT* __restrict__ Y,
                        int64_t n) {
  const int64_t i = ((int64_t)blockIdx.x * 128 + threadIdx.x) * 4;
  if (i >= n) return;
  if (i + 4 <= n) {
    float2 a0 = ls_load2<true>(Ag, i, 1, 0.f), a1 = ls_load2<true>(Ag, i + 2, 1, 0.f);
    float2 u0 = ls_load2<true>(X, i, 1, 0.f), u1 = ls_load2<true>(X, i + 2, 1, 0.f);
    float4 h = *reinterpret_cast<const float4*>(Hs + i);
    if (HAS_B) {
      const float2 b0 = ls_load2<true>(Bg, i, 1, 0.f), b1 = ls_load2<true>(Bg, i + 2, 1, 0.f);
      u0.x *= b0.x, u0.y *= b0.y, u1.x *= b1.x, u1.y *= b1.y;
    }
    h.x = fmaf(a0.x, h.x, u0.x);
    h.y = fmaf(a0.y, h.y, u0.y);
    h.z = fmaf(a1.x, h.z, u1.x);
    h.w = fmaf(a1.y, h.w, u1.y);
    *reinterpret_cast<float4*>(Hs + i) = h;
    ls_store2<true>(Y, i, 1, make_float2(h.x, h.y));
    ls_store2<true>(Y, i + 2, 1, make_float2(h.z, h.w));
    return;
  }
  for (int64_t e = i; e < n; ++e) {
    float u = to_f32<XT>(X[e]);
    if (HAS_B) u *= to_f32<GT>(Bg[e]);
    const float h = fmaf(to_f32<GT>(Ag[e]), Hs[e], u);
    Hs[e] = h;
    if constexpr (sizeof(XT) == 2) Y[e] = __float2bfloat16_rn(h);
    else Y[e] = h;
  }
}

template <typename GT, typename XT, bool HAS_B>
kdn_status step_launch(const void* a, const void* b, const void* x, float* h, void* y, int64_t n,
                       cudaStream_t s) {
  const int64_t blocks = (n + 511) / 512;
  return launch(linear_scan_step_kernel<GT, XT, HAS_B>, blocks, 128, 0, s,
                static_cast<const GT*>(a), static_cast<const GT*>(b), static_cast<const XT*>(x), h,
                static_cast<XT*>(y), n);
}

template <typename GT, typename XT, bool HAS_B, bool PACKED, bool EVEN>
kdn_status forward_go(const LsCall& k) {
  const LsPlan p = ls_plan(k.B, k.T, k.D, kLsFwdSteps * kLsWarps);
  const LsWs ws = ls_ws(k.workspace, p);
  // error word, tile counter and flags (one step range: the kernel itself)
  if (p.chunks > 1) {
    const kdn_status st = enqueued(cudaMemsetAsync(k.workspace, 0, p.map, k.stream));
    if (st != KDN_OK) return st;
  }
  return launch(linear_scan_forward_kernel<GT, XT, HAS_B, PACKED, EVEN>, p.chunks * p.cols,
                kLsThreads, 0, k.stream, static_cast<const GT*>(k.a), static_cast<const GT*>(k.b),
                static_cast<const XT*>(k.x), k.h0, static_cast<XT*>(k.y_out), k.end_out, k.cu, k.N,
                k.T, k.D, (int)(p.cols / k.B), p.chunks, p.cols, ws);
}

template <typename GT, typename XT>
kdn_status forward_types(const LsCall& k) {
  const bool even = (k.D & 1) == 0;
#define KDN_LS_CASE(HB, PK, EV)                                          \
  if ((k.b != nullptr) == HB && (k.cu != nullptr) == PK && even == EV) \
    return forward_go<GT, XT, HB, PK, EV>(k);
  KDN_LS_CASE(false, false, true)
  KDN_LS_CASE(true, false, true)
  KDN_LS_CASE(false, true, true)
  KDN_LS_CASE(true, true, true)
  KDN_LS_CASE(false, false, false)
  KDN_LS_CASE(true, false, false)
  KDN_LS_CASE(false, true, false)
  KDN_LS_CASE(true, true, false)
#undef KDN_LS_CASE
  return KDN_ERR_UNSUPPORTED;
}

}  // namespace

// Of both directions and any types.  Several entries (which are never packed)
// of more than two columns always stream, and then need the error word alone.
size_t linear_scan_workspace_size(int B, int T, int D) {
  const LsPlan p = ls_plan(B, T, D, kLsBwdSteps * kLsWarps);
  const bool streams = B > 1 && p.cols > 2 && (int64_t)B * T < int64_t(1) << 33 && D < 1 << 27;
  return streams ? 256 : p.bytes;
}

// B entries of T steps, or (cu) N sequences packed in T steps with B = 1
kdn_status linear_scan_forward_launch(const void* a, const void* b, kdn_dtype gate_dtype,
                                      const void* x, kdn_dtype in_dtype, const float* h0, void* y,
                                      float* h_out, const int32_t* cu, int N, int B, int T, int D,
                                      void* workspace, cudaStream_t s, int64_t skip) {
  LsCall k{};
  k.a = a;
  k.b = b;
  k.x = x;
  k.gate_dtype = gate_dtype;
  k.in_dtype = in_dtype;
  k.h0 = h0;
  k.y_out = y;
  k.end_out = h_out;
  k.cu = cu;
  k.N = N;
  k.B = B;
  k.T = T;
  k.D = D;
  k.workspace = workspace;
  k.stream = s;
  k.skip = skip;
  kdn_status st = KDN_OK;
  if (D % 8 == 0 ? ls_stream_call<false, true>(k, &st) : ls_stream_call<false, false>(k, &st))
    return st;
  using bf = __nv_bfloat16;
  if (gate_dtype == KDN_F32)
    return in_dtype == KDN_F32 ? forward_types<float, float>(k) : forward_types<float, bf>(k);
  return in_dtype == KDN_F32 ? forward_types<bf, float>(k) : forward_types<bf, bf>(k);
}

kdn_status linear_scan_step_launch(const void* a, const void* b, kdn_dtype gate_dtype,
                                   const void* x, kdn_dtype in_dtype, float* h, void* y, int64_t n,
                                   cudaStream_t s) {
  const int key = (gate_dtype == KDN_BF16 ? 4 : 0) + (in_dtype == KDN_BF16 ? 2 : 0) + (b ? 1 : 0);
  using bf = __nv_bfloat16;
  switch (key) {
    case 0: return step_launch<float, float, false>(a, b, x, h, y, n, s);
    case 1: return step_launch<float, float, true>(a, b, x, h, y, n, s);
    case 2: return step_launch<float, bf, false>(a, b, x, h, y, n, s);
    case 3: return step_launch<float, bf, true>(a, b, x, h, y, n, s);
    case 4: return step_launch<bf, float, false>(a, b, x, h, y, n, s);
    case 5: return step_launch<bf, float, true>(a, b, x, h, y, n, s);
    case 6: return step_launch<bf, bf, false>(a, b, x, h, y, n, s);
    default: return step_launch<bf, bf, true>(a, b, x, h, y, n, s);
  }
}

}  // namespace kdn
