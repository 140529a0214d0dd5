// kdn_linear_scan_backward: the gradients of the gated linear recurrence
// h_t = a_t h_{t-1} + b_t x_t, y = h, from the last step to the first.  With c
// the gradient that reaches the state after step t from the steps behind it
// (dL/dh_T behind the last):
//   g = dy_t + c,   dx_t = b_t g,   db_t = x_t g,   da_t = g h_{t-1},
//   c <- a_t g      (dL/dh0 after the first step)
// so c is itself the recurrence c <- a_t c + a_t dy_t, and the tile and the
// look-back are the forward's (linear_scan.cuh), with the steps counted from
// the end.  h_{t-1} is read from the forward's y: where y is bf16 that is its
// rounded value (half a bf16 step of relative error in da, as da's own
// rounding), which saves running the forward again.
#include "linear_scan.cuh"
#include "linear_scan_call.h"

namespace kdn {
namespace {

template <typename GT, typename XT, bool HAS_B, bool PACKED, bool EVEN>
__global__ void __launch_bounds__(kLsThreads, 2)
linear_scan_backward_kernel(const GT* __restrict__ Ag, const GT* __restrict__ Bg,
                            const XT* __restrict__ X, const XT* __restrict__ Y,
                            const XT* __restrict__ dY, const float* __restrict__ h0,
                            const float* dhT, GT* __restrict__ dA, GT* __restrict__ dB,
                            XT* __restrict__ dX, float* dh0, const int32_t* __restrict__ cu,
                            int N, int T, int D, int groups, int64_t chunks, int64_t cols,
                            LsWs ws) {
  constexpr int L = kLsBwdSteps;
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
  const int end = PACKED ? min(T, __ldg(cu + N)) : T;
  // step i of this warp is token t0 - i
  const int t0 = T - 1 - ((int)(j * (L * kLsWarps)) + warp * L);
  const size_t base = (size_t)bi * T * D + c;

  // tokens that do not exist are identity steps (a = 1, dy = 0)
  float2 a[L], dy[L], hp[L], b[L], x[L];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int t = t0 - i;
    const int hv = t >= 0 && t < end ? have : 0;
    const size_t at = base + (size_t)(hv ? t : 0) * D;
    a[i] = ls_load2<EVEN>(Ag, at, hv, 1.f);
    dy[i] = ls_load2<EVEN>(dY, at, hv, 0.f);
    hp[i] = ls_load2<EVEN>(Y, at - (t > 0 ? D : 0), t > 0 ? hv : 0, 0.f);
    if (HAS_B) {
      b[i] = ls_load2<EVEN>(Bg, at, hv, 0.f);
      x[i] = ls_load2<EVEN>(X, at, hv, 0.f);
    }
  }
  // packed: the sequence of this warp's latest token, and which tokens end one
  int seq = 0;
  uint32_t fin = 0;
  const int ta = min(t0, end - 1);  // the latest token there is (< 0: none)
  if (PACKED && ta >= 0 && ta > t0 - L) {
    seq = ls_sequence_of(cu, N, ta);
    int s = seq, nx = __ldg(cu + seq + 1), lo = __ldg(cu + seq);
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int t = t0 - i;
      if (t >= 0 && t < end) {
        if (t < lo) {
          while (s > 0 && t < lo) lo = __ldg(cu + --s);
          nx = __ldg(cu + s + 1);
        }
        if (t + 1 == nx) {
          fin |= 1u << i;
          if (dhT) {
            const float2 d = ls_load2<false>(dhT, (size_t)s * D + c, have, 0.f);
            dy[i].x += d.x;
            dy[i].y += d.y;
          }
        }
      }
    }
  }

  float A0 = 1.f, H0 = 0.f, A1 = 1.f, H1 = 0.f;
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const bool f = PACKED && ((fin >> i) & 1u);
    ls_compose<PACKED>(A0, H0, f ? ls_const_mark() : (PACKED ? a[i].x + 0.f : a[i].x),
                       a[i].x * dy[i].x);
    ls_compose<PACKED>(A1, H1, f ? ls_const_mark() : (PACKED ? a[i].y + 0.f : a[i].y),
                       a[i].y * dy[i].y);
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
    if (!PACKED && dhT && j == 0) init = ls_load2<false>(dhT, (size_t)bi * D + c, have, 0.f);
    sh.start[lane] = ls_look_back<PACKED>(ws, j, col, cols, j == chunks - 1, m, init);
  }
  __syncthreads();

  float2 cc = sh.start[lane];
  for (int w = 0; w < warp; ++w) {
    const float4 m = sh.warp_map[w][lane];
    cc.x = ls_apply<PACKED>(m.x, m.y, cc.x);
    cc.y = ls_apply<PACKED>(m.z, m.w, cc.y);
  }
  int lo = PACKED ? __ldg(cu + seq) : 0;
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int t = t0 - i;
    if (PACKED && ((fin >> i) & 1u)) cc = make_float2(0.f, 0.f);
    const float2 g = make_float2(dy[i].x + cc.x, dy[i].y + cc.y);
    if (t >= 0 && t < end) {
      if (PACKED) {
        while (seq > 0 && t < lo) lo = __ldg(cu + --seq);
      }
      const size_t at = base + (size_t)t * D;
      const bool is_first = t == lo;
      if (is_first)
        hp[i] = h0 ? ls_load2<false>(h0, (size_t)(PACKED ? seq : bi) * D + c, have, 0.f)
                   : make_float2(0.f, 0.f);
      ls_store2<EVEN>(dA, at, have, make_float2(g.x * hp[i].x, g.y * hp[i].y));
      if (HAS_B) {
        ls_store2<EVEN>(dB, at, have, make_float2(g.x * x[i].x, g.y * x[i].y));
        ls_store2<EVEN>(dX, at, have, make_float2(g.x * b[i].x, g.y * b[i].y));
      } else {
        ls_store2<EVEN>(dX, at, have, g);
      }
      cc = make_float2(a[i].x * g.x, a[i].y * g.y);
      if (is_first) ls_store2<false>(dh0, (size_t)(PACKED ? seq : bi) * D + c, have, cc);
    }
  }
  if (!PACKED && chunks == 1 && tile == 0 && threadIdx.x == 0) *ws.error = DEV_OK;
  // sequences without steps hand the gradient through
  if (!PACKED) {
    if (T == 0 && warp == 0)
      ls_store2<false>(dh0, (size_t)bi * D + c, have,
                       dhT ? ls_load2<false>(dhT, (size_t)bi * D + c, have, 0.f)
                           : make_float2(0.f, 0.f));
  } else if (j == 0) {
    for (int s = warp; s < N; s += kLsWarps)
      if (__ldg(cu + s) >= __ldg(cu + s + 1))
        ls_store2<false>(dh0, (size_t)s * D + c, have,
                         dhT ? ls_load2<false>(dhT, (size_t)s * D + c, have, 0.f)
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

template <typename GT, typename XT, bool HAS_B, bool PACKED, bool EVEN>
kdn_status backward_go(const LsCall& k) {
  const LsPlan p = ls_plan(k.B, k.T, k.D, kLsBwdSteps * kLsWarps);
  const LsWs ws = ls_ws(k.workspace, p);
  // error word, tile counter and flags (one step range: the kernel itself)
  if (p.chunks > 1) {
    const kdn_status st = enqueued(cudaMemsetAsync(k.workspace, 0, p.map, k.stream));
    if (st != KDN_OK) return st;
  }
  return launch(linear_scan_backward_kernel<GT, XT, HAS_B, PACKED, EVEN>, p.chunks * p.cols,
                kLsThreads, 0, k.stream, static_cast<const GT*>(k.a), static_cast<const GT*>(k.b),
                static_cast<const XT*>(k.x), static_cast<const XT*>(k.y),
                static_cast<const XT*>(k.dy), k.h0, k.end_in, static_cast<GT*>(k.da),
                static_cast<GT*>(k.db), static_cast<XT*>(k.dx), k.end_out, k.cu, k.N, k.T, k.D,
                (int)(p.cols / k.B), p.chunks, p.cols, ws);
}

template <typename GT, typename XT>
kdn_status backward_types(const LsCall& k) {
  const bool even = (k.D & 1) == 0;
#define KDN_LS_CASE(HB, PK, EV)                                          \
  if ((k.b != nullptr) == HB && (k.cu != nullptr) == PK && even == EV) \
    return backward_go<GT, XT, HB, PK, EV>(k);
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

// B entries of T steps, or (cu) N sequences packed in T steps with B = 1
kdn_status linear_scan_backward_launch(const void* a, const void* b, kdn_dtype gate_dtype,
                                       const void* x, const void* y, const void* dy,
                                       kdn_dtype in_dtype, const float* h0, const float* dhT,
                                       void* da, void* db, void* dx, float* dh0, const int32_t* cu,
                                       int N, int B, int T, int D, void* workspace,
                                       cudaStream_t s) {
  LsCall k{};
  k.a = a;
  k.b = b;
  k.x = x;
  k.y = y;
  k.dy = dy;
  k.gate_dtype = gate_dtype;
  k.in_dtype = in_dtype;
  k.h0 = h0;
  k.end_in = dhT;
  k.da = da;
  k.db = db;
  k.dx = dx;
  k.end_out = dh0;
  k.cu = cu;
  k.N = N;
  k.B = B;
  k.T = T;
  k.D = D;
  k.workspace = workspace;
  k.stream = s;
  k.skip = -1;
  kdn_status st = KDN_OK;
  if (D % 8 == 0 ? ls_stream_call<true, true>(k, &st) : ls_stream_call<true, false>(k, &st))
    return st;
  using bf = __nv_bfloat16;
  if (gate_dtype == KDN_F32)
    return in_dtype == KDN_F32 ? backward_types<float, float>(k) : backward_types<float, bf>(k);
  return in_dtype == KDN_F32 ? backward_types<bf, float>(k) : backward_types<bf, bf>(k);
}

}  // namespace kdn
