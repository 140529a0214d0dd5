// e4m3 blocks of 128 with one fp32 scale: value = code * scale,
//   scale = max(amax, 2^-100) / 448,  code = e4m3(value / scale).
// 448 is the largest e4m3 number, so a block's largest value uses the whole
// range; the floor keeps a block of zeros from dividing by zero.  An infinity
// or NaN in a block makes its scale infinite or NaN (the maximum propagates
// NaN), which marks every product of that block instead of hiding it.
#pragma once

#include <cuda_fp8.h>

#include "kdn_common.cuh"

namespace kdn {

constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 7.8886090522101181e-31f;  // 2^-100

// the larger of two numbers, NaN if one is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float fp8_scale(float amax) {
  return max_nan(amax, kAmaxFloor) / kE4m3Max;
}
// what a value is multiplied with for its code: 1 / scale from the maximum
// itself, so that the quotient carries two roundings, not three
__device__ __forceinline__ float fp8_inverse(float amax) {
  return kE4m3Max / max_nan(amax, kAmaxFloor);
}
// four codes, the first in the lowest byte
__device__ __forceinline__ uint32_t fp8_pack4(float q0, float q1, float q2, float q3) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q0, q1), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q2, q3), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// A code is the rounding of a quotient that itself carries a few fp32 roundings,
// so near the middle between two codes it may be the other one.  The middle of
// two normal codes has the bits 1000... below the third of the fraction;
// fp8_near tells whether a quotient is within ULPS units in the last place of
// it, and such a quotient is decided again in fp64.  Below 2^-6, the smallest
// normal code, codes are 2^-9 apart whatever the exponent: 2^-6 added (lifted),
// their middles have the same bits, and the few units of a smaller quotient are
// fewer of the sum's.
constexpr float kE4m3Normal = 0.015625f;  // 2^-6
template <uint32_t ULPS>
__device__ __forceinline__ uint32_t fp8_from_middle(float q) {
  return __float_as_uint(q) * 4096u + ((ULPS - 0x80000u) << 12);
}
template <uint32_t ULPS>
__device__ __forceinline__ bool fp8_near(uint32_t from_middle) {
  return from_middle <= 2u * ULPS << 12;
}
template <uint32_t ULPS>
__device__ __forceinline__ bool fp8_near_lifted(float q) {
  const float m = fabsf(q);
  return fp8_near<ULPS>(fp8_from_middle<ULPS>(m < kE4m3Normal ? m + kE4m3Normal : m));
}
// Whether any of the quotients is near a middle (or seems to be: a normal one that
// is lifted all the same, where another is small, may ask without need).  Small
// ones are looked for first: a lift for each of them cost 3 % of fp32 rows.
template <uint32_t ULPS, int N>
__device__ __forceinline__ bool fp8_any_near(const float (&q)[N]) {
  uint32_t near = ~0u;
  float least = kE4m3Normal;
#pragma unroll
  for (int i = 0; i < N; ++i) near = min(near, fp8_from_middle<ULPS>(q[i]));
#pragma unroll
  for (int i = 0; i < N; ++i) least = fminf(least, fabsf(q[i]));
  if (least < kE4m3Normal) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      near = min(near, fp8_from_middle<ULPS>(fabsf(q[i]) + kE4m3Normal));
  }
  return fp8_near<ULPS>(near);
}
// The middle of the two codes that q is between, as a float (it is one).
__device__ __forceinline__ float fp8_middle(float q) {
  const float m = fabsf(q);
  return m < kE4m3Normal ? (floorf(m * 512.f) + 0.5f) / 512.f
                         : __uint_as_float((__float_as_uint(m) & 0xfff00000u) | 0x80000u);
}
// The float nearest to q on the side of its middle that the exact quotient is
// on; over: the sign of the exact magnitude less the middle's.
__device__ __forceinline__ float fp8_side(float q, double over) {
  const uint32_t b = __float_as_uint(fp8_middle(q));
  return copysignf(__uint_as_float(over > 0.0 ? b + 1u : over < 0.0 ? b - 1u : b), q);
}
// The quotients of a block's values, `top` its largest magnitude; and whether a
// code has to be decided in fp64.
// fp32: v * inv has two roundings, at most two units.
// bf16: a quotient of two numbers of eight bits is the middle of two codes or
// 2^-13 of itself away from it, and v hi + v lo, where hi + lo is the inverse to
// more than twice the bits, rounds to the middle where it is one.
template <typename XT>
struct Fp8Block {
  float inv, top;
  __device__ __forceinline__ explicit Fp8Block(float m)
      : inv(fp8_inverse(m)), top(max_nan(m, kAmaxFloor)) {}
  // (through shared memory as two floats)
  __device__ __forceinline__ Fp8Block(float a, float b) : inv(a), top(b) {}
  __device__ __forceinline__ float first() const { return inv; }
  __device__ __forceinline__ float second() const { return top; }
  Fp8Block() = default;
  template <int N>
  __device__ __forceinline__ bool quotients(const float (&v)[N], float (&q)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = v[i] * inv;
    return fp8_any_near<2>(q);
  }
};
template <>
struct Fp8Block<__nv_bfloat16> {
  float hi, lo;
  __device__ __forceinline__ explicit Fp8Block(float m) : hi(fp8_inverse(m)) {
    const float top = max_nan(m, kAmaxFloor);
    const float left = fmaf(-hi, top, kE4m3Max);  // exact
    lo = top <= 3.4e38f ? left * hi * (1.f / kE4m3Max) : 0.f;
  }
  __device__ __forceinline__ Fp8Block(float a, float b) : hi(a), lo(b) {}
  __device__ __forceinline__ float first() const { return hi; }
  __device__ __forceinline__ float second() const { return lo; }
  Fp8Block() = default;
  template <int N>
  __device__ __forceinline__ bool quotients(const float (&v)[N], float (&q)[N]) const {
    const float2 h = make_float2(hi, hi), l = make_float2(lo, lo);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 x = make_float2(v[i], v[i + 1]);
      const float2 r = __ffma2_rn(x, h, __fmul2_rn(x, l));
      q[i] = r.x;
      q[i + 1] = r.y;
    }
    return false;
  }
};
// Eight consecutive elements from `p`: `n` of them exist (the others read as
// 0).  vec: p is 16-byte aligned and all eight exist or none do.  On 32-byte
// boundaries eight floats are one access: two of 16 bytes leave every other
// half of a warp's sectors to the second one (5.6 instead of 6.2 TB/s in the
// norm of fp32 rows).
__device__ __forceinline__ void load8(const float* p, int n, bool vec, float (&v)[8]) {
  if (vec) {
    if (n > 0 && (reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
      asm volatile("ld.global.nc.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                     "=f"(v[6]), "=f"(v[7])
                   : "l"(p));
      return;
    }
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (n > 0) {
      a = __ldg(reinterpret_cast<const float4*>(p));
      b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? __ldg(p + i) : 0.f;
  }
}
__device__ __forceinline__ void unpack_bf16x8(const uint4& a, float (&v)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, int n, bool vec, float (&v)[8]) {
  if (vec) {
    uint4 a = make_uint4(0u, 0u, 0u, 0u);
    if (n > 0) a = __ldg(reinterpret_cast<const uint4*>(p));
    unpack_bf16x8(a, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? __bfloat162float(p[i]) : 0.f;
  }
}
__device__ __forceinline__ void store8(float* p, int n, bool vec, const float (&v)[8]) {
  if (vec) {
    if (n > 0 && (reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
      asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]),
                   "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                   : "memory");
    } else if (n > 0) {
      reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v[i];
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, int n, bool vec, const float (&v)[8]) {
  if (vec) {
    if (n > 0) {
      uint4 a;
      __nv_bfloat162 h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      a.x = *reinterpret_cast<uint32_t*>(&h[0]);
      a.y = *reinterpret_cast<uint32_t*>(&h[1]);
      a.z = *reinterpret_cast<uint32_t*>(&h[2]);
      a.w = *reinterpret_cast<uint32_t*>(&h[3]);
      *reinterpret_cast<uint4*>(p) = a;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = __float2bfloat16_rn(v[i]);
  }
}
__device__ __forceinline__ float amax8(const float (&v)[8]) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(v[i]));
  return m;
}
// the maximum over this thread's half warp (16 threads hold one block of 128)
__device__ __forceinline__ float half_warp_max(float m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

}  // namespace kdn
