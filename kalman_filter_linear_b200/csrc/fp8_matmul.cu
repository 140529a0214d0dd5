// kdn_fp8_matmul: out[m, n] = sum over k of x[m, k] w[n, k], both factors in
// e4m3 with an fp32 scale for each block of 128 along k (x: per row; w: per
// 128 x 128 tile, or per row):
//   out[m, n] = sum_b sx[m, b] sw[n or n/128, b] (sum_{k in block b} x8 w8).
// The inner sum runs on the tensor cores (tcgen05 kind::f8f6f4, fp32 in TMEM);
// products of e4m3 numbers are exact in fp32.  The scales change with every
// block, so each block's product leaves TMEM and is scaled and added in fp32
// registers while the tensor cores work on the next block (two TMEM buffers).
//
// fp8_matmul_wide: 128 x BN outputs a tile, one persistent CTA an SM.  Warp 0
// copies (TMA, 128-byte swizzle), warp 1 issues the MMAs, warps 4-11 scale and
// add: four warps cover the 128 rows (TMEM lanes), each group half the
// columns, so a thread has one row and its row scale, and stores whole
// 32-byte sectors of it.
//
// fp8_matmul_few: for few rows of x the bytes of w are what counts.  w is the
// 128-row operand and up to 64 rows of x are the columns; the blocks of k are
// split over a cluster of up to eight CTAs so that every SM streams w, and the
// parts meet through distributed shared memory, added in rank order.
//
// Every wait is bounded; one that gives up sets the status word.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "kdn_common.cuh"

namespace kdn {
namespace {

constexpr uint32_t kKb = 128;  // bytes (elements) of a block along k

// Instruction descriptor of kind::f8f6f4 with e4m3 A and B (format 0), both
// K-major, fp32 accumulation.
__host__ __device__ constexpr uint32_t umma_idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void umma_f8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t smem_dst, const void* tmap, uint64_t* bar,
                                            int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_dst),
      "l"(tmap), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}
// 32 (or 16) TMEM columns of this warp's lanes.  The wait names the registers,
// so no use of them can move above it.
__device__ __forceinline__ void tmem_ld_async(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_ld_async(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ float2 as_f2(uint32_t a, uint32_t b) {
  return make_float2(__uint_as_float(a), __uint_as_float(b));
}

// 16 outputs of one row from column n (columns below N exist).  align: the
// largest power of two of elements, at most 16, that divides N; less where
// `out` itself is not on a 32-byte boundary.
__device__ __forceinline__ void store16(__nv_bfloat16* p, int n, int N, int align,
                                        const float2* v) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[i].x, v[i].y);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  if (align >= 16 && n + 16 <= N) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else if (align >= 8) {
    if (n < N) reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    if (n + 8 < N) reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (n + 2 * i < N) p[2 * i] = __float2bfloat16_rn(v[i].x);
      if (n + 2 * i + 1 < N) p[2 * i + 1] = __float2bfloat16_rn(v[i].y);
    }
  }
}
__device__ __forceinline__ void store16(float* p, int n, int N, int align, const float2* v) {
  if (align >= 8) {
#pragma unroll
    for (int g = 0; g < 2; ++g)
      if (n + 8 * g < N)
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p + 8 * g),
                     "r"(__float_as_uint(v[4 * g].x)), "r"(__float_as_uint(v[4 * g].y)),
                     "r"(__float_as_uint(v[4 * g + 1].x)), "r"(__float_as_uint(v[4 * g + 1].y)),
                     "r"(__float_as_uint(v[4 * g + 2].x)), "r"(__float_as_uint(v[4 * g + 2].y)),
                     "r"(__float_as_uint(v[4 * g + 3].x)), "r"(__float_as_uint(v[4 * g + 3].y))
                     : "memory");
  } else if (align >= 4) {
#pragma unroll
    for (int g = 0; g < 4; ++g)
      if (n + 4 * g < N)
        reinterpret_cast<float4*>(p)[g] =
            make_float4(v[2 * g].x, v[2 * g].y, v[2 * g + 1].x, v[2 * g + 1].y);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (n + 2 * i < N) p[2 * i] = v[i].x;
      if (n + 2 * i + 1 < N) p[2 * i + 1] = v[i].y;
    }
  }
}

struct Prm {
  const float *sx, *sw;
  void* out;
  int M, N, kbs;         // rows of x, rows of w, blocks along k
  int align;             // elements of out that a vector store may take
  uint32_t* status;      // or null
};

// ------------------------------------------------------------------- wide
template <int BN>
struct Wide {
  static constexpr uint32_t A = 128 * kKb, B = BN * kKb, STAGE = A + B;
  static constexpr int STAGES = BN == 256 ? 4 : 6;
  static constexpr uint32_t OFF_SC = STAGES * STAGE;           // per warp: [2][BN / 2] scales
  static constexpr uint32_t SC = 8 * 2 * (BN / 2) * 4;
  static constexpr uint32_t OFF_BAR = OFF_SC + SC;
  static constexpr uint32_t NBAR = 2 * STAGES + 4;
  static constexpr uint32_t OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr uint32_t SMEM = OFF_MISC + 16 + 1024;       // 1024: alignment
  static_assert(SMEM <= 232448, "shared memory plan");
};

template <int BN, bool TILE, typename OT>
__global__ void __launch_bounds__(384, 1)
fp8_matmul_wide(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                Prm p, int tiles_n, int tiles) {
  using W = Wide<BN>;
  constexpr int S = W::STAGES;
  extern __shared__ uint8_t wsm_raw[];
  uint8_t* sm = wsm_raw + ((1024u - (smem_u32(wsm_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + W::OFF_BAR);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + 2;
  uint32_t* misc = reinterpret_cast<uint32_t*>(sm + W::OFF_MISC);
  volatile uint32_t* abort_flag = misc + 1;
  auto fail = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (*abort_flag) return true;
    if (mbar_wait(bar, parity)) return false;
    *abort_flag = 1u;
    if (p.status) atomicOr(p.status, DEV_TIMEOUT);
    return true;
  };
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 8);
    }
    misc[1] = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&mx);
    tma_prefetch_desc(&mw);
  }
  if (warp == 2) {
    tmem_alloc(misc, 2 * BN);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0 && lane == 0) {
      // copies
      uint32_t it = 0;
      bool bad = false;
      for (int tile = blockIdx.x; tile < tiles && !bad; tile += gridDim.x) {
        const int m0 = tile / tiles_n * 128, n0 = tile % tiles_n * BN;
        for (int kb = 0; kb < p.kbs; ++kb, ++it) {
          const uint32_t st = it % S;
          if (it >= (uint32_t)S && fail(&empty[st], ((it / S) - 1u) & 1u)) { bad = true; break; }
          mbar_expect_tx(&full[st], W::STAGE);
          tma_load_2d(sbase + st * W::STAGE, &mx, &full[st], kb * (int)kKb, m0);
          tma_load_2d(sbase + st * W::STAGE + W::A, &mw, &full[st], kb * (int)kKb, n0);
        }
      }
      // copies in flight land before the CTA's memory goes (bounded)
      if (bad)
        for (uint32_t i = it > (uint32_t)S ? it - S : 0; i < it; ++i)
          mbar_wait(&full[i % S], (i / S) & 1u);
    } else if (warp == 1 && lane == 0) {
      // MMAs
      constexpr uint32_t ID = umma_idesc_e4m3(128, BN);
      uint32_t it = 0;
      bool bad = false;
      for (int tile = blockIdx.x; tile < tiles && !bad; tile += gridDim.x) {
        for (int kb = 0; kb < p.kbs; ++kb, ++it) {
          const uint32_t st = it % S, buf = it & 1u;
          if (it >= 2 && fail(&tempty[buf], ((it >> 1) - 1u) & 1u)) { bad = true; break; }
          if (fail(&full[st], (it / S) & 1u)) { bad = true; break; }
          tc_fence_after();
          const uint32_t a = sbase + st * W::STAGE, b = a + W::A;
#pragma unroll
          for (uint32_t ks = 0; ks < 4; ++ks)
            umma_f8(tmem + buf * BN, umma_desc_sw128(a + 32u * ks, 16, 1024),
                    umma_desc_sw128(b + 32u * ks, 16, 1024), ID, ks > 0);
          umma_commit(&empty[st]);
          umma_commit(&tfull[buf]);
        }
      }
      // nothing may be in flight when TMEM is freed: the last two blocks'
      // commits (bounded)
      for (uint32_t i = it >= 2 ? it - 2 : 0; i < it; ++i) mbar_wait(&tfull[i & 1u], (i >> 1) & 1u);
    }
  } else {
    // scale and add
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    constexpr int CW = BN / 2;  // columns of a thread
    const int g = (warp - 4) >> 2;
    const int q = warp & 3;     // TMEM lane quarter
    const uint32_t tl = ((uint32_t)(32 * q) << 16) + (uint32_t)(g * CW);
    float* sc = reinterpret_cast<float*>(sm + W::OFF_SC) + (warp - 4) * 2 * CW;
    OT* out = static_cast<OT*>(p.out);
    uint32_t it = 0;
    bool bad = false;
    for (int tile = blockIdx.x; tile < tiles && !bad; tile += gridDim.x) {
      const int m = tile / tiles_n * 128 + 32 * q + lane;
      const int n0 = tile % tiles_n * BN + g * CW;
      const float* sxr = p.sx + (size_t)min(m, p.M - 1) * p.kbs;
      // rows of w's scales: one for all columns, or column lane + 32 i
      const float* swr[TILE ? 1 : CW / 32];
      if (TILE) {
        swr[0] = p.sw + (size_t)(min(n0, p.N - 1) >> 7) * p.kbs;
      } else {
#pragma unroll
        for (int i = 0; i < CW / 32; ++i)
          swr[TILE ? 0 : i] = p.sw + (size_t)min(n0 + lane + 32 * i, p.N - 1) * p.kbs;
      }
      float2 acc[CW / 2];
#pragma unroll
      for (int i = 0; i < CW / 2; ++i) acc[i] = make_float2(0.f, 0.f);
      float s_next = __ldg(sxr);
      float w_next[TILE ? 1 : CW / 32];
#pragma unroll
      for (int i = 0; i < (TILE ? 1 : CW / 32); ++i) w_next[i] = __ldg(swr[i]);
      for (int kb = 0; kb < p.kbs; ++kb, ++it) {
        const uint32_t buf = it & 1u;
        float s = s_next;
        float* cs = sc + buf * CW;
        if (TILE) {
          s *= w_next[0];
        } else {
#pragma unroll
          for (int i = 0; i < CW / 32; ++i) cs[lane + 32 * i] = w_next[TILE ? 0 : i];
        }
        if (kb + 1 < p.kbs) {
          s_next = __ldg(sxr + kb + 1);
#pragma unroll
          for (int i = 0; i < (TILE ? 1 : CW / 32); ++i) w_next[i] = __ldg(swr[i] + kb + 1);
        }
        if (!TILE) __syncwarp();
        if (fail(&tfull[buf], (it >> 1) & 1u)) bad = true;
        if (__any_sync(0xffffffffu, bad)) { bad = true; break; }
        tc_fence_after();
        const float2 ss = make_float2(s, s);
        uint32_t r[2][32];
        tmem_ld_async(tmem + tl + buf * BN, r[0]);
#pragma unroll
        for (int c = 0; c < CW / 32; ++c) {
          tmem_ld_wait(r[c & 1]);
          if (c + 1 < CW / 32) tmem_ld_async(tmem + tl + buf * BN + 32 * (c + 1), r[(c + 1) & 1]);
          else {
            // this warp has read the buffer
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[buf]);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float2 d = as_f2(r[c & 1][2 * i], r[c & 1][2 * i + 1]);
            if (!TILE) {
              const float2 cw = *reinterpret_cast<const float2*>(cs + 32 * c + 2 * i);
              d = __fmul2_rn(d, cw);
            }
            acc[16 * c + i] = __ffma2_rn(d, ss, acc[16 * c + i]);
          }
        }
      }
      if (bad) break;
      if (m < p.M) {
        OT* o = out + (size_t)m * p.N + n0;
#pragma unroll
        for (int c = 0; c < CW / 16; ++c) store16(o + 16 * c, n0 + 16 * c, p.N, p.align, acc + 8 * c);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * BN);
  }
}

// -------------------------------------------------------------------- few
// BT: columns of a tile (rows of x), 16, 32 or 64
template <int BT>
struct Few {
  static constexpr uint32_t A = 128 * kKb, B = BT * kKb, STAGE = A + B;
  static constexpr int STAGES = 8;
  static constexpr uint32_t OFF_SC = STAGES * STAGE;      // per warp: [2][BT] scales
  static constexpr uint32_t OFF_BAR = OFF_SC + 4 * 2 * BT * 4;
  static constexpr uint32_t NBAR = 2 * STAGES + 4;
  static constexpr uint32_t OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr uint32_t SMEM = OFF_MISC + 16 + 1024;
  static constexpr uint32_t COLS = 2 * BT;                 // 32, 64 or 128
  static_assert(SMEM <= 232448 && 128u * BT * 4 <= STAGES * STAGE, "shared memory plan");
};

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %1, %2;\n\t"
      "ld.shared::cluster.f32 %0, [a];\n\t}"
      : "=f"(v)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

template <int BT, bool TILE, typename OT>
__global__ void __launch_bounds__(256, 1)
fp8_matmul_few(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
               Prm p, int tiles_n, int split) {
  using F = Few<BT>;
  constexpr int S = F::STAGES;
  extern __shared__ uint8_t fsm_raw[];
  uint8_t* sm = fsm_raw + ((1024u - (smem_u32(fsm_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % split, tile = blockIdx.x / split;
  const int n0 = tile % tiles_n * 128, m0 = tile / tiles_n * BT;
  // this CTA's blocks along k
  const int k0 = (int)((int64_t)p.kbs * rank / split);
  const int nk = (int)((int64_t)p.kbs * (rank + 1) / split) - k0;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + F::OFF_BAR);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + 2;
  uint32_t* misc = reinterpret_cast<uint32_t*>(sm + F::OFF_MISC);
  volatile uint32_t* abort_flag = misc + 1;
  auto fail = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (*abort_flag) return true;
    if (mbar_wait(bar, parity)) return false;
    *abort_flag = 1u;
    if (p.status) atomicOr(p.status, DEV_TIMEOUT);
    return true;
  };
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 4);
    }
    misc[1] = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&mx);
    tma_prefetch_desc(&mw);
  }
  if (warp == 2) {
    tmem_alloc(misc, F::COLS);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];

  float2 acc[BT / 2];
#pragma unroll
  for (int i = 0; i < BT / 2; ++i) acc[i] = make_float2(0.f, 0.f);
  if (warp == 0 && lane == 0) {
    bool bad = false;
    int it = 0;
    for (; it < nk; ++it) {
      const int st = it % S;
      if (it >= S && fail(&empty[st], (uint32_t)((it / S) - 1) & 1u)) { bad = true; break; }
      mbar_expect_tx(&full[st], F::STAGE);
      tma_load_2d(sbase + st * F::STAGE, &mw, &full[st], (k0 + it) * (int)kKb, n0);
      tma_load_2d(sbase + st * F::STAGE + F::A, &mx, &full[st], (k0 + it) * (int)kKb, m0);
    }
    if (bad)
      for (int i = it > S ? it - S : 0; i < it; ++i) mbar_wait(&full[i % S], (uint32_t)(i / S) & 1u);
  } else if (warp == 1 && lane == 0) {
    constexpr uint32_t ID = umma_idesc_e4m3(128, BT);
    int it = 0;
    for (; it < nk; ++it) {
      const int st = it % S, buf = it & 1;
      if (it >= 2 && fail(&tempty[buf], (uint32_t)((it >> 1) - 1) & 1u)) break;
      if (fail(&full[st], (uint32_t)(it / S) & 1u)) break;
      tc_fence_after();
      const uint32_t a = sbase + st * F::STAGE, b = a + F::A;
#pragma unroll
      for (uint32_t ks = 0; ks < 4; ++ks)
        umma_f8(tmem + buf * BT, umma_desc_sw128(a + 32u * ks, 16, 1024),
                umma_desc_sw128(b + 32u * ks, 16, 1024), ID, ks > 0);
      umma_commit(&empty[st]);
      umma_commit(&tfull[buf]);
    }
    for (int i = it >= 2 ? it - 2 : 0; i < it; ++i) mbar_wait(&tfull[i & 1], (uint32_t)(i >> 1) & 1u);
  } else if (warp >= 4) {
    const int q = warp - 4;
    const int n = n0 + 32 * q + lane;  // this thread's row of w
    const uint32_t tl = (uint32_t)(32 * q) << 16;
    float* sc = reinterpret_cast<float*>(sm + F::OFF_SC) + q * 2 * BT;
    const float* swr = p.sw + (size_t)(TILE ? n0 >> 7 : min(n, p.N - 1)) * p.kbs + k0;
    // scales of x's rows: a lane fetches rows lane and lane + 32
    constexpr int NS = BT > 32 ? 2 : 1;
    const float* sxr[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i)
      sxr[i] = p.sx + (size_t)min(m0 + min(lane + 32 * i, BT - 1), p.M - 1) * p.kbs + k0;
    float w_next = __ldg(swr), x_next[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) x_next[i] = __ldg(sxr[i]);
    for (int it = 0; it < nk; ++it) {
      const uint32_t buf = it & 1;
      const float w = w_next;
      float* cs = sc + buf * BT;
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (lane + 32 * i < BT) cs[lane + 32 * i] = x_next[i];
      if (it + 1 < nk) {
        w_next = __ldg(swr + it + 1);
#pragma unroll
        for (int i = 0; i < NS; ++i) x_next[i] = __ldg(sxr[i] + it + 1);
      }
      __syncwarp();
      const bool bad = fail(&tfull[buf], (uint32_t)(it >> 1) & 1u);
      if (__any_sync(0xffffffffu, bad)) break;
      tc_fence_after();
      const float2 ww = make_float2(w, w);
      constexpr int CH = BT >= 32 ? 32 : 16;  // columns of one load
      uint32_t r[BT / CH][CH];
#pragma unroll
      for (int c = 0; c < BT / CH; ++c) tmem_ld_async(tmem + tl + buf * BT + CH * c, r[c]);
#pragma unroll
      for (int c = 0; c < BT / CH; ++c) tmem_ld_wait(r[c]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[buf]);
#pragma unroll
      for (int c = 0; c < BT / CH; ++c)
#pragma unroll
        for (int i = 0; i < CH / 2; ++i) {
          const float2 x2 = *reinterpret_cast<const float2*>(cs + CH * c + 2 * i);
          const float2 d = __fmul2_rn(as_f2(r[c][2 * i], r[c][2 * i + 1]), x2);
          acc[(CH / 2) * c + i] = __ffma2_rn(d, ww, acc[(CH / 2) * c + i]);
        }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, F::COLS);
  }
  // the parts of the cluster, [column][128 rows of w] each, over the stages
  // (all copies have landed and have been read)
  float* part = reinterpret_cast<float*>(sm);
  if (warp >= 4) {
    const int e = tid - 128;
#pragma unroll
    for (int i = 0; i < BT / 2; ++i) {
      part[(2 * i) * 128 + e] = acc[i].x;
      part[(2 * i + 1) * 128 + e] = acc[i].y;
    }
  }
  __syncwarp();
  if (split > 1) cluster_sync_all();
  else __syncthreads();
  {
    // rank r adds and stores columns r, r + split, ...: two at a time, one by
    // each half of the block
    OT* out = static_cast<OT*>(p.out);
    const int e = tid & 127, n = n0 + e;
    const int cols = min(BT, p.M - m0);
    for (int c = rank + split * (tid >> 7); c < cols; c += 2 * split) {
      float v;
      if (split == 1) {
        v = part[c * 128 + e];
      } else {
        const uint32_t at = smem_u32(part + c * 128 + e);
        float t[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) t[r] = r < split ? ld_cluster(at, r) : 0.f;
        v = t[0];
#pragma unroll
        for (int r = 1; r < 8; ++r) v += t[r];
      }
      if (n < p.N) {
        if constexpr (sizeof(OT) == 2) out[(size_t)(m0 + c) * p.N + n] = __float2bfloat16_rn(v);
        else out[(size_t)(m0 + c) * p.N + n] = v;
      }
    }
  }
  // no CTA's shared memory goes while another may read it
  __syncwarp();
  if (split > 1) cluster_sync_all();
}

// ------------------------------------------------------------------- host
PFN_cuTensorMapEncodeTiled_v12000 mm_encoder() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 f = fn.load(std::memory_order_acquire);
  if (!f) {
    void* q = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &q, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return nullptr;
    f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(q);
    fn.store(f, std::memory_order_release);
  }
  return f;
}

// [rows, K] bytes, rows ld bytes apart, boxes of 128 bytes x box rows; what
// lies outside reads as zero.
bool mm_map(CUtensorMap* m, const void* base, int rows, int K, int64_t ld, int box) {
  auto enc = mm_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld};
  cuuint32_t boxes[2] = {kKb, (cuuint32_t)box};
  cuuint32_t estr[2] = {1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, boxes,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The dynamic shared memory limit of a kernel, once for each device.
template <typename K>
bool allow_smem(K kernel, int bytes, int dev, std::atomic<uint64_t>& done) {
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
      cudaSuccess)
    return false;
  done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

template <int BN, bool TILE, typename OT>
kdn_status wide_go(const void* x, int64_t ldx, const void* w, int64_t ldw, int K, const Prm& p,
                   int dev, int sms, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  CUtensorMap mx, mw;
  if (!mm_map(&mx, x, p.M, K, ldx, 128) || !mm_map(&mw, w, p.N, K, ldw, BN) ||
      !allow_smem(fp8_matmul_wide<BN, TILE, OT>, (int)Wide<BN>::SMEM, dev, ready))
    return KDN_ERR_CUDA;
  const int tn = (p.N + BN - 1) / BN;
  const int64_t tiles = (int64_t)((p.M + 127) / 128) * tn;
  const int grid = (int)(tiles < sms ? tiles : sms);
  fp8_matmul_wide<BN, TILE, OT><<<grid, 384, Wide<BN>::SMEM, s>>>(mx, mw, p, tn, (int)tiles);
  return cudaGetLastError() == cudaSuccess ? KDN_OK : KDN_ERR_CUDA;
}

template <int BT, bool TILE, typename OT>
kdn_status few_go(const void* x, int64_t ldx, const void* w, int64_t ldw, int K, const Prm& p,
                  int dev, int sms, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  CUtensorMap mx, mw;
  if (!mm_map(&mx, x, p.M, K, ldx, BT) || !mm_map(&mw, w, p.N, K, ldw, 128) ||
      !allow_smem(fp8_matmul_few<BT, TILE, OT>, (int)Few<BT>::SMEM, dev, ready))
    return KDN_ERR_CUDA;
  const int tn = (p.N + 127) / 128;
  const int64_t tiles = (int64_t)((p.M + BT - 1) / BT) * tn;
  int split = 1;
  while (split < 8 && 2 * split <= p.kbs && tiles * 2 * split <= sms) split *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles * split));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = Few<BT>::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)split;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fp8_matmul_few<BT, TILE, OT>, mx, mw, p, tn, split) ==
                 cudaSuccess
             ? KDN_OK
             : KDN_ERR_CUDA;
}

template <bool TILE, typename OT>
kdn_status mm_go(const void* x, int64_t ldx, const void* w, int64_t ldw, int K, const Prm& p,
                 int dev, int sms, cudaStream_t s) {
  if (p.M <= 16) return few_go<16, TILE, OT>(x, ldx, w, ldw, K, p, dev, sms, s);
  if (p.M <= 32) return few_go<32, TILE, OT>(x, ldx, w, ldw, K, p, dev, sms, s);
  const int64_t rows = (p.M + 127) / 128;
  if (p.M <= 64 || rows * ((p.N + 127) / 128) * 2 <= sms)
    return few_go<64, TILE, OT>(x, ldx, w, ldw, K, p, dev, sms, s);
  // as many tiles as SMs or more: the wide tile (each byte of x feeds twice
  // the columns); fewer: the narrow one, so that more SMs work
  if (rows * ((p.N + 255) / 256) * 4 > (int64_t)sms * 3)
    return wide_go<256, TILE, OT>(x, ldx, w, ldw, K, p, dev, sms, s);
  return wide_go<128, TILE, OT>(x, ldx, w, ldw, K, p, dev, sms, s);
}

}  // namespace

kdn_status fp8_matmul_launch(const void* x, int64_t ldx, const float* sx, const void* w,
                             int64_t ldw, const float* sw, bool tile, void* out, kdn_dtype ot,
                             int M, int N, int K, uint32_t* status, cudaStream_t s) {
  int dev = 0;
  static std::atomic<int> sm_count[64];
  if (cudaGetDevice(&dev) != cudaSuccess) return KDN_ERR_CUDA;
  int sms = sm_count[dev & 63].load(std::memory_order_relaxed);
  if (!sms) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return KDN_ERR_CUDA;
    sm_count[dev & 63].store(sms, std::memory_order_relaxed);
  }
  Prm p{sx, sw, out, M, N, (int)(((int64_t)K + kKb - 1) / kKb), 16, status};
  while (p.align > 1 && N % p.align) p.align >>= 1;
  if (reinterpret_cast<uintptr_t>(out) & 31u) {
    const int most = ot == KDN_F32 ? 4 : 8;
    if (p.align > most) p.align = most;
  }
  using bf = __nv_bfloat16;
  if (ot == KDN_F32)
    return tile ? mm_go<true, float>(x, ldx, w, ldw, K, p, dev, sms, s)
                : mm_go<false, float>(x, ldx, w, ldw, K, p, dev, sms, s);
  return tile ? mm_go<true, bf>(x, ldx, w, ldw, K, p, dev, sms, s)
              : mm_go<false, bf>(x, ldx, w, ldw, K, p, dev, sms, s);
}

}  // namespace kdn
