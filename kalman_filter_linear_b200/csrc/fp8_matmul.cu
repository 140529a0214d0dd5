// kdn_fp8_matmul: out[m, n] = sum over k of x[m, k] w[n, k], both factors in
// e4m3 with an fp32 scale for each block of 128 along k (x: per row; w: per
// 128 x 128 tile, or per row):
//   out[m, n] = sum_b sx[m, b] sw[n or n/128, b] (sum_{k in block b} x8 w8).
// The inner sum runs on the tensor cores (tcgen05 kind::f8f6f4, fp32 in TMEM);
// products of e4m3 numbers are exact in fp32.  The scales change with every
// block, so each block's product leaves TMEM and is scaled and added in fp32
// registers while the tensor cores work on the next block (two TMEM buffers).
//
// fp8_matmul_wide: 256 x BN outputs a tile, by the CTAs of a pair: each has 128
// rows of x and half of w's rows in its shared memory, and one MMA
// (cta_group::2) runs on both, which loads a third less than tiles of one CTA
// (128 x 256 each took 139 us for 32768 x 2048 x 2048, the pairs 132).
// A CTA's warp 0 copies (TMA, 128-byte swizzle), warp 1 of the pair's first CTA
// issues the MMAs, warps 2 and 3 bring the scales, eight blocks at a time and
// turned so that a block's scales are consecutive, warps 4-11 scale and add:
// four warps cover the 128 rows (TMEM lanes), each group half the columns.
// Scaled sums leave through shared memory in bulk copies.
//
// 32768 x 2048 x 2048 takes 136 us (2.0 PFLOP/s; 157 at the 1.5 GHz that the power
// limit leaves after a second of such work), 2048 x 2048 x 32749 with a scale for
// each row of w 209.  Of 130 us in the same run, the loop without scaling took 87;
// with the hand-over of TMEM 96, with its reads still 96, with the multiply-adds
// 125: a warp's own chain of read, scale, add and release bounds it.  Handing TMEM over in parts of 128 columns
// (145), sixteen scaling warps (143) and 128-column tiles with four accumulators
// (152) were no faster.
//
// fp8_matmul_few: for few rows of x the bytes of w are what counts.  w is the
// 128-row operand and up to 64 rows of x are the columns; the blocks of k are
// split over a cluster of up to eight CTAs so that every SM streams w, and the
// parts meet through distributed shared memory, added in rank order.  8 x 2048 x
// 2048 takes 5.8 us, 8 x 8192 x 8192 16 (4.2 TB/s; 12 where w is still in L2).
//
// Every wait is bounded; one that gives up sets the status word.
#include <atomic>

#include "cluster.cuh"
#include "enqueue.h"
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
// 16 lanes x 64 columns: with g = lane / 4 and c = 2 (lane % 4), registers 4 j
// and 4 j + 1 are row g, columns 8 j + c and 8 j + c + 1, the next two row g + 8
__device__ __forceinline__ void tmem_ld_rows16(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32"
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

// the address of `p` in CTA `rank`'s shared memory
__device__ __forceinline__ uint32_t at_rank(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
// An arrival on another CTA's barrier after reads of TMEM (which the tcgen05
// fences order).  No ordinary memory is handed over: a release at cluster scope
// would wait for all of the warp's accesses, a microsecond each time.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// the pair's forms of the calls above; a load signals a barrier of either CTA
__device__ __forceinline__ void umma_f8_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tma_load_pair(uint32_t smem_dst, const void* tmap, uint32_t bar,
                                              int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_dst),
      "l"(tmap), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
// arrives on this barrier of both CTAs when the MMAs so far have finished
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* smem_result, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n\t"
               "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::"r"(
                   smem_u32(smem_result)),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}

// whether a phase is complete, without a wait
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

struct Prm {
  const float *sx, *sw;
  void* out;
  int M, N, kbs;         // rows of x, rows of w, blocks along k
  bool bulk_out;         // out's rows are 16-byte pieces: bulk copies store them
  uint32_t* status;      // or null
  uint32_t skip;         // for tests: the first block's copies that are left out, or ~0
};

// ------------------------------------------------------------------- wide
constexpr int kScaleBlocks = 8;  // blocks along k whose scales come together

template <int BN>
struct Wide {
  static constexpr uint32_t A = 128 * kKb, B = BN / 2 * kKb, STAGE = A + B;
  static constexpr int STAGES = BN == 256 ? 4 : 5;
  static constexpr int BUFS = 512 / BN;  // blocks' products in TMEM
  // scales: two stages of [block][128 rows of x | BN rows or 2 tiles of w]
  static constexpr uint32_t SCV = 128 + BN;
  static constexpr uint32_t OFF_SC = STAGES * STAGE, SC = kScaleBlocks * SCV * 4;
  static constexpr uint32_t OFF_OUT = OFF_SC + 2 * SC;  // per warp: twice 32 rows of 128 bytes of out
  static constexpr uint32_t OFF_BAR = OFF_OUT + 8 * 8192;
  static constexpr uint32_t NBAR = 2 * STAGES + 2 * BUFS + 4;
  static constexpr uint32_t OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr uint32_t SMEM = OFF_MISC + 16 + 1024;  // 1024: alignment
  static_assert(SMEM <= 232448 && OFF_OUT % 1024 == 0, "shared memory plan");
};

template <int BN, bool TILE, typename OT>
__global__ void __launch_bounds__(384, 1)
fp8_matmul_wide(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                const __grid_constant__ CUtensorMap mo, Prm p, int tiles_n, int tiles) {
  using W = Wide<BN>;
  constexpr int S = W::STAGES, BUFS = W::BUFS;
  extern __shared__ uint8_t wsm_raw[];
  uint8_t* sm = wsm_raw + ((1024u - (smem_u32(wsm_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + W::OFF_BAR);  // the first CTA's: both CTAs' bytes
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + BUFS;  // the first CTA's: both CTAs' warps
  uint64_t* sc_full = tempty + BUFS;
  uint64_t* sc_empty = sc_full + 2;
  uint32_t* misc = reinterpret_cast<uint32_t*>(sm + W::OFF_MISC);
  float* scales = reinterpret_cast<float*>(sm + W::OFF_SC);
  volatile uint32_t* abort_flag = misc + 1;
  auto fail = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_try_wait(bar, parity)) return false;
    if (*abort_flag) return true;
    if (mbar_wait(bar, parity)) return false;
    *abort_flag = 1u;
    if (p.status) atomicOr(p.status, DEV_TIMEOUT);
    return true;
  };
  auto warp_fail = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return false;
    return __any_sync(0xffffffffu, fail(bar, parity));
  };
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < BUFS; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 16);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sc_full[i], 2);
      mbar_init(&sc_empty[i], 8);
    }
    misc[1] = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&mx);
    tma_prefetch_desc(&mw);
  }
  __syncthreads();
  cluster_sync_all();
  if (warp == 2) tmem_alloc_pair(misc, 512);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && lane == 0) {
      // copies
      uint32_t it = 0;
      const uint32_t skip = blockIdx.x == 0 ? p.skip : ~0u;
      bool bad = false;
      for (int tile = pair; tile < tiles && !bad; tile += pairs) {
        const int m0 = tile / tiles_n * 256 + (int)rank * 128;
        const int n0 = tile % tiles_n * BN + (int)rank * (BN / 2);
        for (int kb = 0; kb < p.kbs; ++kb, ++it) {
          const uint32_t st = it % S;
          if (it >= (uint32_t)S && fail(&empty[st], ((it / S) - 1u) & 1u)) { bad = true; break; }
          if (rank == 0) mbar_expect_tx(&full[st], 2 * W::STAGE);
          if (it == skip) continue;
          const uint32_t bar = at_rank(&full[st], 0);
          tma_load_pair(sbase + st * W::STAGE, &mx, bar, kb * (int)kKb, m0);
          tma_load_pair(sbase + st * W::STAGE + W::A, &mw, bar, kb * (int)kKb, n0);
        }
      }
      // all copies have landed and been read, and no arrival is under way,
      // when the CTAs go (bounded)
      for (uint32_t i = it > (uint32_t)S ? it - S : 0; i < it; ++i)
        if (!mbar_wait(&empty[i % S], (i / S) & 1u)) break;
    } else if (warp == 1 && rank == 0) {
      // MMAs, by an elected thread of a warp that stays together
      constexpr uint32_t ID = umma_idesc_e4m3(256, BN);
      const uint64_t desc0 = umma_desc_sw128(sbase, 16, 1024);
      uint32_t it = 0, st = 0, st_phase = 0, buf = 0, buf_phase = 1;
      bool bad = false;
      for (int tile = pair; tile < tiles && !bad; tile += pairs) {
        for (int kb = 0; kb < p.kbs; ++kb, ++it) {
          if (warp_fail(&full[st], st_phase)) { bad = true; break; }
          const uint64_t da = desc0 + (uint64_t)(st * (W::STAGE / 16)), db = da + W::A / 16;
          if (it >= (uint32_t)BUFS && warp_fail(&tempty[buf], buf_phase)) { bad = true; break; }
          if (elect_one()) {
            tc_fence_after();
#pragma unroll
            for (uint32_t ks = 0; ks < 4; ++ks)  // (32 bytes along k, in units of 16)
              umma_f8_pair(tmem + buf * BN, da + 2u * ks, db + 2u * ks, ID, ks > 0);
            umma_commit_pair(&tfull[buf]);
            umma_commit_pair(&empty[st]);
          }
          __syncwarp();
          if (++st == (uint32_t)S) {
            st = 0;
            st_phase ^= 1u;
          }
          if (++buf == (uint32_t)BUFS) {
            buf = 0;
            buf_phase ^= 1u;
          }
        }
      }
      // nothing may be in flight when TMEM is freed: the last blocks' commits
      // (bounded)
      if (lane == 0)
        for (uint32_t i = it >= (uint32_t)BUFS ? it - BUFS : 0; i < it; ++i)
          mbar_wait(&tfull[i % BUFS], (i / BUFS) & 1u);
    } else if (warp >= 2) {
      // scales
      const int t = tid - 64;
      uint32_t g = 0;
      bool bad = false;
      for (int tile = pair; tile < tiles && !bad; tile += pairs) {
        const int m0 = tile / tiles_n * 256 + (int)rank * 128, n0 = tile % tiles_n * BN;
        for (int k0 = 0; k0 < p.kbs; k0 += kScaleBlocks, ++g) {
          // three vectors (of 64 at a time) are loaded before their place is free
          constexpr int NV = (128 + (TILE ? 0 : BN)) / 64, AHEAD = NV < 3 ? NV : 3;
          const int nk = min(kScaleBlocks, p.kbs - k0);
          float x[AHEAD][kScaleBlocks], tile_scale = 0.f;
          auto load = [&](int i, float (&to)[kScaleBlocks]) {
            const int v = t + 64 * i;
            const float* from = i < 2 ? p.sx + (size_t)min(m0 + v, p.M - 1) * p.kbs + k0
                                      : p.sw + (size_t)min(n0 + v - 128, p.N - 1) * p.kbs + k0;
#pragma unroll
            for (int k = 0; k < kScaleBlocks; ++k) to[k] = __ldg(from + min(k, nk - 1));
          };
#pragma unroll
          for (int i = 0; i < AHEAD; ++i) load(i, x[i]);
          const int tk = t % kScaleBlocks, th = t / kScaleBlocks;
          if (TILE && th < 2)
            tile_scale = __ldg(p.sw + (size_t)(min(n0 + 128 * th, p.N - 1) >> 7) * p.kbs + k0 +
                               min(tk, nk - 1));
          if (g >= 2 && warp_fail(&sc_empty[g & 1u], ((g >> 1) - 1u) & 1u)) { bad = true; break; }
          float* to = scales + (g & 1u) * (W::SC / 4);
#pragma unroll
          for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int k = 0; k < kScaleBlocks; ++k) to[k * W::SCV + t + 64 * i] = x[i % AHEAD][k];
            if (i + AHEAD < NV) load(i + AHEAD, x[i % AHEAD]);
          }
          if (TILE && th < 2) to[tk * W::SCV + 128 + th] = tile_scale;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_full[g & 1u]);
        }
      }
    }
  } else {
    // scale and add
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    constexpr int CW = BN / 2;  // columns of a thread
    const int h = (warp - 4) >> 2;
    const int q = warp & 3;     // TMEM lane quarter
    const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(h * CW);
    const int gr = lane >> 2, gc = 2 * (lane & 3);
    uint8_t* stage_out = sm + W::OFF_OUT + (warp - 4) * 8192;
    const uint32_t tempty_first = at_rank(tempty, 0);
    // 64 columns are read in two chunks; the next chunk, the next block's first
    // one included, is on its way while one is added.
    // TILE (one scale a row for all columns): a thread has a row, a chunk is 32
    // columns.  Else a thread has the rows gr + 8 i and the columns 8 j + gc and
    // the next, a chunk is 16 rows, and a block's column scales are few loads
    // from shared memory.
    constexpr int CHUNKS = CW / 32;
    uint32_t r[2][32];
    auto read = [&](uint32_t buf, int c) {
      const uint32_t from = tl + buf * BN + 64 * (c >> 1);
      if constexpr (TILE) tmem_ld_async(from + 32 * (c & 1), r[c & 1]);
      else tmem_ld_rows16(from + ((uint32_t)(16 * (c & 1)) << 16), r[c & 1]);
    };
    uint32_t g = 0, buf = 0, phase = 0;
    // Outputs leave by two places in turn, over tiles too: an odd number of pieces
    // (128 columns in bf16: one a warp) begins a tile where the last one ended.
    uint32_t pieces = 0;
    bool bad = false;
    for (int tile = pair; tile < tiles && !bad; tile += pairs) {
      const int mw0 = tile / tiles_n * 256 + (int)rank * 128 + 32 * q;
      const int n0 = tile % tiles_n * BN + h * CW;
      float2 acc[CHUNKS][16];  // [chunk][column pair], or [chunk][2 j + row / 8 of the chunk's]
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[c][j] = make_float2(0.f, 0.f);
      if (warp_fail(&tfull[buf], phase)) break;
      tc_fence_after();
      read(buf, 0);
      const float* sc = nullptr;
      for (int kb = 0, k = 0; kb < p.kbs; ++kb) {
        if (k == 0) {
          if (warp_fail(&sc_full[g & 1u], (g >> 1) & 1u)) {
            tmem_ld_wait(r[0]);  // (nothing may arrive in registers that are used again)
            bad = true;
            break;
          }
          sc = scales + (g & 1u) * (W::SC / 4);
        }
        float s[TILE ? 1 : 4];
        if constexpr (TILE) {
          s[0] = sc[32 * q + lane] * sc[128 + (h * CW >> 7)];
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) s[i] = sc[32 * q + gr + 8 * i];
        }
        const float* cs = sc + 128 + h * CW + gc;
        const uint32_t nbuf = buf + 1 == (uint32_t)BUFS ? 0 : buf + 1;
        const uint32_t nphase = nbuf == 0 ? phase ^ 1u : phase;
        bool ready = false;  // the next block, asked for ahead
        float2 w[8];
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
          if (!TILE && (c & 1) == 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              w[j] = *reinterpret_cast<const float2*>(cs + 64 * (c >> 1) + 8 * j);
          }
          tmem_ld_wait(r[c & 1]);
          if (c + 1 < CHUNKS) {
            read(buf, c + 1);
            if (c + 2 == CHUNKS && kb + 1 < p.kbs) ready = mbar_test_wait(&tfull[nbuf], nphase);
          } else {
            // this warp has read the buffer
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty_first + 8u * buf);
            if (kb + 1 < p.kbs) {
              if (!__all_sync(0xffffffffu, ready) && warp_fail(&tfull[nbuf], nphase)) {
                bad = true;
                break;
              }
              tc_fence_after();
              read(nbuf, 0);
            }
          }
          if constexpr (TILE) {
            const float2 ss = make_float2(s[0], s[0]);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              acc[c][i] = __ffma2_rn(as_f2(r[c & 1][2 * i], r[c & 1][2 * i + 1]), ss, acc[c][i]);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float x = s[2 * (c & 1) + (i & 1)];
              acc[c][i] = __ffma2_rn(__fmul2_rn(as_f2(r[c & 1][2 * i], r[c & 1][2 * i + 1]), w[i >> 1]),
                                     make_float2(x, x), acc[c][i]);
            }
          }
        }
        if (bad) break;
        buf = nbuf;
        phase = nphase;
        sc += W::SCV;
        if (++k == kScaleBlocks || kb == p.kbs - 1) {
          // this warp has used the scales
          k = 0;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_empty[g & 1u]);
          ++g;
        }
      }
      if (bad) break;
      // element pair i of chunk c is at (row, col) of the warp's outputs
      auto row_of = [&](int c, int i) { return TILE ? lane : 16 * (c & 1) + 8 * (i & 1) + gr; };
      auto col_of = [&](int c, int i) {
        return 64 * (c >> 1) + (TILE ? 32 * (c & 1) + 2 * i : 8 * (i >> 1) + gc);
      };
      {
        // 32 rows of 128 bytes through shared memory (16-byte pieces XORed with
        // the row, as the copy's 128-byte swizzle has them), stored by a bulk
        // copy while the next tile begins.  Rows that a bulk copy cannot start at
        // are stored by the warp, one after another: a thread's own stores from
        // its registers are one element of 32 rows each (5695 x 923 x 1316 97 us,
        // so 22).
        constexpr int ES = (int)sizeof(OT), PC = 128 / ES;  // columns of a piece
        constexpr int PER = TILE ? 8 / ES : 1;              // pairs that one store takes
#pragma unroll
        for (int piece = 0; piece < CW / PC; ++piece, ++pieces) {
          // (the copy before the last one has left its place)
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          __syncwarp();
          uint8_t* place = stage_out + (CW / PC % 2 ? pieces & 1u : piece & 1) * 4096;
#pragma unroll
          for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
            for (int i = 0; i < 16; i += PER) {
              // (whole pairs i are in one piece: known when compiled)
              const int first = 64 * (c >> 1) + (TILE ? 32 * (c & 1) + 2 * i : 8 * (i >> 1));
              if (first / PC != piece) continue;
              const int row = row_of(c, i), byte = (col_of(c, i) - PC * piece) * ES;
              uint8_t* to = place + row * 128 + (((byte >> 4) ^ (row & 7)) << 4) + (byte & 15);
              const float2* v = &acc[c][i];
              if constexpr (ES == 2) {
                uint32_t u[PER];
#pragma unroll
                for (int e = 0; e < PER; ++e) {
                  const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[e].x, v[e].y);
                  u[e] = *reinterpret_cast<const uint32_t*>(&b2);
                }
                if constexpr (PER == 4)
                  *reinterpret_cast<uint4*>(to) = make_uint4(u[0], u[1], u[2], u[3]);
                else
                  *reinterpret_cast<uint32_t*>(to) = u[0];
              } else if constexpr (PER == 2) {
                *reinterpret_cast<float4*>(to) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
              } else {
                *reinterpret_cast<float2*>(to) = v[0];
              }
            }
          if (!p.bulk_out) {
            __syncwarp();
            OT* out = static_cast<OT*>(p.out);
            for (int row = 0; row < 32 && mw0 + row < p.M; ++row) {
              OT* o = out + (size_t)(mw0 + row) * p.N + n0 + PC * piece;
#pragma unroll
              for (int e = lane; e < PC; e += 32) {
                const int byte = e * ES;
                const uint8_t* from = place + row * 128 + (((byte >> 4) ^ (row & 7)) << 4) + (byte & 15);
                if (n0 + PC * piece + e < p.N) o[e] = *reinterpret_cast<const OT*>(from);
              }
            }
            __syncwarp();
            continue;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            // (a group for each piece, empty for one outside of out)
            if (mw0 < p.M && n0 + PC * piece < p.N)
              asm volatile(
                  "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::
                      "l"(&mo),
                  "r"(smem_u32(place)), "r"(n0 + PC * piece), "r"(mw0)
                  : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
  __syncwarp();
  cluster_sync_all();
}

// -------------------------------------------------------------------- few
// BT: columns of a tile (rows of x), 16, 32 or 64
template <int BT>
struct Few {
  static constexpr uint32_t A = 128 * kKb, B = BT * kKb, STAGE = A + B;
  static constexpr int STAGES = 4;  // (two CTAs an SM, or eight-CTA clusters would queue)
  static constexpr uint32_t OFF_SC = STAGES * STAGE;      // per warp: [2][BT] scales
  static constexpr uint32_t OFF_BAR = OFF_SC + 4 * 2 * BT * 4;
  static constexpr uint32_t NBAR = 2 * STAGES + 4;
  static constexpr uint32_t OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr uint32_t SMEM = OFF_MISC + 16 + 1024;
  static constexpr uint32_t COLS = 2 * BT;                 // 32, 64 or 128
  static_assert(SMEM <= 232448 && 128u * BT * 4 <= STAGES * STAGE, "shared memory plan");
};

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
    const uint32_t skip = blockIdx.x == 0 ? p.skip : ~0u;
    int it = 0;
    for (; it < nk; ++it) {
      const int st = it % S;
      if (it >= S && fail(&empty[st], (uint32_t)((it / S) - 1) & 1u)) break;
      mbar_expect_tx(&full[st], F::STAGE);
      if ((uint32_t)it == skip) continue;
      tma_load_2d(sbase + st * F::STAGE, &mw, &full[st], (k0 + it) * (int)kKb, n0);
      tma_load_2d(sbase + st * F::STAGE + F::A, &mx, &full[st], (k0 + it) * (int)kKb, m0);
    }
    // copies in flight land before their place is used again, whatever became of
    // the other warps (bounded)
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
// [rows, K] bytes, rows ld bytes apart, boxes of 128 bytes x box rows; what
// lies outside reads as zero.
bool mm_map(CUtensorMap* m, const void* base, int rows, int K, int64_t ld, int box) {
  auto enc = tensor_map_encoder();
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

// out [M, N], boxes of 32 rows x 128 bytes
bool mm_out_map(CUtensorMap* m, void* out, int M, int N, size_t es) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)M};
  cuuint64_t strides[1] = {(cuuint64_t)N * es};
  cuuint32_t boxes[2] = {(cuuint32_t)(128 / es), 32u};
  cuuint32_t estr[2] = {1u, 1u};
  return enc(m, es == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, out,
             dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
kdn_status wide_go(const void* x, int64_t ldx, const void* w, int64_t ldw, int K, const Prm& prm,
                   int dev, int sms, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  CUtensorMap mx, mw, mo{};
  Prm p = prm;
  p.bulk_out = (int64_t)p.N * (int64_t)sizeof(OT) % 16 == 0;
  if (p.bulk_out && !mm_out_map(&mo, p.out, p.M, p.N, sizeof(OT))) return KDN_ERR_CUDA;
  if (!mm_map(&mx, x, p.M, K, ldx, 128) || !mm_map(&mw, w, p.N, K, ldw, BN / 2) ||
      !allow_smem(fp8_matmul_wide<BN, TILE, OT>, (int)Wide<BN>::SMEM, dev, ready))
    return KDN_ERR_CUDA;
  const int tn = (p.N + BN - 1) / BN;
  const int64_t tiles = (int64_t)((p.M + 255) / 256) * tn;
  const int pairs = (int)(tiles < sms / 2 ? tiles : sms / 2);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(384);
  cfg.dynamicSmemBytes = Wide<BN>::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return enqueued(
      cudaLaunchKernelEx(&cfg, fp8_matmul_wide<BN, TILE, OT>, mx, mw, mo, p, tn, (int)tiles));
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
  // Blocks along k of a CTA are halved while its SM would else idle, or while
  // many remain (8 x 8192 x 8192 17.3 us at two CTAs, 12.5 at four), not below
  // two, or four for 64 rows, whose sums cost more to join (64 x 2048 x 2048
  // 7.9 us at four CTAs, 11.5 at eight).
  auto more = [&](int to) {
    return p.kbs >= (BT == 64 ? 4 : 2) * to &&
           (tiles * to <= sms || (tiles * to <= 2 * sms && p.kbs >= 16 * to));
  };
  while (split < 8 && more(2 * split)) split *= 2;
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
  return enqueued(cudaLaunchKernelEx(&cfg, fp8_matmul_few<BT, TILE, OT>, mx, mw, p, tn, split));
}

template <bool TILE, typename OT>
kdn_status mm_go(const void* x, int64_t ldx, const void* w, int64_t ldw, int K, const Prm& p,
                 int dev, int sms, cudaStream_t s) {
  if (p.M <= 16) return few_go<16, TILE, OT>(x, ldx, w, ldw, K, p, dev, sms, s);
  if (p.M <= 32) return few_go<32, TILE, OT>(x, ldx, w, ldw, K, p, dev, sms, s);
  // Where four CTAs can share each tile of 64 rows, k is split; else the pairs'
  // tiles: 128 x 2048 x 2048 (rows, columns, k) 7.9 and 9.7 us, 256 x 512 x 8192
  // 16.5 and 22.6; 256 x 2048 x 2048 11.4 and 9.9, 100 x 8192 x 2048 12.2 and 10.0.
  const int64_t rows = (p.M + 63) / 64;
  if (rows * ((p.N + 127) / 128) * 4 <= sms)
    return few_go<64, TILE, OT>(x, ldx, w, ldw, K, p, dev, sms, s);
  // The wide tile feeds twice the columns from each byte of x; the narrow one
  // puts more SMs to work where there are few: 1200 x 2048 x 2048 13.2 (wide) and
  // 15.0 us, 800 x 2048 x 2048 13.0 and 10.4.
  const int64_t tall = (p.M + 255) / 256;
  if (tall * ((p.N + 127) / 128) > sms / 2)
    return wide_go<256, TILE, OT>(x, ldx, w, ldw, K, p, dev, sms, s);
  return wide_go<128, TILE, OT>(x, ldx, w, ldw, K, p, dev, sms, s);
}

}  // namespace

kdn_status fp8_matmul_launch(const void* x, int64_t ldx, const float* sx, const void* w,
                             int64_t ldw, const float* sw, bool tile, void* out, kdn_dtype ot,
                             int M, int N, int K, uint32_t* status, cudaStream_t s, uint32_t skip) {
  int dev = 0;
  static std::atomic<int> sm_count[64];
  if (cudaGetDevice(&dev) != cudaSuccess) return KDN_ERR_CUDA;
  int sms = sm_count[dev & 63].load(std::memory_order_relaxed);
  if (!sms) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return KDN_ERR_CUDA;
    sm_count[dev & 63].store(sms, std::memory_order_relaxed);
  }
  Prm p{sx, sw, out, M, N, (int)(((int64_t)K + kKb - 1) / kKb), false, status, skip};
  using bf = __nv_bfloat16;
  if (ot == KDN_F32)
    return tile ? mm_go<true, float>(x, ldx, w, ldw, K, p, dev, sms, s)
                : mm_go<false, float>(x, ldx, w, ldw, K, p, dev, sms, s);
  return tile ? mm_go<true, bf>(x, ldx, w, ldw, K, p, dev, sms, s)
              : mm_go<false, bf>(x, ldx, w, ldw, K, p, dev, sms, s);
}

}  // namespace kdn
