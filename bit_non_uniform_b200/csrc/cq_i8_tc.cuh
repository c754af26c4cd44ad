// cq_i8_tc.cuh -- INT8 weights times INT8 activations on the tensor cores
// (tcgen05.mma kind::i8), for more tokens than the streamed product takes.
//
// Operand A is 128 weight rows per CTA, operand B the tokens.  Both come from
// shared memory, K-major with the 128-byte swizzle, loaded by TMA in blocks
// of 128 bytes of K; the INT32 accumulators live in tensor memory.
// Two kernels, chosen by a cost estimate on the host:
//   * i8_split_kernel: one tile of 128 rows x NT tokens per cluster, K split
//     over the cluster's CTAs (1 to 8).  For few tokens or few tiles: weights are
//     read by all SMs although there are fewer tiles than SMs, and the INT32
//     parts are summed through distributed shared memory, each CTA finishing
//     its share of the columns: 13 us at 32 tokens of 6144 x 7168, 17 at 128,
//     against 7 us of HBM time.  (A first version split the K blocks of the
//     persistent kernel over the CTAs and summed partial tiles from global
//     memory: 59 us at 128 tokens, the last CTA of a tile reading its parts.)
//   * i8_pair_kernel: persistent CTA pairs, 256 weight rows x NT tokens per
//     tile (cta_group::2): each CTA loads its 128 weight rows and half of the
//     tokens, which halves the activation traffic and the shared-memory reads
//     per MMA.  Two accumulators, so that a tile's epilogue overlaps the next
//     tile's MMAs.  4096 tokens of 6144 x 7168 take 124 to 134 us (2.7 to 2.9
//     POP/s at 1.65 GHz), the tensor pipe busy in 83% of the active cycles; the
//     rest waits for operands, of which an SM takes in about 50 bytes a cycle.
//
// With SwiGLU a CTA's rows are 8 gate rows, the 8 up rows that belong to
// them, the next 8 gate rows, and so on, so that gate and up of one output
// sit in the same warp of the epilogue, 8 lanes apart.
//
// Warp roles (320 threads): warps 0-7 epilogue (warps w and w + 4 share TMEM
// lanes 32 w .. 32 w + 31, 16 columns each in turn; with four warps the
// epilogue of 128 columns alone took 4 us), warp 8 producer, warp 9 MMA issue
// and TMEM.
#pragma once

#include "cq_a8.cuh"
#include "cq_i8.cuh"

namespace cq {

constexpr int kTcThreads = 320;
constexpr int kTcEpilogue = 256;
constexpr int kTcProducer = 8;
constexpr int kTcMma = 9;
constexpr int kTcBlock = 128;              // bytes of K per stage

enum I8TcSite : int {
  SITE_I8_EMPTY = 50,
  SITE_I8_FULL = 51,
  SITE_I8_DFREE = 52,
  SITE_I8_DFULL = 53,
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Barrier over all threads of the cluster (hardware; every role reaches it).
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of CTA `rank`'s copy of a shared-memory variable.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ int4 ld_cluster_int4(uint32_t cluster_ptr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(cluster_ptr)
               : "memory");
  return v;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
               : "memory");
}

// Tensor copies whose completion counts on an mbarrier of either CTA of the
// pair (`bar` is a cluster address).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int32_t c0,
                                                 int32_t c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, int32_t c0,
                                                 int32_t c1, int32_t c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_load_4d_pair(uint32_t dst, const CUtensorMap* map, int32_t c0,
                                                 int32_t c1, int32_t c2, int32_t c3,
                                                 uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T, kind::i8.
template <int CG>
__device__ __forceinline__ void mma_ss_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive on the barrier (of both CTAs of a pair) when this thread's MMAs are done.
template <int CG>
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  if constexpr (CG == 1)
    mma_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
        ".b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

template <int CG>
__device__ __forceinline__ void tc_alloc(uint32_t slot, uint32_t cols) {
  if constexpr (CG == 1) {
    tmem_alloc(slot, cols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tc_dealloc(uint32_t addr, uint32_t cols) {
  if constexpr (CG == 1)
    tmem_dealloc(addr, cols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
                 : "memory");
}

constexpr int kTcMaxSplit = 8;

struct I8TcParams {
  const float* absmax;      // [M]
  const float* wscale;      // [N]
  void* y;
  int M, N;
  int swiglu, out_bf16;
  int n_rt, n_tt, nkb;      // row tiles, token tiles, K blocks
  int split;                // CTAs per tile (i8_split_kernel)
  int w_boxes;              // SwiGLU: boxes per block of K (1, or 8)
  // i8_pair_kernel: tokens per tile; the first `main_tiles` tiles are whole,
  // each of the others is cut into `cut` parts of tail_nt tokens
  int nt, main_tiles, cut, tail_nt;
  int early_w;              // the weights may be read before griddep_wait
  int withhold;             // test hook: the first stage waits for an arrival that never comes
  uint64_t timeout_ns;
};

// AND-vote and barrier of the epilogue's threads (whole warps).
__device__ __forceinline__ bool tc_epilogue_vote(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 3, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(ok))
      : "memory");
  return r != 0;
}

// A thread's place in a tile of the epilogue.
struct I8Lane {
  int row;                  // TMEM lane
  int half;                 // takes the 16-column chunks of this parity
  int col;                  // output column
  int cols;                 // output columns of y
  int m0, mv;               // first token, valid tokens
  bool live;
  float ws;
};

// `rt0` is the first output column of this CTA's 128 weight rows.
__device__ __forceinline__ I8Lane i8_lane(const I8TcParams& p, int rt0, int m0, int nt) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  I8Lane l;
  l.row = (warp & 3) * 32 + lane;
  l.half = warp >> 2;
  l.cols = p.swiglu ? p.N / 2 : p.N;
  l.m0 = m0;
  l.mv = p.M - m0 < nt ? p.M - m0 : nt;
  l.col = rt0 + (p.swiglu ? (l.row >> 4) * 8 + (lane & 7) : l.row);
  l.live = l.col < l.cols;
  const int wrow = p.swiglu && (lane & 8) ? l.cols + l.col : l.col;
  l.ws = l.live ? p.wscale[wrow] : 0.f;
  return l;
}

template <bool BF16>
__device__ __forceinline__ void i8_put(uint8_t* at, float v) {
  if constexpr (BF16)
    *reinterpret_cast<uint16_t*>(at) = bf16_bits(v);
  else
    *reinterpret_cast<float*>(at) = v;
}

// Scale, SwiGLU and store NQ accumulator columns (tokens m0 + c0 ...) of the
// lane's row; all 32 lanes call it.
template <int NQ, bool BF16>
__device__ __forceinline__ void i8_finish_as(const I8TcParams& p, const I8Lane& l,
                                             const float* s_sx, const int (&a)[NQ], int c0) {
  constexpr int ES = BF16 ? 2 : 4;
  float v[NQ];
#pragma unroll
  for (int q = 0; q < NQ; q += 4) {
    const float4 sx = *reinterpret_cast<const float4*>(s_sx + c0 + q);
    v[q] = __fmul_rn(__fmul_rn(sx.x, l.ws), static_cast<float>(a[q]));
    v[q + 1] = __fmul_rn(__fmul_rn(sx.y, l.ws), static_cast<float>(a[q + 1]));
    v[q + 2] = __fmul_rn(__fmul_rn(sx.z, l.ws), static_cast<float>(a[q + 2]));
    v[q + 3] = __fmul_rn(__fmul_rn(sx.w, l.ws), static_cast<float>(a[q + 3]));
  }
  const int left = l.live ? l.mv - c0 : 0;                  // columns to store
  const int64_t pitch = static_cast<int64_t>(l.cols) * ES;
  uint8_t* at = static_cast<uint8_t*>(p.y) + (l.m0 + c0) * pitch + static_cast<int64_t>(l.col) * ES;
  if (p.swiglu) {
    // lanes 0-7 hold gate and lanes 8-15 up of the same outputs (16-31
    // likewise); of two columns the gate lanes take the first, the up lanes
    // the second
    const int hi = (threadIdx.x >> 3) & 1;
    at += hi * pitch;
#pragma unroll
    for (int q = 0; q < NQ; q += 2) {
      const float other = __shfl_xor_sync(0xffffffffu, hi ? v[q] : v[q + 1], 8);
      const float h = hi ? i8_swiglu_f32(other, v[q + 1]) : i8_swiglu_f32(v[q], other);
      if (q + hi < left) i8_put<BF16>(at, h);
      at += 2 * pitch;
    }
  } else {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      if (q < left) i8_put<BF16>(at, v[q]);
      at += pitch;
    }
  }
}

template <int NQ>
__device__ __forceinline__ void i8_finish(const I8TcParams& p, const I8Lane& l, const float* s_sx,
                                          const int (&a)[NQ], int c0) {
  if (p.out_bf16)
    i8_finish_as<NQ, true>(p, l, s_sx, a, c0);
  else
    i8_finish_as<NQ, false>(p, l, s_sx, a, c0);
}

// The tokens' RN(absmax / 127) of a tile, by the epilogue's threads.
__device__ __forceinline__ void i8_load_scales(const I8TcParams& p, int m0, int mv, int nt,
                                               float* s_sx) {
  for (int c = threadIdx.x; c < nt; c += kTcEpilogue)
    s_sx[c] = c < mv ? __fdiv_rn(p.absmax[m0 + c], 127.0f) : 0.f;
}

// Load this CTA's weight rows of one block of K.  SwiGLU: the tensor map's
// boxes hold 8 gate rows and the 8 up rows of the same outputs; all of them in
// one copy (a fourth dimension counts the groups of 8) where the outputs are a
// multiple of 8, else one copy each (rows past the outputs must read as zero).
template <bool PAIR>
__device__ __forceinline__ void i8_load_w(const I8TcParams& p, uint32_t dst,
                                          const CUtensorMap* map, int k0, int rt0, uint32_t bar) {
  if (!p.swiglu) {
    if constexpr (PAIR) tma_load_2d_pair(dst, map, k0, rt0, bar);
    else tma_load_2d(dst, map, k0, rt0, bar);
  } else if (p.w_boxes == 1) {
    if constexpr (PAIR) tma_load_4d_pair(dst, map, k0, 0, 0, rt0 / 8, bar);
    else tma_load_4d(dst, map, k0, 0, 0, rt0 / 8, bar);
  } else {
    for (int q = 0; q < p.w_boxes; ++q) {
      if constexpr (PAIR) tma_load_3d_pair(dst + q * 2048, map, k0, rt0 + q * 8, 0, bar);
      else tma_load_3d(dst + q * 2048, map, k0, rt0 + q * 8, 0, bar);
    }
  }
}

// ---------------------------------------------------------------------------
// one tile per cluster, K split over its CTAs
// ---------------------------------------------------------------------------
template <int NT>
struct I8SplitCfg {
  static constexpr int A_BYTES = kRows * kTcBlock;
  static constexpr int STAGE = A_BYTES + NT * kTcBlock;
  static constexpr int MISC = 1024 + NT * 4;
  static constexpr int RAW = (220 * 1024 - 1024 - MISC) / STAGE;
  static constexpr int STAGES = RAW > 10 ? 10 : RAW;
  static constexpr int SMEM = 1024 + STAGES * STAGE + MISC;
  static constexpr int DUMP = NT * kRows * 4;                  // the accumulator, over the stages
  static_assert(STAGES >= 4 && DUMP <= STAGES * STAGE && STAGE % 1024 == 0, "shared memory");
  static_assert(NT >= 32 && NT <= 128 && (NT & (NT - 1)) == 0, "TMEM columns");
};

template <int NT>
__global__ void __launch_bounds__(kTcThreads, 1)
    i8_split_kernel(const __grid_constant__ I8TcParams p, const __grid_constant__ CUtensorMap xmap,
                    const __grid_constant__ CUtensorMap wmap) {
  using C = I8SplitCfg<NT>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  const uint32_t misc = base + C::STAGES * C::STAGE;
  const uint32_t bar_full = misc;
  const uint32_t bar_empty = bar_full + 8 * C::STAGES;
  const uint32_t bar_dfull = bar_empty + 8 * C::STAGES;
  const uint32_t slot_tmem = bar_dfull + 8;
  volatile int* const abort_flag =
      reinterpret_cast<volatile int*>(gbase + (slot_tmem + 8 - base));
  float* const s_sx = reinterpret_cast<float*>(gbase + (misc + 1024 - base));   // [NT]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = p.split;
  const int tile = static_cast<int>(blockIdx.x) / S;
  const int part = static_cast<int>(blockIdx.x) - tile * S;   // = rank in the cluster
  const int tt = tile / p.n_rt, rt = tile - tt * p.n_rt;
  const int kb0 = static_cast<int>(static_cast<int64_t>(part) * p.nkb / S);
  const int kb1 = static_cast<int>(static_cast<int64_t>(part + 1) * p.nkb / S);
  const int rt0 = rt * (p.swiglu ? kRows / 2 : kRows);
  const uint64_t tmo = p.timeout_ns;

  if (tid == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(bar_full + 8 * s, s == 0 ? 1 + p.withhold : 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    mbar_init(bar_dfull, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kTcMma) {
    tc_alloc<1>(slot_tmem, NT);
    tc_fence_before();
  }
  if (warp == kTcProducer && lane == 0) {
    prefetch_tensormap(&xmap);
    prefetch_tensormap(&wmap);
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base =
      *reinterpret_cast<volatile uint32_t*>(gbase + (slot_tmem - base));

  bool ok = true;
  I8Lane l = {};
  if (warp == kTcProducer) {
    if (lane == 0) {
      auto load_w = [&](int kb, int st) {
        mbar_arrive_expect_tx(bar_full + 8 * st, C::STAGE);
        i8_load_w<false>(p, base + st * C::STAGE, &wmap, kb * kTcBlock, rt0, bar_full + 8 * st);
      };
      // weights no preceding kernel writes are fetched while it ends
      int early = 0;
      if (p.early_w) {
        for (; early < C::STAGES && kb0 + early < kb1; ++early) load_w(kb0 + early, early);
      }
      griddep_wait();
      int st = 0, loads = 0;
      uint32_t round = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (loads >= early) {
          if (!wait_phase(bar_empty + 8 * st, (round & 1u) ^ 1u, abort_flag, tmo,
                          SITE_I8_EMPTY))
            break;
          load_w(kb, st);
        }
        tma_load_2d(base + st * C::STAGE + C::A_BYTES, &xmap, kb * kTcBlock, tt * NT,
                    bar_full + 8 * st);
        ++loads;
        if (++st == C::STAGES) {
          st = 0;
          ++round;
        }
      }
      if (*abort_flag) {
        // the copies in flight must land before the CTA ends
        const int armed = loads < C::STAGES ? loads : C::STAGES;
        for (int k = 1; k <= armed; ++k) {
          const int idx = loads - k;
          volatile int dummy = 0;
          mbar_wait(bar_full + 8 * (idx % C::STAGES),
                    static_cast<uint32_t>(idx / C::STAGES) & 1u, &dummy, tmo, SITE_TEARDOWN);
        }
      }
    }
    __syncwarp();
  } else if (warp == kTcMma) {
    if (lane == 0) {
      griddep_wait();                       // the bounded waits start after it
      const uint32_t idesc = idesc_s8_s32(kRows, NT);
      int st = 0;
      uint32_t round = 0, acc = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait_phase(bar_full + 8 * st, round & 1u, abort_flag, tmo, SITE_I8_FULL)) break;
        tc_fence_after();
        const uint64_t da = smem_desc_sw128(base + st * C::STAGE);
        const uint64_t db = smem_desc_sw128(base + st * C::STAGE + C::A_BYTES);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          mma_ss_i8<1>(tmem_base, da + 2 * kk, db + 2 * kk, idesc, acc);   // 32 bytes each
          acc = 1;
        }
        tc_commit<1>(bar_empty + 8 * st);
        if (++st == C::STAGES) {
          st = 0;
          ++round;
        }
      }
      tc_commit<1>(bar_dfull);
      volatile int dummy = 0;
      mbar_wait(bar_dfull, 0, &dummy, tmo, SITE_TEARDOWN);
    }
    __syncwarp();
  } else {
    griddep_wait();
    l = i8_lane(p, rt0, tt * NT, NT);
    i8_load_scales(p, l.m0, l.mv, NT, s_sx);
    ok = i8_wait_warp(bar_dfull, 0, abort_flag, tmo, SITE_I8_DFULL);
    ok = tc_epilogue_vote(ok) && *abort_flag == 0;         // also orders s_sx
    tc_fence_after();
    const uint32_t daddr = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    int4* const dump = reinterpret_cast<int4*>(gbase);      // [NT / 4][128]
    for (int cc = l.half; cc * 16 < l.mv; cc += 2) {
      uint32_t r[16];
      tmem_ld16(daddr + cc * 16, r);
      tmem_wait_ld();
      if (S == 1) {
        int a[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) a[q] = static_cast<int>(r[q]);
        if (ok) i8_finish<16>(p, l, s_sx, a, cc * 16);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          dump[(cc * 4 + q) * kRows + l.row] =
              make_int4(static_cast<int>(r[4 * q]), static_cast<int>(r[4 * q + 1]),
                        static_cast<int>(r[4 * q + 2]), static_cast<int>(r[4 * q + 3]));
      }
    }
    tc_fence_before();
  }
  griddep_launch_dependents();
  __syncthreads();
  if (warp == kTcMma) {
    tc_fence_after();
    tc_dealloc<1>(tmem_base, NT);
  }
  if (S > 1) {
    __syncwarp();
    cluster_sync_all();
    if (warp < kTcProducer && ok) {
      // columns in quads, dealt out over the cluster's CTAs
      for (int q = part + S * l.half; q * 4 < l.mv; q += 2 * S) {
        int a[4] = {0, 0, 0, 0};
        const uint32_t at = base + static_cast<uint32_t>(q * kRows + l.row) * 16u;
#pragma unroll
        for (int c = 0; c < kTcMaxSplit; ++c) {
          if (c < S) {
            const int4 v = ld_cluster_int4(cluster_addr(at, c));
            a[0] += v.x;
            a[1] += v.y;
            a[2] += v.z;
            a[3] += v.w;
          }
        }
        i8_finish<4>(p, l, s_sx, a, q * 4);
      }
    }
    cluster_sync_all();                    // nobody leaves while its parts are read
  }
}

// ---------------------------------------------------------------------------
// persistent CTA pairs
// ---------------------------------------------------------------------------
struct I8PairCfg {
  static constexpr int NT = 256;                               // tokens per tile, at most
  static constexpr int A_BYTES = kRows * kTcBlock;             // this CTA's weight rows
  static constexpr int B_BYTES = NT / 2 * kTcBlock;            // this CTA's tokens, at most
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = 6;
  static constexpr int MISC = 1024 + NT * 4;                   // barriers, scales
  static constexpr int SMEM = 1024 + STAGES * STAGE + MISC;
  static_assert(SMEM <= 227 * 1024 && 2 * NT <= kTmemCols, "budgets");
};

// Tile t of the pair kernel.  The last tiles, which would keep only some of
// the pairs busy, may be cut along their tokens: 4096 tokens of 6144 x 7168
// are 384 tiles for 74 pairs, and uncut the sixth round keeps 14 pairs busy.
struct I8Tile {
  int rt, m0, nt;           // row tile, first token, tokens
  bool tail;
};
__device__ __forceinline__ I8Tile i8_tile(const I8TcParams& p, int t) {
  I8Tile i;
  int part = 0, whole = t;
  i.tail = t >= p.main_tiles;
  if (i.tail) {
    const int j = t - p.main_tiles;
    whole = p.main_tiles + j / p.cut;
    part = j % p.cut;
  }
  const int tt = whole / p.n_rt;
  i.rt = whole - tt * p.n_rt;
  i.nt = i.tail ? p.tail_nt : p.nt;
  i.m0 = tt * p.nt + part * p.tail_nt;
  return i;
}

__global__ void __launch_bounds__(kTcThreads, 1)
    i8_pair_kernel(const __grid_constant__ I8TcParams p, const __grid_constant__ CUtensorMap xmap,
                   const __grid_constant__ CUtensorMap xtail,
                   const __grid_constant__ CUtensorMap wmap) {
  using C = I8PairCfg;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  const uint32_t misc = base + C::STAGES * C::STAGE;
  const uint32_t bar_full = misc;                           // the leader's count both CTAs' copies
  const uint32_t bar_empty = bar_full + 8 * C::STAGES;
  const uint32_t bar_dfull = bar_empty + 8 * C::STAGES;     // [2]
  const uint32_t bar_dfree = bar_dfull + 16;                // [2], the leader's
  const uint32_t bar_fin = bar_dfree + 16;
  const uint32_t slot_tmem = bar_fin + 8;
  volatile int* const abort_flag =
      reinterpret_cast<volatile int*>(gbase + (slot_tmem + 8 - base));
  float* const s_sx = reinterpret_cast<float*>(gbase + (misc + 1024 - base));   // [NT]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int unit = static_cast<int>(blockIdx.x) >> 1;
  const int units = static_cast<int>(gridDim.x) >> 1;

  if (tid == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(bar_full + 8 * s, s == 0 ? 1 + p.withhold : 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_dfull + 8 * s, 1);
      mbar_init(bar_dfree + 8 * s, 2 * kTcEpilogue);
    }
    mbar_init(bar_fin, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kTcMma) {
    tc_alloc<2>(slot_tmem, kTmemCols);
    tc_fence_before();
  }
  if (warp == kTcProducer && lane == 0) {
    prefetch_tensormap(&xmap);
    prefetch_tensormap(&xtail);
    prefetch_tensormap(&wmap);
  }
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base =
      *reinterpret_cast<volatile uint32_t*>(gbase + (slot_tmem - base));
  griddep_wait();
  griddep_launch_dependents();

  const int tiles = p.main_tiles + (p.n_rt * p.n_tt - p.main_tiles) * p.cut;
  const uint64_t tmo = p.timeout_ns;
  const int cta_rows = p.swiglu ? 64 : kRows;               // output columns of this CTA's rows

  if (warp == kTcProducer) {
    if (lane == 0) {
      const uint32_t full0 = cluster_addr(bar_full, 0);
      int st = 0, loads = 0;
      uint32_t round = 0;
      bool ok = true;
      for (int t = unit; ok && t < tiles; t += units) {
        const I8Tile tile = i8_tile(p, t);
        const int half = tile.nt / 2, m0 = tile.m0 + rank * half;
        const int w0 = (tile.rt * 2 + rank) * cta_rows;
        const uint32_t bytes = 2u * static_cast<uint32_t>(C::A_BYTES + half * kTcBlock);
        const CUtensorMap* const xm = tile.tail ? &xtail : &xmap;
        for (int kb = 0; kb < p.nkb; ++kb) {
          if (!wait_phase(bar_empty + 8 * st, (round & 1u) ^ 1u, abort_flag, tmo,
                          SITE_I8_EMPTY)) {
            ok = false;
            break;
          }
          const uint32_t a = base + st * C::STAGE;
          const uint32_t bar = full0 + 8 * st;
          if (rank == 0) mbar_arrive_expect_tx(bar_full + 8 * st, bytes);
          i8_load_w<true>(p, a, &wmap, kb * kTcBlock, w0, bar);
          tma_load_2d_pair(a + C::A_BYTES, xm, kb * kTcBlock, m0, bar);
          ++loads;
          if (++st == C::STAGES) {
            st = 0;
            ++round;
          }
        }
      }
      if (*abort_flag) {
        // the copies in flight must land before the CTA ends: the leader sees
        // them on its barriers, the other CTA gives them time
        if (rank == 0) {
          const int armed = loads < C::STAGES ? loads : C::STAGES;
          for (int k = 1; k <= armed; ++k) {
            const int idx = loads - k;
            volatile int dummy = 0;
            mbar_wait(bar_full + 8 * (idx % C::STAGES),
                      static_cast<uint32_t>(idx / C::STAGES) & 1u, &dummy, tmo, SITE_TEARDOWN);
          }
        } else {
          const uint64_t t0 = globaltimer();
          while (globaltimer() - t0 < 1000000ull) {
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == kTcMma) {
    if (lane == 0 && rank == 0) {
      int st = 0;
      uint32_t round = 0, done = 0;
      bool ok = true;
      for (int t = unit; ok && t < tiles; t += units) {
        const uint32_t idesc = idesc_s8_s32(2 * kRows, i8_tile(p, t).nt);
        const uint32_t db = done & 1u;
        if (!wait_phase(bar_dfree + 8 * db, ((done >> 1) & 1u) ^ 1u, abort_flag, tmo,
                        SITE_I8_DFREE))
          break;
        tc_fence_after();
        const uint32_t d = tmem_base + db * C::NT;
        uint32_t acc = 0;
        for (int kb = 0; kb < p.nkb; ++kb) {
          if (!wait_phase(bar_full + 8 * st, round & 1u, abort_flag, tmo, SITE_I8_FULL)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = smem_desc_sw128(base + st * C::STAGE);
          const uint64_t dbs = smem_desc_sw128(base + st * C::STAGE + C::A_BYTES);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            mma_ss_i8<2>(d, da + 2 * kk, dbs + 2 * kk, idesc, acc);        // 32 bytes each
            acc = 1;
          }
          tc_commit<2>(bar_empty + 8 * st);
          if (++st == C::STAGES) {
            st = 0;
            ++round;
          }
        }
        if (!ok) break;
        tc_commit<2>(bar_dfull + 8 * db);
        ++done;
      }
      // the MMAs in flight read both CTAs' shared memory: wait for them
      tc_commit<2>(bar_fin);
      volatile int dummy = 0;
      mbar_wait(bar_fin, 0, &dummy, tmo, SITE_TEARDOWN);
    }
    __syncwarp();
  } else {
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t dfree0 = cluster_addr(bar_dfree, 0);
    uint32_t done = 0;
    for (int t = unit; t < tiles; t += units) {
      const I8Tile tile = i8_tile(p, t);
      const I8Lane l = i8_lane(p, (tile.rt * 2 + rank) * cta_rows, tile.m0, tile.nt);
      i8_load_scales(p, l.m0, l.mv, tile.nt, s_sx);
      const uint32_t db = done & 1u;
      const bool ok = i8_wait_warp(bar_dfull + 8 * db, (done >> 1) & 1u, abort_flag, tmo,
                                   SITE_I8_DFULL);
      if (!tc_epilogue_vote(ok)) break;                     // also orders s_sx
      tc_fence_after();
      const uint32_t daddr = tmem_base + lane_addr + db * C::NT;
      for (int cc = l.half; cc * 16 < l.mv; cc += 2) {
        uint32_t r[16];
        tmem_ld16(daddr + cc * 16, r);
        tmem_wait_ld();
        int a[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) a[q] = static_cast<int>(r[q]);
        i8_finish<16>(p, l, s_sx, a, cc * 16);
      }
      tc_fence_before();
      mbar_arrive_cluster(dfree0 + 8 * db);
      ++done;
      tc_epilogue_vote(true);                               // s_sx is rewritten next
    }
  }

  __syncthreads();
  cluster_sync_all();
  if (warp == kTcMma) {
    tc_fence_after();
    tc_dealloc<2>(tmem_base, kTmemCols);
  }
}

// Per-row INT8 quantization with 16-byte accesses (K a multiple of 8): one
// CTA per row, the row's values kept in registers between the two passes
// while they fit.  The same decisions as quant_rows_kernel.
constexpr int kQvThreads = 128;
constexpr int kQvKeep = 8;                 // 16-byte loads kept per thread

__global__ void __launch_bounds__(kQvThreads)
    quant_rows_vec_kernel(const uint16_t* x, int M, int K, int8_t* xq, float* absmax) {
  __shared__ uint32_t red[kQvThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = blockIdx.x;
  const uint4* xr = reinterpret_cast<const uint4*>(x + row * K);
  uint2* qr = reinterpret_cast<uint2*>(xq + row * K);
  const int nv = K / 8;
  uint4 keep[kQvKeep];
  float mx = 0.f;
  auto top = [&](const uint4& q) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
  };
#pragma unroll
  for (int i = 0; i < kQvKeep; ++i) {
    const int v = threadIdx.x + i * kQvThreads;
    keep[i] = v < nv ? xr[v] : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kQvKeep; ++i) top(keep[i]);
  for (int v = threadIdx.x + kQvKeep * kQvThreads; v < nv; v += kQvThreads) top(xr[v]);
  const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(mx));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  uint32_t mb = red[0];
#pragma unroll
  for (int w = 1; w < kQvThreads / 32; ++w) mb = red[w] > mb ? red[w] : mb;
  mx = __uint_as_float(mb);
  const float inv = mx > 0.f ? __fdiv_rn(127.0f, mx) : 0.f;
  auto code4 = [&](uint32_t a, uint32_t b) {
    return i8_code4(bf16_lo(a), bf16_hi(a), bf16_lo(b), bf16_hi(b), inv);
  };
#pragma unroll
  for (int i = 0; i < kQvKeep; ++i) {
    const int v = threadIdx.x + i * kQvThreads;
    if (v < nv) qr[v] = make_uint2(code4(keep[i].x, keep[i].y), code4(keep[i].z, keep[i].w));
  }
  for (int v = threadIdx.x + kQvKeep * kQvThreads; v < nv; v += kQvThreads) {
    const uint4 q = xr[v];
    qr[v] = make_uint2(code4(q.x, q.y), code4(q.z, q.w));
  }
  if (threadIdx.x == 0) absmax[row] = mx;
}

}  // namespace cq
