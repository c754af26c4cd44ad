// cq_i8_tc.cuh -- INT8 weights times INT8 activations on the tensor cores
// (tcgen05.mma kind::i8), for more tokens than the streamed product takes.
//
// A tile is 128 CG weight rows (the MMA's M) x NT tokens (its N).  Both
// operands come from shared memory, K-major with the 128-byte swizzle, loaded
// by TMA in blocks of 128 bytes of K; the INT32 accumulators live in tensor
// memory, two buffers, so that a tile's epilogue overlaps the next tile's
// MMAs.  With CG = 2 a cluster of two CTAs computes one 256 x NT tile
// (cta_group::2): each CTA loads its 128 weight rows and half of the tokens,
// which halves the activation traffic and the shared-memory reads per MMA.
// The launch's work is the list of (tile, K block) pairs split evenly over
// the CTAs (or pairs); a tile cut by that split is summed from INT32 partial
// tiles by whichever of its CTAs finishes last (integers: the same result in
// any order).
//
// With SwiGLU a CTA's 128 rows are 16 gate rows, the 16 up rows that belong
// to them, the next 16 gate rows, and so on, so that gate and up of one
// output sit in the same warp of the epilogue, 16 lanes apart.
//
// Warp roles (192 threads): warps 0-3 epilogue (TMEM lanes 32 w .. 32 w + 31
// belong to warp w), warp 4 producer, warp 5 MMA issue and TMEM.
#pragma once

#include "cq_i8.cuh"

namespace cq {

constexpr int kTcThreads = 192;
constexpr int kTcProducer = 4;
constexpr int kTcMma = 5;
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

template <int NT, int CG>
struct I8TcCfg {
  static constexpr int A_BYTES = kRows * kTcBlock;             // this CTA's weight rows
  static constexpr int B_ROWS = NT / CG;                       // this CTA's tokens
  static constexpr int B_BYTES = B_ROWS * kTcBlock;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int MISC = 1024 + NT * 4;                   // barriers, scales
  static constexpr int RAW = (220 * 1024 - 1024 - MISC) / STAGE;
  static constexpr int STAGES = RAW > 8 ? 8 : RAW;
  static constexpr int SMEM = 1024 + STAGES * STAGE + MISC;
  static constexpr int TMEM = 2 * NT < 32 ? 32 : 2 * NT;       // two accumulators
  static_assert(STAGES >= 4, "too few stages");
  static_assert(TMEM <= kTmemCols && (TMEM & (TMEM - 1)) == 0, "TMEM columns");
  static_assert(STAGE % 1024 == 0 && B_ROWS % 8 == 0, "swizzle atoms");
};

struct I8TcParams {
  const float* absmax;      // [M]
  const float* wscale;      // [N]
  void* y;
  int* counter;             // [P * CG], zero between launches
  int* partial;             // [2 P CG][NT][128]
  int M, N, K;
  int swiglu, out_bf16;
  int n_rt, n_tt, nkb, P;   // row tiles, token tiles, K blocks, CTAs or pairs
  uint64_t timeout_ns;
};

template <int NT, int CG>
__global__ void __launch_bounds__(kTcThreads, 1)
    i8_tc_kernel(const __grid_constant__ I8TcParams p, const __grid_constant__ CUtensorMap xmap,
                 const __grid_constant__ CUtensorMap wmap) {
  using C = I8TcCfg<NT, CG>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  const uint32_t misc = base + C::STAGES * C::STAGE;
  const uint32_t bar_full = misc;                           // pair: the leader's counts both
  const uint32_t bar_empty = bar_full + 8 * C::STAGES;
  const uint32_t bar_dfull = bar_empty + 8 * C::STAGES;     // [2]
  const uint32_t bar_dfree = bar_dfull + 16;                // [2], the leader's
  const uint32_t bar_fin = bar_dfree + 16;
  const uint32_t slot_tmem = bar_fin + 8;
  volatile int* const abort_flag =
      reinterpret_cast<volatile int*>(gbase + (slot_tmem + 8 - base));
  volatile int* const last_flag =
      reinterpret_cast<volatile int*>(gbase + (slot_tmem + 12 - base));
  float* const s_sx = reinterpret_cast<float*>(gbase + (misc + 1024 - base));   // [NT]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const int unit = CG == 2 ? static_cast<int>(blockIdx.x) >> 1 : static_cast<int>(blockIdx.x);

  if (tid == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_dfull + 8 * s, 1);
      mbar_init(bar_dfree + 8 * s, kEpilogue * CG);
    }
    mbar_init(bar_fin, 1);
    *abort_flag = 0;
    *last_flag = 0;
    fence_mbar_init();
  }
  if (warp == kTcMma) {
    tc_alloc<CG>(slot_tmem, C::TMEM);
    tc_fence_before();
  }
  if (warp == kTcProducer && lane == 0) {
    prefetch_tensormap(&xmap);
    prefetch_tensormap(&wmap);
  }
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base =
      *reinterpret_cast<volatile uint32_t*>(gbase + (slot_tmem - base));
  griddep_wait();
  griddep_launch_dependents();

  const int64_t W = static_cast<int64_t>(p.n_rt) * p.n_tt * p.nkb;
  const int64_t r0 = range_begin(W, p.P, unit);
  const int64_t r1 = range_begin(W, p.P, unit + 1);
  const uint64_t tmo = p.timeout_ns;
  const int hrows = p.swiglu ? p.N / 2 : p.N;               // output columns
  constexpr int SW_ROWS = 64 * CG;                          // outputs of a SwiGLU tile

  if (warp == kTcProducer) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint32_t full0 = CG == 2 ? cluster_addr(bar_full, 0) : bar_full;
      int st = 0, loads = 0;
      uint32_t round = 0;
      bool ok = true;
      for (int64_t x = r0; ok && x < r1;) {
        const Segment sg = segment_at(x, r1, p.nkb);
        const int tt = sg.t / p.n_rt, rt = sg.t - tt * p.n_rt;
        const int m0 = tt * NT + static_cast<int>(rank) * C::B_ROWS;
        const int w0 = p.swiglu ? rt * SW_ROWS + static_cast<int>(rank) * 64
                                : (rt * CG + static_cast<int>(rank)) * kRows;
        for (int kb = sg.s0; kb < sg.s1; ++kb) {
          if (!wait_phase(bar_empty + 8 * st, (round & 1u) ^ 1u, abort_flag, tmo,
                          SITE_I8_EMPTY)) {
            ok = false;
            break;
          }
          const uint32_t a = base + st * C::STAGE, b = a + C::A_BYTES;
          const uint32_t bar = full0 + 8 * st;
          if (rank == 0) mbar_arrive_expect_tx(bar_full + 8 * st, C::STAGE * CG);
          const int k0 = kb * kTcBlock;
          if (p.swiglu) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if constexpr (CG == 2)
                tma_load_3d_pair(a + q * 4096, &wmap, k0, w0 + q * 16, 0, bar);
              else
                tma_load_3d(a + q * 4096, &wmap, k0, w0 + q * 16, 0, bar);
            }
          } else {
            if constexpr (CG == 2)
              tma_load_2d_pair(a, &wmap, k0, w0, bar);
            else
              tma_load_2d(a, &wmap, k0, w0, bar);
          }
          if constexpr (CG == 2)
            tma_load_2d_pair(b, &xmap, k0, m0, bar);
          else
            tma_load_2d(b, &xmap, k0, m0, bar);
          ++loads;
          if (++st == C::STAGES) {
            st = 0;
            ++round;
          }
        }
        x = sg.end;
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
    // ------------------------------------------------------------ MMA issue
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = idesc_s8_s32(kRows * CG, NT);
      int st = 0;
      uint32_t round = 0, tiles = 0;
      bool ok = true;
      for (int64_t x = r0; ok && x < r1;) {
        const Segment sg = segment_at(x, r1, p.nkb);
        const uint32_t db = tiles & 1u;
        if (!wait_phase(bar_dfree + 8 * db, ((tiles >> 1) & 1u) ^ 1u, abort_flag, tmo,
                        SITE_I8_DFREE))
          break;
        tc_fence_after();
        const uint32_t d = tmem_base + db * NT;
        uint32_t acc = 0;
        for (int kb = sg.s0; kb < sg.s1; ++kb) {
          if (!wait_phase(bar_full + 8 * st, round & 1u, abort_flag, tmo, SITE_I8_FULL)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = smem_desc_sw128(base + st * C::STAGE);
          const uint64_t dbs = smem_desc_sw128(base + st * C::STAGE + C::A_BYTES);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            mma_ss_i8<CG>(d, da + 2 * kk, dbs + 2 * kk, idesc, acc);   // 32 bytes = 2 units of 16
            acc = 1;
          }
          tc_commit<CG>(bar_empty + 8 * st);
          if (++st == C::STAGES) {
            st = 0;
            ++round;
          }
        }
        if (!ok) break;
        tc_commit<CG>(bar_dfull + 8 * db);
        ++tiles;
        x = sg.end;
      }
      // the MMAs in flight read both CTAs' shared memory: wait for them
      tc_commit<CG>(bar_fin);
      volatile int dummy = 0;
      mbar_wait(bar_fin, 0, &dummy, tmo, SITE_TEARDOWN);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int i = tid;                                      // TMEM lane
    const uint32_t lane_addr = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t dfree0 = CG == 2 ? cluster_addr(bar_dfree, 0) : bar_dfree;
    const int first_tile = static_cast<int>(r0 / p.nkb);
    const int cta = unit * CG + static_cast<int>(rank);
    uint32_t tiles = 0;
    for (int64_t x = r0; x < r1;) {
      const Segment sg = segment_at(x, r1, p.nkb);
      const int tt = sg.t / p.n_rt, rt = sg.t - tt * p.n_rt;
      const int m0 = tt * NT;
      const int mv = p.M - m0 < NT ? p.M - m0 : NT;
      const int chunks = (mv + 15) >> 4;
      // this lane's weight row, and the output column it stores
      int wrow, col;
      if (p.swiglu) {
        col = rt * SW_ROWS + static_cast<int>(rank) * 64 + warp * 16 + (lane & 15);
        wrow = lane < 16 ? col : hrows + col;
      } else {
        col = wrow = (rt * CG + static_cast<int>(rank)) * kRows + i;
      }
      const bool live = col < hrows;
      const float ws = live ? __ldg(p.wscale + wrow) : 0.f;
      for (int c = i; c < NT; c += kEpilogue)
        s_sx[c] = c < mv ? __fdiv_rn(__ldg(p.absmax + m0 + c), 127.0f) : 0.f;
      const uint32_t db = tiles & 1u;
      const bool ok = wait_phase(bar_dfull + 8 * db, (tiles >> 1) & 1u, abort_flag, tmo,
                                 SITE_I8_DFULL);
      if (!vote_all_epilogue(ok)) break;                    // also orders s_sx
      tc_fence_after();
      const uint32_t daddr = tmem_base + lane_addr + db * NT;
      // scale, SwiGLU and store 16 columns
      auto finish = [&](const int (&a)[16], int c0) {
        float v[16];
#pragma unroll
        for (int q = 0; q < 16; ++q)
          v[q] = __fmul_rn(__fmul_rn(s_sx[c0 + q], ws), static_cast<float>(a[q]));
        if (p.swiglu) {
          // lanes 0-15 hold gate and lanes 16-31 up of the same outputs; of two
          // columns the lower half takes the first and the upper half the second
          const bool hi = lane >= 16;
#pragma unroll
          for (int q = 0; q < 16; q += 2) {
            const float other = __shfl_xor_sync(0xffffffffu, hi ? v[q] : v[q + 1], 16);
            const float h = hi ? i8_swiglu_f32(other, v[q + 1]) : i8_swiglu_f32(v[q], other);
            const int m = c0 + q + (hi ? 1 : 0);
            if (live && m < mv) {
              const int64_t o = static_cast<int64_t>(m0 + m) * hrows + col;
              if (p.out_bf16)
                static_cast<uint16_t*>(p.y)[o] = bf16_bits(h);
              else
                static_cast<float*>(p.y)[o] = h;
            }
          }
        } else if (live) {
          const int64_t o = static_cast<int64_t>(m0 + c0) * hrows + col;
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            if (c0 + q >= mv) break;
            if (p.out_bf16)
              static_cast<uint16_t*>(p.y)[o + static_cast<int64_t>(q) * hrows] = bf16_bits(v[q]);
            else
              static_cast<float*>(p.y)[o + static_cast<int64_t>(q) * hrows] = v[q];
          }
        }
      };
      const bool whole = sg.s0 == 0 && sg.s1 == p.nkb;
      const int slot = 2 * cta + (sg.t == first_tile ? 0 : 1);
      int* const mine = p.partial + static_cast<int64_t>(slot) * NT * kRows;
      for (int cc = 0; cc < chunks; ++cc) {
        uint32_t r[16];
        tmem_ld16(daddr + cc * 16, r);
        tmem_wait_ld();
        int a[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) a[q] = static_cast<int>(r[q]);
        if (whole) {
          finish(a, cc * 16);
        } else {
#pragma unroll
          for (int q = 0; q < 16; ++q)
            if (cc * 16 + q < mv) __stcg(mine + (cc * 16 + q) * kRows + i, a[q]);
        }
      }
      tc_fence_before();
      if constexpr (CG == 2)
        mbar_arrive_cluster(dfree0 + 8 * db);
      else
        mbar_arrive(dfree0 + 8 * db);
      ++tiles;
      if (!whole) {
        __threadfence();
        named_bar_epilogue();
        const int64_t t0 = static_cast<int64_t>(sg.t) * p.nkb;
        const int c_lo = owner_of(W, p.P, t0), c_hi = owner_of(W, p.P, t0 + p.nkb - 1);
        // a unit is the first owner of at most one cut tile: its counter
        int* const cnt = p.counter + c_lo * CG + rank;
        if (i == 0) {
          const int old = atomicAdd(cnt, 1);
          *last_flag = old == c_hi - c_lo;
          if (old == c_hi - c_lo) *cnt = 0;
        }
        named_bar_epilogue();
        if (*last_flag) {
          __threadfence();
          for (int cc = 0; cc < chunks; ++cc) {
            int a[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) a[q] = 0;
            for (int c = c_lo; c <= c_hi; ++c) {
              const int ft = static_cast<int>(range_begin(W, p.P, c) / p.nkb);
              const int sl = 2 * (c * CG + static_cast<int>(rank)) + (sg.t == ft ? 0 : 1);
              const int* src = p.partial + static_cast<int64_t>(sl) * NT * kRows;
#pragma unroll
              for (int q = 0; q < 16; ++q)
                if (cc * 16 + q < mv) a[q] += __ldcg(src + (cc * 16 + q) * kRows + i);
            }
            finish(a, cc * 16);
          }
        }
        named_bar_epilogue();
      } else {
        named_bar_epilogue();                               // s_sx is rewritten next
      }
      x = sg.end;
    }
  }

  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();
  if (warp == kTcMma) {
    tc_fence_after();
    tc_dealloc<CG>(tmem_base, C::TMEM);
  }
}

// Per-row INT8 quantization with 16-byte accesses (K a multiple of 8): one
// CTA per row, the row's values kept in registers between the two passes
// while they fit.  The same decisions as quant_rows_kernel.
constexpr int kQvThreads = 128;
constexpr int kQvKeep = 8;                 // 16-byte loads kept per thread

__global__ void __launch_bounds__(kQvThreads)
    quant_rows_vec_kernel(const uint16_t* __restrict__ x, int M, int K, int8_t* __restrict__ xq,
                          float* __restrict__ absmax) {
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
    return i8_code(bf16_lo(a), inv) | i8_code(bf16_hi(a), inv) << 8 |
           i8_code(bf16_lo(b), inv) << 16 | i8_code(bf16_hi(b), inv) << 24;
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
