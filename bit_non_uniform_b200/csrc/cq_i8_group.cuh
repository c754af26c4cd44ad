// cq_i8_group.cuh -- the INT8 MoE layer for many routes per expert: the same
// values as the streamed layer's, with the products on the tensor cores.
//
// The streamed layer reads an expert's weights from L2 again for every 16
// routes and multiplies on the legacy tensor path: 1024 tokens of 64 experts
// 7168 x 2048 (128 routes each) took 6.3 ms, here 0.83.  HBM bounds it up to
// 32 routes each (256 tokens: 482 us, the weights alone 436), then the copies
// from L2 into shared memory and tiles that are not full (2048 tokens: 1.29 ms,
// 34% of the tensor rate).  The steps:
//   i8_group_plan_kernel   sorts the routes by expert and lists the tiles (up
//                          to NT routes of one expert);
//   i8_group_rows_kernel   quantizes the sorted rows: a token once per route,
//                          so that a tile's rows lie side by side for one copy
//                          (the copies come out of L2);
//   i8_group_kernel        one tile of 128 weight rows x NT routes per CTA,
//                          twice: gate/up with SwiGLU to h (in sorted order),
//                          then, on the codes of h, down to each route's y;
// and the weighted sum is i8_combine_kernel's.  Where the grid ends depends on
// the routes, so that it covers the most tiles there can be; the CTAs past the
// list's end leave at once.
//
// The order of an expert's routes comes from atomics, and no value depends on
// it: a row's codes and sums are its own, and integer.
#pragma once

#include "cq_i8_tc.cuh"

namespace cq {

constexpr int kGpPlanThreads = 1024;
constexpr int kGpRowThreads = 256;
constexpr int kGpRowKeep = 4;              // groups of 8 values kept per thread

struct I8GroupParams {
  const uint16_t* tokens;   // bf16 [T][H]
  const int32_t* ids;       // [T][k]
  const float* wscale;      // the stage's
  float* h;                 // [R][I], sorted
  float* y;                 // [R][H], by route
  int8_t* xq;               // [R][K] codes of the stage's sorted rows
  float* sx;                // [R] RN(absmax / 127)
  int* route;               // [R] the sorted routes, the dropped ones last
  int4* tile;               // expert, first sorted row, rows
  int* n;                   // tiles, routes that are not dropped
  int k, R, E, H, I;
  int nt;
  int n_rt, nkb;            // row tiles, blocks of K
  int clear_y;
  int withhold;             // test hook: the first stage waits for an arrival that never comes
  uint64_t timeout_ns;
};

__global__ void __launch_bounds__(kGpPlanThreads)
    i8_group_plan_kernel(const __grid_constant__ I8GroupParams p) {
  extern __shared__ int s_at[];            // [E] routes, then the next place
  __shared__ int s_sum[2][32];
  __shared__ int s_dropped;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_wait();
  griddep_launch_dependents();
  for (int e = tid; e < p.E; e += kGpPlanThreads) s_at[e] = 0;
  __syncthreads();
  for (int r = tid; r < p.R; r += kGpPlanThreads) {
    const int id = p.ids[r];
    if (id >= 0 && id < p.E) atomicAdd(&s_at[id], 1);
  }
  __syncthreads();
  const int per = (p.E + kGpPlanThreads - 1) / kGpPlanThreads;
  const int e0 = min(tid * per, p.E), e1 = min(e0 + per, p.E);
  int routes = 0, tiles = 0;
  for (int e = e0; e < e1; ++e) {
    routes += s_at[e];
    tiles += (s_at[e] + p.nt - 1) / p.nt;
  }
  const int ir = warp_inclusive_sum(routes), it = warp_inclusive_sum(tiles);
  if (lane == 31) {
    s_sum[0][warp] = ir;
    s_sum[1][warp] = it;
  }
  __syncthreads();
  int row = ir - routes, tile = it - tiles;
  for (int w = 0; w < warp; ++w) {
    row += s_sum[0][w];
    tile += s_sum[1][w];
  }
  if (tid == kGpPlanThreads - 1) {
    p.n[0] = tile + tiles;
    p.n[1] = row + routes;
    s_dropped = row + routes;
  }
  for (int e = e0; e < e1; ++e) {
    const int cnt = s_at[e];
    s_at[e] = row;
    for (int j = 0; j < cnt; j += p.nt)
      p.tile[tile++] = make_int4(e, row + j, min(p.nt, cnt - j), 0);
    row += cnt;
  }
  __syncthreads();
  for (int r = tid; r < p.R; r += kGpPlanThreads) {
    const int id = p.ids[r];
    p.route[atomicAdd(id >= 0 && id < p.E ? &s_at[id] : &s_dropped, 1)] = r;
  }
}

// Codes and scale of one sorted row, with the decisions of i8_stage_rows.  For
// the second product also zeros the y of a dropped route, if the caller sees it.
template <bool DOWN>
__global__ void __launch_bounds__(kGpRowThreads)
    i8_group_rows_kernel(const __grid_constant__ I8GroupParams p) {
  constexpr int SRC = DOWN ? I8_SRC_F32 : I8_SRC_BF16;
  __shared__ uint32_t red[kGpRowThreads / 32];
  const int row = static_cast<int>(blockIdx.x), tid = threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  const int route = p.route[row];
  if (row >= p.n[1]) {
    if (DOWN && p.clear_y)
      for (int i = tid; i < p.H; i += kGpRowThreads)
        p.y[static_cast<int64_t>(route) * p.H + i] = 0.f;
    return;
  }
  const int K = DOWN ? p.I : p.H, nv = K / 8;
  const void* src = DOWN ? static_cast<const void*>(p.h + static_cast<int64_t>(row) * K)
                         : p.tokens + static_cast<int64_t>(route / p.k) * K;
  uint2* const out = reinterpret_cast<uint2*>(p.xq + static_cast<int64_t>(row) * K);
  auto larger = [](float m, float x) {
    if constexpr (DOWN)
      return __uint_as_float(max(__float_as_uint(m), __float_as_uint(x) & 0x7FFFFFFFu));
    else
      return fmaxf(m, fabsf(x));
  };
  float keep[kGpRowKeep][8];
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < kGpRowKeep; ++i) {
    const int v = tid + i * kGpRowThreads;
    if (v < nv) {
      i8_load8<SRC>(src, static_cast<int64_t>(v) * 8, keep[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) mx = larger(mx, keep[i][j]);
    }
  }
  for (int v = tid + kGpRowKeep * kGpRowThreads; v < nv; v += kGpRowThreads) {
    float x[8];
    i8_load8<SRC>(src, static_cast<int64_t>(v) * 8, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) mx = larger(mx, x[j]);
  }
  const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(mx));
  if ((tid & 31) == 0) red[tid >> 5] = m;
  __syncthreads();
  uint32_t mb = red[0];
#pragma unroll
  for (int w = 1; w < kGpRowThreads / 32; ++w) mb = max(mb, red[w]);
  mx = __uint_as_float(mb);
  const float inv = mx > 0.f ? __fdiv_rn(127.0f, mx) : 0.f;
  auto put = [&](int v, const float (&x)[8]) {
    out[v] = make_uint2(i8_code4(x[0], x[1], x[2], x[3], inv),
                        i8_code4(x[4], x[5], x[6], x[7], inv));
  };
#pragma unroll
  for (int i = 0; i < kGpRowKeep; ++i) {
    const int v = tid + i * kGpRowThreads;
    if (v < nv) put(v, keep[i]);
  }
  for (int v = tid + kGpRowKeep * kGpRowThreads; v < nv; v += kGpRowThreads) {
    float x[8];
    i8_load8<SRC>(src, static_cast<int64_t>(v) * 8, x);
    put(v, x);
  }
  if (tid == 0) p.sx[row] = __fdiv_rn(mx, 127.0f);
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int32_t c0,
                                            int32_t c1, int32_t c2, int32_t c3, int32_t c4,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
      : "memory");
}

// Two or three CTAs share an SM, so that one's epilogue runs beside the
// others' products: with tiles of 64 routes 482 us with three, 504 with two
// (256 tokens, 64 experts 7168 x 2048, top 8).
template <int NT>
struct I8GroupCfg {
  static constexpr int CTAS = NT == 64 ? 3 : 2;
  static constexpr int A_BYTES = kRows * kTcBlock;
  static constexpr int STAGE = A_BYTES + NT * kTcBlock;
  static constexpr int MISC = 1024 + NT * 8;                   // barriers, scales, routes
  static constexpr int STAGES = ((CTAS == 3 ? 75 : 112) * 1024 - 1024 - MISC) / STAGE;
  static constexpr int SMEM = 1024 + STAGES * STAGE + MISC;
  static_assert(STAGES >= 3 && STAGE % 1024 == 0 && 16 * STAGES + 24 <= 1024, "shared memory");
  static_assert((NT == 64 || NT == 128) && CTAS * NT <= kTmemCols, "TMEM columns");
};

template <int NT, bool DOWN>
__global__ void __launch_bounds__(kTcThreads, I8GroupCfg<NT>::CTAS)
    i8_group_kernel(const __grid_constant__ I8GroupParams p,
                    const __grid_constant__ CUtensorMap xmap,
                    const __grid_constant__ CUtensorMap wmap) {
  using C = I8GroupCfg<NT>;
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
  int* const s_route = reinterpret_cast<int*>(s_sx + NT);                       // [NT]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = static_cast<int>(blockIdx.x) / p.n_rt;
  const int rt = static_cast<int>(blockIdx.x) - t * p.n_rt;
  griddep_wait();
  if (t >= p.n[0]) return;                 // the whole CTA
  const int4 tile = p.tile[t];
  const int rt0 = rt * (DOWN ? kRows : kRows / 2);             // first output column
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

  if (warp == kTcProducer) {
    if (lane == 0) {
      int st = 0, loads = 0;
      uint32_t round = 0;
      for (int kb = 0; kb < p.nkb; ++kb) {
        if (!wait_phase(bar_empty + 8 * st, (round & 1u) ^ 1u, abort_flag, tmo, SITE_I8_EMPTY))
          break;
        const uint32_t bar = bar_full + 8 * st, dst = base + st * C::STAGE;
        mbar_arrive_expect_tx(bar, C::STAGE);
        if constexpr (DOWN)
          tma_load_3d(dst, &wmap, kb * kTcBlock, rt0, tile.x, bar);
        else
          tma_load_5d(dst, &wmap, kb * kTcBlock, 0, 0, rt0 / 8, tile.x, bar);
        tma_load_2d(dst + C::A_BYTES, &xmap, kb * kTcBlock, tile.y, bar);
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
      const uint32_t idesc = idesc_s8_s32(kRows, NT);
      int st = 0;
      uint32_t round = 0, acc = 0;
      for (int kb = 0; kb < p.nkb; ++kb) {
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
    // TMEM lane `row`; of the 16-column chunks the one half of the warps
    // takes the even, the other the odd ones
    const int row = (warp & 3) * 32 + lane, half = warp >> 2;
    const int cols = DOWN ? p.H : p.I;
    const int col = rt0 + (DOWN ? row : (row >> 4) * 8 + (lane & 7));
    const bool live = col < cols;
    const int hi = (lane >> 3) & 1;        // gate/up: an up row
    const float* const ws = p.wscale + static_cast<int64_t>(tile.x) * (DOWN ? cols : 2 * cols);
    const float w = live ? ws[!DOWN && hi ? cols + col : col] : 0.f;
    for (int c = tid; c < NT; c += kTcEpilogue) {
      s_sx[c] = c < tile.z ? p.sx[tile.y + c] : 0.f;
      if constexpr (DOWN) s_route[c] = c < tile.z ? p.route[tile.y + c] : 0;
    }
    bool ok = i8_wait_warp(bar_dfull, 0, abort_flag, tmo, SITE_I8_DFULL);
    ok = tc_epilogue_vote(ok) && *abort_flag == 0;             // also orders s_sx, s_route
    tc_fence_after();
    const uint32_t daddr = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const float other_w = DOWN ? 0.f : __shfl_xor_sync(0xffffffffu, w, 8);
    for (int c0 = half * 16; c0 < tile.z; c0 += 32) {
      uint32_t r[16];
      tmem_ld16(daddr + c0, r);
      tmem_wait_ld();
      const int left = ok && live ? tile.z - c0 : 0;           // columns to store
      if constexpr (DOWN) {
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          if (q < left)
            p.y[static_cast<int64_t>(s_route[c0 + q]) * cols + col] = __fmul_rn(
                __fmul_rn(s_sx[c0 + q], w), static_cast<float>(static_cast<int>(r[q])));
        }
      } else {
        // of two columns the gate lanes take the first, the up lanes the second
#pragma unroll
        for (int q = 0; q < 16; q += 2) {
          const int own = static_cast<int>(hi ? r[q + 1] : r[q]);
          const int other = __shfl_xor_sync(0xffffffffu, static_cast<int>(hi ? r[q] : r[q + 1]), 8);
          if (q + hi < left) {
            const double sx = s_sx[c0 + q + hi];
            const double a = sx * w * own, b = sx * other_w * other;
            const double gv = hi ? b : a, uv = hi ? a : b;
            p.h[static_cast<int64_t>(tile.y + c0 + q + hi) * cols + col] =
                static_cast<float>(gv / (1.0 + exp(-gv)) * uv);
          }
        }
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
}

}  // namespace cq
