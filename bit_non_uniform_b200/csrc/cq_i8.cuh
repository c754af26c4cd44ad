// cq_i8.cuh -- INT8 weights times INT8 activations for a few tokens: the
// product streamed from memory, used by cq_gemm_i8 / cq_linear_i8 at small M
// and by both stages of the INT8 MoE layer.
//
//   xq[m][k]  = RNE(x[m][k] * RN(127 / absmax[m])), saturated to +-127
//   acc[m][n] = sum_k xq[m][k] * wq[n][k]                 (exact, INT32)
//   y[m][n]   = RN(absmax[m] / 127) * wscale[n] * acc[m][n]
//
// With a handful of tokens every weight byte is read once and used a handful
// of times, so HBM bounds the kernel.  The design only serves the stream:
//   * weight bytes go from global memory straight into the registers that
//     mma.sync.m16n8k32 (S8) takes as its A operand, without shared memory or
//     a barrier in between.  A dot product does not depend on the order of k,
//     so a lane's 16 contiguous bytes serve as the k positions of two MMAs
//     (the activations are read from shared memory under the same order);
//   * rows, not tiles, are split evenly over the CTAs (a tile's missing rows
//     are not loaded), and inside a CTA the 256-byte steps of its rows are
//     split evenly over the warps.  INT32 sums do not depend on their order,
//     so the warps add their parts to the CTA's accumulators with
//     shared-memory atomics and the result is the same on every run;
//   * every CTA quantizes the few activation rows itself (no separate launch).
#pragma once

#include "cq_device.cuh"
#include "cq_engine.cuh"

namespace cq {

constexpr int kI8Threads = 512;
constexpr int kI8Warps = kI8Threads / 32;
constexpr int kI8Step = 256;                 // bytes of K per step
constexpr int kI8AccBytes = 32 * 1024;       // accumulators of one pass over the rows
constexpr int kI8MaxTokens = 16;             // tokens of one pass
constexpr int kI8MaxRoutes = 1024;           // routes of one launch of the MoE layer
constexpr int kI8MaxExperts = 16384;
constexpr int kI8CombineRows = 32;           // output columns of one combine block
constexpr int kI8DoneWords = 16;              // 512 output blocks of a pass, at most
constexpr int kI8SmemLimit = 227 * 1024;

// Bytes between two activation rows in shared memory: whole steps, plus 64 so
// that the eight lanes of a 16-byte read phase (two rows x 64 bytes) touch
// all 32 banks.
__host__ __device__ constexpr int i8_row_stride(int64_t K) {
  return static_cast<int>((K + kI8Step - 1) / kI8Step * kI8Step) + 64;
}

// d += A (16 x 32, row) * B (32 x 8, col), S8 x S8 -> S32.
__device__ __forceinline__ void mma_16832_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// One activation code, as quant_rows_kernel decides it (FP32).
__device__ __forceinline__ uint32_t i8_code(float v, float inv) {
  float r = rintf(__fmul_rn(v, inv));
  r = r > 127.f ? 127.f : (r < -127.f ? -127.f : r);
  return static_cast<uint32_t>(static_cast<int>(r)) & 0xFFu;
}

enum I8Source : int { I8_SRC_BF16 = 0, I8_SRC_F32 = 1, I8_SRC_CODES = 2 };

// Where the rows of a pass come from: row j of the pass is row rows[j] /
// `div` of `base` (rows == null: row j).
struct I8Rows {
  const void* base;
  const float* absmax;     // I8_SRC_CODES: the rows' maxima
  const int* rows;         // shared memory, or null
  int div;
};

// Eight values of a row as FP32.
template <int SRC>
__device__ __forceinline__ void i8_load8(const void* row, int64_t k, float (&v)[8]) {
  if constexpr (SRC == I8_SRC_BF16) {
    const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + k);
    v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x);
    v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
    v[4] = bf16_lo(q.z); v[5] = bf16_hi(q.z);
    v[6] = bf16_lo(q.w); v[7] = bf16_hi(q.w);
  } else {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(row) + k);
    const float4 a = f[0], b = f[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

// Quantize (or copy) `cnt` rows of K elements into shared memory, with each
// row's RN(absmax / 127) in s_scale.  The whole CTA takes part; ends with a
// barrier.  K is a multiple of 16.
template <int SRC>
__device__ __forceinline__ void i8_stage_rows(const I8Rows& src, int cnt, int K, int8_t* xs,
                                              int stride, uint32_t* s_max, float* s_scale) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int ES = SRC == I8_SRC_BF16 ? 2 : (SRC == I8_SRC_F32 ? 4 : 1);
  auto row_ptr = [&](int j) {
    const int r = src.rows ? src.rows[j] / src.div : j;
    return static_cast<const uint8_t*>(src.base) + static_cast<int64_t>(r) * K * ES;
  };
  if constexpr (SRC == I8_SRC_CODES) {
    const int nv = K / 16;
    for (int i = threadIdx.x; i < cnt * nv; i += kI8Threads) {
      const int j = i / nv, v = i - j * nv;
      *reinterpret_cast<uint4*>(xs + j * stride + v * 16) =
          *reinterpret_cast<const uint4*>(row_ptr(j) + v * 16);
    }
    if (threadIdx.x < cnt) s_scale[threadIdx.x] = __fdiv_rn(src.absmax[threadIdx.x], 127.0f);
    __syncthreads();
  } else {
    if (threadIdx.x < kI8MaxTokens) s_max[threadIdx.x] = 0u;
    __syncthreads();
    // each row is shared by `parts` warps
    const int parts = cnt >= kI8Warps ? 1 : kI8Warps / cnt;
    const int nv = K / 8;
    for (int j = warp / parts; j < cnt; j += kI8Warps / parts) {
      const uint8_t* row = row_ptr(j);
      float mx = 0.f;
      for (int v = (warp % parts) * 32 + lane; v < nv; v += parts * 32) {
        float x[8];
        i8_load8<SRC>(row, static_cast<int64_t>(v) * 8, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(x[i]));
      }
      const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(mx));
      if (lane == 0) atomicMax(&s_max[j], m);
    }
    __syncthreads();
    for (int j = warp / parts; j < cnt; j += kI8Warps / parts) {
      const uint8_t* row = row_ptr(j);
      const float mx = __uint_as_float(s_max[j]);
      const float inv = mx > 0.f ? __fdiv_rn(127.0f, mx) : 0.f;
      for (int v = (warp % parts) * 32 + lane; v < nv; v += parts * 32) {
        float x[8];
        i8_load8<SRC>(row, static_cast<int64_t>(v) * 8, x);
        uint2 q;
        q.x = i8_code(x[0], inv) | i8_code(x[1], inv) << 8 | i8_code(x[2], inv) << 16 |
              i8_code(x[3], inv) << 24;
        q.y = i8_code(x[4], inv) | i8_code(x[5], inv) << 8 | i8_code(x[6], inv) << 16 |
              i8_code(x[7], inv) << 24;
        *reinterpret_cast<uint2*>(xs + j * stride + v * 8) = q;
      }
      if (lane == 0 && warp % parts == 0) s_scale[j] = __fdiv_rn(mx, 127.0f);
    }
    __syncthreads();
  }
}

// The rows one pass of a CTA multiplies: `nr` row indices from `wa`.  A tile
// is 16 MMA rows: rows 8 t .. 8 t + 7 of `wa` and the same rows of `wb`
// (paired: gate and up), or 16 consecutive rows of `wa` (wb == null).
struct I8Pass {
  const int8_t* wa;
  const int8_t* wb;
  int nr;
};

// The multiplication of one pass.  begin() issues the warp's first loads, so
// that they are in flight while the CTA stages activations or finishes the
// pass before; run() adds the products of the pass's rows with the `cnt`
// staged activation rows to acc[tile][16][cnt] (zero on entry, complete after
// a barrier).
template <int NB>
struct I8Stream {
  const int8_t *wa, *wb;    // wb == null: not paired
  int nr, K, nk;
  int steps;                // 256-byte steps of this warp
  int tile, kb;             // the next step to multiply
  int lt, lk;               // the step loaded last
  const int8_t *pa, *pb;    // this lane's two rows of tile lt, null past the last row
  uint4 a0[4], w0[4];

  __device__ __forceinline__ void set_tile() {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int ra = lt * (wb ? 8 : 16) + g;
    const int rb = wb ? ra : ra + 8;
    const int8_t* base_b = wb ? wb : wa;
    pa = ra < nr ? wa + static_cast<int64_t>(ra) * K + t * 16 : nullptr;
    pb = rb < nr ? base_b + static_cast<int64_t>(rb) * K + t * 16 : nullptr;
  }
  __device__ __forceinline__ void load(uint4 (&a)[4], uint4 (&b)[4]) const {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k = lk * kI8Step + s * 64;
      const bool in = k + t * 16 < K;
      a[s] = in && pa ? ldg_stream16(pa + k) : make_uint4(0, 0, 0, 0);
      b[s] = in && pb ? ldg_stream16(pb + k) : make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void advance() {
    if (++lk == nk) {
      lk = 0;
      ++lt;
      set_tile();
    }
  }

  __device__ __forceinline__ void begin(const I8Pass& ps, int K_) {
    const int warp = threadIdx.x >> 5;
    wa = ps.wa;
    wb = ps.wb;
    nr = ps.nr;
    K = K_;
    nk = (K + kI8Step - 1) / kI8Step;
    const int rpt = wb ? 8 : 16;
    const int total = (nr + rpt - 1) / rpt * nk;
    const int b0 = static_cast<int>(static_cast<int64_t>(warp) * total / kI8Warps);
    const int b1 = static_cast<int>(static_cast<int64_t>(warp + 1) * total / kI8Warps);
    steps = b1 - b0;
    if (steps == 0) return;
    lt = tile = b0 / nk;
    lk = kb = b0 - tile * nk;
    set_tile();
    load(a0, w0);
  }

  __device__ __forceinline__ void run(int cnt, const int8_t* xs, int stride, int* acc) {
    if (steps == 0) return;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    int d[NB][4];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) d[n][i] = 0;
    auto flush = [&]() {
      int* at = acc + tile * 16 * cnt;
#pragma unroll
      for (int n = 0; n < NB; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col = n * 8 + 2 * t + (i & 1);
          if (col < cnt) atomicAdd(at + (g + 8 * (i >> 1)) * cnt + col, d[n][i]);
          d[n][i] = 0;
        }
      }
    };
    const bool has0 = g < cnt, has1 = NB > 1 && g + 8 < cnt;
    const int8_t* x0 = xs + g * stride + t * 16;
    const int8_t* x1 = xs + (g + 8) * stride + t * 16;
    // multiply the step (tile, kb) and move on
    auto compute = [&](const uint4 (&a)[4], const uint4 (&b)[4]) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int k = kb * kI8Step + s * 64;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (has0) x = *reinterpret_cast<const uint4*>(x0 + k);
        mma_16832_s8(d[0], a[s].x, b[s].x, a[s].y, b[s].y, x.x, x.y);
        mma_16832_s8(d[0], a[s].z, b[s].z, a[s].w, b[s].w, x.z, x.w);
        if constexpr (NB > 1) {
          if (cnt > 8) {
            uint4 z = make_uint4(0, 0, 0, 0);
            if (has1) z = *reinterpret_cast<const uint4*>(x1 + k);
            mma_16832_s8(d[1], a[s].x, b[s].x, a[s].y, b[s].y, z.x, z.y);
            mma_16832_s8(d[1], a[s].z, b[s].z, a[s].w, b[s].w, z.z, z.w);
          }
        }
      }
      if (++kb == nk) {
        flush();
        kb = 0;
        ++tile;
      }
    };
    // two register buffers: the next step's loads are in flight while this
    // one is multiplied
    uint4 a1[4], w1[4];
    for (int b = 0; b < steps; b += 2) {
      const bool two = b + 1 < steps;
      if (two) {
        advance();
        load(a1, w1);
      }
      compute(a0, w0);
      if (b + 2 < steps) {
        advance();
        load(a0, w0);
      }
      if (two) compute(a1, w1);
    }
    if (kb != 0) flush();
  }
};

// silu(g) * u with silu(g) = g / (1 + exp(-g)), in FP32.
__device__ __forceinline__ float i8_swiglu_f32(float g, float u) {
  return g / (1.0f + expf(-g)) * u;
}

// ---------------------------------------------------------------------------
// the product for at most 16 tokens
// ---------------------------------------------------------------------------
struct I8LinearParams {
  const void* x;            // bf16 [M][K], or the codes int8 [M][K]
  const float* absmax;      // with codes
  const int8_t* w;          // [N][K]
  const float* wscale;      // [N]
  void* y;
  int M, N, K;
  int swiglu, out_bf16;
  int stride;               // i8_row_stride(K)
  int acc_off;              // bytes of the staged rows
};

template <int SRC, int NB>
__global__ void __launch_bounds__(kI8Threads, 1)
    i8_linear_kernel(const __grid_constant__ I8LinearParams p) {
  extern __shared__ __align__(128) uint8_t i8_smem[];
  __shared__ uint32_t s_max[kI8MaxTokens];
  __shared__ float s_scale[kI8MaxTokens];
  int8_t* const xs = reinterpret_cast<int8_t*>(i8_smem);
  int* const acc = reinterpret_cast<int*>(i8_smem + p.acc_off);
  const int tid = threadIdx.x;
  const int rows = p.swiglu ? p.N / 2 : p.N;
  const int r0 = static_cast<int>(static_cast<int64_t>(blockIdx.x) * rows / gridDim.x);
  const int r1 = static_cast<int>(static_cast<int64_t>(blockIdx.x + 1) * rows / gridDim.x);
  griddep_wait();
  griddep_launch_dependents();
  if (r0 >= r1) return;
  const int rpt = p.swiglu ? 8 : 16;
  const int per_pass = kI8AccBytes / (64 * p.M) * rpt;      // rows whose accumulators fit
  auto pass_at = [&](int a) {
    I8Pass ps;
    ps.nr = r1 - a < per_pass ? r1 - a : per_pass;
    ps.wa = p.w + static_cast<int64_t>(a) * p.K;
    ps.wb = p.swiglu ? ps.wa + static_cast<int64_t>(rows) * p.K : nullptr;
    return ps;
  };
  I8Pass ps = pass_at(r0);
  I8Stream<NB> stream;
  stream.begin(ps, p.K);
  I8Rows src;
  src.base = p.x;
  src.absmax = p.absmax;
  src.rows = nullptr;
  src.div = 1;
  i8_stage_rows<SRC>(src, p.M, p.K, xs, p.stride, s_max, s_scale);
  for (int a = r0; a < r1;) {
    const int tiles = (ps.nr + rpt - 1) / rpt;
    for (int i = tid; i < tiles * 16 * p.M; i += kI8Threads) acc[i] = 0;
    __syncthreads();
    stream.run(p.M, xs, p.stride, acc);
    const int nr = ps.nr;
    if (a + nr < r1) {
      ps = pass_at(a + nr);
      stream.begin(ps, p.K);
    }
    __syncthreads();
    for (int i = tid; i < nr * p.M; i += kI8Threads) {
      const int m = i / nr, r = i - m * nr;
      const int at = (p.swiglu ? (r >> 3) * 16 + (r & 7) : r) * p.M + m;
      const float sx = s_scale[m];
      float v = __fmul_rn(__fmul_rn(sx, p.wscale[a + r]), static_cast<float>(acc[at]));
      if (p.swiglu) {
        const float u = __fmul_rn(__fmul_rn(sx, p.wscale[rows + a + r]),
                                  static_cast<float>(acc[at + 8 * p.M]));
        v = i8_swiglu_f32(v, u);
      }
      const int64_t o = static_cast<int64_t>(m) * rows + a + r;
      if (p.out_bf16)
        static_cast<uint16_t*>(p.y)[o] = bf16_bits(v);
      else
        static_cast<float*>(p.y)[o] = v;
    }
    __syncthreads();
    a += nr;
  }
}

// ---------------------------------------------------------------------------
// the MoE layer for a few tokens: two launches
// ---------------------------------------------------------------------------
// Both launches read the routes themselves: the experts in use (ascending),
// each with its routes, cut into chunks of at most `nt` routes.  A chunk
// multiplies every row of its expert, so the work is chunks x rows, split
// evenly over the CTAs.
//   gate/up: xq = codes of the chunk's tokens; g, u per (row, route);
//            h[route][row] = RN32(silu(g) u) with g, u and silu in FP64, so
//            that the codes of the second quantization are those of any other
//            FP64 evaluation (a value next to a rounding border would
//            otherwise fall on either side of it);
//   down:    hq = codes of the chunk's h rows; y[route][row], then the
//            weighted sum over a token's routes by the CTA that completes a
//            block of output columns (counted by rows), in the order of the
//            token's routes: no atomics on floats, the same result every run.
struct I8MoeParams {
  const uint16_t* tokens;   // bf16 [T][H]
  const int32_t* ids;       // [T][k]
  const float* topk_w;      // [T][k]
  const int8_t* w;          // the stage's weights: [E][2I][H] or [E][H][I]
  const float* wscale;      // [E][2I] or [E][H]
  float* h;                 // [R][I]
  float* y;                 // [R][H]
  void* out;                // [T][H], or null
  int* done;                // [blocks of output columns], zero between calls
  int T, k, R, E;
  int64_t H, I;
  int nt;                   // routes per chunk
  int out_bf16, clear_y;
  int stride, acc_off;
};

// Shared-memory arrays of the plan.
struct I8PlanSmem {
  uint32_t bits[kI8MaxExperts / 32];       // experts in use
  int pref[kI8MaxExperts / 32 + 1];        // experts in use before each word
  int expert[kI8MaxRoutes];                // the experts in use, ascending
  int cnt[kI8MaxRoutes];                   // their routes
  int off[kI8MaxRoutes + 1];               // first route of each in `route`
  int chunk[kI8MaxRoutes + 1];             // chunks before each
  int route[kI8MaxRoutes];                 // routes by expert
  int16_t dense[kI8MaxRoutes];             // each route's expert, as an index into `expert`
  int16_t rank[kI8MaxRoutes];              // its place among the expert's routes
  int part[kI8Warps + 1];
  int n_experts, n_chunks;
};

// Exclusive prefix over v[0..n) (n <= kI8MaxRoutes) into out[0..n], whole CTA.
template <typename F>
__device__ __forceinline__ void i8_prefix(int n, int* out, int* part, F value) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int PER = kI8MaxRoutes / kI8Threads;
  int v[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = threadIdx.x * PER + i;
    v[i] = at < n ? value(at) : 0;
    sum += v[i];
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  int run = inc - sum;
  for (int w = 0; w < warp; ++w) run += part[w];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = threadIdx.x * PER + i;
    if (at < n) out[at] = run;
    run += v[i];
    if (at == n - 1) out[n] = run;
  }
  if (n == 0 && threadIdx.x == 0) out[0] = 0;
  __syncthreads();
}

// The plan of at most 32 routes, by the first warp (experts in the order of
// their first route; the order only decides which CTA works on what).
__device__ __forceinline__ void i8_plan_small(const I8MoeParams& p, I8PlanSmem& s) {
  const int lane = threadIdx.x;
  if (lane < 32) {
    int id = lane < p.R ? __ldg(p.ids + lane) : -1;
    if (id < 0 || id >= p.E) id = -1;
    const unsigned same = __match_any_sync(0xffffffffu, id);
    const unsigned below = (1u << lane) - 1u;
    const bool first = id >= 0 && (same & below) == 0;
    const unsigned firsts = __ballot_sync(0xffffffffu, first);
    const int cnt = first ? __popc(same) : 0, chunks = (cnt + p.nt - 1) / p.nt;
    int off = cnt, ch = chunks;                  // inclusive prefixes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, off, o), v = __shfl_up_sync(0xffffffffu, ch, o);
      if (lane >= o) {
        off += u;
        ch += v;
      }
    }
    const int leader = __ffs(same) - 1;
    const int base = __shfl_sync(0xffffffffu, off - cnt, leader);
    const int d = __popc(firsts & ((1u << leader) - 1u));
    if (first) {
      s.expert[d] = id;
      s.off[d] = off - cnt;
      s.chunk[d] = ch - chunks;
    }
    s.dense[lane] = static_cast<int16_t>(id >= 0 ? d : -1);
    if (id >= 0) s.route[base + __popc(same & below)] = lane;
    if (lane == 31) {
      const int ne = __popc(firsts);
      s.n_experts = ne;
      s.n_chunks = ch;
      s.off[ne] = off;
      s.chunk[ne] = ch;
    }
  }
  __syncthreads();
}

__device__ __forceinline__ void i8_plan(const I8MoeParams& p, I8PlanSmem& s) {
  if (p.R <= 32) {
    i8_plan_small(p, s);
    return;
  }
  const int tid = threadIdx.x;
  const int words = (p.E + 31) / 32;
  constexpr int PER = kI8MaxRoutes / kI8Threads;
  for (int i = tid; i < words; i += kI8Threads) s.bits[i] = 0u;
  for (int i = tid; i < kI8MaxRoutes; i += kI8Threads) s.cnt[i] = 0;
  __syncthreads();
  int id[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int r = tid + i * kI8Threads;
    id[i] = r < p.R ? __ldg(p.ids + r) : -1;
    if (id[i] >= p.E) id[i] = -1;
    if (id[i] >= 0) atomicOr(&s.bits[id[i] >> 5], 1u << (id[i] & 31));
  }
  __syncthreads();
  i8_prefix(words, s.pref, s.part, [&](int i) { return __popc(s.bits[i]); });
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    int d = -1;
    if (id[i] >= 0) {
      const int w = id[i] >> 5;
      d = s.pref[w] + __popc(s.bits[w] & ((1u << (id[i] & 31)) - 1u));
      s.expert[d] = id[i];
    }
    s.dense[tid + i * kI8Threads] = static_cast<int16_t>(d);
  }
  if (tid == 0) s.n_experts = s.pref[words];
  __syncthreads();
  // each route's place among its expert's routes, in route order: every CTA
  // of both launches has to cut an expert's routes into the same chunks
  if (tid < 32) {
    for (int r0 = 0; r0 < p.R; r0 += 32) {
      const int d = s.dense[r0 + tid];
      const unsigned same = __match_any_sync(0xffffffffu, d);
      const int before = __popc(same & ((1u << tid) - 1u));
      const int base = d >= 0 ? s.cnt[d] : 0;
      __syncwarp();
      if (d >= 0 && before == 0) s.cnt[d] = base + __popc(same);
      s.rank[r0 + tid] = static_cast<int16_t>(base + before);
      __syncwarp();
    }
  }
  __syncthreads();
  const int ne = s.n_experts;
  i8_prefix(ne, s.off, s.part, [&](int i) { return s.cnt[i]; });
  i8_prefix(ne, s.chunk, s.part, [&](int i) { return (s.cnt[i] + p.nt - 1) / p.nt; });
  for (int r = tid; r < p.R; r += kI8Threads) {
    const int d = s.dense[r];
    if (d >= 0) s.route[s.off[d] + s.rank[r]] = r;
  }
  if (tid == 0) s.n_chunks = s.chunk[ne];
  __syncthreads();
}

template <bool DOWN, int NB>
__global__ void __launch_bounds__(kI8Threads, 1)
    i8_moe_kernel(const __grid_constant__ I8MoeParams p) {
  extern __shared__ __align__(128) uint8_t i8_smem[];
  __shared__ I8PlanSmem s;
  __shared__ uint32_t s_max[kI8MaxTokens];
  __shared__ float s_scale[kI8MaxTokens];
  __shared__ uint32_t s_done[kI8DoneWords];      // output blocks this pass completed
  int8_t* const xs = reinterpret_cast<int8_t*>(i8_smem);
  int* const acc = reinterpret_cast<int*>(i8_smem + p.acc_off);
  const int tid = threadIdx.x;
  const int H = static_cast<int>(p.H), I = static_cast<int>(p.I);
  const int K = DOWN ? I : H;
  const int rows = DOWN ? H : I;                 // rows of a chunk (gate/up: pairs)
  constexpr int rpt = DOWN ? 16 : 8;
  if constexpr (!DOWN) {
    griddep_wait();
    griddep_launch_dependents();
  }
  // the second launch may start before the first has ended: the ids are the
  // caller's and were complete before the first began
  i8_plan(p, s);
  const int nc = s.n_chunks;
  const int64_t W = static_cast<int64_t>(nc) * rows;
  int64_t lo = W * blockIdx.x / gridDim.x;       // next row of the chunks' rows
  const int64_t hi = W * (blockIdx.x + 1) / gridDim.x;

  // the passes of this CTA: rows [a, a + nr) of a chunk, all with its routes
  struct Work {
    int ch, first, cnt, a, nr;
    int64_t e;
  };
  auto next = [&](Work& w) {
    const int ch = static_cast<int>(lo / rows);
    if (ch != w.ch) {
      // the chunk's expert: largest d with chunk[d] <= ch
      int d0 = 0, d1 = s.n_experts;
      while (d1 - d0 > 1) {
        const int mid = (d0 + d1) >> 1;
        if (s.chunk[mid] <= ch) d0 = mid; else d1 = mid;
      }
      w.ch = ch;
      w.first = s.off[d0] + (ch - s.chunk[d0]) * p.nt;
      const int left = s.off[d0 + 1] - w.first;
      w.cnt = left < p.nt ? left : p.nt;
      w.e = s.expert[d0];
    }
    const int per_pass = kI8AccBytes / (64 * w.cnt) * rpt;  // rows whose accumulators fit
    w.a = static_cast<int>(lo - static_cast<int64_t>(ch) * rows);
    w.nr = rows - w.a < per_pass ? rows - w.a : per_pass;
    if (hi - lo < w.nr) w.nr = static_cast<int>(hi - lo);
    lo += w.nr;
  };
  auto pass_of = [&](const Work& w) {
    I8Pass ps;
    ps.nr = w.nr;
    if constexpr (DOWN) {
      ps.wa = p.w + (w.e * rows + w.a) * K;
      ps.wb = nullptr;
    } else {
      ps.wa = p.w + (w.e * 2 * rows + w.a) * K;
      ps.wb = ps.wa + static_cast<int64_t>(rows) * K;
    }
    return ps;
  };
  I8Stream<NB> stream;
  Work w;
  w.ch = -1;
  bool more = lo < hi;
  if (more) {
    next(w);
    stream.begin(pass_of(w), K);
  }
  // the second launch's weights are not written by the first: they may be on
  // their way while it ends
  if constexpr (DOWN) griddep_wait();
  if constexpr (DOWN) {
    // rows of dropped routes, and the output where no route is in use
    if (p.clear_y) {
      for (int r = blockIdx.x; r < p.R; r += gridDim.x) {
        if (s.dense[r] >= 0) continue;
        for (int i = tid; i < H; i += kI8Threads) p.y[static_cast<int64_t>(r) * H + i] = 0.f;
      }
    }
    if (nc == 0 && p.out) {
      const int64_t n = static_cast<int64_t>(p.T) * H;
      for (int64_t i = static_cast<int64_t>(blockIdx.x) * kI8Threads + tid; i < n;
           i += static_cast<int64_t>(gridDim.x) * kI8Threads) {
        if (p.out_bf16)
          static_cast<uint16_t*>(p.out)[i] = 0;
        else
          static_cast<float*>(p.out)[i] = 0.f;
      }
    }
  }
  int staged = -1;
  while (more) {
    if (w.ch != staged) {
      staged = w.ch;
      I8Rows src;
      src.absmax = nullptr;
      src.rows = s.route + w.first;
      if constexpr (DOWN) {
        src.base = p.h;
        src.div = 1;
        i8_stage_rows<I8_SRC_F32>(src, w.cnt, K, xs, p.stride, s_max, s_scale);
      } else {
        src.base = p.tokens;
        src.div = p.k;
        i8_stage_rows<I8_SRC_BF16>(src, w.cnt, K, xs, p.stride, s_max, s_scale);
      }
    }
    const int tiles = (w.nr + rpt - 1) / rpt;
    for (int i = tid; i < tiles * 16 * w.cnt; i += kI8Threads) acc[i] = 0;
    if (DOWN && tid < kI8DoneWords) s_done[tid] = 0u;
    __syncthreads();
    stream.run(w.cnt, xs, p.stride, acc);
    const Work cur = w;
    more = lo < hi;
    if (more) {
      next(w);
      stream.begin(pass_of(w), K);
    }
    __syncthreads();
    const float* ws = p.wscale + cur.e * (DOWN ? rows : 2 * rows) + cur.a;
    for (int i = tid; i < cur.nr * cur.cnt; i += kI8Threads) {
      const int j = i / cur.nr, r = i - j * cur.nr;
      const int route = s.route[cur.first + j];
      if constexpr (DOWN) {
        p.y[static_cast<int64_t>(route) * H + cur.a + r] =
            __fmul_rn(__fmul_rn(s_scale[j], ws[r]), static_cast<float>(acc[r * cur.cnt + j]));
      } else {
        const int at = ((r >> 3) * 16 + (r & 7)) * cur.cnt + j;
        const double sx = s_scale[j];
        const double gv = sx * ws[r] * acc[at];
        const double uv = sx * ws[rows + r] * acc[at + 8 * cur.cnt];
        p.h[static_cast<int64_t>(route) * I + cur.a + r] =
            static_cast<float>(gv / (1.0 + exp(-gv)) * uv);
      }
    }
    if constexpr (DOWN) {
      if (p.out) {
        // count the rows of every touched block of output columns; whoever
        // completes a block sums it
        __threadfence();
        __syncthreads();
        const int blk0 = cur.a / kI8CombineRows;
        const int nblk = (cur.a + cur.nr - 1) / kI8CombineRows - blk0 + 1;
        if (tid < nblk) {
          const int c0 = (blk0 + tid) * kI8CombineRows;
          const int c1 = c0 + kI8CombineRows < H ? c0 + kI8CombineRows : H;
          const int m0 = cur.a > c0 ? cur.a : c0;
          const int m1 = cur.a + cur.nr < c1 ? cur.a + cur.nr : c1;
          int* const done = p.done + blk0 + tid;
          if (atomicAdd(done, m1 - m0) + (m1 - m0) == (c1 - c0) * nc) {
            *done = 0;
            atomicOr(&s_done[tid >> 5], 1u << (tid & 31));
          }
        }
        __syncthreads();
        __threadfence();
        constexpr int V = kI8CombineRows / 4;               // float4 columns of a block
        for (int i = tid; i < nblk * p.T * V; i += kI8Threads) {
          const int b = i / (p.T * V), rest = i - b * (p.T * V);
          if (!(s_done[b >> 5] >> (b & 31) & 1u)) continue;
          const int tk = rest / V, c = (blk0 + b) * kI8CombineRows + (rest - tk * V) * 4;
          if (c >= H) continue;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          const float* y = p.y + static_cast<int64_t>(tk) * p.k * H + c;
          for (int j0 = 0; j0 < p.k; j0 += 4) {
            float4 q[4];
            float wj[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int r = tk * p.k + j0 + j;
              const bool live = j0 + j < p.k && s.dense[r] >= 0;
              wj[j] = live ? __ldg(p.topk_w + r) : 0.f;
              q[j] = live ? __ldcg(reinterpret_cast<const float4*>(
                                y + static_cast<int64_t>(j0 + j) * H))
                          : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v.x = fmaf(wj[j], q[j].x, v.x);
              v.y = fmaf(wj[j], q[j].y, v.y);
              v.z = fmaf(wj[j], q[j].z, v.z);
              v.w = fmaf(wj[j], q[j].w, v.w);
            }
          }
          const int64_t o = static_cast<int64_t>(tk) * H + c;
          if (p.out_bf16) {
            uint2 b2;
            b2.x = bf16_bits(v.x) | static_cast<uint32_t>(bf16_bits(v.y)) << 16;
            b2.y = bf16_bits(v.z) | static_cast<uint32_t>(bf16_bits(v.w)) << 16;
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o) = b2;
          } else {
            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = v;
          }
        }
      }
    }
    __syncthreads();
  }
}

}  // namespace cq
