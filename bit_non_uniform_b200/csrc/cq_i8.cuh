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
//   * four producer warps copy the weights into a ring of shared-memory units
//     (16 rows x 512 bytes of K, by 16-byte asynchronous copies; a bulk copy
//     per row took 75 cycles each and held an SM to 13 GB/s) and run on while
//     the other 16 warps stage activations or finish a pass;
//   * the streaming warps take the units in turn and feed them to
//     mma.sync.m16n8k32 (S8).  A dot product does not depend on the order of
//     k, so a lane's 16 contiguous bytes serve as the k positions of two MMAs
//     (the activations are read under the same order);
//   * rows, not tiles, are split evenly over the CTAs (a tile's missing rows
//     are not loaded).  INT32 sums do not depend on their order, so the warps
//     add their parts to the CTA's accumulators with shared-memory atomics and
//     the result is the same on every run;
//   * every CTA quantizes the few activation rows itself (no separate launch).
// Loading straight into the consumers' registers (two buffers of 4 KB a warp)
// kept too little in flight once several tokens made a step's arithmetic
// longer: 4.8 TB/s at 16 tokens of 64 experts against 6.4 now.  Measured: one
// token of 16 experts 7168 x 3072 in 170 us, 6.2 TB/s or 96% of the copy rate;
// 6144 x 7168 for one token in 10.5 us, of which 3.7 are the launch and staging
// that a small matrix takes too.
#pragma once

#include "cq_device.cuh"
#include "cq_engine.cuh"

namespace cq {

constexpr int kI8Consumers = 512;            // threads that multiply
constexpr int kI8Warps = kI8Consumers / 32;
constexpr int kI8Producers = 4;              // producer warps
constexpr int kI8Threads = kI8Consumers + 32 * kI8Producers;
constexpr int kI8Unit = 512;                 // bytes of K of a unit (16 rows)
constexpr int kI8Pitch = kI8Unit + 64;       // 16-byte reads of two rows hit all banks
constexpr int kI8UnitBytes = 16 * kI8Pitch;
constexpr int kI8MaxSlots = 24;              // units in the ring
constexpr int kI8MinSlots = 4;
constexpr int kI8AccBytes = 16 * 1024;       // accumulators of one pass over the rows
constexpr int kI8MaxTokens = 16;             // tokens of one pass
constexpr int kI8MaxRoutes = 1024;           // routes of one launch of the MoE layer
constexpr int kI8MaxExperts = 16384;
constexpr int kI8SmemLimit = 227 * 1024;

// Waits of the streaming kernels; the MoE layer's second launch adds
// kI8SecondSite.
enum I8Site : int { SITE_I8_SLOT_EMPTY = 54, SITE_I8_SLOT_FULL = 55 };
constexpr int kI8SecondSite = 2;

// Bytes between two activation rows in shared memory: whole units (zeros past
// K, where a unit's weights are whatever the slot held before), plus 64 so
// that the eight lanes of a 16-byte read phase (two rows x 64 bytes) touch
// all 32 banks.
__host__ __device__ constexpr int i8_row_stride(int64_t K) {
  return static_cast<int>((K + kI8Unit - 1) / kI8Unit * kI8Unit) + 64;
}

// A bounded wait of a whole warp: every lane waits, then the lanes vote, so
// that they leave together and with one answer (alone, each leaves the spin in
// its own time, and one may see the phase complete where another gives up).
// Warp-wide instructions and barriers follow these waits.
__device__ __forceinline__ bool i8_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort,
                                             uint64_t timeout_ns, int site) {
  const bool ok = *abort == 0 && wait_phase(bar, parity, abort, timeout_ns, site);
  return __all_sync(0xffffffffu, ok) != 0;
}

// Barrier of the consumers.
__device__ __forceinline__ void i8_sync() {
  asm volatile("bar.sync 1, 512;" ::: "memory");
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

// One activation code, as quant_rows_kernel decides it (FP32): the conversion
// rounds to nearest even, takes NaN to 0 and saturates.
__device__ __forceinline__ uint32_t i8_code(float v, float inv) {
  const int r = __float2int_rn(__fmul_rn(v, inv));
  return static_cast<uint32_t>(min(max(r, -127), 127)) & 0xFFu;
}
__device__ __forceinline__ uint32_t i8_code4(float a, float b, float c, float d, float inv) {
  return __byte_perm(__byte_perm(i8_code(a, inv), i8_code(b, inv), 0x0040),
                     __byte_perm(i8_code(c, inv), i8_code(d, inv), 0x0040), 0x5410);
}

enum I8Source : int { I8_SRC_BF16 = 0, I8_SRC_F32 = 1, I8_SRC_CODES = 2 };

// Where the rows of a pass come from: row j of the pass is row rows[j] /
// `div` of `base` (rows == null: row j).
struct I8Rows {
  const void* base;
  const float* absmax;     // I8_SRC_CODES: the rows' maxima
  const int16_t* rows;     // shared memory, or null
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

// Quantize (or copy) `cnt` rows of K elements into shared memory, zeros from
// K to the end of its last unit, with each row's RN(absmax / 127) in s_scale.
// All consumers take part; ends with their barrier.  K is a multiple of 16.
template <int SRC>
__device__ __forceinline__ void i8_stage_rows(const I8Rows& src, int cnt, int K, int8_t* xs,
                                              int stride, uint32_t* s_max, float* s_scale) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int ES = SRC == I8_SRC_BF16 ? 2 : (SRC == I8_SRC_F32 ? 4 : 1);
  auto row_ptr = [&](int j) {
    const int r = src.rows ? src.rows[j] / src.div : j;
    return static_cast<const uint8_t*>(src.base) + static_cast<int64_t>(r) * K * ES;
  };
  const int pad = (stride - 64 - K) / 16;
  for (int i = threadIdx.x; i < cnt * pad; i += kI8Consumers) {
    const int j = i / pad;
    *reinterpret_cast<uint4*>(xs + j * stride + K + (i - j * pad) * 16) = make_uint4(0, 0, 0, 0);
  }
  if constexpr (SRC == I8_SRC_CODES) {
    const int nv = K / 16;
    for (int i = threadIdx.x; i < cnt * nv; i += kI8Consumers) {
      const int j = i / nv, v = i - j * nv;
      *reinterpret_cast<uint4*>(xs + j * stride + v * 16) =
          *reinterpret_cast<const uint4*>(row_ptr(j) + v * 16);
    }
    if (threadIdx.x < cnt) s_scale[threadIdx.x] = __fdiv_rn(src.absmax[threadIdx.x], 127.0f);
    i8_sync();
  } else {
    if (threadIdx.x < kI8MaxTokens) s_max[threadIdx.x] = 0u;
    i8_sync();
    // each row is shared by `parts` warps (cnt <= 16: a warp has one row at
    // most); a thread keeps its first 8 values between the two passes and
    // reads the others again (short loops: a cold instruction cache costs a
    // small call more than that)
    const int parts = kI8Warps / cnt, j = warp / parts;
    const int step = parts * 32, v0 = (warp - j * parts) * 32 + lane, nv = K / 8;
    const uint8_t* const row = j < cnt ? row_ptr(j) : nullptr;
    float first[8];
    // the largest magnitude: of a token's activations as cq_quant_rows takes
    // it (NaN ignored); of computed values NaN counts as the largest, so that
    // what overflowed upstream does not come out as zeros
    auto larger = [](float m, float x) {
      if constexpr (SRC == I8_SRC_F32)
        return __uint_as_float(max(__float_as_uint(m), __float_as_uint(x) & 0x7FFFFFFFu));
      else
        return fmaxf(m, fabsf(x));
    };
    if (row) {
      float mx = 0.f;
      if (v0 < nv) {
        i8_load8<SRC>(row, static_cast<int64_t>(v0) * 8, first);
#pragma unroll 8
        for (int v = v0 + step; v < nv; v += step) {
          float x[8];
          i8_load8<SRC>(row, static_cast<int64_t>(v) * 8, x);
#pragma unroll
          for (int i = 0; i < 8; ++i) mx = larger(mx, x[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = larger(mx, first[i]);
      }
      const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(mx));
      if (lane == 0) atomicMax(&s_max[j], m);
    }
    i8_sync();
    if (row) {
      const float mx = __uint_as_float(s_max[j]);
      const float inv = mx > 0.f ? __fdiv_rn(127.0f, mx) : 0.f;
      auto put = [&](int v, const float (&x)[8]) {
        *reinterpret_cast<uint2*>(xs + j * stride + v * 8) =
            make_uint2(i8_code4(x[0], x[1], x[2], x[3], inv),
                       i8_code4(x[4], x[5], x[6], x[7], inv));
      };
      if (v0 < nv) put(v0, first);
#pragma unroll 4
      for (int v = v0 + step; v < nv; v += step) {
        float x[8];
        i8_load8<SRC>(row, static_cast<int64_t>(v) * 8, x);
        put(v, x);
      }
      if (lane == 0 && v0 == 0) s_scale[j] = __fdiv_rn(mx, 127.0f);
    }
    i8_sync();
  }
}

// The rows one pass of a CTA multiplies: `nr` row indices from `wa`.  A tile
// is 16 MMA rows: rows 8 t .. 8 t + 7 of `wa` and the same rows of `wb`
// (paired: gate and up), or 16 consecutive rows of `wa` (wb == null).  Its
// units are 512 bytes of K each; a pass's units are numbered tile by tile.
struct I8Pass {
  const int8_t* wa;
  const int8_t* wb;
  int nr;
  __device__ __forceinline__ int tiles() const { return wb ? (nr + 7) >> 3 : (nr + 15) >> 4; }
};

// The ring of weight units in shared memory: slot q % slots holds unit q of
// the CTA's passes, numbered through.  Unit q is copied by producer warp
// q % kI8Producers and multiplied by streaming warp q % i8_streamers(slots),
// and slots is a multiple of both: a slot is always filled by one warp and
// emptied by one warp, in order, so that a wait on its parity never meets the
// phase before.
__device__ __forceinline__ int i8_streamers(int slots) {
  return slots <= kI8Warps ? slots : slots / 2;
}
struct I8Ring {
  uint32_t data, full, empty;      // shared addresses: units, barriers
  int slots;
  int site;                        // 0 or kI8SecondSite
  uint64_t timeout_ns;
  volatile int* abort_flag;
};

// Set up by one thread, before a barrier of the whole CTA.
// `withhold` (a test hook): the first slot waits for an arrival that never comes.
__device__ __forceinline__ void i8_ring_init(const I8Ring& r, int withhold) {
  for (int i = 0; i < r.slots; ++i) {
    mbar_init(r.full + 8 * i, 32 + (i == 0 ? withhold : 0));     // the lanes of its producer
    mbar_init(r.empty + 8 * i, 1);
  }
  *r.abort_flag = 0;
  fence_mbar_init();
}

// A producer or streaming warp's place in the units: the next it handles.
struct I8Turn {
  uint32_t q;
  int slot;
  uint32_t round;
  __device__ __forceinline__ void next(int step, int slots) {
    q += step;
    slot += step;
    if (slot >= slots) {
      slot -= slots;
      ++round;
    }
  }
};

// Producer warps: copy this warp's units of the pass, whose first has number q0.
__device__ __forceinline__ void i8_produce(const I8Ring& ring, const I8Pass& ps, int K,
                                           uint32_t q0, I8Turn& turn) {
  const int lane = threadIdx.x & 31;
  const bool paired = ps.wb != nullptr;
  const int per = paired ? 8 : 16, nk = (K + kI8Unit - 1) / kI8Unit;
  const int total = ps.tiles() * nk;
  int u = static_cast<int>(turn.q - q0);
  int tile = u / nk, kk = u - tile * nk;
  for (; u < total; u += kI8Producers) {
    // the first round fills free slots; waiting for one to be emptied has its
    // limit, which must not run while a preceding kernel does (a no-op where
    // the CTA has waited for it already)
    if (turn.round == 1u) griddep_wait();
    if (!i8_wait_warp(ring.empty + 8 * turn.slot, (turn.round & 1u) ^ 1u, ring.abort_flag,
                      ring.timeout_ns, SITE_I8_SLOT_EMPTY + ring.site))
      return;
    const int k = kk * kI8Unit + lane * 16;
    if (k < K) {
      // rows 0-7 and 8-15 of the unit
      const int left = ps.nr - tile * per, left_b = paired ? left : left - 8;
      const int64_t at = static_cast<int64_t>(tile) * per * K + k;
      const int8_t* a = ps.wa + at;
      const int8_t* b = paired ? ps.wb + at : a + static_cast<int64_t>(8) * K;
      const uint32_t dst = ring.data + turn.slot * kI8UnitBytes + lane * 16;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        if (r < left) cp_async16(dst + r * kI8Pitch, a);
        if (r < left_b) cp_async16(dst + (8 + r) * kI8Pitch, b);
        a += K;
        b += K;
      }
    }
    cp_async_mbar_arrive(ring.full + 8 * turn.slot);
    turn.next(kI8Producers, ring.slots);
    kk += kI8Producers;
    while (kk >= nk) {
      kk -= nk;
      ++tile;
    }
  }
}

// Streaming warps: acc[tile][16][cnt] += the products of this warp's units of
// the pass with the `cnt` staged activation rows.  acc is zero on entry and
// complete after the consumers' barrier.  q0: the number of the pass's first
// unit.
template <int NB>
__device__ __forceinline__ void i8_consume(const I8Ring& ring, const uint8_t* ring_data,
                                           const I8Pass& ps, int cnt, int K, const int8_t* xs,
                                           int stride, int* acc, uint32_t q0, I8Turn& turn) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int W = i8_streamers(ring.slots);
  if (warp >= W) return;
  const int nk = (K + kI8Unit - 1) / kI8Unit;
  const int total = ps.tiles() * nk;
  const bool has0 = g < cnt, has1 = NB > 1 && g + 8 < cnt;
  const int8_t* const x0 = xs + g * stride + t * 16;
  const int8_t* const x1 = x0 + 8 * stride;
  int d[NB][4], e[NB][4];                  // two chains of MMAs
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) d[n][i] = e[n][i] = 0;
  int u = static_cast<int>(turn.q - q0);
  int tile = u / nk, kk = u - tile * nk;
  for (; u < total; u += W) {
    if (!i8_wait_warp(ring.full + 8 * turn.slot, turn.round & 1u, ring.abort_flag,
                      ring.timeout_ns, SITE_I8_SLOT_FULL + ring.site))
      return;
    const uint8_t* const w = ring_data + turn.slot * kI8UnitBytes + g * kI8Pitch + t * 16;
    const int8_t* const y0 = x0 + kk * kI8Unit;
    const int8_t* const y1 = x1 + kk * kI8Unit;
#pragma unroll
    for (int s = 0; s < kI8Unit / 64; ++s) {
      const uint4 a = *reinterpret_cast<const uint4*>(w + s * 64);
      const uint4 b = *reinterpret_cast<const uint4*>(w + 8 * kI8Pitch + s * 64);
      uint4 x = make_uint4(0, 0, 0, 0);
      if (has0) x = *reinterpret_cast<const uint4*>(y0 + s * 64);
      mma_16832_s8(d[0], a.x, b.x, a.y, b.y, x.x, x.y);
      mma_16832_s8(e[0], a.z, b.z, a.w, b.w, x.z, x.w);
      if constexpr (NB > 1) {
        uint4 z = make_uint4(0, 0, 0, 0);
        if (has1) z = *reinterpret_cast<const uint4*>(y1 + s * 64);
        mma_16832_s8(d[1], a.x, b.x, a.y, b.y, z.x, z.y);
        mma_16832_s8(e[1], a.z, b.z, a.w, b.w, z.z, z.w);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(ring.empty + 8 * turn.slot);
    turn.next(W, ring.slots);
    const int was = tile;
    kk += W;
    while (kk >= nk) {
      kk -= nk;
      ++tile;
    }
    if (tile != was || u + W >= total) {
      // the warp's last unit of this tile
      int* const at = acc + was * 16 * cnt;
#pragma unroll
      for (int n = 0; n < NB; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col = n * 8 + 2 * t + (i & 1);
          if (col < cnt) atomicAdd(at + (g + 8 * (i >> 1)) * cnt + col, d[n][i] + e[n][i]);
          d[n][i] = e[n][i] = 0;
        }
      }
    }
  }
}

// silu(g) * u with silu(g) = g / (1 + exp(-g)), in FP32.
__device__ __forceinline__ float i8_swiglu_f32(float g, float u) {
  return g / (1.0f + expf(-g)) * u;
}

// ---------------------------------------------------------------------------
// the product for at most 8 tokens
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
  int xs_off, acc_off;      // staged rows and accumulators, behind the ring
  int slots;
  int withhold;             // i8_ring_init
  uint64_t timeout_ns;
};

template <int SRC>
__global__ void __launch_bounds__(kI8Threads, 1)
    i8_linear_kernel(const __grid_constant__ I8LinearParams p) {
  extern __shared__ __align__(128) uint8_t i8_smem[];
  __shared__ uint64_t s_bar[2 * kI8MaxSlots];
  __shared__ uint32_t s_max[kI8MaxTokens];
  __shared__ float s_scale[kI8MaxTokens];
  __shared__ int s_abort;
  int8_t* const xs = reinterpret_cast<int8_t*>(i8_smem + p.xs_off);
  int* const acc = reinterpret_cast<int*>(i8_smem + p.acc_off);
  const int tid = threadIdx.x;
  const int rows = p.swiglu ? p.N / 2 : p.N;
  const int r0 = static_cast<int>(static_cast<int64_t>(blockIdx.x) * rows / gridDim.x);
  const int r1 = static_cast<int>(static_cast<int64_t>(blockIdx.x + 1) * rows / gridDim.x);
  const int rpt = p.swiglu ? 8 : 16, nk = (p.K + kI8Unit - 1) / kI8Unit;
  const int per_pass = kI8AccBytes / (64 * p.M) * rpt;      // rows whose accumulators fit
  auto pass_at = [&](int a) {
    I8Pass ps;
    ps.nr = r1 - a < per_pass ? r1 - a : per_pass;
    ps.wa = p.w + static_cast<int64_t>(a) * p.K;
    ps.wb = p.swiglu ? ps.wa + static_cast<int64_t>(rows) * p.K : nullptr;
    return ps;
  };
  const I8Ring ring = {smem_u32(i8_smem), smem_u32(s_bar), smem_u32(s_bar + kI8MaxSlots), p.slots,
                       0, p.timeout_ns, &s_abort};
  if (tid == 0) i8_ring_init(ring, p.withhold);
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  if (tid >= kI8Consumers) {
    uint32_t q = 0;
    I8Turn turn = {static_cast<uint32_t>(tid >> 5) - kI8Warps, (tid >> 5) - kI8Warps, 0u};
    for (int a = r0; a < r1 && !*ring.abort_flag; a += per_pass) {
      const I8Pass ps = pass_at(a);
      i8_produce(ring, ps, p.K, q, turn);
      q += ps.tiles() * nk;
    }
    cp_async_wait_all();
    return;
  }
  I8Rows src;
  src.base = p.x;
  src.absmax = p.absmax;
  src.rows = nullptr;
  src.div = 1;
  i8_stage_rows<SRC>(src, p.M, p.K, xs, p.stride, s_max, s_scale);
  uint32_t q = 0;
  I8Turn turn = {static_cast<uint32_t>(tid >> 5), tid >> 5, 0u};
  for (int a = r0; a < r1; a += per_pass) {
    const I8Pass ps = pass_at(a);
    const int nr = ps.nr;
    for (int i = tid; i < ps.tiles() * 16 * p.M; i += kI8Consumers) acc[i] = 0;
    i8_sync();
    i8_consume<1>(ring, i8_smem, ps, p.M, p.K, xs, p.stride, acc, q, turn);
    q += ps.tiles() * nk;
    i8_sync();
    for (int i = tid; i < nr * p.M; i += kI8Consumers) {
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
    i8_sync();
  }
}

// ---------------------------------------------------------------------------
// the MoE layer for a few tokens: two launches, and one that sums
// ---------------------------------------------------------------------------
// Both launches read the routes themselves: the experts in use, each with its
// routes, cut into chunks of at most `nt` routes.  A chunk multiplies every
// row of its expert, so the work is chunks x rows, split over the CTAs in
// equal shares of an estimated cost.
//   gate/up: xq = codes of the chunk's tokens; g, u per (row, route);
//            h[route][row] = RN32(silu(g) u) with g, u and silu in FP64, so
//            that the codes of the second quantization are those of any other
//            FP64 evaluation (a value next to a rounding border would
//            otherwise fall on either side of it);
//   down:    hq = codes of the chunk's h rows; y[route][row];
//   then a small kernel sums a token's routes in their order.  (Summed inside
//   the second launch by whichever CTA completes a block of columns, it cost
//   6 us a pass, or a tail of 80 us when left to the end.)
struct I8MoeParams {
  const uint16_t* tokens;   // bf16 [T][H]
  const int32_t* ids;       // [T][k]
  const float* topk_w;      // [T][k]
  const int8_t* w;          // the stage's weights: [E][2I][H] or [E][H][I]
  const float* wscale;      // [E][2I] or [E][H]
  float* h;                 // [R][I]
  float* y;                 // [R][H]
  void* out;                // [T][H], or null
  int T, k, R, E;
  int64_t H, I;
  int nt;                   // routes per chunk
  int wt_row, wt_route;     // i8_weight
  float wt_gap;             // what staging another chunk costs, in units of its rows' weight
  int gap_rows;             // ... in rows
  int out_bf16, clear_y;
  int stride;               // i8_row_stride of the stage's K
  int xs_off, acc_off;      // staged rows and accumulators, behind the ring
  int slots;
  int withhold;             // i8_ring_init
  uint64_t timeout_ns;
};

// Arrays of the plan in shared memory, sized for the launch's routes (in
// whole groups of 32) and experts.
struct I8Plan {
  uint32_t* bits;       // experts in use
  int16_t* pref;        // experts in use before each word
  int16_t* expert;      // the experts in use
  int16_t* cnt;         // their routes
  int16_t* off;         // first route of each in `route`, and the end
  int16_t* chunk;       // chunks before each, and all
  int16_t* route;       // routes by expert
  int16_t* dense;       // each route's expert, as an index into `expert`, or -1
  int16_t* rank;        // its place among the expert's routes
  int* cost;            // i8_weight of the chunks before each expert, and of all
  int* n;               // experts in use, chunks, this CTA's first row and the next one's
};

__host__ __device__ constexpr int i8_plan_routes(int R) { return (R + 31) / 32 * 32; }
__host__ __device__ constexpr int i8_plan_words(int E) { return (E + 31) / 32; }
__host__ __device__ constexpr int i8_plan_bytes(int R, int E) {
  return (i8_plan_words(E) * 6 + i8_plan_routes(R) * 18 + 4 * 2 + 6 * 4 + 15) / 16 * 16;
}

__device__ __forceinline__ I8Plan i8_plan_at(uint8_t* at, int R, int E) {
  const int r = i8_plan_routes(R), w = i8_plan_words(E);
  I8Plan s;
  s.n = reinterpret_cast<int*>(at);
  s.cost = s.n + 4;
  s.bits = reinterpret_cast<uint32_t*>(s.cost + r + 2);
  s.pref = reinterpret_cast<int16_t*>(s.bits + w);
  s.expert = s.pref + w;
  s.cnt = s.expert + r;
  s.off = s.cnt + r;
  s.chunk = s.off + r + 2;
  s.route = s.chunk + r + 2;
  s.dense = s.route + r;
  s.rank = s.dense + r;
  return s;
}

// What a row of a chunk costs: its bytes, a tenth more when its routes take
// two blocks of MMA columns, and its share of the passes (the accumulators
// hold fewer rows, the more routes a chunk has; a pass ends with a gap of some
// 7 us).  Split by rows alone, the CTAs of experts with 9 to 13 routes finished
// at 390 to 410 us, all others at 345 (16 tokens, 64 experts 7168 x 3072).
__device__ __forceinline__ int i8_weight(const I8MoeParams& p, int cnt) {
  return p.wt_row * (cnt > 8 ? 11 : 10) + p.wt_route * cnt;
}
// ... and the chunks of an expert with `cnt` routes.
__device__ __forceinline__ int i8_expert_weight(const I8MoeParams& p, int cnt) {
  if (cnt == 0) return 0;
  const int whole = (cnt - 1) / p.nt;
  return whole * i8_weight(p, p.nt) + i8_weight(p, cnt - whole * p.nt);
}

// The row of the chunks' rows, numbered through, at which CTA b of n begins:
// equal shares of the cost, or of the rows for the few routes of the short
// plan.  A CTA whose rows span two chunks stages activations twice (3 to 4 us, for
// which all others wait), so that chunks are laid out with gaps of that cost
// between them, at most a CTA's share; a CTA that would begin in a gap begins
// behind it: 5 tokens of 40 experts 2064 x 1040 28 us instead of 32.5.  FP32 is
// exact enough (a row or two) and quick, and every step rounds monotonously, so
// that the CTAs' ranges join.
__device__ __forceinline__ int i8_begin(const I8MoeParams& p, const I8Plan& s, int ne, int nc,
                                        int rows, int b, int n) {
  if (b == n || ne == 0) return nc * rows;
  const float all = s.cost[ne], gap = fminf(p.wt_gap, __fdiv_rn(all, n));
  const float at = __fdiv_rn(__fmul_rn(__fadd_rn(all, __fmul_rn(nc - 1, gap)), b), n);
  auto begins = [&](int d) { return __fadd_rn(s.cost[d], __fmul_rn(s.chunk[d], gap)); };
  int d0 = 0, d1 = ne;                     // the expert: largest d that begins at or before it
  while (d1 - d0 > 1) {
    const int mid = (d0 + d1) >> 1;
    if (begins(mid) <= at) d0 = mid; else d1 = mid;
  }
  float left = __fsub_rn(at, begins(d0));
  const int cnt = s.off[d0 + 1] - s.off[d0], whole = (cnt - 1) / p.nt;
  const float w = __fadd_rn(i8_weight(p, p.nt), gap);
  int c = static_cast<int>(__fdiv_rn(left, w));
  c = c < whole ? c : whole;
  left = __fsub_rn(left, __fmul_rn(c, w));
  const float share = __fdiv_rn(left, i8_weight(p, c < whole ? p.nt : cnt - whole * p.nt));
  const int row = static_cast<int>(__fmul_rn(share, rows));
  return (s.chunk[d0] + c) * rows + min(max(row, 0), rows);
}
__device__ __forceinline__ int warp_inclusive_sum(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// The plan of at most 32 routes, by the first warp (experts in the order of
// their first route; the order only decides which CTA works on what).
__device__ __forceinline__ void i8_plan_small(const I8MoeParams& p, const I8Plan& s, int rows) {
  const int lane = threadIdx.x;
  if (lane < 32) {
    int id = lane < p.R ? p.ids[lane] : -1;
    if (id < 0 || id >= p.E) id = -1;
    const unsigned same = __match_any_sync(0xffffffffu, id);
    const unsigned below = (1u << lane) - 1u;
    const bool first = id >= 0 && (same & below) == 0;
    const unsigned firsts = __ballot_sync(0xffffffffu, first);
    const int cnt = first ? __popc(same) : 0, chunks = (cnt + p.nt - 1) / p.nt;
    const int off = warp_inclusive_sum(cnt), ch = warp_inclusive_sum(chunks);
    const int leader = __ffs(same) - 1;
    const int base = __shfl_sync(0xffffffffu, off - cnt, leader);
    const int d = __popc(firsts & ((1u << leader) - 1u));
    if (first) {
      s.expert[d] = static_cast<int16_t>(id);
      s.off[d] = static_cast<int16_t>(off - cnt);
      s.chunk[d] = static_cast<int16_t>(ch - chunks);
    }
    s.dense[lane] = static_cast<int16_t>(id >= 0 ? d : -1);
    if (id >= 0) s.route[base + __popc(same & below)] = static_cast<int16_t>(lane);
    if (lane == 31) {
      const int ne = __popc(firsts);
      s.n[0] = ne;
      s.n[1] = ch;
      s.off[ne] = static_cast<int16_t>(off);
      s.chunk[ne] = static_cast<int16_t>(ch);
      const int n = gridDim.x, gap = min(p.gap_rows, ch * rows / n);
      const int pitch = rows + gap, total = ch * pitch - gap, q = total / n, r = total - q * n;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int b = static_cast<int>(blockIdx.x) + i;
        const int at = ch > 0 ? b * q + b * r / n : 0, c = at / pitch;
        s.n[2 + i] = c * rows + min(at - c * pitch, rows);
      }
    }
  }
  __syncthreads();
}

__device__ __forceinline__ void i8_plan_large(const I8MoeParams& p, const I8Plan& s, int rows) {
  const int tid = threadIdx.x;
  const int words = (p.E + 31) / 32;
  for (int i = tid; i < words; i += kI8Threads) s.bits[i] = 0u;
  __syncthreads();
  for (int r = tid; r < i8_plan_routes(p.R); r += kI8Threads) {
    int id = r < p.R ? p.ids[r] : -1;
    if (id < 0 || id >= p.E) id = -1;
    s.dense[r] = static_cast<int16_t>(id);
    if (id >= 0) atomicOr(&s.bits[id >> 5], 1u << (id & 31));
  }
  __syncthreads();
  // the rest is short enough for one warp
  if (tid < 32) {
    int ne = 0;
    for (int w0 = 0; w0 < words; w0 += 32) {
      const int n = w0 + tid < words ? __popc(s.bits[w0 + tid]) : 0;
      const int inc = warp_inclusive_sum(n);
      if (w0 + tid < words) s.pref[w0 + tid] = static_cast<int16_t>(ne + inc - n);
      ne += __shfl_sync(0xffffffffu, inc, 31);
    }
    for (int i = tid; i < ne; i += 32) s.cnt[i] = 0;
    __syncwarp();
    // each route's expert and its place among the expert's routes, in route
    // order: every CTA of both launches has to cut an expert's routes into
    // the same chunks
    for (int r0 = 0; r0 < p.R; r0 += 32) {
      const int id = s.dense[r0 + tid];
      int d = -1;
      if (id >= 0) {
        d = s.pref[id >> 5] + __popc(s.bits[id >> 5] & ((1u << (id & 31)) - 1u));
        s.expert[d] = static_cast<int16_t>(id);
      }
      const unsigned same = __match_any_sync(0xffffffffu, d);
      const int before = __popc(same & ((1u << tid) - 1u));
      const int base = d >= 0 ? s.cnt[d] : 0;
      __syncwarp();
      if (d >= 0 && before == 0) s.cnt[d] = static_cast<int16_t>(base + __popc(same));
      s.dense[r0 + tid] = static_cast<int16_t>(d);
      s.rank[r0 + tid] = static_cast<int16_t>(base + before);
      __syncwarp();
    }
    int off = 0, ch = 0, cost = 0;
    for (int d0 = 0; d0 < ne; d0 += 32) {
      const int cnt = d0 + tid < ne ? s.cnt[d0 + tid] : 0;
      const int chunks = (cnt + p.nt - 1) / p.nt;
      const int a = warp_inclusive_sum(cnt), b = warp_inclusive_sum(chunks);
      const int weight = i8_expert_weight(p, cnt), c = warp_inclusive_sum(weight);
      if (d0 + tid < ne) {
        s.off[d0 + tid] = static_cast<int16_t>(off + a - cnt);
        s.chunk[d0 + tid] = static_cast<int16_t>(ch + b - chunks);
        s.cost[d0 + tid] = cost + c - weight;
      }
      off += __shfl_sync(0xffffffffu, a, 31);
      ch += __shfl_sync(0xffffffffu, b, 31);
      cost += __shfl_sync(0xffffffffu, c, 31);
    }
    if (tid == 0) {
      s.cost[ne] = cost;
      s.off[ne] = static_cast<int16_t>(off);
      s.chunk[ne] = static_cast<int16_t>(ch);
      s.n[0] = ne;
      s.n[1] = ch;
    }
    __syncwarp();
    if (tid < 2)
      s.n[2 + tid] = i8_begin(p, s, ne, ch, rows, static_cast<int>(blockIdx.x) + tid,
                              static_cast<int>(gridDim.x));
    for (int r = tid; r < p.R; r += 32) {
      const int d = s.dense[r];
      if (d >= 0) s.route[s.off[d] + s.rank[r]] = static_cast<int16_t>(r);
    }
  }
  __syncthreads();
}

template <bool DOWN, int NB>
__global__ void __launch_bounds__(kI8Threads, 1)
    i8_moe_kernel(const __grid_constant__ I8MoeParams p) {
  extern __shared__ __align__(128) uint8_t i8_smem[];
  __shared__ uint32_t s_max[kI8MaxTokens];
  __shared__ float s_scale[kI8MaxTokens];
  __shared__ uint64_t s_bar[2 * kI8MaxSlots];
  __shared__ int s_abort;
  int8_t* const xs = reinterpret_cast<int8_t*>(i8_smem + p.xs_off);
  int* const acc = reinterpret_cast<int*>(i8_smem + p.acc_off);
  const I8Plan s = i8_plan_at(i8_smem + p.acc_off + kI8AccBytes, p.R, p.E);
  const int tid = threadIdx.x;
  const int H = static_cast<int>(p.H), I = static_cast<int>(p.I);
  const int K = DOWN ? I : H;
  const int rows = DOWN ? H : I;                 // rows of a chunk (gate/up: pairs)
  constexpr int rpt = DOWN ? 16 : 8;
  const int nk = (K + kI8Unit - 1) / kI8Unit;
  const I8Ring ring = {smem_u32(i8_smem), smem_u32(s_bar), smem_u32(s_bar + kI8MaxSlots), p.slots,
                       DOWN ? kI8SecondSite : 0, p.timeout_ns, &s_abort};
  if (tid == 0) i8_ring_init(ring, p.withhold);
  if constexpr (!DOWN) {
    griddep_wait();
    griddep_launch_dependents();
  }
  // the second launch may start before the first has ended: the ids are the
  // caller's and were complete before the first began
  if (p.R <= 32)
    i8_plan_small(p, s, rows);
  else
    i8_plan_large(p, s, rows);
  int lo = s.n[2];                               // next row of the chunks' rows (below 2^27)
  const int hi = s.n[3];

  // the passes of this CTA: rows [a, a + nr) of a chunk, all with its routes
  struct Work {
    int ch, first, cnt, a, nr;
    int64_t e;
  };
  auto next = [&](Work& w) {
    const int ch = lo / rows;
    if (ch != w.ch) {
      // the chunk's expert: largest d with chunk[d] <= ch
      int d0 = 0, d1 = s.n[0];
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
    w.a = lo - ch * rows;
    w.nr = rows - w.a < per_pass ? rows - w.a : per_pass;
    if (hi - lo < w.nr) w.nr = hi - lo;
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
  Work w;
  w.ch = -1;
  if (tid >= kI8Consumers) {
    // the second launch's weights are not written by the first: the ring may
    // fill while that ends
    uint32_t q = 0;
    I8Turn turn = {static_cast<uint32_t>(tid >> 5) - kI8Warps, (tid >> 5) - kI8Warps, 0u};
    while (lo < hi && !*ring.abort_flag) {
      next(w);
      const I8Pass ps = pass_of(w);
      i8_produce(ring, ps, K, q, turn);
      q += ps.tiles() * nk;
    }
    cp_async_wait_all();
    return;
  }
  if constexpr (DOWN) {
    griddep_wait();
    griddep_launch_dependents();
    // rows of dropped routes
    if (p.clear_y) {
      for (int r = blockIdx.x; r < p.R; r += gridDim.x) {
        if (s.dense[r] >= 0) continue;
        for (int i = tid; i < H; i += kI8Consumers) p.y[static_cast<int64_t>(r) * H + i] = 0.f;
      }
    }
  }
  int staged = -1;
  uint32_t q = 0;
  I8Turn turn = {static_cast<uint32_t>(tid >> 5), tid >> 5, 0u};
  while (lo < hi) {
    next(w);
    const I8Pass ps = pass_of(w);
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
    for (int i = tid; i < ps.tiles() * 16 * w.cnt; i += kI8Consumers) acc[i] = 0;
    i8_sync();
    if (NB > 1 && w.cnt > 8)
      i8_consume<NB>(ring, i8_smem, ps, w.cnt, K, xs, p.stride, acc, q, turn);
    else
      i8_consume<1>(ring, i8_smem, ps, w.cnt, K, xs, p.stride, acc, q, turn);
    q += ps.tiles() * nk;
    i8_sync();
    const float* ws = p.wscale + w.e * (DOWN ? rows : 2 * rows) + w.a;
    for (int i = tid; i < w.nr * w.cnt; i += kI8Consumers) {
      const int j = i / w.nr, r = i - j * w.nr;
      const int route = s.route[w.first + j];
      if constexpr (DOWN) {
        p.y[static_cast<int64_t>(route) * H + w.a + r] =
            __fmul_rn(__fmul_rn(s_scale[j], ws[r]), static_cast<float>(acc[r * w.cnt + j]));
      } else {
        const int at = ((r >> 3) * 16 + (r & 7)) * w.cnt + j;
        const double sx = s_scale[j];
        const double gv = sx * ws[r] * acc[at];
        const double uv = sx * ws[rows + r] * acc[at + 8 * w.cnt];
        p.h[static_cast<int64_t>(route) * I + w.a + r] =
            static_cast<float>(gv / (1.0 + exp(-gv)) * uv);
      }
    }
    i8_sync();
  }
}

// out[t][c] = sum_j w[t][j] y[t k + j][c] (j ascending, FP32; dropped routes
// contribute nothing): one float4 of columns per thread.
constexpr int kI8CombineThreads = 128;

__global__ void __launch_bounds__(kI8CombineThreads)
    i8_combine_kernel(const __grid_constant__ I8MoeParams p) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kI8CombineThreads + threadIdx.x;
  const int V = static_cast<int>(p.H / 4);
  griddep_wait();
  griddep_launch_dependents();
  if (i >= static_cast<int64_t>(p.T) * V) return;
  const int t = static_cast<int>(i / V), c = static_cast<int>(i - static_cast<int64_t>(t) * V);
  const float4* y = reinterpret_cast<const float4*>(p.y) + static_cast<int64_t>(t) * p.k * V + c;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = 0; j0 < p.k; j0 += 8) {
    float4 q[8];
    float wj[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = t * p.k + j0 + j;
      const int id = j0 + j < p.k ? p.ids[r] : -1;
      const bool live = id >= 0 && id < p.E;
      wj[j] = live ? p.topk_w[r] : 0.f;
      q[j] = live ? __ldcg(y + static_cast<int64_t>(j0 + j) * V) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v.x = fmaf(wj[j], q[j].x, v.x);
      v.y = fmaf(wj[j], q[j].y, v.y);
      v.z = fmaf(wj[j], q[j].z, v.z);
      v.w = fmaf(wj[j], q[j].w, v.w);
    }
  }
  if (p.out_bf16) {
    uint2 b;
    b.x = bf16_bits(v.x) | static_cast<uint32_t>(bf16_bits(v.y)) << 16;
    b.y = bf16_bits(v.z) | static_cast<uint32_t>(bf16_bits(v.w)) << 16;
    static_cast<uint2*>(p.out)[i] = b;
  } else {
    static_cast<float4*>(p.out)[i] = v;
  }
}

}  // namespace cq
