// cq_i8.cu -- host side of the INT8 operators: cq_gemm_i8, cq_linear_i8 and
// the INT8 MoE layer.  Part of libcq's single translation unit.
#include <cuda_runtime.h>

#include "cq.h"
#include "cq_hooks_i8.h"
#include "cq_host.h"
#include "cq_i8.cuh"
#include "cq_i8_group.cuh"
#include "cq_i8_tc.cuh"

namespace cq {

constexpr int kI8Devices = 64;            // devices whose properties are remembered
constexpr int64_t kI8MaxK = 131072;       // one staged row always fits shared memory
static_assert(kI8SmemLimit - 2048 - kI8AccBytes - kI8MinSlots * kI8UnitBytes -
                      i8_plan_bytes(kI8MaxRoutes, kI8MaxExperts) >=
                  i8_row_stride(kI8MaxK),
              "one row");

// What the test hooks choose; a call's own values.
struct I8Hook {
  int path = CQ_I8_AUTO;
  uint64_t timeout_ns = kDefaultTimeoutNs;
  int withhold = 0;
};

// The shared memory of a streaming kernel beside its static arrays: a ring of
// units, `tokens` staged rows, the accumulators, and (MoE) the plan.
constexpr int kI8Smem = kI8SmemLimit - 2048;

// Tokens of one pass: as many as leave room for 12 units (96 KB: what an SM
// needs on its way to take its share of the HBM's rate), or 8 or 4 where long
// rows leave no room for a few tokens beside them.
static int i8_tokens_per_pass(int64_t K, int plan) {
  const int smem = kI8Smem - plan - kI8AccBytes, stride = i8_row_stride(K);
  int n = (smem - 12 * kI8UnitBytes) / stride;
  if (n < 4) n = (smem - 8 * kI8UnitBytes) / stride;
  if (n < 1) n = (smem - kI8MinSlots * kI8UnitBytes) / stride;
  return n < kI8MaxTokens ? n : kI8MaxTokens;
}

template <typename Params>
static int i8_layout(Params& p, int tokens, int64_t K, int plan, uint64_t timeout_ns,
                     bool withhold) {
  p.stride = i8_row_stride(K);
  const int rest = kI8Smem - plan - kI8AccBytes - tokens * p.stride;
  const int slots = rest / kI8UnitBytes < kI8MaxSlots ? rest / kI8UnitBytes : kI8MaxSlots;
  p.slots = slots / kI8MinSlots * kI8MinSlots;   // a multiple of the producers, and even
  p.xs_off = p.slots * kI8UnitBytes;
  p.acc_off = p.xs_off + tokens * p.stride;
  p.timeout_ns = timeout_ns;
  p.withhold = withhold;
  return p.acc_off + kI8AccBytes + plan;
}

static int validate_i8(int64_t M, int64_t N, int64_t K, int epilogue, int out_dtype) {
  if (M < 0 || N < 0 || K <= 0) return CQ_ERR_INVALID_ARG;
  if (epilogue != CQ_EPI_NONE && epilogue != CQ_EPI_SWIGLU) return CQ_ERR_INVALID_ARG;
  if (out_dtype != CQ_DTYPE_F32 && out_dtype != CQ_DTYPE_BF16) return CQ_ERR_INVALID_ARG;
  if (K % 16 != 0 || K > kI8MaxK) return CQ_ERR_UNSUPPORTED;
  if (epilogue == CQ_EPI_SWIGLU && N % 2 != 0) return CQ_ERR_UNSUPPORTED;
  if (M > (int64_t)1 << 24 || N > (int64_t)1 << 24) return CQ_ERR_UNSUPPORTED;
  return CQ_OK;
}

template <int SRC>
static int i8_linear(I8LinearParams p, const I8Hook& hook, int sms, cudaStream_t s) {
  static std::atomic<uint64_t> smem_set{0};
  if (!ensure_smem_limit(i8_linear_kernel<SRC>, kI8Smem, smem_set)) return CQ_ERR_CUDA;
  const int rows = p.swiglu ? p.N / 2 : p.N;
  const int smem = i8_layout(p, p.M, p.K, 0, hook.timeout_ns, hook.withhold);
  return launch_pdl(i8_linear_kernel<SRC>, dim3(rows < sms ? rows : sms), dim3(kI8Threads), smem,
                    s, p);
}

// ---------------------------------------------------------------------------
// the tensor-core product
// ---------------------------------------------------------------------------
struct I8TcPlan {
  bool pair;
  int NT, split;             // tokens of a tile, CTAs per tile (split kernel)
  int n_rt, n_tt, nkb;
  int main_tiles, cut;       // pair kernel: whole tiles, parts of the others
};

static size_t i8_round256(size_t v) { return (v + 255) / 256 * 256; }

// Products streamed from memory: up to 8 tokens, one block of MMA columns, as
// long as their rows fit beside the ring.  6144 x 7168 with SwiGLU takes 10.3
// us at 2 tokens and 12.1 at 8; on the tensor cores 12.5 at 16, and 3 us more
// for rows that have to be quantized first.
static bool i8_streams(int64_t M, int64_t K) { return M <= 8 && M <= i8_tokens_per_pass(K, 0); }

// Clusters of `s` CTAs of the split kernel that run at once (a GPC's SMs need
// not divide evenly): asked once per device and size.
static int i8_clusters_at_once(int s, int sms) {
  static std::atomic<int> known[kI8Devices][kTcMaxSplit + 1];
  int dev = 0;
  if (s == 1 || cudaGetDevice(&dev) != cudaSuccess || dev >= kI8Devices) return sms / s;
  int n = known[dev][s].load(std::memory_order_relaxed);
  if (n > 0) return n;
  static std::atomic<uint64_t> smem_set{0};
  if (!ensure_smem_limit(i8_split_kernel<128>, I8SplitCfg<128>::SMEM, smem_set)) return sms / s;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(sms / s * s));
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = I8SplitCfg<128>::SMEM;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(s);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, i8_split_kernel<128>, &cfg) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return sms / s;
  }
  known[dev][s].store(n, std::memory_order_relaxed);
  return n;
}

// The cheapest kernel and tile by an estimate in cycles.  A block of K of a
// CTA takes the time of its MMAs (2 cycles per token) or of its copies; a
// launch at least the weights' time in HBM (about 3400 bytes a cycle).  The
// copies were measured at 520 cycles a block for 20 KB, 560 for 24 KB and 625
// for 32 KB with all SMs reading (11 to 13 TB/s out of L2: giving the
// activations a producer warp of their own changed nothing).  Over sweeps at
// 24 to 4096 tokens of 6144 x 7168, 7168 x 2048 and 2048 x 7168 the choice is
// within 10% of the best tile and split; tiles of fewer than 128 rows never won.
static int64_t i8_block_cost(int nt, int rows_loaded) {
  const int64_t mma = 2 * nt, copies = 340 + rows_loaded * kTcBlock / 115;
  return mma > copies ? mma : copies;
}

// `path`: CQ_I8_AUTO, or the kernel to choose the tile of.
static I8TcPlan i8_tc_plan(int64_t M, int64_t N, int64_t K, int epilogue, int sms, int path) {
  const bool sw = epilogue == CQ_EPI_SWIGLU;
  const int64_t out = sw ? N / 2 : N;
  const int64_t nkb = (K + kTcBlock - 1) / kTcBlock, hbm = N * K / 3400;
  I8TcPlan best = {};
  int64_t cost = INT64_MAX;
  auto consider = [&](bool pair, int nt, int split, int64_t n_rt, int64_t n_tt, int64_t main,
                      int cut, int64_t c) {
    if (c >= cost || (path != CQ_I8_AUTO && pair != (path == CQ_I8_PAIR))) return;
    cost = c;
    best = {pair, nt, split, static_cast<int>(n_rt), static_cast<int>(n_tt),
            static_cast<int>(nkb), static_cast<int>(main), cut};
  };
  const int64_t per2 = sw ? kRows : 2 * kRows, n_rt2 = (out + per2 - 1) / per2;
  const int64_t units = sms / 2;
  for (int nt = 256; nt >= 128; nt -= 32) {
    const int64_t n_tt = (M + nt - 1) / nt, tiles = n_rt2 * n_tt;
    const int64_t block = i8_block_cost(nt, kRows + nt / 2);
    const int64_t main = tiles / units * units;
    for (int cut = 1; cut <= 4; cut *= 2) {
      if (nt / cut % 32 != 0) break;
      const int64_t rest = ((tiles - main) * cut + units - 1) / units;
      int64_t c = main / units * nkb * block +
                  rest * nkb * i8_block_cost(nt / cut, kRows + nt / cut / 2);
      c = (c > hbm ? c : hbm) + 16000 + 16 * (nt / cut);
      consider(true, nt, 1, n_rt2, n_tt, main, cut, c);
    }
  }
  const int64_t per = sw ? kRows / 2 : kRows, n_rt = (out + per - 1) / per;
  for (int nt = 32; nt <= 128; nt *= 2) {
    const int64_t n_tt = (M + nt - 1) / nt;
    for (int s = 1; s <= kTcMaxSplit && s <= nkb; ++s) {
      const int at_once = i8_clusters_at_once(s, sms);
      const int64_t rounds = (n_rt * n_tt + at_once - 1) / at_once;
      int64_t c = rounds * ((nkb + s - 1) / s) * i8_block_cost(nt, kRows + nt);
      c = (c > hbm ? c : hbm) + rounds * (7500 + 16 * nt) + (s > 1 ? 1500 + 16 * nt : 0);
      consider(false, nt, s, n_rt, n_tt, n_rt * n_tt, 1, c);
    }
  }
  return best;
}

static int i8_encode(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims,
                     const cuuint64_t* strides, const cuuint32_t* box) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return CQ_ERR_CUDA;
  cuuint32_t estr[5] = {1u, 1u, 1u, 1u, 1u};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, static_cast<cuuint32_t>(rank),
                  const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? CQ_OK : CQ_ERR_CUDA;
}

// int8 [rows][K] as boxes of 128 bytes x box_rows rows, 128-byte swizzle.
// Everything outside reads 0.
static int encode_i8_rows(CUtensorMap* map, const void* base, int64_t rows, int64_t K,
                          int box_rows) {
  const cuuint64_t k = static_cast<cuuint64_t>(K);
  const cuuint64_t dims[2] = {k, static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {k};
  const cuuint32_t box[2] = {kTcBlock, static_cast<cuuint32_t>(box_rows)};
  return i8_encode(map, base, 2, dims, strides, box);
}

// Gate and up rows (each `out` of them) in alternating groups of 8: 8 rows of
// both halves per box, and `groups` of these (groups == 0: a map for one at a
// time, which also takes `out` that is not a multiple of 8).
static int encode_i8_gate_up(CUtensorMap* map, const void* base, int64_t out, int64_t K,
                             int groups) {
  const cuuint64_t k = static_cast<cuuint64_t>(K), h = static_cast<cuuint64_t>(out);
  if (groups == 0) {
    const cuuint64_t dims[3] = {k, h, 2};
    const cuuint64_t strides[2] = {k, h * k};
    const cuuint32_t box[3] = {kTcBlock, 8, 2};
    return i8_encode(map, base, 3, dims, strides, box);
  }
  const cuuint64_t dims[4] = {k, 8, 2, h / 8};
  const cuuint64_t strides[3] = {k, h * k, 8 * k};
  const cuuint32_t box[4] = {kTcBlock, 8, 2, static_cast<cuuint32_t>(groups)};
  return i8_encode(map, base, 4, dims, strides, box);
}

template <int NT>
static int launch_i8_split(const I8TcParams& p, const CUtensorMap& xmap, const CUtensorMap& wmap,
                           cudaStream_t s) {
  static std::atomic<uint64_t> smem_set{0};
  if (!ensure_smem_limit(i8_split_kernel<NT>, I8SplitCfg<NT>::SMEM, smem_set)) return CQ_ERR_CUDA;
  return launch_pdl_cluster(i8_split_kernel<NT>,
                            dim3(static_cast<unsigned>(p.n_rt * p.n_tt * p.split)),
                            dim3(kTcThreads), I8SplitCfg<NT>::SMEM, p.split, s, p, xmap, wmap);
}

static int launch_i8_pair(const I8TcParams& p, const CUtensorMap& xmap, const CUtensorMap& xtail,
                          const CUtensorMap& wmap, int sms, cudaStream_t s) {
  static std::atomic<uint64_t> smem_set{0};
  if (!ensure_smem_limit(i8_pair_kernel, I8PairCfg::SMEM, smem_set)) return CQ_ERR_CUDA;
  const int tiles = p.main_tiles + (p.n_rt * p.n_tt - p.main_tiles) * p.cut, units = sms / 2;
  return launch_pdl_cluster(i8_pair_kernel, dim3(2u * (tiles < units ? tiles : units)),
                            dim3(kTcThreads), I8PairCfg::SMEM, 2, s, p, xmap, xtail, wmap);
}

static int i8_tc(const I8LinearParams& q, const I8TcPlan& g, const int8_t* xq,
                 const float* absmax, bool early_w, const I8Hook& hook, int sms,
                 cudaStream_t s) {
  CUtensorMap xmap, xtail, wmap;
  int st = encode_i8_rows(&xmap, xq, q.M, q.K, g.pair ? g.NT / 2 : g.NT);
  if (st != CQ_OK) return st;
  if (g.pair) {
    st = encode_i8_rows(&xtail, xq, q.M, q.K, g.NT / g.cut / 2);
    if (st != CQ_OK) return st;
  }
  const int64_t half = q.N / 2;
  const bool one_box = q.swiglu && half % 8 == 0;
  st = !q.swiglu ? encode_i8_rows(&wmap, q.w, q.N, q.K, kRows)
                 : encode_i8_gate_up(&wmap, q.w, half, q.K, one_box ? kRows / 16 : 0);
  if (st != CQ_OK) return st;
  I8TcParams p = {};
  p.absmax = absmax;
  p.wscale = q.wscale;
  p.y = q.y;
  p.M = q.M;
  p.N = q.N;
  p.swiglu = q.swiglu;
  p.out_bf16 = q.out_bf16;
  p.n_rt = g.n_rt;
  p.n_tt = g.n_tt;
  p.nkb = g.nkb;
  p.split = g.split;
  p.w_boxes = one_box ? 1 : kRows / 16;
  p.nt = g.NT;
  p.main_tiles = g.main_tiles;
  p.cut = g.cut;
  p.tail_nt = g.NT / g.cut;
  p.early_w = early_w;
  p.withhold = hook.withhold != 0;
  p.timeout_ns = hook.timeout_ns;
  if (g.pair) return launch_i8_pair(p, xmap, xtail, wmap, sms, s);
  switch (g.NT) {
    case 32: return launch_i8_split<32>(p, xmap, wmap, s);
    case 64: return launch_i8_split<64>(p, xmap, wmap, s);
    default: return launch_i8_split<128>(p, xmap, wmap, s);
  }
}

static int i8_gemm_impl(const void* x, const float* absmax, int64_t M, const int8_t* wq,
                        const float* wscale, int64_t N, int64_t K, int epilogue, int out_dtype,
                        void* y, void* workspace, size_t ws_bytes, bool codes, cudaStream_t s,
                        const I8Hook& hook = {}) {
  const int st = validate_i8(M, N, K, epilogue, out_dtype);
  if (st != CQ_OK) return st;
  if (M == 0 || N == 0) return CQ_OK;
  if (!x || !wq || !wscale || !y || (codes && !absmax)) return CQ_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(wq, 16) || !aligned(wscale, 4) || !aligned(y, 16) ||
      (codes && !aligned(absmax, 4)))
    return CQ_ERR_UNSUPPORTED;
  const int sms = num_sms();
  if (sms <= 0) return CQ_ERR_CUDA;
  I8LinearParams p = {};
  p.x = x;
  p.absmax = absmax;
  p.w = wq;
  p.wscale = wscale;
  p.y = y;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.swiglu = epilogue == CQ_EPI_SWIGLU;
  p.out_bf16 = out_dtype == CQ_DTYPE_BF16;
  const bool streams = i8_streams(M, K);
  if (hook.path == CQ_I8_STREAM && !streams) return CQ_ERR_UNSUPPORTED;
  if (streams && (hook.path == CQ_I8_AUTO || hook.path == CQ_I8_STREAM))
    return codes ? i8_linear<I8_SRC_CODES>(p, hook, sms, s)
                 : i8_linear<I8_SRC_BF16>(p, hook, sms, s);
  const I8TcPlan g = i8_tc_plan(M, N, K, epilogue, sms, hook.path);
  if (static_cast<int64_t>(g.n_rt) * g.n_tt * g.split >= (int64_t)1 << 28)
    return CQ_ERR_UNSUPPORTED;
  const int8_t* xq = static_cast<const int8_t*>(x);
  if (!codes) {
    const size_t o_absmax = i8_round256(static_cast<size_t>(M) * K);
    if (!workspace || ws_bytes < o_absmax + static_cast<size_t>(M) * sizeof(float))
      return CQ_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return CQ_ERR_UNSUPPORTED;
    int8_t* q = static_cast<int8_t*>(workspace);
    float* a = reinterpret_cast<float*>(q + o_absmax);
    const int e = launch_pdl(quant_rows_vec_kernel, dim3(static_cast<unsigned>(M)),
                             dim3(kQvThreads), 0, s, static_cast<const uint16_t*>(x), p.M, p.K, q,
                             a);
    if (e != CQ_OK) return e;
    xq = q;
    absmax = a;
  }
  // behind the quantization the weights may be fetched early: it ends only
  // after the kernel before it
  return i8_tc(p, g, xq, absmax, !codes, hook, sms, s);
}

// ---------------------------------------------------------------------------
// the MoE layer
// ---------------------------------------------------------------------------
struct I8MoePlan {
  int64_t T;                 // tokens of one launch
  int nt;                    // routes per tile on the tensor cores; 0: streamed
  int tiles;                 // ... and tiles, at most
  size_t o_y, o_xq, o_sx, o_route, o_tile, o_n, total;         // h comes first
};

// Streamed or sorted?  Streaming takes one launch less per stage and reads the
// routes' experts at the HBM's rate, but a CTA stages activations for every
// chunk it works on, and a launch holds kI8MaxRoutes routes: a second one
// would read most experts again.  Sorted tiles cost some 5 us more at a few
// routes and next to nothing per expert.  Measured on weights not in L2,
// streamed / sorted in us (uniform routes):
//   * up to 32 routes, which one warp plans: 13.7 / 17.5 (4 experts 512 x 256,
//     32 routes), 19.6 / 25.4 (16 of 1024 x 1024), 112 / 130 (16 of 7168 x
//     2048); just above, 20.4 / 17.6 (16 of 512 x 256, 48 routes);
//   * experts of 2 MB and more, up to 5 routes each: 54 / 55 (128 routes of 32
//     experts 2048 x 1024), 231 / 238 (of 32 experts 7168 x 2048), 1665 / 1656
//     (1024 of 256); at 8 each 255 / 242 (256 of 32);
//   * experts of 0.5 to 2 MB, up to 128 routes and 5 each: within 12%, 34.3 /
//     31.2 at 96 and 44.6 / 42.4 at 128 routes (64 and 128 experts 1024 x 512),
//     and ahead when some routes are dropped (22.9 / 24.8: 108 routes, three
//     quarters dropped, 50 of 336 x 1040).  Above, 55 / 49 at 256.  Smaller ones
//     leave no such range: 24.6 / 17.5 at 64 routes of 128 experts 256 x 128;
//   * in several streamed launches: 2472 / 1720 at 144 tokens, top 8 of 256
//     experts 7168 x 2048; 15976 / 5793 at 256 tokens, top 16 of 896.
// Dropped routes count in all this: the host does not know them.
// Tiles of 64 routes up to 96 each: 531 us against 562 with 128 at 48 routes
// each (64 experts 7168 x 2048), 720 against 722 at 96, 1007 against 831 at
// 128.  (256 routes, one CTA per SM: 1470 us at 256 each, 1293 with 128.)
static bool i8_moe_sorted(int64_t routes, int64_t E, int64_t H, int64_t I, int k) {
  const int64_t bytes = 3 * H * I;
  if (routes <= 32) return false;
  if (routes > kI8MaxRoutes / k * k || bytes < (1 << 19)) return true;
  return routes > 5 * E || (bytes < (2 << 20) && routes > 128);
}

// Routes of one sorted launch: every further launch reads the experts again,
// so 128 for each of them (then the products take as long as the weights), at
// most as many as keep the workspace near 3 GB for rows of 7168.  With 16384
// for any number of experts 2048 tokens, top 16 of 896 experts 7168 x 2048,
// took 13.1 ms instead of 7.0.
static int64_t i8_group_routes(int64_t E) {
  const int64_t r = 128 * E;
  return r < 16384 ? 16384 : (r < 65536 ? r : 65536);
}

static I8MoePlan i8_moe_plan(int64_t T, int k, int E, int64_t H, int64_t I,
                             int path = CQ_I8_AUTO) {
  I8MoePlan m = {};
  const int64_t e = E;
  const bool sorted =
      path == CQ_I8_AUTO ? i8_moe_sorted(T * k, E, H, I, k) : path == CQ_I8_SORTED;
  const int64_t most = (sorted ? i8_group_routes(e) : kI8MaxRoutes) / k;
  m.T = T < most ? T : most;
  const size_t R = static_cast<size_t>(m.T) * k;
  if (sorted) m.nt = m.T * k > 96 * e ? 128 : 64;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += i8_round256(bytes);
    return o;
  };
  take(R * I * sizeof(float));
  m.o_y = take(R * H * sizeof(float));
  if (m.nt) {
    m.tiles = static_cast<int>(R / m.nt + (R < static_cast<size_t>(E) ? R : E));
    m.o_xq = take(R * (H > I ? H : I));
    m.o_sx = take(R * sizeof(float));
    m.o_route = take(R * sizeof(int));
    // room for the smallest tiles: no fewer tokens need a larger workspace
    m.o_tile = take((R / 64 + (R < static_cast<size_t>(E) ? R : E)) * sizeof(int4));
    m.o_n = take(2 * sizeof(int));
  }
  m.total = at;
  return m;
}

static int validate_i8_moe(int64_t T, int k, int E, int64_t H, int64_t I) {
  if (T < 0 || k <= 0 || E <= 0 || H <= 0 || I <= 0) return CQ_ERR_INVALID_ARG;
  if (E > kI8MaxExperts || k > kI8MaxRoutes) return CQ_ERR_UNSUPPORTED;
  if (H % 16 != 0 || I % 16 != 0 || H > kI8MaxK || I > kI8MaxK) return CQ_ERR_UNSUPPORTED;
  if (T > (int64_t)1 << 24) return CQ_ERR_UNSUPPORTED;
  return CQ_OK;
}

template <bool DOWN, int NB>
static int launch_i8_moe(const I8MoeParams& p, int grid, int smem, cudaStream_t s) {
  static std::atomic<uint64_t> smem_set{0};
  if (!ensure_smem_limit(i8_moe_kernel<DOWN, NB>, kI8Smem, smem_set)) return CQ_ERR_CUDA;
  return launch_pdl(i8_moe_kernel<DOWN, NB>, dim3(grid), dim3(kI8Threads), smem, s, p);
}

// A launch's share of the hook: the one that loses operands has the whole limit.
template <bool DOWN>
static bool i8_stage_withheld(const I8Hook& hook) {
  return hook.withhold == (DOWN ? 2 : 1);
}
template <bool DOWN>
static uint64_t i8_stage_limit(const I8Hook& hook) {
  return hook.withhold == 0 || i8_stage_withheld<DOWN>(hook) ? hook.timeout_ns
                                                             : hook.timeout_ns / 4;
}

template <bool DOWN>
static int i8_moe_stage(I8MoeParams p, const int8_t* w, const float* wscale, const I8Hook& hook,
                        int sms, cudaStream_t s) {
  const int64_t K = DOWN ? p.I : p.H;
  p.w = w;
  p.wscale = wscale;
  // an expert sees a token once as a rule: T <= 8 needs one block of columns
  const int plan = i8_plan_bytes(p.R, p.E);
  p.nt = i8_tokens_per_pass(K, plan);
  if (p.T <= 8 && p.nt > 8) p.nt = 8;
  if (p.R < p.nt) p.nt = p.R;
  // nanoseconds x 10 per row and per route of a row, at 50 bytes a nanosecond
  // and 7 us a pass
  constexpr int rpt = DOWN ? 16 : 8;
  p.wt_row = static_cast<int>((DOWN ? K : 2 * K) / 50) + 1;
  p.wt_route = 70000 / (kI8AccBytes / 64 * rpt);
  p.wt_gap = 35000.f / static_cast<float>(DOWN ? p.H : p.I);
  p.gap_rows = static_cast<int>(3500 * 50 / (DOWN ? K : 2 * K));
  const int smem = i8_layout(p, p.nt, K, plan, i8_stage_limit<DOWN>(hook),
                             i8_stage_withheld<DOWN>(hook));
  return p.nt <= 8 ? launch_i8_moe<DOWN, 1>(p, sms, smem, s)
                   : launch_i8_moe<DOWN, 2>(p, sms, smem, s);
}

// The weights [E][rows][K] of a stage: boxes of 128 rows of an expert (down),
// or of 8 groups of 8 gate rows and the 8 up rows that belong to them.  What
// is outside an expert's rows reads 0.
static int encode_i8_experts(CUtensorMap* map, const int8_t* w, bool down, int64_t E, int64_t rows,
                             int64_t K) {
  const cuuint64_t k = static_cast<cuuint64_t>(K), n = static_cast<cuuint64_t>(rows),
                   e = static_cast<cuuint64_t>(E);
  if (down) {
    const cuuint64_t dims[3] = {k, n, e};
    const cuuint64_t strides[2] = {k, n * k};
    const cuuint32_t box[3] = {kTcBlock, kRows, 1};
    return i8_encode(map, w, 3, dims, strides, box);
  }
  const cuuint64_t dims[5] = {k, 8, 2, n / 8, e};
  const cuuint64_t strides[4] = {k, n * k, 8 * k, 2 * n * k};
  const cuuint32_t box[5] = {kTcBlock, 8, 2, kRows / 16, 1};
  return i8_encode(map, w, 5, dims, strides, box);
}

template <int NT, bool DOWN>
static int i8_group_stage(I8GroupParams p, const int8_t* w, const float* wscale,
                          const I8Hook& hook, int tiles, cudaStream_t s) {
  static std::atomic<uint64_t> smem_set{0};
  if (!ensure_smem_limit(i8_group_kernel<NT, DOWN>, I8GroupCfg<NT>::SMEM, smem_set))
    return CQ_ERR_CUDA;
  const int64_t K = DOWN ? p.I : p.H, rows = DOWN ? p.H : p.I, per = DOWN ? kRows : kRows / 2;
  CUtensorMap xmap, wmap;
  int st = encode_i8_rows(&xmap, p.xq, p.R, K, NT);
  if (st == CQ_OK) st = encode_i8_experts(&wmap, w, DOWN, p.E, rows, K);
  if (st != CQ_OK) return st;
  p.wscale = wscale;
  p.withhold = i8_stage_withheld<DOWN>(hook);
  p.timeout_ns = i8_stage_limit<DOWN>(hook);
  p.n_rt = static_cast<int>((rows + per - 1) / per);
  p.nkb = static_cast<int>((K + kTcBlock - 1) / kTcBlock);
  st = launch_pdl(i8_group_rows_kernel<DOWN>, dim3(static_cast<unsigned>(p.R)),
                  dim3(kGpRowThreads), 0, s, p);
  if (st != CQ_OK) return st;
  return launch_pdl(i8_group_kernel<NT, DOWN>,
                    dim3(static_cast<unsigned>(tiles) * static_cast<unsigned>(p.n_rt)),
                    dim3(kTcThreads), I8GroupCfg<NT>::SMEM, s, p, xmap, wmap);
}

template <int NT>
static int i8_group_nt(const I8GroupParams& p, const int8_t* w_gu, const float* s_gu,
                       const int8_t* w_dn, const float* s_dn, const I8Hook& hook, int tiles,
                       cudaStream_t s) {
  const int st = i8_group_stage<NT, false>(p, w_gu, s_gu, hook, tiles, s);
  return st != CQ_OK ? st : i8_group_stage<NT, true>(p, w_dn, s_dn, hook, tiles, s);
}

// The routes' outputs of `q`'s tokens on the tensor cores.
static int i8_group(const I8MoeParams& q, const I8MoePlan& m, uint8_t* ws, const int8_t* w_gu,
                    const float* s_gu, const int8_t* w_dn, const float* s_dn,
                    const I8Hook& hook, cudaStream_t s) {
  static std::atomic<uint64_t> smem_set{0};
  if (!ensure_smem_limit(i8_group_plan_kernel, kI8MaxExperts * 4, smem_set)) return CQ_ERR_CUDA;
  I8GroupParams p = {};
  p.tokens = q.tokens;
  p.ids = q.ids;
  p.h = q.h;
  p.y = q.y;
  p.xq = reinterpret_cast<int8_t*>(ws + m.o_xq);
  p.sx = reinterpret_cast<float*>(ws + m.o_sx);
  p.route = reinterpret_cast<int*>(ws + m.o_route);
  p.tile = reinterpret_cast<int4*>(ws + m.o_tile);
  p.n = reinterpret_cast<int*>(ws + m.o_n);
  p.k = q.k;
  p.R = q.R;
  p.E = q.E;
  p.H = static_cast<int>(q.H);
  p.I = static_cast<int>(q.I);
  p.nt = m.nt;
  p.clear_y = q.clear_y;
  const int st = launch_pdl(i8_group_plan_kernel, dim3(1), dim3(kGpPlanThreads), p.E * 4, s, p);
  if (st != CQ_OK) return st;
  switch (m.nt) {
    case 64: return i8_group_nt<64>(p, w_gu, s_gu, w_dn, s_dn, hook, m.tiles, s);
    default: return i8_group_nt<128>(p, w_gu, s_gu, w_dn, s_dn, hook, m.tiles, s);
  }
}

static int i8_moe_impl(const uint16_t* tokens, int64_t T, const int32_t* topk_ids,
                       const float* topk_w, int k, int E, const int8_t* w_gu, const float* s_gu,
                       const int8_t* w_dn, const float* s_dn, int64_t H, int64_t I, int out_dtype,
                       float* route_out, void* out, void* workspace, size_t ws_bytes,
                       cudaStream_t s, const I8Hook& hook = {}) {
  int st = validate_i8_moe(T, k, E, H, I);
  if (st != CQ_OK) return st;
  if (out_dtype != CQ_DTYPE_F32 && out_dtype != CQ_DTYPE_BF16) return CQ_ERR_INVALID_ARG;
  if (T == 0) return CQ_OK;
  if (!tokens || !topk_ids || !w_gu || !s_gu || !w_dn || !s_dn || !workspace)
    return CQ_ERR_INVALID_ARG;
  if (out && !topk_w) return CQ_ERR_INVALID_ARG;
  if (!aligned(tokens, 16) || !aligned(topk_ids, 4) || !aligned(w_gu, 16) || !aligned(s_gu, 4) ||
      !aligned(w_dn, 16) || !aligned(s_dn, 4) || !aligned(workspace, 256) ||
      (topk_w && !aligned(topk_w, 4)) || (route_out && !aligned(route_out, 16)) ||
      (out && !aligned(out, 16)))
    return CQ_ERR_UNSUPPORTED;
  const int sms = num_sms();
  if (sms <= 0) return CQ_ERR_CUDA;
  const I8MoePlan m = i8_moe_plan(T, k, E, H, I, hook.path);
  if (ws_bytes < m.total) return CQ_ERR_WORKSPACE;
  if (!out && !route_out) return CQ_OK;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int os = out_dtype == CQ_DTYPE_BF16 ? 2 : 4;
  for (int64_t t = 0; t < T; t += m.T) {
    I8MoeParams p = {};
    p.T = static_cast<int>(T - t < m.T ? T - t : m.T);
    p.k = k;
    p.R = p.T * k;
    p.E = E;
    p.H = H;
    p.I = I;
    p.tokens = tokens + t * H;
    p.ids = topk_ids + t * k;
    p.topk_w = topk_w ? topk_w + t * k : nullptr;
    p.h = reinterpret_cast<float*>(ws);
    p.y = route_out ? route_out + t * k * H : reinterpret_cast<float*>(ws + m.o_y);
    p.out = out ? static_cast<uint8_t*>(out) + t * H * os : nullptr;
    p.out_bf16 = out_dtype == CQ_DTYPE_BF16;
    p.clear_y = route_out != nullptr;
    if (m.nt) {
      st = i8_group(p, m, ws, w_gu, s_gu, w_dn, s_dn, hook, s);
    } else {
      st = i8_moe_stage<false>(p, w_gu, s_gu, hook, sms, s);
      if (st == CQ_OK) st = i8_moe_stage<true>(p, w_dn, s_dn, hook, sms, s);
    }
    if (st != CQ_OK) return st;
    if (!out) continue;
    const int64_t n = p.T * (H / 4);
    st = launch_pdl(i8_combine_kernel,
                    dim3(static_cast<unsigned>((n + kI8CombineThreads - 1) / kI8CombineThreads)),
                    dim3(kI8CombineThreads), 0, s, p);
    if (st != CQ_OK) return st;
  }
  return CQ_OK;
}

}  // namespace cq

using namespace cq;

extern "C" CQ_API size_t cq_gemm_i8_workspace_size(int64_t M, int64_t N, int64_t K, int epilogue) {
  if (validate_i8(M, N, K, epilogue, CQ_DTYPE_F32) != CQ_OK || M == 0 || N == 0 || i8_streams(M, K))
    return 0;
  return i8_round256(static_cast<size_t>(M) * K) +
         i8_round256(static_cast<size_t>(M) * sizeof(float));
}

extern "C" CQ_API int cq_gemm_i8(const int8_t* xq, const float* absmax, int64_t M,
                                 const int8_t* wq, const float* wscale, int64_t N, int64_t K,
                                 int epilogue, int out_dtype, void* y, void* workspace,
                                 size_t ws_bytes, void* stream) {
  return i8_gemm_impl(xq, absmax, M, wq, wscale, N, K, epilogue, out_dtype, y, workspace,
                      ws_bytes, true, static_cast<cudaStream_t>(stream));
}

extern "C" CQ_API int cq_linear_i8(const uint16_t* x, int64_t M, const int8_t* wq,
                                   const float* wscale, int64_t N, int64_t K, int epilogue,
                                   int out_dtype, void* y, void* workspace, size_t ws_bytes,
                                   void* stream) {
  return i8_gemm_impl(x, nullptr, M, wq, wscale, N, K, epilogue, out_dtype, y, workspace,
                      ws_bytes, false, static_cast<cudaStream_t>(stream));
}

extern "C" CQ_API size_t cq_moe_i8_workspace_size(int64_t T, int k, int E, int64_t H, int64_t I) {
  if (validate_i8_moe(T, k, E, H, I) != CQ_OK) return 0;
  return i8_moe_plan(T, k, E, H, I).total;
}

extern "C" CQ_API int cq_moe_i8(const uint16_t* tokens, int64_t T, const int32_t* topk_ids,
                                const float* topk_w, int k, int E, const int8_t* w_gu,
                                const float* s_gu, const int8_t* w_dn, const float* s_dn,
                                int64_t H, int64_t I, int out_dtype, float* route_out, void* out,
                                void* workspace, size_t ws_bytes, void* stream) {
  return i8_moe_impl(tokens, T, topk_ids, topk_w, k, E, w_gu, s_gu, w_dn, s_dn, H, I, out_dtype,
                     route_out, out, workspace, ws_bytes, static_cast<cudaStream_t>(stream));
}

// ---------------------------------------------------------------------------
// test hooks (declared in cq_hooks_i8.h)
// ---------------------------------------------------------------------------
static I8Hook i8_hook(int path, uint64_t timeout_ns, int withhold) {
  I8Hook hook;
  hook.path = path;
  if (timeout_ns) hook.timeout_ns = timeout_ns;
  hook.withhold = withhold;
  return hook;
}

extern "C" CQ_API int cq_test_product_i8_path(int64_t M, int64_t N, int64_t K, int epilogue) {
  if (validate_i8(M, N, K, epilogue, CQ_DTYPE_F32) != CQ_OK || M == 0 || N == 0) return 0;
  if (i8_streams(M, K)) return CQ_I8_STREAM;
  int sms = num_sms();
  if (sms <= 0) sms = 148;
  return i8_tc_plan(M, N, K, epilogue, sms, CQ_I8_AUTO).pair ? CQ_I8_PAIR : CQ_I8_SPLIT;
}

extern "C" CQ_API int cq_test_product_i8(const void* x, const float* absmax, int64_t M,
                                         const int8_t* wq, const float* wscale, int64_t N,
                                         int64_t K, int epilogue, int out_dtype, void* y,
                                         void* workspace, size_t ws_bytes, int path,
                                         uint64_t timeout_ns, int withhold, void* stream) {
  if (path < CQ_I8_AUTO || path > CQ_I8_PAIR) return CQ_ERR_INVALID_ARG;
  return i8_gemm_impl(x, absmax, M, wq, wscale, N, K, epilogue, out_dtype, y, workspace, ws_bytes,
                      absmax != nullptr, static_cast<cudaStream_t>(stream),
                      i8_hook(path, timeout_ns, withhold));
}

static bool i8_moe_path_ok(int path) {
  return path == CQ_I8_AUTO || path == CQ_I8_STREAM || path == CQ_I8_SORTED;
}

extern "C" CQ_API int cq_test_moe_i8_path(int64_t T, int k, int E, int64_t H, int64_t I,
                                          int64_t* tokens_per_launch) {
  if (validate_i8_moe(T, k, E, H, I) != CQ_OK || T == 0) return 0;
  const I8MoePlan m = i8_moe_plan(T, k, E, H, I);
  if (tokens_per_launch) *tokens_per_launch = m.T;
  return m.nt ? CQ_I8_SORTED : CQ_I8_STREAM;
}

extern "C" CQ_API size_t cq_test_moe_i8_workspace_size(int64_t T, int k, int E, int64_t H,
                                                       int64_t I, int path) {
  if (validate_i8_moe(T, k, E, H, I) != CQ_OK || !i8_moe_path_ok(path)) return 0;
  return i8_moe_plan(T, k, E, H, I, path).total;
}

extern "C" CQ_API int cq_test_moe_i8(const uint16_t* tokens, int64_t T, const int32_t* topk_ids,
                                     const float* topk_w, int k, int E, const int8_t* w_gu,
                                     const float* s_gu, const int8_t* w_dn, const float* s_dn,
                                     int64_t H, int64_t I, int out_dtype, float* route_out,
                                     void* out, void* workspace, size_t ws_bytes, int path,
                                     uint64_t timeout_ns, int withhold, void* stream) {
  if (!i8_moe_path_ok(path)) return CQ_ERR_INVALID_ARG;
  return i8_moe_impl(tokens, T, topk_ids, topk_w, k, E, w_gu, s_gu, w_dn, s_dn, H, I, out_dtype,
                     route_out, out, workspace, ws_bytes, static_cast<cudaStream_t>(stream),
                     i8_hook(path, timeout_ns, withhold));
}
