// cq_i8.cu -- host side of the INT8 operators: cq_gemm_i8, cq_linear_i8 and
// the INT8 MoE layer.  Part of libcq's single translation unit.
#include <cuda_runtime.h>

#include "cq.h"
#include "cq_host.h"
#include "cq_i8.cuh"
#include "cq_i8_tc.cuh"

namespace cq {

constexpr int64_t kI8MaxK = 131072;       // one staged row always fits shared memory

// Shared memory left for staged rows beside the accumulators and a kernel's
// static arrays.
constexpr int kI8LinearRowBytes = kI8SmemLimit - 1024 - kI8AccBytes;
constexpr int kI8MoeRowBytes =
    kI8SmemLimit - 1024 - kI8AccBytes - static_cast<int>(sizeof(I8PlanSmem));

static int i8_tokens_per_pass(int64_t K, int row_bytes) {
  const int n = row_bytes / i8_row_stride(K);
  return n < kI8MaxTokens ? n : kI8MaxTokens;
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

template <int SRC, int NB>
static int launch_i8_linear(const I8LinearParams& p, int grid, cudaStream_t s) {
  static std::atomic<uint64_t> smem_set{0};
  if (!ensure_smem_limit(i8_linear_kernel<SRC, NB>, kI8SmemLimit - 1024, smem_set))
    return CQ_ERR_CUDA;
  return launch_pdl(i8_linear_kernel<SRC, NB>, dim3(grid), dim3(kI8Threads),
                    p.acc_off + kI8AccBytes, s, p);
}

template <int SRC>
static int i8_linear(I8LinearParams p, int sms, cudaStream_t s) {
  const int64_t M = p.M, rows = p.swiglu ? p.N / 2 : p.N;
  const int es = SRC == I8_SRC_CODES ? 1 : 2, os = p.out_bf16 ? 2 : 4;
  const int nt = i8_tokens_per_pass(p.K, kI8LinearRowBytes);
  const int grid = static_cast<int>(rows < sms ? rows : sms);
  p.stride = i8_row_stride(p.K);
  for (int64_t m = 0; m < M; m += nt) {
    I8LinearParams q = p;
    q.M = static_cast<int>(M - m < nt ? M - m : nt);
    q.x = static_cast<const uint8_t*>(p.x) + m * p.K * es;
    q.absmax = p.absmax ? p.absmax + m : nullptr;
    q.y = static_cast<uint8_t*>(p.y) + m * rows * os;
    q.acc_off = q.M * p.stride;
    const int st = q.M <= 8 ? launch_i8_linear<SRC, 1>(q, grid, s)
                            : launch_i8_linear<SRC, 2>(q, grid, s);
    if (st != CQ_OK) return st;
  }
  return CQ_OK;
}

// ---------------------------------------------------------------------------
// the tensor-core product
// ---------------------------------------------------------------------------
// Every workspace of the INT8 operators begins with the same counter area,
// so that one buffer may serve calls of different sizes: counters return to
// zero, and nothing else is ever written there.
constexpr size_t kI8CounterBytes = 16384;

struct I8TcPlan {
  int NT, CG;
  int n_rt, n_tt, nkb, P;
  size_t o_xq, o_absmax, o_partial, total;
};

static size_t i8_round256(size_t v) { return (v + 255) / 256 * 256; }

// Tokens up to which the product is streamed from memory.
static bool i8_streams(int64_t M) { return M <= kI8MaxTokens; }

static I8TcPlan i8_tc_plan(int64_t M, int64_t N, int64_t K, int epilogue, int sms) {
  I8TcPlan g;
  g.NT = M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256;
  g.CG = g.NT == 256 ? 2 : 1;
  const int64_t out = epilogue == CQ_EPI_SWIGLU ? N / 2 : N;
  const int64_t rows = epilogue == CQ_EPI_SWIGLU ? 64 * g.CG : kRows * g.CG;
  g.n_rt = static_cast<int>((out + rows - 1) / rows);
  g.n_tt = static_cast<int>((M + g.NT - 1) / g.NT);
  g.nkb = static_cast<int>((K + kTcBlock - 1) / kTcBlock);
  const int64_t W = static_cast<int64_t>(g.n_rt) * g.n_tt * g.nkb;
  const int units = sms / g.CG;
  g.P = static_cast<int>(W < units ? W : units);
  g.o_xq = kI8CounterBytes;
  g.o_absmax = g.o_xq + i8_round256(static_cast<size_t>(M) * K);
  g.o_partial = g.o_absmax + i8_round256(static_cast<size_t>(M) * sizeof(float));
  g.total = g.o_partial + static_cast<size_t>(2) * g.P * g.CG * g.NT * kRows * sizeof(int);
  return g;
}

// int8 [rows][K] as boxes of 128 bytes x box_rows rows, 128-byte swizzle; with
// halves == 2, box_rows rows of each half of the rows (gate, then up).
// Everything outside reads 0.
static int encode_i8_operand(CUtensorMap* map, const void* base, int64_t rows, int64_t K,
                             int box_rows, int halves) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return CQ_ERR_CUDA;
  const cuuint64_t per = static_cast<cuuint64_t>(rows / halves);
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), per, 2};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(K), per * static_cast<cuuint64_t>(K)};
  cuuint32_t box[3] = {kTcBlock, static_cast<cuuint32_t>(box_rows), 2};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, halves == 2 ? 3u : 2u,
                  const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? CQ_OK : CQ_ERR_CUDA;
}

template <int NT, int CG>
static int launch_i8_tc(const I8TcParams& p, const CUtensorMap& xmap, const CUtensorMap& wmap,
                        cudaStream_t s) {
  using C = I8TcCfg<NT, CG>;
  static std::atomic<uint64_t> smem_set{0};
  if (!ensure_smem_limit(i8_tc_kernel<NT, CG>, C::SMEM, smem_set)) return CQ_ERR_CUDA;
  return launch_pdl_cluster(i8_tc_kernel<NT, CG>, dim3(p.P * CG), dim3(kTcThreads), C::SMEM, CG,
                            s, p, xmap, wmap);
}

static int i8_tc(const I8LinearParams& q, const I8TcPlan& g, const int8_t* xq,
                 const float* absmax, uint8_t* ws, cudaStream_t s) {
  CUtensorMap xmap, wmap;
  int st = encode_i8_operand(&xmap, xq, q.M, q.K, g.NT / g.CG, 1);
  if (st != CQ_OK) return st;
  st = q.swiglu ? encode_i8_operand(&wmap, q.w, q.N, q.K, 16, 2)
                : encode_i8_operand(&wmap, q.w, q.N, q.K, kRows, 1);
  if (st != CQ_OK) return st;
  I8TcParams p = {};
  p.absmax = absmax;
  p.wscale = q.wscale;
  p.y = q.y;
  p.counter = reinterpret_cast<int*>(ws);
  p.partial = reinterpret_cast<int*>(ws + g.o_partial);
  p.M = q.M;
  p.N = q.N;
  p.K = q.K;
  p.swiglu = q.swiglu;
  p.out_bf16 = q.out_bf16;
  p.n_rt = g.n_rt;
  p.n_tt = g.n_tt;
  p.nkb = g.nkb;
  p.P = g.P;
  p.timeout_ns = kDefaultTimeoutNs;
  switch (g.NT) {
    case 32: return launch_i8_tc<32, 1>(p, xmap, wmap, s);
    case 64: return launch_i8_tc<64, 1>(p, xmap, wmap, s);
    case 128: return launch_i8_tc<128, 1>(p, xmap, wmap, s);
    default: return launch_i8_tc<256, 2>(p, xmap, wmap, s);
  }
}

static int i8_gemm_impl(const void* x, const float* absmax, int64_t M, const int8_t* wq,
                        const float* wscale, int64_t N, int64_t K, int epilogue, int out_dtype,
                        void* y, void* workspace, size_t ws_bytes, bool codes, cudaStream_t s) {
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
  if (i8_streams(M))
    return codes ? i8_linear<I8_SRC_CODES>(p, sms, s) : i8_linear<I8_SRC_BF16>(p, sms, s);
  const I8TcPlan g = i8_tc_plan(M, N, K, epilogue, sms);
  if (static_cast<int64_t>(g.n_rt) * g.n_tt >= (int64_t)1 << 31) return CQ_ERR_UNSUPPORTED;
  if (!workspace) return CQ_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return CQ_ERR_UNSUPPORTED;
  if (ws_bytes < g.total) return CQ_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int8_t* xq = static_cast<const int8_t*>(x);
  if (!codes) {
    int8_t* q = reinterpret_cast<int8_t*>(ws + g.o_xq);
    float* a = reinterpret_cast<float*>(ws + g.o_absmax);
    const int e = launch_pdl(quant_rows_vec_kernel, dim3(static_cast<unsigned>(M)),
                             dim3(kQvThreads), 0, s, static_cast<const uint16_t*>(x), p.M, p.K, q,
                             a);
    if (e != CQ_OK) return e;
    xq = q;
    absmax = a;
  }
  return i8_tc(p, g, xq, absmax, ws, s);
}

// ---------------------------------------------------------------------------
// the MoE layer
// ---------------------------------------------------------------------------
struct I8MoePlan {
  int64_t T;                 // tokens of one launch
  size_t o_h, o_y, total;    // the counters come first
};

static I8MoePlan i8_moe_plan(int64_t T, int k, int64_t H, int64_t I) {
  I8MoePlan m;
  const int64_t most = kI8MaxRoutes / k;
  m.T = T < most ? T : most;
  const size_t R = static_cast<size_t>(m.T) * k;
  static_assert(kI8MaxK / kI8CombineRows * sizeof(int) <= kI8CounterBytes, "counter area");
  m.o_h = kI8CounterBytes;
  m.o_y = m.o_h + i8_round256(R * I * sizeof(float));
  m.total = m.o_y + i8_round256(R * H * sizeof(float));
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
static int launch_i8_moe(const I8MoeParams& p, int grid, cudaStream_t s) {
  static std::atomic<uint64_t> smem_set{0};
  if (!ensure_smem_limit(i8_moe_kernel<DOWN, NB>,
                         kI8SmemLimit - 1024 - static_cast<int>(sizeof(I8PlanSmem)), smem_set))
    return CQ_ERR_CUDA;
  return launch_pdl(i8_moe_kernel<DOWN, NB>, dim3(grid), dim3(kI8Threads),
                    p.acc_off + kI8AccBytes, s, p);
}

template <bool DOWN>
static int i8_moe_stage(I8MoeParams p, const int8_t* w, const float* wscale, int sms,
                        cudaStream_t s) {
  const int64_t K = DOWN ? p.I : p.H;
  p.w = w;
  p.wscale = wscale;
  p.stride = i8_row_stride(K);
  // an expert sees a token once as a rule: T <= 8 needs one block of columns
  p.nt = i8_tokens_per_pass(K, kI8MoeRowBytes);
  if (p.T <= 8 && p.nt > 8) p.nt = 8;
  p.acc_off = p.nt * p.stride;
  return p.nt <= 8 ? launch_i8_moe<DOWN, 1>(p, sms, s) : launch_i8_moe<DOWN, 2>(p, sms, s);
}

}  // namespace cq

using namespace cq;

extern "C" CQ_API size_t cq_gemm_i8_workspace_size(int64_t M, int64_t N, int64_t K, int epilogue) {
  if (validate_i8(M, N, K, epilogue, CQ_DTYPE_F32) != CQ_OK || M == 0 || N == 0 || i8_streams(M))
    return 0;
  int sms = num_sms();
  if (sms <= 0) sms = 148;
  return i8_tc_plan(M, N, K, epilogue, sms).total;
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
  return i8_moe_plan(T, k, H, I).total;
}

extern "C" CQ_API int cq_moe_i8(const uint16_t* tokens, int64_t T, const int32_t* topk_ids,
                                const float* topk_w, int k, int E, const int8_t* w_gu,
                                const float* s_gu, const int8_t* w_dn, const float* s_dn,
                                int64_t H, int64_t I, int out_dtype, float* route_out, void* out,
                                void* workspace, size_t ws_bytes, void* stream) {
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
  const I8MoePlan m = i8_moe_plan(T, k, H, I);
  if (ws_bytes < m.total) return CQ_ERR_WORKSPACE;
  if (!out && !route_out) return CQ_OK;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
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
    p.h = reinterpret_cast<float*>(ws + m.o_h);
    p.y = route_out ? route_out + t * k * H : reinterpret_cast<float*>(ws + m.o_y);
    p.out = out ? static_cast<uint8_t*>(out) + t * H * os : nullptr;
    p.done = reinterpret_cast<int*>(ws);
    p.out_bf16 = out_dtype == CQ_DTYPE_BF16;
    p.clear_y = route_out != nullptr;
    st = i8_moe_stage<false>(p, w_gu, s_gu, sms, s);
    if (st != CQ_OK) return st;
    st = i8_moe_stage<true>(p, w_dn, s_dn, sms, s);
    if (st != CQ_OK) return st;
  }
  return CQ_OK;
}
