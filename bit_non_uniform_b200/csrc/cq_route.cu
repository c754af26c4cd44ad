// cq_route.cu -- host side of the MoE router (cq_moe_route).  Part of
// libcq's single translation unit.
#include <cuda_runtime.h>

#include "cq.h"
#include "cq_host.h"
#include "cq_route.cuh"

namespace cq {

template <int NV>
static int launch_route(const RouteParams& p, cudaStream_t s) {
  return launch_pdl(route_topk_kernel<NV>,
                    dim3(static_cast<unsigned>((p.T + kRtWarps - 1) / kRtWarps)),
                    dim3(kRtWarps * 32), 0, s, p);
}

}  // namespace cq

using namespace cq;

extern "C" CQ_API int cq_moe_route(const void* logits, int logits_dtype, int64_t T, int E, int k,
                                   const float* bias, int scoring, int renorm, float scale,
                                   int32_t* topk_ids, float* topk_w, void* stream) {
  if (T < 0 || E <= 0 || k <= 0 || k > E) return CQ_ERR_INVALID_ARG;
  if (logits_dtype != CQ_DTYPE_F32 && logits_dtype != CQ_DTYPE_BF16) return CQ_ERR_INVALID_ARG;
  if (scoring != CQ_SCORE_SOFTMAX && scoring != CQ_SCORE_SIGMOID) return CQ_ERR_INVALID_ARG;
  if (renorm != 0 && renorm != 1) return CQ_ERR_INVALID_ARG;
  if (E > kRtMaxExperts || k > kRtMaxTopk || T > (int64_t)1 << 31) return CQ_ERR_UNSUPPORTED;
  if (T == 0) return CQ_OK;
  if (!logits || !topk_ids || !topk_w) return CQ_ERR_INVALID_ARG;
  if (!aligned(logits, logits_dtype == CQ_DTYPE_BF16 ? 2 : 4) || !aligned(topk_ids, 4) ||
      !aligned(topk_w, 4) || (bias && !aligned(bias, 4)))
    return CQ_ERR_UNSUPPORTED;
  RouteParams p = {};
  p.logits = logits;
  p.bias = bias;
  p.ids = topk_ids;
  p.w = topk_w;
  p.T = T;
  p.E = E;
  p.k = k;
  p.sigmoid = scoring == CQ_SCORE_SIGMOID;
  p.renorm = renorm;
  p.bf16 = logits_dtype == CQ_DTYPE_BF16;
  p.scale = scale;
  p.vec4 = E % 4 == 0 && aligned(logits, p.bf16 ? 8 : 16);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // NV values in each of 32 lanes, in whole vectors: as few as hold the row.
  // 4096 tokens, top 8, sigmoid and bias, 384 experts: 7.5 us with 12 values,
  // 8.0 with 16; 768 experts: 8.4 with 24, 8.9 with 28.
  switch ((E + 127) / 128) {
    case 1: return launch_route<4>(p, s);
    case 2: return launch_route<8>(p, s);
    case 3: return launch_route<12>(p, s);
    case 4: return launch_route<16>(p, s);
    case 5: return launch_route<20>(p, s);
    case 6: return launch_route<24>(p, s);
    case 7: return launch_route<28>(p, s);
    default: return launch_route<32>(p, s);
  }
}
