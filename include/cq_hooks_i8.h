/*
 * cq_hooks_i8.h -- test hooks of the INT8 operators.
 *
 * Like those of cq_hooks.h, these entry points are not part of the product
 * interface (include/cq.h): they let the test suite run a product or a layer
 * on a chosen kernel, ask which kernel a call takes, and make the kernels'
 * bounded waits run out.  Arguments are validated as those of the calls in
 * cq.h that they stand for.
 */
#ifndef CQ_HOOKS_I8_H_
#define CQ_HOOKS_I8_H_

#include "cq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Kernels: what the call itself picks; the streaming kernels; K split over a
 * cluster, and CTA pairs (products); sorted routes (the MoE layer). */
enum {
  CQ_I8_AUTO = 0,
  CQ_I8_STREAM = 1,
  CQ_I8_SPLIT = 2,
  CQ_I8_PAIR = 3,
  CQ_I8_SORTED = 4
};

/*
 * cq_test_product_i8 -- cq_gemm_i8 (absmax given) or cq_linear_i8 (absmax
 * NULL: x is bfloat16) on the kernel `path`, with `timeout_ns` as the limit of
 * every device-side wait (0: the default).  With withhold != 0 every CTA waits
 * for an arrival on its first piece of operands that never comes: the waits run
 * out, and the kernel records CQ_ERR_TIMEOUT (read with cq_get_device_error) and
 * returns.  A path that does not take the problem returns CQ_ERR_UNSUPPORTED.
 * cq_test_product_i8_path gives the path of a call (148 SMs without a GPU), or
 * 0 where there is none to run.
 */
CQ_API int cq_test_product_i8_path(int64_t M, int64_t N, int64_t K, int epilogue);
CQ_API int cq_test_product_i8(const void *x, const float *absmax, int64_t M, const int8_t *wq,
                              const float *wscale, int64_t N, int64_t K, int epilogue,
                              int out_dtype, void *y, void *workspace, size_t ws_bytes, int path,
                              uint64_t timeout_ns, int withhold, void *stream);

/*
 * cq_test_moe_i8 -- cq_moe_i8 likewise.  withhold = 1 or 2: in the gate/up or the
 * down launch; its limit is `timeout_ns`, that of the
 * other launch a quarter of it.
 * cq_test_moe_i8_path gives the path of a layer (0 where there is none to run)
 * and, in *tokens_per_launch, how many tokens one launch takes.
 */
CQ_API int cq_test_moe_i8_path(int64_t T, int k, int E, int64_t H, int64_t I,
                               int64_t *tokens_per_launch);
CQ_API size_t cq_test_moe_i8_workspace_size(int64_t T, int k, int E, int64_t H, int64_t I,
                                            int path);
CQ_API int cq_test_moe_i8(const uint16_t *tokens, int64_t T, const int32_t *topk_ids,
                          const float *topk_w, int k, int E, const int8_t *w_gu,
                          const float *s_gu, const int8_t *w_dn, const float *s_dn, int64_t H,
                          int64_t I, int out_dtype, float *route_out, void *out, void *workspace,
                          size_t ws_bytes, int path, uint64_t timeout_ns, int withhold,
                          void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CQ_HOOKS_I8_H_ */
