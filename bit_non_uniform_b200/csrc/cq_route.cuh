// cq_route.cuh -- a MoE router's logits to the top-k expert ids and weights.
//
//   score_e = sigmoid(l_e)  or  softmax(l)_e
//   pick_e  = score_e + bias_e   (without a bias: l_e, which orders the same)
//   ids     = the k experts of largest pick, descending, ties to the lower id
//   w_j     = scale * score_(ids_j)  [/ sum_j score_(ids_j) with renorm]
// Picks are compared in FP64, so the ids are those of any other FP64
// evaluation; an expert whose logit is -inf or NaN (or whose pick is) is
// never chosen, and slots without an expert get id -1 and weight 0, which the
// MoE layers drop.
//
// One warp per token, the logits in registers.  The FP32 picks only cut the
// field: the k-th largest of the 32 lanes' own maxima is a lower bound of the
// k-th largest pick, so every expert that can be chosen lies above it less
// the FP32 error.  The few candidates left (about 1.5 k) are evaluated in
// FP64, one per lane, and ranked by counting.  Reading the logits bounds the
// kernel at many tokens; at a few it is the latency of that chain.
#pragma once

#include "cq_device.cuh"

namespace cq {

constexpr int kRtWarps = 4;
constexpr int kRtCand = 256;             // candidates ranked by counting
constexpr int kRtMaxExperts = 1024;
constexpr int kRtMaxTopk = 32;

struct RouteParams {
  const void* logits;       // [T][E]
  const float* bias;        // [E], or null
  int32_t* ids;             // [T][k]
  float* w;                 // [T][k]
  int64_t T;
  int E, k;
  int sigmoid, renorm, bf16;
  float scale;
};

struct RouteSmem {
  double pick[kRtCand];
  float logit[kRtCand];
  int id[kRtCand];
  double sel_score[kRtMaxTopk];
  int sel_id[kRtMaxTopk];
};

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// exp(l - top) where equal infinities count as 1 (the limit).
__device__ __forceinline__ double route_exp64(float l, float top) {
  return l == top ? 1.0 : exp(static_cast<double>(l) - static_cast<double>(top));
}

template <int NV>
__global__ void __launch_bounds__(kRtWarps * 32)
    route_topk_kernel(const __grid_constant__ RouteParams p) {
  __shared__ RouteSmem smem[kRtWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  RouteSmem& s = smem[warp];
  const float NEG = -INFINITY;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRtWarps + warp;
  if (t >= p.T) return;
  float l[NV], key[NV];
  const int64_t base = t * p.E;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = i * 32 + lane;
    float v = NEG;
    if (e < p.E)
      v = p.bf16 ? __uint_as_float(static_cast<uint32_t>(
                       __ldg(static_cast<const uint16_t*>(p.logits) + base + e)) << 16)
                 : __ldg(static_cast<const float*>(p.logits) + base + e);
    l[i] = v == v ? v : NEG;
  }
  float top = NEG;
  double sum = 0.0;                      // softmax: sum of exp(l - top)
  if (!p.sigmoid) {
#pragma unroll
    for (int i = 0; i < NV; ++i) top = fmaxf(top, l[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (p.bias) {
      // picks compare p + bias: the sum in FP64
#pragma unroll 1
      for (int i = 0; i < NV; ++i)
        if (l[i] > NEG) sum += route_exp64(l[i], top);
      sum = warp_sum_f64(sum);
    } else if (!p.renorm) {
      float f = 0.f;                     // only scales the weights: FP32
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (l[i] > NEG) f += l[i] == top ? 1.f : expf(l[i] - top);
      sum = warp_sum_f64(static_cast<double>(f));
    }
  }
  auto score64 = [&](float v) -> double {
    if (p.sigmoid) return 1.0 / (1.0 + exp(-static_cast<double>(v)));
    return p.bias ? route_exp64(v, top) / sum : route_exp64(v, top);
  };
  auto pick64 = [&](float v, int e) -> double {
    return p.bias ? score64(v) + static_cast<double>(__ldg(p.bias + e))
                  : static_cast<double>(v);
  };
  // FP32 picks (clamped, so that the margin below stays finite)
  const float inv_sum = static_cast<float>(1.0 / sum);
  float best = NEG;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = i * 32 + lane;
    float v = l[i];
    if (p.bias && v > NEG) {
      const float sc = p.sigmoid ? 1.0f / (1.0f + expf(-v))
                                 : (v == top ? 1.f : expf(v - top)) * inv_sum;
      v = sc + __ldg(p.bias + e);
      v = v == v ? fminf(v, 3e38f) : NEG;
    }
    key[i] = v;
    best = fmaxf(best, v);
  }
  // the k-th largest lane maximum
  int rank = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const float o = __shfl_sync(0xffffffffu, best, j);
    rank += o > best || (o == best && j < lane);
  }
  const unsigned at = __ballot_sync(0xffffffffu, rank == p.k - 1);
  float cut = __shfl_sync(0xffffffffu, best, __ffs(at) - 1);
  // FP32 picks are off by a few units of 2^-24 (1 + |bias|), the score being
  // at most 1: twice that on either side, rounded up
  if (p.bias && cut > NEG) cut -= 2e-6f * (2.0f + fabsf(cut));
  int n = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool in = key[i] > NEG && key[i] >= cut;
    const unsigned m = __ballot_sync(0xffffffffu, in);
    const int pos = n + __popc(m & ((1u << lane) - 1u));
    if (in && pos < kRtCand) {
      s.id[pos] = i * 32 + lane;
      s.logit[pos] = l[i];
    }
    n += __popc(m);
  }
  if (lane < p.k) s.sel_id[lane] = -1;
  __syncwarp();
  if (n <= kRtCand) {
    for (int c = lane; c < n; c += 32) s.pick[c] = pick64(s.logit[c], s.id[c]);
    __syncwarp();
    // candidates are in the order of their ids, so position breaks ties
    for (int c = lane; c < n; c += 32) {
      const double mine = s.pick[c];
      int r = 0;
      for (int j = 0; j < n; ++j) {
        const double o = s.pick[j];
        r += o > mine || (o == mine && j < c);
      }
      if (r < p.k && mine > -static_cast<double>(INFINITY)) {
        s.sel_id[r] = s.id[c];
        s.sel_score[r] = score64(s.logit[c]);
      }
    }
  } else {
    // more equal (or nearly equal) picks than are ranked at once: take the
    // best k one by one
    uint32_t taken = 0;
    for (int r = 0; r < p.k; ++r) {
      double bp = -static_cast<double>(INFINITY);
      int be = kRtMaxExperts, bi = -1;
      float bl = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!(key[i] > NEG && key[i] >= cut) || (taken >> i & 1u)) continue;
        const double v = pick64(l[i], i * 32 + lane);
        if (v > bp) {
          bp = v;
          be = i * 32 + lane;
          bi = i;
          bl = l[i];
        }
      }
      double wp = bp;
      int we = be;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const double op = __shfl_xor_sync(0xffffffffu, wp, o);
        const int oe = __shfl_xor_sync(0xffffffffu, we, o);
        if (op > wp || (op == wp && oe < we)) {
          wp = op;
          we = oe;
        }
      }
      if (we == be && bi >= 0) {
        taken |= 1u << bi;
        s.sel_id[r] = be;
        s.sel_score[r] = score64(bl);
      }
    }
  }
  __syncwarp();
  int id = -1;
  double sc = 0.0;
  if (lane < p.k) {
    id = s.sel_id[lane];
    if (id >= 0) sc = s.sel_score[lane];
  }
  if (p.renorm) {
    const double total = warp_sum_f64(sc);
    sc = total > 0.0 ? sc / total : 0.0;
  } else if (!p.sigmoid && !p.bias && id >= 0) {
    sc /= sum;
  }
  if (lane < p.k) {
    p.ids[t * p.k + lane] = id;
    p.w[t * p.k + lane] = static_cast<float>(sc * static_cast<double>(p.scale));
  }
}

}  // namespace cq
