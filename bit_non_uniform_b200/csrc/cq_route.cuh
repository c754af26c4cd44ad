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
  int sigmoid, renorm, bf16, vec4;
  float scale;
};

struct RouteSmem {
  double pick[kRtCand];
  double score[kRtCand];
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

// Plain global loads (not the read-only path: a preceding kernel may still be
// writing the data when this one starts), kept behind griddep_wait.
__device__ __forceinline__ uint32_t route_ld16(const void* at) {
  uint16_t v;
  asm volatile("ld.global.b16 %0, [%1];" : "=h"(v) : "l"(at));
  return v;
}
__device__ __forceinline__ float route_ld32(const void* at) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(at));
  return v;
}
__device__ __forceinline__ uint2 route_ld64(const void* at) {
  uint2 v;
  asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(at));
  return v;
}
__device__ __forceinline__ float4 route_ld128(const void* at) {
  float4 v;
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(at));
  return v;
}

// One logit, NaN as -inf.
__device__ __forceinline__ float route_logit(const RouteParams& p, int64_t at) {
  const float v =
      p.bf16 ? __uint_as_float(route_ld16(static_cast<const uint16_t*>(p.logits) + at) << 16)
             : route_ld32(static_cast<const float*>(p.logits) + at);
  return fmaxf(v, -INFINITY);
}

// 2^x and 1/x by the approximate units (2 and 1 units in the last place;
// 2^x of +inf is inf, 1/inf is 0).
__device__ __forceinline__ float route_ex2(float x) {
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float route_rcp(float x) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The warp's values in descending order, one per lane.
__device__ __forceinline__ float warp_sort_desc(float v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size *= 2) {
#pragma unroll
    for (int o = size / 2; o > 0; o /= 2) {
      const float u = __shfl_xor_sync(0xffffffffu, v, o);
      const bool first = (lane & o) == 0, down = (lane & size) == 0;
      v = first == down ? fmaxf(v, u) : fminf(v, u);
    }
  }
  return v;
}

// NV values per lane, a multiple of 4.  The lane's value i is expert ((i / 4) 32 + lane) 4 + i % 4
// where rows and bias can be read in fours (vec4), else i 32 + lane.
template <int NV>
__global__ void __launch_bounds__(kRtWarps * 32)
    route_topk_kernel(const __grid_constant__ RouteParams p) {
  __shared__ RouteSmem smem[kRtWarps];
  __shared__ float4 s_bias[NV * 8];      // zeros past E
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  RouteSmem& s = smem[warp];
  const float NEG = -INFINITY;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRtWarps + warp;
  const bool live = t < p.T;
  const int64_t base = t * p.E;
  auto expert = [&](int i) {
    return p.vec4 ? ((i >> 2) * 32 + lane) * 4 + (i & 3) : i * 32 + lane;
  };
  float key[NV];                         // the logits, then the FP32 picks
  if (p.vec4) {
#pragma unroll
    for (int i = 0; i < NV; i += 4) {
      const int e = expert(i);
      float4 v = make_float4(NEG, NEG, NEG, NEG);
      if (live && e < p.E) {
        if (p.bf16) {
          const uint2 q = route_ld64(static_cast<const uint16_t*>(p.logits) + base + e);
          v = make_float4(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xFFFF0000u),
                          __uint_as_float(q.y << 16), __uint_as_float(q.y & 0xFFFF0000u));
        } else {
          v = route_ld128(static_cast<const float*>(p.logits) + base + e);
        }
      }
      key[i] = v.x;
      key[i + 1] = v.y;
      key[i + 2] = v.z;
      key[i + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = fmaxf(key[i], NEG);      // NaN becomes -inf
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = i * 32 + lane;
      key[i] = live && e < p.E ? route_logit(p, base + e) : NEG;
    }
  }
  // the CTA's bias, on its way together with the logits (read where it is
  // used, it cost one token 2 us)
  float* const bias = reinterpret_cast<float*>(s_bias);
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < NV / kRtWarps; ++i) {
      const int e = i * kRtWarps * 32 + threadIdx.x;
      bias[e] = e < p.E ? route_ld32(p.bias + e) : 0.f;
    }
  }
  __syncthreads();
  if (!live) return;
  float top = NEG;
  double sum = 0.0;                      // softmax: sum of exp(l - top)
  if (!p.sigmoid) {
#pragma unroll
    for (int i = 0; i < NV; ++i) top = fmaxf(top, key[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (p.bias) {
      // picks compare p + bias: the sum in FP64 (the logits read again, so
      // that the loop stays rolled)
      if (top > NEG) {
        for (int e = lane; e < p.E; e += 128) {
          double x[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float v = e + 32 * j < p.E ? route_logit(p, base + e + 32 * j) : NEG;
            // (equal infinities count as 1)
            x[j] = v == top ? 0.0 : static_cast<double>(v) - static_cast<double>(top);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = exp(x[j]);
          sum += (x[0] + x[1]) + (x[2] + x[3]);
        }
      }
      sum = warp_sum_f64(sum);
    } else if (!p.renorm) {
      float f = 0.f;                     // only scales the weights: FP32
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (key[i] > NEG) f += key[i] == top ? 1.f : expf(key[i] - top);
      sum = warp_sum_f64(static_cast<double>(f));
    }
  }
  auto score64 = [&](float v) -> double {
    if (p.sigmoid) return 1.0 / (1.0 + exp(-static_cast<double>(v)));
    return p.bias ? route_exp64(v, top) / sum : route_exp64(v, top);
  };
  if (p.bias) {
    // FP32 picks
    constexpr float LOG2E = 1.44269504f;
    const float inv_sum = p.sigmoid ? 0.f : static_cast<float>(1.0 / sum);
#pragma unroll
    for (int i = 0; i < NV; i += 4) {
      float b[4];
      if (p.vec4) {
        const float4 q = s_bias[expert(i) >> 2];
        b[0] = q.x;
        b[1] = q.y;
        b[2] = q.z;
        b[3] = q.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = bias[expert(i + j)];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v = key[i + j];
        const float sc = p.sigmoid ? route_rcp(1.0f + route_ex2(-LOG2E * v))
                                   : (v == top ? 1.0f : route_ex2(LOG2E * (v - top))) * inv_sum;
        key[i + j] = v > NEG ? fmaxf(sc + b[j], NEG) : NEG;
      }
    }
  }
  float best = NEG;
#pragma unroll
  for (int i = 0; i < NV; ++i) best = fmaxf(best, key[i]);
  // the k-th largest lane maximum, and its margin.  An FP32 pick is off by at
  // most 5e-7 (1 + |bias|): the score is at most 1, its exponential within
  // 2^-21 + 2^-22 |l| (relative, and s (1 - s) |l| < 0.23), the reciprocal and
  // the sums within a few 2^-24.  Twice that on either side, with
  // |bias| <= 1 + |pick|.
  float cut = __shfl_sync(0xffffffffu, warp_sort_desc(best), p.k - 1);
  if (p.bias) {
    cut = fminf(cut, 3e38f);
    cut -= 2e-6f * (2.0f + fabsf(cut));
  }
  cut = fmaxf(cut, -3.402823466e38f);        // -inf is never a candidate
  uint32_t mask = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) mask |= key[i] >= cut ? 1u << i : 0u;
  const int mine = __popc(mask);
  int n = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, n, o);
    if (lane >= o) n += u;
  }
  int pos = n - mine;
  n = __shfl_sync(0xffffffffu, n, 31);
  if (lane < p.k) s.sel_id[lane] = -1;
  if (n <= kRtCand) {
    for (uint32_t m = mask; m; m &= m - 1) s.id[pos++] = expert(__ffs(m) - 1);
    __syncwarp();
    for (int c = lane; c < n; c += 32) {
      const int e = s.id[c];
      const float v = route_logit(p, base + e);
      const double sc = score64(v);
      s.score[c] = sc;
      s.pick[c] = p.bias ? sc + static_cast<double>(bias[e]) : static_cast<double>(v);
    }
    __syncwarp();
    for (int c = lane; c < n; c += 32) {
      const double pick = s.pick[c];
      const int e = s.id[c];
      int r = 0;
      for (int j = 0; j < n; ++j) {
        const double o = s.pick[j];
        r += o > pick || (o == pick && s.id[j] < e);
      }
      if (r < p.k && pick > -static_cast<double>(INFINITY)) {
        s.sel_id[r] = e;
        s.sel_score[r] = s.score[c];
      }
    }
  } else {
    // more equal (or nearly equal) picks than are ranked at once: take the
    // best k one by one
    __syncwarp();
    for (int r = 0; r < p.k; ++r) {
      double wp = -static_cast<double>(INFINITY);
      int we = kRtMaxExperts, wi = 0;
      for (uint32_t m = mask; m; m &= m - 1) {
        const int i = __ffs(m) - 1, e = expert(i);
        const float v = route_logit(p, base + e);
        const double pick = p.bias ? score64(v) + static_cast<double>(bias[e])
                                   : static_cast<double>(v);
        if (pick > wp || (pick == wp && e < we)) {
          wp = pick;
          we = e;
          wi = i;
        }
      }
      const int own = we;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const double op = __shfl_xor_sync(0xffffffffu, wp, o);
        const int oe = __shfl_xor_sync(0xffffffffu, we, o);
        if (op > wp || (op == wp && oe < we)) {
          wp = op;
          we = oe;
        }
      }
      if (we == own && we < kRtMaxExperts && wp > -static_cast<double>(INFINITY)) {
        mask &= ~(1u << wi);
        s.sel_id[r] = we;
        s.sel_score[r] = score64(route_logit(p, base + we));
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
