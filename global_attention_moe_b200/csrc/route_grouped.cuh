// route_grouped.cuh -- routing with sigmoid or softmax scores, group-limited choice and a scale factor,
// and the gradient of its weights.
//
//   s_e   = sigmoid(x_e)  or  exp(x_e - max x) / sum_i exp(x_i - max x)          (FP64)
//   key_e = fp32(s_e) + bias_e                                                   (FP32)
//   group score = its largest key + its second largest (FP32; a group of one expert: its key); the
//   top_groups largest groups are kept, ties to the lower group
//   ids = the top_k largest keys of the kept groups, ties to the lower expert; a NaN key counts as -inf
//   w_j = scale s_j / sum_i s_i over the chosen (normalize; all scores zero: zero), or scale s_j
//
// The choice is defined on FP32 keys of FP64 scores, as the ungrouped router's is, so it does not depend
// on how the scores are computed, and the tests can ask for equal ids.
#pragma once

#include <stdint.h>

#include "neighbors.cuh"

namespace mimo {
namespace rg {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxExperts = 512;
constexpr int kMaxPerLane = kMaxExperts / 32;
constexpr int kMaxGroups = 32;

struct RouteParams {
  const float* logits;  // [T, E]
  const float* bias;    // [E] or nullptr
  int32_t* ids;         // [T, top_k]
  float* weights;       // [T, top_k]
  int64_t T;
  int E, top_k, groups, top_groups;
  int softmax, normalize;
  float scale;
};

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The definition for one token, by one warp: lane holds experts lane + 32 m; s_key: E floats of the warp's.
__device__ __forceinline__ void route_exact(const RouteParams& P, int64_t tok, int lane, float* s_key) {
  const float* x = P.logits + tok * P.E;
  double sc[kMaxPerLane];
  if (P.softmax) {
    float mx = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int m = 0; m < kMaxPerLane; ++m) {
      const float v = lane + 32 * m < P.E ? __ldg(x + lane + 32 * m) : -INFINITY;
      sc[m] = v;
      nan |= v != v;
      mx = fmaxf(mx, v);
    }
    mx = warp_max(mx);
    nan = __any_sync(0xffffffffu, nan);
    double sum = 0.0;
#pragma unroll
    for (int m = 0; m < kMaxPerLane; ++m) {
      sc[m] = lane + 32 * m < P.E ? exp(sc[m] - static_cast<double>(mx)) : 0.0;  // all -inf: NaN, as the formula says
      sum += sc[m];
    }
    sum = warp_sum_f64(sum);
#pragma unroll
    for (int m = 0; m < kMaxPerLane; ++m) sc[m] /= sum;
  } else {
#pragma unroll
    for (int m = 0; m < kMaxPerLane; ++m)
      sc[m] = lane + 32 * m < P.E ? nb::route_sigmoid_f64(static_cast<double>(__ldg(x + lane + 32 * m))) : 0.0;
  }
  float key[kMaxPerLane];
#pragma unroll
  for (int m = 0; m < kMaxPerLane; ++m) {
    key[m] = -INFINITY;
    const int e = lane + 32 * m;
    if (e < P.E) {
      const float k = static_cast<float>(sc[m]) + (P.bias != nullptr ? __ldg(P.bias + e) : 0.f);
      key[m] = k == k ? k : -INFINITY;
    }
  }
  uint32_t open = 0;  // this lane's experts that may be chosen
#pragma unroll
  for (int m = 0; m < kMaxPerLane; ++m)
    if (lane + 32 * m < P.E) open |= 1u << m;
  if (P.top_groups < P.groups) {
    const int size = P.E / P.groups;
#pragma unroll
    for (int m = 0; m < kMaxPerLane; ++m)
      if (lane + 32 * m < P.E) s_key[lane + 32 * m] = key[m];
    __syncwarp();
    float a = -INFINITY, b = -INFINITY;  // lane g: the two largest keys of group g
    if (lane < P.groups)
      for (int i = 0; i < size; ++i) {
        const float k = s_key[lane * size + i];
        b = fmaxf(b, fminf(a, k));
        a = fmaxf(a, k);
      }
    float gs = size > 1 ? a + b : a;
    if (gs != gs) gs = -INFINITY;  // +inf and -inf keys in one group
    int rank = 0;
    for (int j = 0; j < P.groups; ++j) {
      const float o = __shfl_sync(0xffffffffu, gs, j);
      rank += (o > gs || (o == gs && j < lane)) ? 1 : 0;
    }
    const uint32_t kept = __ballot_sync(0xffffffffu, lane < P.groups && rank < P.top_groups);
#pragma unroll
    for (int m = 0; m < kMaxPerLane; ++m)
      if (lane + 32 * m < P.E && !((kept >> ((lane + 32 * m) / size)) & 1u)) open &= ~(1u << m);
    __syncwarp();  // s_key is written again for the next token
  }
  double chosen = 0.0, total = 0.0;
  int my_id = 0;
#pragma unroll 1
  for (int c = 0; c < P.top_k; ++c) {
    float bk = -INFINITY;
    int be = 0x7fffffff;
#pragma unroll
    for (int m = 0; m < kMaxPerLane; ++m)
      if (((open >> m) & 1u) && (be == 0x7fffffff || key[m] > bk)) {
        bk = key[m];
        be = lane + 32 * m;
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float ok = __shfl_xor_sync(0xffffffffu, bk, o);
      const int oe = __shfl_xor_sync(0xffffffffu, be, o);
      if (oe != 0x7fffffff && (be == 0x7fffffff || ok > bk || (ok == bk && oe < be))) {
        bk = ok;
        be = oe;
      }
    }
    // top_k <= the experts of the kept groups, so some expert was open
    double s = 0.0;
    if ((be & 31) == lane) {
#pragma unroll
      for (int m = 0; m < kMaxPerLane; ++m)
        if (m == be >> 5) s = sc[m];
      open &= ~(1u << (be >> 5));
    }
    s = __shfl_sync(0xffffffffu, s, be & 31);
    total += s;
    if (lane == c) {
      my_id = be;
      chosen = s;
    }
  }
  if (lane < P.top_k) {
    const double w = P.normalize ? (total == 0.0 ? 0.0 : chosen / total) : chosen;
    P.ids[tok * P.top_k + lane] = my_id;
    P.weights[tok * P.top_k + lane] = static_cast<float>(w * static_cast<double>(P.scale));
  }
}

// One warp per token.
__global__ void __launch_bounds__(kThreads) route_grouped_kernel(const __grid_constant__ RouteParams P) {
  extern __shared__ __align__(16) float sm[];  // E keys per warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t tok = static_cast<int64_t>(blockIdx.x) * kWarps + warp; tok < P.T; tok += step)
    route_exact(P, tok, lane, sm + warp * P.E);
}

struct RouteBwdParams {
  const float* logits;    // [T, E]
  const int32_t* ids;     // [T, top_k]
  const float* dweights;  // [T, top_k]
  float* dlogits;         // [T, E]
  int64_t T;
  int E, top_k;
  int softmax, normalize;
  float scale;
};

// Gradient of the weights with respect to the logits (the choice itself has none).  With g = dw, p_j =
// s_j / sum of the chosen s and gm = sum_i g_i p_i:
//   sigmoid, normalised   dx_j = scale (g_j - gm) p_j (1 - s_j)      (from ds_j = scale (g_j - gm) / S)
//   sigmoid               dx_j = scale g_j s_j (1 - s_j)
//   softmax, normalised   dx_j = scale (g_j - gm) p_j                (the softmax's own sum cancels)
//   softmax               dx_e = scale s_e (sum of g_j with id_j = e - sum_j g_j s_j)     every expert
// An id outside [0, E) is an empty place: it takes no part.  The same id twice adds up.
// One warp per token; the row is put together in shared memory and written whole.
__global__ void __launch_bounds__(kThreads) route_bwd_kernel(const __grid_constant__ RouteBwdParams P) {
  extern __shared__ __align__(16) float sm[];  // E per warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row = sm + warp * P.E;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t tok = static_cast<int64_t>(blockIdx.x) * kWarps + warp; tok < P.T; tok += step) {
    const float* x = P.logits + tok * P.E;
    int id = -1;
    double g = 0.0;
    if (lane < P.top_k) {
      id = __ldg(P.ids + tok * P.top_k + lane);
      if (id < 0 || id >= P.E) id = -1;
      if (id >= 0) g = static_cast<double>(P.scale) * static_cast<double>(__ldg(P.dweights + tok * P.top_k + lane));
    }
    const double xj = id >= 0 ? static_cast<double>(__ldg(x + id)) : -INFINITY;
    for (int e = lane; e < P.E; e += 32) row[e] = 0.f;
    __syncwarp();
    double d = 0.0;  // this place's share of dx[id]
    if (!P.softmax) {
      const double s = id >= 0 ? nb::route_sigmoid_f64(xj) : 0.0, c = id >= 0 ? nb::route_sigmoid_f64(-xj) : 0.0;
      if (P.normalize) {
        const double S = warp_sum_f64(s);
        const double p = S == 0.0 ? 0.0 : s / S;
        const double gm = warp_sum_f64(g * p);
        d = (g - gm) * p * c;
      } else {
        d = g * s * c;
      }
    } else if (P.normalize) {
      double mx = xj;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmax(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const double s = id >= 0 && mx > -INFINITY ? exp(xj - mx) : 0.0;
      const double S = warp_sum_f64(s);
      const double p = S == 0.0 ? 0.0 : s / S;
      const double gm = warp_sum_f64(g * p);
      d = (g - gm) * p;
    } else {
      float mx = -INFINITY;
      for (int e = lane; e < P.E; e += 32) mx = fmaxf(mx, __ldg(x + e));
      const double m = static_cast<double>(warp_max(mx));
      double S = 0.0;
      for (int e = lane; e < P.E; e += 32) S += exp(static_cast<double>(__ldg(x + e)) - m);
      S = warp_sum_f64(S);
      const double s = id >= 0 ? exp(xj - m) / S : 0.0;
      const double gm = warp_sum_f64(g * s);
      for (int e = lane; e < P.E; e += 32)
        row[e] = static_cast<float>(-gm * (exp(static_cast<double>(__ldg(x + e)) - m) / S));
      __syncwarp();
      d = g * s;
    }
    // places in turn, so that the same id twice adds up in a fixed order
    for (int j = 0; j < P.top_k; ++j) {
      if (lane == j && id >= 0) row[id] += static_cast<float>(d);
      __syncwarp();
    }
    for (int e = lane; e < P.E; e += 32) P.dlogits[tok * P.E + e] = row[e];
    __syncwarp();
  }
}

}  // namespace rg
}  // namespace mimo
