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
//
// route_fast_kernel takes it on approximate FP32 keys whose error is bounded, one warp per token:
//   1. a lane holds P experts of one group in a row (L lanes to a group), forms their approximate keys,
//      moved up by a constant so that they are positive and order like their bits as integers, puts the
//      expert's place in the lane into the low bits, and sorts them;
//   2. a group's two largest come from its lanes' first two by exchanges; its rank among the groups by
//      comparing with each; lanes of the groups that are not kept drop out;
//   3. top_k times, the warp's largest first key (one integer reduction) is taken from its lane;
//   4. where every two neighbours of the k + 1 largest differ by more than twice the error bound, their
//      order is that of the exact keys: the chosen experts' scores are formed in FP32 and written.
// Otherwise the experts within the bound of the k-th key (at most 32) take their exact keys in FP64 and are
// ranked; and where that does not decide either (group scores within the bound, more than 32 candidates,
// keys that are NaN, infinite or far below the others), route_exact states the definition.
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

// The definition alone, one warp per token: shapes that the fast kernel's lanes do not hold.
__global__ void __launch_bounds__(kThreads) route_grouped_kernel(const __grid_constant__ RouteParams P) {
  extern __shared__ __align__(16) float sm[];  // E keys per warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t tok = static_cast<int64_t>(blockIdx.x) * kWarps + warp; tok < P.T; tok += step)
    route_exact(P, tok, lane, sm + warp * P.E);
}

// ---------------------------------------------------------------- the fast kernel
// What the lanes hold: S = E / groups experts to a group, L lanes to a group, P experts to a lane.
struct FastShape {
  int S, L, P, vec;  // vec: every lane holds exactly P experts, a multiple of 4
};

// Descending compare-exchange network (Batcher's odd-even merge sort), N a power of two.
template <int N>
__device__ __forceinline__ void sort_desc(int (&k)[N]) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1)
#pragma unroll
    for (int q = p; q >= 1; q >>= 1)
#pragma unroll
      for (int j = q % p; j <= N - 1 - q; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const int a = k[i + j], b = k[i + j + q];
            k[i + j] = max(a, b);
            k[i + j + q] = min(a, b);
          }
}

__device__ __forceinline__ float as_float(int k) { return __uint_as_float(static_cast<uint32_t>(k)); }

constexpr int kNone = static_cast<int>(0x80000000u);  // below every key (as a float -0)
constexpr int kInf = 0x7F800000;
constexpr float kLog2e = 1.4426950408889634f;

// The exact keys of the experts within `margin` of the k-th approximate one, ranked.  sorted[32 m + lane]: the
// lane's m-th largest key.  Returns false when there are more than 32 of them.
template <int P>
__device__ __noinline__ bool route_candidates(const RouteParams& R, const FastShape& F, int64_t tok, int lane,
                                              const int* sorted, float margin) {
  constexpr int mask = P - 1;
  const float* x = R.logits + tok * R.E;
  int at = 0, n = 0, mine = 0;  // the lane's next key; candidates; this lane's candidate
  float cut = -INFINITY;
#pragma unroll 1
  while (true) {
    const int a = at < P ? sorted[32 * at + lane] : kNone;
    const int M = __reduce_max_sync(0xffffffffu, a);
    if (M < 0 || as_float(M) < cut) break;
    if (n == 32) return false;
    const int first = __ffs(__ballot_sync(0xffffffffu, a == M)) - 1;
    if (lane == first) ++at;
    if (lane == n) mine = (first / F.L) * F.S + (first % F.L) * F.P + (P - 1 - (M & mask));
    if (++n == R.top_k) cut = as_float(M) - margin;
  }
  if (n < R.top_k) return false;
  double sc = 0.0;
  if (R.softmax) {
    float mx = -INFINITY;
    for (int e = lane; e < R.E; e += 32) mx = fmaxf(mx, __ldg(x + e));
    const double m = static_cast<double>(warp_max(mx));
    double S = 0.0;
    for (int e = lane; e < R.E; e += 32) S += exp(static_cast<double>(__ldg(x + e)) - m);
    S = warp_sum_f64(S);
    sc = exp(static_cast<double>(__ldg(x + mine)) - m) / S;
  } else {
    sc = nb::route_sigmoid_f64(static_cast<double>(__ldg(x + mine)));
  }
  const float key = static_cast<float>(sc) + (R.bias != nullptr ? __ldg(R.bias + mine) : 0.f);
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const float o = __shfl_sync(0xffffffffu, key, j);
    const int e = __shfl_sync(0xffffffffu, mine, j);
    rank += (o > key || (o == key && e < mine)) ? 1 : 0;
  }
  const bool chosen = lane < n && rank < R.top_k;
  const double total = warp_sum_f64(chosen ? sc : 0.0);
  if (chosen) {
    const double w = R.normalize ? (total == 0.0 ? 0.0 : sc / total) : sc;
    R.ids[tok * R.top_k + rank] = mine;
    R.weights[tok * R.top_k + rank] = static_cast<float>(w * static_cast<double>(R.scale));
  }
  return true;
}

__device__ __noinline__ void route_exact_call(const RouteParams& R, int64_t tok, int lane, float* s_key) {
  route_exact(R, tok, lane, s_key);
}

template <int P, bool kSoftmax>
__global__ void __launch_bounds__(kThreads, P <= 8 ? 4 : 2) route_fast_kernel(const __grid_constant__ RouteParams R,
                                                              const __grid_constant__ FastShape F) {
  extern __shared__ __align__(16) float sm[];  // per warp: E keys (route_exact) or 32 P sorted ones
  constexpr int kMask = P - 1;                 // low bits of a key: P - 1 - place in the lane
  constexpr int kDepth = P < 4 ? P : 4;        // keys of a lane that the fast path can take
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* s_key = sm + warp * (32 * P > R.E ? 32 * P : R.E);
  const int g = lane / F.L, in_group = (lane % F.L) * F.P;
  const int count = g < R.groups ? max(0, min(F.P, F.S - in_group)) : 0;
  const int e0 = count > 0 ? g * F.S + in_group : 0;
  // biases moved up by the least of them (those far below all others aside), so that keys are positive
  float bl[P], low = 0.f;
#pragma unroll
  for (int m = 0; m < P; ++m) bl[m] = 0.f;
  if (R.bias != nullptr) {
    low = INFINITY;
#pragma unroll
    for (int m = 0; m < P; ++m)
      if (m < count) {
        bl[m] = __ldg(R.bias + e0 + m);
        if (bl[m] > -1024.f) low = fminf(low, bl[m]);
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
    if (!(fabsf(low) < 1e30f)) low = 0.f;
#pragma unroll
    for (int m = 0; m < P; ++m) bl[m] -= low;
  }
  const float off = fabsf(low);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  int64_t tok = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  float xn[P];  // the next token's logits
  auto load = [&](int64_t t) {
    if (P >= 4 && F.vec) {
      const float4* p = reinterpret_cast<const float4*>(R.logits + t * R.E + e0);
#pragma unroll
      for (int m = 0; m < P / 4; ++m) {
        const float4 v = t < R.T ? __ldg(p + m) : make_float4(0.f, 0.f, 0.f, 0.f);
        xn[4 * m] = v.x, xn[4 * m + 1] = v.y, xn[4 * m + 2] = v.z, xn[4 * m + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int m = 0; m < P; ++m) xn[m] = t < R.T && m < count ? __ldg(R.logits + t * R.E + e0 + m) : -INFINITY;
    }
  };
  load(tok);
#pragma unroll 1
  for (; tok < R.T; tok += step) {
    float sc[P];
#pragma unroll
    for (int m = 0; m < P; ++m) sc[m] = xn[m];
    load(tok + step);  // in flight meanwhile
    float mx = 0.f, inv = 1.f;
    if (kSoftmax) {
      mx = sc[0];
#pragma unroll
      for (int m = 1; m < P; ++m) mx = fmaxf(mx, sc[m]);
      mx = warp_max(mx);
      float sum = 0.f;
#pragma unroll
      for (int m = 0; m < P; ++m) {
        sc[m] = ex2_approx((sc[m] - mx) * kLog2e);
        sum += sc[m];
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      inv = rcp_approx(sum);
#pragma unroll
      for (int m = 0; m < P; ++m) sc[m] *= inv;
    } else {
#pragma unroll
      for (int m = 0; m < P; ++m) sc[m] = rcp_approx(1.f + ex2_approx(sc[m] * -kLog2e));
    }
    int key[P];
#pragma unroll
    for (int m = 0; m < P; ++m) {
      const int k = static_cast<int>(__float_as_uint(sc[m] + bl[m]));
      key[m] = m < count ? (k & ~kMask) | (P - 1 - m) : kNone;
    }
    sort_desc<P>(key);
    // A bound on twice the error of a key.  2^y is within 2 ulp and its exponent rounded twice, so exp(-x) is
    // within (2 + 2 |x|) 2^-23 and the sigmoid, with 1 / y within 1 ulp, within 2^-21 (exp's error reaches it
    // times at most e^-|x|); for softmax, with d = max - x, (2 + 2 d) 2^-23 of the score, the sum's the same
    // averaged over the scores (d below ln 512 there) and the reciprocal's: under 2^-18 of the score up to d = 12,
    // and past that the score is below 2^-17 of the largest.  Then the place in the low bits, at most 15 2^-23
    // of the key, and FP32 roundings of the score, the bias's move and the sums.
    const int top = __reduce_max_sync(0xffffffffu, key[0]);
    const float margin = (kSoftmax ? 0.f : 0x1p-19f) + 0x1p-16f * (as_float(top) + off);
    bool slow = top >= kInf;
    if (R.top_groups < R.groups) {
      float a = as_float(key[0]), b = P > 1 ? as_float(key[P > 1 ? 1 : 0]) : -0.f;
      for (int o = 1; o < F.L; o <<= 1) {
        const float a2 = __shfl_xor_sync(0xffffffffu, a, o), b2 = __shfl_xor_sync(0xffffffffu, b, o);
        b = fmaxf(fminf(a, a2), fmaxf(b, b2));
        a = fmaxf(a, a2);
      }
      const float gs = F.S > 1 ? a + b : a;
      // the lower group ahead in the low bits (31 2^-23 of the score), so that exactly top_groups are kept
      const int mine = g < R.groups ? (static_cast<int>(__float_as_uint(gs)) & ~31) | (31 - g) : kNone;
      int left = mine, least = 0;
      for (int j = 0; j < R.top_groups; ++j) {
        least = __reduce_max_sync(0xffffffffu, left);
        left = left == least ? kNone : left;
      }
      const int most = max(0, __reduce_max_sync(0xffffffffu, left));
      const bool kept = mine >= least;
      slow = slow || least < 0 || !(as_float(least) - as_float(most) > 2.f * margin);
      if (!kept) {
#pragma unroll
        for (int m = 0; m < P; ++m) key[m] = kNone;
      }
    }
    if (!slow) {
      int h[kDepth];
#pragma unroll
      for (int m = 0; m < kDepth; ++m) h[m] = key[m];
      int M = 0;
      unsigned from = 0;  // lane c: the c-th largest key and the lane it came from
#pragma unroll 1
      for (int c = 0; c < R.top_k; ++c) {
        const int best = __reduce_max_sync(0xffffffffu, h[0]);
        const bool here = h[0] == best;
        const unsigned who = __ballot_sync(0xffffffffu, here);
        if (lane == c) {
          M = best;
          from = who;
        }
#pragma unroll
        for (int m = 0; m + 1 < kDepth; ++m) h[m] = here ? h[m + 1] : h[m];
        h[kDepth - 1] = here ? kNone : h[kDepth - 1];
      }
      const int next = __reduce_max_sync(0xffffffffu, h[0]);
      const int after = __shfl_sync(0xffffffffu, M, lane + 1 < 32 ? lane + 1 : 31);
      const float gap = as_float(M) - as_float(lane == R.top_k - 1 ? next : after);
      const float kth = as_float(__shfl_sync(0xffffffffu, M, R.top_k - 1));
      bool unsure = P > kDepth && as_float(key[P > kDepth ? kDepth : 0]) > kth - margin;
      int id = 0;
      float x = 0.f;
      if (lane < R.top_k) {
        unsure = unsure || M < 0 || !(gap > margin) || __popc(from) != 1;
        const int src = __ffs(from) - 1;
        id = (src / F.L) * F.S + (src % F.L) * F.P + (P - 1 - (M & kMask));
        if (!unsure) x = __ldg(R.logits + tok * R.E + id);
        unsure = unsure || x - mx < -80.f;  // scores that FP32 may not hold
      }
      if (!__any_sync(0xffffffffu, unsure)) {
        float s = 0.f;
        if (lane < R.top_k) s = kSoftmax ? expf(x - mx) * inv : rcp_approx(1.f + expf(-x));
        if (R.normalize) {
          float total = s;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
          s *= rcp_approx(total);
        }
        if (lane < R.top_k) {
          R.ids[tok * R.top_k + lane] = id;
          R.weights[tok * R.top_k + lane] = s * R.scale;
        }
      } else {
        int* sorted = reinterpret_cast<int*>(s_key);
#pragma unroll
        for (int m = 0; m < P; ++m) sorted[32 * m + lane] = key[m];
        __syncwarp();
        slow = !route_candidates<P>(R, F, tok, lane, sorted, margin);
        __syncwarp();
      }
    }
    if (slow) route_exact_call(R, tok, lane, s_key);
  }
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
