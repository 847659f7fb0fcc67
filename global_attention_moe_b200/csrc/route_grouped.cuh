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
//      order is that of the exact keys: the chosen experts' scores are formed in FP32 and written (exponentials
//      and reciprocals of 1 to 2 ulp: weights within 2^-19, where FP64 would cost as much as the choice; only the
//      order needs more).
// Other tokens are marked in ids and taken up after the loop, whose registers then hold no call: the experts
// within the bound of the k-th key (at most 32) take their exact keys in FP64 and are ranked; and where that
// does not decide either (group scores within the bound, more than 32 candidates, keys that are NaN,
// infinite or far below the others), route_exact states the definition.
#pragma once

#include <stdint.h>

#include "cp_async.cuh"
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

// e^(x - m), with the difference's rounding (which alone puts it off by |x - m| 2^-24) made good; m finite.
__device__ __forceinline__ float exp_diff(float x, float m) {
  const float t = x - m, e = expf(t);
  if (!(t > -104.f)) return e;  // 0, or NaN
  const float b = t - x, rest = (x - (t - b)) - (m + b);
  return fmaf(e, rest, e);
}

// The definition for one token, by one warp: lane holds experts lane + 32 m; s_key: E floats of the warp's.
__device__ __forceinline__ void route_exact(const RouteParams& P, int64_t tok, int lane, float* s_key) {
  const float* x = P.logits + tok * P.E;
  double sc[kMaxPerLane];
  if (P.softmax) {
    float mx = -INFINITY;
#pragma unroll
    for (int m = 0; m < kMaxPerLane; ++m) {
      const float v = lane + 32 * m < P.E ? __ldg(x + lane + 32 * m) : -INFINITY;
      sc[m] = v;
      mx = fmaxf(mx, v);
    }
    mx = warp_max(mx);
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
// What the lanes hold: S = E / groups experts to a group, L = 2^lg lanes to a group, P experts to a lane.
struct FastShape {
  int S, lg, P;
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

constexpr int kNone = static_cast<int>(0x80000000u);  // below every key
__device__ __forceinline__ float as_float(int k) { return __uint_as_float(static_cast<uint32_t>(k)); }  // kNone: -0
constexpr int kInf = 0x7F800000;
constexpr float kLog2e = 1.4426950408889634f;
// Negative keys (biases at most kFarBias, -1024) count as none, and a group whose second key is one as below all
// others.  With high the largest moved bias and low the move, its sum is at most high + 1 and kFarBias - low + 1,
// which is negative, as that says, while high + |low| is below this.
constexpr float kMaxSpread = 1000.f, kFarBias = -1024.f;

// A lane's experts (e0 .. e0 + count - 1, count <= P) and their biases, moved up by the least of them (those
// far below all others aside) so that keys are positive; `most` bounds the moved biases' size and the move.
template <int P>
struct Lane {
  int g, e0, count;
  float bias[P];
  float most;
  __device__ __forceinline__ Lane(const RouteParams& R, const FastShape& F, int lane) {
    g = lane >> F.lg;
    const int in_group = (lane & ((1 << F.lg) - 1)) * F.P;
    count = g < R.groups ? max(0, min(F.P, F.S - in_group)) : 0;
    e0 = count > 0 ? g * F.S + in_group : 0;
    most = 0.f;
#pragma unroll
    for (int m = 0; m < P; ++m) bias[m] = 0.f;
    if (R.bias == nullptr) return;
    float low = INFINITY;
#pragma unroll
    for (int m = 0; m < P; ++m)
      if (m < count) {
        bias[m] = __ldg(R.bias + e0 + m);
        if (bias[m] > kFarBias) low = fminf(low, bias[m]);
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
    if (!(fabsf(low) < 1e30f)) low = 0.f;
    float high = 0.f;
#pragma unroll
    for (int m = 0; m < P; ++m) {
      // finite, so that the place in the low bits of a key does not make a NaN of -inf
      bias[m] = bias[m] - low < -1e30f ? -1e30f : bias[m] - low;
      high = fmaxf(high, bias[m]);
    }
    most = warp_max(high) + fabsf(low);
    if (!(most < kMaxSpread)) most = INFINITY;  // no bound: every token takes the exact path
  }
  template <bool kFull>
  __device__ __forceinline__ void load(const RouteParams& R, int64_t tok, float (&x)[P]) const {
    const float* p = R.logits + tok * R.E + e0;
    const bool in = tok < R.T;
    if (kFull && P >= 4) {
#pragma unroll
      for (int m = 0; m < P / 4; ++m) {
        const float4 v = in ? __ldg(reinterpret_cast<const float4*>(p) + m) : make_float4(0.f, 0.f, 0.f, 0.f);
        x[4 * m] = v.x, x[4 * m + 1] = v.y, x[4 * m + 2] = v.z, x[4 * m + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int m = 0; m < P; ++m) x[m] = in && (kFull || m < count) ? __ldg(p + m) : -INFINITY;
    }
  }
  // The approximate keys of logits x, sorted, their places in the low bits; and a bound on twice their error.
  // 2^y is within 2 ulp and its exponent rounded twice, so exp(-x) is within (2 + 2 |x|) 2^-23 and the
  // sigmoid, with 1 / y within 1 ulp, within 2^-21 (exp's error reaches it times at most e^-|x|); for softmax,
  // with d = max - x, (2 + 2 d) 2^-23 of the score, the sum's the same averaged over the scores (d below
  // ln 512 there) and the reciprocal's: under 2^-18 of the score up to d = 12, and past that the score is
  // below 2^-17 of the largest.  Then the place in the low bits, at most 15 2^-23 of the key, and FP32
  // roundings of the score, the bias's move and the sums.  mx and inv: softmax's maximum and 1 / sum.
  template <bool kSoftmax, bool kFull>
  __device__ __forceinline__ float keys(float (&x)[P], int (&key)[P], float& mx, float& inv) const {
    mx = 0.f;
    inv = 1.f;
    if (kSoftmax) {
      mx = x[0];
#pragma unroll
      for (int m = 1; m < P; ++m) mx = fmaxf(mx, x[m]);
      mx = warp_max(mx);
      float sum = 0.f;
#pragma unroll
      for (int m = 0; m < P; ++m) {
        x[m] = ex2_approx((x[m] - mx) * kLog2e);
        sum += x[m];
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      inv = rcp_approx(sum);
#pragma unroll
      for (int m = 0; m < P; ++m) x[m] = fmaf(x[m], inv, bias[m]);
    } else {
#pragma unroll
      for (int m = 0; m < P; ++m) x[m] = rcp_approx(1.f + ex2_approx(x[m] * -kLog2e)) + bias[m];
    }
#pragma unroll
    for (int m = 0; m < P; ++m) {
      const int k = (static_cast<int>(__float_as_uint(x[m])) & ~(P - 1)) | (P - 1 - m);
      key[m] = kFull || m < count ? k : kNone;
    }
    sort_desc<P>(key);
    return kSoftmax ? 0x1p-16f * (inv + most) : 0x1p-19f + 0x1p-16f * (1.f + most);
  }
};

// Which groups are kept, by the lanes' first two keys: false when the scores at the border are within the
// error.  kept: whether this lane's is.
template <int P>
__device__ __forceinline__ bool choose_groups(const RouteParams& R, const FastShape& F, const int (&key)[P], int g,
                                              float margin, bool& kept) {
  auto or_none = [](int k) { return k == kNone ? -INFINITY : as_float(k); };
  float a = or_none(key[0]), b = P > 1 ? or_none(key[P > 1 ? 1 : 0]) : -INFINITY;
#pragma unroll 1
  for (int o = 1; o < (1 << F.lg); o <<= 1) {
    const float a2 = __shfl_xor_sync(0xffffffffu, a, o), b2 = __shfl_xor_sync(0xffffffffu, b, o);
    b = fmaxf(fminf(a, a2), fmaxf(b, b2));
    a = fmaxf(a, a2);
  }
  const float gs = F.S > 1 ? a + b : a;
  // the lower group ahead in the low bits (31 2^-23 of the score), so that exactly top_groups are kept
  const int mine = g < R.groups ? (static_cast<int>(__float_as_uint(gs)) & ~31) | (31 - g) : kNone;
  int left = mine, least = 0;
#pragma unroll 4
  for (int j = 0; j < R.top_groups; ++j) {
    least = __reduce_max_sync(0xffffffffu, left);
    left = left == least ? kNone : left;
  }
  const int most = max(0, __reduce_max_sync(0xffffffffu, left));
  kept = mine >= least;
  return least >= 0 && as_float(least) - as_float(most) > 2.f * margin;
}

// A token that the fast path left: the exact keys of the experts within the error of the k-th approximate
// one, ranked.  Returns false when that does not decide: group scores at the border within the error, over 32
// candidates, keys that are not ordinary numbers.  s_key: 32 P words of the warp's.
template <int P, bool kSoftmax>
__device__ __noinline__ bool route_candidates(const RouteParams& R, const FastShape& F, int64_t tok, int lane,
                                              int* s_key) {
  const Lane<P> mine(R, F, lane);
  float v[P], mx, inv;
  int key[P];
  mine.template load<false>(R, tok, v);
  const float margin = mine.template keys<kSoftmax, false>(v, key, mx, inv);
  if (!(mine.most < kMaxSpread) || __any_sync(0xffffffffu, key[0] >= kInf)) return false;
  bool kept = true;
  if (R.top_groups < R.groups && !choose_groups<P>(R, F, key, mine.g, margin, kept)) return false;
#pragma unroll
  for (int m = 0; m < P; ++m) s_key[32 * m + lane] = kept ? key[m] : kNone;
  __syncwarp();
  int at = 0, n = 0, e = 0;  // the lane's next key; candidates; this lane's candidate
  float cut = -INFINITY;
#pragma unroll 1
  while (true) {
    const int a = at < P ? s_key[32 * at + lane] : kNone;
    const int M = __reduce_max_sync(0xffffffffu, a);
    if (M < 0 || as_float(M) < cut) break;
    if (n == 32) return false;
    const int first = __ffs(__ballot_sync(0xffffffffu, a == M)) - 1;
    if (lane == first) ++at;
    const int e1 = __shfl_sync(0xffffffffu, mine.e0, first) + P - 1 - (M & (P - 1));
    if (lane == n) e = e1;
    if (++n == R.top_k) cut = as_float(M) - margin;
  }
  if (n < R.top_k) return false;
  const float* x = R.logits + tok * R.E;
  double sc = 0.0;
  if (kSoftmax) {
    const double m = static_cast<double>(mx);
    double S = 0.0;
    for (int i = lane; i < R.E; i += 32) S += exp(static_cast<double>(__ldg(x + i)) - m);
    S = warp_sum_f64(S);
    sc = exp(static_cast<double>(__ldg(x + e)) - m) / S;
  } else {
    sc = nb::route_sigmoid_f64(static_cast<double>(__ldg(x + e)));
  }
  const float exact = static_cast<float>(sc) + (R.bias != nullptr ? __ldg(R.bias + e) : 0.f);
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const float o = __shfl_sync(0xffffffffu, exact, j);
    const int i = __shfl_sync(0xffffffffu, e, j);
    rank += (o > exact || (o == exact && i < e)) ? 1 : 0;
  }
  const bool chosen = lane < n && rank < R.top_k;
  const double total = warp_sum_f64(chosen ? sc : 0.0);
  if (chosen) {
    const double w = R.normalize ? (total == 0.0 ? 0.0 : sc / total) : sc;
    R.ids[tok * R.top_k + rank] = e;
    R.weights[tok * R.top_k + rank] = static_cast<float>(w * static_cast<double>(R.scale));
  }
  return true;
}

__device__ __noinline__ void route_exact_call(const RouteParams& R, int64_t tok, int lane, float* s_key) {
  route_exact(R, tok, lane, s_key);
}

template <int P, bool kSoftmax, bool kFull>  // kFull: every lane holds exactly P experts
__global__ void __launch_bounds__(kThreads, P <= 8 ? 4 : 2) route_fast_kernel(const __grid_constant__ RouteParams R,
                                                                              const __grid_constant__ FastShape F) {
  extern __shared__ __align__(16) float sm[];    // per warp: E keys (route_exact) or 32 P sorted ones
  __shared__ int2 s_pick[kWarps][32];            // the largest keys in turn, and the lanes that held them
  constexpr int kDepth = P < 4 ? P : 4;          // keys of a lane that the fast path can take
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2* pick = s_pick[warp];
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  {
    const Lane<P> mine(R, F, lane);
    float xn[P];  // the next token's logits
    mine.template load<kFull>(R, first, xn);
#pragma unroll 1
    for (int64_t tok = first; tok < R.T; tok += step) {
      float v[P], mx, inv;
#pragma unroll
      for (int m = 0; m < P; ++m) v[m] = xn[m];
      mine.template load<kFull>(R, tok + step, xn);  // in flight meanwhile
      int key[P];
      const float margin = mine.template keys<kSoftmax, kFull>(v, key, mx, inv);
      bool sure = !__any_sync(0xffffffffu, key[0] >= kInf);
      bool kept = true;
      if (R.top_groups < R.groups) sure = choose_groups<P>(R, F, key, mine.g, margin, kept) && sure;
      int h[kDepth];
#pragma unroll
      for (int m = 0; m < kDepth; ++m) h[m] = kept ? key[m] : kNone;
      const int deep = P > kDepth && kept ? key[P > kDepth ? kDepth : 0] : kNone;
      int taken = 0;
      __syncwarp();  // the last token's picks are read
#pragma unroll 4
      for (int c = 0; c < R.top_k; ++c) {
        const int best = __reduce_max_sync(0xffffffffu, h[0]);
        if (h[0] == best) {
          pick[c] = make_int2(best, lane);
          ++taken;
#pragma unroll
          for (int m = 0; m + 1 < kDepth; ++m) h[m] = h[m + 1];
          h[kDepth - 1] = kNone;
        }
      }
      const int next = __reduce_max_sync(0xffffffffu, h[0]);
      const int count = __reduce_add_sync(0xffffffffu, taken);  // over top_k: one key in two lanes
      __syncwarp();
      const int2 own = lane < R.top_k ? pick[lane] : make_int2(0, 0);
      const int after = lane + 1 < R.top_k ? pick[lane + 1].x : next;
      const float kth = as_float(pick[R.top_k - 1].x);
      sure = sure && count == R.top_k && !(P > kDepth && as_float(deep) > kth - margin);
      const int e = __shfl_sync(0xffffffffu, mine.e0, own.y) + P - 1 - (own.x & (P - 1));
      float x = 0.f;
      if (lane < R.top_k) {
        sure = sure && own.x >= 0 && as_float(own.x) - as_float(after) > margin;
        if (sure) x = __ldg(R.logits + tok * R.E + e);
        sure = sure && x - mx > -80.f;  // scores that FP32 holds
      }
      if (__all_sync(0xffffffffu, sure)) {
        float s = 0.f;
        if (lane < R.top_k) s = kSoftmax ? exp_diff(x, mx) * inv : rcp_approx(1.f + expf(-x));
        if (R.normalize) {
          float total = s;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
          s *= rcp_approx(total);
        }
        if (lane < R.top_k) {
          R.ids[tok * R.top_k + lane] = e;
          R.weights[tok * R.top_k + lane] = s * R.scale;
        }
      } else if (lane == 0) {
        R.ids[tok * R.top_k] = -1;  // left for below
      }
    }
  }
  __syncwarp();
  // the tokens of this warp that were left
  float* s_key = sm + warp * (32 * P > R.E ? 32 * P : R.E);
#pragma unroll 1
  for (int64_t t0 = first; t0 < R.T; t0 += 32 * step) {
    const int64_t t = t0 + lane * step;
    unsigned left = __ballot_sync(0xffffffffu, t < R.T && *(R.ids + t * R.top_k) < 0);
    for (; left; left &= left - 1) {
      const int64_t tok = t0 + (__ffs(left) - 1) * step;
      if (!route_candidates<P, kSoftmax>(R, F, tok, lane, reinterpret_cast<int*>(s_key))) {
        __syncwarp();
        route_exact_call(R, tok, lane, s_key);
      }
      __syncwarp();
    }
  }
}

// ---------------------------------------------------------------- many tokens: four threads per token
// The warp kernel spends most of its instructions on exchanges between lanes.  With enough tokens to fill the
// GPU with eight to a warp, four threads take a token: rows come into shared memory (cp.async), keys become
// integers of 23 bits above 8 bits of 255 - expert, and every choice is minimum and maximum of integers:
//   1. keys, kept in place, and each group's two largest (a group's blocks of eight experts go round the four);
//   2. the groups by their sums;
//   3. the kept groups' keys in blocks of eight: sorted, then merged into the thread's sorted eight largest, at
//      the end into the token's; the largest of what falls out is kept too, so that the k-th and the next can
//      be compared.
// Errors, and what is left for the exact paths, as in the warp kernel, with the keys' spacing 2^-23 of their
// range.  One thread per token takes fewer instructions (226 a token against 474 of the warp kernel at 256
// experts in 8 groups), but 32 rows to a warp leave six warps to an SM, and it was slower than the warp kernel
// (185 against 160 us for 262144 tokens).
constexpr int kBulkWarps = 4;  // per CTA
constexpr int kBulkThreads = 32 * kBulkWarps;
constexpr int kBulkH = 4;                // threads to a token
constexpr int kBulkTokens = 32 / kBulkH;  // tokens to a warp
constexpr int kBulkPad = 4;              // floats: rows 16 bytes apart in the banks
constexpr float kBulkOne = 8388608.f;    // 2^23: adds an integer into the low bits

__device__ __forceinline__ int max3(int a, int b, int c) { return max(a, max(b, c)); }

// The eight largest of two descending lists of eight, descending, and the largest of the rest.
__device__ __forceinline__ void merge8(int (&r)[8], const int (&k)[8], int& rest) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int a = r[i], b = k[7 - i];
    r[i] = max(a, b);
    rest = max(rest, min(a, b));
  }
#pragma unroll
  for (int d = 4; d > 0; d >>= 1)  // r is bitonic
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i & d) == 0) {
        const int a = r[i], b = r[i + d];
        r[i] = max(a, b);
        r[i + d] = min(a, b);
      }
}

template <int P, bool kSoftmax>
__global__ void __launch_bounds__(kBulkThreads) route_bulk_kernel(const __grid_constant__ RouteParams R,
                                                                  const __grid_constant__ FastShape F) {
  extern __shared__ __align__(16) float sm[];  // per warp 8 rows of E + 4; then E biases
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, stride = R.E + kBulkPad;
  const int own = lane / kBulkH, h = lane % kBulkH;
  float* rows = sm + warp * kBulkTokens * stride;
  float* mine = rows + own * stride;
  float* s_bias = sm + kBulkWarps * kBulkTokens * stride;
  // biases moved up by the least of them (those far below all others aside: -inf, a negative key)
  float low = 0.f, high = 0.f;
  if (R.bias != nullptr) {
    low = INFINITY;
    high = -INFINITY;
    for (int e = lane; e < R.E; e += 32) {
      const float b = __ldg(R.bias + e);
      if (b > kFarBias) low = fminf(low, b);
      high = fmaxf(high, b == b ? b : INFINITY);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
    high = warp_max(high);
  }
  const bool plain = high - low + fabsf(low) < kMaxSpread;  // else every token is left for the exact paths
  const float range = plain ? high - low : 1.f, off = plain ? fabsf(low) : 0.f;
  for (int e = threadIdx.x; e < R.E; e += kBulkThreads) {
    const float b = R.bias != nullptr ? __ldg(R.bias + e) : 0.f;
    s_bias[e] = b >= low ? b - low : -INFINITY;
  }
  __syncthreads();
  const int groups = R.top_groups < R.groups ? R.groups : 1, S = R.E / groups;
  const int64_t tiles = (R.T + kBulkTokens - 1) / kBulkTokens, step = static_cast<int64_t>(gridDim.x) * kBulkWarps;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kBulkWarps + warp;
  const int chunks = R.E / 4;
#pragma unroll 1
  for (int64_t tile = first; tile < tiles; tile += step) {
    const int64_t t0 = tile * kBulkTokens, tok = t0 + own;
    const int live = static_cast<int>(min(static_cast<int64_t>(kBulkTokens), R.T - t0));
    const float* from = R.logits + t0 * R.E;
    for (int r = 0; r < live; ++r, from += R.E)
      for (int c = lane; c < chunks; c += 32) cp_async_16(smem_u32(rows + r * stride + 4 * c), from + 4 * c, 16u);
    cp_async_commit();
    cp_async_wait<0>();
    __syncwarp();
    float mx = 0.f, inv = 1.f;
    if (kSoftmax) {
      mx = -INFINITY;
      for (int e = 4 * h; e < R.E; e += 4 * kBulkH) {
        const float4 v = *reinterpret_cast<const float4*>(mine + e);
        mx = fmaxf(fmaxf(mx, fmaxf(v.x, v.y)), fmaxf(v.z, v.w));
      }
#pragma unroll
      for (int o = 1; o < kBulkH; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      float sum = 0.f;
      for (int e = 4 * h; e < R.E; e += 4 * kBulkH) {
        const float4 v = *reinterpret_cast<const float4*>(mine + e);
        sum += (ex2_approx((v.x - mx) * kLog2e) + ex2_approx((v.y - mx) * kLog2e)) +
               (ex2_approx((v.z - mx) * kLog2e) + ex2_approx((v.w - mx) * kLog2e));
      }
#pragma unroll
      for (int o = 1; o < kBulkH; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      inv = rcp_approx(sum);
      __syncwarp();  // the row is rewritten below
    }
    // keys as integers: 2^23 - 2048 for the largest possible score and bias
    const float scale = (kBulkOne - 2048.f) / ((kSoftmax ? inv : 1.f) + range);
    // twice a key's error, in steps: the sigmoid's 2^-21 or the softmax's 2^-18 of the score (Lane::keys), the
    // roundings of the bias's move and of the sum
    const float err = scale * ((kSoftmax ? 0x1p-17f * inv : 0x1p-20f) + 0x1p-22f * (range + off)) + 6.f;
    const int margin = static_cast<int>(err) + 1;
    bool sure = plain && (!kSoftmax || (inv > 0.f && inv <= 1.5f));
    int v[8];  // the groups: the sum of the two largest (24 bits), the lower group ahead; a negative key: none
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      v[g] = kNone;
      if (g >= groups) continue;
      int a = kNone, b = kNone;  // the group's two largest
#pragma unroll 1
      for (int e = g * S + 8 * h; e < (g + 1) * S; e += 8 * kBulkH) {
        int k[8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float4 v4 = *reinterpret_cast<const float4*>(mine + e + 4 * u);
          const float4 w4 = *reinterpret_cast<const float4*>(s_bias + e + 4 * u);
          const float x[4] = {v4.x, v4.y, v4.z, v4.w}, bias[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float s = kSoftmax ? ex2_approx((x[i] - mx) * kLog2e) * inv : rcp_approx(1.f + ex2_approx(x[i] * -kLog2e));
            const uint32_t q = __float_as_uint(fmaf(s + bias[i], scale, kBulkOne));
            k[4 * u + i] = static_cast<int>(q * 256u + static_cast<uint32_t>(255 - (e + 4 * u + i)));
          }
          *reinterpret_cast<int4*>(mine + e + 4 * u) = make_int4(k[4 * u], k[4 * u + 1], k[4 * u + 2], k[4 * u + 3]);
        }
        if (groups > 1) {
          int p[4], q[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[i] = max(k[2 * i], k[2 * i + 1]);
            q[i] = min(k[2 * i], k[2 * i + 1]);
          }
#pragma unroll
          for (int d = 2; d > 0; d >>= 1)
#pragma unroll
            for (int i = 0; i < d; ++i) {
              q[i] = max3(min(p[i], p[i + d]), q[i], q[i + d]);
              p[i] = max(p[i], p[i + d]);
            }
          b = max3(min(a, p[0]), b, q[0]);
          a = max(a, p[0]);
        }
      }
      if (groups > 1) {
#pragma unroll
        for (int o = 1; o < kBulkH; o <<= 1) {
          const int a2 = __shfl_xor_sync(0xffffffffu, a, o), b2 = __shfl_xor_sync(0xffffffffu, b, o);
          b = max3(min(a, a2), b, b2);
          a = max(a, a2);
        }
        v[g] = b < 0 ? kNone : (((a >> 8) + (b >> 8)) << 3) | (7 - g);
      }
    }
    uint32_t kept = 1u;
    if (groups > 1) {
      kept = 0;
      int least = 0x7FFFFFFF, most = 0;
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        int rank = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) rank += v[j] > v[g] ? 1 : 0;
        const bool in = g < groups && rank < R.top_groups;
        kept |= in ? 1u << g : 0u;
        least = min(least, in ? v[g] : 0x7FFFFFFF);
        most = max(most, in ? 0 : v[g]);
      }
      sure = sure && least >= 0 && __popc(kept) == R.top_groups && (least >> 3) - (most >> 3) > 2 * margin;
    }
    int r[8], rest = kNone;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = kNone;
    for (int j = 0; j < (groups > 1 ? R.top_groups : 1); ++j) {
      // the token's j-th kept group (where there are fewer, the token is left anyway)
      const int g = kept ? __ffs(kept) - 1 : 0;
      kept &= kept - 1;
#pragma unroll 1
      for (int e = g * S + 8 * h; e < (g + 1) * S; e += 8 * kBulkH) {
        const int4 u = *reinterpret_cast<const int4*>(mine + e), w = *reinterpret_cast<const int4*>(mine + e + 4);
        int k[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
        sort_desc<8>(k);
        merge8(r, k, rest);
      }
    }
#pragma unroll
    for (int o = 1; o < kBulkH; o <<= 1) {
      int k[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) k[i] = __shfl_xor_sync(0xffffffffu, r[i], o);
      rest = max(rest, __shfl_xor_sync(0xffffffffu, rest, o));
      merge8(r, k, rest);
    }
    // neighbours that are too near one another, or a key that is none
    const int64_t gap = static_cast<int64_t>(margin) * 256 + 255;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < R.top_k) {
        const int next = i < 7 ? r[i < 7 ? i + 1 : 7] : rest;
        sure = sure && r[i] >= 0 && static_cast<int64_t>(r[i]) - next > gap;
      }
    // choices 2 h and 2 h + 1 are this thread's to write
    int e2[2];
    float w2[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int key = h == 0 ? r[u] : h == 1 ? r[2 + u] : h == 2 ? r[4 + u] : r[6 + u];
      e2[u] = 255 - (key & 255);
      w2[u] = 0.f;
      if (2 * h + u < R.top_k && sure && tok < R.T) {
        const float x = __ldg(R.logits + tok * R.E + e2[u]);
        sure = x - mx > -80.f;  // a score that FP32 holds
        w2[u] = kSoftmax ? exp_diff(x, mx) * inv : rcp_approx(1.f + expf(-x));
      }
    }
    float total = w2[0] + w2[1];
    int all = sure ? 1 : 0;
#pragma unroll
    for (int o = 1; o < kBulkH; o <<= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, o);
      all &= __shfl_xor_sync(0xffffffffu, all, o);
    }
    if (tok < R.T) {
      const float f = R.normalize ? rcp_approx(total) : 1.f;  // (times the scale it could overflow)
      int32_t* ids = R.ids + tok * R.top_k;
      float* out = R.weights + tok * R.top_k;
      if (!all) {
        if (h == 0) ids[0] = -1;  // left for below
      } else {
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (2 * h + u < R.top_k) {
            ids[2 * h + u] = e2[u];
            out[2 * h + u] = w2[u] * f * R.scale;
          }
      }
    }
    __syncwarp();  // the rows are read
  }
  __syncwarp();
  // the tokens of this warp that were left
#pragma unroll 1
  for (int64_t tile = first; tile < tiles; tile += step) {
    const int64_t t = tile * kBulkTokens + lane;
    unsigned left = __ballot_sync(0xffffffffu, lane < kBulkTokens && t < R.T && *(R.ids + t * R.top_k) < 0);
    for (; left; left &= left - 1) {
      const int64_t tok = tile * kBulkTokens + __ffs(left) - 1;
      if (!route_candidates<P, kSoftmax>(R, F, tok, lane, reinterpret_cast<int*>(rows))) {
        __syncwarp();
        route_exact_call(R, tok, lane, rows);
      }
      __syncwarp();
    }
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

// Gradient of the weights with respect to the logits (the choice itself has none).  With g = scale dw and p_j =
// s_j / sum of the chosen s:
//   sigmoid, normalised   dx_j = p_j (1 - s_j) (g_j - sum_i g_i p_i)
//   sigmoid               dx_j = g_j s_j (1 - s_j)
//   softmax, normalised   dx_j = p_j (g_j - sum_i g_i p_i)             (the softmax's own sum cancels)
//   softmax               dx_e = s_e (g_e - sum_i g_i s_i)             every expert, g_e = 0 for those not chosen
// Where one expert has nearly all of the sum, g_j and the mean agree in all bits that FP32 has, and what is left
// is the row.  So the differences are formed first: with D the chosen expert of the largest logit and
// dev_i = g_i - g_D (zero for D), g_j - sum_i g_i p_i = dev_j - sum_i p_i dev_i, where no term but D's has a p
// above one half; for the plain softmax, with C and U the scores of the chosen and of the others (C + U = 1),
// g_j - sum_i g_i s_i = g_j U + C dev_j - sum_i s_i dev_i.  1 - s is formed as a score, not by subtraction.
// An id outside [0, E) is an empty place: it takes no part.  The same id several times is one place with the sum of
// the gradients: score m s and the mean gradient for m places.
//
// FP32 throughout: sigmoid scores below one half enter p as e^(x - max x), so that p is as exact far below zero;
// plain sigmoid scores that FP32 does not hold (x below -80) are formed in FP64.
//
// Both kernels are bound by the rows they write.

// The places of one expert (lanes with the same tag; empty places: tags of their own) become one: the first takes
// the mean (kMean) or the sum of their gradients and their number, the others are emptied.  The result is in two
// floats, g + rest, so that its difference from another's is as exact as that of single places.
template <bool kMean>
__device__ __forceinline__ void join_same(int tag, int lane, bool& has, float& g, float& rest, float& count) {
  count = 1.f;
  rest = 0.f;
  const unsigned peers = __match_any_sync(0xffffffffu, tag);
  if (__all_sync(0xffffffffu, peers == (1u << lane))) return;
  double s = 0.0;
  for (int j = 0; j < 32; ++j) {
    const float o = __shfl_sync(0xffffffffu, g, j);
    if ((peers >> j) & 1u) s += static_cast<double>(o);
  }
  count = static_cast<float>(__popc(peers));
  if (kMean) s /= static_cast<double>(count);
  has = has && __ffs(peers) - 1 == lane;
  g = has ? static_cast<float>(s) : 0.f;
  if (has && fabsf(g) < INFINITY) rest = static_cast<float>(s - static_cast<double>(g));
}

// s (1 - s) g of a sigmoid score, in FP64 (few places).
__device__ __noinline__ float sigmoid_place_f64(float g, float x) {
  const double xd = static_cast<double>(x);
  return static_cast<float>(static_cast<double>(g) * nb::route_sigmoid_f64(xd) * nb::route_sigmoid_f64(-xd));
}

// All but the plain softmax: few elements of a row are not zero.  W lanes to a token (top_k <= W), 32 / W
// tokens to a warp; the rows are put together in shared memory, which is zero between uses, and written
// whole with 16-byte stores.
template <int W>
__global__ void __launch_bounds__(kThreads) route_bwd_sparse_kernel(const __grid_constant__ RouteBwdParams P) {
  constexpr int kTokens = 32 / W;
  extern __shared__ __align__(16) float sm[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / W, j = lane % W;
  float* rows = sm + warp * ((kTokens * P.E + 3) & ~3);
  const int n = kTokens * P.E;
  for (int e = lane; e < n; e += 32) rows[e] = 0.f;
  __syncwarp();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * kTokens;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kTokens; t0 < P.T; t0 += step) {
    const int64_t tok = t0 + sub;
    int id = -1;
    float g = 0.f, x = -INFINITY, rest, count;
    if (tok < P.T && j < P.top_k) {
      id = __ldg(P.ids + tok * P.top_k + j);
      g = __ldg(P.dweights + tok * P.top_k + j);
      if (id < 0 || id >= P.E) id = -1;
      if (id >= 0) x = __ldg(P.logits + tok * P.E + id);
      else g = 0.f;
    }
    bool has = id >= 0;
    join_same<true>(has ? sub * P.E + id : -1 - lane, lane, has, g, rest, count);
    auto sum = [](float v) {
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      return v;
    };
    // sigmoid: r is the larger of s and 1 - s, e r the smaller
    const float e = P.softmax ? 0.f : expf(-fabsf(x)), r = P.softmax ? 1.f : __fdiv_rn(1.f, 1.f + e);
    const float c = P.softmax ? 1.f : x >= 0.f ? e * r : r;
    float d;
    if (P.normalize) {
      float mx = has ? x : -INFINITY;
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const unsigned tops = __ballot_sync(0xffffffffu, has && x == mx) >> (sub * W) & (0xffffffffu >> (32 - W));
      const int D = sub * W + (tops ? __ffs(tops) - 1 : j);
      const float diff = (g - __shfl_sync(0xffffffffu, g, D)) + (rest - __shfl_sync(0xffffffffu, rest, D));
      const float dev = has ? diff * P.scale : 0.f;
      const float base = P.softmax ? mx : fminf(mx, 0.f);
      float s = !P.softmax && x >= 0.f ? r : base == 0.f ? e * r : exp_diff(x, base) * r;
      s = has && mx > -INFINITY ? s * count : 0.f;
      if (has && x != x) s = x;
      const float S = sum(s);
      const float p = S == 0.f ? 0.f : __fdiv_rn(s, S);
      d = (dev - sum(p * dev)) * p * c;
    } else {
      g *= count * P.scale;
      d = g * (x >= 0.f ? r : e * r) * c;
      if (__any_sync(0xffffffffu, has && x < -80.f && x > -INFINITY) && has && x < -80.f) d = sigmoid_place_f64(g, x);
    }
    float* at = rows + sub * P.E + id;
    if (has) *at = d;
    __syncwarp();
    const int64_t left = (P.T - t0) * P.E;
    float* out = P.dlogits + t0 * P.E;
    if ((P.E & 3) == 0) {
      const int m = static_cast<int>(min(static_cast<int64_t>(n), left)) / 4;
      for (int e = lane; e < m; e += 32) reinterpret_cast<float4*>(out)[e] = reinterpret_cast<const float4*>(rows)[e];
    } else {
      const int m = static_cast<int>(min(static_cast<int64_t>(n), left));
      for (int e = lane; e < m; e += 32) out[e] = rows[e];
    }
    __syncwarp();
    if (has) *at = 0.f;
    __syncwarp();
  }
}

// Softmax weights that were not renormalised: every element of the row.  One warp per token, kM >= E / 32 experts to
// a lane (with 16 for every E, 128 experts of 4099 tokens take 5.7 us instead of 4.8; 65536 x 256: 59 us).
template <int kM>
__global__ void __launch_bounds__(kThreads) route_bwd_dense_kernel(const __grid_constant__ RouteBwdParams P) {
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t tok = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); tok < P.T; tok += step) {
    const float* x = P.logits + tok * P.E;
    float v[kM];
    int id = -1;
    float g = 0.f, xj = -INFINITY, rest, count;
    if (lane < P.top_k) {
      id = __ldg(P.ids + tok * P.top_k + lane);
      g = __ldg(P.dweights + tok * P.top_k + lane);
      if (id < 0 || id >= P.E) id = -1;
    }
    float mx = -INFINITY;
#pragma unroll
    for (int m = 0; m < kM; ++m)
      if (32 * m < P.E) {
        v[m] = lane + 32 * m < P.E ? __ldg(x + lane + 32 * m) : -INFINITY;
        mx = fmaxf(mx, v[m]);
      }
    if (id >= 0) xj = __ldg(x + id);
    else g = 0.f;
    bool has = id >= 0;
    join_same<false>(has ? id : -1 - lane, lane, has, g, rest, count);
    uint32_t mine = 0;  // bit m: this lane's expert lane + 32 m is chosen
#pragma unroll 4
    for (int c = 0; c < P.top_k; ++c) {
      const int o = __shfl_sync(0xffffffffu, id, c);
      if (o >= 0 && (o & 31) == lane) mine |= 1u << (o >> 5);
    }
    float xm = has ? xj : -INFINITY;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      xm = fmaxf(xm, __shfl_xor_sync(0xffffffffu, xm, o));
    }
    const unsigned tops = __ballot_sync(0xffffffffu, has && xj == xm);
    const int D = tops ? __ffs(tops) - 1 : lane;
    const float dev = ((g - __shfl_sync(0xffffffffu, g, D)) + (rest - __shfl_sync(0xffffffffu, rest, D))) * P.scale;
    g *= P.scale;
    // sums over the exponentials as they are; 1 / (U + C) comes in at the end
    float U = 0.f;
#pragma unroll
    for (int m = 0; m < kM; ++m)
      if (32 * m < P.E) {
        v[m] = lane + 32 * m < P.E ? expf(v[m] - mx) : 0.f;
        U += (mine >> m) & 1u ? 0.f : v[m];
      }
    const float s = has ? exp_diff(xj, mx) : 0.f;
    float C = s, gm = g * s, dm = has ? dev * s : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      U += __shfl_xor_sync(0xffffffffu, U, o);
      C += __shfl_xor_sync(0xffffffffu, C, o);
      gm += __shfl_xor_sync(0xffffffffu, gm, o);
      dm += __shfl_xor_sync(0xffffffffu, dm, o);
    }
    const float inv = __fdiv_rn(1.f, U + C), inv2 = inv * inv;
    float* out = P.dlogits + tok * P.E;
    const float f = -gm * inv2;
#pragma unroll
    for (int m = 0; m < kM; ++m)
      if (lane + 32 * m < P.E && !((mine >> m) & 1u)) out[lane + 32 * m] = f * v[m];
    if (has) out[id] = s * inv2 * (fmaf(g, U, C * dev) - dm);
  }
}

}  // namespace rg
}  // namespace mimo
