// kv_evict.cuh -- eviction from the page-size-1 KV cache by accumulated attention weight.
//
// Sequence b's n_b entries of the index list stay as they are when n_b <= budget; else its first
// keep_first, its last keep_recent and, of the rest, those with the largest weights (ties to the earlier
// entry, NaN below everything) stay, budget in all, in their order.  The kept rows and weights are packed
// without gaps, and the rows that left are packed in a list of their own.
#pragma once

#include <stdint.h>

#include "params.cuh"
#include "sm100.cuh"

namespace mimo {
namespace ev {

constexpr int kThreads = 1024;

struct EvictParams {
  const float* weights;       // [total_kv]
  const int32_t* kv_indices;  // [total_kv]
  const int32_t* kv_indptr;   // [num_seqs + 1]
  int32_t* new_indices;       // kept rows
  float* new_weights;         // their weights
  int32_t* new_indptr;        // [num_seqs + 1]
  int32_t* freed;             // rows that left
  int32_t num_seqs, total_kv, max_kv_len;
  int32_t budget, first, recent;
};

// Bits that order like the weight as unsigned integers: 0 for NaN, then from -inf up; +0 and -0 the same.
__device__ __forceinline__ uint32_t order_bits(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Inclusive sums of two counts over the CTA's threads (packed in one 64-bit word), and the totals.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, unsigned long long* s_warp,
                                                         unsigned long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  unsigned long long before = 0, all = 0;
  for (int k = 0; k < kThreads / 32; ++k) {
    if (k < warp) before += s_warp[k];
    all += s_warp[k];
  }
  __syncthreads();
  total = all;
  return v + before;
}

// One CTA per sequence.
__global__ void __launch_bounds__(kThreads) kv_evict_kernel(const __grid_constant__ EvictParams P) {
  __shared__ uint32_t s_hist[256];
  __shared__ unsigned long long s_warp[kThreads / 32];
  __shared__ uint32_t s_pick[2];
  const int b = blockIdx.x, tid = threadIdx.x;
  // where the sequence's entries go: the kept lengths of the sequences before it
  long long before = 0;
  bool ok = true;
  {
    unsigned long long mine = 0, all = 0;
    for (int i = tid; i < P.num_seqs; i += kThreads) {
      const int lo = __ldg(P.kv_indptr + i), hi = __ldg(P.kv_indptr + i + 1);
      if (lo < 0 || hi < lo || hi > P.total_kv || hi - lo > P.max_kv_len || (i == 0 && lo != 0)) ok = false;
      if (i < b && hi > lo) mine += static_cast<unsigned long long>(min(hi - lo, P.budget));
    }
    block_scan(mine, s_warp, all);
    before = static_cast<long long>(all);
  }
  if (__syncthreads_or(!ok)) {  // an inconsistent index list: report and write nothing
    if (tid == 0 && b == 0) atomicOr(&g_mimo_error, kErrSeqlens);
    return;
  }
  const int beg = __ldg(P.kv_indptr + b), n = __ldg(P.kv_indptr + b + 1) - beg;
  const int kept = min(n, P.budget);
  if (tid == 0) {
    if (b == 0) P.new_indptr[0] = 0;
    P.new_indptr[b + 1] = static_cast<int32_t>(before + kept);
  }
  const float* w = P.weights + beg;
  const int32_t* idx = P.kv_indices + beg;
  int32_t* to_idx = P.new_indices + before;
  float* to_w = P.new_weights + before;
  int32_t* away = P.freed + (beg - before);
  if (n <= P.budget) {
    for (int i = tid; i < n; i += kThreads) {
      to_idx[i] = __ldg(idx + i);
      to_w[i] = __ldg(w + i);
    }
    return;
  }
  // the (budget - first - recent)-th largest weight of entries first .. n - recent - 1, digit by digit
  const int lo = P.first, hi = n - P.recent;
  uint32_t need = static_cast<uint32_t>(P.budget - P.first - P.recent), prefix = 0;
  for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
    for (int i = tid; i < 256; i += kThreads) s_hist[i] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    for (int i = lo + tid; i < hi; i += kThreads) {
      const uint32_t o = order_bits(__ldg(w + i));
      if ((o & mask) == prefix) atomicAdd(&s_hist[(o >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t left = need;
      int d = 255;
      for (; d > 0 && s_hist[d] < left; --d) left -= s_hist[d];
      s_pick[0] = static_cast<uint32_t>(d);
      s_pick[1] = left;
    }
    __syncthreads();
    prefix |= s_pick[0] << shift;
    need = s_pick[1];
    __syncthreads();
  }
  // of the entries equal to the threshold, the first `need` stay
  const bool any = P.budget > P.first + P.recent;
  uint32_t ties = 0, out = 0;
  for (int base = 0; base < n; base += kThreads) {
    const int i = base + tid;
    float v = 0.f;
    bool keep = false, tie = false;
    if (i < n) {
      v = __ldg(w + i);
      keep = i < lo || i >= hi;
      if (!keep && any) {
        const uint32_t o = order_bits(v);
        keep = o > prefix;
        tie = o == prefix;
      }
    }
    unsigned long long total;
    const unsigned long long t = block_scan(tie ? 1u : 0u, s_warp, total);
    if (tie && ties + static_cast<uint32_t>(t) <= need) keep = true;
    ties += static_cast<uint32_t>(total);
    const unsigned long long k = block_scan(keep ? 1u : 0u, s_warp, total);
    if (i < n) {
      const uint32_t at = out + static_cast<uint32_t>(k);  // kept entries up to and with this one
      if (keep) {
        to_idx[at - 1] = __ldg(idx + i);
        to_w[at - 1] = v;
      } else {
        away[i - at] = __ldg(idx + i);
      }
    }
    out += static_cast<uint32_t>(total);
  }
}

}  // namespace ev
}  // namespace mimo
