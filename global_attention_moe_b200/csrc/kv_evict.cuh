// kv_evict.cuh -- eviction from the page-size-1 KV cache by accumulated attention weight.
//
// Sequence b's n_b entries of the index list stay as they are when n_b <= budget; else its first
// keep_first, its last keep_recent and, of the rest, those with the largest weights (ties to the earlier
// entry, NaN below everything) stay, budget in all, in their order.  The kept rows and weights are packed
// without gaps, and the rows that left are packed in a list of their own.
//
// A cluster of C CTAs takes one sequence, each warp a contiguous piece of it.  Weights become unsigned
// integers of the same order (entries that must stay: the largest), are kept in shared memory, and the
// budget-th largest is found by a radix select of 11 + 11 + 10 bits: each CTA counts its digits in shared
// memory, and every CTA adds the cluster's counts over distributed shared memory.  With S(i) and E(i) the
// entries before i that are above / equal to that threshold and m the equal ones that stay, entry i's place
// is S(i) + min(E(i), m), so one count per warp and one exchange of the warps' counts place every entry.
// All of it is integer arithmetic: the result is the same for any C, which goes by the sequences' length and number
// (launch_evict).  64 sequences of 1024 to 8192 entries: 11.4 us, a chain of barriers; 131072 entries on eight SMs:
// 26 us.
#pragma once

#include <stdint.h>

#include "params.cuh"
#include "sm100.cuh"

namespace mimo {
namespace ev {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;  // CTAs to a sequence
constexpr int kBins = 2048;
constexpr int kAhead = 8;  // loads of 32 entries that a warp has in flight
constexpr uint32_t kMust = 0xFFFFFFFFu;  // above every weight's bits

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
  int32_t key_cap;            // weights' bits that fit in a CTA's shared memory
};

struct Shared {
  uint32_t hist[3 * kBins];  // of the three digits
  uint32_t scan[2][kWarps];   // block-wide sums
  uint32_t above[kWarps], equal[kWarps];  // the warps' counts
  uint32_t pick[2];           // digit, entries of it that stay
};
// then key_cap words: the bits of the CTA's entries
constexpr uint32_t kFixedBytes = (sizeof(Shared) + 15) / 16 * 16;

// Bits that order like the weight as unsigned integers: 0 for NaN, then from -inf up; +0 and -0 the same.
__device__ __forceinline__ uint32_t order_bits(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t warp_scan(uint32_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// Inclusive sum over the CTA's threads; `buf` alternates between calls.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* buf, int lane, int warp) {
  v = warp_scan(v, lane);
  if (lane == 31) buf[warp] = v;
  __syncthreads();
  const uint32_t w = warp_scan(buf[lane], lane);
  const uint32_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return warp > 0 ? v + before : v;
}

template <int C>
__global__ void __cluster_dims__(C, 1, 1) __launch_bounds__(kThreads, 1)
    kv_evict_kernel(const __grid_constant__ EvictParams P) {
  extern __shared__ __align__(16) float sm[];
  Shared* S = reinterpret_cast<Shared*>(sm);
  const int b = blockIdx.x / C, r = C > 1 ? blockIdx.x % C : 0, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 3 * kBins; i += kThreads) S->hist[i] = 0;
  // the index list's bounds, and where this sequence's entries go: the kept lengths before it
  uint32_t mine = 0;
  bool ok = true;
  for (int i = tid; i < P.num_seqs; i += kThreads) {
    const int lo = __ldg(P.kv_indptr + i), hi = __ldg(P.kv_indptr + i + 1);
    if (lo < 0 || hi < lo || hi > P.total_kv || hi - lo > P.max_kv_len || (i == 0 && lo != 0)) ok = false;
    if (i < b && hi > lo) mine += static_cast<uint32_t>(min(hi - lo, P.budget));
  }
  const uint32_t sum = block_scan(mine, S->scan[0], lane, warp);
  if (tid == kThreads - 1) S->pick[0] = sum;
  if (__syncthreads_or(!ok)) {  // inconsistent (every CTA sees the same list): report and write nothing
    if (tid == 0 && blockIdx.x == 0) atomicOr(&g_mimo_error, kErrSeqlens);
    return;
  }
  const int before = static_cast<int>(S->pick[0]);
  const int beg = __ldg(P.kv_indptr + b), n = __ldg(P.kv_indptr + b + 1) - beg;
  if (tid == 0 && r == 0) {
    if (b == 0) P.new_indptr[0] = 0;
    P.new_indptr[b + 1] = before + min(n, P.budget);
  }
  const float* w = P.weights + beg;
  const int32_t* idx = P.kv_indices + beg;
  int32_t* to_idx = P.new_indices + before;
  float* to_w = P.new_weights + before;
  int32_t* away = P.freed + (beg - before);
  if (n <= P.budget) {  // the same for every CTA of the cluster
    for (int i = r * kThreads + tid; i < n; i += C * kThreads) {
      to_idx[i] = __ldg(idx + i);
      to_w[i] = __ldg(w + i);
    }
    return;
  }
  // this warp's piece [i0, i1), a multiple of 32 entries; its bits are at keys[i - base]
  const int piece = static_cast<int>(((static_cast<int64_t>(n) + C * kWarps - 1) / (C * kWarps) + 31) / 32 * 32);
  const int64_t start = static_cast<int64_t>(r * kWarps + warp) * piece;
  const int i0 = static_cast<int>(min(start, static_cast<int64_t>(n)));
  const int i1 = static_cast<int>(min(start + piece, static_cast<int64_t>(n)));
  const bool stored = static_cast<int64_t>(piece) * kWarps <= P.key_cap;
  uint32_t* keys = reinterpret_cast<uint32_t*>(sm) + kFixedBytes / 4 + warp * piece;
  const int must_from = n - P.recent;
  auto bits_at = [&](int i) -> uint32_t {
    const uint32_t o = order_bits(__ldg(w + i));
    return (i < P.first || i >= must_from) ? kMust : o;
  };
  // f of every entry's bits, in any order: the lane's share of the piece
  auto each_key = [&](auto f) {
    if (stored) {
      const uint4* k4 = reinterpret_cast<const uint4*>(keys);
      const int n4 = (i1 - i0) / 4;
      for (int q = lane; q < n4; q += 32) {
        const uint4 v = k4[q];
        f(v.x), f(v.y), f(v.z), f(v.w);
      }
      if (lane < (i1 - i0) % 4) f(keys[4 * n4 + lane]);
    } else {
      for (int i = i0 + lane; i < i1; i += 32) f(bits_at(i));
    }
  };
  auto key_at = [&](int i) -> uint32_t { return stored ? keys[i - i0] : bits_at(i); };
  // first digit, while the bits are stored
  for (int i = i0; i < i1; i += 32 * kAhead) {
    uint32_t o[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) o[k] = i + 32 * k + lane < i1 ? bits_at(i + 32 * k + lane) : 0u;
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i + 32 * k + lane < i1) {
        if (stored) keys[i + 32 * k + lane - i0] = o[k];
        atomicAdd(&S->hist[o[k] >> 21], 1u);
      }
  }
  __syncwarp();  // a lane reads the others' bits from here on
  uint32_t need = static_cast<uint32_t>(P.budget), prefix = 0;
  // pass p: digit of `width` bits at `shift`, over the entries that agree with the prefix above it
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    const int shift = p == 0 ? 21 : p == 1 ? 10 : 0;
    if (p > 0) {
      const int above = p == 1 ? 21 : 10;
      const uint32_t digit_mask = p == 1 ? 2047u : 1023u;
      each_key([&](uint32_t o) {
        if ((o >> above) == (prefix >> above)) atomicAdd(&S->hist[p * kBins + ((o >> shift) & digit_mask)], 1u);
      });
    }
    if (C > 1) cluster_sync();
    else __syncthreads();
    // the largest digits first: thread t adds bins 2047 - 2t and 2046 - 2t over the cluster
    const int hi = kBins - 1 - 2 * tid;
    uint32_t a = 0, c = 0;
    if (C > 1) {
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const uint2 v = ld_cluster_u32x2(&S->hist[p * kBins + hi - 1], k);
        a += v.x;
        c += v.y;
      }
    } else {
      c = S->hist[p * kBins + hi];
      a = S->hist[p * kBins + hi - 1];
    }
    const uint32_t upto = block_scan(a + c, S->scan[(p + 1) & 1], lane, warp), from = upto - a - c;
    if (from < need && upto >= need) {  // one thread, for need >= 1
      const bool first = from + c >= need;
      S->pick[0] = static_cast<uint32_t>(first ? hi : hi - 1);
      S->pick[1] = need - (first ? from : from + c);
    }
    __syncthreads();
    if (need > 0) {
      prefix |= S->pick[0] << shift;
      need = S->pick[1];
    } else {
      prefix = kMust;  // nothing stays (budget 0: no entry must)
    }
    // pick is written again only after the next pass's barriers
  }
  // counts of entries above and equal to the threshold
  uint32_t above = 0, equal = 0;
  each_key([&](uint32_t o) {
    above += o > prefix ? 1u : 0u;
    equal += o == prefix ? 1u : 0u;
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    above += __shfl_xor_sync(0xffffffffu, above, o);
    equal += __shfl_xor_sync(0xffffffffu, equal, o);
  }
  if (lane == 0) {
    S->above[warp] = above;
    S->equal[warp] = equal;
  }
  if (C > 1) cluster_sync();
  else __syncthreads();
  above = equal = 0;  // those of the warps before this one
#pragma unroll
  for (int k = 0; k < C; ++k) {
    const bool mine_too = k < r || (k == r && lane < warp);
    if (C > 1) {
      if (mine_too) {
        above += ld_cluster_u32(&S->above[lane], k);
        equal += ld_cluster_u32(&S->equal[lane], k);
      }
    } else if (mine_too) {
      above += S->above[lane];
      equal += S->equal[lane];
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    above += __shfl_xor_sync(0xffffffffu, above, o);
    equal += __shfl_xor_sync(0xffffffffu, equal, o);
  }
  if (C > 1) cluster_arrive();  // this thread reads no other CTA's memory any more
  const unsigned below = (1u << lane) - 1u;
  for (int i = i0; i < i1; i += 32 * kAhead) {
    int32_t row[kAhead];
    float wt[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int at = i + 32 * k + lane;
      row[k] = at < i1 ? __ldg(idx + at) : 0;
      wt[k] = at < i1 ? __ldg(w + at) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int at = i + 32 * k + lane;
      const bool in = at < i1;
      const uint32_t o = in ? key_at(at) : 0u;
      const unsigned ma = __ballot_sync(0xffffffffu, in && o > prefix), me = __ballot_sync(0xffffffffu, in && o == prefix);
      const uint32_t e = equal + __popc(me & below);  // equal ones before this entry
      const uint32_t place = above + __popc(ma & below) + min(e, need);
      if (in) {
        if (o > prefix || (o == prefix && e < need)) {
          to_idx[place] = row[k];
          to_w[place] = wt[k];
        } else {
          away[at - place] = row[k];
        }
      }
      above += __popc(ma);
      equal += __popc(me);
    }
  }
  if (C > 1) cluster_wait();  // the cluster's other CTAs may still read this one's memory
}

}  // namespace ev
}  // namespace mimo
