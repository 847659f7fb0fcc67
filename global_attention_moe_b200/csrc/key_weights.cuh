// key_weights.cuh -- the attention weight each cached key receives from a step's new queries, for the
// page-size-1 KV cache:
//
//   w_j = prev_j + sum over the sequence's query heads h and new queries i that see key j of
//         exp(q~_{i,h} . k~_j / sqrt(192) - lse_{h,i})
//
// with q~, k~, positions, window and masking as in the KV-cache attention (attn_decode.cuh) and lse the
// normaliser that it returned (the sink included), so a query's weights over its keys sum to one (less
// the sink's share).
//
// Precision: the weights are FP32 and are summed over many steps, so the scores are formed more exactly
// than the attention's: the rotated dims of Q and K are each split into an FP16 value and what is left, times
// 2^11 and rounded to FP16 (22 bits from 2^-14 on, 2^-36 below: unscaled, the rest would run out of FP16's
// exponents from about 1 down, and queries of 3000 with keys of 3e-4 were off by 1.5e-5).  Three products hi hi +
// 2^-11 (hi lo + lo hi) take the place of one, the last two first: the MMA that starts hi hi takes the accumulator
// times 2^-11.  The pass-through dims are exact in BF16.  Rotation angles come from FP64-reduced positions.
// Exponentials are ex2.approx (2 ulp); sums are FP32, four chains to a key and part.
//
// Three launches:
//   1. kw_prep_kernel: Q rotated and split once, into rows of 256 16-bit values (hi 64, lo 64, pass 128)
//      ordered by (KV head, token, head of the group), lse in log2 units beside it, and the running count
//      of work units per sequence;
//   2. kw_main_kernel: persistent, one CTA per SM.  A unit is (sequence, KV head, part f of the query
//      tiles, tile of 128 keys).  The keys are the M = 128 rows of the tcgen05 product and the queries its
//      N columns, so that a thread owns one key (a TMEM lane) and adds that key's exponentials in a
//      register, with no reduction across threads.  Each unit writes its sums to a partial row [f, KV
//      head][key];
//   3. kw_join_kernel: adds the partial rows in a fixed order, and prev; writes nothing if launch 2 gave up.
//
// Warp roles of the main kernel (24 warps; registers are dealt out by warpgroup):
//   warp 0       TMEM owner; issues the MMAs (A = K from TMEM, B = Q from shared memory)
//   warp 1       Q loader: TMA boxes of the prepared rows, and their lse
//   warp 2       angles of the key tiles' first positions
//   warps 4-11   sums (thread = key = TMEM lane): two groups of four that take the score tiles in turn, since
//                one group's sums take longer than a tile's products (1550 cycles)
//   warps 12-19  K rotation, two threads to a key: rows from shared memory, BF16 -> FP16 hi and lo (angle
//                addition from the tile's first key; paired FP32 arithmetic), into TMEM with the pass dims
//   warps 20-23  K fetcher: gathers the tile's rows by index with cp.async into the 128-byte-swizzled layout
// Units are walked in order by every role.  A gathered K tile (48 KB) stays in its stage only until it has been
// rotated into one of two TMEM buffers (128 columns: hi, lo, pass): the gather's latency, about 2.5 us for rows
// spread over the cache, is what has to be covered, and the stages are what covers it.  It also leaves the
// tensor cores one operand to read from shared memory instead of two, whose 128 bytes a cycle they would
// take whole.  CTA c takes KV head c % hkv and a run of that head's units, so that CTAs side by side read the
// same cache rows.  With one query tile per sequence (decode steps, QS = 1) the Q tile stays in shared memory
// while the keys of its sequence stream through KS stages; with more (chunked prefill, QS = 2) a key tile stays
// in TMEM while the query tiles stream through two Q stages.
//
// 64 sequences of 8 tokens on 1024 to 8192 keys (470 MB of rows, 59 us of three-product MMAs): 134 us at 1965 MHz,
// 157 to 161 where the power cap holds the clock at 1590, the gather and the sums' exponentials about level; a chunk
// of 300 tokens on 5000 keys: 84 to 88 us.  The role loops are kept short: unrolled further, their instructions no
// longer fit the SM's cache and the decode case took 228 us.
#pragma once

#include "attn_decode.cuh"
#include "cp_async.cuh"

namespace mimo {
namespace kw {

constexpr int kThreads = 768;
constexpr int kTile = 128;             // keys per unit
constexpr uint32_t kUnit = 16384;      // 128 rows x 64 dims x 2 B
constexpr uint32_t kStage = 3 * kUnit;  // a gathered K tile: dims 0..63, 64..127, 128..191
constexpr uint32_t kCtrlOff = 14 * kUnit;  // KS stages, then QS Q tiles
constexpr int kLseSlots = 4;
constexpr uint32_t kTmemCols = 512;        // two score tiles of at most 128 columns, then two K tiles
constexpr uint32_t kColK = 256;
constexpr int kRotThreads = 256;
// registers of a thread, by warpgroup: 80 at launch; 56 + 2 x 80 + 2 x 104 + 56 = 6 x 80
constexpr uint32_t kRegsSmall = 56, kRegsRotate = 104, kRegsFetch = 56;
constexpr int kMaxKS = 4;
constexpr int kMaxSplits = 16;

struct Params {
  const uint16_t* q;          // bf16 [Tq, hq, 192]
  const uint16_t* k_cache;    // bf16 [cache_rows, hkv, 192]
  const int32_t* kv_indices;  // [total_kv]
  const int32_t* kv_indptr;   // [num_seqs + 1]
  const int32_t* cu_q;        // [num_seqs + 1]
  const float* lse;           // [hq, Tq]
  const float* prev;          // [total_kv] or nullptr
  float* out;                 // [total_kv]
  uint16_t* qs;               // workspace: [hkv * Tq * group, 256]
  float* lse2;                // workspace: [hkv * Tq * group], log2 units
  long long* units;           // workspace: [num_seqs + 1], running count of units; then whether launch 2 gave up
  float* partial;             // workspace: [parts * hkv, total_kv]
  int32_t num_seqs, total_q, total_kv, cache_rows, max_q_len, max_kv_len;
  int32_t hq, hkv, group;
  int32_t window;             // < 0: global causal layer
  int32_t splits;             // parts of the query tiles
  int32_t parts;              // partial rows to a KV head: 1, or two to a split
  int32_t ntile;              // query rows per tile (MMA N): multiple of 16, at most 128
  float scale_log2;
  uint64_t wait_limit_ns;
  double theta[kRopeDims / 2];
};

// Sequence b: false when its bounds are inconsistent.
struct Seq {
  int q_beg, q_len, kv_beg, kv_len;
  int lo;     // first key that any of its queries sees
  int tiles;  // 128-key tiles of the keys that are seen
};
__device__ __forceinline__ bool load_seq(const Params& P, int b, Seq& s) {
  s.q_beg = __ldg(P.cu_q + b);
  s.q_len = __ldg(P.cu_q + b + 1) - s.q_beg;
  s.kv_beg = __ldg(P.kv_indptr + b);
  s.kv_len = __ldg(P.kv_indptr + b + 1) - s.kv_beg;
  s.lo = 0;
  s.tiles = 0;
  if (s.q_beg < 0 || s.q_len < 0 || s.q_len > P.max_q_len || s.q_len > P.total_q - s.q_beg || s.kv_beg < 0 ||
      s.kv_len < s.q_len || s.kv_len > P.max_kv_len || s.kv_len > P.total_kv - s.kv_beg)
    return false;
  if (s.q_len == 0) {
    s.lo = s.kv_len;  // no query sees any key
    return true;
  }
  s.lo = dec::key_lo(s.kv_len, s.q_len, P.window);
  s.tiles = (s.kv_len - s.lo + kTile - 1) / kTile;
  return true;
}

// cos / sin of pos theta, the angle reduced in FP64.
__device__ __forceinline__ float2 angle(int pos, double theta) {
  const double a = static_cast<double>(pos) * theta;
  const double n = rint(a * kInvTwoPi);
  float s, c;
  sincosf(static_cast<float>(fma(-n, kTwoPi, a)), &s, &c);
  return make_float2(c, s);
}

constexpr int kLoBits = 11;  // the rest is held times 2^kLoBits, at most as large as x

// x as an FP16 value and the FP16 rounding of the rest, scaled.
__device__ __forceinline__ void split16(float x, __half& hi, __half& lo) {
  hi = __float2half_rn(x);
  lo = __float2half_rn((x - __half2float(hi)) * static_cast<float>(1 << kLoBits));
}

// ---------------------------------------------------------------- launch 1
// Blocks 0 .. gridDim - 2: one warp per (token, kPrepHeads query heads), lane = RoPE pair; the rows are loaded
// before the token's sequence is looked up.  Last block: the running count of units.
constexpr int kPrepThreads = 256;
constexpr int kPrepHeads = 4;

// The last entry of the ascending list at most t (n >= 1 entries, the first taken as at most t), by a warp.
__device__ __forceinline__ int find_seq(const int32_t* list, int n, int t, int lane) {
  int a = 0;
  while (n > 1) {
    const int stride = (n + 31) / 32;  // a + lane stride, the ones at most t
    const int at = lane * stride;
    const unsigned m = __ballot_sync(0xffffffffu, at < n && (at == 0 || __ldg(list + a + at) <= t));
    const int k = 31 - __clz(m);
    a += k * stride;
    n = min(stride, n - k * stride);
  }
  return a;
}

__global__ void __launch_bounds__(kPrepThreads) kw_prep_kernel(const __grid_constant__ Params P) {
  __shared__ long long s_warp[kPrepThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == gridDim.x - 1) {
    long long before = 0;
    bool bad = false;
    for (int b0 = 0; b0 < P.num_seqs; b0 += kPrepThreads) {
      const int b = b0 + static_cast<int>(threadIdx.x);
      long long v = 0;
      if (b < P.num_seqs) {
        Seq s;
        bad |= !load_seq(P, b, s);
        v = static_cast<long long>(s.tiles) * P.hkv * P.splits;
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      if (lane == 31) s_warp[warp] = v;
      __syncthreads();
      for (int k = 0; k < warp; ++k) v += s_warp[k];
      if (b < P.num_seqs) P.units[b + 1] = before + v;
      for (int k = 0; k < kPrepThreads / 32; ++k) before += s_warp[k];
      __syncthreads();
    }
    if (threadIdx.x == 0) P.units[0] = P.units[P.num_seqs + 1] = 0;
    if (bad) atomicOr(&g_mimo_error, kErrSeqlens);
    return;
  }
  const int hblocks = (P.hq + kPrepHeads - 1) / kPrepHeads;
  const long long item = static_cast<long long>(blockIdx.x) * (kPrepThreads / 32) + warp;
  const int t = static_cast<int>(item / hblocks);
  const int h0 = static_cast<int>(item % hblocks) * kPrepHeads;
  if (t >= P.total_q) return;
  const int nh = min(kPrepHeads, P.hq - h0);
  const uint16_t* src = P.q + (static_cast<size_t>(t) * P.hq + h0) * kHeadDimQK;
  uint16_t x16[kPrepHeads], y16[kPrepHeads];
  uint2 pass[kPrepHeads];
#pragma unroll
  for (int i = 0; i < kPrepHeads; ++i)
    if (i < nh) {
      x16[i] = __ldg(src + i * kHeadDimQK + lane);
      y16[i] = __ldg(src + i * kHeadDimQK + lane + 32);
      pass[i] = __ldg(reinterpret_cast<const uint2*>(src + i * kHeadDimQK + 64) + lane);
    }
  const float l = lane < nh ? __ldg(P.lse + static_cast<size_t>(h0 + lane) * P.total_q + t) * dec::kLog2e : 0.f;
  const double theta = P.theta[lane];
  Seq s;
  const bool ok = load_seq(P, find_seq(P.cu_q, P.num_seqs, t, lane), s) && t >= s.q_beg && t < s.q_beg + s.q_len;
  if (!ok) return;  // rows of no sequence are never read as queries
  const float2 cs = angle(s.kv_len - s.q_len + (t - s.q_beg), theta);
  float amax = 0.f;
  int g = h0 / P.group, hh = h0 - g * P.group;  // KV head, head in the group
#pragma unroll
  for (int i = 0; i < kPrepHeads; ++i)
    if (i < nh) {
      const size_t row = (static_cast<size_t>(g) * P.total_q + t) * P.group + hh;
      if (++hh == P.group) {
        hh = 0;
        ++g;
      }
      uint16_t* dst = P.qs + row * 256;
      const float x = __uint_as_float(static_cast<uint32_t>(x16[i]) << 16);
      const float y = __uint_as_float(static_cast<uint32_t>(y16[i]) << 16);
      const float u = x * cs.x - y * cs.y, v = y * cs.x + x * cs.y;
      amax = fmaxf(amax, fmaxf(fabsf(u), fabsf(v)));
      __half uh, ul, vh, vl;
      split16(u, uh, ul);
      split16(v, vh, vl);
      __half* d = reinterpret_cast<__half*>(dst);
      d[lane] = uh;
      d[lane + 32] = vh;
      d[lane + 64] = ul;
      d[lane + 96] = vl;
      reinterpret_cast<uint2*>(dst + 128)[lane] = pass[i];
      if (lane == i) P.lse2[row] = l;
    }
  if (amax > 65504.f) atomicOr(&g_mimo_error, kErrRange);
}

// ---------------------------------------------------------------- launch 2
struct Ctrl {
  uint64_t k_landed[kMaxKS], k_empty[kMaxKS];  // stages
  uint64_t k_full[2], k_free[2];               // K tiles in TMEM
  uint64_t a_full[2], a_empty[2];              // angles of a tile's first key
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], s_empty[2];
  uint64_t lse_full[kLseSlots];
  uint32_t tmem_base;
  int abort;
  alignas(16) float k_cos[2][kRopeDims / 2], k_sin[2][kRopeDims / 2];  // at the tile's first key, by tile parity
  alignas(16) float lse2[kLseSlots][kTile];                // of the Q loads, in turn (read as float4)
};
constexpr uint32_t kSmemBytes = kCtrlOff + ((sizeof(Ctrl) + 15) & ~size_t(15));
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

struct Unit {
  int kv_beg, k0, nk;  // index-list offset, first key, keys of the tile
  int kv_len;
  int p0, rows;        // position of query 0, query rows of the sequence (q_len * group)
  int g, f;
  int qt0, qt1;        // query tiles of this unit that see any of its keys
  long long row0;      // first prepared row of (KV head, sequence)
};

// The units of this CTA, in order.  QS = 1 (one query tile to a sequence, one split): CTA c takes KV head c % hkv
// and the (c / hkv)-th run of its key tiles, so that hkv CTAs read the same cache rows, which lie side by side, at
// about the same time (DRAM sees 384 hkv bytes in a row).  QS = 2: every gridDim-th unit.  Every role has its
// own walk in its loop, so the run's step is kept to a few instructions: the roles' loops together have to fit
// the SM's instruction cache.
template <int QS>
struct Walker {
  long long u, left;
  int b, kt, g, f, nq;
  long long lo, hi;  // QS = 2: units of sequence b
  Seq s;
  __device__ __forceinline__ explicit Walker(const Params& P) {
    const long long total = P.units[P.num_seqs];
    if (QS == 1) {  // the grid is a multiple of hkv
      const int runs = static_cast<int>(gridDim.x) / P.hkv, run = static_cast<int>(blockIdx.x) / P.hkv;
      const long long tiles = total / P.hkv;
      u = tiles * run / runs;
      left = tiles * (run + 1) / runs - u;
      u *= P.hkv;
    } else {
      u = blockIdx.x;
      left = u < total ? (total - u + gridDim.x - 1) / gridDim.x : 0;
    }
    b = kt = g = f = nq = 0;
    lo = hi = 0;
    if (left == 0) return;
    int a = 0, z = P.num_seqs;  // the sequence of the first unit
    while (z - a > 1) {
      const int m = (a + z) / 2;
      if (P.units[m] <= u) a = m;
      else z = m;
    }
    b = a;
    if (QS == 1) {
      load_seq(P, b, s);
      kt = static_cast<int>((u - P.units[b]) / P.hkv);
      g = static_cast<int>(blockIdx.x) % P.hkv;
    } else {
      --b;  // entered by the first step
    }
  }
  __device__ __forceinline__ bool next(const Params& P, Unit& w) {
    if (left == 0) return false;
    --left;
    if (QS == 1) {
      while (kt == s.tiles) {  // the next sequence that has tiles
        load_seq(P, ++b, s);
        kt = 0;
      }
    } else {
      while (u >= hi) {
        ++b;
        lo = P.units[b];
        hi = P.units[b + 1];
        load_seq(P, b, s);
        nq = (s.q_len * P.group + P.ntile - 1) / P.ntile;
      }
      const int r = static_cast<int>(u - lo), r2 = r / s.tiles;
      kt = r - r2 * s.tiles;
      g = r2 / P.splits;
      f = r2 - g * P.splits;
      u += gridDim.x;
    }
    w.f = f;
    w.g = g;
    w.kv_beg = s.kv_beg;
    w.kv_len = s.kv_len;
    w.k0 = s.lo + kt * kTile;
    w.nk = min(kTile, s.kv_len - w.k0);
    w.p0 = s.kv_len - s.q_len;
    w.rows = s.q_len * P.group;
    w.row0 = (static_cast<long long>(g) * P.total_q + s.q_beg) * P.group;
    w.qt0 = 0;
    w.qt1 = 1;
    if (QS == 1) {
      ++kt;
    } else {
      w.qt0 = static_cast<int>(static_cast<long long>(nq) * f / P.splits);
      w.qt1 = static_cast<int>(static_cast<long long>(nq) * (f + 1) / P.splits);
      if (w.k0 > w.p0)  // causal: rows from the query at the tile's first key on
        w.qt0 = max(w.qt0, static_cast<int>(static_cast<long long>(w.k0 - w.p0) * P.group / P.ntile));
      if (P.window >= 0) {  // rows up to the last query whose window reaches the tile's last key
        const long long end = (static_cast<long long>(w.k0) + w.nk + P.window - w.p0) * P.group;
        w.qt1 = static_cast<int>(min(static_cast<long long>(w.qt1), (end + P.ntile - 1) / P.ntile));
      }
    }
    return true;
  }
  // The next unit that has query tiles.
  __device__ __forceinline__ bool next_busy(const Params& P, Unit& w) {
    while (next(P, w))
      if (QS == 1 || w.qt1 > w.qt0) return true;
    return false;
  }
};

// Bounded wait; gives up once another role has aborted.
__device__ __forceinline__ bool wait(Ctrl* C, uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait_sleep(bar, parity, kWaitSliceNs)) return true;
    if (*reinterpret_cast<volatile int*>(&C->abort)) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      *reinterpret_cast<volatile int*>(&C->abort) = 1;
      atomicOr(&g_mimo_error, kErrTimeout);
      return false;
    }
  }
}

// Warp wv gathers rows 32 wv .. 32 wv + 31 of each tile, lane l holding the cache row of the l-th (-1: none),
// loaded two units ahead of its copies (its latency is about a unit's whole time).  A loop over the rows, four
// at a time with eight lanes to a row, keeps the code short.
template <int KS, int QS>
__device__ __forceinline__ void role_fetch(uint8_t* smem, Ctrl* C, const Params& P, int lt) {
  const int lane = lt & 31, row0 = lt & ~31, l8 = lane & 7, r4 = lane >> 3;
  const size_t stride = static_cast<size_t>(P.hkv) * kHeadDimQK;
  Walker<QS> walk(P);
  Unit w;
  bool bad = false, more = true;
  int row[3], g[3], n[3];  // of the unit to copy, and the next two
  auto load = [&](int i) {
    g[i] = -1;
    if (more) more = walk.next_busy(P, w);
    if (!more) return;
    g[i] = w.g;
    n[i] = w.nk - row0;
    row[i] = lane < n[i] ? __ldg(P.kv_indices + w.kv_beg + w.k0 + row0 + lane) : -1;
  };
  uint32_t c = 0;
  auto copy = [&](int i) -> bool {  // false at the end, or when the wait gave up
    if (g[i] < 0) return false;
    const uint32_t st = c % KS;
    const bool ok = c < KS || wait(C, &C->k_empty[st], (c / KS - 1) & 1, P.wait_limit_ns);
    if (!__all_sync(0xffffffffu, ok)) return false;
    const uint16_t* from = P.k_cache + g[i] * kHeadDimQK + 8 * l8;
    const uint32_t dst = smem_u32(smem + st * kStage) + static_cast<uint32_t>(row0 + r4) * 128u;
#pragma unroll 4
    for (int p = 0; p < 8; ++p) {
      const int k = __shfl_sync(0xffffffffu, row[i], 4 * p + r4);
      const bool in = static_cast<uint32_t>(k) < static_cast<uint32_t>(P.cache_rows);
      bad |= !in && 4 * p + r4 < n[i];  // an index outside the cache: zeros, reported
      const uint16_t* src = from + static_cast<size_t>(in ? k : 0) * stride;
      const uint32_t nb = in ? 16u : 0u, at = dst + 512u * p + ((l8 ^ ((4 * p + r4) & 7)) << 4);
#pragma unroll
      for (int u = 0; u < 3; ++u) cp_async_16(at + u * kUnit, src + 64 * u, nb);
    }
    cp_async_mbar_arrive_noinc(&C->k_landed[st]);
    ++c;
    load(i);
    return true;
  };
  load(0);
  load(1);
  load(2);
#pragma unroll 1
  while (true) {  // the three sets by turns, so that none has to be moved before it has come
    if (!copy(0) || !copy(1) || !copy(2)) break;  // the same for every lane
  }
  cp_async_commit();
  cp_async_wait<0>();  // nothing of ours stays in flight, on every path
  if (bad) atomicOr(&g_mimo_error, kErrSeqlens);
}

// Cos / sin of every frequency (lane) at each tile's first key, one tile ahead of the rotation.
template <int QS>
__device__ __forceinline__ void role_angles(Ctrl* C, const Params& P, int lane) {
  const double theta = P.theta[lane];
  Walker<QS> walk(P);
  Unit w;
#pragma unroll 1
  for (uint32_t c = 0; walk.next_busy(P, w); ++c) {
    const uint32_t buf = c & 1;
    const float2 a = angle(w.k0, theta);
    if (c >= 2 && !wait(C, &C->a_empty[buf], ((c >> 1) - 1) & 1, P.wait_limit_ns)) return;
    C->k_cos[buf][lane] = a.x;
    C->k_sin[buf][lane] = a.y;
    mbar_arrive(&C->a_full[buf]);
  }
}

// Thread: key r = t % 128 of the tile (the TMEM lane), h = t / 128: chunk pairs 2h and 2h + 1 (dims 16h ..
// 16h + 15 and their partners) and pass dims 64 + 64h .. 127 + 64h.  oc, os: cos / sin of the key's offset from
// the tile's first key for those dims, two frequencies to a pair.
template <int KS, int QS>
__device__ __forceinline__ void role_rotate(uint8_t* smem, Ctrl* C, uint32_t tmem, const Params& P, int t,
                                            const float2 (&oc)[8], const float2 (&os)[8]) {
  const int r = t & 127, h = t >> 7;
  const uint32_t lane_base = static_cast<uint32_t>(r & ~31) << 16;
  Walker<QS> walk(P);
  Unit w;
  __half2 amax = __floats2half2_rn(0.f, 0.f);
#pragma unroll 1
  for (uint32_t c = 0; walk.next_busy(P, w); ++c) {
    const uint32_t st = c % KS, buf = c & 1;
    bool ok = wait(C, &C->a_full[buf], (c >> 1) & 1, P.wait_limit_ns);
    ok = ok && wait(C, &C->k_landed[st], (c / KS) & 1, P.wait_limit_ns);
    // the products with the tile before last are done: with one query tile to a unit its score tile says so
    if (ok && c >= 2) ok = wait(C, QS == 1 ? &C->s_full[buf] : &C->k_free[buf], ((c >> 1) - 1) & 1, P.wait_limit_ns);
    if (!__all_sync(0xffffffffu, ok)) break;
    tc_fence_after_sync();
    const uint8_t* row = smem + st * kStage + r * 128;
    const uint32_t dst = tmem + lane_base + kColK + 128u * buf;
    {
      uint32_t pass[32];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + (1 + h) * kUnit + ((k ^ (r & 7)) << 4));
        pass[4 * k] = v.x, pass[4 * k + 1] = v.y, pass[4 * k + 2] = v.z, pass[4 * k + 3] = v.w;
      }
      tmem_st32(dst + 64 + 32 * h, pass);
    }
    uint32_t ah[8], al[8], bh[8], bl[8];  // dims 16h .. 16h + 15 and partners, two to a word
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int p = 2 * h + q;
      const uint4 a = *reinterpret_cast<const uint4*>(row + ((p ^ (r & 7)) << 4));
      const uint4 b = *reinterpret_cast<const uint4*>(row + (((p + 4) ^ (r & 7)) << 4));
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 bc = *reinterpret_cast<const float2*>(&C->k_cos[buf][8 * p + 2 * e]);
        const float2 bs = *reinterpret_cast<const float2*>(&C->k_sin[buf][8 * p + 2 * e]);
        const float2 kc = oc[4 * q + e], ks = os[4 * q + e];
        const float2 cs = ffma2(bc, kc, fmul2(make_float2(-bs.x, -bs.y), ks));
        const float2 sn = ffma2(bs, kc, fmul2(bc, ks));
        const float2 x = unpack_bf16x2(aw[e]), y = unpack_bf16x2(bw[e]);
        const float2 ny = unpack_bf16x2(bw[e] ^ 0x80008000u);
        const float2 u = ffma2(x, cs, fmul2(ny, sn)), v = ffma2(y, cs, fmul2(x, sn));
        const __half2 uh = __floats2half2_rn(u.x, u.y), vh = __floats2half2_rn(v.x, v.y);
        amax = __hmax2(amax, __hmax2(__habs2(uh), __habs2(vh)));
        const float2 m1 = make_float2(-1.f, -1.f);
        const float2 up = make_float2(1 << kLoBits, 1 << kLoBits);
        const float2 ul = fmul2(ffma2(__half22float2(uh), m1, u), up), vl = fmul2(ffma2(__half22float2(vh), m1, v), up);
        const __half2 uln = __floats2half2_rn(ul.x, ul.y), vln = __floats2half2_rn(vl.x, vl.y);
        ah[4 * q + e] = *reinterpret_cast<const uint32_t*>(&uh);
        al[4 * q + e] = *reinterpret_cast<const uint32_t*>(&uln);
        bh[4 * q + e] = *reinterpret_cast<const uint32_t*>(&vh);
        bl[4 * q + e] = *reinterpret_cast<const uint32_t*>(&vln);
      }
    }
    tmem_st8(dst + 8 * h, ah);
    tmem_st8(dst + 16 + 8 * h, bh);
    tmem_st8(dst + 32 + 8 * h, al);
    tmem_st8(dst + 48 + 8 * h, bl);
    tmem_st_wait();
    mbar_arrive(&C->k_empty[st]);  // the stage is read
    mbar_arrive(&C->a_empty[buf]);
    tc_fence_before_sync();
    mbar_arrive(&C->k_full[buf]);
  }
  const float2 top = __half22float2(amax);
  if (fmaxf(top.x, top.y) > 65504.f) atomicOr(&g_mimo_error, kErrRange);  // infinite: rounded past FP16's range
}

template <int KS, int QS>
__device__ __forceinline__ void role_load_q(uint8_t* smem, Ctrl* C, const Params& P, const CUtensorMap* tq, int lane) {
  const uint32_t unit = static_cast<uint32_t>(P.ntile) * 128u;  // 64 dims of the tile's rows: a multiple of 2 KB
  uint8_t* ring = smem + KS * kStage;
  Walker<QS> walk(P);
  Unit w;
  long long have = -1;
  uint32_t loads = 0;
  bool ok = true;
#pragma unroll 1
  while (ok && walk.next_busy(P, w)) {
#pragma unroll 1
    for (int qt = w.qt0; qt < w.qt1; ++qt) {
      const long long row = w.row0 + static_cast<long long>(qt) * P.ntile;
      if (QS == 1 && row == have) continue;
      have = row;
      const uint32_t st = loads % QS;
      ok = loads < QS || wait(C, &C->q_empty[st], (loads / QS - 1) & 1, P.wait_limit_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      // the products that this stage waited for are QS tiles back, and the sums two behind those: the slot's
      // last reader is done
      for (int c = lane; c < P.ntile; c += 32)
        C->lse2[loads % kLseSlots][c] = qt * P.ntile + c < w.rows ? __ldg(P.lse2 + row + c) : 0.f;
      if (lane == 0) {
        mbar_arrive_expect_tx(&C->q_full[st], 4 * unit);
        for (int u = 0; u < 4; ++u)
          tma_load_2d(ring + (4 * st + u) * unit, tq, &C->q_full[st], 64 * u, static_cast<int32_t>(row));
      }
      mbar_arrive(&C->lse_full[loads % kLseSlots]);
      ++loads;
    }
  }
  // nothing of ours stays in flight, on every path
  for (uint32_t i = loads > QS ? loads - QS : 0; i < loads; ++i)
    wait(C, &C->q_full[i % QS], (i / QS) & 1, P.wait_limit_ns);
}

// S = K Q^T of one tile: Q hi with K lo and Q lo with K hi, then, with those times 2^-11, Q hi with K hi, pass with
// pass.  k: K's TMEM columns (hi 0, lo 32, pass 64 and 96); q: Q's descriptor (hi, lo, pass, pass, qu apart).  All
// 20 in a row: the issue of an MMA from a rolled loop takes about 250 cycles, in a row about 90.
__device__ __forceinline__ void issue_tile(uint32_t acc, uint32_t k, uint32_t q, uint32_t qu, uint32_t idesc_f16,
                                           uint32_t idesc_bf16) {
#pragma unroll
  for (int s = 0; s < 4; ++s) mma_ts_lo(acc, k + 32 + 8 * s, q + 2 * s, idesc_f16, s > 0 ? 1u : 0u);
#pragma unroll
  for (int s = 0; s < 4; ++s) mma_ts_lo(acc, k + 8 * s, q + qu + 2 * s, idesc_f16, 1u);
  mma_ts_lo_scaled<kLoBits>(acc, k, q, idesc_f16);
#pragma unroll
  for (int s = 1; s < 4; ++s) mma_ts_lo(acc, k + 8 * s, q + 2 * s, idesc_f16, 1u);
  q += 2 * qu;
#pragma unroll
  for (int s = 0; s < 4; ++s) mma_ts_lo(acc, k + 64 + 8 * s, q + 2 * s, idesc_bf16, 1u);
  q += qu;
#pragma unroll
  for (int s = 0; s < 4; ++s) mma_ts_lo(acc, k + 96 + 8 * s, q + 2 * s, idesc_bf16, 1u);
}

// The whole warp walks the units and waits; one lane issues.  What the MMAs' operands are formed from is made
// uniform over the warp first, so that they are formed in the uniform registers that the MMAs read.
template <int KS, int QS>
__device__ __forceinline__ void role_mma(uint8_t* smem, Ctrl* C, uint32_t tmem, const Params& P) {
  const uint32_t idesc_f16 = make_idesc_f32acc(0, 0, 128, P.ntile), idesc_bf16 = make_idesc_f32acc(1, 0, 128, P.ntile);
  const uint32_t unit = static_cast<uint32_t>(P.ntile) * 128u;
  const uint32_t q0 = sdesc_lo(smem_u32(smem + KS * kStage), 16), qu = unit >> 4;
  const uint32_t t0 = __shfl_sync(0xffffffffu, tmem, 0);
  Walker<QS> walk(P);
  Unit w;
  long long have = -1;
  uint32_t loads = 0, d = 0;
#pragma unroll 1
  for (uint32_t c = 0; walk.next_busy(P, w); ++c) {
    const uint32_t buf = c & 1;
    if (!__all_sync(0xffffffffu, wait(C, &C->k_full[buf], (c >> 1) & 1, P.wait_limit_ns))) return;
#pragma unroll 1
    for (int qt = w.qt0; qt < w.qt1; ++qt, ++d) {
      const long long row = w.row0 + static_cast<long long>(qt) * P.ntile;
      bool ok = true;
      if (QS > 1 || row != have) {
        // a commit takes about 50 cycles of the tensor pipe: one stage is handed back only where Q changes
        if (QS == 1 && loads > 0 && elect_one()) tc_commit(&C->q_empty[0]);
        have = row;
        ok = wait(C, &C->q_full[loads % QS], (loads / QS) & 1, P.wait_limit_ns);
        ++loads;
      }
      if (ok && d >= 2) ok = wait(C, &C->s_empty[d & 1], ((d >> 1) - 1) & 1, P.wait_limit_ns);
      if (!__all_sync(0xffffffffu, ok)) return;
      tc_fence_after_sync();
      const uint32_t st = __shfl_sync(0xffffffffu, (loads - 1) % QS, 0);
      const uint32_t acc = t0 + __shfl_sync(0xffffffffu, 128u * (d & 1), 0);
      const uint32_t k = t0 + __shfl_sync(0xffffffffu, kColK + 128u * buf, 0);
      if (elect_one()) {
        issue_tile(acc, k, q0 + 4 * st * qu, qu, idesc_f16, idesc_bf16);
        tc_commit(&C->s_full[d & 1]);
        if (QS > 1) tc_commit(&C->q_empty[st]);
        if (QS > 1 && qt + 1 == w.qt1) tc_commit(&C->k_free[buf]);
      }
      __syncwarp();
    }
  }
}

// Adds 2^(s sl2 - lse2) over N score columns; masked: of those in [lo, hi) only.  (Half of the exponentials as
// polynomials on the FMA pipe, so that ex2's 16 a cycle are not what two groups at work share, was slower: 96
// against 90 us for a 300-token chunk.)
template <int N, bool kMasked>
__device__ __forceinline__ void add_columns(const uint32_t (&s)[N], const float* lse2, float sl2, int lo, int hi,
                                            float2& a0, float2& a1) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 l = *reinterpret_cast<const float4*>(lse2 + i);
    const float2 k = make_float2(sl2, sl2);
    const float2 e0 = ffma2(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), k, make_float2(-l.x, -l.y));
    const float2 e1 =
        ffma2(make_float2(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), k, make_float2(-l.z, -l.w));
    float2 p0 = make_float2(ex2_approx(e0.x), ex2_approx(e0.y)), p1 = make_float2(ex2_approx(e1.x), ex2_approx(e1.y));
    if (kMasked) {
      p0.x = i >= lo && i < hi ? p0.x : 0.f;
      p0.y = i + 1 >= lo && i + 1 < hi ? p0.y : 0.f;
      p1.x = i + 2 >= lo && i + 2 < hi ? p1.x : 0.f;
      p1.y = i + 3 >= lo && i + 3 < hi ? p1.y : 0.f;
    }
    a0 = fadd2(a0, p0);
    a1 = fadd2(a1, p1);
  }
}

// Group grp takes the score tiles of its parity.  With one tile to a unit (QS = 1) it writes the whole sums of
// its units; else each group writes its own partial row of every unit.
template <int QS>
__device__ __forceinline__ void role_sum(Ctrl* C, uint32_t tmem, const Params& P, int r, uint32_t grp) {
  const uint32_t acc = tmem + (static_cast<uint32_t>(r & ~31) << 16) + 128u * grp;
  const float sl2 = P.scale_log2;
  Walker<QS> walk(P);
  Unit w;
  long long have = -1;
  uint32_t loads = 0, d = 0;
#pragma unroll 1
  while (walk.next(P, w)) {
    const int key = w.k0 + r;
    // all queries of a tile see all keys of the unit from row see_all on, and up to row win_all
    const long long see_all = (static_cast<long long>(w.k0) + w.nk - 1 - w.p0) * P.group;
    const long long win_all = (static_cast<long long>(w.k0) + P.window + 1 - w.p0) * P.group;
    float2 a0 = make_float2(0.f, 0.f), a1 = a0;
    bool mine = false;
#pragma unroll 1
    for (int qt = w.qt0; qt < w.qt1; ++qt, ++d) {
      const int base = qt * P.ntile;
      if (QS > 1 || w.row0 + base != have) {
        have = w.row0 + base;
        ++loads;
      }
      if ((d & 1) != grp) continue;
      mine = true;
      const int cols = min(P.ntile, w.rows - base);  // query rows of the tile
      const bool all = base >= see_all && (P.window < 0 || base + cols <= win_all);
      int c_lo = 0, c_hi = cols;
      if (!all) {  // columns (query rows) that see this key: a run
        const long long seen = (static_cast<long long>(key) - w.p0) * P.group - base;
        c_lo = static_cast<int>(max(0LL, min(seen, 128LL)));
        if (P.window >= 0) {
          const long long end = (static_cast<long long>(key) + P.window + 1 - w.p0) * P.group - base;
          c_hi = static_cast<int>(max(0LL, min(static_cast<long long>(cols), end)));
        }
      }
      // this load's lse; the loader is at most two loads ahead (its rows wait for the products of the loads
      // before, and those for the score tiles), so the slot still holds it
      const uint32_t slot = (loads - 1) % kLseSlots;
      bool ok = wait(C, &C->lse_full[slot], ((loads - 1) / kLseSlots) & 1, P.wait_limit_ns);
      ok = ok && wait(C, &C->s_full[grp], (d >> 1) & 1, P.wait_limit_ns);
      if (!__all_sync(0xffffffffu, ok)) return;
      tc_fence_after_sync();
      const float* lse2 = C->lse2[slot];
      int c0 = 0;
#pragma unroll 1
      for (; c0 + 32 <= cols; c0 += 32) {
        uint32_t s[32];
        tmem_ld32(acc + c0, s);
        tmem_ld_wait(s);
        if (all) add_columns<32, false>(s, lse2 + c0, sl2, 0, 0, a0, a1);
        else add_columns<32, true>(s, lse2 + c0, sl2, c_lo - c0, c_hi - c0, a0, a1);
      }
#pragma unroll 1
      for (; c0 < cols; c0 += 16) {  // ntile is a multiple of 16
        uint32_t s[16];
        tmem_ld16(acc + c0, s);
        tmem_ld16_wait(s);
        add_columns<16, true>(s, lse2 + c0, sl2, c_lo - c0, c_hi - c0, a0, a1);
      }
      tc_fence_before_sync();
      mbar_arrive(&C->s_empty[grp]);
    }
    if (r < w.nk && (QS > 1 || mine)) {
      const int part = QS > 1 ? 2 * w.f + static_cast<int>(grp) : 0;
      P.partial[(static_cast<size_t>(part) * P.hkv + w.g) * P.total_kv + w.kv_beg + key] =
          (a0.x + a0.y) + (a1.x + a1.y);
    }
  }
}

template <int KS, int QS>
__global__ void __launch_bounds__(kThreads, 1) kw_main_kernel(const __grid_constant__ CUtensorMap tq,
                                                              const __grid_constant__ Params P) {
  static_assert(KS <= kMaxKS, "stages");  // what Q takes goes by ntile: the launch keeps to kCtrlOff
  extern __shared__ __align__(1024) uint8_t smem[];
  Ctrl* C = reinterpret_cast<Ctrl*>(smem + kCtrlOff);
  const int tid = threadIdx.x, warp = tid >> 5;
  int skip = 0;
  if (tid == 0) {
    skip = (*reinterpret_cast<volatile unsigned int*>(&g_mimo_error) & kErrTimeout) != 0;
    if (smem_u32(smem) & 1023u) skip = 1;  // swizzled operands need a 1 KB aligned base
  }
  if (__syncthreads_or(skip)) {
    if (tid == 0) P.units[P.num_seqs + 1] = 1;
    return;
  }
  if (tid == 0) {
    for (int s = 0; s < KS; ++s) {
      mbar_init(&C->k_landed[s], 128);  // one cp.async arrival per fetcher thread
      mbar_init(&C->k_empty[s], kRotThreads);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&C->q_full[s], 1);
      mbar_init(&C->q_empty[s], 1);
      mbar_init(&C->k_full[s], kRotThreads);
      mbar_init(&C->k_free[s], 1);
      mbar_init(&C->a_full[s], 32);
      mbar_init(&C->a_empty[s], kRotThreads);
      mbar_init(&C->s_full[s], 1);
      mbar_init(&C->s_empty[s], 128);
    }
    for (int s = 0; s < kLseSlots; ++s) mbar_init(&C->lse_full[s], 32);
    C->abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(&C->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  // cos / sin of every offset within a tile, by everyone into the rings' memory; the rotation's threads keep theirs
  float2* table = reinterpret_cast<float2*>(smem);  // [offset][frequency]
#pragma unroll 1
  for (int i = tid; i < kTile * (kRopeDims / 2); i += kThreads)
    table[i] = angle(i / (kRopeDims / 2), P.theta[i % (kRopeDims / 2)]);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = C->tmem_base;
  float2 oc[8], os[8];
  if (warp >= 12 && warp < 20) {
    const int t = tid - 384;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(&table[(t & 127) * (kRopeDims / 2) + 16 * (t >> 7) + 2 * i]);
      oc[i] = make_float2(v.x, v.z);
      os[i] = make_float2(v.y, v.w);
    }
  }
  fence_proxy_async_smem();  // the Q tiles come by TMA into the same memory
  __syncthreads();
  if (warp < 4) {
    setmaxnreg_dec<kRegsSmall>();
    if (warp == 0) role_mma<KS, QS>(smem, C, tmem, P);
    else if (warp == 1) role_load_q<KS, QS>(smem, C, P, &tq, tid & 31);
    else if (warp == 2) role_angles<QS>(C, P, tid & 31);
  } else if (warp < 12) {
    role_sum<QS>(C, tmem, P, tid & 127, warp >= 8 ? 1u : 0u);
  } else if (warp < 20) {
    setmaxnreg_inc<kRegsRotate>();
    role_rotate<KS, QS>(smem, C, tmem, P, tid - 384, oc, os);
  } else {
    setmaxnreg_dec<kRegsFetch>();
    role_fetch<KS, QS>(smem, C, P, tid - 640);
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (tid == 0 && *reinterpret_cast<volatile int*>(&C->abort)) P.units[P.num_seqs + 1] = 1;
  if (warp == 0) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------- launch 3
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) kw_join_kernel(const __grid_constant__ Params P) {
  const long long i = static_cast<long long>(blockIdx.x) * kJoinThreads + threadIdx.x;
  const int lane = threadIdx.x & 31;
  const bool in = i < P.total_kv;
  const int rows = P.parts * P.hkv;
  // the partial rows are read before the entry's sequence is known: where no query sees the key they were not
  // written, and what is read does not count
  float v = 0.f;
  if (in) {
#pragma unroll 8
    for (int k = 0; k < rows; ++k) v += P.partial[static_cast<size_t>(k) * P.total_kv + i];
  }
  const float p = in && P.prev != nullptr ? P.prev[i] : 0.f;
  // the sequence of the warp's first entry, and from there on to this entry's
  const long long i0 = i - lane;
  // where launch 2 gave up (a bounded wait ran out, in it or before it) partial rows are missing: out, which may be
  // prev, stays as it was
  if (i0 >= P.total_kv || P.units[P.num_seqs + 1] != 0) return;
  int b = find_seq(P.kv_indptr, P.num_seqs, static_cast<int>(i0), lane);
  if (!in) return;
  while (b + 1 < P.num_seqs && __ldg(P.kv_indptr + b + 1) <= i) ++b;
  Seq s;
  if (!load_seq(P, b, s) || i < s.kv_beg || i >= s.kv_beg + s.kv_len) return;  // left as it was
  P.out[i] = i - s.kv_beg >= s.lo ? p + v : p;
}

}  // namespace kw
}  // namespace mimo
