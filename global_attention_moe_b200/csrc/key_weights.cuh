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
// than the attention's: the rotated dims of Q and K are each split into an FP16 value and the FP16
// rounding of what is left (22 bits), and three products hi hi + hi lo + lo hi take the place of one; the
// pass-through dims are exact in BF16.  Rotation angles come from FP64-reduced positions.
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
//   3. kw_join_kernel: adds the partial rows in a fixed order, and prev.
//
// Warp roles of the main kernel (14 warps):
//   warps 0-3   sums (thread = key = TMEM lane)
//   warps 4-7   K fetcher: gathers the tile's rows by index with cp.async into the 128-byte-swizzled layout
//   warps 8-11  K rotation: BF16 -> FP16 hi in place, lo beside it (angle addition from the tile's start)
//   warp 12     TMEM owner; lane 0 issues the MMAs
//   warp 13     Q loader: TMA boxes of the prepared rows, and their lse
// Units are walked in order by every role.  With one query tile per sequence (decode steps) a CTA takes a
// contiguous run of units, so Q stays in shared memory while the keys of a (sequence, KV head) stream
// through two K stages; with more (chunked prefill) the key tile stays while the query tiles stream
// through two Q stages.
#pragma once

#include "attn_decode.cuh"
#include "cp_async.cuh"

namespace mimo {
namespace kw {

constexpr int kThreads = 448;
constexpr int kTile = 128;                 // keys per unit
constexpr uint32_t kUnit = 16384;          // 128 rows x 64 dims x 2 B
constexpr uint32_t kStage = 4 * kUnit;     // K: hi, pass, pass, lo; Q: hi, lo, pass, pass
constexpr uint32_t kCtrlOff = 3 * kStage;  // two K stages and one Q stage, or one and two
constexpr int kLseSlots = 4;
constexpr uint32_t kTmemCols = 256;        // two score tiles of at most 128 columns
constexpr uint32_t kRotBar = 1;            // named barrier of the rotation warps
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
  long long* units;           // workspace: [num_seqs + 1], running count of units
  float* partial;             // workspace: [splits * hkv, total_kv]
  int32_t num_seqs, total_q, total_kv, cache_rows, max_q_len, max_kv_len;
  int32_t hq, hkv, group;
  int32_t window;             // < 0: global causal layer
  int32_t splits;             // parts of the query tiles
  int32_t ntile;              // query rows per tile (MMA N): multiple of 16, at most 128
  int32_t contiguous;         // a CTA's units: a run (1) or every gridDim-th (0)
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

// x as an FP16 value and the FP16 rounding of the rest.
__device__ __forceinline__ void split16(float x, __half& hi, __half& lo) {
  hi = __float2half_rn(x);
  lo = __float2half_rn(x - __half2float(hi));
}

// ---------------------------------------------------------------- launch 1
// Blocks 0 .. gridDim - 2: one warp per (token, 8 query heads), lane = RoPE pair.  Last block: the running
// count of units.
constexpr int kPrepThreads = 256;
constexpr int kPrepHeads = 8;
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
    if (threadIdx.x == 0) P.units[0] = 0;
    if (bad) atomicOr(&g_mimo_error, kErrSeqlens);
    return;
  }
  const int hblocks = (P.hq + kPrepHeads - 1) / kPrepHeads;
  const long long item = static_cast<long long>(blockIdx.x) * (kPrepThreads / 32) + warp;
  const int t = static_cast<int>(item / hblocks);
  const int h0 = static_cast<int>(item % hblocks) * kPrepHeads;
  if (t >= P.total_q) return;
  // the token's sequence: the last one that starts at or before it
  int a = 0, z = P.num_seqs;
  while (z - a > 1) {
    const int m = (a + z) / 2;
    if (__ldg(P.cu_q + m) <= t) a = m;
    else z = m;
  }
  Seq s;
  const bool ok = load_seq(P, a, s) && t >= s.q_beg && t < s.q_beg + s.q_len;
  if (!ok) return;  // rows of no sequence are never read as queries
  const float2 cs = angle(s.kv_len - s.q_len + (t - s.q_beg), P.theta[lane]);
  float amax = 0.f;
#pragma unroll 4
  for (int h = h0; h < min(h0 + kPrepHeads, P.hq); ++h) {
    const uint16_t* src = P.q + (static_cast<size_t>(t) * P.hq + h) * kHeadDimQK;
    const size_t row = (static_cast<size_t>(h / P.group) * P.total_q + t) * P.group + h % P.group;
    uint16_t* dst = P.qs + row * 256;
    const float x = __uint_as_float(static_cast<uint32_t>(__ldg(src + lane)) << 16);
    const float y = __uint_as_float(static_cast<uint32_t>(__ldg(src + lane + 32)) << 16);
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
    reinterpret_cast<uint2*>(dst + 128)[lane] = __ldg(reinterpret_cast<const uint2*>(src + 64) + lane);
    if (lane == 0) P.lse2[row] = __ldg(P.lse + static_cast<size_t>(h) * P.total_q + t) * dec::kLog2e;
  }
  if (amax > 65504.f) atomicOr(&g_mimo_error, kErrRange);
}

// ---------------------------------------------------------------- launch 2
struct Ctrl {
  uint64_t k_landed[2], k_full[2], k_empty[2];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], s_empty[2];
  uint64_t lse_full[kLseSlots];
  uint32_t tmem_base;
  int abort;
  float2 k_base[2][kRopeDims / 2];  // cos / sin at the tile's first key, by unit parity
  double theta[kRopeDims / 2];
  float lse2[kLseSlots][kTile];     // of the Q loads, in turn
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

// The units of this CTA, in order.
struct Walker {
  long long u, step, left;
  int b = -1;
  long long lo = 0, hi = 0;  // units of sequence b
  Seq s;
  __device__ __forceinline__ explicit Walker(const Params& P) {
    const long long total = P.units[P.num_seqs];
    if (P.contiguous) {
      u = total * blockIdx.x / gridDim.x;
      left = total * (blockIdx.x + 1) / gridDim.x - u;
      step = 1;
    } else {
      u = blockIdx.x;
      step = gridDim.x;
      left = u < total ? (total - u + step - 1) / step : 0;
    }
    if (left > 0) {  // the sequence of the first unit
      int a = 0, z = P.num_seqs;
      while (z - a > 1) {
        const int m = (a + z) / 2;
        if (P.units[m] <= u) a = m;
        else z = m;
      }
      b = a - 1;
    }
  }
  __device__ __forceinline__ bool next(const Params& P, Unit& w) {
    if (left == 0) return false;
    while (u >= hi) {
      ++b;
      lo = P.units[b];
      hi = P.units[b + 1];
      load_seq(P, b, s);
    }
    const int r = static_cast<int>(u - lo);
    const int kt = r % s.tiles, r2 = r / s.tiles;
    w.f = r2 % P.splits;
    w.g = r2 / P.splits;
    w.kv_beg = s.kv_beg;
    w.kv_len = s.kv_len;
    w.k0 = s.lo + kt * kTile;
    w.nk = min(kTile, s.kv_len - w.k0);
    w.p0 = s.kv_len - s.q_len;
    w.rows = s.q_len * P.group;
    const int nq = (w.rows + P.ntile - 1) / P.ntile;
    w.qt0 = static_cast<int>(static_cast<long long>(nq) * w.f / P.splits);
    w.qt1 = static_cast<int>(static_cast<long long>(nq) * (w.f + 1) / P.splits);
    if (w.k0 > w.p0)  // causal: rows from the query at the tile's first key on
      w.qt0 = max(w.qt0, static_cast<int>(static_cast<long long>(w.k0 - w.p0) * P.group / P.ntile));
    if (P.window >= 0) {  // rows up to the last query whose window reaches the tile's last key
      const long long end = (static_cast<long long>(w.k0) + w.nk + P.window - w.p0) * P.group;
      w.qt1 = static_cast<int>(min(static_cast<long long>(w.qt1), (end + P.ntile - 1) / P.ntile));
    }
    w.row0 = (static_cast<long long>(w.g) * P.total_q + s.q_beg) * P.group;
    u += step;
    --left;
    return true;
  }
  // The next unit that has query tiles.
  __device__ __forceinline__ bool next_busy(const Params& P, Unit& w) {
    while (next(P, w))
      if (w.qt1 > w.qt0) return true;
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

__device__ __forceinline__ void load_idx(const Params& P, const Unit& w, int rsub, int (&idx)[8]) {
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int j = 16 * p + rsub;
    idx[p] = j < w.nk ? __ldg(P.kv_indices + w.kv_beg + w.k0 + j) : -1;
  }
}

template <int KS>
__device__ __forceinline__ void role_fetch(uint8_t* smem, Ctrl* C, const Params& P, int lt) {
  const int l8 = lt & 7, rsub = lt >> 3;
  Walker walk(P);
  Unit w;
  bool bad = false;
  bool more = walk.next_busy(P, w);
  int idx[8];
  if (more) load_idx(P, w, rsub, idx);
#pragma unroll 1
  for (uint32_t c = 0; more; ++c) {
    const uint32_t st = c % KS;
    if (c >= KS && !wait(C, &C->k_empty[st], (c / KS - 1) & 1, P.wait_limit_ns)) break;
    const uint32_t dst = smem_u32(smem + st * kStage);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const int j = 16 * p + rsub;
      const bool in = idx[p] >= 0 && idx[p] < P.cache_rows;
      bad |= j < w.nk && !in;  // an index outside the cache: zeros, reported
      const uint16_t* src = in ? P.k_cache + (static_cast<size_t>(idx[p]) * P.hkv + w.g) * kHeadDimQK : P.k_cache;
      const uint32_t sw = static_cast<uint32_t>(j * 128 + ((l8 ^ (j & 7)) << 4));
#pragma unroll
      for (int u = 0; u < 3; ++u) cp_async_16(dst + u * kUnit + sw, src + 64 * u + 8 * l8, in ? 16u : 0u);
    }
    cp_async_mbar_arrive_noinc(&C->k_landed[st]);
    more = walk.next_busy(P, w);
    if (more) load_idx(P, w, rsub, idx);  // in flight while this thread waits for the next stage
  }
  cp_async_commit();
  cp_async_wait<0>();  // nothing of ours stays in flight, on every path
  if (bad) atomicOr(&g_mimo_error, kErrSeqlens);
}

template <int KS>
__device__ __forceinline__ void role_rotate(uint8_t* smem, Ctrl* C, const Params& P, int r) {
  // cos / sin of this row's offset from the tile's first key
  float2 off[kRopeDims / 2];
#pragma unroll
  for (int i = 0; i < kRopeDims / 2; ++i) off[i] = angle(r, C->theta[i]);
  Walker walk(P);
  Unit w;
  float amax = 0.f;
  bool ok = true;
#pragma unroll 1
  for (uint32_t c = 0; walk.next_busy(P, w); ++c) {
    const uint32_t st = c % KS;
    if (r < kRopeDims / 2) C->k_base[c & 1][r] = angle(w.k0, C->theta[r]);
    if (ok) ok = wait(C, &C->k_landed[st], (c / KS) & 1, P.wait_limit_ns);
    // this tile's base angles written, those of two tiles back read; all leave together
    if (!named_bar_and(kRotBar, 128, ok)) break;
    const float2* base = C->k_base[c & 1];
    uint8_t* hi_row = smem + st * kStage + r * 128;
    uint8_t* lo_row = hi_row + 3 * kUnit;
#pragma unroll
    for (int p = 0; p < 4; ++p) {  // chunk pair (p, p + 4): dims 8p .. 8p + 7 and their partners
      const uint32_t ca = (p ^ (r & 7)) << 4, cb = ((p + 4) ^ (r & 7)) << 4;
      const uint4 a = *reinterpret_cast<const uint4*>(hi_row + ca), b = *reinterpret_cast<const uint4*>(hi_row + cb);
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
      uint32_t ah[4], al[4], bh[4], bl[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float u[2], v[2];
        const float2 x = unpack_bf16x2(aw[e]), y = unpack_bf16x2(bw[e]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 t = base[8 * p + 2 * e + k], o = off[8 * p + 2 * e + k];
          const float cs = t.x * o.x - t.y * o.y, sn = t.y * o.x + t.x * o.y;
          const float xx = k ? x.y : x.x, yy = k ? y.y : y.x;
          u[k] = xx * cs - yy * sn;
          v[k] = yy * cs + xx * sn;
          amax = fmaxf(amax, fmaxf(fabsf(u[k]), fabsf(v[k])));
        }
        const __half2 uh = __floats2half2_rn(u[0], u[1]), vh = __floats2half2_rn(v[0], v[1]);
        const float2 uf = __half22float2(uh), vf = __half22float2(vh);
        const __half2 ul = __floats2half2_rn(u[0] - uf.x, u[1] - uf.y), vl = __floats2half2_rn(v[0] - vf.x, v[1] - vf.y);
        ah[e] = *reinterpret_cast<const uint32_t*>(&uh);
        al[e] = *reinterpret_cast<const uint32_t*>(&ul);
        bh[e] = *reinterpret_cast<const uint32_t*>(&vh);
        bl[e] = *reinterpret_cast<const uint32_t*>(&vl);
      }
      *reinterpret_cast<uint4*>(hi_row + ca) = make_uint4(ah[0], ah[1], ah[2], ah[3]);
      *reinterpret_cast<uint4*>(hi_row + cb) = make_uint4(bh[0], bh[1], bh[2], bh[3]);
      *reinterpret_cast<uint4*>(lo_row + ca) = make_uint4(al[0], al[1], al[2], al[3]);
      *reinterpret_cast<uint4*>(lo_row + cb) = make_uint4(bl[0], bl[1], bl[2], bl[3]);
    }
    fence_proxy_async_smem();  // the fetcher's copies and these writes, before the MMA reads the stage
    mbar_arrive(&C->k_full[st]);
  }
  if (amax > 65504.f) atomicOr(&g_mimo_error, kErrRange);
}

template <int QS>
__device__ __forceinline__ void role_load_q(uint8_t* smem, Ctrl* C, const Params& P, const CUtensorMap* tq, int lane) {
  Walker walk(P);
  Unit w;
  long long have = -1;
  uint32_t loads = 0;
  const uint32_t unit_bytes = static_cast<uint32_t>(P.ntile) * 128u;
  bool ok = true;
#pragma unroll 1
  while (ok && walk.next_busy(P, w)) {
#pragma unroll 1
    for (int qt = w.qt0; qt < w.qt1; ++qt) {
      const long long row = w.row0 + static_cast<long long>(qt) * P.ntile;
      if (row == have) continue;
      have = row;
      const uint32_t st = loads % QS;
      ok = loads < QS || wait(C, &C->q_empty[st], (loads / QS - 1) & 1, P.wait_limit_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      for (int c = lane; c < P.ntile; c += 32)
        C->lse2[loads % kLseSlots][c] = qt * P.ntile + c < w.rows ? __ldg(P.lse2 + row + c) : 0.f;
      uint8_t* dst = smem + (3 - QS + st) * kStage;
      if (lane == 0) {
        mbar_arrive_expect_tx(&C->q_full[st], 4 * unit_bytes);
        for (int u = 0; u < 4; ++u)
          tma_load_2d(dst + u * kUnit, tq, &C->q_full[st], 64 * u, static_cast<int32_t>(row));
      }
      mbar_arrive(&C->lse_full[loads % kLseSlots]);
      ++loads;
    }
  }
  // nothing of ours stays in flight, on every path
  if (loads > 0) wait(C, &C->q_full[(loads - 1) % QS], ((loads - 1) / QS) & 1, P.wait_limit_ns);
  if (QS > 1 && loads > 1) wait(C, &C->q_full[(loads - 2) % QS], ((loads - 2) / QS) & 1, P.wait_limit_ns);
}

template <int KS, int QS>
__device__ __forceinline__ void role_mma(uint8_t* smem, Ctrl* C, uint32_t tmem, const Params& P) {
  const uint32_t idesc_f16 = make_idesc_f32acc(0, 0, 128, P.ntile), idesc_bf16 = make_idesc_f32acc(1, 0, 128, P.ntile);
  constexpr uint32_t kStep = kUnit >> 4;
  Walker walk(P);
  Unit w;
  long long have = -1;
  uint32_t loads = 0, d = 0;
#pragma unroll 1
  for (uint32_t c = 0; walk.next_busy(P, w); ++c) {
    const uint32_t st = c % KS;
    if (!wait(C, &C->k_full[st], (c / KS) & 1, P.wait_limit_ns)) return;
    const uint32_t k_lo = sdesc_lo(smem_u32(smem + st * kStage), 16);
#pragma unroll 1
    for (int qt = w.qt0; qt < w.qt1; ++qt, ++d) {
      const long long row = w.row0 + static_cast<long long>(qt) * P.ntile;
      if (row != have) {
        if (loads > 0) tc_commit(&C->q_empty[(loads - 1) % QS]);  // the last product with those rows is issued
        have = row;
        if (!wait(C, &C->q_full[loads % QS], (loads / QS) & 1, P.wait_limit_ns)) return;
        ++loads;
      }
      if (d >= 2 && !wait(C, &C->s_empty[d & 1], ((d >> 1) - 1) & 1, P.wait_limit_ns)) return;
      tc_fence_after_sync();
      const uint32_t q_lo = sdesc_lo(smem_u32(smem + (3 - QS + (loads - 1) % QS) * kStage), 16);
      const uint32_t acc = tmem + 128u * (d & 1);
      // rotated dims: hi hi, hi lo, lo hi; then the pass-through dims
#pragma unroll
      for (int k = 0; k < 4; ++k) mma_ss_lo(acc, k_lo + 2 * k, q_lo + 2 * k, idesc_f16, k > 0 ? 1u : 0u);
#pragma unroll
      for (int k = 0; k < 4; ++k) mma_ss_lo(acc, k_lo + 2 * k, q_lo + kStep + 2 * k, idesc_f16, 1u);
#pragma unroll
      for (int k = 0; k < 4; ++k) mma_ss_lo(acc, k_lo + 3 * kStep + 2 * k, q_lo + 2 * k, idesc_f16, 1u);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ss_lo(acc, k_lo + (1 + u) * kStep + 2 * k, q_lo + (2 + u) * kStep + 2 * k, idesc_bf16, 1u);
      tc_commit(&C->s_full[d & 1]);
    }
    tc_commit(&C->k_empty[st]);
  }
}

__device__ __forceinline__ void role_sum(Ctrl* C, uint32_t tmem, const Params& P, int r, int wq) {
  const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
  const float sl2 = P.scale_log2;
  Walker walk(P);
  Unit w;
  long long have = -1;
  uint32_t loads = 0, d = 0;
#pragma unroll 1
  while (walk.next(P, w)) {
    const int key = w.k0 + r;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int qt = w.qt0; qt < w.qt1; ++qt, ++d) {
      const long long row = w.row0 + static_cast<long long>(qt) * P.ntile;
      bool ok = true;
      if (row != have) {
        // this load's lse; the loader is at most three loads ahead (its rows wait for the products of the
        // load before, and those for the score tiles), so the slot still holds it
        have = row;
        ok = wait(C, &C->lse_full[loads % kLseSlots], (loads / kLseSlots) & 1, P.wait_limit_ns);
        ++loads;
      }
      const float* lse2 = C->lse2[(loads - 1) % kLseSlots];
      // columns (query rows) that see this key: a run
      const long long base = static_cast<long long>(qt) * P.ntile;
      const long long seen = (static_cast<long long>(key) - w.p0) * P.group - base;
      const int c_lo = static_cast<int>(max(0LL, min(seen, 128LL)));
      long long c_end = min(static_cast<long long>(P.ntile), w.rows - base);
      if (P.window >= 0) c_end = min(c_end, (static_cast<long long>(key) + P.window + 1 - w.p0) * P.group - base);
      const int c_hi = static_cast<int>(max(0LL, c_end));
      if (!__all_sync(0xffffffffu, ok && wait(C, &C->s_full[d & 1], (d >> 1) & 1, P.wait_limit_ns))) return;
      tc_fence_after_sync();
#pragma unroll 1
      for (int c0 = 0; c0 < P.ntile; c0 += 16) {
        uint32_t s[16];
        tmem_ld16(tmem + lane_base + 128u * (d & 1) + c0, s);
        tmem_ld16_wait(s);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float p = ex2_approx(fmaf(__uint_as_float(s[i]), sl2, -lse2[c0 + i]));
          acc[i & 3] += (c0 + i >= c_lo && c0 + i < c_hi) ? p : 0.f;
        }
      }
      tc_fence_before_sync();
      mbar_arrive(&C->s_empty[d & 1]);
    }
    if (r < w.nk)
      P.partial[(static_cast<size_t>(w.f) * P.hkv + w.g) * P.total_kv + w.kv_beg + key] =
          (acc[0] + acc[1]) + (acc[2] + acc[3]);
  }
}

template <int KS, int QS>
__global__ void __launch_bounds__(kThreads, 1) kw_main_kernel(const __grid_constant__ CUtensorMap tq,
                                                              const __grid_constant__ Params P) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Ctrl* C = reinterpret_cast<Ctrl*>(smem + kCtrlOff);
  const int tid = threadIdx.x, warp = tid >> 5;
  int skip = 0;
  if (tid == 0) {
    skip = (*reinterpret_cast<volatile unsigned int*>(&g_mimo_error) & kErrTimeout) != 0;
    if (smem_u32(smem) & 1023u) skip = 1;  // swizzled operands need a 1 KB aligned base
  }
  if (__syncthreads_or(skip)) return;
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&C->k_landed[s], 128);  // one cp.async arrival per fetcher thread
      mbar_init(&C->k_full[s], 128);
      mbar_init(&C->k_empty[s], 1);
      mbar_init(&C->q_full[s], 1);
      mbar_init(&C->q_empty[s], 1);
      mbar_init(&C->s_full[s], 1);
      mbar_init(&C->s_empty[s], 128);
    }
    for (int s = 0; s < kLseSlots; ++s) mbar_init(&C->lse_full[s], 32);
    C->abort = 0;
    fence_barrier_init();
  }
  if (tid < kRopeDims / 2) C->theta[tid] = P.theta[tid];
  if (warp == 12) {
    tmem_alloc(&C->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = C->tmem_base;
  if (warp < 4) {
    role_sum(C, tmem, P, tid, warp);
  } else if (warp < 8) {
    role_fetch<KS>(smem, C, P, tid - 128);
  } else if (warp < 12) {
    role_rotate<KS>(smem, C, P, tid - 256);
  } else if (warp == 12) {
    if ((tid & 31) == 0) role_mma<KS, QS>(smem, C, tmem, P);
  } else {
    role_load_q<QS>(smem, C, P, &tq, tid & 31);
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------- launch 3
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) kw_join_kernel(const __grid_constant__ Params P) {
  const long long i = static_cast<long long>(blockIdx.x) * kJoinThreads + threadIdx.x;
  if (i >= P.total_kv) return;
  int a = 0, z = P.num_seqs;
  while (z - a > 1) {
    const int m = (a + z) / 2;
    if (__ldg(P.kv_indptr + m) <= i) a = m;
    else z = m;
  }
  Seq s;
  if (!load_seq(P, a, s) || i < s.kv_beg || i >= s.kv_beg + s.kv_len) return;  // left as it was
  float v = 0.f;
  if (i - s.kv_beg >= s.lo)
    for (int k = 0; k < P.splits * P.hkv; ++k) v += P.partial[static_cast<size_t>(k) * P.total_kv + i];
  P.out[i] = P.prev != nullptr ? P.prev[i] + v : v;
}

}  // namespace kw
}  // namespace mimo
