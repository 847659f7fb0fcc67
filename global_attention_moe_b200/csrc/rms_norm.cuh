// rms_norm.cuh -- the norm in front of the attention and of the experts: RMS norm with the residual's
// addition, an output in BF16 and / or in E4M3 with one scale per 1 x 128 block, and its gradient.
//
//   h    = bf16(x + r)                      (h = x without a residual)
//   rstd = 1 / sqrt(mean(h^2) + eps)
//   y    = h rstd w
//   FP8:  scale = max(max|y| / 448, 2^-126) over 128 consecutive columns, code = e4m3(y / scale)
//   gradient, with g = dy w:  dx = rstd g - h rstd^3 (sum g h) / H + dh,  dw = sum_t dy h rstd
//
// The norm is taken of h as it is stored (rounded to BF16 once), so the gradient, which reads h, is that
// of exactly the function computed.  Sums, rstd and y are FP32; y is rounded once, to BF16 and to E4M3
// each from the FP32 value.
//
// Both directions are bound by HBM: a row is read once and kept in registers (as BF16 pairs) between the
// reduction and the output.  A row whose sum of squares passes FP32's range (values near 2^64 and more)
// is reduced once more with its values times 2^-80; eps is at least 1e-18, so that squares too small for
// FP32 do not matter beside it.  TPR threads share a row, vector v of 8 columns belonging to thread v % TPR,
// at most 4 vectors each.  16384 x 4096 with a residual to FP8: 73 us, 6.4 TB/s (98% of a copy's rate).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "sm100.cuh"

namespace mimo {
namespace rms {

constexpr int kMaxFeatures = 16384;  // 512 threads x 4 vectors x 8 columns
constexpr int kFp8Block = 128;       // columns per scale: 16 vectors, one half-warp
constexpr float kFp8Max = 448.f;
constexpr int kBwdThreads = 512;

struct NormParams {
  const uint16_t* x;       // bf16 [T, H]
  const uint16_t* r;       // bf16 [T, H] or nullptr
  const void* w;           // bf16 or fp32 [H]
  uint16_t* h;             // bf16 [T, H] or nullptr
  uint16_t* y;             // bf16 [T, H] or nullptr
  uint8_t* codes;          // e4m3 [T, H] or nullptr
  float* scale;            // fp32 [T, ceil(H / 128)]
  int64_t T;
  int H;
  float eps;
};

struct NormBwdParams {
  const uint16_t* h;   // bf16 [T, H]
  const uint16_t* dy;  // bf16 [T, H]
  const uint16_t* dh;  // bf16 [T, H] or nullptr
  const void* w;       // bf16 or fp32 [H]
  uint16_t* dx;        // bf16 [T, H]
  float* partial;      // fp32 [CTAs, H]
  int64_t T;
  int H;
  float eps;
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(w[e] << 16);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// Weights of vector v (8 columns).
template <class WT>
__device__ __forceinline__ void load_w(const void* w, int v, float (&f)[8]);
template <>
__device__ __forceinline__ void load_w<uint16_t>(const void* w, int v, float (&f)[8]) {
  unpack8(__ldg(static_cast<const uint4*>(w) + v), f);
}
template <>
__device__ __forceinline__ void load_w<float>(const void* w, int v, float (&f)[8]) {
  const float4 a = __ldg(static_cast<const float4*>(w) + 2 * v), b = __ldg(static_cast<const float4*>(w) + 2 * v + 1);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The row's sum over its TPR threads; every thread of the row calls it.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* s_sum) {
  v = warp_sum(v);
  if (TPR > 32) {
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int k = 0; k < TPR / 32; ++k) v += s_sum[k];
  }
  return v;
}

template <int V>
__device__ __forceinline__ float squares(const uint4 (&hv)[V]) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float f[8];
    unpack8(hv[i], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
  }
  return ss;
}

constexpr float kDown = 0x1p-80f;
// Values times 2^-80 (exact, but for values that this makes too small to matter beside the row's largest).
template <int V>
__device__ __forceinline__ void scale_down(uint4 (&hv)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float f[8];
    unpack8(hv[i], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= kDown;
    hv[i] = pack8(f);
  }
}

// TPR threads per row, V vectors of 8 columns per thread (V TPR >= H / 8); rows of a CTA in parallel.
// x, r and h may be the same memory (each thread reads its columns before it writes them), so they are
// read with ordinary loads.
template <int TPR, int V, bool kFp8, class WT>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) rms_norm_kernel(const __grid_constant__ NormParams P) {
  constexpr int kThreads = TPR < 128 ? 128 : TPR;
  __shared__ float s_sum[2][kThreads / 32];
  const int t = threadIdx.x % TPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / TPR) + threadIdx.x / TPR;
  if (row >= P.T) return;  // whole warps; with more than one warp per row the CTA has only this row
  const int n = P.H / 8;
  const uint4* x = reinterpret_cast<const uint4*>(P.x + row * P.H);
  uint4 hv[V];
#pragma unroll
  for (int i = 0; i < V; ++i) hv[i] = t + i * TPR < n ? x[t + i * TPR] : make_uint4(0, 0, 0, 0);
  if (P.r != nullptr) {
    const uint4* r = reinterpret_cast<const uint4*>(P.r + row * P.H);
    uint4 rv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) rv[i] = t + i * TPR < n ? r[t + i * TPR] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float a[8], b[8];
      unpack8(hv[i], a);
      unpack8(rv[i], b);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 h2 = fadd2(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]));
        a[e] = h2.x, a[e + 1] = h2.y;
      }
      hv[i] = pack8(a);
    }
  }
  if (P.h != nullptr) {
    uint4* h = reinterpret_cast<uint4*>(P.h + row * P.H);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (t + i * TPR < n) h[t + i * TPR] = hv[i];
  }
  float ss = row_sum<TPR>(squares(hv), s_sum[0]);
  float eps = P.eps;
  if (!(ss <= 3.4e38f)) {  // the same for every thread of the row
    scale_down(hv);
    eps *= kDown;
    eps *= kDown;
    ss = row_sum<TPR>(squares(hv), s_sum[1]);
  }
  const float rstd = 1.f / sqrtf(ss / static_cast<float>(P.H) + eps);
  const int blocks = (P.H + kFp8Block - 1) / kFp8Block;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = t + i * TPR;
    const bool in = v < n;
    if (!kFp8 && !in) break;
    float f[8];
    unpack8(hv[i], f);
    if (in) {
      float w[8];
      load_w<WT>(P.w, v, w);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {  // (f rstd) w
        const float2 y2 = fmul2(fmul2(make_float2(f[e], f[e + 1]), make_float2(rstd, rstd)), make_float2(w[e], w[e + 1]));
        f[e] = y2.x, f[e + 1] = y2.y;
      }
    }
    if (P.y != nullptr && in) reinterpret_cast<uint4*>(P.y + row * P.H)[v] = pack8(f);
    if (kFp8) {
      // the block's 16 vectors are in the 16 lanes of this half-warp (those past the row hold zeros)
      float a = 0.f;
#pragma unroll
      for (int e = 0; e < 8; e += 2) a = fmax3(a, fabsf(f[e]), fabsf(f[e + 1]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      const float scale = fmaxf(__fdiv_rn(a, kFp8Max), 0x1p-126f);  // a block of zeros: the smallest normal scale
      if (in) {
        // The quotients, negated: q = y (1 / scale) and one step with the remainder y - q scale, which is exact
        // (Markstein), so that they are the rounded y / scale.  With BF16 rows and weights 2 to 4 of 10000 lie on a
        // midpoint of two codes, where the reciprocal's rounding would decide.  Negated, so that zeros keep their
        // sign; an infinite scale takes no step (codes 0, and NaN where y is infinite).  A division for each: 82 us,
        // for those near a midpoint 79 to 90, this, as the reciprocal alone, 73 (16384 x 4096).
        const float ninv = -1.f / scale, sc = scale < INFINITY ? scale : 0.f;
        uint32_t c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 y2 = make_float2(f[2 * e], f[2 * e + 1]), ninv2 = make_float2(ninv, ninv);
          float2 q = fmul2(y2, ninv2);
          q = ffma2(ffma2(q, make_float2(sc, sc), y2), ninv2, q);
          c[e] = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
        }
        reinterpret_cast<uint2*>(P.codes + row * P.H)[v] =
            make_uint2((c[0] | (c[1] << 16)) ^ 0x80808080u, (c[2] | (c[3] << 16)) ^ 0x80808080u);
        if ((v & 15) == 0) P.scale[row * blocks + (v >> 4)] = scale;
      }
    }
  }
}

// Gradient.  A CTA of 512 threads holds 512 / TPR row groups; each group walks rows with a stride over
// the grid, each thread keeping the dw sums of its columns in registers; at the end the groups' sums are
// added in shared memory in a fixed order and written as the CTA's partial row.  rms_norm_dw_kernel adds
// the partial rows, also in a fixed order, so dw does not change from run to run.  dx may be dy's or dh's
// memory (a thread reads its columns before it writes them), so those are read with ordinary loads.
// 16384 x 4096 with dh: 96 us, 5.6 TB/s; a CTA of 16 warps an SM, at 126 registers the row and its dw sums.
template <int TPR, int V, class WT>
__global__ void __launch_bounds__(kBwdThreads, 1) rms_norm_bwd_kernel(const __grid_constant__ NormBwdParams P) {
  constexpr int kGroups = kBwdThreads / TPR;
  extern __shared__ __align__(16) float sm[];  // H floats
  __shared__ float2 s_sum[2][kBwdThreads / 32];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const int n = P.H / 8;
  float acc[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[i][e] = 0.f;
  int par = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kGroups + grp; row < P.T;
       row += static_cast<int64_t>(gridDim.x) * kGroups) {
    const uint4* h = reinterpret_cast<const uint4*>(P.h + row * P.H);
    const uint4* dy = reinterpret_cast<const uint4*>(P.dy + row * P.H);
    uint4 hv[V], gv[V], dv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool in = t + i * TPR < n;
      hv[i] = in ? __ldg(h + t + i * TPR) : make_uint4(0, 0, 0, 0);
      gv[i] = in ? dy[t + i * TPR] : make_uint4(0, 0, 0, 0);
    }
    if (P.dh != nullptr) {
      const uint4* dh = reinterpret_cast<const uint4*>(P.dh + row * P.H);
#pragma unroll
      for (int i = 0; i < V; ++i) dv[i] = t + i * TPR < n ? dh[t + i * TPR] : make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) dv[i] = make_uint4(0, 0, 0, 0);
    }
    float ss, gh;
    auto sums = [&] {
      ss = gh = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (t + i * TPR >= n) break;
        float f[8], g[8], w[8];
        unpack8(hv[i], f);
        unpack8(gv[i], g);
        load_w<WT>(P.w, t + i * TPR, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ss = fmaf(f[e], f[e], ss);
          gh = fmaf(g[e] * w[e], f[e], gh);
        }
      }
      ss = warp_sum(ss);
      gh = warp_sum(gh);
      if (TPR > 32) {
        // two buffers: a group's warps may be one reduction apart, never two
        if ((threadIdx.x & 31) == 0) s_sum[par][threadIdx.x >> 5] = make_float2(ss, gh);
        named_bar_sync(1 + grp, TPR);
        ss = gh = 0.f;
#pragma unroll
        for (int k = 0; k < TPR / 32; ++k) {
          const float2 p = s_sum[par][grp * (TPR / 32) + k];
          ss += p.x;
          gh += p.y;
        }
        par ^= 1;
      }
    };
    sums();
    float eps = P.eps, down = 1.f;
    if (!(ss <= 3.4e38f)) {  // the same for every thread of the row
      scale_down(hv);
      down = kDown;
      eps *= kDown;
      eps *= kDown;
      sums();
    }
    // n = h rstd does not change with the scale of h; dx does, as rstd
    const float rstd = 1.f / sqrtf(ss / static_cast<float>(P.H) + eps), rout = rstd * down;
    const float c = rstd * rstd * gh / static_cast<float>(P.H);  // dx = rstd (g - h c)
    uint4* dx = reinterpret_cast<uint4*>(P.dx + row * P.H);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (t + i * TPR >= n) break;
      float f[8], g[8], d[8], w[8];
      unpack8(hv[i], f);
      unpack8(gv[i], g);
      unpack8(dv[i], d);
      load_w<WT>(P.w, t + i * TPR, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        acc[i][e] = fmaf(g[e], f[e] * rstd, acc[i][e]);
        d[e] = fmaf(rout, g[e] * w[e] - f[e] * c, d[e]);
      }
      dx[t + i * TPR] = pack8(d);
    }
  }
  // the groups' dw sums, added in the order of the groups
  for (int g = 0; g < kGroups; ++g) {
    if (g > 0) __syncthreads();
    if (grp == g) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = t + i * TPR;
        if (v >= n) break;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float s = g > 0 ? sm[8 * v + e] + acc[i][e] : acc[i][e];
          if (g == kGroups - 1)
            P.partial[static_cast<int64_t>(blockIdx.x) * P.H + 8 * v + e] = s;
          else
            sm[8 * v + e] = s;
        }
      }
    }
  }
}

// dw[c] = sum over the partial rows, in order: 64 columns per CTA, 16 threads (4 columns each) x 16
// interleaved row chains, then the chains in order.
constexpr int kDwThreads = 256;
__global__ void __launch_bounds__(kDwThreads) rms_norm_dw_kernel(const float* __restrict__ partial, float* __restrict__ dw,
                                                                 int rows, int H) {
  __shared__ float4 s[16][16];
  const int q = threadIdx.x & 15, k = threadIdx.x >> 4;
  const int c = blockIdx.x * 64 + 4 * q;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < H)
    for (int i = k; i < rows; i += 16) {
      const float4 p = *reinterpret_cast<const float4*>(partial + static_cast<int64_t>(i) * H + c);
      a.x += p.x, a.y += p.y, a.z += p.z, a.w += p.w;
    }
  s[k][q] = a;
  __syncthreads();
  if (k == 0 && c < H) {
    for (int i = 1; i < 16; ++i) {
      const float4 p = s[i][q];
      a.x += p.x, a.y += p.y, a.z += p.z, a.w += p.w;
    }
    *reinterpret_cast<float4*>(dw + c) = a;
  }
}

}  // namespace rms
}  // namespace mimo
