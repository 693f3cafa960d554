// Layer norm of rows of `dim` values and its gradient:
//   mean = sum x / dim, var = sum (x - mean)^2 / dim, rstd = 1 / sqrt(var + eps)
//   xh = (x - mean) rstd,   y = xh weight + bias
//   g = dy weight,  dx = rstd (g - sum(g) / dim - xh sum(g xh) / dim)
//   dweight = sum over rows of dy xh,   dbias = sum over rows of dy
// (the indexer's key norm, and its gradient from the warm-up loss's dk).
//
// Floor: HBM, each row read once and written once. Wide aligned rows come near it
// (8191 fp32 rows of 4096, the gradient: 5.7 TB/s; 16384 of 8192: 6.6); narrow rows wait
// for their loads, with 28 and, in the gradient, 16 warps per SM (65536 bf16 rows of
// 128: 8.4 us, and 16.8 with the weights' sums). A row stays in registers
// between its passes (two passes for the variance: sum of squares minus
// squared mean would cancel in fp32 when |mean| >> sigma). TPR threads share a
// row and hold 8 NV elements each. Arithmetic is fp32 but for the gradient of rows of
// up to four values; bf16 only at loads and stores.
//
// The weight's gradient: a thread keeps the sums of its columns over all the
// rows its CTA walks, the CTA writes one partial row, and a second kernel adds
// the partial rows in order (the same bits on every call).
#pragma once

#include <cuda_bf16.h>

#include "ptx.cuh"

namespace dsa {

constexpr int kNormMaxDim = 16384;

struct NormParams {
  const void* x;
  const float* w;
  const float* b;
  void* y;
  float* mean;
  float* rstd;
  long long rows, xs, ys;          // row strides in elements
  int dim;
  int x_bf16, y_bf16;
  float eps;
};

struct NormBwdParams {
  const void* dy;
  const void* x;
  const float* w;
  const float* mean;
  const float* rstd;
  void* dx;
  float* part;                     // [CTA][2][dim]: partial dweight, dbias
  long long rows, dys, xs, dxs;
  int dim;
  int dy_bf16, x_bf16, dx_bf16;
};

// Element types of a row tensor as a template argument; kAny: told at run time.
enum { kRowF32 = 0, kRowBf16 = 1, kRowAny = 2 };

// One thread's elements of a row as loaded: 8 NV of them in chunks of E (VEC),
// or one by one, TPR apart. E = 8 makes 16-byte accesses of bf16 but leaves the
// halves of fp32 sectors to two instructions, so rows with an fp32 tensor among
// theirs take E = 4.
template <bool VEC, int TPR, int NV, int TYPE, int E>
struct NormRow {
  static constexpr int EPT = 8 * NV, CHUNKS = EPT / E;
  static constexpr int PER = VEC && TYPE == kRowBf16 ? E / 2 : E;    // words per chunk
  uint32_t w[PER * CHUNKS];        // fp32 bits, or for VEC bf16 pairs in a chunk's first half

  __device__ __forceinline__ static int elem(int lane, int j) {
    return VEC ? ((j / E) * TPR + lane) * E + j % E : j * TPR + lane;
  }
  __device__ __forceinline__ static bool is_bf16(int flag) {
    return TYPE == kRowAny ? flag != 0 : TYPE == kRowBf16;
  }
  __device__ __forceinline__ void load(const void* base, long long off, int flag, int lane, int dim) {
    if constexpr (VEC) {
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) {
        const int e = elem(lane, c * E);
        uint32_t* v = w + c * PER;
#pragma unroll
        for (int k = 0; k < PER; ++k) v[k] = 0u;
        if (e >= dim) continue;
        if (is_bf16(flag)) {
          const uint16_t* s = static_cast<const uint16_t*>(base) + off + e;
          if constexpr (E == 8) {
            const uint4 u = *reinterpret_cast<const uint4*>(s);
            v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
          } else {
            const uint2 u = *reinterpret_cast<const uint2*>(s);
            v[0] = u.x; v[1] = u.y;
          }
        } else if constexpr (PER == E) {
          const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + off + e);
#pragma unroll
          for (int k = 0; k < E; k += 4) {
            const uint4 u = s[k / 4];
            v[k] = u.x; v[k + 1] = u.y; v[k + 2] = u.z; v[k + 3] = u.w;
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < EPT; ++j) {
        const int e = elem(lane, j);
        w[j] = 0u;
        if (e < dim)
          w[j] = is_bf16(flag) ? static_cast<uint32_t>(static_cast<const uint16_t*>(base)[off + e]) << 16
                               : __float_as_uint(static_cast<const float*>(base)[off + e]);
      }
    }
  }
  // Elements past dim read as 0.
  __device__ __forceinline__ void get(float (&f)[EPT], int flag) const {
    if (VEC && is_bf16(flag)) {
#pragma unroll
      for (int j = 0; j < EPT; ++j) {
        const uint32_t u = w[(j / E) * PER + (j % E) / 2];
        f[j] = __uint_as_float((j & 1) ? (u & 0xffff0000u) : (u << 16));
      }
    } else if constexpr (!VEC || TYPE != kRowBf16) {
#pragma unroll
      for (int j = 0; j < EPT; ++j) f[j] = __uint_as_float(w[j]);
    }
  }
};

// Stores one thread's elements of a row in the same arrangement.
template <bool VEC, int TPR, int NV, int E>
__device__ __forceinline__ void norm_store(void* base, long long off, int bf16, int lane, int dim,
                                           const float (&f)[8 * NV]) {
  using Row = NormRow<VEC, TPR, NV, kRowAny, E>;
  if constexpr (VEC) {
#pragma unroll
    for (int c = 0; c < 8 * NV / E; ++c) {
      const int e = Row::elem(lane, c * E);
      if (e >= dim) continue;
      const float* v = f + c * E;
      if (bf16) {
        uint32_t u[E / 2];
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
          u[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        uint16_t* d = static_cast<uint16_t*>(base) + off + e;
        if constexpr (E == 8) *reinterpret_cast<uint4*>(d) = make_uint4(u[0], u[1], u[E / 2 - 2], u[E / 2 - 1]);
        else *reinterpret_cast<uint2*>(d) = make_uint2(u[0], u[1]);
      } else {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(base) + off + e);
#pragma unroll
        for (int k = 0; k < E; k += 4) d[k / 4] = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8 * NV; ++j) {
      const int e = Row::elem(lane, j);
      if (e >= dim) continue;
      if (bf16) static_cast<__nv_bfloat16*>(base)[off + e] = __float2bfloat16_rn(f[j]);
      else static_cast<float*>(base)[off + e] = f[j];
    }
  }
}

// One thread's fp32 weights in a row's arrangement: `fill` where there are none.
template <bool VEC, int TPR, int NV, int E>
__device__ __forceinline__ void norm_weights(const float* w, float fill, int lane, int dim,
                                             float (&f)[8 * NV]) {
  using Row = NormRow<VEC, TPR, NV, kRowAny, E>;
#pragma unroll
  for (int j = 0; j < 8 * NV; j += VEC ? 4 : 1) {
    const int e = Row::elem(lane, j);
    if constexpr (VEC) {
      float4 v = make_float4(fill, fill, fill, fill);
      if (w && e < dim) v = __ldg(reinterpret_cast<const float4*>(w + e));
      f[j] = v.x; f[j + 1] = v.y; f[j + 2] = v.z; f[j + 3] = v.w;
    } else {
      f[j] = w && e < dim ? __ldg(w + e) : fill;
    }
  }
}

// Sums over the TPR threads of a row. More than a warp: through shared memory,
// `buf` alternating between two sets of slots so that one barrier per sum
// suffices.
template <int TPR>
__device__ __forceinline__ float2 norm_sum2(float a, float b, float2* slots, int& buf) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    float2* s = slots + buf * W;
    buf ^= 1;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float2 v = s[i];
      a += v.x;
      b += v.y;
    }
  }
  return make_float2(a, b);
}
template <int TPR>
__device__ __forceinline__ float norm_sum(float a, float2* slots, int& buf) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    float2* s = slots + buf * W;
    buf ^= 1;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5].x = a;
    __syncthreads();
    a = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) a += s[i].x;
  }
  return a;
}

// Threads per CTA: rows of up to a warp's threads share one.
template <int TPR>
constexpr int norm_threads() { return TPR <= 32 ? 256 : TPR; }

// CTAs per SM that the registers are bounded for, without and with the gradient.
constexpr int norm_ctas(int tpr, bool gradient) {
  return gradient ? (tpr <= 32 ? 2 : tpr == 128 ? 4 : 1) : (tpr <= 32 ? 4 : tpr == 128 ? 6 : tpr == 512 ? 2 : 1);
}

// How a group keeps bytes in flight: narrow rows are loaded U at a time, wide
// ones one row ahead (PRE), the others rely on the other CTAs.
template <int TPR, int NV, int TYPE>
struct NormFlow {
  static constexpr int U = TPR <= 32 && NV == 1 ? (TYPE == kRowBf16 ? 4 : 2) : 1;
  static constexpr bool PRE = U == 1 && NV == 1;
  static constexpr bool KEEP = NV == 1;                  // weights stay in registers
};

template <bool VEC, int TPR, int NV, int TYPE>
__global__ void __launch_bounds__(norm_threads<TPR>(), norm_ctas(TPR, false))
    norm_kernel(const NormParams p) {
  constexpr int E = TYPE == kRowBf16 ? 8 : 4;
  using Row = NormRow<VEC, TPR, NV, TYPE, E>;
  using F = NormFlow<TPR, NV, TYPE>;
  constexpr int EPT = Row::EPT, GROUPS = norm_threads<TPR>() / TPR;
  __shared__ float2 slots[TPR > 32 ? 2 * TPR / 32 : 1];
  int buf = 0;
  const int lane = threadIdx.x % TPR;
  const long long step = static_cast<long long>(gridDim.x) * GROUPS;
  // A whole warp stays in the loop (the sums use full-warp shuffles): a group
  // past the last row loads nothing and stores nothing.
  const long long base = static_cast<long long>(blockIdx.x) * GROUPS;
  const int g = threadIdx.x / TPR;
  Row raw[F::U], next;
  if (F::PRE && base + g < p.rows) raw[0].load(p.x, (base + g) * p.xs, p.x_bf16, lane, p.dim);
  float w[EPT], b[EPT];
  if constexpr (F::KEEP) {
    norm_weights<VEC, TPR, NV, E>(p.w, 1.f, lane, p.dim, w);
    norm_weights<VEC, TPR, NV, E>(p.b, 0.f, lane, p.dim, b);
  }
  const float inv = 1.0f / static_cast<float>(p.dim);
  for (long long r0 = base; r0 < p.rows; r0 += step * F::U) {
    if constexpr (F::PRE) {
      if (r0 + g + step < p.rows) next.load(p.x, (r0 + g + step) * p.xs, p.x_bf16, lane, p.dim);
    } else {
#pragma unroll
      for (int u = 0; u < F::U; ++u) {
        const long long r = r0 + g + u * step;
        if (r < p.rows) raw[u].load(p.x, r * p.xs, p.x_bf16, lane, p.dim);
      }
    }
#pragma unroll
    for (int u = 0; u < F::U; ++u) {
      if (u > 0 && r0 + u * step >= p.rows) break;       // the same in the whole CTA
      const long long r = r0 + g + u * step;
      float x[EPT];
      raw[u].get(x, p.x_bf16);
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < EPT; ++j) s += x[j];
      const float mean = norm_sum<TPR>(s, slots, buf) * inv;
      float q = 0.f;
#pragma unroll
      for (int j0 = 0; j0 < EPT; j0 += VEC ? E : 1) {
        float part = 0.f;
#pragma unroll
        for (int j = j0; j < j0 + (VEC ? E : 1); ++j) {
          x[j] -= mean;
          part = fmaf(x[j], x[j], part);
        }
        if (Row::elem(lane, j0) < p.dim) q += part;      // a chunk is inside the row or outside
      }
      const float var = norm_sum<TPR>(q, slots, buf) * inv;
      const float rstd = rsqrtf(var + p.eps);
      if (r < p.rows) {
        if constexpr (!F::KEEP) {
          norm_weights<VEC, TPR, NV, E>(p.w, 1.f, lane, p.dim, w);
          norm_weights<VEC, TPR, NV, E>(p.b, 0.f, lane, p.dim, b);
        }
#pragma unroll
        for (int j = 0; j < EPT; ++j) x[j] = fmaf(x[j] * rstd, w[j], b[j]);
        norm_store<VEC, TPR, NV, E>(p.y, r * p.ys, p.y_bf16, lane, p.dim, x);
        if (lane == 0) {
          if (p.mean) p.mean[r] = mean;
          if (p.rstd) p.rstd[r] = rstd;
        }
      }
    }
    if constexpr (F::PRE) raw[0] = next;
  }
}

// Whether the places past a row's end, which hold (0 - mean) rstd and are multiplied
// by 0, would overflow to infinity and make their products NaN: rows of equal values
// past 1e35, say. Such a row's sum is formed again without them. PADS: compiled
// only into the kernels of rows that leave places empty, as the branch alone costs
// registers (8191 fp32 rows of 4096: 70.0 us, 72.9 with it, 80.8 with a test at
// every place).
__device__ __forceinline__ bool norm_pads_overflow(float mean, float rstd) {
  return !(fabsf(mean * rstd) < INFINITY);
}

// The same for the gradient, which loads two rows and keeps column sums.
template <int TPR, int NV>
struct NormBwdFlow {
  static constexpr int U = TPR <= 32 && NV == 1 ? 2 : 1;
  static constexpr bool PRE = U == 1 && NV == 1;
  static constexpr bool KEEP = NV == 1;
};

template <bool VEC, bool PADS, int TPR, int NV, int XT, int GT>
__global__ void __launch_bounds__(norm_threads<TPR>(), norm_ctas(TPR, true))
    norm_bwd_kernel(const NormBwdParams p) {
  constexpr int E = XT == kRowBf16 && GT == kRowBf16 ? 8 : 4;
  using RowX = NormRow<VEC, TPR, NV, XT, E>;
  using RowG = NormRow<VEC, TPR, NV, GT, E>;
  using F = NormBwdFlow<TPR, NV>;
  constexpr int EPT = RowX::EPT, THREADS = norm_threads<TPR>(), GROUPS = THREADS / TPR;
  constexpr int COLS = TPR * EPT;                       // columns a group covers, >= dim
  __shared__ float2 slots[TPR > 32 ? 2 * TPR / 32 : 1];
  int buf = 0;
  const int lane = threadIdx.x % TPR;
  const long long step = static_cast<long long>(gridDim.x) * GROUPS;
  const long long base = static_cast<long long>(blockIdx.x) * GROUPS;
  const int g = threadIdx.x / TPR;
  RowX cx[F::U], nx;
  RowG cy[F::U], ny;
  float mean[F::U], rstd[F::U], nmean = 0.f, nrstd = 0.f;
  auto fetch = [&](long long r, RowX& rx, RowG& ry, float& m, float& s) {
    if (r < p.rows) {
      rx.load(p.x, r * p.xs, p.x_bf16, lane, p.dim);
      ry.load(p.dy, r * p.dys, p.dy_bf16, lane, p.dim);
      m = p.mean[r];
      s = p.rstd[r];
    }
  };
  if constexpr (F::PRE) fetch(base + g, cx[0], cy[0], mean[0], rstd[0]);
  float w[EPT], aw[EPT], ab[EPT];
  if constexpr (F::KEEP) norm_weights<VEC, TPR, NV, E>(p.w, 1.f, lane, p.dim, w);
#pragma unroll
  for (int j = 0; j < EPT; ++j) aw[j] = ab[j] = 0.f;
  const float inv = 1.0f / static_cast<float>(p.dim);
  for (long long r0 = base; r0 < p.rows; r0 += step * F::U) {
    if constexpr (F::PRE) {
      fetch(r0 + g + step, nx, ny, nmean, nrstd);
    } else {
#pragma unroll
      for (int u = 0; u < F::U; ++u) fetch(r0 + g + u * step, cx[u], cy[u], mean[u], rstd[u]);
    }
#pragma unroll
    for (int u = 0; u < F::U; ++u) {
      if (u > 0 && r0 + u * step >= p.rows) break;       // the same in the whole CTA
      const long long r = r0 + g + u * step;
      const bool there = r < p.rows;
      float x[EPT], d[EPT];
      cx[u].get(x, p.x_bf16);
      cy[u].get(d, p.dy_bf16);
      if constexpr (!F::KEEP) norm_weights<VEC, TPR, NV, E>(p.w, 1.f, lane, p.dim, w);
      float sg = 0.f, sgx = 0.f;
#pragma unroll
      for (int j = 0; j < EPT; ++j) {
        // past the row's end d is 0, and with it every product (see norm_pads_overflow)
        x[j] = (x[j] - mean[u]) * rstd[u];
        if (there) {
          aw[j] = fmaf(d[j], x[j], aw[j]);
          ab[j] += d[j];
        }
        d[j] *= w[j];
        sg += d[j];
        sgx = fmaf(d[j], x[j], sgx);
      }
      if (PADS && norm_pads_overflow(mean[u], rstd[u])) {
        sgx = 0.f;
#pragma unroll
        for (int j = 0; j < EPT; ++j)
          if (RowX::elem(lane, j) < p.dim) sgx = fmaf(d[j], x[j], sgx);
      }
      const float2 s = norm_sum2<TPR>(sg, sgx, slots, buf);
      const float mg = s.x * inv, mgx = s.y * inv;
      if (there) {
#pragma unroll
        for (int j = 0; j < EPT; ++j) d[j] = rstd[u] * (d[j] - mg - x[j] * mgx);
        norm_store<VEC, TPR, NV, E>(p.dx, r * p.dxs, p.dx_bf16, lane, p.dim, d);
      }
    }
    if constexpr (F::PRE) {
      cx[0] = nx;
      cy[0] = ny;
      mean[0] = nmean;
      rstd[0] = nrstd;
    }
  }
  griddep_launch_dependents();
  if (!p.part) return;
  // the CTA's partial sums: groups of a CTA hold the same columns
  float* part = p.part + static_cast<size_t>(blockIdx.x) * 2 * p.dim;
  if constexpr (GROUPS > 1) {
    constexpr int WARPS = THREADS / 32;
    __shared__ float acc[WARPS][COLS];                 // one quantity at a time
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int j = 0; j < EPT; ++j) {
        float v = k == 0 ? aw[j] : ab[j];
#pragma unroll
        for (int o = TPR; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        acc[threadIdx.x >> 5][RowX::elem(lane, j)] = v;
      }
      __syncthreads();
      for (int e = threadIdx.x; e < p.dim; e += THREADS) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) v += acc[i][e];
        part[k * p.dim + e] = v;
      }
      __syncthreads();
    }
  } else {
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
      const int e = RowX::elem(lane, j);
      if (e < p.dim) {
        part[e] = aw[j];
        part[p.dim + e] = ab[j];
      }
    }
  }
}

// ---------------------------------------------------------------- rows of a few values

// The gradient of rows of at most kNormFewDim values, a thread per row in fp64.
// dx is what g keeps without its parts along 1 and xh, and xh is orthogonal to 1, so
// rows of two values keep next to nothing of it: dx = rstd (g1 - g2) / 2 (1 - xh^2)
// with 1 - xh^2 = eps rstd^2, 1e-6 and less, which the rounding of xh to fp32
// (2^-24) buries: of 200 K such rows the median was off by 6 %. Rows of three or
// four values lose the digits where g happens to lie near the two directions (3 in
// 1000 and 1 in 100000 off by more than 2e-5), rows of five no longer (none). fp64
// costs nothing here: 65536 fp32 rows of two take 5.0 us (12.4 with 16 threads a row
// in fp32), one row 3.7 (3.1).
constexpr int kNormFewDim = 4, kNormFewThreads = 256, kNormFewCtas = 2;

__device__ __forceinline__ double norm_elem(const void* base, long long at, int bf16) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at]) : static_cast<const float*>(base)[at];
}

__global__ void __launch_bounds__(kNormFewThreads, kNormFewCtas) norm_bwd_few_kernel(const NormBwdParams p) {
  constexpr int D = kNormFewDim, WARPS = kNormFewThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double w[D], acc[2][D];          // acc: this thread's rows' dweight, dbias
#pragma unroll
  for (int j = 0; j < D; ++j) {
    w[j] = p.w && j < p.dim ? p.w[j] : 1.f;
    acc[0][j] = acc[1][j] = 0.0;
  }
  const double inv = 1.0 / p.dim;
  const long long step = static_cast<long long>(gridDim.x) * kNormFewThreads;
  for (long long r = static_cast<long long>(blockIdx.x) * kNormFewThreads + threadIdx.x; r < p.rows; r += step) {
    const double mean = p.mean[r], rstd = p.rstd[r];
    double h[D], g[D], sg = 0.0, sgx = 0.0;
#pragma unroll
    for (int j = 0; j < D; ++j) {
      if (j >= p.dim) continue;
      const double d = norm_elem(p.dy, r * p.dys + j, p.dy_bf16);
      h[j] = (norm_elem(p.x, r * p.xs + j, p.x_bf16) - mean) * rstd;
      acc[0][j] = fma(d, h[j], acc[0][j]);
      acc[1][j] += d;
      g[j] = d * w[j];
      sg += g[j];
      sgx = fma(g[j], h[j], sgx);
    }
    const double mg = sg * inv, mgx = sgx * inv;
#pragma unroll
    for (int j = 0; j < D; ++j) {
      if (j >= p.dim) continue;
      const float dx = static_cast<float>(rstd * (g[j] - mg - h[j] * mgx));
      if (p.dx_bf16) static_cast<__nv_bfloat16*>(p.dx)[r * p.dxs + j] = __float2bfloat16_rn(dx);
      else static_cast<float*>(p.dx)[r * p.dxs + j] = dx;
    }
  }
  griddep_launch_dependents();
  if (!p.part) return;
  __shared__ double sums[WARPS][2 * D];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < D; ++j) {
      double v = acc[k][j];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) sums[warp][k * D + j] = v;
    }
  __syncthreads();
  if (threadIdx.x < 2 * D && threadIdx.x % D < p.dim) {
    double v = 0.0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) v += sums[i][threadIdx.x];
    p.part[(static_cast<size_t>(blockIdx.x) * 2 + threadIdx.x / D) * p.dim + threadIdx.x % D] = static_cast<float>(v);
  }
}

// ---------------------------------------------------------------- wide rows

// Wide rows whose every 16-byte chunk is aligned. A CTA has
// one row at a time, with many elements per thread (the sums over threads cost
// the same for any number of them), while the rows to come are on their way into
// a ring of stages in shared memory (bulk copies, one stage per row). A stage is
// loaded anew after the barrier of its row's first sum, when every thread holds
// its part of the row in registers. Issuing a copy takes a thread about 290
// cycles, so the gradient's two are issued by two warps.
constexpr int kNormMaxStages = 8;
// Threads of an SM that the registers allow, without and with the gradient.
constexpr int kNormWideThreads = 768, kNormBwdWideThreads = 512;
constexpr int norm_wide_ctas(int tpr, bool gradient) {
  const int n = (gradient ? kNormBwdWideThreads : kNormWideThreads) / tpr;
  return n > 1 ? n : 1;
}

// Sums of N values per thread over the CTA's TPR threads, one barrier (`buf`
// alternates between two sets of slots).
template <int TPR, int N>
__device__ __forceinline__ void norm_sums(float (&v)[N], float* slots, int& buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  constexpr int W = TPR / 32;
  float* s = slots + buf * W * N;
  buf ^= 1;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i * W + (threadIdx.x >> 5)] = v[i];
  }
  __syncthreads();
  // lane k < W of every warp takes warp k's sum
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float t = (threadIdx.x & 31) < W ? s[i * W + (threadIdx.x & 31)] : 0.f;
#pragma unroll
    for (int o = (W > 1 ? W / 2 : 0); o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    v[i] = __shfl_sync(0xffffffffu, t, 0);
  }
}

struct NormRing {
  uint8_t* data;
  uint64_t* full;
  int st, stages;
  uint32_t phase;
  bool ok;

  // Every thread; `copies` arrivals complete a stage.
  __device__ __forceinline__ void init(uint8_t* smem, int n, int copies) {
    full = reinterpret_cast<uint64_t*>(smem);
    data = smem + 128;
    st = 0;
    stages = n;
    phase = 0;
    ok = true;
    if (threadIdx.x == 0) {
      for (int k = 0; k < kNormMaxStages; ++k) mbar_init(&full[k], copies);
      fence_mbar_init();
    }
    __syncthreads();
  }
  // The current stage, of row r, has landed. A wait that runs out is reported; the
  // thread waits once more for every copy in flight, issues none any more and goes
  // on without waiting, so that every thread meets every barrier.
  __device__ __forceinline__ void wait(long long r, long long step, long long rows) {
    if (!ok) return;
    ok = mbar_wait(&full[st], phase);
    if (ok) return;
#pragma unroll 1
    for (int k = 0; k < stages && r + k * step < rows; ++k)
      mbar_wait(&full[st + k < stages ? st + k : st + k - stages], st + k < stages ? phase : phase ^ 1);
  }
  __device__ __forceinline__ void next() {
    if (++st == stages) {
      st = 0;
      phase ^= 1;
    }
  }
};

template <int TPR, int NV>
__global__ void __launch_bounds__(TPR, norm_wide_ctas(TPR, false)) norm_wide_kernel(const NormParams p, int stages) {
  constexpr int E = 4, EPT = 8 * NV;
  constexpr bool KEEP = TPR < 1024;              // weights stay in registers
  using Row = NormRow<true, TPR, NV, kRowAny, E>;
  extern __shared__ __align__(128) uint8_t norm_smem[];
  __shared__ float slots[2 * TPR / 32];
  int buf = 0;
  const int lane = threadIdx.x;
  const long long step = gridDim.x;
  const uint32_t bytes = p.dim * (p.x_bf16 ? 2 : 4);
  NormRing ring;
  ring.init(norm_smem, stages, 1);
  auto copy_in = [&](long long r, int st) {
    if (r >= p.rows) return;
    mbar_arrive_expect_tx(&ring.full[st], bytes);
    bulk_load(smem_u32(ring.data + st * bytes), static_cast<const uint8_t*>(p.x) + r * p.xs * (p.x_bf16 ? 2 : 4),
              bytes, &ring.full[st]);
  };
  if ((lane & 31) == 0)
    for (int k = lane >> 5; k < stages; k += TPR / 32) copy_in(blockIdx.x + k * step, k);
  float w[EPT], b[EPT];
  if constexpr (KEEP) {
    norm_weights<true, TPR, NV, E>(p.w, 1.f, lane, p.dim, w);
    norm_weights<true, TPR, NV, E>(p.b, 0.f, lane, p.dim, b);
  }
  const float inv = 1.0f / static_cast<float>(p.dim);
  for (long long r = blockIdx.x; r < p.rows; r += step) {
    float x[EPT], s[1] = {0.f}, q[1] = {0.f};
    ring.wait(r, step, p.rows);
    {
      Row raw;
      raw.load(ring.data + ring.st * bytes, 0, p.x_bf16, lane, p.dim);
      raw.get(x, p.x_bf16);
    }
#pragma unroll
    for (int j = 0; j < EPT; ++j) s[0] += x[j];
    norm_sums<TPR, 1>(s, slots, buf);
    if (lane == 0 && ring.ok) copy_in(r + stages * step, ring.st);
    ring.next();
    const float mean = s[0] * inv;
#pragma unroll
    for (int j0 = 0; j0 < EPT; j0 += E) {
      float part = 0.f;
#pragma unroll
      for (int j = j0; j < j0 + E; ++j) {
        x[j] -= mean;
        part = fmaf(x[j], x[j], part);
      }
      if (Row::elem(lane, j0) < p.dim) q[0] += part;
    }
    norm_sums<TPR, 1>(q, slots, buf);
    const float rstd = rsqrtf(q[0] * inv + p.eps);
    if constexpr (!KEEP) {
      norm_weights<true, TPR, NV, E>(p.w, 1.f, lane, p.dim, w);
      norm_weights<true, TPR, NV, E>(p.b, 0.f, lane, p.dim, b);
    }
#pragma unroll
    for (int j = 0; j < EPT; ++j) x[j] = fmaf(x[j] * rstd, w[j], b[j]);
    norm_store<true, TPR, NV, E>(p.y, r * p.ys, p.y_bf16, lane, p.dim, x);
    if (lane == 0) {
      if (p.mean) p.mean[r] = mean;
      if (p.rstd) p.rstd[r] = rstd;
    }
  }
}

template <int TPR, int NV, bool PADS>
__global__ void __launch_bounds__(TPR, norm_wide_ctas(TPR, true))
    norm_bwd_wide_kernel(const NormBwdParams p, int stages) {
  constexpr int E = 4, EPT = 8 * NV;
  // Weights stay in registers where rows are short (2048: 50 us, 54 with reloads);
  // beside 256 or more threads' rows they cost more than their reloads (8191 fp32
  // rows of 4096: 77 us, 70 with reloads).
  constexpr bool KEEP = TPR == 128;
  using Row = NormRow<true, TPR, NV, kRowAny, E>;
  extern __shared__ __align__(128) uint8_t norm_smem[];
  __shared__ float slots[2 * 2 * TPR / 32];
  int buf = 0;
  const int lane = threadIdx.x, warp = threadIdx.x >> 5;
  const long long step = gridDim.x;
  const uint32_t x_bytes = p.dim * (p.x_bf16 ? 2 : 4), dy_bytes = p.dim * (p.dy_bf16 ? 2 : 4);
  NormRing ring;
  ring.init(norm_smem, stages, 2);
  auto copy_in = [&](long long r, int st, int dy) {
    if (r >= p.rows) return;
    uint8_t* dst = ring.data + st * (x_bytes + dy_bytes) + (dy ? x_bytes : 0);
    const uint32_t bytes = dy ? dy_bytes : x_bytes;
    const uint8_t* src = dy ? static_cast<const uint8_t*>(p.dy) + r * p.dys * (p.dy_bf16 ? 2 : 4)
                            : static_cast<const uint8_t*>(p.x) + r * p.xs * (p.x_bf16 ? 2 : 4);
    mbar_arrive_expect_tx(&ring.full[st], bytes);
    bulk_load(smem_u32(dst), src, bytes, &ring.full[st]);
  };
  if ((lane & 31) == 0)
    for (int k = warp; k < 2 * stages; k += TPR / 32) copy_in(blockIdx.x + (k >> 1) * step, k >> 1, k & 1);
  float w[EPT], aw[EPT], ab[EPT];
  if constexpr (KEEP) norm_weights<true, TPR, NV, E>(p.w, 1.f, lane, p.dim, w);
#pragma unroll
  for (int j = 0; j < EPT; ++j) aw[j] = ab[j] = 0.f;
  const float inv = 1.0f / static_cast<float>(p.dim);
  float nmean = 0.f, nrstd = 0.f;                        // of the row to come
  auto stats = [&](long long r) {
    if (r < p.rows) {
      nmean = __ldg(p.mean + r);
      nrstd = __ldg(p.rstd + r);
    }
  };
  stats(blockIdx.x);
  for (long long r = blockIdx.x; r < p.rows; r += step) {
    const float mean = nmean, rstd = nrstd;
    stats(r + step);
    float x[EPT], d[EPT], s[2] = {0.f, 0.f};
    ring.wait(r, step, p.rows);
    {
      const uint8_t* src = ring.data + ring.st * (x_bytes + dy_bytes);
      Row raw;
      raw.load(src, 0, p.x_bf16, lane, p.dim);
      raw.get(x, p.x_bf16);
      raw.load(src + x_bytes, 0, p.dy_bf16, lane, p.dim);
      raw.get(d, p.dy_bf16);
    }
    if constexpr (!KEEP) norm_weights<true, TPR, NV, E>(p.w, 1.f, lane, p.dim, w);
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
      // past the row's end d is 0, and with it every product (see norm_pads_overflow)
      x[j] = (x[j] - mean) * rstd;
      aw[j] = fmaf(d[j], x[j], aw[j]);
      ab[j] += d[j];
      d[j] *= w[j];
      s[0] += d[j];
      s[1] = fmaf(d[j], x[j], s[1]);
    }
    if (PADS && norm_pads_overflow(mean, rstd)) {
      s[1] = 0.f;
#pragma unroll
      for (int j = 0; j < EPT; ++j)
        if (Row::elem(lane, j) < p.dim) s[1] = fmaf(d[j], x[j], s[1]);
    }
    norm_sums<TPR, 2>(s, slots, buf);
    if ((lane & 31) == 0 && warp < 2 && ring.ok) copy_in(r + stages * step, ring.st, warp);
    ring.next();
    const float mg = s[0] * inv, mgx = s[1] * inv;
#pragma unroll
    for (int j = 0; j < EPT; ++j) d[j] = rstd * (d[j] - mg - x[j] * mgx);
    norm_store<true, TPR, NV, E>(p.dx, r * p.dxs, p.dx_bf16, lane, p.dim, d);
  }
  griddep_launch_dependents();
  if (!p.part) return;
  float* part = p.part + static_cast<size_t>(blockIdx.x) * 2 * p.dim;
#pragma unroll
  for (int j = 0; j < EPT; ++j) {
    const int e = Row::elem(lane, j);
    if (e < p.dim) {
      part[e] = aw[j];
      part[p.dim + e] = ab[j];
    }
  }
}

constexpr int kNormReduceUnroll = 10;   // partial rows a thread loads before it adds

// dweight, dbias: the n partial rows [2][dim] added in a fixed order, 32
// columns per CTA (of the 2 dim), 32 warps over the rows.
__global__ void __launch_bounds__(1024)
    norm_bwd_reduce_kernel(const float* __restrict__ part, float* dw, float* db, int dim, int n) {
  __shared__ float acc[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  griddep_wait();
  float v = 0.f;
  for (int i0 = warp; i0 < n; i0 += 32 * kNormReduceUnroll) {
    float t[kNormReduceUnroll];
#pragma unroll
    for (int k = 0; k < kNormReduceUnroll; ++k) {
      const int i = i0 + 32 * k;
      t[k] = i < n && c < 2 * dim ? part[static_cast<size_t>(i) * 2 * dim + c] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kNormReduceUnroll; ++k) v += t[k];
  }
  acc[warp][lane] = v;
  __syncthreads();
  // column `warp` of the CTA: its 32 sums by a warp reduction
  v = acc[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int cw = blockIdx.x * 32 + warp;
  if (lane == 0 && cw < 2 * dim) {
    if (cw < dim) {
      if (dw) dw[cw] = v;
    } else if (db) {
      db[cw - dim] = v;
    }
  }
}

}  // namespace dsa
