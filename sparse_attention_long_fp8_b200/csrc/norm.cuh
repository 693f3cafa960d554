// Layer norm of rows of `dim` values and its gradient:
//   mean = sum x / dim, var = sum (x - mean)^2 / dim, rstd = 1 / sqrt(var + eps)
//   xh = (x - mean) rstd,   y = xh weight + bias
//   g = dy weight,  dx = rstd (g - sum(g) / dim - xh sum(g xh) / dim)
//   dweight = sum over rows of dy xh,   dbias = sum over rows of dy
// (the indexer's key norm, and its gradient from the warm-up loss's dk).
//
// Bound: HBM, each row read once and written once. A row stays in registers
// between its passes (two passes for the variance: sum of squares minus
// squared mean would cancel in fp32 when |mean| >> sigma). TPR threads share a
// row and hold 8 NV elements each. All arithmetic is fp32; bf16 only at loads and stores.
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

// One thread's elements of a row as loaded: 8 NV of them in chunks of 8
// (VEC, 16-byte loads) or one by one, TPR apart.
template <bool VEC, int TPR, int NV, int TYPE>
struct NormRow {
  static constexpr int EPT = 8 * NV;
  static constexpr int PER = VEC && TYPE == kRowBf16 ? 4 : 8;    // words per chunk
  uint32_t w[PER * NV];            // fp32 bits, or for VEC bf16 pairs in a chunk's first 4

  __device__ __forceinline__ static int elem(int lane, int j) {
    return VEC ? ((j >> 3) * TPR + lane) * 8 + (j & 7) : j * TPR + lane;
  }
  __device__ __forceinline__ static bool is_bf16(int flag) {
    return TYPE == kRowAny ? flag != 0 : TYPE == kRowBf16;
  }
  __device__ __forceinline__ void load(const void* base, long long off, int flag, int lane, int dim) {
    if constexpr (VEC) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int e = elem(lane, 8 * v);
        uint4 u = make_uint4(0, 0, 0, 0), t = u;
        if (is_bf16(flag)) {
          if (e < dim) u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + off + e);
        } else if (e < dim) {
          const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + off + e);
          u = s[0];
          t = s[1];
        }
        w[PER * v] = u.x; w[PER * v + 1] = u.y; w[PER * v + 2] = u.z; w[PER * v + 3] = u.w;
        if constexpr (PER == 8) {
          w[8 * v + 4] = t.x; w[8 * v + 5] = t.y; w[8 * v + 6] = t.z; w[8 * v + 7] = t.w;
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
        const uint32_t u = w[(j >> 3) * PER + ((j & 7) >> 1)];
        f[j] = __uint_as_float((j & 1) ? (u & 0xffff0000u) : (u << 16));
      }
    } else if constexpr (!VEC || TYPE != kRowBf16) {
#pragma unroll
      for (int j = 0; j < EPT; ++j) f[j] = __uint_as_float(w[j]);
    }
  }
};

// Stores one thread's elements of a row in the same arrangement.
template <bool VEC, int TPR, int NV>
__device__ __forceinline__ void norm_store(void* base, long long off, int bf16, int lane, int dim,
                                           const float (&f)[8 * NV]) {
  using Row = NormRow<VEC, TPR, NV, kRowAny>;
  if constexpr (VEC) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = Row::elem(lane, 8 * v);
      if (e >= dim) continue;
      if (bf16) {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(f[8 * v + 2 * j], f[8 * v + 2 * j + 1]);
          u[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + off + e) = make_uint4(u[0], u[1], u[2], u[3]);
      } else {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(base) + off + e);
        d[0] = make_float4(f[8 * v], f[8 * v + 1], f[8 * v + 2], f[8 * v + 3]);
        d[1] = make_float4(f[8 * v + 4], f[8 * v + 5], f[8 * v + 6], f[8 * v + 7]);
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
template <bool VEC, int TPR, int NV>
__device__ __forceinline__ void norm_weights(const float* w, float fill, int lane, int dim,
                                             float (&f)[8 * NV]) {
  using Row = NormRow<VEC, TPR, NV, kRowAny>;
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

// How a group keeps bytes in flight: narrow rows are loaded U at a time, wide
// ones one row ahead (PRE), the others rely on the other CTAs. MIN_CTAS per SM
// bounds the registers.
template <int TPR, int NV, int TYPE>
struct NormFlow {
  static constexpr int U = TPR <= 32 && NV == 1 ? (TYPE == kRowBf16 ? 4 : 2) : 1;
  static constexpr bool PRE = U == 1 && NV == 1;
  static constexpr bool KEEP = NV == 1;                  // weights stay in registers
  static constexpr int MIN_CTAS = TPR <= 32 ? 4 : (TPR == 128 ? 6 : (TPR == 512 ? 2 : 1));
};

template <bool VEC, int TPR, int NV, int TYPE>
__global__ void __launch_bounds__(norm_threads<TPR>(), NormFlow<TPR, NV, TYPE>::MIN_CTAS)
    norm_kernel(const NormParams p) {
  using Row = NormRow<VEC, TPR, NV, TYPE>;
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
    norm_weights<VEC, TPR, NV>(p.w, 1.f, lane, p.dim, w);
    norm_weights<VEC, TPR, NV>(p.b, 0.f, lane, p.dim, b);
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
      for (int j0 = 0; j0 < EPT; j0 += VEC ? 8 : 1) {
        float part = 0.f;
#pragma unroll
        for (int j = j0; j < j0 + (VEC ? 8 : 1); ++j) {
          x[j] -= mean;
          part = fmaf(x[j], x[j], part);
        }
        if (Row::elem(lane, j0) < p.dim) q += part;      // a chunk is inside the row or outside
      }
      const float var = norm_sum<TPR>(q, slots, buf) * inv;
      const float rstd = rsqrtf(var + p.eps);
      if (r < p.rows) {
        if constexpr (!F::KEEP) {
          norm_weights<VEC, TPR, NV>(p.w, 1.f, lane, p.dim, w);
          norm_weights<VEC, TPR, NV>(p.b, 0.f, lane, p.dim, b);
        }
#pragma unroll
        for (int j = 0; j < EPT; ++j) x[j] = fmaf(x[j] * rstd, w[j], b[j]);
        norm_store<VEC, TPR, NV>(p.y, r * p.ys, p.y_bf16, lane, p.dim, x);
        if (lane == 0) {
          if (p.mean) p.mean[r] = mean;
          if (p.rstd) p.rstd[r] = rstd;
        }
      }
    }
    if constexpr (F::PRE) raw[0] = next;
  }
}

// The same for the gradient, which loads two rows and keeps column sums.
template <int TPR, int NV>
struct NormBwdFlow {
  static constexpr int U = TPR <= 32 && NV == 1 ? 2 : 1;
  static constexpr bool PRE = U == 1 && NV == 1;
  static constexpr bool KEEP = NV == 1;
  static constexpr int MIN_CTAS = TPR <= 32 ? 2 : (TPR == 128 ? 4 : 1);
};

template <bool VEC, int TPR, int NV, int XT, int GT>
__global__ void __launch_bounds__(norm_threads<TPR>(), NormBwdFlow<TPR, NV>::MIN_CTAS)
    norm_bwd_kernel(const NormBwdParams p) {
  using RowX = NormRow<VEC, TPR, NV, XT>;
  using RowG = NormRow<VEC, TPR, NV, GT>;
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
  if constexpr (F::KEEP) norm_weights<VEC, TPR, NV>(p.w, 1.f, lane, p.dim, w);
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
      if constexpr (!F::KEEP) norm_weights<VEC, TPR, NV>(p.w, 1.f, lane, p.dim, w);
      float sg = 0.f, sgx = 0.f;
#pragma unroll
      for (int j = 0; j < EPT; ++j) {
        // past the row's end d is 0, and with it every product
        x[j] = (x[j] - mean[u]) * rstd[u];
        if (there) {
          aw[j] = fmaf(d[j], x[j], aw[j]);
          ab[j] += d[j];
        }
        d[j] *= w[j];
        sg += d[j];
        sgx = fmaf(d[j], x[j], sgx);
      }
      const float2 s = norm_sum2<TPR>(sg, sgx, slots, buf);
      const float mg = s.x * inv, mgx = s.y * inv;
      if (there) {
#pragma unroll
        for (int j = 0; j < EPT; ++j) d[j] = rstd[u] * (d[j] - mg - x[j] * mgx);
        norm_store<VEC, TPR, NV>(p.dx, r * p.dxs, p.dx_bf16, lane, p.dim, d);
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
