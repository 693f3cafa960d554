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
// row and hold 8 NV elements each; with NV = 1 the next row's loads are issued
// before this row is reduced (wider rows have more CTAs' loads in flight). All arithmetic is fp32; bf16 only at loads and stores.
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

// One thread's elements of a row as loaded: 8 NV of them in chunks of 8
// (VEC, 16-byte loads) or one by one, TPR apart.
template <bool VEC, int TPR, int NV>
struct NormRow {
  static constexpr int EPT = 8 * NV;
  uint32_t w[EPT];                 // fp32 bits, or for VEC bf16 pairs in the first half

  __device__ __forceinline__ static int elem(int lane, int j) {
    return VEC ? ((j >> 3) * TPR + lane) * 8 + (j & 7) : j * TPR + lane;
  }
  __device__ __forceinline__ void load(const void* base, long long off, int bf16, int lane, int dim) {
    if constexpr (VEC) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int e = elem(lane, 8 * v);
        if (bf16) {
          uint4 u = make_uint4(0, 0, 0, 0);
          if (e < dim) u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + off + e);
          w[8 * v] = u.x; w[8 * v + 1] = u.y; w[8 * v + 2] = u.z; w[8 * v + 3] = u.w;
        } else {
          uint4 u = make_uint4(0, 0, 0, 0), t = u;
          if (e < dim) {
            const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + off + e);
            u = s[0];
            t = s[1];
          }
          w[8 * v] = u.x; w[8 * v + 1] = u.y; w[8 * v + 2] = u.z; w[8 * v + 3] = u.w;
          w[8 * v + 4] = t.x; w[8 * v + 5] = t.y; w[8 * v + 6] = t.z; w[8 * v + 7] = t.w;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < EPT; ++j) {
        const int e = elem(lane, j);
        w[j] = 0u;
        if (e < dim)
          w[j] = bf16 ? static_cast<uint32_t>(static_cast<const uint16_t*>(base)[off + e]) << 16
                      : __float_as_uint(static_cast<const float*>(base)[off + e]);
      }
    }
  }
  // Elements past dim read as 0.
  __device__ __forceinline__ void get(float (&f)[EPT], int bf16) const {
    if (VEC && bf16) {
#pragma unroll
      for (int j = 0; j < EPT; ++j) {
        const uint32_t u = w[(j & ~7) + ((j & 7) >> 1)];
        f[j] = __uint_as_float((j & 1) ? (u & 0xffff0000u) : (u << 16));
      }
    } else {
#pragma unroll
      for (int j = 0; j < EPT; ++j) f[j] = __uint_as_float(w[j]);
    }
  }
  __device__ __forceinline__ static void store(void* base, long long off, int bf16, int lane, int dim,
                                               const float (&f)[EPT]) {
    if constexpr (VEC) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int e = elem(lane, 8 * v);
        if (e >= dim) continue;
        if (bf16) {
          uint32_t u[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[8 * v + 2 * j], f[8 * v + 2 * j + 1]);
            u[j] = *reinterpret_cast<const uint32_t*>(&h);
          }
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + off + e) =
              make_uint4(u[0], u[1], u[2], u[3]);
        } else {
          float4* d = reinterpret_cast<float4*>(static_cast<float*>(base) + off + e);
          d[0] = make_float4(f[8 * v], f[8 * v + 1], f[8 * v + 2], f[8 * v + 3]);
          d[1] = make_float4(f[8 * v + 4], f[8 * v + 5], f[8 * v + 6], f[8 * v + 7]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < EPT; ++j) {
        const int e = elem(lane, j);
        if (e >= dim) continue;
        if (bf16) static_cast<__nv_bfloat16*>(base)[off + e] = __float2bfloat16_rn(f[j]);
        else static_cast<float*>(base)[off + e] = f[j];
      }
    }
  }
};

// Sum of (a, b) over the TPR threads of a row. More than a warp: through
// shared memory, `buf` alternating between two sets of slots so that one
// barrier per sum suffices.
template <int TPR>
__device__ __forceinline__ float2 norm_sum(float a, float b, float2* slots, int& buf) {
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

// Threads per CTA: rows of up to a warp's threads share one.
template <int TPR>
constexpr int norm_threads() { return TPR <= 32 ? 256 : TPR; }

template <bool VEC, int TPR, int NV>
__global__ void __launch_bounds__(norm_threads<TPR>()) norm_kernel(const NormParams p) {
  using Row = NormRow<VEC, TPR, NV>;
  constexpr int EPT = Row::EPT, GROUPS = norm_threads<TPR>() / TPR;
  constexpr bool PRE = NV == 1;    // the next row and the weights in registers
  __shared__ float2 slots[TPR > 32 ? 2 * TPR / 32 : 1];
  int buf = 0;
  const int lane = threadIdx.x % TPR;
  const long long step = static_cast<long long>(gridDim.x) * GROUPS;
  // A whole warp stays in the loop (the sums use full-warp shuffles): a group
  // past the last row loads nothing and stores nothing.
  const long long base = static_cast<long long>(blockIdx.x) * GROUPS;
  const int g = threadIdx.x / TPR;
  Row cur, next;
  if (PRE && base + g < p.rows) cur.load(p.x, (base + g) * p.xs, p.x_bf16, lane, p.dim);
  auto weight = [&](int j) {
    const int e = Row::elem(lane, j);
    return p.w && e < p.dim ? __ldg(p.w + e) : 1.f;
  };
  auto bias = [&](int j) {
    const int e = Row::elem(lane, j);
    return p.b && e < p.dim ? __ldg(p.b + e) : 0.f;
  };
  float w[PRE ? EPT : 1], b[PRE ? EPT : 1];
  if constexpr (PRE) {
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
      w[j] = weight(j);
      b[j] = bias(j);
    }
  }
  const float inv = 1.0f / static_cast<float>(p.dim);
  for (long long r0 = base; r0 < p.rows; r0 += step) {
    const long long r = r0 + g;
    if constexpr (PRE) {
      if (r + step < p.rows) next.load(p.x, (r + step) * p.xs, p.x_bf16, lane, p.dim);
    } else {
      if (r < p.rows) cur.load(p.x, r * p.xs, p.x_bf16, lane, p.dim);
    }
    float x[EPT];
    cur.get(x, p.x_bf16);
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < EPT; ++j) s += x[j];
    const float mean = norm_sum<TPR>(s, 0.f, slots, buf).x * inv;
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
      x[j] -= mean;
      if (Row::elem(lane, j) < p.dim) q = fmaf(x[j], x[j], q);
    }
    const float var = norm_sum<TPR>(q, 0.f, slots, buf).x * inv;
    const float rstd = 1.0f / sqrtf(var + p.eps);
    if (r < p.rows) {
#pragma unroll
      for (int j = 0; j < EPT; ++j) {
        if constexpr (PRE) x[j] = fmaf(x[j] * rstd, w[j], b[j]);
        else x[j] = fmaf(x[j] * rstd, weight(j), bias(j));
      }
      Row::store(p.y, r * p.ys, p.y_bf16, lane, p.dim, x);
      if (lane == 0) {
        if (p.mean) p.mean[r] = mean;
        if (p.rstd) p.rstd[r] = rstd;
      }
    }
    if constexpr (PRE) cur = next;
  }
}

template <bool VEC, int TPR, int NV>
__global__ void __launch_bounds__(norm_threads<TPR>(), 1) norm_bwd_kernel(const NormBwdParams p) {
  using Row = NormRow<VEC, TPR, NV>;
  constexpr int EPT = Row::EPT, THREADS = norm_threads<TPR>(), GROUPS = THREADS / TPR;
  constexpr int COLS = TPR * EPT;                       // columns a group covers, >= dim
  constexpr bool PRE = NV == 1;    // the next row and the weights in registers
  __shared__ float2 slots[TPR > 32 ? 2 * TPR / 32 : 1];
  int buf = 0;
  const int lane = threadIdx.x % TPR;
  const long long step = static_cast<long long>(gridDim.x) * GROUPS;
  const long long base = static_cast<long long>(blockIdx.x) * GROUPS;
  const int g = threadIdx.x / TPR;
  Row cx, cy, nx, ny;
  float mean = 0.f, rstd = 0.f, nmean = 0.f, nrstd = 0.f;
  auto fetch = [&](long long r, Row& rx, Row& ry, float& m, float& s) {
    if (r < p.rows) {
      rx.load(p.x, r * p.xs, p.x_bf16, lane, p.dim);
      ry.load(p.dy, r * p.dys, p.dy_bf16, lane, p.dim);
      m = p.mean[r];
      s = p.rstd[r];
    }
  };
  if constexpr (PRE) fetch(base + g, cx, cy, mean, rstd);
  auto weight = [&](int j) {
    const int e = Row::elem(lane, j);
    return p.w && e < p.dim ? __ldg(p.w + e) : 1.f;
  };
  float w[PRE ? EPT : 1], aw[EPT], ab[EPT];
#pragma unroll
  for (int j = 0; j < EPT; ++j) {
    if constexpr (PRE) w[j] = weight(j);
    aw[j] = ab[j] = 0.f;
  }
  const float inv = 1.0f / static_cast<float>(p.dim);
  for (long long r0 = base; r0 < p.rows; r0 += step) {
    const long long r = r0 + g;
    const bool there = r < p.rows;
    if constexpr (PRE) fetch(r + step, nx, ny, nmean, nrstd);
    else fetch(r, cx, cy, mean, rstd);
    float x[EPT], d[EPT];
    cx.get(x, p.x_bf16);
    cy.get(d, p.dy_bf16);
    float sg = 0.f, sgx = 0.f;
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
      // past the row's end d is 0 and so are its products
      x[j] = Row::elem(lane, j) < p.dim ? (x[j] - mean) * rstd : 0.f;
      if (there) {
        aw[j] = fmaf(d[j], x[j], aw[j]);
        ab[j] += d[j];
      }
      if constexpr (PRE) d[j] *= w[j];
      else d[j] *= weight(j);
      sg += d[j];
      sgx = fmaf(d[j], x[j], sgx);
    }
    const float2 s = norm_sum<TPR>(sg, sgx, slots, buf);
    const float mg = s.x * inv, mgx = s.y * inv;
    if (there) {
#pragma unroll
      for (int j = 0; j < EPT; ++j) d[j] = rstd * (d[j] - mg - x[j] * mgx);
      Row::store(p.dx, r * p.dxs, p.dx_bf16, lane, p.dim, d);
    }
    if constexpr (PRE) {
      cx = nx;
      cy = ny;
      mean = nmean;
      rstd = nrstd;
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
        if constexpr (TPR == 16) v += __shfl_xor_sync(0xffffffffu, v, 16);
        acc[threadIdx.x >> 5][Row::elem(lane, j)] = v;
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
      const int e = Row::elem(lane, j);
      if (e < p.dim) {
        part[e] = aw[j];
        part[p.dim + e] = ab[j];
      }
    }
  }
}

// dweight, dbias: the n partial rows [2][dim] added in a fixed order, 32
// columns per CTA (of the 2 dim), 32 warps over the rows.
__global__ void __launch_bounds__(1024)
    norm_bwd_reduce_kernel(const float* __restrict__ part, float* dw, float* db, int dim, int n) {
  __shared__ float acc[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  griddep_wait();
  float v = 0.f;
  if (c < 2 * dim)
#pragma unroll 4
    for (int i = warp; i < n; i += 32) v += part[static_cast<size_t>(i) * 2 * dim + c];
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
