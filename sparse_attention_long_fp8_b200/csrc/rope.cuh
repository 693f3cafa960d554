// Rotary positions: each pair (a, b) of a head's rotated part turns by
// angle = pos * freq[i] and is scaled by the amplitude A:
//     a' = A (a cos - b sin),   b' = A (a sin + b cos)
// (the gradient is the transpose, the same with -angle). Pairs are the two
// halves' elements i and i + rot/2 (half layout) or neighbours 2i and 2i + 1
// (interleaved).
//
// The angle is formed in turns, pos * (freq / 2 pi), in fp64 and only its
// fraction goes on in fp32: at position 2^20 an fp32 product would be off by
// 2^-4 radians, the fraction is off by 2^-25 turns at any position. Every
// (token, pair) is evaluated once per CTA, into shared memory, and used by
// all heads of the CTA's rows.
//
// Bound: HBM, one read and one write per element (in place: of the rotated
// part only). Threads move 16-byte chunks when every address allows it (the
// rotated part's halves and the strides are multiples of a chunk), single
// elements otherwise; several rows are loaded before the first is turned.
#pragma once

#include <cuda_bf16.h>

#include "layout.cuh"

namespace dsa {

constexpr int kRopeMaxPairs = 128;
constexpr int kRopeThreads = 256;
constexpr int kRopeTableBytes = 32768;   // cos / sin of one CTA's tokens
constexpr int kRopeMaxTokens = 512;      // tokens of one CTA
// Rows a thread loads before it turns any: 64 bytes of 16-byte chunks.
template <int E, bool HALF>
constexpr int rope_unroll() { return HALF && E > 1 ? 2 : 4; }

// One rotation as the kernels take it (from dsa_rope_spec).
struct RopeAngles {
  int32_t begin, pairs;            // rotated dims [begin, begin + 2 pairs)
  int32_t half;                    // 1: pairs (i, i + pairs), 0: (2i, 2i + 1)
  float amplitude;
  double turns[kRopeMaxPairs];     // turns per position of each pair
};

// (A cos, A sin) of pos positions at `turns` turns per position. The fraction of
// a turn, in [-1/2, 1/2], is cut to the nearest quarter q and a rest of at most
// 1/8, x = 2 pi rest in [-pi/4, pi/4]; sin x and cos x by their Taylor series (the
// first terms left out are below x^11 / 11! = 2e-9 and x^10 / 10! = 3e-8), turned
// by q quarters. Off by at most about 2^-23 with the rounding of the fraction.
__device__ __forceinline__ float2 rope_cos_sin(double turns, int pos, float amplitude) {
  double t = static_cast<double>(pos) * turns;
  t -= rint(t);
  const float f = static_cast<float>(t);
  const float qf = rintf(4.0f * f);
  const float x = 6.28318531f * fmaf(-0.25f, qf, f);          // the difference is exact
  const float x2 = x * x;
  float s = fmaf(x2, 1.0f / 362880.0f, -1.0f / 5040.0f);
  s = fmaf(x2, s, 1.0f / 120.0f);
  s = fmaf(x2, s, -1.0f / 6.0f);
  s = fmaf(x2 * s, x, x);
  float c = fmaf(x2, 1.0f / 40320.0f, -1.0f / 720.0f);
  c = fmaf(x2, c, 1.0f / 24.0f);
  c = fmaf(x2, c, -0.5f);
  c = fmaf(x2, c, 1.0f);
  const int q = static_cast<int>(qf);
  const float cc = (q & 1) ? s : c, ss = (q & 1) ? c : s;
  return make_float2(amplitude * (((q + 1) & 2) ? -cc : cc), amplitude * ((q & 2) ? -ss : ss));
}

// n / d for n < 2^31 by a multiplication: m = ceil(2^(32 + sh) / d) with
// 2^sh >= d leaves n * m / 2^(32 + sh) within 1/d of n / d from above.
struct FastDiv {
  uint32_t d, m, sh;
  __host__ static FastDiv make(uint32_t d) {
    FastDiv f{d, 0, 0};
    while ((1ull << f.sh) < d) ++f.sh;
    const uint64_t full = ((1ull << (32 + f.sh)) + d - 1) / d;   // 2^32 <= full <= 2^33
    f.m = static_cast<uint32_t>(full - (1ull << 32));
    return f;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return static_cast<uint32_t>((static_cast<uint64_t>(__umulhi(n, m)) + n) >> sh);
  }
};

struct RopeParams {
  const void* x;
  void* out;
  int64_t xs[3], os[3];            // element strides of batch, token, head
  RowPos rp;
  uint32_t rows;                   // batch * tokens * heads
  int32_t heads, n_q, dim;
  int32_t rows_per_cta;
  int32_t copy;                    // out of place: the other dims are copied
  float sign;                      // -1: the transpose
  FastDiv by_heads, by_tokens;
  RopeAngles a;
};

template <class T>
__device__ __forceinline__ float rope_to_float(T v) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(v);
  else return v;
}
template <class T>
__device__ __forceinline__ T rope_from_float(float v) {
  if constexpr (sizeof(T) == 2) return __float2bfloat16_rn(v);
  else return v;
}

template <class T, int E>
struct alignas(E * sizeof(T)) RopeChunk {
  T v[E];
};

// E elements per chunk: 16 bytes of T, or 1. An item is E pairs (half: a chunk
// of each half) or max(E / 2, 1) pairs (interleaved: one chunk, or two
// neighbouring elements).
template <class T, int E, bool HALF>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kUnroll = rope_unroll<E, HALF>();
  constexpr int HP = HALF ? E : (E > 1 ? E / 2 : 1);
  using Chunk = RopeChunk<T, E>;
  extern __shared__ float2 cs[];                       // [tokens][pairs]
  __shared__ double turns[kRopeMaxPairs];
  __shared__ uint8_t live[kRopeMaxTokens];
  const int P = p.a.pairs;
  const uint32_t row0 = blockIdx.x * static_cast<uint32_t>(p.rows_per_cta);
  const uint32_t row1 = min(row0 + static_cast<uint32_t>(p.rows_per_cta), p.rows);
  const uint32_t tok0 = p.by_heads.div(row0);
  const int ntok = static_cast<int>(p.by_heads.div(row1 - 1) - tok0) + 1;
  for (int i = threadIdx.x; i < P; i += kRopeThreads) turns[i] = p.a.turns[i];
  __syncthreads();
  for (int i = threadIdx.x; i < ntok * P; i += kRopeThreads) {
    const int tk = i / P, pr = i - tk * P;
    const uint32_t tok = tok0 + tk;
    const uint32_t b = p.by_tokens.div(tok);
    const int pos = p.rp.pos(static_cast<int>(b), static_cast<int>(tok - b * p.n_q));
    if (pr == 0) live[tk] = pos >= 0;
    float2 v = rope_cos_sin(turns[pr], pos, p.a.amplitude);
    v.y *= p.sign;
    cs[i] = v;
  }
  __syncthreads();

  const T* x = static_cast<const T*>(p.x);
  T* out = static_cast<T*>(p.out);
  // Offsets of a row in x and out; -1 for a row past the end or a padding token.
  auto locate = [&](uint32_t row, int64_t& xo, int64_t& oo, int& tk) -> bool {
    if (row >= row1) return false;
    const uint32_t tok = p.by_heads.div(row);
    tk = static_cast<int>(tok - tok0);
    if (!live[tk]) return false;
    const int64_t h = row - tok * static_cast<uint32_t>(p.heads);
    const uint32_t b = p.by_tokens.div(tok);
    const int64_t t = tok - b * static_cast<uint32_t>(p.n_q);
    xo = b * p.xs[0] + t * p.xs[1] + h * p.xs[2];
    oo = b * p.os[0] + t * p.os[1] + h * p.os[2];
    return true;
  };

  {
    const int items = P / HP;
    const int lanes = kRopeThreads / items;            // rows side by side (items <= 128)
    const int item = threadIdx.x % items, ry = threadIdx.x / items;
    const int first = p.a.begin + (HALF ? item * E : 2 * item * HP);
    const int second = HALF ? first + P : first + 1;   // second: halves, or the scalar neighbour
    if (ry < lanes)
      for (uint32_t r = row0 + ry; r < row1; r += lanes * kUnroll) {
        Chunk u[kUnroll], w[kUnroll];
        int64_t oo[kUnroll];
        int tk[kUnroll];
        bool on[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
          int64_t xo;
          on[k] = locate(r + k * lanes, xo, oo[k], tk[k]);
          if (on[k]) {
            u[k] = *reinterpret_cast<const Chunk*>(x + xo + first);
            if constexpr (HALF || E == 1) w[k] = *reinterpret_cast<const Chunk*>(x + xo + second);
          }
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
          if (!on[k]) continue;
          const float2* t = cs + tk[k] * P + item * HP;
#pragma unroll
          for (int j = 0; j < HP; ++j) {
            const float2 v = t[j];
            if constexpr (HALF || E == 1) {
              const float a = rope_to_float(u[k].v[j]), b = rope_to_float(w[k].v[j]);
              u[k].v[j] = rope_from_float<T>(a * v.x - b * v.y);
              w[k].v[j] = rope_from_float<T>(a * v.y + b * v.x);
            } else {
              const float a = rope_to_float(u[k].v[2 * j]), b = rope_to_float(u[k].v[2 * j + 1]);
              u[k].v[2 * j] = rope_from_float<T>(a * v.x - b * v.y);
              u[k].v[2 * j + 1] = rope_from_float<T>(a * v.y + b * v.x);
            }
          }
          *reinterpret_cast<Chunk*>(out + oo[k] + first) = u[k];
          if constexpr (HALF || E == 1) *reinterpret_cast<Chunk*>(out + oo[k] + second) = w[k];
        }
      }
  }
  if (!p.copy) return;
  // the dims outside the rotated part, two chunks of a row per thread and step
  const int chunks = (p.dim - 2 * P) / E;
  if (chunks == 0) return;
  const int wide = min((chunks + 1) / 2, kRopeThreads);
  const int lanes = kRopeThreads / wide;
  const int c0 = threadIdx.x % wide, ry = threadIdx.x / wide;
  if (ry >= lanes) return;
  auto at = [&](int c) { return c * E < p.a.begin ? c * E : c * E + 2 * P; };
  for (int c = c0; c < chunks; c += 2 * wide) {
    const bool two = c + wide < chunks;
    const int e0 = at(c), e1 = at(two ? c + wide : c);
    for (uint32_t r = row0 + ry; r < row1; r += lanes * kUnroll) {
      Chunk u[kUnroll], w[kUnroll];
      int64_t oo[kUnroll];
      bool on[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        int64_t xo;
        int tk;
        on[k] = locate(r + k * lanes, xo, oo[k], tk);
        if (on[k]) {
          u[k] = *reinterpret_cast<const Chunk*>(x + xo + e0);
          w[k] = *reinterpret_cast<const Chunk*>(x + xo + e1);
        }
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
        if (on[k]) {
          *reinterpret_cast<Chunk*>(out + oo[k] + e0) = u[k];
          if (two) *reinterpret_cast<Chunk*>(out + oo[k] + e1) = w[k];
        }
    }
  }
}

}  // namespace dsa
