// Rotary positions: each pair (a, b) of a head's rotated part turns by
// angle = pos * freq[i] and is scaled by the amplitude A:
//     a' = A (a cos - b sin),   b' = A (a sin + b cos)
// (the gradient is the transpose, the same with -angle). Pairs are the two
// halves' elements i and i + rot/2 (half layout) or neighbours 2i and 2i + 1
// (interleaved).
//
// The angle is formed in turns, pos * (freq / 2 pi), in fp64 and reduced there to
// an eighth of a turn, which goes on in fp32. An fp32 product would be off by 2^-4
// radians at position 2^20. The reduced angle is off by 2^-25 for its rounding to
// fp32, and by 2^-52 of the whole angle for the roundings of freq / 2 pi and of the
// product: as much again at 2^27 radians, 2^-21 at the last position (freq = 1).
// Every (token, pair) is evaluated once per CTA, into shared memory, and used by
// all heads of the CTA's rows.
//
// Bound: HBM, one read and one write per element (in place: of the rotated
// part only): 16384 x 64 heads of 128 bf16 in 91.5 us, 5.87 TB/s. Threads move the
// longest chunks, up to 16 bytes, that every address allows (the rotated part's
// halves and the strides are multiples of one; interleaved pairs: 16 bytes or
// single elements); several rows are loaded before the first is turned. Rows at
// odd addresses are bound by sectors written in parts and by how little single
// elements keep on its way: 8192 x 64 rows of 133 bf16 in 89 us, 3.1 TB/s (116 us
// with every thread forming its rows' offsets and four rows on their way; 219 us
// with a thread per element, whose stores would be whole but whose loads double).
#pragma once

#include <cuda_bf16.h>

#include "layout.cuh"

namespace dsa {

constexpr int kRopeMaxPairs = 128;
constexpr int kRopeThreads = 256;
// Shared memory of one CTA: below 48 KB with both at their largest.
constexpr int kRopeTableBytes = 28672;   // cos / sin of its tokens
constexpr int kRopeMaxRows = 1024;       // its rows: offsets and token of each
constexpr int kRopeMaxTokens = 512;
// Chunks below 16 bytes: many per row, so a row's offsets are formed once.
constexpr bool rope_rows_in_smem(int bytes) { return bytes < 16; }
constexpr int rope_smem(int bytes, int rows, int tokens, int pairs) {
  return (rope_rows_in_smem(bytes) ? rows * 18 : 0) + tokens * pairs * 8;
}
// Rows a thread loads before it turns any: 64 bytes of 16-byte chunks, 4 rows of
// shorter chunks, 8 of single elements, which would else leave too little on its
// way (8192 x 64 rows of 133 bf16: 89 us, 92 with 4 rows, 127 with 12).
template <int E, int BYTES, bool HALF>
constexpr int rope_unroll() { return BYTES == 16 ? (HALF ? 2 : 4) : E == 1 ? 8 : 4; }

// One rotation as the kernels take it (from dsa_rope_spec).
struct RopeAngles {
  int32_t begin, pairs;            // rotated dims [begin, begin + 2 pairs)
  int32_t half;                    // 1: pairs (i, i + pairs), 0: (2i, 2i + 1)
  float amplitude;
  double turns[kRopeMaxPairs];     // turns per position of each pair
};

// (A cos, A sin) of pos positions at `turns` turns per position. The fraction of
// a turn, in [-1/2, 1/2], is cut to the nearest quarter q and a rest of at most
// 1/8, x = 2 pi rest in [-pi/4, pi/4], in fp64 up to the one rounding of x; sin x
// and cos x by their Taylor series (the first terms left out are below
// x^11 / 11! = 2e-9 and x^12 / 12! = 2e-10), turned by q quarters. Off by about an
// ulp of 1, and by the angle's own error far out (see the top). (With the fraction itself rounded to fp32 the angle is off by up to 1e-7: of
// 80 M appended E4M3 codes 148 instead of 121 miss the 64-bit formula's; a form with
// cos and sin rounded from 64 bits misses 128.)
__device__ __forceinline__ float2 rope_cos_sin(double turns, int pos, float amplitude) {
  double t = static_cast<double>(pos) * turns;
  t -= rint(t);
  const float qf = rintf(4.0f * static_cast<float>(t));
  const float x = static_cast<float>(fma(-0.25, static_cast<double>(qf), t) * 6.283185307179586);
  const float x2 = x * x;
  float s = fmaf(x2, 1.0f / 362880.0f, -1.0f / 5040.0f);
  s = fmaf(x2, s, 1.0f / 120.0f);
  s = fmaf(x2, s, -1.0f / 6.0f);
  s = fmaf(x2 * s, x, x);
  float c = fmaf(x2, -1.0f / 3628800.0f, 1.0f / 40320.0f);
  c = fmaf(x2, c, -1.0f / 720.0f);
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

// E elements per chunk. An item is E pairs (half: a chunk of each half) or
// max(E / 2, 1) pairs (interleaved: one chunk, or two neighbouring elements).
template <class T, int E, bool HALF>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kUnroll = rope_unroll<E, E * sizeof(T), HALF>();
  constexpr int HP = HALF ? E : (E > 1 ? E / 2 : 1);
  using Chunk = RopeChunk<T, E>;
  constexpr bool ROWS = rope_rows_in_smem(E * sizeof(T));
  extern __shared__ __align__(16) uint8_t rope_smem_base[];
  longlong2* const offs = reinterpret_cast<longlong2*>(rope_smem_base);       // [rows] x, out
  float2* const cs = reinterpret_cast<float2*>(offs + (ROWS ? p.rows_per_cta : 0));   // [tokens][pairs]
  __shared__ double turns[kRopeMaxPairs];
  __shared__ uint8_t live[kRopeMaxTokens];
  const int P = p.a.pairs;
  const uint32_t row0 = blockIdx.x * static_cast<uint32_t>(p.rows_per_cta);
  const int nrow = static_cast<int>(min(static_cast<uint32_t>(p.rows_per_cta), p.rows - row0));
  const uint32_t tok0 = p.by_heads.div(row0);
  const int ntok = static_cast<int>(p.by_heads.div(row0 + nrow - 1) - tok0) + 1;
  int16_t* const token = reinterpret_cast<int16_t*>(cs + ntok * P);           // [rows]
  auto place = [&](int i, int64_t& xo, int64_t& oo) -> int {
    const uint32_t row = row0 + i, tok = p.by_heads.div(row), b = p.by_tokens.div(tok);
    const int64_t h = row - tok * static_cast<uint32_t>(p.heads);
    const int64_t t = tok - b * static_cast<uint32_t>(p.n_q);
    xo = b * p.xs[0] + t * p.xs[1] + h * p.xs[2];
    oo = b * p.os[0] + t * p.os[1] + h * p.os[2];
    return static_cast<int>(tok - tok0);
  };
  for (int i = threadIdx.x; i < P; i += kRopeThreads) turns[i] = p.a.turns[i];
  if constexpr (ROWS)
    for (int i = threadIdx.x; i < nrow; i += kRopeThreads) {
      int64_t xo, oo;
      token[i] = static_cast<int16_t>(place(i, xo, oo));
      offs[i] = make_longlong2(xo, oo);
    }
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
  // Offset in x of the CTA's row i; false past the end and for padding. The
  // offset in out and the token are kept beside it, or (ROWS) looked up again.
  auto locate = [&](int i, int64_t& xo, int64_t& oo, int& tk) -> bool {
    if (i >= nrow) return false;
    if constexpr (ROWS) {
      if (!live[token[i]]) return false;
      xo = offs[i].x;
    } else {
      tk = static_cast<int>(p.by_heads.div(row0 + i) - tok0);
      if (!live[tk]) return false;
      place(i, xo, oo);
    }
    return true;
  };
  auto target = [&](int i, int64_t& oo, int& tk) {
    if constexpr (ROWS) {
      tk = token[i];
      oo = offs[i].y;
    }
  };

  {
    const int items = P / HP;
    const int lanes = kRopeThreads / items;            // rows side by side (items <= 128)
    const int item = threadIdx.x % items, ry = threadIdx.x / items;
    const int first = p.a.begin + (HALF ? item * E : 2 * item * HP);
    const int second = HALF ? first + P : first + 1;   // second: halves, or the scalar neighbour
    if (ry < lanes)
      for (int r = ry; r < nrow; r += lanes * kUnroll) {
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
          target(r + k * lanes, oo[k], tk[k]);
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
    for (int r = ry; r < nrow; r += lanes * kUnroll) {
      Chunk u[kUnroll], w[kUnroll];
      int64_t oo[kUnroll];
      int tk[kUnroll];
      bool on[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        int64_t xo;
        on[k] = locate(r + k * lanes, xo, oo[k], tk[k]);
        if (on[k]) {
          u[k] = *reinterpret_cast<const Chunk*>(x + xo + e0);
          w[k] = *reinterpret_cast<const Chunk*>(x + xo + e1);
        }
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
        if (on[k]) {
          target(r + k * lanes, oo[k], tk[k]);
          *reinterpret_cast<Chunk*>(out + oo[k] + e0) = u[k];
          if (two) *reinterpret_cast<Chunk*>(out + oo[k] + e1) = w[k];
        }
    }
  }
}

}  // namespace dsa
