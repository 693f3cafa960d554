// New tokens into the caches, one launch: of token i of sequence b at position
// s = q_pos0[b] + i,
//   latent row    kv[s]    = the given row with its RoPE part turned by s;
//   indexer key   k_fp8[s], k_scale[s] = E4M3 row encoding (scale amax / 448)
//                 of RoPE(LayerNorm(k)).
// The norm, the rotation and the encoding of a key are one pass in fp32: the
// only roundings are the e4m3 codes and the bf16 of the rotated latent dims
// (the others are copied).
//
// A warp takes one token. Floor: HBM, 2 (d^I + D_qk) bytes read and d^I + 4 + 2
// D_qk written per token. What bounds it is issuing, 445 instructions per token
// and warp, in a chain of two loads, reductions and stores that 32 warps per SM
// hide in part: 19.7 us for 26 K tokens, 3.55 TB/s (without the key's part or
// without the latent row's it would be 14.9). Two tokens per warp, 16 lanes each:
// 21 us, the registers spill; the next token's loads issued ahead: 21 us; 40 or 48
// warps per SM: 23 us, spills; loads behind the test of n_new: 20.1 us.
// A decode step is bound by its launch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "layout.cuh"
#include "rope.cuh"

namespace dsa {

constexpr int kAppendWarps = 4;    // warps (tokens) per CTA

struct AppendParams {
  const __nv_bfloat16* k;          // [B, n_q, DI]
  const __nv_bfloat16* c;          // [B, n_q, DQK]
  const float* w;
  const float* b;
  const int32_t* q_pos0;
  const int32_t* n_new;
  uint8_t* k_fp8;
  float* k_scale;
  __nv_bfloat16* kv;
  KeyMap km;
  int32_t n_q, n_kv;
  uint32_t tokens;                 // B * n_q
  FastDiv by_tokens;               // n_q
  int32_t same_angles;             // ak and ac turn by the same angles
  int32_t key_vec;                 // the key's pairs lie in aligned groups of four dims
  float eps;
  RopeAngles ak, ac;               // of the key, of the latent row
};

// Token `tok` by one warp; key, cs: its scratch (DI values, pairs).
template <int DI, int DQK>
__device__ __forceinline__ void append_token(const AppendParams& p, uint32_t tok, int lane, float* key,
                                             float2* cs, const double* tk, const double* tc,
                                             const float (&w)[DI / 32], const float (&bias)[DI / 32]) {
  constexpr int PER = DI / 32;     // key values of a lane
  const uint32_t b = p.by_tokens.div(tok);
  const int i = static_cast<int>(tok - b * static_cast<uint32_t>(p.n_q));
  const int n_new = p.n_new ? p.n_new[b] : p.n_q;
  // past INT_MAX it turns negative, and is reported like any position past the cache
  const int pos = static_cast<int>(static_cast<uint32_t>(p.q_pos0 ? p.q_pos0[b] : 0) + static_cast<uint32_t>(i));
  // loads first, of a padded token's rows too: the key, and the latent row's 16-byte chunks
  const __nv_bfloat16* kr = p.k + static_cast<size_t>(tok) * DI + lane * PER;
  float v[PER];
  if constexpr (PER == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(kr);
    v[0] = __uint_as_float(u.x << 16);
    v[1] = __uint_as_float(u.x & 0xffff0000u);
    v[2] = __uint_as_float(u.y << 16);
    v[3] = __uint_as_float(u.y & 0xffff0000u);
  } else {
    v[0] = __bfloat162float(*kr);
  }
  constexpr int CHUNKS = DQK / 8, ROUNDS = (CHUNKS + 31) / 32;
  const __nv_bfloat16* cr = p.c + static_cast<size_t>(tok) * DQK;
  uint4 row[ROUNDS];
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r)
    if (r * 32 + lane < CHUNKS) row[r] = reinterpret_cast<const uint4*>(cr)[r * 32 + lane];
  if (i >= n_new) return;
  if (pos < 0 || pos >= p.n_kv) {  // past the cache: reported, nothing written
    if (lane == 0) raise_error(kErrBadInput);
    return;
  }
  const int64_t at = p.km.row(static_cast<int>(b), pos, p.n_kv);
  if (at < 0) return;              // page outside the pool (reported by the map)

  // ---- latent row: whole chunks outside the rotated part as they are
  const int c0 = p.ac.begin, c1 = c0 + 2 * p.ac.pairs;
  __nv_bfloat16* kvr = p.kv + at * DQK;
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int e = (r * 32 + lane) * 8;
    if (e >= DQK || (e >= c0 && e + 8 <= c1)) continue;
    if (e + 8 <= c0 || e >= c1) {
      reinterpret_cast<uint4*>(kvr)[r * 32 + lane] = row[r];
    } else {
      for (int j = e; j < e + 8; ++j)     // a chunk that the part's border cuts
        if (j < c0 || j >= c1) kvr[j] = cr[j];
    }
  }
  for (int j = lane; j < p.ac.pairs; j += 32) {
    const int ea = c0 + (p.ac.half ? j : 2 * j), eb = p.ac.half ? ea + p.ac.pairs : ea + 1;
    const float2 t = rope_cos_sin(tc[j], pos, p.ac.amplitude);
    if (p.same_angles) cs[j] = t;
    const float x = __bfloat162float(cr[ea]), y = __bfloat162float(cr[eb]);
    kvr[ea] = __float2bfloat16_rn(x * t.x - y * t.y);
    kvr[eb] = __float2bfloat16_rn(x * t.y + y * t.x);
  }

  // ---- indexer key: norm, rotation, encoding
  auto warp_sum = [](float s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
  };
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < PER; ++j) s += v[j];
  const float mean = warp_sum(s) * (1.0f / DI);
  s = 0.f;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    v[j] -= mean;
    s = fmaf(v[j], v[j], s);
  }
  const float rstd = rsqrtf(warp_sum(s) * (1.0f / DI) + p.eps);
#pragma unroll
  for (int j = 0; j < PER; ++j) v[j] = fmaf(v[j] * rstd, w[j], bias[j]);
  if (!p.same_angles)
    for (int j = lane; j < p.ak.pairs; j += 32) cs[j] = rope_cos_sin(tk[j], pos, p.ak.amplitude);
  const int P = p.ak.pairs;
  if (PER == 4 && p.key_vec) {
    // the lane's four dims are inside or outside together, and so are their pairs
    const int e = lane * 4 - p.ak.begin;
    const bool in = e >= 0 && e < 2 * P;
    if (p.ak.half) {
      *reinterpret_cast<float4*>(key + lane * 4) = make_float4(v[0], v[1], v[2], v[3]);
      __syncwarp();
      if (in) {
        const bool second = e >= P;
        const int pr = second ? e - P : e;
        const float4 o = *reinterpret_cast<const float4*>(key + p.ak.begin + (second ? e - P : e + P));
        const float4 t0 = *reinterpret_cast<const float4*>(cs + pr);
        const float4 t1 = *reinterpret_cast<const float4*>(cs + pr + 2);
        const float sg = second ? 1.f : -1.f;
        v[0] = fmaf(v[0], t0.x, sg * o.x * t0.y);
        v[1] = fmaf(v[1], t0.z, sg * o.y * t0.w);
        v[2] = fmaf(v[2], t1.x, sg * o.z * t1.y);
        v[3] = fmaf(v[3], t1.z, sg * o.w * t1.w);
      }
    } else {
      __syncwarp();
      if (in) {
        const float4 t = *reinterpret_cast<const float4*>(cs + (e >> 1));
        const float a = v[0], c = v[2];
        v[0] = a * t.x - v[1] * t.y;
        v[1] = a * t.y + v[1] * t.x;
        v[2] = c * t.z - v[3] * t.w;
        v[3] = c * t.w + v[3] * t.z;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < PER; ++j) key[lane * PER + j] = v[j];
    __syncwarp();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = lane * PER + j - p.ak.begin;      // within the rotated part
      if (e < 0 || e >= 2 * P) continue;
      const bool second = p.ak.half ? e >= P : (e & 1);
      const int pr = p.ak.half ? (second ? e - P : e) : e >> 1;
      const int other = p.ak.begin + (p.ak.half ? (second ? e - P : e + P) : e ^ 1);
      const float2 t = cs[pr];
      const float o = key[other];
      v[j] = second ? o * t.y + v[j] * t.x : v[j] * t.x - o * t.y;
    }
  }
  // the sizes as bit patterns: non-negative floats order like these, and NaN is above all
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
  const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, top));
  const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;     // 1 with NaN
  // v / scale to 2^-23 by one reciprocal, unless that would overflow
  const bool tiny = scale < 1e-37f;
  const float inv = __frcp_rn(tiny ? 1.f : scale);
  uint32_t packed = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    // saturates at 448, which is in reach by a rounding only; NaN stays NaN
    const float y = tiny ? __fdiv_rn(v[j], scale) : v[j] * inv;
    packed |= static_cast<uint32_t>(__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3)) << (8 * j);
  }
  uint8_t* codes = p.k_fp8 + at * DI + lane * PER;
  if constexpr (PER == 4) *reinterpret_cast<uint32_t*>(codes) = packed;
  else *codes = static_cast<uint8_t>(packed);
  if (lane == 0) p.k_scale[at] = scale;
}

template <int DI, int DQK>
__global__ void __launch_bounds__(32 * kAppendWarps, 8) append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ __align__(16) float skey[kAppendWarps][DI];
  __shared__ __align__(16) float2 scs[kAppendWarps][kRopeMaxPairs];
  __shared__ double tk[kRopeMaxPairs], tc[kRopeMaxPairs];    // turns per position
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int j = threadIdx.x; j < p.ak.pairs; j += 32 * kAppendWarps) tk[j] = p.ak.turns[j];
  for (int j = threadIdx.x; j < p.ac.pairs; j += 32 * kAppendWarps) tc[j] = p.ac.turns[j];
  constexpr int PER = DI / 32;
  float w[PER], bias[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    w[j] = p.w ? p.w[lane * PER + j] : 1.f;
    bias[j] = p.b ? p.b[lane * PER + j] : 0.f;
  }
  __syncthreads();
  // no barrier below spans warps
  for (uint32_t tok = blockIdx.x * kAppendWarps + warp; tok < p.tokens; tok += gridDim.x * kAppendWarps) {
    append_token<DI, DQK>(p, tok, lane, skey[warp], scs[warp], tk, tc, w, bias);
    __syncwarp();                  // the scratch has been read
  }
}

}  // namespace dsa
