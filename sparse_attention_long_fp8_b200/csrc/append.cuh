// New tokens into the caches, one launch: of token i of sequence b at position
// s = q_pos0[b] + i,
//   latent row    kv[s]    = the given row with its RoPE part turned by s;
//   indexer key   k_fp8[s], k_scale[s] = E4M3 row encoding (scale amax / 448)
//                 of RoPE(LayerNorm(k)).
// The norm, the rotation and the encoding of a key are one pass in fp32: the
// only roundings are the e4m3 codes and the bf16 of the rotated latent dims
// (the others are copied).
//
// A warp takes one token. Bound: HBM, 2 (d^I + D_qk) bytes read and
// d^I + 4 + 2 D_qk written per token; a decode step is bound by its launch.
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
  long long tokens;                // B * n_q
  float eps;
  RopeAngles ak, ac;               // of the key, of the latent row
};

// Token `tok` by one warp; key, cs: its scratch (DI values, DI / 2 pairs).
template <int DI, int DQK>
__device__ __forceinline__ void append_token(const AppendParams& p, long long tok, int lane, float* key,
                                             float2* cs, const double* tk, const double* tc) {
  constexpr int PER = DI / 32;     // key values of a lane
  const int b = static_cast<int>(tok / p.n_q), i = static_cast<int>(tok - static_cast<long long>(b) * p.n_q);
  if (p.n_new && i >= p.n_new[b]) return;
  const int pos = (p.q_pos0 ? p.q_pos0[b] : 0) + i;
  // loads first: the key, and the latent row's 16-byte chunks
  const __nv_bfloat16* kr = p.k + tok * DI + lane * PER;
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
  const __nv_bfloat16* cr = p.c + tok * DQK;
  uint4 row[ROUNDS];
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r)
    if (r * 32 + lane < CHUNKS) row[r] = reinterpret_cast<const uint4*>(cr)[r * 32 + lane];
  if (pos < 0 || pos >= p.n_kv) {  // past the cache: reported, nothing written
    if (lane == 0) raise_error(kErrBadInput);
    return;
  }
  const int64_t at = p.km.row(b, pos, p.n_kv);
  if (at < 0) return;              // page outside the pool (reported by the map)

  // ---- latent row: whole chunks outside the rotated part as they are
  const int c0 = p.ac.begin, c1 = c0 + 2 * p.ac.pairs;
  __nv_bfloat16* kvr = p.kv + at * DQK;
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int e = (r * 32 + lane) * 8;
    if (e >= DQK) continue;
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
  const float rstd = 1.0f / sqrtf(warp_sum(s) * (1.0f / DI) + p.eps);
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = lane * PER + j;
    v[j] = fmaf(v[j] * rstd, p.w ? p.w[e] : 1.f, p.b ? p.b[e] : 0.f);
    key[e] = v[j];
  }
  for (int j = lane; j < p.ak.pairs; j += 32)
    cs[j] = rope_cos_sin(tk[j], pos, p.ak.amplitude);
  __syncwarp();
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = lane * PER + j - p.ak.begin;        // within the rotated part
    if (e < 0 || e >= 2 * p.ak.pairs) continue;
    const bool second = p.ak.half ? e >= p.ak.pairs : (e & 1);
    const int pr = p.ak.half ? (second ? e - p.ak.pairs : e) : e >> 1;
    const int other = p.ak.begin + (p.ak.half ? (second ? e - p.ak.pairs : e + p.ak.pairs) : e ^ 1);
    const float2 t = cs[pr];
    const float o = key[other];
    v[j] = second ? o * t.y + v[j] * t.x : v[j] * t.x - o * t.y;
  }
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < PER; ++j) amax = fmaxf(amax, fabsf(v[j]));
  // non-negative floats order like their bit patterns
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
  uint32_t packed = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const float y = fminf(448.f, fmaxf(-448.f, __fdiv_rn(v[j], scale)));
    packed |= static_cast<uint32_t>(__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3)) << (8 * j);
  }
  uint8_t* codes = p.k_fp8 + at * DI + lane * PER;
  if constexpr (PER == 4) *reinterpret_cast<uint32_t*>(codes) = packed;
  else *codes = static_cast<uint8_t>(packed);
  if (lane == 0) p.k_scale[at] = scale;
}

template <int DI, int DQK>
__global__ void __launch_bounds__(32 * kAppendWarps) append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ float skey[kAppendWarps][DI];
  __shared__ float2 scs[kAppendWarps][DI / 2];
  __shared__ double tk[kRopeMaxPairs], tc[kRopeMaxPairs];    // turns per position
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int j = threadIdx.x; j < p.ak.pairs; j += 32 * kAppendWarps) tk[j] = p.ak.turns[j];
  for (int j = threadIdx.x; j < p.ac.pairs; j += 32 * kAppendWarps) tc[j] = p.ac.turns[j];
  __syncthreads();
  // no barrier below spans warps
  for (long long tok = static_cast<long long>(blockIdx.x) * kAppendWarps + warp; tok < p.tokens;
       tok += static_cast<long long>(gridDim.x) * kAppendWarps) 
{
    append_token<DI, DQK>(p, tok, lane, skey[warp], scs[warp], tk, tc);
    __syncwarp();                  // the scratch has been read
  }
}

}  // namespace dsa
