// Dense MQA attention of a few new tokens over every visible row of the latent
// cache (576 dims, V = the first 512; contiguous or paged):
//     s_k = scale q . kv[k],  out = sum_k softmax(s)_k kv[k, :512]
// with the online softmax: running maximum m and sum l per head, O rescaled
// when m grows.
//
// The work is cut along the caches. All query rows' 64-key blocks, row after
// row, form one line; CTA pair p takes blocks [p share, (p + 1) share) of it,
// whatever rows they belong to, so ragged lengths keep every SM equally busy
// and one long sequence spreads over the whole GPU. A row that lies inside one
// share is written directly; the (at most two) rows that a share's ends cut
// leave an fp32 partial O and LSE in the workspace, and dense_combine_kernel
// joins them in key order. Both kernels derive the cut from kv_len and the
// positions on the device: the host never needs the lengths.
//
// Inside a pair, CTA v owns value half v: it forms the complete logits and
// accumulates O for its 256 value dims (O 256 + S 64 + Q 192 TMEM columns =
// 512; an O of 512 dims would leave no column for S). Warp roles: 0 loads key
// blocks by TMA (nine 64-dim boxes per block, 128-byte swizzle, two stages,
// each released in two parts); 1 issues S = Q K^T; 2 issues O += P V; 4-11 run
// the softmax and the epilogue. S, P, Q and O are laid out as in
// sparse_attn_vh.cuh.
//
// Rows behind a sequence's last key may hold anything, NaN and infinities too:
// the producer overwrites them with zeros in shared memory before the block
// is used (0 * NaN in P V would reach the output), and their logits are
// masked by selection, not by adding.
#pragma once

#include "layout.cuh"
#include "sparse_attn_vh.cuh"

namespace dsa {

struct DenseParams {
  const __nv_bfloat16* q;      // [rows, H, 576]
  KeyMap km;
  RowPos rp;
  const int32_t* kv_len;
  void* out;                   // [rows, H, 512]
  float* lse;                  // [rows, H] or null
  float* part_o;               // [2 pairs][H][512]: slot 2 p: the row that share p begins
  float* part_lse;             // [2 pairs][H]       inside of, 2 p + 1: the row it ends inside of
  int32_t rows, n_q, n_kv, H;
  int32_t out_bf16;
  int32_t pairs;               // CTA pairs of the attention kernel
  int32_t min_share;           // blocks
  float scale_log2;

  // Keys that query row r sees, and the 64-key blocks they fill.
  __device__ __forceinline__ int visible(int r) const {
    const int b = r / n_q;
    const int last = min(rp.pos(b, r - b * n_q), n_kv - 1);     // no overflow at INT_MAX
    const int len = kv_len ? kv_len[b] : n_kv;
    return max(0, min(last + 1, len));
  }
  __device__ __forceinline__ int blocks(int r) const { return (visible(r) + 63) >> 6; }
  __device__ __forceinline__ long long share(long long total) const {
    return max(static_cast<long long>(min_share), (total + pairs - 1) / pairs);
  }
};

struct DenseTile : VhTile {
  static constexpr int THREADS = 384;           // TMA 0, S MMA 1, PV MMA 2, softmax 4-11
  static constexpr int AHEAD = 5;               // blocks whose lines are on their way into L2
  static constexpr int SM0 = 4;                 // first softmax warp
  static constexpr int NUM_BARS = 4 * STAGES + 8;
  static constexpr int OFF_SCAN = OFF_BAR + NUM_BARS * 8;      // [12] sums, then the start
  static constexpr int SMEM_BYTES = OFF_SCAN + 12 * 8 + 32;
  static_assert(SMEM_BYTES <= 232448, "shared memory");
};

// Sum of v over the CTA's threads; every thread calls it.
template <int WARPS>
__device__ __forceinline__ long long dense_block_sum(long long v, long long* scan) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();               // the previous sum has been read
  if ((threadIdx.x & 31) == 0) scan[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) v += scan[i];
  return v;
}

// A share's segments: blocks [blk, blk + n) of row `row`, one row after the other.
struct DenseSeg {
  int row, blk, n, vis;
  bool whole;                    // the row's blocks are all in this segment
};
struct DenseWalk {
  int row, blk;
  long long left;
  __device__ __forceinline__ bool next(const DenseParams& p, DenseSeg& s) {
    if (left <= 0) return false;
    int v = p.visible(row);
    while (v == 0) v = p.visible(++row);     // blocks are left, so such a row follows
    const int nb = (v + 63) >> 6;
    s.row = row;
    s.blk = blk;
    s.n = static_cast<int>(min(left, static_cast<long long>(nb - blk)));
    s.vis = v;
    s.whole = s.n == nb;
    left -= s.n;
    ++row;
    blk = 0;
    return true;
  }
};

// tmap_kv: the cache as bf16 rows of 576, box 64 dims x 64 rows. tmap_o and
// tmap_p: out and part_o as byte rows of 512 elements, box 128 bytes x H rows.
// All with the 128-byte swizzle.
__global__ void __launch_bounds__(384, 1)
    dense_attn_kernel(const __grid_constant__ CUtensorMap tmap_kv,
                      const __grid_constant__ CUtensorMap tmap_o,
                      const __grid_constant__ CUtensorMap tmap_p, const DenseParams p) {
  using T = DenseTile;
  constexpr int NK = T::NK;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  uint8_t* c_smem = smem + T::OFF_C;
  uint8_t* qs_smem = smem + T::OFF_QS;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + T::OFF_BAR);
  uint64_t* cx_full = bars;                      // [2] logit-only blocks of the stage landed
  uint64_t* cv_full = bars + T::STAGES;          // [2] V-half blocks landed
  uint64_t* cx_empty = bars + 2 * T::STAGES;     // [2] S of the stage's block finished
  uint64_t* cv_empty = bars + 3 * T::STAGES;     // [2] PV of the stage's block finished
  uint64_t* s_full = bars + 4 * T::STAGES;       // S tile written
  uint64_t* s_free = s_full + 1;                 // S tile loaded by all softmax warps
  uint64_t* p_full = s_full + 2;                 // [2] P tile of buffer b written
  uint64_t* pv_done = s_full + 4;                // [2] PV of buffer b finished (buffer free, O updated)
  uint64_t* q_ready = s_full + 6;                // Q of a segment in TMEM and shared memory
  uint64_t* tail = s_full + 7;                   // a row's last, partly filled block landed
  long long* scan = reinterpret_cast<long long*>(smem + T::OFF_SCAN);
  int* start = reinterpret_cast<int*>(scan + 12);               // row, block of the share's begin
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(start + 2);

  if ((smem_u32(smem_raw) & 1023u) != 0) {      // see VhTile::SMEM_BYTES: no slack to realign
    if (threadIdx.x == 0) raise_error(kErrInternal);
    return;
  }
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int pair = blockIdx.x >> 1, vh = blockIdx.x & 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < T::STAGES; ++s) {
      mbar_init(&cx_full[s], 1);
      mbar_init(&cv_full[s], 1);
      mbar_init(&cx_empty[s], 1);
      mbar_init(&cv_empty[s], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_free, T::SOFTMAX_WARPS);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&p_full[s], T::SOFTMAX_WARPS);
      mbar_init(&pv_done[s], 1);
    }
    mbar_init(q_ready, T::SOFTMAX_WARPS);
    mbar_init(tail, 1);
    fence_mbar_init();
    prefetch_tmap(&tmap_kv);
  }
  griddep_launch_dependents();                   // the join may be launched (it waits for this grid)
  // ---- the share: blocks [begin, end) of the line of all rows' blocks
  constexpr int kWarps = T::THREADS / 32;
  long long mine = 0;
  for (int r = threadIdx.x; r < p.rows; r += T::THREADS) mine += p.blocks(r);
  const long long total = dense_block_sum<kWarps>(mine, scan);
  const long long share = p.share(total);
  const long long begin = pair * share;
  DenseWalk walk{0, 0, max(0ll, min(total, begin + share) - begin)};
  if (walk.left == 0) return;                    // the same in every thread: no TMEM, no copies yet
  for (long long base = 0, r0 = 0; r0 < p.rows; r0 += T::THREADS) {
    // exclusive prefix of this thread's row within the tile of rows
    const int r = static_cast<int>(r0) + threadIdx.x;
    const int nb = r < p.rows ? p.blocks(r) : 0;
    long long incl = nb;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    long long before = base;
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) before += scan[i];
      base += scan[i];
    }
    const long long at = before + incl - nb;
    if (nb > 0 && at <= begin && begin < at + nb) {
      start[0] = r;
      start[1] = static_cast<int>(begin - at);
    }
    if (base > begin) break;                     // the same in every thread
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, T::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  walk.row = start[0];
  walk.blk = start[1];

  // Every role walks the same segments and counts their blocks alike: g is
  // the CTA's running block number, which picks the stage, the P buffer and
  // the barrier phases.
  if (warp == 0) {
    // ------------------------------------------------------------ key blocks by TMA
    uint32_t g = 0, tails = 0;
    uint32_t nx = 0, nv = 0;                     // loads issued on cx_full, on cv_full
    bool ok = true;
    DenseSeg w;
    while (ok && walk.next(p, w)) {
      const int b = w.row / p.n_q;
      // The pool row of a block's first key: a block of 64 lies inside one
      // page. A page outside the pool reads as zeros (the rows past the end).
      auto locate = [&](int blk) -> int {
        const int64_t r = p.km.row(b, blk * NK, p.n_kv);
        return static_cast<int>(r >= 0 ? r : p.km.pool_rows);
      };
      int at = locate(w.blk);
      for (int i = 0; i < w.n; ++i, ++g) {
        const int blk = w.blk + i;
        const int st = g % T::STAGES;
        const uint32_t ph = ((g / T::STAGES) & 1) ^ 1;
        const int valid = w.vis - blk * NK;
        const int y = at;
        if (i + 1 < w.n) at = locate(blk + 1);   // one block ahead
        uint8_t* dst = c_smem + st * T::STAGE_BYTES;
        if (i + T::AHEAD < w.n) {
          const int yp = locate(blk + T::AHEAD);
          if (lane < T::NDB && (lane & 1) == vh) tma_prefetch_2d(&tmap_kv, lane * 64, yp);
        }
        ok = mbar_wait(&cx_empty[st], ph);
        if (!ok) break;
        if (valid >= NK) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&cx_full[st], T::XDB * T::DB_BYTES);
#pragma unroll
            for (int t = 0; t < T::XDB; ++t) {
              const int db = t == 4 ? 8 : t + 4 * (1 - vh);
              tma_load_2d(dst + db * T::DB_BYTES, &tmap_kv, &cx_full[st], db * 64, y);
            }
          }
          ++nx;
          ok = mbar_wait(&cv_empty[st], ph);
          if (!ok) break;
          ++nv;
          if (lane == 0) {
            mbar_arrive_expect_tx(&cv_full[st], T::VDB * T::DB_BYTES);
#pragma unroll
            for (int t = 0; t < T::VDB; ++t) {
              const int db = 4 * vh + t;
              tma_load_2d(dst + db * T::DB_BYTES, &tmap_kv, &cv_full[st], db * 64, y);
            }
          }
        } else {
          ok = mbar_wait(&cv_empty[st], ph);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(tail, T::NDB * T::DB_BYTES);
            for (int db = 0; db < T::NDB; ++db)
              tma_load_2d(dst + db * T::DB_BYTES, &tmap_kv, tail, db * 64, y);
          }
          ok = mbar_wait(tail, tails & 1);
          if (!ok) {
            mbar_wait(tail, tails & 1);          // in flight: once more before the CTA ends
            break;
          }
          ++tails;
          ++nx;
          ++nv;
          // rows valid .. 63 of every box become zeros
          const int words = (NK - valid) * 8;    // 16-byte words per box
          for (int db = 0; db < T::NDB; ++db) {
            const uint32_t a = smem_u32(dst) + db * T::DB_BYTES + valid * 128;
            for (int k = lane; k < words; k += 32) sts_v4(a + k * 16, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&cx_full[st]);
            mbar_arrive(&cv_full[st]);
          }
        }
        __syncwarp();
      }
    }
    // A wait that ran out leaves copies in flight: they end before the CTA does
    // (the last two uses of each barrier).
    if (!ok)
      for (uint32_t d = 1; d <= 2; ++d) {
        if (nx >= d) mbar_wait(&cx_full[(nx - d) % T::STAGES], ((nx - d) / T::STAGES) & 1);
        if (nv >= d) mbar_wait(&cv_full[(nv - d) % T::STAGES], ((nv - d) / T::STAGES) & 1);
      }
  } else if (warp == 1) {
    // ------------------------------------------------------------ S = Q K^T issuer
    // One elected lane runs the whole loop (see elect_one). Descriptors are
    // formed once: adding (byte offset >> 4) moves the start address.
    if (elect_one()) {
      constexpr uint32_t idesc_s = umma_idesc(128, NK, 1u, 1u, 0u, 0u);
      const uint64_t c_desc0 = umma_desc(smem_u32(c_smem), 16, 1024, 2);
      const uint64_t q_desc0 = umma_desc(smem_u32(qs_smem), 16, 1024, 2);
      const uint32_t d_s = tmem_base + T::COL_S;
      const uint32_t x_shift = static_cast<uint32_t>(4 * (1 - vh) * T::DB_BYTES) >> 4;
      const uint32_t v_shift = static_cast<uint32_t>(4 * vh * T::DB_BYTES) >> 4;
      uint32_t g = 0, k = 0;
      bool ok = true;
      DenseSeg w;
      while (ok && walk.next(p, w)) {
        ok = mbar_wait(q_ready, k & 1);
        ++k;
        tc_fence_after();
        for (int i = 0; i < w.n && ok; ++i, ++g) {
          const int st = g % T::STAGES;
          const uint32_t ph = (g / T::STAGES) & 1;
          // the S buffer is free once every softmax warp has loaded S(g - 1)
          ok = (g == 0 || mbar_wait(s_free, (g - 1) & 1)) && mbar_wait(&cx_full[st], ph);
          if (!ok) break;
          tc_fence_after();
          const uint64_t cd = c_desc0 + static_cast<uint32_t>(st * (T::STAGE_BYTES >> 4));
#pragma unroll
          for (int t = 0; t < T::XDB; ++t)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint32_t off = (t < 4 ? t * T::DB_BYTES : 8 * T::DB_BYTES) + kk * 32;
              const uint64_t bd = cd + (t < 4 ? x_shift : 0u) + (off >> 4);
              umma_bf16_ts(d_s, tmem_base + T::COL_Q + t * 32 + kk * 8, bd, idesc_s,
                           (t | kk) ? 1u : 0u);
            }
          umma_commit(&cx_empty[st]);
          ok = mbar_wait(&cv_full[st], ph);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t bd = cd + v_shift + ((kk * 32) >> 4);
            umma_bf16_ts(d_s, tmem_base + T::COL_Q + T::XDB * 32 + kk * 8, bd, idesc_s, 1u);
          }
#pragma unroll
          for (int uq = 0; uq < T::QSB; ++uq)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint64_t ad = q_desc0 + ((uq * T::M * 128 + kk * 32) >> 4);
              const uint64_t bd = cd + v_shift + (((uq + 1) * T::DB_BYTES + kk * 32) >> 4);
              umma_bf16_ss(d_s, ad, bd, idesc_s, 1u);
            }
          umma_commit(s_full);
        }
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ O += P V issuer
    // P(g) exists only after S(g) was read, so when PV(g) completes both
    // readers of the V-half blocks are done and P buffer g & 1 is free. The
    // first PV of a segment overwrites O: the softmax warps write its P only
    // after they have read out the previous segment's O.
    if (elect_one()) {
      constexpr uint32_t idesc_pv = umma_idesc(128, T::VH, 1u, 1u, 0u, 1u);
      const uint64_t p_desc0 = umma_desc(smem_u32(smem + T::OFF_P), 16, 1024, 2);
      const uint64_t v_desc0 = umma_desc(smem_u32(c_smem) + 4 * vh * T::DB_BYTES, T::DB_BYTES, 1024, 2);
      uint32_t g = 0;
      bool ok = true;
      DenseSeg w;
      while (ok && walk.next(p, w)) {
        for (int i = 0; i < w.n; ++i, ++g) {
          const int st = g % T::STAGES;
          if (!(ok = mbar_wait(&p_full[g & 1], (g >> 1) & 1))) break;
          tc_fence_after();
          const uint64_t vd = v_desc0 + static_cast<uint32_t>(st * (T::STAGE_BYTES >> 4));
          const uint64_t pd = p_desc0 + static_cast<uint32_t>((g & 1) * (T::P_BYTES >> 4));
#pragma unroll
          for (int kk = 0; kk < NK / 16; ++kk)
            umma_bf16_ss(tmem_base + T::COL_O, pd + ((kk * 32) >> 4), vd + ((kk * 2048) >> 4),
                         idesc_pv, (i > 0 || kk > 0) ? 1u : 0u);
          umma_commit(&cv_empty[st]);
          umma_commit(&pv_done[g & 1]);
        }
      }
    }
    __syncwarp();
  } else if (warp >= T::SM0) {
    // ------------------------------------------------------------ softmax / epilogue
    const int quarter = warp & 3;
    const int half = (warp - T::SM0) >> 2;                   // which 32 keys of a block
    const int h = quarter * 32 + lane;                       // head row = TMEM lane
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t pair_bar = 1u + static_cast<uint32_t>(quarter);   // the quarter's two warps
    float* red = reinterpret_cast<float*>(smem + T::OFF_RED);   // [parity][half][128]
    const int stid = threadIdx.x - T::SM0 * 32;              // 0..255 over the softmax warps
    constexpr uint32_t kAllBar = 5u;                         // named barrier of the 8 warps
    constexpr uint32_t kAllThreads = 32u * T::SOFTMAX_WARPS;

    // Q of a row, three 64-dim blocks at a time through the Q area of shared
    // memory: twice as staging for the six TMEM blocks, once for the three
    // that stay there.
    auto copy_q3 = [&](int row, int first, bool tmem_part) {
      const __nv_bfloat16* qrow = p.q + static_cast<size_t>(row) * p.H * T::DQK;
      const int r4 = stid >> 3, ch = stid & 7;
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const int db = tmem_part ? vh_tblock(first + j, vh) : vh_sblock(first + j, vh);
#pragma unroll
        for (int it = 0; it < T::M / 32; ++it) {
          const int r = it * 32 + r4;
          const __nv_bfloat16* src = qrow + static_cast<size_t>(min(r, p.H - 1)) * T::DQK + db * 64 + ch * 8;
          const uint32_t dst = smem_u32(qs_smem) + j * (T::M * 128) + (r >> 3) * 1024 + (r & 7) * 128 +
                               ((ch ^ (r & 7)) << 4);
          cp_async_16(dst, src, r < p.H ? 16u : 0u);
        }
      }
      cp_async_wait_all();
    };
    auto load_q = [&](int row) {
#pragma unroll 1
      for (int round = 0; round < 2; ++round) {
        copy_q3(row, 3 * round, true);
        named_bar_sync(kAllBar, kAllThreads);
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          const uint32_t rowp = smem_u32(qs_smem) + j * (T::M * 128) + (h >> 3) * 1024 + (h & 7) * 128;
          uint32_t v[16];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 x = lds_v4(rowp + (((4 * half + c) ^ (h & 7)) << 4));
            v[4 * c] = x.x; v[4 * c + 1] = x.y; v[4 * c + 2] = x.z; v[4 * c + 3] = x.w;
          }
          tmem_st16(tmem_base + lane_addr + T::COL_Q + (2 * (3 * round + j) + half) * 16, v);
        }
        named_bar_sync(kAllBar, kAllThreads);      // staging read before it is overwritten
      }
      copy_q3(row, 0, false);
      fence_proxy_async_smem();
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
    };

    uint32_t sr[32];
    float z[32];
    const uint32_t p_row = smem_u32(smem + T::OFF_P) + (h >> 3) * 1024 + (h & 7) * 128;
    uint32_t g = 0;
    bool ok = true;
    DenseSeg w;
    bool more = walk.next(p, w);
    if (more) load_q(w.row);
    while (more && ok) {
      float m_used = -INFINITY;   // running max (log2 domain) the P values are relative to
      float l = 0.f;              // this warp's share of the sum of the fp32 p (LSE)
      float l_mma = 0.f;          // ... of the bf16-rounded p the PV MMA used (normalises O)
      for (int i = 0; i < w.n; ++i, ++g) {
        // ---- logits of this warp's 32 keys; the S buffer is released at
        // once. A failed wait does not leave the loop before the partner
        // exchange: the quarter's two warps leave together.
        const int valid = w.vis - (w.blk + i) * NK - half * 32;   // of this warp's 32 keys
        if (ok) ok = mbar_wait(s_full, g & 1);
        tc_fence_after();
        tmem_ld32(tmem_base + lane_addr + T::COL_S + half * 32, sr);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free);
        // ---- block max over the 64 keys, shared with the partner warp (over
        // the unscaled logits: the scale is not negative, see the host's check)
#pragma unroll
        for (int j = 0; j < 32; ++j) z[j] = __uint_as_float(sr[j]);
        if (valid < 32) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j >= valid) z[j] = -INFINITY;
        }
        float mx[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          mx[r] = fmaxf(fmaxf(fmaxf(z[r], z[r + 4]), fmaxf(z[r + 8], z[r + 12])),
                        fmaxf(fmaxf(z[r + 16], z[r + 20]), fmaxf(z[r + 24], z[r + 28])));
        const float hmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
        float* red_i = red + (g & 1) * (2 * T::M);
        red_i[half * T::M + h] = hmax;
        if (!named_bar_and(pair_bar, 64u, ok)) {
          ok = false;
          break;
        }
        const float bmax = fmaxf(hmax, red_i[(half ^ 1) * T::M + h]);
        // ---- online softmax. Rescaling O needs PV(g - 1) finished; writing
        // P buffer g & 1 needs PV(g - 2) finished.
        const bool grow = bmax > m_used + 8.0f;
        const float m_new = grow ? bmax : m_used;
        if (i > 0 && __any_sync(0xffffffffu, grow)) {
          if (ok) ok = mbar_wait(&pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
          tc_fence_after();
          const float alpha = grow ? ex2_approx(m_used - m_new) : 1.0f;
#pragma unroll 1
          for (int c = half * (T::VH / 2); c < (half + 1) * (T::VH / 2) && ok; c += 16) {
            uint32_t o[16];
            tmem_ld16(tmem_base + lane_addr + T::COL_O + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
            tmem_st16(tmem_base + lane_addr + T::COL_O + c, o);
          }
          tmem_wait_st();
          l *= alpha;
          l_mma *= alpha;
        } else if (g > 1 && ok) {
          ok = mbar_wait(&pv_done[g & 1], ((g >> 1) & 1) ^ 1);
        }
        m_used = m_new;
        uint32_t pk[16];
        float ls[4] = {0.f, 0.f, 0.f, 0.f}, lm[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float p0 = ex2_approx(fmaf(z[2 * j], p.scale_log2, -m_used));
          const float p1 = ex2_approx(fmaf(z[2 * j + 1], p.scale_log2, -m_used));
          const __nv_bfloat162 pb2 = __floats2bfloat162_rn(p0, p1);
          ls[j & 3] += p0 + p1;
          lm[j & 3] += __low2float(pb2) + __high2float(pb2);
          pk[j] = *reinterpret_cast<const uint32_t*>(&pb2);
        }
        float lsum = (ls[0] + ls[1]) + (ls[2] + ls[3]);
        float lsum_mma = (lm[0] + lm[1]) + (lm[2] + lm[3]);
        if (m_used == -INFINITY) {
#pragma unroll
          for (int j = 0; j < 16; ++j) pk[j] = 0u;
          lsum = lsum_mma = hmax != hmax ? hmax : 0.f;    // all -inf, or NaN among them
        }
        l += lsum;
        l_mma += lsum_mma;
        const uint32_t pb = p_row + (g & 1) * T::P_BYTES;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          sts_v4(pb + (((4 * half + c) ^ (h & 7)) << 4), pk[4 * c], pk[4 * c + 1], pk[4 * c + 2],
                 pk[4 * c + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[g & 1]);
      }
      // all softmax warps go on, or stop, together
      if (!named_bar_and(kAllBar, kAllThreads, ok)) {
        ok = false;
        break;
      }
      // ---- the next segment's Q: this segment's S MMAs have all completed
      // (the last S was loaded above), so its logits may start during this
      // epilogue
      const DenseSeg done = w;
      more = walk.next(p, w);
      if (more) load_q(w.row);
      // ---- epilogue: O of the segment, once its last PV has finished
      ok = mbar_wait(&pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
      tc_fence_after();
      red[half * T::M + h] = l;
      red[(2 + half) * T::M + h] = l_mma;
      named_bar_sync(pair_bar, 64u);
      const float l_o = red[(half ^ 1) * T::M + h];
      const float lm_o = red[(2 + (half ^ 1)) * T::M + h];
      const bool pv_ok = ok;
      named_bar_sync(pair_bar, 64u);
      const float l_all = half == 0 ? l + l_o : l_o + l;
      const float lm_all = half == 0 ? l_mma + lm_o : lm_o + l_mma;
      // O / sum(rounded p) is an exact convex combination of the V rows; the
      // LSE keeps the unrounded sum.
      const bool has = pv_ok && l_all != 0.f && lm_all != 0.f;   // true for NaN
      const float inv_l = has ? 1.0f / lm_all : 0.f;
      const uint32_t keep = has ? 0xffffffffu : 0u;
      const float lse_v = has ? (m_used + log2f(l_all)) * 0.69314718055994531f : -INFINITY;
      // O leaves by TMA stores of 128-byte-wide column slices staged in the
      // swizzled layout the store reads: one slice per round, alternating
      // between the two P buffers (free: the last PV has finished); after the
      // last segment all slices at once through the stage area.
      const bool direct = done.whole;
      const int slot = 2 * pair + (done.blk > 0 ? 0 : 1);
      const bool bf16_out = direct && p.out_bf16;
      const int esz = bf16_out ? 2 : 4;
      const int slice_cols = 128 / esz;
      const int n_slices = T::VH / slice_cols;
      const int per_round = more ? 1 : n_slices;
      const int32_t y_row = (direct ? done.row : slot) * p.H;
#pragma unroll 1
      for (int s0 = 0, rnd = 0; s0 < n_slices; s0 += per_round, ++rnd) {
        const uint32_t stage =
            more ? smem_u32(smem + T::OFF_P) + (rnd & 1) * T::P_BYTES : smem_u32(c_smem);
        if (more && stid == 0) bulk_wait_read<1>();     // the store of round rnd - 2 has read it
        named_bar_sync(kAllBar, kAllThreads);
        for (int sl = s0; sl < s0 + per_round; ++sl) {
          const uint32_t srow = stage + (sl - s0) * (T::M * 128) + h * 128;
#pragma unroll 1
          for (int c = half * (slice_cols / 2); c < (half + 1) * (slice_cols / 2); c += 16) {
            uint32_t o[16];
            tmem_ld16(tmem_base + lane_addr + T::COL_O + sl * slice_cols + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j] & keep) * inv_l);
            const int cc = c * esz / 16;                   // its first 16-byte chunk in the row
            if (bf16_out) {
              uint32_t pkd[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const __nv_bfloat162 v =
                    __floats2bfloat162_rn(__uint_as_float(o[2 * j]), __uint_as_float(o[2 * j + 1]));
                pkd[j] = *reinterpret_cast<const uint32_t*>(&v);
              }
#pragma unroll
              for (int q2 = 0; q2 < 2; ++q2)
                sts_v4(srow + (((cc + q2) ^ (h & 7)) << 4), pkd[4 * q2], pkd[4 * q2 + 1],
                       pkd[4 * q2 + 2], pkd[4 * q2 + 3]);
            } else {
#pragma unroll
              for (int q2 = 0; q2 < 4; ++q2)
                sts_v4(srow + (((cc + q2) ^ (h & 7)) << 4), o[4 * q2], o[4 * q2 + 1], o[4 * q2 + 2],
                       o[4 * q2 + 3]);
            }
          }
        }
        fence_proxy_async_smem();
        named_bar_sync(kAllBar, kAllThreads);
        if (stid == 0) {
          const void* map = direct ? static_cast<const void*>(&tmap_o) : static_cast<const void*>(&tmap_p);
          for (int sl = s0; sl < s0 + per_round; ++sl)
            tma_store_2d(map, stage + (sl - s0) * (T::M * 128), (vh * T::VH + sl * slice_cols) * esz, y_row);
          bulk_commit();
        }
      }
      // every staged byte read before the next segment writes P
      if (stid == 0) bulk_wait_read<0>();
      named_bar_sync(kAllBar, kAllThreads);
      if (vh == 0 && half == 0 && h < p.H) {
        if (!direct) p.part_lse[static_cast<size_t>(slot) * p.H + h] = lse_v;
        else if (p.lse) p.lse[static_cast<size_t>(done.row) * p.H + h] = lse_v;
      }
      ok = named_bar_and(kAllBar, kAllThreads, ok);
    }
  }

  if (threadIdx.x == T::SM0 * 32) bulk_wait<0>();   // the output stores have completed
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, T::TMEM_COLS);
  }
}

// Joins the partials of the rows that more than one share holds, in key order,
// and writes the rows that see no key (out = 0, LSE = -inf). G warps per (row,
// head) take every G-th partial, a lane 16 of the 512 value dims; their sums
// meet in shared memory. The shares are derived as the attention kernel derives
// them. Few rows may have a partial from every pair (one long sequence: 74 of
// them), so they get more warps: 36 -> 8 us with G = 8 against one thread
// walking all partials.
template <int G>
__global__ void __launch_bounds__(256) dense_combine_kernel(const DenseParams p) {
  constexpr int HEADS = 8 / G;                   // heads per CTA
  __shared__ longlong2 scan[8];
  __shared__ float4 acc_s[G > 1 ? 8 : 1][4][32];
  __shared__ float sum_s[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x;
  const int h = blockIdx.y * HEADS + warp / G, sub = warp % G;
  long long total = 0, first = 0;                // blocks of all rows, of the rows ahead
  for (int r = threadIdx.x; r < p.rows; r += 256) {
    const int nb = p.blocks(r);
    total += nb;
    if (r < row) first += nb;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    first += __shfl_xor_sync(0xffffffffu, first, o);
  }
  if (lane == 0) scan[warp] = make_longlong2(total, first);
  __syncthreads();
  total = first = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    total += scan[i].x;
    first += scan[i].y;
  }
  const int nb = p.blocks(row);
  const long long share = p.share(total);
  const int p0 = static_cast<int>(first / share);
  const int np = nb > 0 ? static_cast<int>((first + nb - 1) / share) - p0 + 1 : 0;
  griddep_wait();                                // every CTA: this grid ends after the attention
  if (np == 1) return;                           // written by the attention kernel
  // the row begins in share p0 (slot 2 p0 + 1); the others begin inside of it
  auto slot = [&](int i) {
    return (static_cast<size_t>(2 * (p0 + i)) + (i == 0 ? 1 : 0)) * p.H + h;
  };
  const bool there = h < p.H;
  float m = -INFINITY;
  if (there)
    for (int i = lane; i < np; i += 32) m = fmaxf(m, p.part_lse[slot(i)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float4 acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  if (there) {
#pragma unroll 2
    for (int i = sub; i < np; i += G) {
      const size_t at = slot(i);
      const float ls = p.part_lse[at];
      const float wgt = ls == -INFINITY ? 0.f : __expf(ls - m);
      sum += wgt;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(p.part_o + at * 512 + j * 128 + lane * 4);
        acc[j].x = fmaf(wgt, v.x, acc[j].x);
        acc[j].y = fmaf(wgt, v.y, acc[j].y);
        acc[j].z = fmaf(wgt, v.z, acc[j].z);
        acc[j].w = fmaf(wgt, v.w, acc[j].w);
      }
    }
  }
  if constexpr (G > 1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) acc_s[warp][j][lane] = acc[j];
    if (lane == 0) sum_s[warp] = sum;
    __syncthreads();
    if (sub != 0) return;
#pragma unroll
    for (int k = 1; k < G; ++k) {
      sum += sum_s[warp + k];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 v = acc_s[warp + k][j][lane];
        acc[j].x += v.x; acc[j].y += v.y; acc[j].z += v.z; acc[j].w += v.w;
      }
    }
  }
  if (!there) return;
  const float inv = sum != 0.f ? 1.0f / sum : 0.f;     // NaN goes through
  const size_t o = (static_cast<size_t>(row) * p.H + h) * 512;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 v = make_float4(acc[j].x * inv, acc[j].y * inv, acc[j].z * inv, acc[j].w * inv);
    const size_t at = o + j * 128 + lane * 4;
    if (p.out_bf16) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = v;
    }
  }
  if (lane == 0 && p.lse)
    p.lse[static_cast<size_t>(row) * p.H + h] = sum != 0.f ? m + logf(sum) : -INFINITY;
}

}  // namespace dsa
