// Dense MQA attention of a few new tokens over every visible row of the latent
// cache (576 dims, V = the first 512; contiguous or paged):
//     s_k = scale q . kv[k],  out = sum_k softmax(s)_k kv[k, :512]
// with the online softmax: running maximum m and sum l per head, O rescaled
// when m grows.
//
// The work is cut along the caches. All query rows' 128-key blocks, row after
// row, form one line; CTA pair p takes blocks [p share, (p + 1) share) of it,
// whatever rows they belong to, so ragged lengths keep every SM equally busy
// and one long sequence spreads over the whole GPU. A row that lies inside one
// share is written directly; the (at most two) rows that a share's ends cut
// leave an fp32 partial O and LSE in the workspace, and dense_combine_kernel
// joins them in key order. Both kernels derive the cut from kv_len and the
// positions on the device: the host never needs the lengths.
//
// The two CTAs of a pair (a cluster, two SMs) work on one block together with
// tcgen05 over both (cta_group::2, M = 128 heads, 64 per CTA):
//   S [128 x 128 keys] = Q K^T   each CTA holds Q of its 64 heads and loads 64
//                                of the block's keys;
//   O [128 x 512]     += P V     each CTA holds P of its heads and loads half
//                                of the value dims of all 128 keys.
// So every product is formed once, the softmax of a head stays inside one CTA,
// and no partial result crosses SMs. (Two independent CTAs, one per value half,
// form S twice: 2.9 K cycles per 64 keys, 0.69 ms for 64 sequences of 16-32 K
// keys.) What bounds a block: shared memory, 147 KB of operand reads for S, 98
// for PV, 138 KB of loads and 16 KB of P at 128 bytes a cycle = 3.1 K cycles,
// then the tensor pipe with 2.2 K.
//
// TMEM per CTA (M = 128 over a pair keeps 64 rows per CTA: lanes 0-63 hold the
// first half of the N columns of rows 0-63, lanes 64-127 the second half): O
// 256 columns (two N = 256 accumulators), S 2 x 64.
//
// Key blocks stream through one ring of 16 KB entries, one TMA copy each, in the
// order the MMAs read them: S(i + 1) as five entries (64 keys x 128 dims, the
// last one 64), then V(i) as four (64 keys x 128 dims). V is loaded a second time
// (from L2) rather than kept from S: held back until its P exists it would
// leave no room to load ahead.
//
// Rows behind a sequence's last key may hold anything, NaN and infinities too:
// their logits are masked by selection, and the producer overwrites them with
// zeros in V entries before the MMA reads those (0 * NaN would reach O).
//
// Warp roles: 0 and 2 load by TMA; 1 of CTA 0 issues every MMA (one elected lane), 1
// of CTA 1 passes on its CTA's arrivals to CTA 0; 4-11 run the softmax and the
// epilogue.
#pragma once

#include "layout.cuh"
#include "ptx.cuh"

#include <cuda_bf16.h>

namespace dsa {

struct DenseParams {
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

  // Keys that query row r sees, and the 128-key blocks they fill.
  __device__ __forceinline__ int visible(int r) const {
    const int b = r / n_q;
    const int last = min(rp.pos(b, r - b * n_q), n_kv - 1);     // no overflow at INT_MAX
    const int len = kv_len ? kv_len[b] : n_kv;
    return max(0, min(last + 1, len));
  }
  __device__ __forceinline__ int blocks(int r) const { return (visible(r) + 127) >> 7; }
  __device__ __forceinline__ long long share(long long total) const {
    return max(static_cast<long long>(min_share), (total + pairs - 1) / pairs);
  }
};

struct DenseTile {
  static constexpr int NK = 128;                // keys per block, 64 loaded by each CTA for S
  static constexpr int HB = 64;                 // heads per CTA
  static constexpr int DQK = 576, DV = 512;
  static constexpr int QB = DQK / 64;           // 9 dim blocks of Q
  static constexpr int BOX = 64 * 128;          // 64 rows x 64 dims
  static constexpr int ENTRY = 2 * BOX;
  static constexpr int RING = 8;
  static constexpr int SE = 5, VE = 4;          // entries of S, of V per block
  static constexpr int THREADS = 384;
  static constexpr int SM0 = 4, SOFTMAX_WARPS = 8;
  static constexpr int COL_O = 0, COL_S = 256;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr int OFF_RING = 0;
  static constexpr int OFF_Q = RING * ENTRY;
  static constexpr int OFF_P = OFF_Q + QB * BOX;               // [2 key halves][64 heads][64 keys]
  static constexpr int P_BYTES = HB * NK * 2;
  static constexpr int OFF_RED = OFF_P + P_BYTES;              // [2 parity][4 parts][64 heads] fp32
  static constexpr int OFF_BAR = OFF_RED + 2 * 4 * HB * 4;
  static constexpr int NUM_BARS = 3 * RING + 10;
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
    const int nb = (v + 127) >> 7;
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

// tmap_kv: the cache as [9 dim blocks][rows][64], box 64 dims x 64 rows x 2
// blocks (blocks past the ninth read as zero). tmap_q: Q as
// [rows][H][576], box 64 dims x 64 heads. tmap_o, tmap_p: out and part_o as
// [rows or slots][H][512 elements in bytes], box 128 bytes x 64 heads. All with
// the 128-byte swizzle; heads past H read as zero and are not stored.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(384, 1)
    dense_attn_kernel(const __grid_constant__ CUtensorMap tmap_kv,
                      const __grid_constant__ CUtensorMap tmap_q,
                      const __grid_constant__ CUtensorMap tmap_o,
                      const __grid_constant__ CUtensorMap tmap_p, const DenseParams p) {
  using T = DenseTile;
  constexpr int NK = T::NK;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  uint8_t* ring = smem + T::OFF_RING;
  uint8_t* q_smem = smem + T::OFF_Q;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + T::OFF_BAR);
  uint64_t* full = bars;                         // [RING] this CTA's part of the entry landed
  uint64_t* far_full = bars + T::RING;           // [RING] (CTA 0) the other CTA's part landed
  uint64_t* empty = bars + 2 * T::RING;          // [RING] the MMAs have read the entry
  uint64_t* q_full = bars + 3 * T::RING;         // this CTA's Q of a segment landed
  uint64_t* far_q = q_full + 1;                  // (CTA 0) the other CTA's Q landed
  uint64_t* q_empty = q_full + 2;                // the segment's last S has read Q
  uint64_t* s_full = q_full + 3;                 // [2] S of buffer b written
  uint64_t* s_free = q_full + 5;                 // [2] (CTA 0) both CTAs' softmax warps have loaded it
  uint64_t* p_full = q_full + 7;                 // (CTA 0) both CTAs' P written
  uint64_t* pv_done = q_full + 8;                // O += P V finished
  uint64_t* tail = q_full + 9;                   // a partly filled V entry landed
  long long* scan = reinterpret_cast<long long*>(smem + T::OFF_SCAN);
  int* start = reinterpret_cast<int*>(scan + 12);              // row, block of the share's begin
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(start + 2);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int pair = blockIdx.x >> 1;
  const uint32_t rank = cluster_ctarank();       // = blockIdx.x & 1

  if (threadIdx.x == 0) {
    if ((smem_u32(smem_raw) & 1023u) != 0) raise_error(kErrInternal);   // see SMEM_BYTES: no slack
    for (int s = 0; s < T::RING; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&far_full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(far_q, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&s_free[s], 2 * T::SOFTMAX_WARPS);
    }
    mbar_init(p_full, 2 * T::SOFTMAX_WARPS);
    mbar_init(pv_done, 1);
    mbar_init(tail, 1);
    fence_mbar_init();
    prefetch_tmap(&tmap_kv);
    prefetch_tmap(&tmap_q);
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
  // the same in every thread of both CTAs: no TMEM, no copies yet
  if (walk.left == 0 || (smem_u32(smem_raw) & 1023u) != 0) return;
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
    tmem_alloc_pair(tmem_slot, T::TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();                                // also: both CTAs' barriers are initialised
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  walk.row = start[0];
  walk.blk = start[1];

  // Every role walks the same segments and counts alike: g is the pair's
  // running block number, e the running ring entry. In a segment of n blocks
  // the entries are those of S(0), S(1), V(0), S(2), V(1), ..., V(n - 1).
  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ loads
    // Warp 0 loads Q and the S entries, warp 2 the V entries: issuing a copy
    // takes one thread about 290 cycles, nine of them would bound a block.
    // Both walk every entry and wait until it is free, so that a barrier is
    // never two phases ahead of a waiting thread.
    const bool for_s = warp == 0;
    uint32_t e = 0, segs = 0, tails = 0;
    uint32_t mine = 0, phase = 0;                // slots this warp has filled, and their phases
    bool ok = true;
    DenseSeg w;
    // One entry: waits until its slot is free and returns it.
    auto slot_free = [&]() -> uint32_t {
      const uint32_t st = e % T::RING;
      ok = mbar_wait(&empty[st], ((e / T::RING) & 1) ^ 1);
      return st;
    };
    auto filled = [&](uint32_t st) {
      mine |= 1u << st;
      phase = (phase & ~(1u << st)) | (((e / T::RING) & 1) << st);
    };
    while (ok && walk.next(p, w)) {
      const int b = w.row / p.n_q;
      // The pool row of a block's first key: a block of 128 lies inside one
      // page. A page outside the pool reads as zeros (the rows past the end).
      auto locate = [&](int blk) -> int {
        const int64_t r = p.km.row(b, blk * NK, p.n_kv);
        return static_cast<int>(r >= 0 ? r : p.km.pool_rows);
      };
      if (for_s) {
        // Q of this CTA's heads, once the previous segment's last S has read it
        if (segs > 0) ok = mbar_wait(q_empty, (segs - 1) & 1);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full, T::QB * T::BOX);
          for (int t = 0; t < T::QB; ++t)
            tma_load_3d(q_smem + t * T::BOX, &tmap_q, q_full, t * 64, static_cast<int>(rank) * T::HB, w.row);
        }
      }
      ++segs;
      int y = locate(w.blk);                     // of the block this warp loads next
      for (int i = 0; i <= w.n && ok; ++i) {
        if (i < w.n) {
          // S(i): this CTA's 64 keys, dims 128 t .. + 127 (the last entry: 64)
          for (int t = 0; t < T::SE; ++t, ++e) {
            const uint32_t st = slot_free();
            if (!ok) break;
            if (!for_s) continue;
            filled(st);
            if (lane == 0) {
              mbar_arrive_expect_tx(&full[st], T::ENTRY);
              tma_load_3d(ring + st * T::ENTRY, &tmap_kv, &full[st], 0, y + static_cast<int>(rank) * 64, 2 * t);
            }
          }
          if (!ok) break;
          if (for_s && i + 1 < w.n) y = locate(w.blk + i + 1);
        }
        if (i == 0) continue;
        // V(i - 1): entry (key half kh, accumulator j): dims 256 j + 128 rank .. + 127
        const int valid = w.vis - (w.blk + i - 1) * NK;
        for (int t = 0; t < T::VE; ++t, ++e) {
          const uint32_t st = slot_free();
          if (!ok) break;
          if (for_s) continue;
          filled(st);
          const int kh = t >> 1, zb = 4 * (t & 1) + 2 * static_cast<int>(rank);
          const int rows = valid - 64 * kh;      // of this half that hold keys
          uint8_t* dst = ring + st * T::ENTRY;
          if (rows >= 64 || rows <= 0) {
            // a half without keys reads as zeros: past the end of the pool
            if (lane == 0) {
              mbar_arrive_expect_tx(&full[st], T::ENTRY);
              tma_load_3d(dst, &tmap_kv, &full[st], 0, rows > 0 ? y + 64 * kh : static_cast<int>(p.km.pool_rows), zb);
            }
          } else {
            if (lane == 0) {
              mbar_arrive_expect_tx(tail, T::ENTRY);
              tma_load_3d(dst, &tmap_kv, tail, 0, y + 64 * kh, zb);
            }
            ok = mbar_wait(tail, tails & 1) || mbar_wait(tail, tails & 1);
            ++tails;
            for (int k = lane; k < (64 - rows) * 8; k += 32) {
              sts_v4(smem_u32(dst) + rows * 128 + k * 16, 0u, 0u, 0u, 0u);
              sts_v4(smem_u32(dst) + T::BOX + rows * 128 + k * 16, 0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[st]);
          }
        }
        if (!for_s && i < w.n) y = locate(w.blk + i);
      }
      __syncwarp();
    }
    // A wait that ran out leaves copies in flight: they end before the CTA does.
    if (!ok) {
      for (uint32_t st = 0; st < T::RING; ++st)
        if ((mine >> st) & 1u) mbar_wait(&full[st], (phase >> st) & 1u);
      if (for_s && segs > 0) mbar_wait(q_full, (segs - 1) & 1);
    }
  } else if (warp == 1 && rank == 1) {
    // ------------------------------------------------------------ arrivals passed on to CTA 0
    if (elect_one()) {
      uint32_t e = 0, segs = 0;
      bool ok = true;
      DenseSeg w;
      while (ok && walk.next(p, w)) {
        ok = mbar_wait(q_full, segs & 1);
        if (!ok) break;
        mbar_arrive_at(far_q, 0);
        ++segs;
        const uint32_t last = e + static_cast<uint32_t>(w.n) * (T::SE + T::VE);
        for (; e < last; ++e) {
          ok = mbar_wait(&full[e % T::RING], (e / T::RING) & 1);
          if (!ok) break;
          mbar_arrive_at(&far_full[e % T::RING], 0);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (CTA 0)
    if (elect_one()) {
      constexpr uint32_t idesc_s = umma_idesc(128, NK, 1u, 1u, 0u, 0u);
      constexpr uint32_t idesc_pv = umma_idesc(128, 256, 1u, 1u, 0u, 1u);
      const uint64_t k_desc0 = umma_desc(smem_u32(ring), 16, 1024, 2);
      const uint64_t v_desc0 = umma_desc(smem_u32(ring), T::BOX, 1024, 2);
      const uint64_t q_desc0 = umma_desc(smem_u32(q_smem), 16, 1024, 2);
      const uint64_t p_desc0 = umma_desc(smem_u32(smem + T::OFF_P), 16, 1024, 2);
      uint32_t e = 0, g = 0, segs = 0;
      bool ok = true;
      DenseSeg w;
      auto landed = [&]() {
        const uint32_t st = e % T::RING, ph = (e / T::RING) & 1;
        ok = mbar_wait(&full[st], ph) && mbar_wait(&far_full[st], ph);
        tc_fence_after();
        return ok;
      };
      while (ok && walk.next(p, w)) {
        ok = mbar_wait(q_full, segs & 1) && mbar_wait(far_q, segs & 1);
        ++segs;
        tc_fence_after();
        for (int i = 0; i <= w.n && ok; ++i) {
          if (i < w.n) {
            // S(g + i) into buffer b, free once S(g + i - 2) has been loaded
            const uint32_t gs = g + i, b = gs & 1;
            if (gs > 1) ok = mbar_wait(&s_free[b], ((gs >> 1) & 1) ^ 1);
            tc_fence_after();
            const uint32_t d = tmem_base + T::COL_S + b * 64;
#pragma unroll
            for (int t = 0; t < T::SE; ++t) {
              if (!landed()) break;
              const uint64_t kd = k_desc0 + static_cast<uint32_t>((e % T::RING) * (T::ENTRY >> 4));
#pragma unroll
              for (int kk = 0; kk < (t < 4 ? 8 : 4); ++kk) {
                const uint32_t off = ((kk >> 2) * T::BOX + (kk & 3) * 32) >> 4;
                umma_bf16_ss_pair(d, q_desc0 + (t * (T::ENTRY >> 4) + off), kd + off, idesc_s,
                                  (t | kk) ? 1u : 0u);
              }
              umma_commit_pair(&empty[e % T::RING]);
              ++e;
            }
            if (!ok) break;
            umma_commit_pair(&s_full[b]);
            if (i + 1 == w.n) umma_commit_pair(q_empty);
          }
          if (i == 0) continue;
          // O += P V of block g + i - 1
          const uint32_t gp = g + i - 1;
          if (!(ok = mbar_wait(p_full, gp & 1))) break;
          tc_fence_after();
          const uint32_t more_o = i > 1 ? 1u : 0u;   // a segment's first product overwrites O
#pragma unroll
          for (int t = 0; t < T::VE; ++t) {
            if (!landed()) break;
            const uint64_t vd = v_desc0 + static_cast<uint32_t>((e % T::RING) * (T::ENTRY >> 4));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_bf16_ss_pair(tmem_base + T::COL_O + (t & 1) * 128,
                                p_desc0 + (((t >> 1) * T::BOX + kk * 32) >> 4), vd + ((kk * 2048) >> 4),
                                idesc_pv, (t > 1 || kk > 0) ? 1u : more_o);
            umma_commit_pair(&empty[e % T::RING]);
            ++e;
          }
          if (ok) umma_commit_pair(pv_done);
        }
        g += w.n;
      }
    }
    __syncwarp();
  } else if (warp >= T::SM0) {
    // ------------------------------------------------------------ softmax / epilogue
    const int quarter = warp & 3;
    const int half = (warp - T::SM0) >> 2;                   // which 32 of a lane's 64 keys
    const int row = quarter * 32 + lane;                     // TMEM lane
    const int h = row & 63, side = row >> 6;                 // head of this CTA; key / dim half
    const int part = side * 2 + half;                        // of the four threads of a head
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t head_bar = 1u + static_cast<uint32_t>(quarter & 1);   // the four warps of its heads
    float* red = reinterpret_cast<float*>(smem + T::OFF_RED);   // [parity][part][64]
    const int stid = threadIdx.x - T::SM0 * 32;              // 0..255 over the softmax warps
    constexpr uint32_t kAllBar = 5u;                         // named barrier of the 8 warps
    constexpr uint32_t kAllThreads = 32u * T::SOFTMAX_WARPS;
    const int head = static_cast<int>(rank) * T::HB + h;     // of the row

    uint32_t sr[32];
    float z[32];
    const uint32_t p_row = smem_u32(smem + T::OFF_P) + side * T::BOX + (h >> 3) * 1024 + (h & 7) * 128;
    uint32_t g = 0;
    bool ok = true;
    DenseSeg w;
    bool more = walk.next(p, w);
    while (more && ok) {
      float m_used = -INFINITY;   // running max (log2 domain) the P values are relative to
      float l = 0.f;              // this thread's share of the sum of the fp32 p (LSE)
      float l_mma = 0.f;          // ... of the bf16-rounded p the PV MMA used (normalises O)
      for (int i = 0; i < w.n; ++i, ++g) {
        // ---- logits of this thread's 32 keys; the S buffer is released at
        // once. A failed wait does not leave the loop before the exchange:
        // the four warps of a head leave together.
        const uint32_t b = g & 1;
        const int valid = w.vis - (w.blk + i) * NK - part * 32;
        if (ok) ok = mbar_wait(&s_full[b], (g >> 1) & 1);
        tc_fence_after();
        tmem_ld32(tmem_base + lane_addr + T::COL_S + b * 64 + half * 32, sr);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(&s_free[b], 0);
        // ---- block max over the 128 keys, shared among the head's threads
        // (over the unscaled logits: the scale is positive)
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
        float* red_i = red + (g & 1) * (4 * T::HB) + h;
        red_i[part * T::HB] = hmax;
        if (!named_bar_and(head_bar, 128u, ok)) {
          ok = false;
          break;
        }
        const float bmax = fmaxf(fmaxf(red_i[0], red_i[T::HB]), fmaxf(red_i[2 * T::HB], red_i[3 * T::HB]));
        // ---- online softmax: both rescaling O and writing P need PV(g - 1)
        // finished
        const bool grow = bmax > m_used + 8.0f;
        const float m_new = grow ? bmax : m_used;
        if (g > 0 && ok) ok = mbar_wait(pv_done, (g - 1) & 1);
        if (i > 0 && __any_sync(0xffffffffu, grow)) {
          tc_fence_after();
          const float alpha = grow ? ex2_approx(m_used - m_new) : 1.0f;
#pragma unroll 1
          for (int c = half * 128; c < (half + 1) * 128 && ok; c += 16) {
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
#pragma unroll
        for (int c = 0; c < 4; ++c)
          sts_v4(p_row + (((4 * half + c) ^ (h & 7)) << 4), pk[4 * c], pk[4 * c + 1], pk[4 * c + 2],
                 pk[4 * c + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(p_full, 0);
      }
      // all softmax warps go on, or stop, together
      if (!named_bar_and(kAllBar, kAllThreads, ok)) {
        ok = false;
        break;
      }
      const DenseSeg done = w;
      more = walk.next(p, w);
      // ---- epilogue: O of the segment, once its last PV has finished
      ok = mbar_wait(pv_done, (g - 1) & 1);
      tc_fence_after();
      red[part * T::HB + h] = l;
      red[(4 + part) * T::HB + h] = l_mma;
      const bool pv_ok = named_bar_and(kAllBar, kAllThreads, ok);
      float l_all = 0.f, lm_all = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        l_all += red[k * T::HB + h];
        lm_all += red[(4 + k) * T::HB + h];
      }
      named_bar_sync(kAllBar, kAllThreads);      // read before the next segment's maxima
      // O / sum(rounded p) is an exact convex combination of the V rows; the
      // LSE keeps the unrounded sum.
      const bool has = pv_ok && l_all != 0.f && lm_all != 0.f;   // true for NaN
      const float inv_l = has ? 1.0f / lm_all : 0.f;
      const uint32_t keep = has ? 0xffffffffu : 0u;
      const float lse_v = has ? (m_used + log2f(l_all)) * 0.69314718055994531f : -INFINITY;
      // O leaves by TMA stores of 128-byte-wide column slices of the 64 heads,
      // staged in the swizzled layout the store reads. A round covers the
      // same slice of both lane halves (dims 128 apart): through the P area (free: the
      // last PV has finished), one round at a time; after the last segment
      // every round at once through the ring.
      const bool direct = done.whole;
      const int slot = 2 * pair + (done.blk > 0 ? 0 : 1);
      const bool bf16_out = direct && p.out_bf16;
      const int esz = bf16_out ? 2 : 4;
      const int cols = 128 / esz;                // of a slice
      const int rounds = 256 / cols;             // slices of a lane's 256 columns
      const int per_step = more ? 1 : rounds;
      const int z0 = direct ? done.row : slot;
#pragma unroll 1
      for (int r0 = 0; r0 < rounds; r0 += per_step) {
        const uint32_t stage = more ? smem_u32(smem + T::OFF_P) : smem_u32(ring);
        if (r0 > 0 && stid == 0) bulk_wait_read<0>();    // the last step's stores have read it
        if (r0 > 0) named_bar_sync(kAllBar, kAllThreads);
        for (int r = r0; r < r0 + per_step; ++r) {
          const uint32_t srow = stage + ((r - r0) * 2 + side) * T::BOX + h * 128;
#pragma unroll 1
          for (int c = half * (cols / 2); c < (half + 1) * (cols / 2); c += 16) {
            uint32_t o[16];
            tmem_ld16(tmem_base + lane_addr + T::COL_O + r * cols + c, o);
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
        if (stid == 0 && static_cast<int>(rank) * T::HB < p.H) {
          const void* map = direct ? static_cast<const void*>(&tmap_o) : static_cast<const void*>(&tmap_p);
          for (int r = r0; r < r0 + per_step; ++r)
#pragma unroll
            for (int sd = 0; sd < 2; ++sd) {
              // lane half sd of columns [r cols, + cols): accumulator j = column / 128
              const int col = r * cols;
              const int dim = (col >> 7) * 256 + sd * 128 + (col & 127);
              tma_store_3d(map, stage + ((r - r0) * 2 + sd) * T::BOX, dim * esz,
                           static_cast<int>(rank) * T::HB, z0);
            }
          bulk_commit();
        }
      }
      // every staged byte read before the next segment writes P
      if (stid == 0) bulk_wait_read<0>();
      if (part == 0 && head < p.H) {
        if (!direct) p.part_lse[static_cast<size_t>(slot) * p.H + head] = lse_v;
        else if (p.lse) p.lse[static_cast<size_t>(done.row) * p.H + head] = lse_v;
      }
      ok = named_bar_and(kAllBar, kAllThreads, ok);
    }
  }

  if (threadIdx.x == T::SM0 * 32) bulk_wait<0>();   // the output stores have completed
  tc_fence_before();
  __syncwarp();
  cluster_sync();                                // no arrival or MMA of the pair is outstanding
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, T::TMEM_COLS);
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
