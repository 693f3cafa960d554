// Dense MQA attention of a few new tokens over every visible row of the latent
// cache (576 dims, V = the first 512; contiguous or paged):
//     s_k = scale q . kv[k],  out = sum_k softmax(s)_k kv[k, :512]
// with the online softmax: running maximum m and sum l per head, O rescaled
// when m grows.
//
// The work is cut along the caches. All query rows' 128-key blocks, row after
// row, form one line; CTA pair p takes units [p share, (p + 1) share) of it,
// whatever rows they belong to, so ragged lengths keep every SM equally busy
// and one long sequence spreads over the whole GPU. A row counts kDenseRowCost
// units more than its blocks, at its beginning: taking up a row (its Q, the
// first block's latency, its output) costs about as much as that many blocks
// (32 rows of up to 1500 keys: 29.7 us without, 27.2 us with 3). A row that lies
// inside one share is written directly; the (at most two) rows that a share's
// ends cut leave an fp32 partial O and LSE in the workspace, and
// dense_combine_kernel joins them in key order. Where no row is longer than a few
// blocks, rows are not cut and nothing is joined. The cut is derived from kv_len
// and the positions on the device: the host never needs the lengths.
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
// leave no room to load ahead. (A ring of four entries for each of the two:
// 0.60 ms where the shared ring takes 0.49.)
//
// Rows behind a sequence's last key may hold anything, NaN and infinities too:
// their logits are masked by selection, and the producer overwrites them with
// zeros in V entries before the MMA reads those (0 * NaN would reach O).
//
// Warp roles: 0 and 2 load by TMA; 1 of CTA 0 issues every MMA (one elected lane), 1
// of CTA 1 passes on its CTA's arrivals to CTA 0; 3 notes the cut and writes the
// rows that see no key; 4-11 run the softmax and the epilogue.
#pragma once

#include "dense_loads.cuh"
#include "layout.cuh"
#include "ptx.cuh"

#include <cuda_bf16.h>

namespace dsa {

constexpr int kDenseRowCost = 3;               // blocks
constexpr int kDenseCutCost = 5;               // units
constexpr unsigned long long kDenseDrainNs = 100'000'000ull;   // for a copy in flight, after a wait has run out
constexpr int kDenseMinShare = 1;              // units (one row of 4000 keys: 14.8 us, 18.4 with 4)

struct DenseParams {
  KeyMap km;
  RowPos rp;
  const int32_t* kv_len;
  void* out;                   // [rows, H, 512]
  float* lse;                  // [rows, H] or null
  float* part_o;               // [2 pairs][H][512]: slot 2 p: the row that share p begins
  float* part_lse;             // [2 pairs][H]       inside of, 2 p + 1: the row it ends inside of
  int2* cut;                   // [pairs] row and block that share p begins with; row -1: no blocks
  int32_t rows, n_q, n_kv, H;
  int32_t out_bf16;
  int32_t pairs;               // CTA pairs of the attention kernel
  int32_t whole;               // rows are never cut (the host's bound on their length says so)
  float scale_log2;

  // Keys that query row r sees, and the 128-key blocks they fill.
  __device__ __forceinline__ int visible(int r) const {
    const int b = r / n_q;
    const int last = min(rp.pos(b, r - b * n_q), n_kv - 1);     // no overflow at INT_MAX
    const int len = kv_len ? kv_len[b] : n_kv;
    return max(0, min(last + 1, len));
  }
  __device__ __forceinline__ int blocks(int r) const { return (visible(r) + 127) >> 7; }
  // Length on the line of a row that sees `vis` keys.
  __device__ static __forceinline__ int units_of(int vis) {
    return vis > 0 ? ((vis + 127) >> 7) + kDenseRowCost : 0;
  }
  __device__ __forceinline__ int units(int r) const { return units_of(visible(r)); }
  __device__ __forceinline__ long long share(long long total) const {
    return max(static_cast<long long>(kDenseMinShare), (total + pairs - 1) / pairs);
  }
  // Whether rows stay whole (the longest has `most` units). Uncut, every row has
  // a pair to itself when there are enough, else a share runs over by half a
  // row; cutting costs kDenseCutCost and an eighth of a unit per row for the
  // partials and their join (64 rows of 500 to 1000 keys: 39.5 us cut, 29.3
  // whole; one row of 2000: 14.0 cut, 33 whole).
  __device__ __forceinline__ bool keep_whole(long long share, int most) const {
    const long long whole_cost = rows <= pairs ? most : share + most / 2;
    return whole || whole_cost <= share + kDenseCutCost + min(rows, pairs) / 8;
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
  static constexpr int NUM_BARS = 4 * RING + 10;
  static constexpr int OFF_SCAN = OFF_BAR + NUM_BARS * 8;      // dense_share_block's scratch, TMEM address
  static constexpr int SMEM_BYTES = OFF_SCAN + (THREADS / 32 + 2) * 8 + 8;
  static_assert(SMEM_BYTES <= 232448, "shared memory");
};

// A share's segments: blocks [blk, blk + n) of row `row`, one row after the other.
struct DenseSeg {
  int row, blk, n, vis;
  bool whole;                    // the row's blocks are all in this segment
};
// What is left of a share: `left` units from unit `off` of row `row`.
struct DenseWalk {
  int row;
  long long off, left;
  bool whole;                    // rows are not cut: those that begin in the share
  int vis;                       // keys that `row` sees, -1: to be looked up
  __device__ __forceinline__ bool next(const DenseParams& p, DenseSeg& s) {
    while (left > 0) {
      int v = vis >= 0 ? vis : p.visible(row);
      while (v == 0) v = p.visible(++row);   // units are left, so such a row follows
      vis = -1;
      const int nb = (v + 127) >> 7;
      const long long end = min(off + left, static_cast<long long>(nb + kDenseRowCost));
      s.row = row;
      s.vis = v;
      s.blk = static_cast<int>(max(0ll, off - kDenseRowCost));
      s.n = static_cast<int>(max(0ll, end - kDenseRowCost)) - s.blk;
      if (whole) {                           // the whole row if it begins here, else none of it
        s.blk = 0;
        s.n = off == 0 ? nb : 0;
      }
      s.whole = s.n == nb;
      left -= end - off;
      ++row;
      off = 0;
      if (s.n > 0) return true;              // 0 also where a share ends before the row's first block
    }
    return false;
  }
};

// The share of pair `pair`. With few rows every warp finds it by itself, 32 rows
// at a time: no barrier. This runs once per launch, with cold instruction
// caches, so it is kept short rather than unrolled (1 to 2 us). The sums fit 32
// bits: batch * n_kv is at most 2^30, so 256 rows have at most 2^31 + 768 units.
constexpr int kDenseWarpRows = 256;
__device__ __forceinline__ DenseWalk dense_share_warp(const DenseParams& p, int pair) {
  const int lane = threadIdx.x & 31;
  uint32_t total = 0, most = 0;
  int vis0 = 0;                                  // of the first 32 rows
#pragma unroll 1
  for (int r = lane; r - lane < p.rows; r += 32) {
    const int v = r < p.rows ? p.visible(r) : 0;
    if (r < 32) vis0 = v;
    const uint32_t len = DenseParams::units_of(v);
    total += __reduce_add_sync(0xffffffffu, len);
    most = max(most, __reduce_max_sync(0xffffffffu, len));
  }
  const uint32_t share = static_cast<uint32_t>(p.share(total));
  const bool whole = p.keep_whole(share, static_cast<int>(most));
  DenseWalk w{pair, 0, 0, whole, -1};
  if (whole && p.rows <= p.pairs) {              // a pair per row
    w.vis = pair >= p.rows ? 0 : pair < 32 ? __shfl_sync(0xffffffffu, vis0, pair & 31) : p.visible(pair);
    w.left = DenseParams::units_of(w.vis);
    return w;
  }
  const uint32_t begin = pair * share;
  if (begin >= total) return w;
  w.left = min(share, total - begin);
  uint32_t base = 0;                             // units of the tiles before
#pragma unroll 1
  for (int r = lane; r - lane < p.rows; r += 32) {
    const int v = r < 32 ? vis0 : (r < p.rows ? p.visible(r) : 0);
    const uint32_t len = DenseParams::units_of(v);
    const uint32_t sum = __reduce_add_sync(0xffffffffu, len);
    if (begin < base + sum) {
      uint32_t incl = len;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
      }
      const uint32_t at = base + incl - len;
      const int src = __ffs(__ballot_sync(0xffffffffu, at <= begin && begin < at + len)) - 1;
      w.row = r - lane + src;
      w.off = __shfl_sync(0xffffffffu, begin - at, src);
      w.vis = __shfl_sync(0xffffffffu, v, src);
      break;
    }
    base += sum;
  }
  return w;
}
// Any number of rows: block-wide sums through `scan` (WARPS + 2 words, the last
// two for the start); every thread calls it.
template <int WARPS>
__device__ __forceinline__ DenseWalk dense_share_block(const DenseParams& p, int pair, long long* scan) {
  constexpr int THREADS = 32 * WARPS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long total = 0;
  int most = 0;
  for (int r = threadIdx.x; r < p.rows; r += THREADS) {
    const int len = p.units(r);
    total += len;
    most = max(most, len);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  most = __reduce_max_sync(0xffffffffu, most);
  // a row has at most 2^23 + 3 units, all of them fewer than 2^39
  if (lane == 0) scan[warp] = (total << 24) | most;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    total += scan[i] >> 24;
    most = max(most, static_cast<int>(scan[i] & 0xffffff));
  }
  const long long share = p.share(total), begin = pair * share;
  // more rows than pairs here (see the caller)
  DenseWalk w{0, 0, max(0ll, min(total, begin + share) - begin), p.keep_whole(share, most), -1};
  for (long long base = 0, r0 = 0; r0 < p.rows && w.left > 0; r0 += THREADS) {
    // exclusive prefix of this thread's row within the tile of rows
    const int r = static_cast<int>(r0) + threadIdx.x;
    const int len = r < p.rows ? p.units(r) : 0;
    long long incl = len;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    long long before = base;
    for (int i = 0; i < WARPS; ++i) {
      if (i < warp) before += scan[i];
      base += scan[i];
    }
    const long long at = before + incl - len;
    if (at <= begin && begin < at + len) {
      scan[WARPS] = r;
      scan[WARPS + 1] = begin - at;
    }
    if (base > begin) break;                     // the same in every thread
  }
  __syncthreads();
  if (w.left > 0) {
    w.row = static_cast<int>(scan[WARPS]);
    w.off = scan[WARPS + 1];
  }
  return w;
}

// out = 0 and LSE = -inf for CTA `rank`'s heads of row r, by one warp.
__device__ __forceinline__ void dense_empty_row(const DenseParams& p, int r, int rank, int lane) {
  const int h0 = rank * DenseTile::HB, h1 = min(p.H, h0 + DenseTile::HB);
  const size_t bytes = p.out_bf16 ? 1024 : 2048;
  const size_t first = static_cast<size_t>(r) * p.H;
  if (h0 >= h1) return;
  uint4* o = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + (first + h0) * bytes);
  const int n = (h1 - h0) * static_cast<int>(bytes / 16);
  for (int i = lane; i < n; i += 32) o[i] = make_uint4(0, 0, 0, 0);
  if (p.lse)
    for (int h = h0 + lane; h < h1; h += 32) p.lse[first + h] = -INFINITY;
}

// tmap_kv: the cache as [9 dim blocks][rows][64], box 64 dims x 64 rows x 2
// blocks (blocks past the ninth read as zero). tmap_q: Q as
// [rows][9 dim blocks][H][64], box 64 dims x 64 heads x 9 blocks; heads past H
// read as zero. Both with the 128-byte swizzle.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(384, 1)
    dense_attn_kernel(const __grid_constant__ CUtensorMap tmap_kv,
                      const __grid_constant__ CUtensorMap tmap_q, const DenseParams p) {
  using T = DenseTile;
  constexpr int NK = T::NK;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  uint8_t* ring = smem + T::OFF_RING;
  uint8_t* q_smem = smem + T::OFF_Q;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + T::OFF_BAR);
  uint64_t* full = bars;                         // [RING] this CTA's part of the entry landed
  uint64_t* far_full = bars + T::RING;           // [RING] (CTA 0) the other CTA's part landed
  uint64_t* empty = bars + 2 * T::RING;          // [RING][2] the MMAs have read the entry's even, odd use
  uint64_t* q_full = bars + 4 * T::RING;         // this CTA's Q of a segment landed
  uint64_t* far_q = q_full + 1;                  // (CTA 0) the other CTA's Q landed
  uint64_t* q_empty = q_full + 2;                // the segment's last S has read Q
  uint64_t* s_full = q_full + 3;                 // [2] S of buffer b written
  uint64_t* s_free = q_full + 5;                 // [2] (CTA 0) both CTAs' softmax warps have loaded it
  uint64_t* p_full = q_full + 7;                 // (CTA 0) both CTAs' P written
  uint64_t* pv_done = q_full + 8;                // O += P V finished
  uint64_t* tail = q_full + 9;                   // a partly filled V entry landed
  long long* scan = reinterpret_cast<long long*>(smem + T::OFF_SCAN);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(scan + T::THREADS / 32 + 2);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int pair = blockIdx.x >> 1;
  const uint32_t rank = cluster_ctarank();       // = blockIdx.x & 1

  if ((smem_u32(smem_raw) & 1023u) != 0) {       // see SMEM_BYTES: no slack to realign; in both CTAs
    if (threadIdx.x == 0) raise_error(kErrInternal);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < T::RING; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&far_full[s], 1);
      mbar_init(&empty[2 * s], 1);
      mbar_init(&empty[2 * s + 1], 1);
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
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, T::TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncwarp();
  cluster_arrive();                              // barriers initialised, TMEM allocated; the wait is below
  DenseWalk walk = p.rows <= kDenseWarpRows ? dense_share_warp(p, pair)
                                            : dense_share_block<T::THREADS / 32>(p, pair, scan);
  __syncwarp();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // Every role walks the same segments and counts alike: g is the pair's
  // running block number, e the ring's running entry. A segment of n blocks is
  // computed as S(0), S(1), V(0), S(2), V(1), ..., V(n - 1).
  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ loads
    // Warp 0 loads Q and the S entries, warp 2 the V entries: issuing a copy
    // takes one thread about 290 cycles, nine of them would bound a block. A
    // loader waits for its own entries only: the other's may pass by more than
    // one phase meanwhile. `empty` has a barrier for the even and one for the odd
    // uses of a slot, so a wait for use u - 1 could be mistaken only for use u - 5,
    // 24 entries and more before, while a loader's entries are at most 11 apart.
    // One elected lane makes the S loads. The V loads take the whole warp, which also
    // zeroes the ends of partly filled entries: each of its waits is voted on, as a lane
    // whose wait ran out while the others' just did not would leave the loop, and the
    // warp's barriers, by itself. (Votes in both: 480 to 500 us for 64 sequences of
    // 16-32 K keys, none in either 530 to 610, one lane for both 475; this 448.)
    const bool for_s = warp == 0, lead = elect_one();
    uint32_t e0 = 0, segs = 0, tails = 0;        // e0: the segment's first entry
    DenseLoads<T::RING> loads;
    bool ok = true;
    DenseSeg w;
    auto voted = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0;
    };
    // The slot of entry e, once its last use has been read by `wait`; not ok:
    // nothing is issued.
    auto claim = [&](uint32_t e, auto wait) -> uint32_t {
      uint32_t st;
      ok = loads.claim(e, st, [&](uint32_t slot, uint32_t use) {
        return wait(&empty[2 * slot + (use & 1)], (use >> 1) & 1);
      });
      return st;
    };
    while (ok && walk.next(p, w)) {
      const int b = w.row / p.n_q;
      // The pool row of a block's first key: a block of 128 lies inside one
      // page. A page outside the pool reads as zeros (the rows past the end).
      auto locate = [&](int blk) -> int {
        const int64_t r = p.km.row(b, blk * NK, p.n_kv);
        return static_cast<int>(r >= 0 ? r : p.km.pool_rows);
      };
      int y = locate(w.blk);
      if (for_s) {
        if (lead) {
          // Q of this CTA's heads, once the previous segment's last S has read it
          if (segs > 0) ok = mbar_wait(q_empty, (segs - 1) & 1);
          if (ok) {
            mbar_arrive_expect_tx(q_full, T::QB * T::BOX);
            tma_load_4d(q_smem, &tmap_q, q_full, 0, static_cast<int>(rank) * T::HB, 0, w.row);
            ++segs;
          }
          for (int i = 0; i < w.n && ok; ++i) {
            // S(i): this CTA's 64 keys, dims 128 t .. + 127 (the last entry: 64)
            const uint32_t e = e0 + (i == 0 ? 0 : T::SE + (i - 1) * (T::SE + T::VE));
            for (int t = 0; t < T::SE; ++t) {
              const uint32_t st = claim(e + t, mbar_wait);
              if (!ok) break;
              mbar_arrive_expect_tx(&full[st], T::ENTRY);
              tma_load_3d(ring + st * T::ENTRY, &tmap_kv, &full[st], 0, y + static_cast<int>(rank) * 64, 2 * t);
            }
            if (i + 1 < w.n) y = locate(w.blk + i + 1);
          }
        }
        ok = __all_sync(0xffffffffu, ok);        // the other lanes' is true
      } else {
        for (int i = 0; i < w.n && ok; ++i) {
          // V(i): entry (key half kh, accumulator j): dims 256 j + 128 rank .. + 127
          const int valid = w.vis - (w.blk + i) * NK;
          const uint32_t e = e0 + (i + 1 < w.n ? T::SE + i * (T::SE + T::VE) + T::SE
                                               : w.n * (T::SE + T::VE) - T::VE);
          for (int t = 0; t < T::VE; ++t) {
            const uint32_t st = claim(e + t, voted);
            if (!ok) break;
            const int kh = t >> 1, zb = 4 * (t & 1) + 2 * static_cast<int>(rank);
            const int rows = valid - 64 * kh;    // of this half that hold keys
            uint8_t* dst = ring + st * T::ENTRY;
            if (rows >= 64 || rows <= 0) {
              // a half without keys reads as zeros: past the end of the pool
              if (lead) {
                mbar_arrive_expect_tx(&full[st], T::ENTRY);
                tma_load_3d(dst, &tmap_kv, &full[st], 0,
                            rows > 0 ? y + 64 * kh : static_cast<int>(p.km.pool_rows), zb);
              }
            } else {
              loads.by_tail(st);
              if (lead) {
                mbar_arrive_expect_tx(tail, T::ENTRY);
                tma_load_3d(dst, &tmap_kv, tail, 0, y + 64 * kh, zb);
              }
              ok = voted(tail, tails & 1);
              if (!ok) break;
              loads.tail_landed();
              ++tails;
              for (int k = lane; k < (64 - rows) * 8; k += 32) {
                sts_v4(smem_u32(dst) + rows * 128 + k * 16, 0u, 0u, 0u, 0u);
                sts_v4(smem_u32(dst) + T::BOX + rows * 128 + k * 16, 0u, 0u, 0u, 0u);
              }
              fence_proxy_async_smem();
              __syncwarp();
              if (lead) mbar_arrive(&full[st]);
            }
          }
          if (i + 1 < w.n) y = locate(w.blk + i + 1);
        }
      }
      e0 += static_cast<uint32_t>(w.n) * (T::SE + T::VE);
    }
    // A wait that ran out leaves copies in flight: they end before the CTA does. (A
    // slot that the other loader has used since has nothing of this one's in flight,
    // and may count a phase more: its wait runs out after kDenseDrainNs.)
    if (!ok && lead) {
      loads.drain([&](uint32_t st, uint32_t ph) { mbar_wait_limit(&full[st], ph, kDenseDrainNs); },
                  [&] { mbar_wait_limit(tail, tails & 1, kDenseDrainNs); });
      if (for_s && segs > 0) mbar_wait_limit(q_full, (segs - 1) & 1, kDenseDrainNs);
    }
    __syncwarp();
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
      // Entry e has landed in both CTAs; its slot.
      auto landed = [&]() -> uint32_t {
        const uint32_t st = e % T::RING, ph = (e / T::RING) & 1;
        ok = mbar_wait(&full[st], ph) && mbar_wait(&far_full[st], ph);
        tc_fence_after();
        return st;
      };
      // Its MMAs have been issued: free once they finish.
      auto release = [&]() {
        umma_commit_pair(&empty[2 * (e % T::RING) + ((e / T::RING) & 1)]);
        ++e;
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
              const uint32_t st = landed();
              if (!ok) break;
              const uint64_t kd = k_desc0 + static_cast<uint32_t>(st * (T::ENTRY >> 4));
#pragma unroll
              for (int kk = 0; kk < (t < 4 ? 8 : 4); ++kk) {
                const uint32_t off = ((kk >> 2) * T::BOX + (kk & 3) * 32) >> 4;
                umma_bf16_ss_pair(d, q_desc0 + (t * (T::ENTRY >> 4) + off), kd + off, idesc_s,
                                  (t | kk) ? 1u : 0u);
              }
              release();
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
            const uint32_t st = landed();
            if (!ok) break;
            const uint64_t vd = v_desc0 + static_cast<uint32_t>(st * (T::ENTRY >> 4));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_bf16_ss_pair(tmem_base + T::COL_O + (t & 1) * 128,
                                p_desc0 + (((t >> 1) * T::BOX + kk * 32) >> 4), vd + ((kk * 2048) >> 4),
                                idesc_pv, (t > 1 || kk > 0) ? 1u : more_o);
            release();
          }
          if (ok) umma_commit_pair(pv_done);
        }
        g += w.n;
      }
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------ the cut; rows that see no key
    DenseSeg w;
    const bool any = walk.next(p, w);
    if (lane == 0 && rank == 0 && !p.whole) p.cut[pair] = any ? make_int2(w.row, w.blk) : make_int2(-1, 0);
    for (int r = pair; r < p.rows; r += p.pairs)
      if (p.blocks(r) == 0) dense_empty_row(p, r, static_cast<int>(rank), lane);
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
          const bool all_ok = __all_sync(0xffffffffu, ok);       // the loads take whole warps
#pragma unroll 1
          for (int c = half * 128; c < (half + 1) * 128 && all_ok; c += 16) {
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
          // no finite maximum so far: all visible logits are -inf, or NaN is among
          // them (fmaxf leaves it out beside -inf, a masked key's among them)
          bool nan = false;
#pragma unroll
          for (int j = 0; j < 32; ++j) nan |= z[j] != z[j];
          lsum = lsum_mma = nan ? __int_as_float(0x7fffffff) : 0.f;
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
      // O / sum(rounded p) is an exact convex combination of the V rows; the
      // LSE keeps the unrounded sum. O goes straight from TMEM to memory: in the
      // 16x256b shape four lanes hold 8 neighbouring columns of a row, a full
      // sector of fp32 per row and store. (Staged through shared memory for TMA
      // stores it took 2 us at the end of a share and 5 us between two rows.)
      const bool direct = done.whole;
      const int slot = 2 * pair + (done.blk > 0 ? 0 : 1);
      const bool bf16_out = direct && p.out_bf16;
      const size_t out_row = static_cast<size_t>(direct ? done.row : slot) * p.H;
      uint8_t* const out_base = static_cast<uint8_t*>(direct ? p.out : static_cast<void*>(p.part_o));
      const int esz = bf16_out ? 2 : 4;
#pragma unroll 1
      for (int rb = 0; rb < 2; ++rb) {
        // this thread's two heads of the 16 lanes
        float inv[2];
        uint8_t* at[2];
        bool there[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int hh = (quarter & 1) * 32 + rb * 16 + 8 * k + (lane >> 2);
          float lm = 0.f;
#pragma unroll
          for (int q = 0; q < 4; ++q) lm += red[(4 + q) * T::HB + hh];
          inv[k] = pv_ok && lm != 0.f ? 1.0f / lm : 0.f;                 // NaN goes through
          const int hd = static_cast<int>(rank) * T::HB + hh;
          there[k] = hd < p.H;
          at[k] = out_base + ((out_row + hd) * T::DV + half * 256 + side * 128 + (lane & 3) * 2) * esz;
        }
#pragma unroll 1
        for (int c = 0; c < 128; c += 64) {
          uint32_t o[32];
          tmem_ld_16x256b_x8(tmem_base + lane_addr + (static_cast<uint32_t>(rb * 16) << 16) + T::COL_O +
                                 half * 128 + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (there[k]) {
              if (bf16_out) {
#pragma unroll
                for (int b = 0; b < 8; ++b)
                  *reinterpret_cast<__nv_bfloat162*>(at[k] + b * 16) =
                      __floats2bfloat162_rn(__uint_as_float(o[4 * b + 2 * k]) * inv[k],
                                            __uint_as_float(o[4 * b + 2 * k + 1]) * inv[k]);
              } else {
#pragma unroll
                for (int b = 0; b < 8; ++b)
                  *reinterpret_cast<float2*>(at[k] + b * 32) =
                      make_float2(__uint_as_float(o[4 * b + 2 * k]) * inv[k],
                                  __uint_as_float(o[4 * b + 2 * k + 1]) * inv[k]);
              }
            }
            at[k] += 64 * esz;
          }
        }
      }
      if (part == 0 && head < p.H) {
        float l_all = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) l_all += red[k * T::HB + h];
        const float lse_v = pv_ok && l_all != 0.f ? (m_used + log2f(l_all)) * 0.69314718055994531f : -INFINITY;
        if (!direct) p.part_lse[static_cast<size_t>(slot) * p.H + head] = lse_v;
        else if (p.lse) p.lse[static_cast<size_t>(done.row) * p.H + head] = lse_v;
      }
      tc_fence_before();
      // red and O read before the next segment's maxima and its first P V
      ok = named_bar_and(kAllBar, kAllThreads, ok);
    }
  }

  tc_fence_before();
  __syncwarp();
  cluster_sync();                                // no arrival or MMA of the pair is outstanding
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, T::TMEM_COLS);
  }
}

constexpr int kDenseMaxPairs = 128;

// Joins the partials of the rows that more than one share holds, in key order.
// blockIdx.x counts those rows: row k is the k-th whose beginning lies in a
// share that does not hold its end. A head's 512 value dims go to 512 / (32 VW)
// warps with VW dims per lane. Few rows may have a partial from every pair (one
// long sequence: 74 of them), so they get eight warps a head (VW = 2), many
// rows two (VW = 8). Like the share search it runs once with cold instruction
// caches: its loop over partials is not unrolled (3 us). No shared memory: the
// attention kernel leaves none for a CTA that waits beside it.
template <int VW>
__global__ void __launch_bounds__(256) dense_combine_kernel(const DenseParams p) {
  constexpr int WPH = 512 / (32 * VW);           // warps per head
  constexpr int V = VW < 4 ? VW : 4;             // dims per load
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y * (8 / WPH) + warp / WPH;
  const int dim0 = (warp % WPH) * 32 * VW;
  constexpr int K = kDenseMaxPairs / 32;
  griddep_wait();                                // every CTA: this grid ends after the attention
  // the cuts, lane q % 32 of word q / 32 for share q. `inside`: the share begins
  // inside a row; `opens`: and the row begins in the share before
  int2 c[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int q = k * 32 + lane;
    c[k] = q < p.pairs ? p.cut[q] : make_int2(-1, 0);
  }
  int found = -1, row = 0, seen = 0, np = 1;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    int2 b = make_int2(__shfl_up_sync(0xffffffffu, c[k].x, 1), __shfl_up_sync(0xffffffffu, c[k].y, 1));
    if (k > 0) {
      const int bx = __shfl_sync(0xffffffffu, c[k > 0 ? k - 1 : 0].x, 31);
      const int by = __shfl_sync(0xffffffffu, c[k > 0 ? k - 1 : 0].y, 31);
      if (lane == 0) b = make_int2(bx, by);
    }
    const bool inside = c[k].x >= 0 && c[k].y > 0;     // never so for share 0
    const uint32_t opens = __ballot_sync(0xffffffffu, inside && !(b.y > 0 && b.x == c[k].x));
    if (found < 0) {
      const int nth = static_cast<int>(blockIdx.x) - seen;
      seen += __popc(opens);
      if (nth < __popc(opens)) {
        const bool is_nth = ((opens >> lane) & 1u) && __popc(opens & ((1u << lane) - 1u)) == nth;
        const int bit = __ffs(__ballot_sync(0xffffffffu, is_nth)) - 1;
        found = k * 32 + bit - 1;                // the share the row begins in
        row = __shfl_sync(0xffffffffu, c[k].x, bit);
      }
    }
    // a row's shares follow one another, so counting them all is counting its own
    if (found >= 0) np += __popc(__ballot_sync(0xffffffffu, inside && c[k].x == row));
  }
  if (found < 0 || h >= p.H) return;
  // the row begins in share `found` (slot 2 found + 1); the others begin inside of it
  auto slot = [&](int i) {
    return (static_cast<size_t>(2 * (found + i)) + (i == 0 ? 1 : 0)) * p.H + h;
  };
  float w[K];                                    // LSE, then weight, of partial 32 k + lane
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    w[k] = k * 32 + lane < np ? p.part_lse[slot(k * 32 + lane)] : -INFINITY;
    m = fmaxf(m, w[k]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    w[k] = w[k] == -INFINITY ? 0.f : __expf(w[k] - m);
    sum += w[k];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  float acc[VW];
#pragma unroll
  for (int j = 0; j < VW; ++j) acc[j] = 0.f;
  constexpr int UN = VW <= 2 ? 16 : 4;           // partials loaded before the first is added
#pragma unroll 1
  for (int i0 = 0; i0 < np; i0 += UN) {
    float wk = w[0];                             // of the 32 partials that i0 is among
#pragma unroll
    for (int k = 1; k < K; ++k) wk = (i0 >> 5) == k ? w[k] : wk;
    float v[UN][VW];
    const float* src = p.part_o + (static_cast<size_t>(2 * (found + i0)) * p.H + h) * 512 + dim0 + lane * V;
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const bool on = i0 + u < np;
      const float* s_u = src + (i0 + u == 0 ? static_cast<size_t>(p.H) * 512 : 0);
#pragma unroll
      for (int j = 0; j < VW; j += V) {
        if constexpr (V == 4) {
          const float4 t = on ? __ldcg(reinterpret_cast<const float4*>(s_u + j * 32)) : make_float4(0.f, 0.f, 0.f, 0.f);
          v[u][j] = t.x; v[u][j + 1] = t.y; v[u][j + 2] = t.z; v[u][j + 3] = t.w;
        } else {
          const float2 t = on ? __ldcg(reinterpret_cast<const float2*>(s_u + j * 32)) : make_float2(0.f, 0.f);
          v[u][j] = t.x; v[u][j + 1] = t.y;
        }
      }
      src += static_cast<size_t>(2 * p.H) * 512;
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const float wgt = __shfl_sync(0xffffffffu, wk, (i0 + u) & 31);
#pragma unroll
      for (int j = 0; j < VW; ++j) acc[j] = fmaf(wgt, v[u][j], acc[j]);
    }
  }
  const float inv = sum != 0.f ? 1.0f / sum : 0.f;     // NaN goes through
  const size_t o = (static_cast<size_t>(row) * p.H + h) * 512 + dim0;
#pragma unroll
  for (int j = 0; j < VW; j += V) {
    const size_t at = o + (j / V) * 32 * V + lane * V;
    if (p.out_bf16) {
      uint32_t w[V / 2];
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(acc[j + 2 * k] * inv, acc[j + 2 * k + 1] * inv);
        w[k] = *reinterpret_cast<const uint32_t*>(&t);
      }
      uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + at);
      if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      else *dst = w[0];
    } else {
      float* dst = static_cast<float*>(p.out) + at;
      if constexpr (V == 4)
        *reinterpret_cast<float4*>(dst) =
            make_float4(acc[j] * inv, acc[j + 1] * inv, acc[j + 2] * inv, acc[j + 3] * inv);
      else *reinterpret_cast<float2*>(dst) = make_float2(acc[j] * inv, acc[j + 1] * inv);
    }
  }
  if (dim0 == 0 && lane == 0 && p.lse)
    p.lse[static_cast<size_t>(row) * p.H + h] = sum != 0.f ? m + logf(sum) : -INFINITY;
}

}  // namespace dsa
