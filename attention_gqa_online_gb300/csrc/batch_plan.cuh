// batch_plan.cuh -- how the batched paged attention divides a ragged batch
// over a fixed grid, from lengths that only the device knows.
//
// The query rows of sequence s and kv head g are flattened as r = t * gs + j
// (token t, head g * gs + j) and cut into blocks of ROWS; an item is one
// (sequence, row block, kv head).  Its keys are the union of its rows'
// windows, and of the first positions that stay visible behind them, walked in tiles of KEYS.  Every item weighs its tiles plus item_cost (what
// its Q load, epilogue and masked tiles take, in tiles); the weights of all items, laid end to end in (sequence,
// row block, kv head) order, are cut into equal ranges, one per thread block.  A
// range boundary inside an item splits its keys: each part is a piece, whose
// unnormalised output and (max, sum) go to a partial slot, and the block that
// arrives last (batch_mma.cu: a second kernel) joins the pieces of an item in key
// order (so results do not depend on the order in which blocks run; the cuts, and
// with them a sequence's last bits, depend on the whole batch).  An item of at most item_cost tiles is not split:
// the block of its first unit takes it whole.
#pragma once

#include <cstdint>

#include "batch.h"
#include "common.cuh"
#include "internal.h"

namespace attn {
namespace plan {

struct SeqInfo {
  int row0;   // first row of the token batch
  int q_len;  // new tokens
  int len;    // cached positions, the new ones included
  int pfx;    // keys below it are visible to every row
};

__device__ __forceinline__ SeqInfo load_seq(const BatchArgs& a, int s) {
  SeqInfo q;
  const uint32_t b = a.q_start[s], e = a.q_start[s + 1], n = a.kv_len[s];
  const bool ok = b <= e && e <= a.total_rows && n <= (uint32_t)a.capacity && n >= e - b;
  if (!ok) record_status(a.status, ATTN_ERR_INVALID_ARG);
  q.row0 = (int)b;
  q.q_len = (b <= e && e <= a.total_rows) ? (int)(e - b) : 0;
  q.len = (int)min(n, (uint32_t)a.capacity);
  q.pfx = a.prefix_len != nullptr ? (int)min(a.prefix_len[s], (uint32_t)q.len) : 0;
  return q;
}

// Token of flattened row f, and the page of a position.
__device__ __forceinline__ int token_of(const BatchArgs& a, int f) { return (int)divide((uint32_t)f, a.by_gs); }
__device__ __forceinline__ int page_of(const BatchArgs& a, int key) { return (int)divide((uint32_t)key, a.by_page); }

// Keys [lo, hi) of the row of token t (empty when hi <= lo).
__device__ __forceinline__ int row_hi(const SeqInfo& q, int t) { return max(q.len - q.q_len + t + 1, q.pfx); }
__device__ __forceinline__ int row_lo(const BatchArgs& a, const SeqInfo& q, int t) {
  const int n = q.len - q.q_len + t + 1;
  return (a.window > 0 && n > a.window) ? n - a.window : 0;
}

// Keys of a block's rows: [0, se) and [lo_min, hi_max), se < lo_min or se == 0.  (SINKS false, here and below: a call
// without first positions, se == 0 everywhere; that in the lookups cost a mixed batch of short pieces 3% of its time.)
struct BlockKeys {
  int lo_min, lo_max, hi_min, hi_max;  // extremes over the rows' windows (lo_min 0 where the first positions reach them)
  int se;                              // end of the first positions in sight of a row
  int ns, skip, nt;                    // tiles: nt in all, the first ns from tile 0 on, the others `skip` later
};
// Key tile of tile t, which the item's tiles are counted from: of the nt (SINKS), or key tiles as they are.
template <bool SINKS>
__device__ __forceinline__ int first_tile(const BlockKeys& k) { return SINKS ? 0 : k.skip; }
template <bool SINKS>
__device__ __forceinline__ int tile_at(int t, int ns, int skip) { return SINKS && t >= ns ? t + skip : t; }
// Can no row see, or can some row see all of, keys [key, key + n)?  (Of one of the two ranges.)
template <bool SINKS>
__device__ __forceinline__ bool keys_hidden(int key, int n, int se, int lo, int hi) {
  return (key + n <= lo || key >= hi) && (!SINKS || key >= se);
}
template <bool SINKS>
__device__ __forceinline__ bool keys_inside(int key, int n, int se, int lo, int hi) {
  return (key >= lo && key + n <= hi) || (SINKS && key + n <= se);
}

template <int ROWS>
__device__ __forceinline__ int row_blocks(const BatchArgs& a, const SeqInfo& q) {
  return (q.q_len * a.gs + ROWS - 1) / ROWS;
}

template <int ROWS, int KEYS, bool SINKS>
__device__ __forceinline__ BlockKeys block_keys(const BatchArgs& a, const SeqInfo& q, int b) {
  const int t0 = token_of(a, b * ROWS);
  const int t1 = token_of(a, min(q.q_len * a.gs, (b + 1) * ROWS) - 1);
  BlockKeys k;
  k.lo_min = row_lo(a, q, t0);
  k.lo_max = row_lo(a, q, t1);
  k.hi_min = row_hi(q, t0);
  k.hi_max = row_hi(q, t1);
  const bool any = k.hi_max > k.lo_min;
  k.se = k.ns = 0;
  if (SINKS) {
    k.se = min(a.sinks, k.lo_max);
    if (k.se >= k.lo_min) k.lo_min = k.se = 0;
  }
  const int kt0 = k.lo_min / KEYS;
  if (SINKS) k.ns = min((k.se + KEYS - 1) / KEYS, kt0);
  k.skip = kt0 - k.ns;
  k.nt = any ? (k.hi_max + KEYS - 1) / KEYS - k.skip : 0;
  return k;
}

// 64-bit quotient; unit counts nearly always fit in 32 bits, where a division takes a quarter of the time.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((unsigned long long)(a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

struct Piece {
  SeqInfo q;
  BlockKeys k;
  int s, b, g;
  int t0, t1;     // tiles [t0, t1) of the item's nt
  int slot;       // partial slot of a piece that is not the whole item
  bool whole;
  // The item's pieces, when there are several: blocks first .. last, the first one's in slot slot0, the others in
  // slot 0.
  int first, last, slot0;
};

// What a block needs to walk its range; written by make_plan.
struct Start {
  long long left;  // units of this block
  long long x;     // offset into the first item
  long long u0;    // the range's first unit
  long long per;   // units per block
  int s, b, g;
};

// Inclusive scan of one value a thread over the whole block; *total gets the sum.
template <int THREADS>
__device__ __forceinline__ long long block_scan(long long v, long long* warp_sums, long long* total) {
  static_assert(THREADS % 32 == 0 && THREADS <= 1024, "whole warps");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();  // warp_sums may still be read by an earlier scan
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const long long x = warp_sums[w];
    if (w < warp) before += x;
    all += x;
  }
  *total = all;
  return v + before;
}

// Range of block c when the items weigh `units` in all.
__device__ __forceinline__ long long units_per_block(long long units, int blocks, int cost) {
  return max(quotient(units + blocks - 1, blocks), (long long)(cost + 1));
}
__device__ __forceinline__ void set_start(Start* start, int s, int b, long long offset, int w, long long u0, long long per,
                                          long long units) {
  start->g = (int)quotient(offset, w);
  start->x = offset - (long long)start->g * w;
  start->s = s;
  start->b = b;
  start->u0 = u0;
  start->per = per;
  start->left = min(per, units - u0);
}

// The plan by one warp, for batches of at most kWarpSeqs sequences with few
// row blocks each (a lane takes consecutive sequences): no block barriers, so a
// single-token step starts about a microsecond sooner.  Returns false (to every
// lane) when the batch is too large for it.
constexpr int kWarpSeqs = 512, kWarpBlocks = 32;
template <int ROWS, int KEYS, bool SINKS>
__device__ __forceinline__ bool warp_plan(const BatchArgs& a, int c, int blocks, Start* start) {
  const int lane = threadIdx.x & 31;
  if (a.n_seqs > kWarpSeqs) return false;
  const int share = (a.n_seqs + 31) / 32;
  const int s0 = min(a.n_seqs, lane * share), s1 = min(a.n_seqs, s0 + share);
  int nb = 0;
  long long mine = 0;
  for (int s = s0; s < s1; ++s) {
    const SeqInfo q = load_seq(a, s);
    const int n = row_blocks<ROWS>(a, q);
    nb += n;
    if (nb <= kWarpBlocks)
      for (int b = 0; b < n; ++b) mine += block_keys<ROWS, KEYS, SINKS>(a, q, b).nt + a.item_cost;
  }
  if (__any_sync(0xffffffffu, nb > kWarpBlocks)) return false;
  mine *= a.G;
  long long upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += o;
  }
  const long long units = __shfl_sync(0xffffffffu, upto, 31);
  const long long per = units_per_block(units, blocks, a.item_cost), u0 = per * c;
  if (lane == 0 && u0 >= units) start->left = 0;
  long long at = upto - mine;
  if (u0 >= at && u0 < upto) {
    bool found = false;
    for (int s = s0; s < s1 && !found; ++s) {
      const SeqInfo q = load_seq(a, s);
      const int n = row_blocks<ROWS>(a, q);
      for (int b = 0; b < n && !found; ++b) {
        const int w = block_keys<ROWS, KEYS, SINKS>(a, q, b).nt + a.item_cost;
        found = u0 < at + (long long)w * a.G;
        if (found) set_start(start, s, b, u0 - at, w, u0, per, units);
        at += (long long)w * a.G;
      }
    }
  }
  return true;
}

// The range of thread block `c` of `blocks`.  Every thread of the block calls it;
// first_block holds n_seqs + 1 ints and warp_sums THREADS/32 values in shared
// memory.  On return (after its final barrier) *start is valid.
template <int ROWS, int KEYS, int THREADS, bool SINKS>
__device__ void make_plan(const BatchArgs& a, int c, int blocks, int* first_block, long long* warp_sums, Start* start) {
  const int tid = threadIdx.x;
  if (tid < 32) {
    const bool done = warp_plan<ROWS, KEYS, SINKS>(a, c, blocks, start);
    if (tid == 0) first_block[0] = done ? 1 : 0;
  }
  __syncthreads();
  if (first_block[0]) return;
  __syncthreads();
  // Row blocks before each sequence.
  long long carry = 0;
  for (int s0 = 0; s0 < a.n_seqs; s0 += THREADS) {
    const int s = s0 + tid;
    const int nb = s < a.n_seqs ? row_blocks<ROWS>(a, load_seq(a, s)) : 0;
    long long sum;
    const long long incl = block_scan<THREADS>(nb, warp_sums, &sum);
    if (s < a.n_seqs) first_block[s] = (int)(carry + incl - nb);
    carry += sum;
  }
  // Sequences that do not overlap have at most total_rows * gs / ROWS + n_seqs blocks. A q_start that goes up and down
  // can give every second sequence all the rows: more blocks than 32 bits count, or than a call should take.
  const bool fits = carry <= (long long)a.total_rows * a.gs / ROWS + a.n_seqs;
  const int n_blk = fits ? (int)carry : 0;
  if (tid == 0) {
    if (!fits) record_status(a.status, ATTN_ERR_INVALID_ARG);
    first_block[a.n_seqs] = n_blk;
    start->left = 0;
  }
  __syncthreads();
  if (!fits) return;
  // Weights of this thread's share of the row blocks (all kv heads of each).
  const int share = (n_blk + THREADS - 1) / THREADS;
  const int i0 = min(n_blk, tid * share), i1 = min(n_blk, i0 + share);
  int s = 0;
  if (i0 < i1) {  // last sequence whose first block is at or before i0
    int lo = 0, hi = a.n_seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first_block[mid] <= i0)
        lo = mid;
      else
        hi = mid;
    }
    s = lo;
  }
  long long mine = 0;
  {
    int ss = s;
    SeqInfo q{};
    int have = -1;
    for (int i = i0; i < i1; ++i) {
      while (first_block[ss + 1] <= i) ++ss;
      if (have != ss) q = load_seq(a, have = ss);
      mine += (long long)(block_keys<ROWS, KEYS, SINKS>(a, q, i - first_block[ss]).nt + a.item_cost) * a.G;
    }
  }
  long long units;
  const long long upto = block_scan<THREADS>(mine, warp_sums, &units);
  const long long per = units_per_block(units, blocks, a.item_cost), u0 = per * c;
  long long at = upto - mine;
  if (u0 >= at && u0 < upto) {  // this thread's share holds the range's start
    int ss = s;
    for (int i = i0; i < i1; ++i) {
      while (first_block[ss + 1] <= i) ++ss;
      const int w = block_keys<ROWS, KEYS, SINKS>(a, load_seq(a, ss), i - first_block[ss]).nt + a.item_cost;
      if (u0 < at + (long long)w * a.G) {
        set_start(start, ss, i - first_block[ss], u0 - at, w, u0, per, units);
        break;
      }
      at += (long long)w * a.G;
    }
  }
  __syncthreads();
}

// The call's tag, one larger (by 2^16) than any before on this workspace.  Each block adds its part of 2^16, once, so
// until the last has all read the same multiple; nothing has to be put back, whatever becomes of the call.
__device__ __forceinline__ unsigned long long begin_call(const BatchArgs& a) {
  const unsigned long long mine = blockIdx.x == 0 ? 65536ull - (gridDim.x - 1) : 1ull;
  return (atomicAdd(a.calls, mine) >> 16) << 16;
}
// One more piece of the item that begins in counter `c`'s block: how many were seen before.  Releases what the thread
// (and those that it is ordered after) wrote, acquires what the earlier pieces' threads did.
__device__ __forceinline__ unsigned piece_arrives(unsigned long long* c, unsigned long long tag) {
  unsigned long long seen;
  asm volatile(
      "red.relaxed.gpu.global.max.u64 [%1], %2;\n\t"
      "atom.acq_rel.gpu.global.add.u64 %0, [%1], 1;"
      : "=l"(seen)
      : "l"(c), "l"(tag)
      : "memory");
  return (unsigned)(seen - tag);
}

// Walks the pieces of a block's range, in order.  Warps of different roles
// walk it independently and see the same pieces.
template <int ROWS, int KEYS, bool SINKS>
struct Walker {
  const BatchArgs& a;
  SeqInfo q;
  long long left, x, u, per;
  int s, b, g, nb, index;

  __device__ __forceinline__ Walker(const BatchArgs& args, const Start& st)
      : a(args), q{}, left(st.left), x(st.x), u(st.u0), per(st.per), s(st.s), b(st.b), g(st.g), nb(0), index(0) {
    if (left > 0) {
      q = load_seq(a, s);
      nb = row_blocks<ROWS>(a, q);
    }
  }

  // The next piece, or false.  `split` (may be nullptr) receives the record of
  // an item that starts here and ends in a later block.
  __device__ __forceinline__ bool next(Piece& p, BatchSplit* split = nullptr) {
    while (left > 0) {
      const BlockKeys k = block_keys<ROWS, KEYS, SINKS>(a, q, b);
      const long long w = k.nt + a.item_cost;
      const long long take = min(left, w - x);
      p.q = q;
      p.k = k;
      p.s = s;
      p.b = b;
      p.g = g;
      const bool one_piece = k.nt <= a.item_cost;
      p.t0 = one_piece ? 0 : (int)max(0ll, x - a.item_cost);
      p.t1 = one_piece ? (x == 0 ? k.nt : 0) : (int)max(0ll, x + take - a.item_cost);
      p.slot = index == 0 ? 0 : 1;
      p.whole = p.t0 == 0 && p.t1 == k.nt;
      const bool have = p.t1 > p.t0 || (k.nt == 0 && x == 0);
      if (!p.whole && have) {
        p.first = (int)quotient(u - x + a.item_cost, per);  // the block that holds tile 0
        p.last = (int)quotient(u - x + w - 1, per);
        p.slot0 = (long long)p.first * per >= u - x ? 0 : 1;  // is the item the first of its first block's range?
      }
      if (split != nullptr && p.t0 == 0 && p.t1 > 0 && p.t1 < k.nt) {
        split->valid = 1;
        split->seq = s;
        split->blk = b;
        split->g = g;
        split->slot0 = p.slot0;
        split->last = p.last;
      }
      ++index;
      x += take;
      u += take;
      left -= take;
      if (x == w) {
        x = 0;
        if (++g == a.G) {
          g = 0;
          if (++b == nb) {
            b = 0;
            do {
              if (++s >= a.n_seqs) {
                left = 0;
                break;
              }
              q = load_seq(a, s);
              nb = row_blocks<ROWS>(a, q);
            } while (nb == 0);
          }
        }
      }
      if (have) return true;
    }
    return false;
  }
};

}  // namespace plan
}  // namespace attn
