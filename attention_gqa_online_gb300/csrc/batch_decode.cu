// batch_decode.cu -- single-token attention of a batch over its pages: the
// operation of batch_mma.cu where each sequence has about one new token, so an
// item has at most 16 rows (the query heads of one kv head) and its time is the
// stream of K and V. D is the head dimension rounded up to 64 or 128 (the
// columns past the head are zeros and not stored).
//
// One block per multiprocessor: four producer warps keep 128 KB of K/V tiles in
// flight (TMA boxes of page parts, 128-byte swizzle; a warp issues one in
// about 100 cycles, so small pages need several) and eight warps consume them,
// tile J by warps 4 (J & 1) .. + 3, 16 keys a warp, or 32 at D = 64, where the
// fixed costs of a 64-key tile outweigh its products (33 sequences, 14 heads
// over 2, window 4096, capped: 28 us with 16 keys a warp, 23 with 32). The 16
// rows fill the M of m16n8k16, whose products cost a fraction of the tile's
// transfer time, so the whole tile's softmax runs on all lanes (on the tcgen05
// kernel the rows would be 4 to 16 of 128 lanes). Each warp keeps its own
// running reference, sum and output in registers: no exchange per tile. The
// reference moves only when a score exceeds it by more than kSlack (log2
// units), so the row maximum is not reduced over lanes on every tile.
//
// At a piece's end the eight states are joined in shared memory, in two steps.
// Pieces of a split item go to the workspace; the block that arrives last (a
// counter per item, which each call numbers anew) joins them in key order, so one launch
// does everything and results do not depend on the order of arrival.
//
// Bound by HBM on large batches: 64 sequences of up to 16384 positions, 8 kv
// heads of 128, read 1.69 GB in 259 us, 6.5 TB/s (96% of a copy's rate; pages of
// 16 rows). A small call is bound by its latency: one sequence of 1536
// positions takes 9.0 us, from launch and plan through the first tiles' trip
// to HBM to the join.
//
// Codes (C8). K's words become fp16 on the way into the products, V's too, whose
// scale joins the key's weight instead. The conversion no longer hides behind the
// stream: the same 64 sequences take 161 us, 5.2 TB/s (issue 43% busy; scales of
// single positions 9% more).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "batch.h"
#include "batch_plan.cuh"
#include "batch_score.cuh"
#include "batch_wait.cuh"
#include "cache8.cuh"
#include "common.cuh"
#include "internal.h"
#include "mma16.cuh"

namespace attn {
namespace {

constexpr int kRows = 16;
// What a piece takes beyond its tiles, in tiles. At 2, 3, 4, 6 one sequence of 1536 positions takes 9.3, 8.9, 9.0, 9.6 us,
// of 8000 13.7, 13.4, 13.0, 12.3; 64 of up to 16384 take 256 to 258.
constexpr int kItemCost = 4;
constexpr int kConsumers = 256, kThreads = kConsumers + 128;
constexpr int kDescs = 4;
constexpr int kRingBytes = 128 * 1024;
constexpr int kMaxStages = 4;

struct DecodeDesc {
  int end, whole, n, tile0, ns, skip;  // tiles tile0 .. tile0 + n - 1 of the item's (plan::tile_at)
  int seq, g, row0, q_len, len, pfx, first_row, rows;
  int lo_min, lo_max, hi_min, hi_max, se;
  int slot, first, last, slot0;
};

template <int D, bool C8>
struct __align__(1024) DecodeSmem {
  // Keys of a warp and of a tile: a tile is 16 KB of K and 16 KB of V either way.  Rows are 128 bytes a chunk (codes: one
  // chunk, at D = 64 half of it zeros).
  static constexpr int chunks = C8 || D == 64 ? 1 : 2;
  static constexpr int warp_keys = chunks == 1 ? 32 : 16, keys = 4 * warp_keys;
  static constexpr int tile_bytes = keys * chunks * 128;  // K or V
  static constexpr int stages = kRingBytes / (2 * tile_bytes);
  // A group waits on every use of its own stages only (a parity wait that skips a phase is no wait).
  static_assert(stages % 2 == 0 && stages <= kMaxStages, "tile J and tile J + stages belong to one group");
  static constexpr int q_stride = D + 8;   // elements; 16 bytes off a multiple of 128: rows start in different banks
  static constexpr int o_stride = D + 8;   // floats
  unsigned char ring[stages][2][tile_bytes];
  float4 scale[kMaxStages][C8 ? keys : 1];  // of a tile's keys: K's scale, log2 of V's, one over V's
  uint16_t q[2][kRows * q_stride];
  float o[4][kRows * o_stride];
  float2 ml[8][kRows];  // reference and sum of each warp's rows
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t q_ready[2], q_free[2];
  uint64_t desc_full[kDescs], desc_free[kDescs];
  DecodeDesc desc[kDescs];
  plan::Start start;
  long long warp_sums[kThreads / 32];
  unsigned long long tag;  // this call's (plan::begin_call)
  int abort;
  int issued[4];  // tiles whose copies each producer warp issued
  int share[4];   // bytes of a tile that are a producer warp's
  int go;       // there is a piece
  int is_last;  // this block joins the item
};

// T: of Q and the result.  C8: K and V are codes of cache8.cuh.
template <typename T, int D, bool C8, bool SINKS, bool BRIEF = false>
__global__ void __launch_bounds__(kThreads, 1)
    batch_decode_kernel(const BatchArgs a, const ScoreMap sc, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_v1, const __grid_constant__ CUtensorMap tm_v8,
                        const int box_rows) {
  using S = DecodeSmem<D, C8>;
  using TO = typename std::conditional<C8, __half, T>::type;  // operands
  constexpr bool kHalf = std::is_same<TO, __half>::value;
  constexpr float kSlack = kHalf ? 8.f : 24.f;  // P <= 2^8 (times 2^7) or 2^24: inside the operand type's range
  constexpr int kKeys = S::keys, kChunkBytes = kKeys * 128;
  constexpr int kTiles = S::warp_keys / 8, kSteps = S::warp_keys / 16;  // n-tiles of a warp's scores, k-steps of P V
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  allow_dependent_launch();
  if (tid == 0) {
    for (int i = 0; i < S::stages; ++i) {
      mbar_init(&sm.full[i], C8 ? 5 : 1);  // the copies; codes: four warps' scales, too
      mbar_init(&sm.empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_ready[i], 1);
      mbar_init(&sm.q_free[i], 8);
    }
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(&sm.desc_full[i], 1);
      mbar_init(&sm.desc_free[i], 11);  // eight consumers, three producers
    }
    sm.abort = 0;
    fence_mbar_init();
  }
  if (tid == kConsumers) prefetch_tmap(&tm_k);
  // Columns of Q past the head stay zeros.
  for (int i = tid; i < 2 * kRows * S::q_stride; i += kThreads) sm.q[0][i] = 0;
  grid_dependency_wait();  // lengths, tables and pages may be the previous kernel's output
  if (tid == 32) sm.tag = plan::begin_call(a);
  plan::make_plan<kRows, S::keys, kThreads, SINKS>(a, blockIdx.x, gridDim.x, reinterpret_cast<int*>(sm.ring[0][0]), sm.warp_sums,
                                          &sm.start);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the plan's scratch is where the tiles land
  __syncthreads();
  // Warps wait as a whole: lanes that left a wait at different times could arrive for, or part from, the others.
  const unsigned long long limit = BRIEF ? a.wait_ns : kWaitLimitNs;
  auto wait = [&](uint64_t* bar, int phase) {
    return warp_wait<BRIEF>(bar, (unsigned)(phase & 1), a.status, &sm.abort, limit);
  };

  if (warp >= kConsumers / 32) {
    // ------------------------------------------------------------ producers
    // Warps 0, 1 fetch K and 2, 3 fetch V: at D = 128 a column chunk each, at D = 64 every other part.  Warp 0 is also
    // the planner and loads Q.
    const int pw = warp - kConsumers / 32, sub = pw & 1;
    const bool is_v = pw >= 2;
    const CUtensorMap* tm = is_v ? &tm_v : &tm_k;
    const int outside = a.num_pages * a.page_rows;  // a row past the pool: arrives as zeros
    const int parts = kKeys / box_rows;             // page parts of a tile, at most 16
    const int parts_log2 = __ffs(parts) - 1;
    const int chunk = S::chunks == 2 ? sub : 0;
    const bool my_part = lane < parts && (S::chunks == 2 || (lane & 1) == sub);
    // Tiles of one piece, from tile number J on.
    auto load_tiles = [&](int n, int seq, int g, int se, int lo, int hi, int tile0, int ns, int skip, int J) {
      // First key of part q.
      auto key_of = [&](int q) {
        if (!SINKS) return tile0 * kKeys + q * box_rows;
        return plan::tile_at<SINKS>(tile0 + (q >> parts_log2), ns, skip) * kKeys + (q & (parts - 1)) * box_rows;
      };
      const uint32_t* table = a.block_table + (long long)seq * a.max_blocks;
      // Pool rows of the page parts, 32 at a time (one a lane), read at least 32 parts ahead.
      auto rows_of = [&](int q0) {
        const int q = q0 + lane, key = key_of(q);
        const bool seen = q < n * parts && !plan::keys_hidden<SINKS>(key, box_rows, se, lo, hi);
        const int col = seen ? plan::page_of(a, key) : 0;
        const uint32_t pg = table[col];  // (no branch around it: two such reads overlap)
        return !seen ? outside : pg < (uint32_t)a.num_pages ? (int)pg * a.page_rows + key - col * a.page_rows : -1;
      };
      int now = rows_of(0), next = n * parts > 32 ? rows_of(32) : outside;
      // Codes: the lane's key of each tile, 32 pw + lane; its scales are looked up a tile ahead (a trip to L2).
      const int box_log2 = __ffs(box_rows) - 1, mine = 32 * pw + lane;
      uint32_t k_byte = 0, v_byte = 0;
      auto look = [&](int rows, int i) {  // rows: of the 32 parts that hold tile i's
        const int row = __shfl_sync(0xffffffffu, rows, (i * parts + (mine >> box_log2)) & 31);
        if (row < 0 || row == outside) return;  // (the codes arrive as zeros)
        const long long b = (long long)divide((uint32_t)(row + (mine & (box_rows - 1))), a.by_scale) * a.G + g;
        k_byte = a.k_scales[b];
        v_byte = a.v_scales[b];
      };
      if constexpr (C8) look(now, 0);
      for (int i = 0; i < n; ++i, ++J) {
        const int q0 = i * parts;
        if (i > 0 && q0 % 32 == 0) {
          now = next;
          next = rows_of(q0 + 32);
        }
        int row = __shfl_sync(0xffffffffu, now, (q0 + lane) % 32);
        if (!my_part) row = outside;
        if (row < 0) {  // a page outside the pool
          record_status(a.status, ATTN_ERR_INVALID_ARG);
          row = outside;
        }
        const int key = key_of(q0) + lane * box_rows, st = J % S::stages;
        // A wait that ran out ends the role: a slot in use must not be written, nor a phase arrived at twice.
        if (J >= S::stages && !wait(&sm.empty[st], J / S::stages - 1)) return J;
        if (pw == 0 && lane == 0) mbar_arrive_expect_tx(&sm.full[st], (unsigned)(2 * S::tile_bytes));
        __syncwarp();
        unsigned char* dst = sm.ring[st][is_v ? 1 : 0] + chunk * kChunkBytes;
        // V rows of a fetched part that lie outside the windows are replaced by zeros (0 * NaN), by eights or single
        // rows.
        const bool edge = is_v && row != outside && !plan::keys_inside<SINKS>(key, box_rows, se, lo, hi);
        if (my_part && !edge) tma_load_3d(dst + lane * box_rows * 128, tm, 64 * chunk, g, row, &sm.full[st]);
        unsigned edges = __ballot_sync(0xffffffffu, edge);
        while (edges) {
          const int e = __ffs(edges) - 1;
          edges &= edges - 1;
          const int row_e = __shfl_sync(0xffffffffu, row, e), key_e = __shfl_sync(0xffffffffu, key, e);
          const int key_8 = key_e + 8 * lane;  // eight rows a lane; those that are not all of one kind, row by row
          const bool inside = plan::keys_inside<SINKS>(key_8, 8, se, lo, hi), outer = plan::keys_hidden<SINKS>(key_8, 8, se, lo, hi);
          if (8 * lane < box_rows && (inside || outer)) {
            const int y = inside ? row_e + 8 * lane : outside;
            tma_load_3d(dst + (e * box_rows + 8 * lane) * 128, &tm_v8, 64 * chunk, g, y, &sm.full[st]);
          }
          unsigned mixed = __ballot_sync(0xffffffffu, 8 * lane < box_rows && !inside && !outer);
          while (mixed) {
            const int r = 8 * (__ffs(mixed) - 1) + lane;
            mixed &= mixed - 1;
            if (lane < 8) {
              const int y = plan::keys_inside<SINKS>(key_e + r, 1, se, lo, hi) ? row_e + r : outside;
              tma_load_3d(dst + (e * box_rows + r) * 128, &tm_v1, 64 * chunk, g, y, &sm.full[st]);
            }
          }
        }
        if constexpr (C8) {
          const int ev = c8::exp_of(v_byte);
          sm.scale[st][mine] = make_float4(pow2f(c8::exp_of(k_byte)), (float)ev, pow2f(-ev), 0.f);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.full[st]);
          if (i + 1 < n) look(((i + 1) * parts) % 32 == 0 ? next : now, i + 1);
        }
      }
      return J;
    };
    int x = 0, J = 0;
    if (pw != 0) {
      if (lane == 0) {
        prefetch_tmap(tm);
        if (is_v) prefetch_tmap(&tm_v1);
      }
      for (;; ++x) {
        const DecodeDesc& d = sm.desc[x % kDescs];
        if (!wait(&sm.desc_full[x % kDescs], x / kDescs) || !warp_whole(&sm.abort) || d.end) break;
        J = load_tiles(d.n, d.seq, d.g, d.se, d.lo_min, d.hi_max, d.tile0, d.ns, d.skip, J);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.desc_free[x % kDescs]);
      }
    }
    plan::Walker<kRows, kKeys, SINKS> walk(a, sm.start);
    plan::Piece p;
    while (pw == 0) {
      const bool more = walk.next(p) && warp_whole(&sm.abort);
      const int first_row = p.b * kRows;
      const int rows = more ? min(kRows, p.q.q_len * a.gs - first_row) : 0;
      if (more && p.t1 == p.t0) {  // rows without keys
        for (int r = 0; r < rows; ++r) {
          const int f = first_row + r, t = plan::token_of(a, f), h = p.g * a.gs + f - t * a.gs;
          T* dst = static_cast<T*>(a.out) + (long long)(p.q.row0 + t) * a.out_stride + (long long)h * a.D;
          if (lane < a.D / 8) *reinterpret_cast<uint4*>(dst + 8 * lane) = make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      if (x >= kDescs && !wait(&sm.desc_free[x % kDescs], x / kDescs - 1)) break;
      if (lane == 0) {
        DecodeDesc& d = sm.desc[x % kDescs];
        d.end = !more;
        if (more) {
          d.whole = p.whole;
          d.n = p.t1 - p.t0;
          d.tile0 = plan::first_tile<SINKS>(p.k) + p.t0;
          d.ns = p.k.ns;
          d.skip = p.k.skip;
          d.se = p.k.se;
          d.seq = p.s;
          d.g = p.g;
          d.row0 = p.q.row0;
          d.q_len = p.q.q_len;
          d.len = p.q.len;
          d.pfx = p.q.pfx;
          d.first_row = first_row;
          d.rows = rows;
          d.lo_min = p.k.lo_min;
          d.lo_max = p.k.lo_max;
          d.hi_min = p.k.hi_min;
          d.hi_max = p.k.hi_max;
          d.slot = p.slot;
          d.first = p.first;
          d.last = p.last;
          d.slot0 = p.slot0;
        }
        mbar_arrive(&sm.desc_full[x % kDescs]);
      }
      __syncwarp();
      if (!more) break;
      // Q rows, one copy each.
      if (x >= 2 && !wait(&sm.q_free[x & 1], (x >> 1) - 1)) break;
      if (lane == 0) mbar_arrive_expect_tx(&sm.q_ready[x & 1], (unsigned)(rows * a.D * 2));
      __syncwarp();
      if (lane < rows) {
        const int f = first_row + lane, t = plan::token_of(a, f), h = p.g * a.gs + f - t * a.gs;
        bulk_g2s(&sm.q[x & 1][lane * S::q_stride],
                 static_cast<const T*>(a.q) + (long long)(p.q.row0 + t) * a.q_stride + (long long)h * a.D, a.D * 2,
                 &sm.q_ready[x & 1]);
      }
      J = load_tiles(p.t1 - p.t0, p.s, p.g, p.k.se, p.k.lo_min, p.k.hi_max, plan::first_tile<SINKS>(p.k) + p.t0,
                     p.k.ns, p.k.skip, J);
      ++x;
      if (!warp_whole(&sm.abort)) break;
    }
    const int share = __popc(__ballot_sync(0xffffffffu, my_part)) * box_rows * 128;
    if (lane == 0) {
      sm.issued[pw] = J;
      sm.share[pw] = share;
    }
    __syncwarp();
    named_barrier(2, kThreads);
    // No copy may still be landing in shared memory when the block exits.  The consumers have read every tile, unless
    // the pipeline broke.  Then some producers may have issued a tile that others have not: its barrier was armed for
    // all of them, or not at all.  (They are at most a ring apart, since a slot falls free when a whole tile is read.)
    if (*(volatile int*)&sm.abort != 0 && tid == kConsumers) {
      int lo = J, hi = J;
      for (int w = 1; w < 4; ++w) {
        lo = min(lo, sm.issued[w]);
        hi = max(hi, sm.issued[w]);
      }
      for (int j = lo; j < hi; ++j) {
        unsigned missing = 0;
        for (int w = 0; w < 4; ++w) missing += sm.issued[w] <= j ? sm.share[w] : 0;
        settle_tile(&sm.full[j % S::stages], J > j, 2 * S::tile_bytes, missing);
        for (int w = 0; C8 && w < 4; ++w)
          if (sm.issued[w] <= j) mbar_arrive(&sm.full[j % S::stages]);
      }
      drain_ring(sm.full, S::stages, hi, a.status);
      drain_ring(sm.q_ready, 2, x, a.status);
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int grp = warp >> 2, kw = S::warp_keys * (warp & 3);  // group, and the warp's first key of the tile
  const int lr = lane >> 2, lc = 2 * (lane & 3);
  int J = 0;
  for (int x = 0;; ++x) {
    const DecodeDesc& d = sm.desc[x % kDescs];
    // One thread decides for all whether there is a piece: the warps meet at barriers that none may miss.  (The
    // joining buffers are free again after this barrier, too.)
    if (tid == 0)
      sm.go = wait_phase<BRIEF>(&sm.desc_full[x % kDescs], (unsigned)(x / kDescs & 1), a.status, &sm.abort, limit) &&
              *(volatile int*)&sm.abort == 0 && !d.end;
    __syncwarp();
    named_barrier(1, kConsumers);
    if (!sm.go) break;
    const int n = d.n, rows = d.rows;
    // This thread's rows lr and lr + 8 (past the piece's: no keys).
    int lo[2], hi[2], pos[2];
    float slope[2], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = lr + 8 * e, f = d.first_row + min(r, rows - 1), t = plan::token_of(a, f);
      const plan::SeqInfo q{d.row0, d.q_len, d.len, d.pfx};
      lo[e] = plan::row_lo(a, q, t);
      hi[e] = r < rows ? plan::row_hi(q, t) : 0;
      pos[e] = d.len - d.q_len + t;
      slope[e] = a.slopes != nullptr ? -kLog2e * a.slopes[d.g * a.gs + f - t * a.gs] : 0.f;
    }
    const int lo_max = d.lo_max, hi_min = rows < kRows ? 0 : d.hi_min;
    bool ok = wait(&sm.q_ready[x & 1], x >> 1);
    // Codes: a lane's word of a row of K is four columns, so its columns of a step are 4 (lane % 4) + 0 .. 3.
    uint32_t qa[D / 16][4];
    {
      const uint16_t* q = sm.q[x & 1] + (C8 ? 2 * lc : lc);
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          qa[c][e] = *reinterpret_cast<const uint32_t*>(q + (lr + 8 * (e & 1)) * S::q_stride + 16 * c +
                                                        (C8 ? 2 : 8) * (e >> 1));
    }
    __syncwarp();
    float qf[2] = {1.f, 1.f};  // powers of two that came off the rows; without a cap, with the scores' scale
    if constexpr (C8 && !std::is_same<T, __half>::value) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float big = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) big = max3(big, q16::largest2(qa[c][h]), q16::largest2(qa[c][2 + h]));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        const int E = pow2_scale_exp(big);
        const float mul = pow2f(14 - E);
        qf[h] = pow2f(E - 14);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          qa[c][h] = q16::to_half2(qa[c][h], mul);
          qa[c][2 + h] = q16::to_half2(qa[c][2 + h], mul);
        }
      }
    }
    if (C8 && !(a.softcap > 0.f)) {
      qf[0] *= sc.scale2;
      qf[1] *= sc.scale2;
    }
    // (After a wait that ran out a warp frees no slot any more, since copies may still be landing there, but keeps to
    // the block's barriers until the next piece.)
    if (ok && lane == 0) mbar_arrive(&sm.q_free[x & 1]);
    float o[D / 8][4];
#pragma unroll
    for (int c = 0; c < D / 8; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c][e] = 0.f;

    for (int i = (J & 1) ^ grp; ok && i < n; i += 2) {
      const int j = J + i, st = j % S::stages;
      ok = wait(&sm.full[st], j / S::stages);
      if (!ok) break;
      const uint32_t k_base = smem_u32(sm.ring[st][0]), v_base = smem_u32(sm.ring[st][1]);
      // Codes: V's scale 2^v of a key joins its score, so weights are p 2^v against the largest of these and V stays as it
      // is; sums of p take 2^-v off again.
      float4 ks[C8 ? kTiles : 1][2];  // of the keys 8 y + lc + {0, 1}
      // With two n-tiles, even and odd column steps accumulate apart: the chain of dependent products is half as long.
      constexpr int kSets = kTiles == 2 ? 2 : 1;
      float s[kTiles][4], s1[kTiles][4];
#pragma unroll
      for (int y = 0; y < kTiles; ++y)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[y][e] = s1[y][e] = 0.f;
      if constexpr (C8) {
        // Eight keys, four steps of 16 columns: a lane's four words are its columns of each.
#pragma unroll
        for (int y = 0; y < kTiles; ++y)
#pragma unroll
          for (int c4 = 0; c4 < D / 64; ++c4) {
            const int r = kw + 8 * y + (lane & 7), u = 4 * c4 + (lane >> 3);
            uint32_t kb[4];
            ldsm4(kb, k_base + r * 128 + 16 * (u ^ (r & 7)));
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t b0, b1;
              c8::to_half4(kb[c], b0, b1);
              mma16816<TO>(s[y], qa[4 * c4 + c], b0, b1);
            }
          }
      } else
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
#pragma unroll
        for (int g = 0; g < kSteps; ++g) {  // 16 keys
          const int r = kw + 16 * g + (lane & 7) + 8 * (lane >> 4), u = 2 * (c & 3) + ((lane >> 3) & 1);
          uint32_t kb[4];
          ldsm4(kb, k_base + (c >> 2) * kChunkBytes + r * 128 + 16 * (u ^ (r & 7)));
          mma16816<TO>(c % kSets ? s1[2 * g] : s[2 * g], qa[c], kb[0], kb[1]);
          mma16816<TO>(c % kSets ? s1[2 * g + 1] : s[2 * g + 1], qa[c], kb[2], kb[3]);
        }
      }
      if (kSets == 2) {
#pragma unroll
        for (int y = 0; y < kTiles; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[y][e] += s1[y][e];
      }
      if constexpr (C8) {
#pragma unroll
        for (int y = 0; y < kTiles; ++y) {
          ks[y][0] = sm.scale[st][kw + 8 * y + lc];
          ks[y][1] = sm.scale[st][kw + 8 * y + lc + 1];
#pragma unroll
          for (int e = 0; e < 4; ++e) s[y][e] *= ks[y][e & 1].x * qf[e >> 1];
        }
      }
      const int tile_key = plan::tile_at<SINKS>(d.tile0 + i, d.ns, d.skip) * kKeys, key0 = tile_key + kw + lc;
      if (a.softcap > 0.f) {
#pragma unroll
        for (int y = 0; y < kTiles; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[y][e] = sc.out_mul * tanh_score(s[y][e] * sc.in_mul);
      } else if (!C8) {
#pragma unroll
        for (int y = 0; y < kTiles; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[y][e] *= sc.scale2;
      }
      if (a.slopes != nullptr) {
#pragma unroll
        for (int y = 0; y < kTiles; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[y][e] = fmaf(slope[e >> 1], fabsf((float)(pos[e >> 1] - (key0 + 8 * y + (e & 1)))), s[y][e]);
      }
      if constexpr (C8) {
#pragma unroll
        for (int y = 0; y < kTiles; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[y][e] += ks[y][e & 1].y;
      }
      if (tile_key + kKeys > hi_min || tile_key < lo_max) {
#pragma unroll
        for (int y = 0; y < kTiles; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + 8 * y + (e & 1);
            if (key >= hi[e >> 1] || (key < lo[e >> 1] && (!SINKS || key >= a.sinks))) s[y][e] = -INFINITY;
          }
      }
      float t[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int y = 0; y < kTiles; ++y)
#pragma unroll
        for (int h = 0; h < 2; ++h) t[h] = max3(t[h], s[y][2 * h], s[y][2 * h + 1]);
      if (__any_sync(0xffffffffu, t[0] > m[0] + kSlack || t[1] > m[1] + kSlack)) {  // some reference moves
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          t[h] = fmaxf(t[h], __shfl_xor_sync(0xffffffffu, t[h], 1));
          t[h] = fmaxf(t[h], __shfl_xor_sync(0xffffffffu, t[h], 2));
          const float mn = fmaxf(m[h], t[h]), f = mn == m[h] ? 1.f : ex2(m[h] - mn);
          m[h] = mn;
          l[h] *= f;
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            o[c][2 * h] *= f;
            o[c][2 * h + 1] *= f;
          }
        }
      }
      constexpr float kHead = kHalf ? kF16Head : 0.f;
      const float sub[2] = {m[0] == -INFINITY ? 0.f : m[0] - kHead, m[1] == -INFINITY ? 0.f : m[1] - kHead};
#pragma unroll
      for (int y = 0; y < kTiles; ++y)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[y][e] = ex2(s[y][e] - sub[e >> 1]);
          if constexpr (C8)
            l[e >> 1] = fmaf(s[y][e], ks[y][e & 1].z, l[e >> 1]);
          else
            l[e >> 1] += s[y][e];
        }
#pragma unroll
      for (int g = 0; g < kSteps; ++g) {
        const uint32_t pa[4] = {pack2<TO>(s[2 * g][0], s[2 * g][1]), pack2<TO>(s[2 * g][2], s[2 * g][3]),
                                pack2<TO>(s[2 * g + 1][0], s[2 * g + 1][1]), pack2<TO>(s[2 * g + 1][2], s[2 * g + 1][3])};
        if constexpr (C8) {
          // A transposed word is two neighbouring columns of two keys; their even columns make one product, the odd ones
          // another: o[2 u] and o[2 u + 1] hold columns 16 u + 2 n and 16 u + 2 n + 1.
#pragma unroll
          for (int u2 = 0; u2 < D / 32; ++u2) {
            const int r = kw + 16 * g + (lane & 15), u = 2 * u2 + (lane >> 4);
            uint32_t vb[4];
            ldsm4_t(vb, v_base + r * 128 + 16 * (u ^ (r & 7)));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t even0, odd0, even1, odd1;
              c8::to_half4(__byte_perm(vb[2 * e], 0, 0x3120), even0, odd0);
              c8::to_half4(__byte_perm(vb[2 * e + 1], 0, 0x3120), even1, odd1);
              mma16816<TO>(o[4 * u2 + 2 * e], pa, even0, even1);
              mma16816<TO>(o[4 * u2 + 2 * e + 1], pa, odd0, odd1);
            }
          }
        } else
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const int r = kw + 16 * g + (lane & 15), u = 2 * (c & 3) + (lane >> 4);
          uint32_t vb[4];
          ldsm4_t(vb, v_base + (c >> 2) * kChunkBytes + r * 128 + 16 * (u ^ (r & 7)));
          mma16816<TO>(o[2 * c], pa, vb[0], vb[1]);
          mma16816<TO>(o[2 * c + 1], pa, vb[2], vb[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[st]);
    }
    J += n;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }

    // Join of the eight warps: warps 4-7 hand over to 0-3, then four states are summed by all threads.
    auto put = [&](int w) {
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float* row = &sm.o[w][(lr + 8 * h) * S::o_stride];
          if constexpr (!C8)
            *reinterpret_cast<float2*>(row + 8 * c + lc) = make_float2(o[c][2 * h], o[c][2 * h + 1]);
          else if (c % 2 == 0)
            *reinterpret_cast<float4*>(row + 8 * c + 2 * lc) =
                make_float4(o[c][2 * h], o[c + 1][2 * h], o[c][2 * h + 1], o[c + 1][2 * h + 1]);
        }
      if ((lane & 3) == 0) {
        sm.ml[w][lr] = make_float2(m[0], l[0]);
        sm.ml[w][lr + 8] = make_float2(m[1], l[1]);
      }
    };
    if (warp >= 4) put(warp - 4);
    named_barrier(1, kConsumers);
    if (warp < 4) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 other = sm.ml[warp][lr + 8 * h];
        const float mn = fmaxf(m[h], other.x);
        const float f0 = l[h] == 0.f ? 0.f : ex2(m[h] - mn), f1 = other.y == 0.f ? 0.f : ex2(other.x - mn);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const float* row = &sm.o[warp][(lr + 8 * h) * S::o_stride];
          if constexpr (!C8) {
            const float2 v = *reinterpret_cast<const float2*>(row + 8 * c + lc);
            o[c][2 * h] = o[c][2 * h] * f0 + v.x * f1;
            o[c][2 * h + 1] = o[c][2 * h + 1] * f0 + v.y * f1;
          } else if (c % 2 == 0) {
            const float4 v = *reinterpret_cast<const float4*>(row + 8 * c + 2 * lc);
            o[c][2 * h] = o[c][2 * h] * f0 + v.x * f1;
            o[c + 1][2 * h] = o[c + 1][2 * h] * f0 + v.y * f1;
            o[c][2 * h + 1] = o[c][2 * h + 1] * f0 + v.z * f1;
            o[c + 1][2 * h + 1] = o[c + 1][2 * h + 1] * f0 + v.w * f1;
          }
        }
        l[h] = l[h] * f0 + other.y * f1;
        m[h] = mn;
      }
      __syncwarp();
      put(warp);
    }
    named_barrier(1, kConsumers);
    constexpr int kPerRow = D / 8;  // threads of a row, eight columns each
    const int r = tid / kPerRow, c0 = 8 * (tid % kPerRow);
    const bool mine = tid < kRows * kPerRow && r < rows;
    const bool inside = c0 < a.D;  // the others are columns past the head
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, m_all = -INFINITY, l_all = 0.f;
    // Adds state (m, l, eight columns) to the thread's.
    auto add = [&](float2 ml, float4 v0, float4 v1) {
      if (ml.y == 0.f) return;  // none of the row's keys
      const float mn = fmaxf(m_all, ml.x);
      const float f0 = l_all == 0.f ? 0.f : ex2(m_all - mn), f1 = ex2(ml.x - mn);
      const float w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = acc[k] * f0 + w[k] * f1;
      l_all = l_all * f0 + ml.y * f1;
      m_all = mn;
    };
    auto store = [&]() {
      const float inv = l_all == 0.f ? 0.f : 1.f / l_all;
      const int f = d.first_row + r, t = plan::token_of(a, f), h = d.g * a.gs + f - t * a.gs;
      T* dst = static_cast<T*>(a.out) + (long long)(d.row0 + t) * a.out_stride + (long long)h * a.D + c0;
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = l_all == 0.f ? 0u : pack2<T>(acc[2 * k] * inv, acc[2 * k + 1] * inv);
      if (inside) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    };
    if (mine) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float4* v = reinterpret_cast<const float4*>(&sm.o[w][r * S::o_stride + c0]);
        add(sm.ml[w][r], v[0], v[1]);
      }
    }
    if (d.whole) {
      if (mine) store();
    } else {
      constexpr long long kSlotFloats = kRows * (D + 2);
      float* part = a.partial + (2ll * blockIdx.x + d.slot) * kSlotFloats;
      if (mine) {
        *reinterpret_cast<float4*>(part + r * D + c0) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        *reinterpret_cast<float4*>(part + r * D + c0 + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (c0 == 0) *reinterpret_cast<float2*>(part + kRows * D + 2 * r) = make_float2(m_all, l_all);
      }
      named_barrier(1, kConsumers);
      if (tid == 0) {
        // Releases the block's part (its writes are ordered before by the barrier) and acquires the others'.
        sm.is_last = plan::piece_arrives(a.arrived + d.first, sm.tag) == (unsigned)(d.last - d.first);
      }
      named_barrier(1, kConsumers);
      if (sm.is_last && mine) {
        m_all = -INFINITY;
        l_all = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = 0.f;
        // Eight pieces' loads at a time: one by one each would wait for its own trip to L2 (one sequence of 8000
        // positions, 19 pieces an item: 19.4 us, 13.0 this way).
        const int first = d.first, last = d.last, slot0 = d.slot0;
#pragma unroll 1
        for (int c8 = first; c8 <= last; c8 += 8) {
          float2 ml[8];
          float4 v[8][2];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int c = min(c8 + i, last);
            const float* q = a.partial + (2ll * c + (c == first ? slot0 : 0)) * kSlotFloats;
            ml[i] = __ldcg(reinterpret_cast<const float2*>(q + kRows * D + 2 * r));
            v[i][0] = __ldcg(reinterpret_cast<const float4*>(q + r * D + c0));
            v[i][1] = __ldcg(reinterpret_cast<const float4*>(q + r * D + c0 + 4));
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c8 + i <= last) add(ml[i], v[i][0], v[i][1]);
        }
        store();
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.desc_free[x % kDescs]);
  }
  __syncwarp();
  named_barrier(2, kThreads);  // the producers wait for the last tiles' readers
}

template <typename T, int D, bool C8>
int launch_decode_t(const BatchArgs& a, int blocks, int box_rows, cudaStream_t s) {
  using S = DecodeSmem<D, C8>;
  if (box_rows > S::keys) box_rows = S::keys;
  // K and V: [rows][G][head_dim]; columns past the head (head_dim < D) arrive as zeros.  16-bit elements are only moved:
  // one element type serves both, and pairs of codes.
  constexpr int kBytes = C8 ? 1 : 2;
  const uint64_t dims[3] = {(uint64_t)a.D * kBytes / 2, (uint64_t)a.G, (uint64_t)a.num_pages * a.page_rows};
  const uint64_t strides[2] = {(uint64_t)a.D * kBytes, (uint64_t)a.kv_dim * kBytes};
  const uint32_t box[3] = {64, 1, (uint32_t)box_rows}, one_row[3] = {64, 1, 1}, eight[3] = {64, 1, 8};
  CUtensorMap tm_k, tm_v, tm_v1, tm_v8;
  const int l2 = kv_l2_bytes(a.D * kBytes / 2);
  if (!make_tmap(&tm_k, a.k_pages, 3, dims, strides, box, true, kSwizzle128, l2) ||
      !make_tmap(&tm_v, a.v_pages, 3, dims, strides, box, true, kSwizzle128, l2) ||
      !make_tmap(&tm_v8, a.v_pages, 3, dims, strides, eight, true, kSwizzle128, l2) ||
      !make_tmap(&tm_v1, a.v_pages, 3, dims, strides, one_row, true, kSwizzle128, l2))
    return ATTN_ERR_CUDA;
  auto of_form = [&](auto brief) {
    constexpr bool B = decltype(brief)::value;
    if (C8 || a.sinks > 0) return reinterpret_cast<const void*>(batch_decode_kernel<T, D, C8, true, B>);
    return reinterpret_cast<const void*>(batch_decode_kernel<T, D, C8, C8, B>);  // (codes have one form)
  };
  const void* kern = of_form(std::false_type{});
  if constexpr (std::is_same<T, __nv_bfloat16>::value)  // the failure-path test
    if (a.wait_ns != 0) kern = of_form(std::true_type{});
  const size_t smem = sizeof(S) + 1024;
  if (!set_smem_limit(kern, smem)) return ATTN_ERR_CUDA;
  BatchArgs aa = a;
  aa.item_cost = kItemCost;
  ScoreMap sc = score_map(a);
  void* args[] = {&aa, &sc, &tm_k, &tm_v, &tm_v1, &tm_v8, &box_rows};
  return launch_pdl(kern, dim3(blocks), dim3(kThreads), smem, s, args) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

template <bool C8>
int launch_decode(const BatchArgs& a, int dtype, int blocks, int box_rows, cudaStream_t s) {
  if (dtype == ATTN_DT_BF16)
    return a.D <= 64 ? launch_decode_t<__nv_bfloat16, 64, C8>(a, blocks, box_rows, s)
                     : launch_decode_t<__nv_bfloat16, 128, C8>(a, blocks, box_rows, s);
  return a.D <= 64 ? launch_decode_t<__half, 64, C8>(a, blocks, box_rows, s)
                   : launch_decode_t<__half, 128, C8>(a, blocks, box_rows, s);
}

}  // namespace

int launch_batch_decode(const BatchArgs& a, int dtype, int blocks, int box_rows, cudaStream_t s) {
  return a.k_scales != nullptr ? launch_decode<true>(a, dtype, blocks, box_rows, s)
                               : launch_decode<false>(a, dtype, blocks, box_rows, s);
}

}  // namespace attn
