// batch_tc.cuh -- attention of each sequence's new tokens over its pages on
// the tcgen05 tensor cores (D = 64 or 128, pages of whole 8-row groups).
//
// The operation and the division of work are those of batch_mma.cu and
// batch_plan.cuh; here a row block is 128 flattened rows (the M of one MMA)
// and a key tile 128 keys.  One persistent block per multiprocessor walks its
// range of pieces, and every stage runs ahead across piece borders: while the last tiles of
// one piece are in the softmax, the next piece's Q block, K tiles and first
// scores are already being made.
//
// Warp roles (384 threads; three warpgroups, so registers can be split):
//   warp 0      K producer: one TMA box per page part and 64-column chunk
//               (lane l takes the l-th part; a part no row of the block sees is
//               fetched from outside the pool, which arrives as zeros)
//   warp 1      issues both products of every tile, S_(J+2) = Q K^T before O += P_J V
//   warp 2      V producer
//   warp 3      planner: walks the pieces, writes their descriptors into a
//               four-deep ring, and loads each piece's Q block (two buffers)
//   warps 4-7,
//   warps 8-11  softmax groups 0 and 1: tile J (counted over all pieces of
//               the block) belongs to group J & 1; a thread owns a whole row
// Tensor memory (512 columns): S_b [128 b, +128), P_b [256 + 64 b, +64), b = J & 1,
// O [384, +D).
//
// Softmax.  P is taken against a reference that moves to the tile's maximum only
// when that exceeds it by more than kRescale (log2 units), so O is rarely
// rescaled; the reference passes from tile to tile between the two groups,
// and each group sums its own tiles' P in fp32.  P is rounded to the operand
// type of V (bf16 <= 2^24, fp16 <= 2^8; both operands of an MMA share a type):
// an error of half a step per weight, linear in the output.
//
// End of a piece.  The group that owns the last tile reads its half of O's
// columns as soon as P V lands; the other group first does the next piece's first
// tile, so the exponentials continue.  The next piece's first P V waits for
// both reads.  A whole item is normalised and stored in the output's type, a split
// one goes to its partial slot in fp32.
//
// Rows of V that lie in a fetched page part but outside the block's windows
// hold whatever the page holds; the issuing warp zeroes them in shared memory
// (0 * NaN would reach every row).  The same rows of K only make scores that are masked.
//
// Every wait is bounded; a block whose pipeline breaks drains its copies and
// MMAs, frees its tensor memory and leaves the status word set.
#pragma once

#include <cfloat>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "batch.h"
#include "batch_plan.cuh"
#include "batch_score.cuh"
#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace attn {
namespace {

constexpr int kTcRows = 128, kTcKeys = 128, kTcThreads = 384;
constexpr int kDescs = 4;        // piece descriptors in flight
constexpr int kChain = 4;        // reference maxima in flight
constexpr int kPColumn = 256, kOColumn = 384;
constexpr int kMaxSlots = 4;     // K (and V) tiles in flight, at most
// Registers: 128 threads * 104 + 256 * 200 = 384 * 168, the block's allocation at launch.
constexpr int kCtrlRegs = 104, kSoftmaxRegs = 200;

// A piece as the roles see it.
struct PieceDesc {
  int end;         // no more pieces
  int whole;       // the item's only piece
  int seq, g, slot;
  int row0, q_len, len, pfx, blk;
  int rows;        // valid rows of the block
  int lo_min, lo_max, hi_min, hi_max;
  int tile0, n;    // key tiles tile0 .. tile0 + n - 1 of the sequence
};

template <int D>
struct TcLayout {
  static constexpr int chunks = D / 64;               // 128-byte column chunks of a row
  static constexpr int chunk_bytes = 128 * 128;       // 128 rows of one chunk
  static constexpr int tile_bytes = chunks * chunk_bytes;
  static constexpr int slots = D == 128 ? 2 : 4;      // K tiles (and V tiles) in flight
  static constexpr int operand_bytes = (2 + 2 * slots) * tile_bytes;
};

template <int D>
struct __align__(1024) TcSmem {
  unsigned char q[2][TcLayout<D>::tile_bytes];
  unsigned char k[TcLayout<D>::slots][TcLayout<D>::tile_bytes];
  unsigned char v[TcLayout<D>::slots][TcLayout<D>::tile_bytes];
  uint64_t k_full[kMaxSlots], k_empty[kMaxSlots], v_full[kMaxSlots], v_empty[kMaxSlots];
  uint64_t q_ready[2], q_free[2];
  uint64_t desc_full[kDescs], desc_free[kDescs];
  uint64_t s_full[2], s_free[2], p_ready[2], pv_done[2];
  uint64_t chain_bar[4][kChain];  // [row quarter][J & 3]
  uint64_t stat_bar[4][2][2];     // [row quarter][piece & 1][group]
  uint64_t o_free;                // both groups have read O
  uint64_t drain;
  float chain[kChain][kTcRows];
  float2 stat[2][2][kTcRows];  // [piece & 1][group][row]: reference, sum
  PieceDesc desc[kDescs];
  plan::Start start;
  long long warp_sums[kTcThreads / 32];
  uint32_t tmem_base;
  int abort;
};

template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  return std::is_same<T, __half>::value ? tc::pack_f16(lo, hi) : tc::pack_bf16(lo, hi);
}

// MODE 0: scores are scale2 * S with scale2 > 0 (folded into the exponent's
// fma); 1: scaled, with an optional distance bias; 2: capped, with an optional
// distance bias.
template <typename T, int D, int MODE>
__global__ void __launch_bounds__(kTcThreads, 1)
    batch_tc_kernel(const BatchArgs a, const ScoreMap sc, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_q,
                    const int box_rows, const int q_box) {
  using L = TcLayout<D>;
  constexpr bool kHalf = std::is_same<T, __half>::value;
  constexpr float kRescale = kHalf ? 8.f : 24.f;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  TcSmem<D>& sm = *reinterpret_cast<TcSmem<D>*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  allow_dependent_launch();
  if (warp == 0) {
    for (int i = lane; i < kMaxSlots; i += 32) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_full[i], 1);
      mbar_init(&sm.v_empty[i], 1);
    }
    if (lane < 2) {
      mbar_init(&sm.q_ready[lane], 1);
      mbar_init(&sm.q_free[lane], 1);
      mbar_init(&sm.s_full[lane], 1);
      mbar_init(&sm.s_free[lane], 4);
      mbar_init(&sm.p_ready[lane], 4);
      mbar_init(&sm.pv_done[lane], 1);
    }
    if (lane < kDescs) {
      mbar_init(&sm.desc_full[lane], 1);
      mbar_init(&sm.desc_free[lane], 11);  // K, MMA, V warps and eight softmax warps
    }
    if (lane < 16) {
      mbar_init(&sm.chain_bar[lane >> 2][lane & 3], 1);
      mbar_init(&sm.stat_bar[lane >> 2][(lane >> 1) & 1][lane & 1], 1);
    }
    if (lane == 31) {
      mbar_init(&sm.o_free, 8);
      mbar_init(&sm.drain, 1);
      sm.abort = 0;
    }
    fence_mbar_init();
  }
  if (warp == 1) tc::tmem_alloc(&sm.tmem_base, 512);
  // Lengths, tables and pages may be the previous kernel's output.
  grid_dependency_wait();
  plan::make_plan<kTcRows, kTcKeys, kTcThreads>(a, blockIdx.x, gridDim.x, reinterpret_cast<int*>(sm.q[0]), sm.warp_sums,
                                                &sm.start);
  // The plan's scratch is where Q and the K/V tiles land.
  fence_async_smem();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sm.tmem_base;
  auto wait = [&](uint64_t* bar, int phase) { return mbar_wait_bounded(bar, (unsigned)(phase & 1), a.status, &sm.abort); };
  // Descriptor of piece x (its slot stays valid until every role has released it).
  auto piece = [&](int x) -> const PieceDesc& {
    wait(&sm.desc_full[x % kDescs], x / kDescs);
    return sm.desc[x % kDescs];
  };

  if (warp < 4) {
    regs_dec<kCtrlRegs>();
    if (warp == 0 || warp == 2) {
      // ---------------------------------------------------------- K and V producers
      const bool is_v = warp == 2;
      const CUtensorMap* tm = is_v ? &tm_v : &tm_k;
      unsigned char* ring = is_v ? &sm.v[0][0] : &sm.k[0][0];
      uint64_t* full = is_v ? sm.v_full : sm.k_full;
      uint64_t* empty = is_v ? sm.v_empty : sm.k_empty;
      if (lane == 0) prefetch_tmap(tm);
      const int parts = kTcKeys / box_rows;
      const int outside = a.num_pages * a.page_rows;  // a row past the pool: arrives as zeros
      int J = 0;
      for (int x = 0; !*(volatile int*)&sm.abort; ++x) {
        const PieceDesc& d = piece(x);
        if (d.end || *(volatile int*)&sm.abort) break;
        const uint32_t* table = a.block_table + (long long)d.seq * a.max_blocks;
        const int lo = d.lo_min, hi = d.hi_max, col = d.g * D, n = d.n, tile0 = d.tile0;
        for (int i = 0; i < n; ++i, ++J) {
          int row = outside;
          const int key = (tile0 + i) * kTcKeys + lane * box_rows;
          if (lane < parts && key < hi && key + box_rows > lo) {
            const uint32_t pg = table[key / a.page_rows];
            if (pg < (uint32_t)a.num_pages)
              row = (int)pg * a.page_rows + key % a.page_rows;
            else
              record_status(a.status, ATTN_ERR_INVALID_ARG);
          }
          const int slot = J % L::slots, use = J / L::slots;
          if (use >= 1) wait(&empty[slot], use - 1);
          if (lane == 0) mbar_arrive_expect_tx(&full[slot], (unsigned)L::tile_bytes);
          __syncwarp();
          if (lane < parts) {
            unsigned char* dst = ring + slot * L::tile_bytes + lane * box_rows * 128;
#pragma unroll
            for (int c = 0; c < L::chunks; ++c)
              tma_load_2d(dst + c * L::chunk_bytes, tm, col + 64 * c, row, &full[slot]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.desc_free[x % kDescs]);
      }
      // No copy may still be landing in shared memory when the block exits.
      for (int s = 0; s < L::slots && s < J; ++s) {
        const int last = s + ((J - 1 - s) / L::slots) * L::slots;
        mbar_wait_bounded(&full[s], (unsigned)((last / L::slots) & 1), a.status);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issue
      constexpr uint32_t fmt = kHalf ? tc::kFmtF16 : tc::kFmtBF16;
      constexpr uint32_t idesc_qk = tc::idesc_f32acc(fmt, false, kTcRows, kTcKeys);
      constexpr uint32_t idesc_pv = tc::idesc_f32acc(fmt, true, kTcRows, D);
      const uint64_t dq0 = tc::sdesc_sw128(smem_u32(sm.q[0]), 16, 1024);
      const uint64_t dk0 = tc::sdesc_sw128(smem_u32(sm.k[0]), 16, 1024);
      const uint64_t dv0 = tc::sdesc_sw128(smem_u32(sm.v[0]), L::chunk_bytes, 1024);
      constexpr uint64_t tile16 = L::tile_bytes >> 4;
      auto wait_all = [&](uint64_t* bar, int phase) { return __all_sync(0xffffffffu, wait(bar, phase)); };
      int jq = 0, xq = 0, iq = 0, nq = 0;  // the next Q K^T: tile jq, the iq-th of piece xq
      bool more_q = true, ok = true;
      auto issue_qk = [&]() {
        if (!more_q || !ok) return;
        if (iq == 0) {
          const PieceDesc& d = piece(xq);
          if (d.end || *(volatile int*)&sm.abort) {
            more_q = false;
            return;
          }
          nq = d.n;
          ok = wait_all(&sm.q_ready[xq & 1], xq >> 1);
        }
        const int slot = jq % L::slots, b = jq & 1;
        ok = ok && wait_all(&sm.k_full[slot], jq / L::slots) && (jq < 2 || wait_all(&sm.s_free[b], (jq - 2) >> 1));
        if (!ok) return;
        tc::fence_after_sync();
        const uint64_t dq = dq0 + (xq & 1) * tile16, dk = dk0 + slot * tile16;
#pragma unroll
        for (int c4 = 0; c4 < L::chunks; ++c4) {
          const uint64_t c = (uint64_t)((c4 * L::chunk_bytes) >> 4);
          tc::mma4_f16_ss(tmem + kTcKeys * b, dq + c, dq + c + 2, dq + c + 4, dq + c + 6, dk + c, dk + c + 2, dk + c + 4,
                          dk + c + 6, idesc_qk, c4 > 0 ? 1u : 0u);
        }
        tc::commit_elect(&sm.s_full[b]);
        tc::commit_elect(&sm.k_empty[slot]);
        ++jq;
        if (++iq == nq) {
          tc::commit_elect(&sm.q_free[xq & 1]);
          iq = 0;
          ++xq;
        }
      };
      issue_qk();
      issue_qk();
      int J = 0;
      for (int x = 0; ok; ++x) {
        const PieceDesc& d = piece(x);
        if (d.end || *(volatile int*)&sm.abort) break;
        const int n = d.n, lo = d.lo_min, hi = d.hi_max, tile0 = d.tile0;
        for (int i = 0; ok && i < n; ++i, ++J) {
          // S_(J+2) first: its buffer is free before P_J is written.
          issue_qk();
          const int slot = J % L::slots, b = J & 1;
          ok = ok && wait_all(&sm.v_full[slot], J / L::slots);
          if (!ok) break;
          const int key0 = (tile0 + i) * kTcKeys;
          if (key0 < lo || key0 + kTcKeys > hi) {
            // Rows of fetched page parts outside the windows of every row.
            const int za = max(0, (lo - key0) / box_rows * box_rows), zb = max(0, lo - key0);
            const int zc = min(kTcKeys, hi - key0), zd = min(kTcKeys, (zc + box_rows - 1) / box_rows * box_rows);
            for (int r = za + (lane >> 3); r < zd; r += 4) {
              if (r >= zb && r < zc) continue;
#pragma unroll
              for (int c = 0; c < L::chunks; ++c)
                *reinterpret_cast<uint4*>(sm.v[slot] + c * L::chunk_bytes + r * 128 + 16 * (lane & 7)) =
                    make_uint4(0u, 0u, 0u, 0u);
            }
            fence_async_smem();
            __syncwarp();
          }
          // The first product of a piece replaces O: both groups have read the last one.
          if (i == 0 && x > 0) ok = wait_all(&sm.o_free, x - 1);
          ok = ok && wait_all(&sm.p_ready[b], J >> 1);
          if (!ok) break;
          tc::fence_after_sync();
          const uint64_t dv = dv0 + slot * tile16;
          constexpr uint64_t st = (16 * 128) >> 4;  // one K step: 16 key rows of 128 bytes
#pragma unroll
          for (int c4 = 0; c4 < kTcKeys / 64; ++c4) {
            const uint64_t c = 4 * st * c4;
            const uint32_t pa = tmem + kPColumn + 64 * b + 32 * c4;  // P: 8 columns (16 keys) per K step
            tc::mma4_f16_ts(tmem + kOColumn, pa, pa + 8, pa + 16, pa + 24, dv + c, dv + c + st, dv + c + 2 * st,
                            dv + c + 3 * st, idesc_pv, (i > 0 || c4 > 0) ? 1u : 0u);
          }
          tc::commit_elect(&sm.pv_done[b]);
          tc::commit_elect(&sm.v_empty[slot]);
        }
        if (lane == 0) mbar_arrive(&sm.desc_free[x % kDescs]);
      }
      tc::commit_elect(&sm.drain);
      mbar_wait_bounded(&sm.drain, 0, a.status);
    } else {
      // ---------------------------------------------------------- planner, Q loads
      if (lane == 0 && q_box) prefetch_tmap(&tm_q);
      BatchSplit split{};
      plan::Walker<kTcRows, kTcKeys> walk(a, sm.start);
      plan::Piece p;
      int x = 0;
      bool more = true;
      while (more) {
        more = walk.next(p, &split) && !*(volatile int*)&sm.abort;
        const int rows = more ? min(kTcRows, p.q.q_len * a.gs - p.b * kTcRows) : 0;
        if (more && p.t1 == p.t0) {  // rows without keys
          for (int r = lane >> 2; r < rows; r += 8) {
            const int f = p.b * kTcRows + r, t = f / a.gs, h = p.g * a.gs + f % a.gs;
            T* dst = static_cast<T*>(a.out) + (long long)(p.q.row0 + t) * a.out_stride + (long long)h * D;
            for (int u = lane & 3; u < D / 8; u += 4) *reinterpret_cast<uint4*>(dst + 8 * u) = make_uint4(0u, 0u, 0u, 0u);
          }
          continue;
        }
        if (x >= kDescs) wait(&sm.desc_free[x % kDescs], x / kDescs - 1);
        if (lane == 0) {
          PieceDesc& d = sm.desc[x % kDescs];
          d.end = !more;
          if (more) {
            d.whole = p.whole;
            d.seq = p.s;
            d.g = p.g;
            d.slot = p.slot;
            d.row0 = p.q.row0;
            d.q_len = p.q.q_len;
            d.len = p.q.len;
            d.pfx = p.q.pfx;
            d.blk = p.b;
            d.rows = rows;
            d.lo_min = p.k.lo_min;
            d.lo_max = p.k.lo_max;
            d.hi_min = p.k.hi_min;
            d.hi_max = p.k.hi_max;
            d.tile0 = p.k.kt0 + p.t0;
            d.n = p.t1 - p.t0;
          }
          mbar_arrive(&sm.desc_full[x % kDescs]);
        }
        __syncwarp();
        if (!more) break;
        // Q block, 128-byte swizzle.  Rows past the piece's are left as they are or hold other rows (an MMA row
        // only feeds itself, and those rows are not stored).
        if (x >= 2) wait(&sm.q_free[x & 1], (x >> 1) - 1);
        if (q_box) {  // whole tokens a block: one box per column chunk
          if (lane == 0) {
            mbar_arrive_expect_tx(&sm.q_ready[x & 1], (unsigned)L::tile_bytes);
#pragma unroll
            for (int c = 0; c < L::chunks; ++c)
              tma_load_3d(sm.q[x & 1] + c * L::chunk_bytes, &tm_q, 64 * c, p.g * a.gs, p.q.row0 + p.b * (kTcRows / a.gs),
                          &sm.q_ready[x & 1]);
          }
          __syncwarp();
          ++x;
          continue;
        }
        constexpr int units = D / 8, rows_per = 32 / units;  // units of a row over the lanes
        const int u = lane % units;
        unsigned char* qt = sm.q[x & 1] + (u >> 3) * L::chunk_bytes;
        const T* src = static_cast<const T*>(a.q) + (long long)p.q.row0 * a.q_stride + (long long)p.g * a.gs * D + 8 * u;
        for (int r = lane / units; r < rows; r += rows_per) {
          const int f = p.b * kTcRows + r, t = f / a.gs;
          cp_async16(qt + r * 128 + 16 * ((u & 7) ^ (r & 7)), src + (long long)t * a.q_stride + (f - t * a.gs) * D, 16u);
        }
        cp_async_commit();
        cp_async_wait<0>();
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_ready[x & 1]);
        ++x;
      }
      if (lane == 0) a.split[blockIdx.x] = split;
      // The Q copies of the last pieces have landed before the block exits.
      for (int y = max(0, x - 2); q_box && y < x; ++y) mbar_wait_bounded(&sm.q_ready[y & 1], (unsigned)((y >> 1) & 1), a.status);
    }
  } else {
    // ------------------------------------------------------------ softmax groups
    regs_inc<kSoftmaxRegs>();
    const int grp = (warp - 4) >> 2, qd = warp & 3;
    const int r = 32 * qd + lane;  // row == TMEM lane
    const uint32_t lane_base = (uint32_t)(32 * qd) << 16;
    const uint32_t o_col = tmem + lane_base + kOColumn;
    constexpr int kHalfD = D / 2;

    // Reads this group's half of O of piece x, whose last tile is jl, and stores it.
    auto epilogue = [&](int x, int jl) {
      const PieceDesc& d = sm.desc[x % kDescs];
      const bool busy = 32 * qd < d.rows;
      float inv = 0.f, m_fin = -INFINITY, l_row = 0.f;
      // A parity wait needs the phase before it to be over: for the other group's tile jl that follows from P V
      // of this group's tile jl - 1 (products complete in order).
      if (jl > 0 && (jl & 1) != grp) wait(&sm.pv_done[(jl - 1) & 1], (jl - 1) >> 1);
      wait(&sm.pv_done[jl & 1], jl >> 1);
      tc::fence_after_sync();
      T* dst = nullptr;
      float* part = nullptr;
      if (busy) {
        wait(&sm.stat_bar[qd][x & 1][grp ^ 1], x >> 1);
        const float2 s0 = sm.stat[x & 1][0][r], s1 = sm.stat[x & 1][1][r];
        m_fin = fmaxf(s0.x, s1.x);
        if (s0.y != 0.f) l_row += s0.y * ex2(s0.x - m_fin);
        if (s1.y != 0.f) l_row += s1.y * ex2(s1.x - m_fin);
        inv = l_row == 0.f ? 0.f : 1.f / l_row;
        if (d.whole) {
          const int f = d.blk * kTcRows + r, t = f / a.gs, h = d.g * a.gs + f % a.gs;
          dst = static_cast<T*>(a.out) + (long long)(d.row0 + t) * a.out_stride + (long long)h * D + grp * kHalfD;
        } else {
          part = a.partial + (long long)(2 * blockIdx.x + d.slot) * kTcRows * (D + 2);
          if (grp == 0 && r < d.rows) *reinterpret_cast<float2*>(part + kTcRows * D + 2 * r) = make_float2(m_fin, l_row);
          part += r * D + grp * kHalfD;
        }
      }
      const bool store = r < d.rows;
#pragma unroll
      for (int c = 0; c < kHalfD / 32; ++c) {  // 32 columns at a time; O is free after the last read
        uint32_t o[32];
        if (busy) {
          tc::tmem_ld32(o_col + grp * kHalfD + 32 * c, o);
          tc::tmem_ld_wait();
          tc::reg_fence(o);
        }
        if (c == kHalfD / 32 - 1) {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.o_free);
        }
        if (store && dst != nullptr) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = l_row == 0.f
                         ? 0u
                         : pack_pair<T>(__uint_as_float(o[e + 2 * k]) * inv, __uint_as_float(o[e + 2 * k + 1]) * inv);
            *reinterpret_cast<uint4*>(dst + 32 * c + e) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else if (store) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4*>(part + 32 * c + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.desc_free[x % kDescs]);
    };

    // One pass of this loop is at most one own tile and one epilogue.  pend: the
    // piece whose epilogue waits for this group's next tile (its last tile is J - 1).
    int x = -1, J = 0, n = 0, i = 0, pend = -1;
    bool busy = false, done = false;
    int lo_r = 0, hi_r = 0, pos_r = 0;
    float slope = 0.f, m_ref = -INFINITY, l = 0.f;
    auto open_piece = [&]() {  // the next piece's row data
      const PieceDesc& d = piece(++x);
      done = d.end || *(volatile int*)&sm.abort;
      n = done ? 0 : d.n;
      i = (J & 1) ^ grp;
      busy = !done && 32 * qd < d.rows;
      m_ref = -INFINITY;
      l = 0.f;
      lo_r = hi_r = pos_r = 0;
      slope = 0.f;
      if (!done && r < d.rows) {
        const int f = d.blk * kTcRows + r, t = f / a.gs;
        const plan::SeqInfo q{d.row0, d.q_len, d.len, d.pfx};
        lo_r = plan::row_lo(a, q, t);
        hi_r = plan::row_hi(q, t);
        pos_r = d.len - d.q_len + t;
        if (MODE != 0 && a.slopes != nullptr) slope = -kLog2e * a.slopes[d.g * a.gs + f % a.gs];
      }
    };
    open_piece();
    while (!done || pend >= 0) {
      if (i < n) {
        const PieceDesc& d = sm.desc[x % kDescs];
        const int j = J + i, b = j & 1;
        wait(&sm.s_full[b], j >> 1);
        tc::fence_after_sync();
        if (!busy) {
          // No valid row in this warp: only keep the barriers going (P_b of tile j - 2 must have been read
          // before this tile's arrival).
          if (lane == 0) {
            mbar_arrive(&sm.s_free[b]);
            mbar_arrive(&sm.chain_bar[qd][j % kChain]);
          }
          if (j >= 2) wait(&sm.pv_done[b], (j - 2) >> 1);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_ready[b]);
        } else {
          const uint32_t s_col = tmem + lane_base + kTcKeys * b;
          uint32_t s[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tc::tmem_ld32(s_col + 32 * c, s[c]);
          tc::tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 4; ++c) tc::reg_fence(s[c]);
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.s_free[b]);

          const int key0 = (d.tile0 + i) * kTcKeys;
          if (MODE == 1) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e) s[c][e] = __float_as_uint(__uint_as_float(s[c][e]) * sc.scale2);
          } else if (MODE == 2) {
            float big = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; e += 2)
                big = max3(big, fabsf(__uint_as_float(s[c][e])), fabsf(__uint_as_float(s[c][e + 1])));
            if (!__any_sync(0xffffffffu, big * sc.in_mul > kTanhPolyMax)) {
              // tanh_poly on pairs: y = out_mul (x + x u q(u)).
              const float xo = sc.in_mul * sc.out_mul;
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                  const float s0 = __uint_as_float(s[c][e]), s1 = __uint_as_float(s[c][e + 1]);
                  s[c][e] = __float_as_uint(s0 * xo);
                  s[c][e + 1] = __float_as_uint(s1 * xo);
                  float x0 = s0 * sc.in_mul, x1 = s1 * sc.in_mul;
                  const float u0 = x0 * x0, u1 = x1 * x1;
                  float q0 = kTanhQ4, q1 = kTanhQ4;
                  fma2(q0, q1, u0, u1, kTanhQ3, kTanhQ3);
                  fma2(q0, q1, u0, u1, kTanhQ2, kTanhQ2);
                  fma2(q0, q1, u0, u1, kTanhQ1, kTanhQ1);
                  fma2(q0, q1, u0, u1, kTanhQ0, kTanhQ0);
                  q0 *= u0;
                  q1 *= u1;
                  x0 = __uint_as_float(s[c][e]);
                  x1 = __uint_as_float(s[c][e + 1]);
                  fma2(q0, q1, x0, x1, x0, x1);
                  s[c][e] = __float_as_uint(q0);
                  s[c][e + 1] = __float_as_uint(q1);
                }
            } else {
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  s[c][e] = __float_as_uint(sc.out_mul * tanh_score(__uint_as_float(s[c][e]) * sc.in_mul));
            }
          }
          if (MODE != 0 && a.slopes != nullptr) {
            const float dist = (float)(key0 - pos_r);
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                s[c][e] = __float_as_uint(fmaf(slope, fabsf(dist + (float)(32 * c + e)), __uint_as_float(s[c][e])));
          }
          if (key0 + kTcKeys > d.hi_min) {  // the tile crosses some row's window end
            const int lim = hi_r - key0;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (32 * c + e >= lim) s[c][e] = __float_as_uint(-INFINITY);
          }
          if (key0 < d.lo_max) {  // ... or some row's window start
            const int lim = lo_r - key0;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (32 * c + e < lim) s[c][e] = __float_as_uint(-INFINITY);
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 128; e += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mx[k] = max3(mx[k], __uint_as_float(s[e >> 5][(e & 31) + 2 * k]),
                           __uint_as_float(s[e >> 5][(e & 31) + 2 * k + 1]));
          const float cf = MODE == 0 ? sc.scale2 : 1.f;
          const float tmax = cf * max3(mx[0], mx[1], fmaxf(mx[2], mx[3]));

          // The reference of the tile before (left by the other group), then this tile's.
          float m_prev = -INFINITY;
          if (i > 0) {
            wait(&sm.chain_bar[qd][(j - 1) % kChain], (j - 1) / kChain);
            m_prev = sm.chain[(j - 1) % kChain][r];
          }
          const float m_new = (tmax > m_prev + kRescale) ? tmax : m_prev;  // also for the first finite maximum
          sm.chain[j % kChain][r] = m_new;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.chain_bar[qd][j % kChain]);
          const float neg_m = (m_new == -INFINITY) ? 0.f : -m_new;

          float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float x0 = __uint_as_float(s[c][e]), x1 = __uint_as_float(s[c][e + 1]);
              if (MODE == 0)
                fma2(x0, x1, cf, cf, neg_m, neg_m);
              else
                add2(x0, x1, neg_m, neg_m);
              const float p0 = ex2(x0), p1 = ex2(x1);
              const int k = (e >> 1) & 3;
              add2(sum[2 * k], sum[2 * k + 1], p0, p1);
              s[c][e >> 1] = pack_pair<T>(p0, p1);
            }
          // P_b was last read by P V of tile j - 2.
          if (j >= 2) {
            wait(&sm.pv_done[b], (j - 2) >> 1);
            tc::fence_after_sync();
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) tc::tmem_st16(tmem + lane_base + kPColumn + 64 * b + 16 * c, s[c]);
          const float tsum = ((sum[0] + sum[1]) + (sum[2] + sum[3])) + ((sum[4] + sum[5]) + (sum[6] + sum[7]));
          l = l * ((m_new != m_ref) ? ex2(m_ref - m_new) : 1.f) + tsum;
          m_ref = m_new;
          // O holds the piece's earlier tiles against m_prev.
          if (i > 0 && __any_sync(0xffffffffu, m_new != m_prev)) {
            const float corr = (m_new != m_prev) ? ex2(m_prev - m_new) : 1.f;  // m_prev = -inf gives 0
            wait(&sm.pv_done[b ^ 1], (j - 1) >> 1);
            tc::fence_after_sync();
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tc::tmem_ld32(o_col + 32 * c, o);
              tc::tmem_ld_wait();
              tc::reg_fence(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
              tc::tmem_st32(o_col + 32 * c, o);
            }
          }
          tc::tmem_st_wait();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_ready[b]);
        }
        i += 2;
      }
      int ep = -1;
      if (pend >= 0) {  // the first tile of this piece is done; O still holds the last piece
        ep = pend;
        pend = -1;
      } else if (i >= n) {
        sm.stat[x & 1][grp][r] = make_float2(m_ref, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.stat_bar[qd][x & 1][grp]);
        J += n;
        if (((J - 1) & 1) == grp)
          ep = x;
        else
          pend = x;
        open_piece();
      }
      if (ep >= 0) epilogue(ep, J - 1);
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
    tc::tmem_relinquish();
  }
}

template <typename T, int D>
int launch_tc_t(const BatchArgs& a, int blocks, int box_rows, cudaStream_t s) {
  const uint64_t dims[2] = {(uint64_t)a.kv_dim, (uint64_t)a.num_pages * a.page_rows};
  const uint64_t strides[1] = {(uint64_t)a.kv_dim * 2};
  const uint32_t box[2] = {64, (uint32_t)box_rows};
  CUtensorMap tm_k, tm_v;  // 16-bit elements are only moved: one element type serves both
  if (!make_tmap(&tm_k, a.k_pages, 2, dims, strides, box, true, kSwizzle128) ||
      !make_tmap(&tm_v, a.v_pages, 2, dims, strides, box, true, kSwizzle128))
    return ATTN_ERR_CUDA;
  // Q: [rows][H][D]; a row block is one box of gs heads x 128/gs tokens when gs divides 128.
  int q_box = kTcRows % a.gs == 0 ? 1 : 0;
  CUtensorMap tm_q = tm_k;
  if (q_box) {
    const uint64_t qdims[3] = {(uint64_t)D, (uint64_t)a.H, (uint64_t)a.total_rows};
    const uint64_t qstrides[2] = {(uint64_t)D * 2, (uint64_t)a.q_stride * 2};
    const uint32_t qbox[3] = {64, (uint32_t)a.gs, (uint32_t)(kTcRows / a.gs)};
    if (!make_tmap(&tm_q, a.q, 3, qdims, qstrides, qbox, true, kSwizzle128)) return ATTN_ERR_CUDA;
  }
  ScoreMap sc = score_map(a);
  const void* kern;
  if (a.softcap > 0.f)
    kern = reinterpret_cast<const void*>(batch_tc_kernel<T, D, 2>);
  else if (a.slopes != nullptr || !(sc.scale2 >= FLT_MIN))
    kern = reinterpret_cast<const void*>(batch_tc_kernel<T, D, 1>);
  else
    kern = reinterpret_cast<const void*>(batch_tc_kernel<T, D, 0>);
  const size_t smem = sizeof(TcSmem<D>) + 1024;
  if (!set_smem_limit(kern, smem)) return ATTN_ERR_CUDA;
  BatchArgs aa = a;
  void* args[] = {&aa, &sc, &tm_k, &tm_v, &tm_q, &box_rows, &q_box};
  return launch_pdl(kern, dim3(blocks), dim3(kTcThreads), smem, s, args) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace
}  // namespace attn
