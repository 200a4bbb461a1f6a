// batch_tc.cuh -- attention of each sequence's new tokens over its pages on
// the tcgen05 tensor cores (pages of whole 8-row groups). D is the head
// dimension rounded up to 64 or 128. A smaller head (FULL false) takes TMA maps
// that end at the head: the columns past it are zeros in Q, K and V, and are
// not stored. 4 sequences of 512 new tokens at 8192, 32 heads over 8: 222 us at
// 96 columns and 190 at 40 (batch_mma.cu: 1425 and 917). Heads of 128 and 64
// keep a form with widths known at compile time: 220 and 188 us, against 227
// and 192 in this one.  Calls with first positions (SINKS) take the smaller
// heads' form at every width.
//
// The operation and the division of work are those of batch_mma.cu and
// batch_plan.cuh; here a row block is 128 flattened rows (the M of one MMA)
// and a key tile 128 keys.  One persistent block per multiprocessor walks its
// range of pieces, and every stage runs ahead across piece borders: while the last tiles of
// one piece are in the softmax, the next piece's Q block, K tiles and first
// scores are already being made.
//
// Warp roles (512 threads; four warpgroups, so registers can be split):
//   warp 0      planner and K producer: walks the pieces, writes their descriptors
//               into a four-deep ring, loads each piece's Q block (two buffers) and
//               its K tiles, one TMA box per page part and 64-column chunk (lane l takes
//               the l-th part; a part no row of the block sees is fetched from outside
//               the pool, which arrives as zeros)
//   warp 1      issues S_J = Q K^T, up to two tiles ahead of
//   warp 2      which issues O += P_J V
//   warp 3      V producer
//   warps 4-7,
//   warps 8-11  softmax groups 0 and 1: tile J (counted over all pieces of
//               the block) belongs to group J & 1; a thread owns a whole row
//   warps 12-15 output: O to memory at a piece's end, joins of split items
// Tensor memory (512 columns): S_b [128 b, +128), P_b [256 + 64 b, +64), b = J & 1,
// O [384, +D).
//
// Softmax.  P is taken against a reference that moves to the tile's maximum only
// when that exceeds it by more than kRescale (log2 units), so O is rarely
// rescaled; the reference passes from tile to tile between the two groups,
// and each group sums its own tiles' P in fp32.  P is rounded to the operand
// type of V (bf16 <= 2^24, fp16 <= 2^15; both operands of an MMA share a type):
// an error of half a step per weight, linear in the output (fp16 weights below
// 2^-21 of the reference: 2^-32 each, kF16Head).
//
// End of a piece.  The output warps read O as soon as the last P V lands, and
// the next piece's first P V waits for that read only; the softmax groups go
// straight on to the next piece.
//
// Rows of V that lie in a fetched page part but outside the block's windows
// hold whatever the page holds (0 * NaN would reach every row): such parts are
// fetched eight rows or one row at a time, those rows from outside the pool, as
// zeros. The same rows of K only make scores that are masked.
//
// Bound by the softmax warps: a prompt of 8192, 32 heads over 8 of 128, bf16,
// takes 373 to 384 us (1.43 to 1.48 PFLOP/s, 74 to 77% of the measured bf16
// rate; tensor pipe 65% busy, special-function unit 33%, issue 47%), two chunks
// of 512 behind 16k to 32k keys 235 us (75%), at heads of 64 a prompt 445 us (32%:
// the softmax takes as long a tile, the products half). With the exponentials left out a chunk took seven
// eighths of its time, with tile loads and hand-overs alone two thirds.
//
// Codes (C8: pools of cache8.cuh).  K and V arrive as bytes in a ring of their
// own and warps 12-15 make fp16 operand tiles of them (every value is an fp16
// number), and fp16 of a bf16 Q block, whose rows' powers of two the softmax
// multiplies scores by (q16).  They convert a piece's first tiles before they
// store the last piece's O: as many as there are operand slots, since those wait for
// products of earlier pieces only.  Rows of V out of sight become zeros there.
// In a pair each block fetches and converts its own halves.  Bound by that
// conversion: the same prompt 768 us, the chunks 438 (tensor pipe 33% busy).
//
// Every wait is bounded; a block whose pipeline breaks drains its copies and
// MMAs, frees its tensor memory and leaves the status word set.  A role whose
// wait ran out frees no slot that copies land in any more.
#pragma once

#include <cfloat>
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
#include "tc.cuh"

namespace attn {
namespace {

constexpr int kTcRows = 128, kTcKeys = 128, kTcThreads = 512;
// What an item takes beyond its tiles, in tiles; kItemCostRows where a block's rows are no whole tokens (gs does not
// divide 128) and Q is copied by a warp. At 2, 3, 4, 5: 17 prompts of 512, 32 heads over 8, 123, 110, 99, 99 us; mixed
// batch of chunks 218, 219, 214, 213; prompt of 8192 alike. kItemCostRows at 2, 4, 7, 10, 16, prompt of 8192 with 20 heads
// over 4: 588, 453, 344, 324, 321. At 4, 7, 10, 16: 12 heads over 4, the prompt 274, 214, 208, 204, 32 chunks of 100 at 1000
// 69, 66, 54, 54, 8 x 4 tokens at 4000 24, 24, 25, 28; 14 over 2 of 64: 223, 198, 198, 199; 48, 47, 38, 38; 18, 20, 20, 24.
// Codes, at 2, 3, 4, 5, 6, 8, 10, 16: 17 prompts of 512 160, 156, 152, 155, 152, 158, 158, 168; prompt of 8192 783, 771, 777,
// 783, 789, 799, 812, 850; 20 heads over 4 980, 812, 746, 752, 763, 772, 787, 832; 32 chunks of 100, 12 heads over 4, 124, 122,
// 124, 122, 115, 105, 105, 103.
constexpr int kItemCost = 4, kItemCostRows = 10;
constexpr int kDescs = 4;        // piece descriptors in flight
constexpr int kChain = 4;        // reference maxima in flight
constexpr int kPColumn = 256, kOColumn = 384;
constexpr int kMaxSlots = 4;     // K (and V) tiles in flight, at most
// Registers: 128 threads * (72 + 72) + 256 * 184 = 512 * 128, the block's allocation at launch.
// Codes: 128 * (72 + 104) + 256 * 168, for the warps that make operand tiles.
constexpr int kCtrlRegs = 72, kOutRegs = 72, kSoftmaxRegs = 184, kOutRegsC8 = 104, kSoftmaxRegsC8 = 168;
static_assert(128 * (kCtrlRegs + kOutRegs) + 256 * kSoftmaxRegs == 65536 &&
                  128 * (kCtrlRegs + kOutRegsC8) + 256 * kSoftmaxRegsC8 == 65536, "the block's registers at launch");

// A piece as the roles see it.
struct PieceDesc {
  int end;         // no more pieces
  int whole;       // the item's only piece
  int seq, g, slot;
  int row0, q_len, len, pfx;
  int first_row;   // first flattened row of this block
  int rows;        // valid rows from there on, at most 128
  int lo_min, lo_max, hi_min, hi_max;
  int first, last, slot0;  // the item's pieces (plan::Piece)
  int tile_last, n;  // tiles tile_last, tile_last - 1, ... (n of them) of the item's (plan::tile_at)
  int pos_min;       // position of the block's first row
  int se, ns, skip;  // with first positions (plan::BlockKeys); other calls leave them as they are
};

// Shared memory of one block.  A pair splits the keys of a K tile and the
// columns of a V tile, so each block holds half of both.
template <int D, bool PAIR, bool C8>
struct TcLayout {
  static constexpr int rows = PAIR ? 256 : 128;       // flattened rows of an item
  static constexpr int chunks = D / 64;               // 128-byte column chunks of a row
  static constexpr int q_chunk = 128 * 128;           // bytes of one chunk of the Q block
  static constexpr int q_bytes = chunks * q_chunk;
  static constexpr int k_rows = PAIR ? 64 : 128;      // keys of a tile held here
  static constexpr int k_chunk = k_rows * 128;
  static constexpr int k_bytes = chunks * k_chunk;
  static constexpr int v_chunks = PAIR ? chunks / 2 : chunks;
  static constexpr int v_chunk = kTcKeys * 128;
  static constexpr int v_bytes = v_chunks * v_chunk;
  // K tiles (and V tiles) in flight: 128 KB or 64 KB in all; codes: as operands, 96 KB or 128 KB.
  static constexpr int slots = k_bytes == 32768 ? 2 : C8 ? 3 : 4;
  static constexpr int q_bufs = C8 && k_bytes == 32768 ? 1 : 2;
  // Codes as they come, in units of 8 KB of K or V: row bytes, rows and units of a tile, units in flight.
  static constexpr int kr_bytes = D, vr_bytes = 64 * v_chunks;
  static constexpr int kr_rows = C8 ? 8192 / kr_bytes : 1, vr_rows = C8 ? 8192 / vr_bytes : 1;
  static constexpr int kr_units = C8 ? k_rows / kr_rows : 1, vr_units = C8 ? kTcKeys / vr_rows : 1;
  static constexpr int raw_slots = !C8 ? 1 : D == 64 ? 3 : 2;
};
constexpr int kMaxRaw = 4;

template <int D, bool PAIR, bool C8>
struct __align__(1024) TcSmem {
  using L = TcLayout<D, PAIR, C8>;
  unsigned char q[L::q_bufs][L::q_bytes];
  unsigned char k[L::slots][L::k_bytes];
  unsigned char v[L::slots][L::v_bytes];
  alignas(128) unsigned char raw[2][L::raw_slots][C8 ? 8192 : 128];  // [K, V]
  alignas(8) uint16_t scale[2][L::raw_slots][C8 ? (D == 64 || PAIR ? 128 : 64) : 1];  // of each row of a unit, fp16; 0: out of sight
  uint64_t raw_full[2][kMaxRaw], raw_empty[2][kMaxRaw], q_raw[2], qf_bar[kDescs];  // codes
  uint64_t k_made[kMaxSlots], v_made[kMaxSlots], q_made[2];  // codes: operands written by the pair's second block
  uint64_t k_full[kMaxSlots], k_empty[kMaxSlots], v_full[kMaxSlots], v_empty[kMaxSlots];
  uint64_t q_ready[2], q_free[2];
  uint64_t desc_full[kDescs], desc_free[kDescs];
  uint64_t s_full[2], s_free[2], p_ready[2], pv_done[2];
  uint64_t chain_bar[4][kChain];  // [row quarter][J & 3]
  uint64_t stat_bar[4][kDescs][2];  // [row quarter][piece % kDescs][group]
  uint64_t o_ready;               // the piece's last P V has completed
  uint64_t o_free;                // O has been read
  uint64_t join_bar[kDescs];      // [piece % kDescs] whether this block joins the piece's item is known
  uint64_t drain[2];
  alignas(128) unsigned char out[4][32 * 128];  // [row quarter]: 64 columns of its rows on their way out, 128-byte swizzle
  float chain[kChain][kTcRows];
  float2 stat[kDescs][2][kTcRows];  // [piece % kDescs][group][row]: reference, sum
  int8_t qf[C8 ? kDescs : 1][C8 ? kTcRows : 1];  // [piece % kDescs] powers of two that came off the rows of Q: 2^(qf - 14)
  int4 row[256];               // each softmax thread's own row: window [x, y), position z, slope w (as float bits)
  PieceDesc desc[kDescs];
  int joins[kDescs];
  plan::Start start;
  long long warp_sums[kTcThreads / 32];
  unsigned long long tag;  // this call's (plan::begin_call)
  uint32_t tmem_base;
  int abort;
  int broken;     // a wait of either block of the pair ran out
  int issued[3];  // K tiles, V tiles (codes: units) and Q blocks whose copies this block issued
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

// ---------------------------------------------------------------- block pairs
__device__ __forceinline__ uint32_t pair_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Address, in the cluster's shared window, of the same object in the pair's first block.
__device__ __forceinline__ uint32_t in_leader(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The same object in block `rank` of the pair: a store to it, a load from it.
__device__ __forceinline__ uint32_t in_block(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void store_in_block(int* p, uint32_t rank, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(in_block(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ int load_in_block(const int* p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(in_block(p, rank)) : "memory");
  return v;
}
// Arrives on a barrier of the first block.  These barriers hand over tensor
// memory only, which tcgen05's own fences order, so neither the arrival needs a
// cluster-scope release (it would wait for every store of the thread) nor the
// wait a cluster-scope acquire (it would invalidate L1).
template <bool PAIR>
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
  if (PAIR)
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(in_leader(smem_u32(bar)))
                 : "memory");
  else
    mbar_arrive(bar);
}
// As arrive_leader, for tiles that this thread's warp wrote.
template <bool PAIR>
__device__ __forceinline__ void arrive_leader_release(uint64_t* bar) {
  if (PAIR)
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(in_leader(smem_u32(bar)))
                 : "memory");
  else
    mbar_arrive(bar);
}
// Tensor copies into this block's shared memory that complete on `bar` (a
// barrier of the first block, by its cluster address, when PAIR).
template <bool PAIR>
__device__ __forceinline__ void load_2d(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
            "r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  if (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// Rows of a kv head: column x of whole rows (FULL), or of head g in a map that
// ends at the head.
template <bool PAIR, bool FULL>
__device__ __forceinline__ void load_rows(void* dst, const CUtensorMap* map, int x, int g, int row, uint32_t bar) {
  if (FULL)
    load_2d<PAIR>(dst, map, x, row, bar);
  else
    load_3d<PAIR>(dst, map, x, g, row, bar);
}
// Tensor-memory allocation and commits of a pair: both blocks allocate, the
// first one issues, and a commit arrives in both.
template <bool PAIR>
__device__ __forceinline__ void tmem_alloc_all(uint32_t* dst) {
  if (PAIR)
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(dst)) : "memory");
  else
    tc::tmem_alloc(dst, 512);
}
template <bool PAIR>
__device__ __forceinline__ void tmem_free_all(uint32_t tmem) {
  if (PAIR) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tc::tmem_dealloc(tmem, 512);
    tc::tmem_relinquish();
  }
}
template <bool PAIR>
__device__ __forceinline__ void commit_all(uint64_t* bar) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
            smem_u32(bar))
        : "memory");
  else
    tc::commit_elect(bar);
}
// Four MMAs into one accumulator, issued by one lane of the converged warp
// (mma4_f16_* of tc.cuh for a pair).
#define ATTN_PAIR_MMA4(AFORM)                                                          \
  asm volatile(                                                                        \
      "{\n\t.reg .pred p, t, e;\n\telect.sync _|e, 0xffffffff;\n\t"                    \
      "setp.ne.b32 p, %10, 0;\n\tsetp.eq.b32 t, %10, %10;\n\t"                         \
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], " AFORM(1) ", %5, %9, p;\n\t"       \
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], " AFORM(2) ", %6, %9, t;\n\t"       \
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], " AFORM(3) ", %7, %9, t;\n\t"       \
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], " AFORM(4) ", %8, %9, t;\n\t}"
#define ATTN_A_DESC(i) "%" #i
#define ATTN_A_TMEM(i) "[%" #i "]"
template <bool PAIR>
__device__ __forceinline__ void mma4_ss(uint32_t d, uint64_t a0, uint64_t b0, uint32_t idesc, uint32_t accumulate) {
  if (PAIR)
    ATTN_PAIR_MMA4(ATTN_A_DESC)::"r"(d), "l"(a0), "l"(a0 + 2), "l"(a0 + 4), "l"(a0 + 6), "l"(b0), "l"(b0 + 2),
        "l"(b0 + 4), "l"(b0 + 6), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    tc::mma4_f16_ss(d, a0, a0 + 2, a0 + 4, a0 + 6, b0, b0 + 2, b0 + 4, b0 + 6, idesc, accumulate);
}
template <bool PAIR>
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint64_t b0, uint64_t st, uint32_t idesc,
                                        uint32_t accumulate) {
  if (PAIR)
    ATTN_PAIR_MMA4(ATTN_A_TMEM)::"r"(d), "r"(a), "r"(a + 8), "r"(a + 16), "r"(a + 24), "l"(b0), "l"(b0 + st),
        "l"(b0 + 2 * st), "l"(b0 + 3 * st), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    tc::mma4_f16_ts(d, a, a + 8, a + 16, a + 24, b0, b0 + st, b0 + 2 * st, b0 + 3 * st, idesc, accumulate);
}
#undef ATTN_A_TMEM
#undef ATTN_A_DESC
#undef ATTN_PAIR_MMA4

// ---------------------------------------------------------------- codes
// Row r of Q buffer qb, bf16, becomes fp16, times 2^(14 - the result).
template <int D, bool PAIR, typename S>
__device__ __forceinline__ int q_to_half(S& sm, int qb, int r) {
  using L = TcLayout<D, PAIR, true>;
  unsigned char* row = sm.q[qb] + r * 128;
  float m = 0.f;
#pragma unroll 8
  for (int u = 0; u < D / 8; ++u) m = fmaxf(m, q16::largest(row + (u >> 3) * L::q_chunk + 16 * ((u & 7) ^ (r & 7))));
  const int E = pow2_scale_exp(m);
  const float mul = pow2f(14 - E);
#pragma unroll 4
  for (int u = 0; u < D / 8; ++u) q16::to_half(row + (u >> 3) * L::q_chunk + 16 * ((u & 7) ^ (r & 7)), mul);
  return E;
}

// Operand tiles of tile J (K, then V), this warp's quarter of each unit's rows.  One piece of code for both, and short:
// a warp alone runs at three or four clocks an instruction, and all roles of the block share the instruction cache (both
// unrolled apart, and scales looked up here: 2 chunks of 512 behind 16k to 32k 706 us).
template <int D, bool PAIR, typename S, typename W>
__device__ __forceinline__ bool make_operands(S& sm, uint64_t* k_made, uint64_t* v_made, int J, int w,
                                              W& wait) {
  using L = TcLayout<D, PAIR, true>;
  const int slot = J % L::slots, lane = threadIdx.x & 31;
#pragma unroll 1
  for (int t = 0; t < 2; ++t) {
    // Lanes of a row, 16 columns each: 8, or 4 where rows are 64 bytes.  A warp makes 2 KB of a unit.
    const int lanes_log2 = (t ? L::vr_bytes : L::kr_bytes) == 128 ? 3 : 2;
    const int u = lane & ((1 << lanes_log2) - 1), at_once = 32 >> lanes_log2;
    const int in_unit = 4 * at_once * w + (lane >> lanes_log2);  // the lane's first row
    // Lanes of the second chunk (columns from 64 on) store their halves the other way round: eight lanes, eight bank
    // groups.  Every row of a lane has the same place among eight, or that four further, by turns.
    const bool swap = (u >> 2) != 0;
    const int at = 16 * ((2 * (u & 3) + (u >> 2)) ^ (in_unit & 7)), flip = at_once == 4 ? 64 : 0;
    unsigned char* dst = (t ? sm.v[slot] + (u >> 2) * L::v_chunk : sm.k[slot] + (u >> 2) * L::k_chunk) + 128 * in_unit;
    if (J >= L::slots && !wait(t ? &sm.v_empty[slot] : &sm.k_empty[slot], J / L::slots - 1)) return false;
#pragma unroll 1
    for (int h = 0; h < (t ? L::vr_units : L::kr_units); ++h) {
      const int Ju = (t ? L::vr_units : L::kr_units) * J + h, st = Ju % L::raw_slots;
      if (!wait(&sm.raw_full[t][st], Ju / L::raw_slots)) return false;
      const unsigned char* src = sm.raw[t][st] + 2048 * w + 16 * lane;
      const uint16_t* scale = sm.scale[t][st] + in_unit;
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        uint4 c = *reinterpret_cast<const uint4*>(src + 512 * it);
        const uint32_t m = scale[at_once * it] * 0x10001u;
        if (__any_sync(0xffffffffu, m == 0u))
          if (m == 0u) c = make_uint4(0u, 0u, 0u, 0u);  // (not 0 * code: that may be NaN)
        if (swap) c = make_uint4(c.z, c.w, c.x, c.y);
        uint32_t x[8];
        c8::to_half4(c.x, x[0], x[1]);
        c8::to_half4(c.y, x[2], x[3]);
        c8::to_half4(c.z, x[4], x[5]);
        c8::to_half4(c.w, x[6], x[7]);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = c8::mul_half2(x[e], m);
        unsigned char* to = dst + 128 * at_once * it;
        const int a0 = it & 1 ? at ^ flip : at;
        *reinterpret_cast<uint4*>(to + a0) = make_uint4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<uint4*>(to + (a0 ^ 16)) = make_uint4(x[4], x[5], x[6], x[7]);
      }
      dst += 128 * 16 * at_once;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.raw_empty[t][st]);
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(t ? &v_made[slot] : &k_made[slot]);
  }
  return true;
}

// MODE 0: scores are scale2 * S with scale2 > 0 (folded into the exponent's
// fma); 1: scaled, with an optional distance bias; 2: capped, with an optional
// distance bias.
// T: of Q and the result.
template <typename T, int D, int MODE, bool PAIR, bool FULL, bool SINKS, bool C8, bool BRIEF = false>
__global__ void __launch_bounds__(kTcThreads, 1)
    batch_tc_kernel(const BatchArgs a, const ScoreMap score, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_v1, const __grid_constant__ CUtensorMap tm_v8,
                    const __grid_constant__ CUtensorMap tm_q, const int box_rows, const int q_box) {
  static_assert(!C8 || (!FULL && SINKS), "codes have one form");
  using L = TcLayout<D, PAIR, C8>;
  using TO = typename std::conditional<C8, __half, T>::type;  // operands
  const int hd = FULL ? D : a.D;  // columns of a head
  constexpr bool kHalf = std::is_same<TO, __half>::value;
  constexpr int kQBufs = L::q_bufs;
  constexpr float kRescale = kHalf ? 8.f : 24.f;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  using S = TcSmem<D, PAIR, C8>;
  S& sm = *reinterpret_cast<S*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // The block (or pair) of the plan, and this block's place in its pair.
  const int unit = PAIR ? (int)blockIdx.x >> 1 : (int)blockIdx.x, units = PAIR ? (int)gridDim.x >> 1 : (int)gridDim.x;
  const int rank = PAIR ? (int)pair_rank() : 0;

  allow_dependent_launch();
  if (warp == 0) {
    constexpr int kMakers = !C8 ? 1 : PAIR ? 5 : 4;  // arrivals that make an operand whole: four warps, the second block
    for (int i = lane; i < kMaxSlots; i += 32) {
      mbar_init(&sm.k_full[i], kMakers);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_full[i], kMakers);
      mbar_init(&sm.v_empty[i], 1);
      if (C8) {
        mbar_init(&sm.k_made[i], 4);
        mbar_init(&sm.v_made[i], 4);
      }
    }
    if (C8 && lane < 2 * kMaxRaw) {
      mbar_init(&sm.raw_full[lane & 1][lane >> 1], 2);  // the copy, and the scales
      mbar_init(&sm.raw_empty[lane & 1][lane >> 1], 4);
    }
    if (C8 && lane < kDescs) mbar_init(&sm.qf_bar[lane], 4);
    if (lane < 2) {
      mbar_init(&sm.q_ready[lane], kMakers);
      if (C8) mbar_init(&sm.q_raw[lane], 1);
      if (C8) mbar_init(&sm.q_made[lane], 4);
      mbar_init(&sm.q_free[lane], 1);
      mbar_init(&sm.s_full[lane], 1);
      mbar_init(&sm.s_free[lane], PAIR ? 8 : 4);  // the group's warps, of both blocks
      mbar_init(&sm.p_ready[lane], PAIR ? 8 : 4);
      mbar_init(&sm.pv_done[lane], 1);
    }
    if (lane < kDescs) {
      mbar_init(&sm.desc_full[lane], 1);
      mbar_init(&sm.join_bar[lane], 1);
      // V, (first block) P V, eight softmax and four output warps; codes: the second block's idle issue warps, too
      mbar_init(&sm.desc_free[lane], rank == 0 ? 14 : C8 ? 15 : 13);
    }
    if (lane < 16) mbar_init(&sm.chain_bar[lane >> 2][lane & 3], 1);
    mbar_init(&sm.stat_bar[lane >> 3][(lane >> 1) & 3][lane & 1], 1);
    if (lane == 31) {
      mbar_init(&sm.o_ready, 1);
      mbar_init(&sm.o_free, PAIR ? 8 : 4);
      mbar_init(&sm.drain[0], 1);
      mbar_init(&sm.drain[1], 1);
      sm.abort = sm.broken = 0;
    }
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_all<PAIR>(&sm.tmem_base);
  // Lengths, tables and pages may be the previous kernel's output.
  grid_dependency_wait();
  if (tid == 32) sm.tag = plan::begin_call(a);
  plan::make_plan<L::rows, kTcKeys, kTcThreads, SINKS>(a, unit, units, reinterpret_cast<int*>(sm.q[0]), sm.warp_sums, &sm.start);
  // The plan's scratch is where Q and the K/V tiles land.
  fence_async_smem();
  tc::fence_before_sync();
  if (PAIR)
    pair_sync();  // the other block's barriers are initialised, too
  else
    __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sm.tmem_base;
  // Warps wait as a whole.  Were lanes to leave a wait at different times, one could arrive somewhere for the warp, the
  // barrier complete its next phase and the others wait for a phase that is past.
  const unsigned long long limit = BRIEF ? a.wait_ns : kWaitLimitNs;
  // The forms with more code wait in less of it (17 ragged chunks with a bias 218 us, 202 so; a prompt of 8192 with a window
  // and first positions 237 and 226); the plainest one does not gain (prompt of 8192 395 and 405).
  constexpr bool kShortWaits = C8 || SINKS || MODE != 0;
  auto wait = [&](uint64_t* bar, int phase) {
    return warp_wait<BRIEF, kShortWaits>(bar, (unsigned)(phase & 1), a.status, &sm.abort, limit);
  };
  // Without the vote, where no answer is asked for, nothing warp-wide follows at once and a __syncwarp comes before a lane
  // arrives for the warp (17 ragged chunks with a bias, 16 heads: 223 us with votes there too, 219 this way).
  auto lane_wait = [&](uint64_t* bar, int phase) {
    if constexpr (kShortWaits)
      wait_phase_short<BRIEF>(bar, (unsigned)(phase & 1), a.status, &sm.abort, (unsigned)limit);
    else
      wait_phase<BRIEF>(bar, (unsigned)(phase & 1), a.status, &sm.abort, limit);
  };
  // Is there a piece x?  Its descriptor is then valid until every role has released it.  If not, there are no more or
  // the pipeline broke: the role, all lanes of it, leaves.
  auto next_piece = [&](int x) {
    return wait(&sm.desc_full[x % kDescs], x / kDescs) && warp_whole(&sm.abort) && !sm.desc[x % kDescs].end;
  };

  if (warp < 4) {
    regs_dec<kCtrlRegs>();
    // The producers (warps 0 and 3) walk a piece's page parts.  Pool rows are read from the block table 32 parts at a
    // time (one a lane), at least 32 parts ahead: a table read is a trip to L2, longer than a tile's products.
    const int outside = a.num_pages * a.page_rows;  // a row past the pool: arrives as zeros
    struct Parts {
      int shift;             // log2 of the page parts of a tile held here
      int n, se, lo, hi;     // tiles; what the rows see: keys [0, se) and [lo, hi)
      int last, ns, skip;    // the item's tile that is tile 0 here, and plan::tile_at's
      int off;               // first key held here of a tile
      const uint32_t* table;
      int now, next;         // pool rows of 32 parts, and of the 32 after
    };
    auto first_key_of = [&](const Parts& w, int i) {
      return plan::tile_at<SINKS>(w.last - i, w.ns, w.skip) * kTcKeys + w.off;
    };
    auto rows_of = [&](const Parts& w, int q0) {
      const int q = q0 + lane, i = q >> w.shift, key = first_key_of(w, i) + (q - (i << w.shift)) * box_rows;
      const bool seen = i < w.n && !plan::keys_hidden<SINKS>(key, box_rows, w.se, w.lo, w.hi);
      const int col = seen ? plan::page_of(a, key) : 0;
      const uint32_t pg = w.table[col];  // (no branch around it: two such reads overlap)
      return !seen ? outside : pg < (uint32_t)a.num_pages ? (int)pg * a.page_rows + key - col * a.page_rows : -1;
    };
    auto open_parts = [&](int keys, int n, int se, int lo, int hi, int last, int ns, int skip, int off, int seq) {
      Parts w{__ffs(keys) - __ffs(box_rows), n, se, lo, hi, last, ns, skip, off,
              a.block_table + (long long)seq * a.max_blocks, 0, 0};
      w.now = rows_of(w, 0);
      w.next = rows_of(w, 32);
      return w;
    };
    // Pool row of this lane's part of tile i (tiles in order).
    auto part_row = [&](Parts& w, int i) {
      const int q0 = i << w.shift;
      if (i > 0 && q0 % 32 == 0) {
        w.now = w.next;
        w.next = rows_of(w, q0 + 32);
      }
      int row = __shfl_sync(0xffffffffu, w.now, (q0 + lane) % 32);
      if (lane >> w.shift) row = outside;
      if (row < 0) {  // a page outside the pool
        record_status(a.status, ATTN_ERR_INVALID_ARG);
        row = outside;
      }
      return row;
    };
    // Codes of a piece's tiles of K (v 0) or V (1) and their rows' scales, unit by unit; J counts units.  A lane looks up
    // the scales of four rows of a unit, one tile ahead (a trip to L2); four rows of one page share one where the blocks of
    // the scales are whole fours.
    auto load_codes = [&](Parts& w, int v, int g, int& J) {
      const int rows = v ? L::vr_rows : L::kr_rows, r = 4 * lane;
      constexpr int kUnits = L::vr_units;  // (of K, too, but for a pair's)
      const int units = v ? L::vr_units : L::kr_units;
      const uint8_t* scales = (v ? a.v_scales : a.k_scales) + g;
      const int box_log2 = __ffs(box_rows) - 1, parts_log2 = __ffs(rows) - 1 - box_log2;
      const bool quad = (a.scale_rows & 3) == 0;
      auto look = [&](int row, int h) {  // bytes of the lane's four rows
        const int part = __shfl_sync(0xffffffffu, row, ((h << parts_log2) + (r >> box_log2)) & 31);
        if (r >= rows || part == outside) return 0u;
        const uint32_t at = (uint32_t)(part + (r & (box_rows - 1)));
        if (quad) return 0x01010101u * scales[(long long)divide(at, a.by_scale) * a.G];
        uint32_t b = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) b |= (uint32_t)scales[(long long)divide(at + k, a.by_scale) * a.G] << (8 * k);
        return b;
      };
      int row = part_row(w, 0);
      uint32_t bytes[kUnits];
#pragma unroll
      for (int h = 0; h < kUnits; ++h) bytes[h] = look(row, h);
#pragma unroll 1
      for (int i = 0; i < w.n; ++i) {
        const int key0 = first_key_of(w, i);
        const bool cut = v && !plan::keys_inside<SINKS>(key0, kTcKeys, w.se, w.lo, w.hi);
#pragma unroll
        for (int h = 0; h < kUnits; ++h) {
          if (h >= units) break;
          const int st = J % L::raw_slots;
          if (J >= L::raw_slots && !wait(&sm.raw_empty[v][st], J / L::raw_slots - 1)) return false;
          if (lane == 0) mbar_arrive_expect_tx(&sm.raw_full[v][st], 8192u);
          __syncwarp();
          if (lane >> parts_log2 == h && (lane >> w.shift) == 0)
            load_3d<false>(sm.raw[v][st] + (lane - (h << parts_log2)) * box_rows * (8192 / rows), v ? &tm_v : &tm_k,
                           PAIR ? 32 * rank * v : 0, g, row, smem_u32(&sm.raw_full[v][st]));
          if (r < rows) {
            uint32_t x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[k] = (uint32_t)(c8::exp_of((bytes[h] >> (8 * k)) & 0xffu) + 15) << 10;
              if (cut && plan::keys_hidden<SINKS>(key0 + rows * h + r + k, 1, w.se, w.lo, w.hi)) x[k] = 0u;
            }
            *reinterpret_cast<uint2*>(&sm.scale[v][st][r]) = make_uint2(x[0] | x[1] << 16, x[2] | x[3] << 16);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.raw_full[v][st]);
          ++J;
        }
        if (i + 1 < w.n) {
          row = part_row(w, i + 1);
#pragma unroll
          for (int h = 0; h < kUnits; ++h) bytes[h] = look(row, h);
        }
      }
      return true;
    };
    auto barrier_of = [&](uint64_t* full) { return PAIR ? in_leader(smem_u32(full)) : smem_u32(full); };
    struct Planned {
      plan::Piece p;
      int first_row, rows;  // this block's of p: 128 flattened rows from first_row on
    };
    using Walk = plan::Walker<L::rows, kTcKeys, SINKS>;
    // Planner: descriptor x, of the next piece.  False: the role ends.  (A wait that ran out ends it at once: writing over a
    // descriptor or a slot in use, or arriving twice in one phase, would turn a late block into a fault.)
    auto plan_piece = [&](Walk& walk, Planned& at, int x) {
      plan::Piece& p = at.p;
      int &first_row = at.first_row, &rows = at.rows;
      bool more;
      while (true) {
        more = walk.next(p) && warp_whole(&sm.abort);
        first_row = p.b * L::rows + rank * kTcRows;
        rows = more ? max(0, min(kTcRows, p.q.q_len * a.gs - first_row)) : 0;
        if (!more || p.t1 != p.t0) break;
        for (int r = lane >> 2; r < rows; r += 8) {  // rows without keys
          const int f = first_row + r, t = plan::token_of(a, f), h = p.g * a.gs + f - t * a.gs;
          T* dst = static_cast<T*>(a.out) + (long long)(p.q.row0 + t) * a.out_stride + (long long)h * hd;
          for (int u = lane & 3; u < hd / 8; u += 4) *reinterpret_cast<uint4*>(dst + 8 * u) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      if (x >= kDescs && !wait(&sm.desc_free[x % kDescs], x / kDescs - 1)) return false;
      if (lane == 0) {
        PieceDesc& d = sm.desc[x % kDescs];
        d.end = !more;
        if (more) {
          d.whole = p.whole;
          d.seq = p.s;
          d.g = p.g;
          d.slot = p.slot;
          d.first = p.first;
          d.last = p.last;
          d.slot0 = p.slot0;
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
          d.tile_last = plan::first_tile<SINKS>(p.k) + p.t1 - 1;
          d.n = p.t1 - p.t0;
          d.pos_min = p.q.len - p.q.q_len + plan::token_of(a, first_row);
          if (SINKS) {
            d.se = p.k.se;
            d.ns = p.k.ns;
            d.skip = p.k.skip;
          }
        }
        mbar_arrive(&sm.desc_full[x % kDescs]);
      }
      __syncwarp();
      return more;
    };
    // Q block of piece x, 128-byte swizzle.  Rows past the piece's are left as they are or hold other rows (an MMA row only
    // feeds itself, and those rows are not stored).  False: its buffer did not fall free.
    auto load_q = [&](const Planned& at, int x) {
      const plan::Piece& p = at.p;
      const int first_row = at.first_row, rows = at.rows;
      const int qb = x % kQBufs;
      if (x >= kQBufs && !wait(&sm.q_free[qb], x / kQBufs - 1)) return false;
      if (PAIR || q_box) {  // whole tokens a block: one box per column chunk
        if (lane == 0) {
          constexpr bool kShared = PAIR && !C8;  // both blocks' halves complete on the first one's barrier
          uint64_t* full = C8 ? &sm.q_raw[qb] : &sm.q_ready[qb];
          const uint32_t bar = kShared ? barrier_of(full) : smem_u32(full);
          if (C8 || rank == 0) mbar_arrive_expect_tx(full, (unsigned)(kShared ? 2 : 1) * L::q_bytes);
#pragma unroll
          for (int c = 0; c < L::chunks; ++c)
            load_3d<kShared>(sm.q[qb] + c * L::q_chunk, &tm_q, 64 * c, p.g * a.gs, p.q.row0 + plan::token_of(a, first_row), bar);
        }
        __syncwarp();
      } else {
        constexpr int kUnits = D / 8, kRowsPer = 32 / kUnits;  // units of a row over the lanes
        const int u = lane % kUnits;
        unsigned char* qt = sm.q[qb] + (u >> 3) * L::q_chunk;
        const T* src = static_cast<const T*>(a.q) + (long long)p.q.row0 * a.q_stride + (long long)p.g * a.gs * hd;
        const bool inside = 8 * u < hd;  // columns past the head are zeros
        for (int r = lane / kUnits; r < rows; r += kRowsPer) {
          const int f = first_row + r, t = plan::token_of(a, f);
          cp_async16(qt + r * 128 + 16 * ((u & 7) ^ (r & 7)),
                     src + (long long)t * a.q_stride + (f - t * a.gs) * hd + (inside ? 8 * u : 0), inside ? 16u : 0u);
        }
        cp_async_commit();
        cp_async_wait<0>();
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(C8 ? &sm.q_raw[qb] : &sm.q_ready[qb]);
      }
      return true;
    };
    if (C8 && (warp == 0 || warp == 3)) {
      // ---------------------------------------------------------- codes: planner, Q and K producer; V producer
      if constexpr (C8) {
        const int v = warp == 3 ? 1 : 0;
        if (lane == 0) prefetch_tmap(v ? &tm_v : &tm_k);
        Walk walk(a, sm.start);
        Planned at;
        int x = 0, J = 0;
        for (bool ok = true; ok; ++x) {
          if (v) {
            if (!next_piece(x)) break;
          } else {
            if (!plan_piece(walk, at, x)) break;
            if (!load_q(at, x)) break;
          }
          // (One piece of code for K and V.)
          const PieceDesc& d = sm.desc[x % kDescs];
          Parts w = open_parts(v ? kTcKeys : L::k_rows, d.n, d.se, d.lo_min, d.hi_max, d.tile_last, d.ns, d.skip,
                               PAIR && !v ? rank * L::k_rows : 0, d.seq);
          ok = load_codes(w, v, d.g, J);
          if (v && ok && lane == 0) mbar_arrive(&sm.desc_free[x % kDescs]);
        }
        if (lane == 0) {
          sm.issued[v] = J;
          if (!v) sm.issued[2] = PAIR || q_box ? x : 0;
        }
      }
    } else if (!C8 && warp == 0) {
      // ---------------------------------------------------------- planner, Q and K producer
      if (lane == 0) {
        prefetch_tmap(&tm_k);
        if (q_box) prefetch_tmap(&tm_q);
      }
      Walk walk(a, sm.start);
      Planned at;
      const plan::Piece& p = at.p;
      int x = 0, J = 0;
      for (bool ok = true; ok && plan_piece(walk, at, x); ++x) {
        // The piece's first page parts are looked up while its Q buffer falls free.
        const int n = p.t1 - p.t0, col = FULL ? p.g * D : 0;
        Parts w = open_parts(L::k_rows, n, p.k.se, p.k.lo_min, p.k.hi_max, plan::first_tile<SINKS>(p.k) + p.t1 - 1, p.k.ns,
                             p.k.skip, PAIR ? rank * L::k_rows : 0, p.s);
        if (!load_q(at, x)) break;
        for (int i = 0; i < n; ++i, ++J) {
          const int row = part_row(w, i), slot = J % L::slots;
          if (J >= L::slots) ok = wait(&sm.k_empty[slot], J / L::slots - 1);
          if (!ok) break;
          if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&sm.k_full[slot], (unsigned)(PAIR ? 2 : 1) * L::k_bytes);
          __syncwarp();
          if ((lane >> w.shift) == 0) {
            const uint32_t bar = barrier_of(&sm.k_full[slot]);
#pragma unroll
            for (int c = 0; c < L::chunks; ++c)
              load_rows<PAIR, FULL>(sm.k[slot] + c * L::k_chunk + lane * box_rows * 128, &tm_k, col + 64 * c, p.g, row, bar);
          }
        }
      }
      if (lane == 0) {
        sm.issued[0] = J;
        sm.issued[2] = PAIR || q_box ? x : 0;
      }
    } else if (!C8 && warp == 3) {
      // ---------------------------------------------------------- V producer
      if (lane == 0) {
        prefetch_tmap(&tm_v);
        prefetch_tmap(&tm_v1);
      }
      int J = 0;
      bool ok = true;
      for (int x = 0; ok; ++x) {
        if (!next_piece(x)) break;
        const PieceDesc& d = sm.desc[x % kDescs];
        const int n = d.n, g = FULL ? 0 : d.g, col = (FULL ? d.g * D : 0) + (PAIR ? rank * 64 * L::v_chunks : 0);
        Parts w = open_parts(kTcKeys, n, d.se, d.lo_min, d.hi_max, d.tile_last, d.ns, d.skip, 0, d.seq);
        for (int i = 0; i < n; ++i, ++J) {
          const int row = part_row(w, i), key = first_key_of(w, i) + lane * box_rows, slot = J % L::slots;
          if (J >= L::slots) ok = wait(&sm.v_empty[slot], J / L::slots - 1);
          if (!ok) break;
          if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&sm.v_full[slot], (unsigned)(PAIR ? 2 : 1) * L::v_bytes);
          __syncwarp();
          const uint32_t bar = barrier_of(&sm.v_full[slot]);
          // A part that reaches outside the block's windows goes by eights or single rows: what the page holds there (0 * NaN would
          // reach every row) is replaced by zeros from outside the pool.
          const bool edge = row != outside && !plan::keys_inside<SINKS>(key, box_rows, w.se, w.lo, w.hi);
          if ((lane >> w.shift) == 0 && !edge) {
#pragma unroll
            for (int c = 0; c < L::v_chunks; ++c)
              load_rows<PAIR, FULL>(sm.v[slot] + c * L::v_chunk + lane * box_rows * 128, &tm_v, col + 64 * c, g, row,
                                       bar);
          }
          unsigned edges = __ballot_sync(0xffffffffu, edge);
          while (edges) {
            const int p = __ffs(edges) - 1;
            edges &= edges - 1;
            const int row_p = __shfl_sync(0xffffffffu, row, p), key_p = __shfl_sync(0xffffffffu, key, p);
            const int key_8 = key_p + 8 * lane;  // eight rows a lane; those that are not all of one kind, row by row
            const bool inside = plan::keys_inside<SINKS>(key_8, 8, w.se, w.lo, w.hi);
            const bool outer = plan::keys_hidden<SINKS>(key_8, 8, w.se, w.lo, w.hi);
            if (8 * lane < box_rows && (inside || outer)) {
              const int y = inside ? row_p + 8 * lane : outside;
#pragma unroll
              for (int c = 0; c < L::v_chunks; ++c)
                load_rows<PAIR, FULL>(sm.v[slot] + c * L::v_chunk + (p * box_rows + 8 * lane) * 128, &tm_v8, col + 64 * c, g,
                                      y, bar);
            }
            unsigned mixed = __ballot_sync(0xffffffffu, 8 * lane < box_rows && !inside && !outer);
            while (mixed) {
              const int r = 8 * (__ffs(mixed) - 1) + lane;
              mixed &= mixed - 1;
              if (lane < 8) {
                const int y = plan::keys_inside<SINKS>(key_p + r, 1, w.se, w.lo, w.hi) ? row_p + r : outside;
#pragma unroll
                for (int c = 0; c < L::v_chunks; ++c)
                  load_rows<PAIR, FULL>(sm.v[slot] + c * L::v_chunk + (p * box_rows + r) * 128, &tm_v1, col + 64 * c, g, y,
                                        bar);
              }
            }
          }
        }
        if (ok && lane == 0) mbar_arrive(&sm.desc_free[x % kDescs]);
      }
      if (lane == 0) sm.issued[1] = J;
    } else {
      // ---------------------------------------------------------- MMA issue (the first block's, in a pair)
      // Two warps, one a product, so that neither holds up the other; warp-uniform loops, one elected lane issues.
      constexpr uint32_t fmt = kHalf ? tc::kFmtF16 : tc::kFmtBF16;
      // Codes: operands are whole when the first block's four warps have written their parts and, in a pair, the second
      // block's, whose idle issue warps pass that on (*_made): released to the cluster by a thread that has no loads in
      // flight, which a release would wait for, and acquired for the cluster by the warp that issues the products (the
      // test after the wait, whose phase cannot end before that warp goes on; as a fence it took 2 chunks of 512 from
      // 444 to 470 us, this way nothing).
      auto wait_operand = [&](uint64_t* bar, int phase) {
        const bool ok = wait(bar, phase);
        if constexpr (C8 && PAIR) return ok && __all_sync(0xffffffffu, mbar_test_wait_cluster(bar, (unsigned)(phase & 1))) != 0;
        return ok;
      };
      if (rank != 0) {
        if constexpr (C8) {
          bool ok = true;
          int j = 0;
          for (int x = 0; ok; ++x) {
            if (!next_piece(x)) break;
            const int n = sm.desc[x % kDescs].n, qb = x % kQBufs;
            if (warp == 1) {
              ok = wait(&sm.q_made[qb], x / kQBufs);
              if (ok && lane == 0) arrive_leader_release<PAIR>(&sm.q_ready[qb]);
            }
            for (int i = 0; ok && i < n; ++i, ++j) {
              const int slot = j % L::slots;
              ok = wait(warp == 1 ? &sm.k_made[slot] : &sm.v_made[slot], j / L::slots);
              if (ok && lane == 0) arrive_leader_release<PAIR>(warp == 1 ? &sm.k_full[slot] : &sm.v_full[slot]);
            }
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(&sm.desc_free[x % kDescs]);
          }
        }
      } else if (warp == 1) {
        constexpr uint32_t idesc_qk = tc::idesc_f32acc(fmt, false, L::rows, kTcKeys);
        const uint64_t dq0 = tc::sdesc_sw128(smem_u32(sm.q[0]), 16, 1024);
        const uint64_t dk0 = tc::sdesc_sw128(smem_u32(sm.k[0]), 16, 1024);
        bool ok = true;
        int j = 0;
        for (int x = 0; ok; ++x) {
          if (!next_piece(x)) break;
          const PieceDesc& d = sm.desc[x % kDescs];
          const int n = d.n;
          const int qb = x % kQBufs;
          const uint64_t dq = dq0 + (uint64_t)(qb * (L::q_bytes >> 4));
          ok = wait_operand(&sm.q_ready[qb], x / kQBufs);
          for (int i = 0; ok && i < n; ++i, ++j) {
            const int slot = j % L::slots, b = j & 1;
            ok = wait_operand(&sm.k_full[slot], j / L::slots) && (j < 2 || wait(&sm.s_free[b], (j - 2) >> 1));
            if (!ok) break;
            tc::fence_after_sync();
            const uint64_t dk = dk0 + (uint64_t)(slot * (L::k_bytes >> 4));
#pragma unroll
            for (int c = 0; c < L::chunks; ++c)
              mma4_ss<PAIR>(tmem + kTcKeys * b, dq + (uint64_t)((c * L::q_chunk) >> 4),
                            dk + (uint64_t)((c * L::k_chunk) >> 4), idesc_qk, c > 0 ? 1u : 0u);
            commit_all<PAIR>(&sm.s_full[b]);
            commit_all<PAIR>(&sm.k_empty[slot]);
          }
          if (ok) commit_all<PAIR>(&sm.q_free[qb]);  // (after a failed wait the block may still be landing)
        }
      } else {
        constexpr uint32_t idesc_pv = tc::idesc_f32acc(fmt, true, L::rows, D);
        const uint64_t dv0 = tc::sdesc_sw128(smem_u32(sm.v[0]), L::v_chunk, 1024);
        bool ok = true;
        int j = 0;
        for (int x = 0; ok; ++x) {
          if (!next_piece(x)) break;
          const PieceDesc& d = sm.desc[x % kDescs];
          const int n = d.n;
          // The first product of a piece replaces O.
          if (x > 0) ok = wait(&sm.o_free, x - 1);
          for (int i = 0; ok && i < n; ++i, ++j) {
            const int slot = j % L::slots, b = j & 1;
            ok = wait_operand(&sm.v_full[slot], j / L::slots) && wait(&sm.p_ready[b], j >> 1);
            if (!ok) break;
            tc::fence_after_sync();
            const uint64_t dv = dv0 + (uint64_t)(slot * (L::v_bytes >> 4));
            constexpr uint64_t st = (16 * 128) >> 4;  // one K step: 16 key rows of 128 bytes
#pragma unroll
            for (int c4 = 0; c4 < kTcKeys / 64; ++c4)  // P: 8 columns (16 keys) per K step
              mma4_ts<PAIR>(tmem + kOColumn, tmem + kPColumn + 64 * b + 32 * c4, dv + 4 * st * c4, st, idesc_pv,
                            (i > 0 || c4 > 0) ? 1u : 0u);
            commit_all<PAIR>(&sm.pv_done[b]);
            commit_all<PAIR>(&sm.v_empty[slot]);
          }
          if (ok) commit_all<PAIR>(&sm.o_ready);
          if (ok && lane == 0) mbar_arrive(&sm.desc_free[x % kDescs]);
        }
      }
      if (rank == 0) {
        commit_all<PAIR>(&sm.drain[warp - 1]);
        mbar_wait_bounded(&sm.drain[warp - 1], 0, a.status);
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ softmax groups
    regs_inc<C8 ? kSoftmaxRegsC8 : kSoftmaxRegs>();
    const int grp = (warp - 4) >> 2, qd = warp & 3;
    const int r = 32 * qd + lane;  // row == TMEM lane
    const uint32_t lane_base = (uint32_t)(32 * qd) << 16;
    const uint32_t o_col = tmem + lane_base + kOColumn;
    int J = 0;
    for (int x = 0;; ++x) {
      if (!next_piece(x)) break;
      const PieceDesc& d = sm.desc[x % kDescs];
      const int n = d.n;
      const bool busy = 32 * qd < d.rows;
      float m_ref = -INFINITY, l = 0.f;
      int4 info = make_int4(0, 0, 0, 0);
      if (r < d.rows) {
        const int f = d.first_row + r, t = plan::token_of(a, f);
        const plan::SeqInfo q{d.row0, d.q_len, d.len, d.pfx};
        info.x = plan::row_lo(a, q, t);
        info.y = plan::row_hi(q, t);
        info.z = d.len - d.q_len + t;
        if (MODE != 0 && a.slopes != nullptr) info.w = __float_as_int(-kLog2e * a.slopes[d.g * a.gs + f - t * a.gs]);
      }
      ScoreMap sc = score;  // codes: with what came off the row
      if constexpr (C8) {
        lane_wait(&sm.qf_bar[x % kDescs], x / kDescs);
        const float f = pow2f(sm.qf[x % kDescs][r] - 14);
        // (Masked scores are -inf before they are multiplied: not by zero, and a row this small has scores of zero.)
        sc.scale2 = MODE == 0 ? fmaxf(sc.scale2 * f, FLT_MIN) : sc.scale2 * f;
        sc.in_mul *= f;
      }
      sm.row[128 * grp + r] = info;  // read on the tiles that need it: kept in registers it would spill scores
      for (int i = (J & 1) ^ grp; i < n; i += 2) {
        const int j = J + i, b = j & 1;
        const int key0 = plan::tile_at<SINKS>(d.tile_last - i, d.ns, d.skip) * kTcKeys;
        // Does the tile cross some row's window end, or start?
        const bool cut_hi = key0 + kTcKeys > d.hi_min, cut_lo = key0 < d.lo_max;
        wait(&sm.s_full[b], j >> 1);
        tc::fence_after_sync();
        if (!busy) {
          // No valid row in this warp: only keep the barriers going (P_b of tile j - 2 must have been read
          // before this tile's arrival).
          if (j > 0) lane_wait(&sm.chain_bar[qd][(j - 1) % kChain], (j - 1) / kChain);
          __syncwarp();
          if (lane == 0) {
            arrive_leader<PAIR>(&sm.s_free[b]);
            mbar_arrive(&sm.chain_bar[qd][j % kChain]);
          }
          if (j >= 2) wait(&sm.pv_done[b], (j - 2) >> 1);
          __syncwarp();
          if (lane == 0) arrive_leader<PAIR>(&sm.p_ready[b]);
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
          if (lane == 0) arrive_leader<PAIR>(&sm.s_free[b]);

          if (MODE == 1 && a.slopes == nullptr) {
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
            if (!__any_sync(0xffffffffu, big * fabsf(sc.in_mul) > kTanhPolyMax)) {
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
                  s[c][e] = __float_as_uint(capped_score(__uint_as_float(s[c][e]), sc));
            }
          }
          float fold = 0.f;  // to be added to every score of the row
          if (MODE != 0 && a.slopes != nullptr) {
            // slope = -slopes[h] log2 e.  In a tile wholly behind (or ahead of) the rows |p - j| is linear in the column;
            // in one that crosses them, slope |d| is slope d with the sign of slope.
            const int4 info = sm.row[128 * grp + r];
            const float slope = __int_as_float(info.w), mul = MODE == 1 ? sc.scale2 : 1.f;
            const bool behind = a.prefix_len == nullptr || key0 + kTcKeys - 1 <= d.pos_min;
            const float step = behind ? -slope : slope, first = step * (float)(key0 - info.z);
            if (behind || key0 >= d.pos_min + (kTcRows - 1) / a.gs + 1) {
              // What the whole tile shares joins the reference; the rest grows along the row by additions, from an
              // exact value every 32 columns (at most 15 roundings of a bias within 128 keys).
              fold = first;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                float b0 = step * (float)(32 * c), b1 = step * (float)(32 * c + 1);
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                  float x0 = __uint_as_float(s[c][e]), x1 = __uint_as_float(s[c][e + 1]);
                  fma2(x0, x1, mul, mul, b0, b1);
                  add2(b0, b1, 2.f * step, 2.f * step);
                  s[c][e] = __float_as_uint(x0);
                  s[c][e + 1] = __float_as_uint(x1);
                }
              }
            } else {
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                  float x0 = __uint_as_float(s[c][e]), x1 = __uint_as_float(s[c][e + 1]);
                  float b0 = step, b1 = step;
                  fma2(b0, b1, (float)(32 * c + e), (float)(32 * c + e + 1), first, first);
                  b0 = copysignf(b0, slope);
                  b1 = copysignf(b1, slope);
                  fma2(x0, x1, mul, mul, b0, b1);
                  s[c][e] = __float_as_uint(x0);
                  s[c][e + 1] = __float_as_uint(x1);
                }
            }
          }
          if (cut_hi) {
            const int lim = sm.row[128 * grp + r].y - key0;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (32 * c + e >= lim) s[c][e] = __float_as_uint(-INFINITY);
          }
          if (cut_lo) {
            // Keys [sinks, lo) of the sequence: columns [from, lim) of the tile.
            const int lim = sm.row[128 * grp + r].x - key0, from = SINKS ? a.sinks - key0 : 0;
            const unsigned count = (unsigned)max(0, lim - from);
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (SINKS ? (unsigned)(32 * c + e - from) < count : 32 * c + e < lim) s[c][e] = __float_as_uint(-INFINITY);
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 128; e += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mx[k] = max3(mx[k], __uint_as_float(s[e >> 5][(e & 31) + 2 * k]),
                           __uint_as_float(s[e >> 5][(e & 31) + 2 * k + 1]));
          const float cf = MODE == 0 ? sc.scale2 : 1.f;
          const float tmax = cf * max3(mx[0], mx[1], fmaxf(mx[2], mx[3])) + fold;

          // The reference of the tile before (left by the other group), then this tile's.
          // (The first tile of a piece, and warps without rows, wait too, for nothing but order: a group must not get
          // two tiles ahead of the other one's wait on the same slot of the ring.)
          float m_prev = -INFINITY;
          if (j > 0) lane_wait(&sm.chain_bar[qd][(j - 1) % kChain], (j - 1) / kChain);
          if (i > 0) m_prev = sm.chain[(j - 1) % kChain][r];
          const float m_new = (tmax > m_prev + kRescale) ? tmax : m_prev;  // also for the first finite maximum
          sm.chain[j % kChain][r] = m_new;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.chain_bar[qd][j % kChain]);
          const float neg_m = (m_new == -INFINITY) ? 0.f : kHalf ? fold - m_new + kF16Head : fold - m_new;

          // Exponentials run kLag scores ahead of their sum and packing (in place: packed pair k of a chunk replaces
          // its score k, long done), so the special-function unit, 4 cycles an instruction, is never waited for.
          constexpr int kLag = 16;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int e = 0; e < 128 + kLag; e += 2) {
            if (e < 128) {
              float x0 = __uint_as_float(s[e >> 5][e & 31]), x1 = __uint_as_float(s[e >> 5][(e & 31) + 1]);
              if (MODE == 0)
                fma2(x0, x1, cf, cf, neg_m, neg_m);
              else
                add2(x0, x1, neg_m, neg_m);
              s[e >> 5][e & 31] = __float_as_uint(ex2(x0));
              s[e >> 5][(e & 31) + 1] = __float_as_uint(ex2(x1));
            }
            if (e >= kLag) {
              const int k = e - kLag;
              const float p0 = __uint_as_float(s[k >> 5][k & 31]), p1 = __uint_as_float(s[k >> 5][(k & 31) + 1]);
              add2(sum[k & 2], sum[(k & 2) + 1], p0, p1);
              s[k >> 5][(k & 31) >> 1] = pack_pair<TO>(p0, p1);
            }
          }
          // P_b was last read by P V of tile j - 2.
          if (j >= 2) {
            wait(&sm.pv_done[b], (j - 2) >> 1);
            tc::fence_after_sync();
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) tc::tmem_st16(tmem + lane_base + kPColumn + 64 * b + 16 * c, s[c]);
          const float tsum = (sum[0] + sum[1]) + (sum[2] + sum[3]);
          l = l * ((m_new != m_ref) ? ex2(m_ref - m_new) : 1.f) + tsum;
          m_ref = m_new;
          // O holds the piece's earlier tiles against m_prev.
          // (A row that had no keys yet holds zeros there, whatever the factor.)
          const bool moved = m_new != m_prev && m_prev != -INFINITY;
          if (i > 0 && __any_sync(0xffffffffu, moved)) {
            const float corr = moved ? ex2(m_prev - m_new) : 1.f;
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
          if (lane == 0) arrive_leader<PAIR>(&sm.p_ready[b]);
        }
      }
      sm.stat[x % kDescs][grp][r] = make_float2(m_ref, l);
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.stat_bar[qd][x % kDescs][grp]);
        mbar_arrive(&sm.desc_free[x % kDescs]);
      }
      J += n;
    }
  } else {
    // ------------------------------------------------------------ output warps
    // O of each piece as soon as its last product lands: whole items leave normalised in the output's type, pieces of
    // a split one in fp32 to the workspace, where the warp that arrives last joins its 32 rows in key order.
    regs_dec<C8 ? kOutRegsC8 : kOutRegs>();
    const int qd = warp & 3, r = 32 * qd + lane;
    const uint32_t o_col = tmem + ((uint32_t)(32 * qd) << 16) + kOColumn;
    constexpr int kCols = 16, kChunks = D / kCols;  // columns at a time: few registers
    auto output = [&](int x) {
      const PieceDesc& d = sm.desc[x % kDescs];
      const bool busy = 32 * qd < d.rows, store = r < d.rows;
      lane_wait(&sm.stat_bar[qd][x % kDescs][0], x / kDescs);
      lane_wait(&sm.stat_bar[qd][x % kDescs][1], x / kDescs);
      const float2 s0 = sm.stat[x % kDescs][0][r], s1 = sm.stat[x % kDescs][1][r];
      const float m_fin = fmaxf(s0.x, s1.x);
      float l_row = 0.f;
      if (s0.y != 0.f) l_row += s0.y * ex2(s0.x - m_fin);
      if (s1.y != 0.f) l_row += s1.y * ex2(s1.x - m_fin);
      const float inv = l_row == 0.f ? 0.f : 1.f / l_row;
      long long dst = 0;  // the row's first element of the output
      if (busy) {
        const int f = d.first_row + min(r, d.rows - 1), t = plan::token_of(a, f), h = d.g * a.gs + (f - t * a.gs);
        dst = (long long)(d.row0 + t) * a.out_stride + (long long)h * hd;
      }
      const bool whole = d.whole;
      const int pr = rank * kTcRows + r, rows_here = d.rows - 32 * qd;  // row of the item; rows of this warp
      constexpr long long kSlotFloats = (long long)L::rows * (D + 2);
      // Partial slots hold four columns of all rows, then the next four, so a warp's accesses are consecutive.
      float* part = a.partial + (2ll * unit + d.slot) * kSlotFloats + 4 * pr;
      unsigned char* stage = sm.out[qd];
      // 16 columns of the row, rounded.
      auto round16 = [&](const float* v, float mul, bool empty, uint32_t* w) {
#pragma unroll
        for (int e = 0; e < kCols; e += 2) w[e >> 1] = empty ? 0u : pack_pair<T>(v[e] * mul, v[e + 1] * mul);
      };
      auto to_stage = [&](const uint32_t* w, int c) {  // columns [16 c, +16) of the 64
#pragma unroll
        for (int u = 0; u < 2; ++u)
          *reinterpret_cast<uint4*>(stage + lane * 128 + 16 * ((2 * c + u) ^ (lane & 7))) =
              make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
      };
      // The 64 columns from col0 on, eight lanes a row: a lane a row would touch 32 lines a store (prompt of 8192: 469
      // us so, 452 this way).
      auto from_stage = [&](int col0) {
        __syncwarp();
        const int u = lane & 7;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int row = 4 * k + (lane >> 3);
          const long long to = __shfl_sync(0xffffffffu, dst, row);
          const uint4 v = *reinterpret_cast<const uint4*>(stage + row * 128 + 16 * (u ^ (row & 7)));
          if (row < rows_here && col0 + 8 * u < hd)
            *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + to + col0 + 8 * u) = v;
        }
        __syncwarp();
      };
      auto read16 = [&](int c, float* v) {
        uint32_t o[32];
        tc::tmem_ld16(o_col + kCols * c, o);
        tc::tmem_ld_wait();
        tc::reg_fence16(o);
#pragma unroll
        for (int e = 0; e < kCols; ++e) v[e] = __uint_as_float(o[e]);
      };
      auto free_o = [&] {
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive_leader<PAIR>(&sm.o_free);
      };
      wait(&sm.o_ready, x);
      tc::fence_after_sync();
      if (!busy) {
        free_o();
      } else if (whole) {
        float v[kCols];
        uint32_t w[8], held[D == 128 ? 32 : 1];  // columns 64 on wait in registers, so O is free before any store
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          read16(c, v);
          round16(v, inv, l_row == 0.f, w);
          to_stage(w, c);
        }
        if constexpr (D == 128) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            read16(4 + c, v);
            round16(v, inv, l_row == 0.f, held + 8 * c);
          }
        }
        free_o();
        from_stage(0);
        if constexpr (D == 128) {
#pragma unroll
          for (int c = 0; c < 4; ++c) to_stage(held + 8 * c, c);
          from_stage(64);
        }
      } else {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          float v[kCols];
          read16(c, v);
          if (c == kChunks - 1) free_o();
          if (store) {
#pragma unroll
            for (int e = 0; e < kCols; e += 4)
              *reinterpret_cast<float4*>(part + (kCols * c + e) * L::rows) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          }
        }
      }
      // Pieces of at most 32 rows are the first warp's, but all four warps join them, each some of the columns (4
      // new tokens behind 16000, 4 heads a kv head, items of 19 pieces: 100 us with one warp, 32
      // with four).
      const bool shared_join = !whole && d.rows > 0 && d.rows <= 32;
      const int first = d.first, last = d.last;
      bool join = false;
      if (!whole && busy) {
        if (store) *reinterpret_cast<float2*>(part + (long long)L::rows * D - 2 * pr) = make_float2(m_fin, l_row);
        __syncwarp();
        unsigned seen = 0;
        // Releases this warp's rows, acquires the other pieces'.
        if (lane == 0) seen = plan::piece_arrives(a.arrived + ((PAIR ? 2 * first + rank : first) * 4 + qd), sm.tag);
        seen = __shfl_sync(0xffffffffu, seen, 0);
        join = seen == (unsigned)(last - first);
      }
      if (qd == 0) {
        if (lane == 0) {
          sm.joins[x % kDescs] = join ? 1 : 0;
          mbar_arrive(&sm.join_bar[x % kDescs]);
        }
      } else if (shared_join) {
        lane_wait(&sm.join_bar[x % kDescs], x / kDescs);
        __syncwarp();
        join = *(volatile int*)&sm.joins[x % kDescs] != 0;
      }
      if (join) {
        const int jr = shared_join ? lane : r, jpr = rank * kTcRows + jr;  // row of the block and of the item
        const bool mine = jr < d.rows;
        const long long ml_off = (long long)L::rows * D - 2 * jpr;
        const int slot0 = d.slot0;
        const float* row0 = a.partial + 4 * jpr;
        auto piece_of = [&](int c) { return row0 + (2 * c + (c == first ? slot0 : 0)) * kSlotFloats; };
        // Several pieces' loads go out together, a trip to L2 each.
        float m_all = -INFINITY, l_all = 0.f;
#pragma unroll 1
        for (int c0 = first; c0 <= last; c0 += 4) {
          float2 ml[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            ml[i] = __ldcg(reinterpret_cast<const float2*>(piece_of(min(c0 + i, last)) + ml_off));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (!mine || c0 + i > last || ml[i].y == 0.f) continue;  // none of the row's keys
            const float mn = fmaxf(m_all, ml[i].x);
            l_all = (l_all == 0.f ? 0.f : l_all * ex2(m_all - mn)) + ml[i].y * ex2(ml[i].x - mn);
            m_all = mn;
          }
        }
        const float inv_all = l_all == 0.f ? 0.f : 1.f / l_all;
        const int k0 = shared_join ? qd * (kChunks / 4) : 0, k1 = shared_join ? k0 + kChunks / 4 : kChunks;
#pragma unroll 1
        for (int k = k0; k < k1; ++k) {
          float acc[kCols];
#pragma unroll
          for (int e = 0; e < kCols; ++e) acc[e] = 0.f;
#pragma unroll 1
          for (int c0 = first; c0 <= last; c0 += 2) {
            float2 ml[2];
            float4 v[2][kCols / 4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float* q = piece_of(min(c0 + i, last));
              ml[i] = __ldcg(reinterpret_cast<const float2*>(q + ml_off));
#pragma unroll
              for (int e = 0; e < kCols / 4; ++e)
                v[i][e] = __ldcg(reinterpret_cast<const float4*>(q + (kCols * k + 4 * e) * L::rows));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (!mine || c0 + i > last || ml[i].y == 0.f) continue;
              const float f = ex2(ml[i].x - m_all);
#pragma unroll
              for (int e = 0; e < kCols / 4; ++e) {
                acc[4 * e] = fmaf(v[i][e].x, f, acc[4 * e]);
                acc[4 * e + 1] = fmaf(v[i][e].y, f, acc[4 * e + 1]);
                acc[4 * e + 2] = fmaf(v[i][e].z, f, acc[4 * e + 2]);
                acc[4 * e + 3] = fmaf(v[i][e].w, f, acc[4 * e + 3]);
              }
            }
          }
          uint32_t w[8];
          round16(acc, inv_all, l_all == 0.f, w);
          if (shared_join) {
            const int f = d.first_row + min(jr, d.rows - 1), t = plan::token_of(a, f), h = d.g * a.gs + (f - t * a.gs);
            T* to = static_cast<T*>(a.out) + (long long)(d.row0 + t) * a.out_stride + (long long)h * hd + kCols * k;
#pragma unroll
            for (int u = 0; u < 2; ++u)
              if (mine && kCols * k + 8 * u < hd)
                *reinterpret_cast<uint4*>(to + 8 * u) = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
          } else {
            to_stage(w, k & 3);
            if ((k & 3) == 3) from_stage(16 * (k - 3));
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.desc_free[x % kDescs]);
    };
    if constexpr (!C8) {
      for (int x = 0;; ++x) {
        if (!next_piece(x)) break;
        output(x);
      }
    } else {
      int J = 0;
      for (int x = 0;; ++x) {
        const bool more = next_piece(x);
        bool ok = more;
        if (more) {
          const int qb = x % kQBufs;
          ok = wait(&sm.q_raw[qb], x / kQBufs);
          if (ok) {
            int E = 14;
            if constexpr (!std::is_same<T, __half>::value) E = q_to_half<D, PAIR, S>(sm, qb, r);
            sm.qf[x % kDescs][r] = (int8_t)E;
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&sm.qf_bar[x % kDescs]);
              mbar_arrive(rank == 0 ? &sm.q_ready[qb] : &sm.q_made[qb]);
            }
          }
        }
        // The piece's first tiles (no more than there are slots), the last piece's output, the other tiles.
        const int n = more ? sm.desc[x % kDescs].n : 0, ahead = min(n, L::slots);
#pragma unroll 1
        for (int i = 0; more ? ok : warp_whole(&sm.abort); ++i) {
          if (i == ahead && x > 0) output(x - 1);
          if (i >= n) break;
          ok = make_operands<D, PAIR>(sm, rank == 0 ? sm.k_full : sm.k_made, rank == 0 ? sm.v_full : sm.v_made, J++, qd,
                                       wait);
        }
        if (!more || !ok) break;
      }
    }
  }

  __syncwarp();
  tc::fence_before_sync();
  // No copy may still be landing in shared memory when the block exits.  Products have read every tile, unless the
  // pipeline broke.
  auto drain_codes = [&] {
    drain_ring(sm.raw_full[0], L::raw_slots, sm.issued[0], a.status);
    drain_ring(sm.raw_full[1], L::raw_slots, sm.issued[1], a.status);
    drain_ring(sm.q_raw, kQBufs, sm.issued[2], a.status);
  };
  if (PAIR) {
    // Arrivals, commits and copies cross the pair: it leaves together.
    if (lane == 0 && *(volatile int*)&sm.abort != 0)
      for (int b = 0; b < 2; ++b) store_in_block(&sm.broken, b, 1);
    pair_sync();
    if constexpr (C8) {  // (each block's copies are its own)
      if (*(volatile int*)&sm.broken != 0) {
        if (tid == 0) drain_codes();
        __syncwarp();
        pair_sync();
      }
    } else if (*(volatile int*)&sm.broken != 0) {
      // A tile that only one block issued would never complete: its barrier was armed for both halves, or not at all.
      // (One block is at most a ring ahead of the other, since a slot falls free by a product that read both halves.)
      if (rank == 0 && tid == 0) {
        auto settle = [&](uint64_t* full, int slots, int which, unsigned half) {
          const int mine = sm.issued[which], other = load_in_block(&sm.issued[which], 1);
          for (int j = min(mine, other); j < max(mine, other); ++j) settle_tile(&full[j % slots], mine > j, 2 * half, half);
          drain_ring(full, slots, max(mine, other), a.status);
        };
        settle(sm.k_full, L::slots, 0, L::k_bytes);
        settle(sm.v_full, L::slots, 1, L::v_bytes);
        settle(sm.q_ready, 2, 2, L::q_bytes);
      }
      __syncwarp();
      pair_sync();
    }
    // The first block's last commits arrive here, too.
    if (rank != 0 && (warp == 1 || warp == 2)) mbar_wait_bounded(&sm.drain[warp - 1], 0, a.status);
    __syncwarp();
  } else {
    __syncthreads();
    if (C8 && *(volatile int*)&sm.abort != 0 && tid == 0) {
      drain_codes();
    } else if (*(volatile int*)&sm.abort != 0 && tid == 0) {
      drain_ring(sm.k_full, L::slots, sm.issued[0], a.status);
      drain_ring(sm.v_full, L::slots, sm.issued[1], a.status);
      drain_ring(sm.q_ready, 2, sm.issued[2], a.status);
    }
  }
  if (warp == 1) {
    tc::fence_after_sync();
    tmem_free_all<PAIR>(tmem);
  }
}

template <typename T, int D, bool PAIR, bool FULL, bool SINKS, bool C8 = false>
int launch_tc_t(const BatchArgs& a, int blocks, int box_rows, cudaStream_t s) {
  // K and V: whole rows, or [rows][G][head_dim], where columns past the head arrive as zeros.
  const int rank = FULL ? 2 : 3;
  using L = TcLayout<D, PAIR, C8>;
  const uint64_t pool = (uint64_t)a.num_pages * a.page_rows;
  constexpr int kBytes = C8 ? 1 : 2;
  const uint64_t dims[3] = {(uint64_t)(FULL ? a.kv_dim : a.D) * kBytes / 2, FULL ? pool : (uint64_t)a.G, pool};
  const uint64_t strides[2] = {(uint64_t)(FULL ? a.kv_dim : a.D) * kBytes, (uint64_t)a.kv_dim * kBytes};
  if (PAIR && box_rows > 64) box_rows = 64;  // a block holds 64 keys of a K tile
  if (C8 && box_rows > L::kr_rows) box_rows = L::kr_rows;
  if (C8 && box_rows > L::vr_rows) box_rows = L::vr_rows;
  const uint32_t box[3] = {64, FULL ? (uint32_t)box_rows : 1, (uint32_t)box_rows}, one_row[3] = {64, 1, 1};
  const uint32_t eight[3] = {64, FULL ? 8u : 1u, 8};
  CUtensorMap tm_k, tm_v, tm_v1, tm_v8;  // 16-bit elements are only moved: one element type serves both, and pairs of codes
  const int l2 = kv_l2_bytes(a.D * kBytes / 2);
  if constexpr (C8) {
    const uint32_t kbox[3] = {L::kr_bytes / 2, 1, (uint32_t)box_rows}, vbox[3] = {L::vr_bytes / 2, 1, (uint32_t)box_rows};
    if (!make_tmap(&tm_k, a.k_pages, 3, dims, strides, kbox, true, kSwizzleNone, l2) ||
        !make_tmap(&tm_v, a.v_pages, 3, dims, strides, vbox, true, kSwizzleNone, l2))
      return ATTN_ERR_CUDA;
    tm_v1 = tm_v8 = tm_v;
  } else if (!make_tmap(&tm_k, a.k_pages, rank, dims, strides, box, true, kSwizzle128, l2) ||
      !make_tmap(&tm_v, a.v_pages, rank, dims, strides, box, true, kSwizzle128, l2) ||
      !make_tmap(&tm_v8, a.v_pages, rank, dims, strides, eight, true, kSwizzle128, l2) ||
      !make_tmap(&tm_v1, a.v_pages, rank, dims, strides, one_row, true, kSwizzle128, l2))
    return ATTN_ERR_CUDA;
  // Q: [rows][H][D]; a row block is one box of gs heads x 128/gs tokens when gs divides 128.
  int q_box = kTcRows % a.gs == 0 ? 1 : 0;
  CUtensorMap tm_q = tm_k;
  if (q_box) {
    const uint64_t qdims[3] = {(uint64_t)a.D, (uint64_t)a.H, (uint64_t)a.total_rows};
    const uint64_t qstrides[2] = {(uint64_t)a.D * 2, (uint64_t)a.q_stride * 2};
    const uint32_t qbox[3] = {64, (uint32_t)a.gs, (uint32_t)(kTcRows / a.gs)};
    if (!make_tmap(&tm_q, a.q, 3, qdims, qstrides, qbox, true, kSwizzle128)) return ATTN_ERR_CUDA;
  }
  ScoreMap sc = score_map(a);
  auto of_mode = [&](auto brief) {
    constexpr bool B = decltype(brief)::value;
    if (a.softcap > 0.f) return reinterpret_cast<const void*>(batch_tc_kernel<T, D, 2, PAIR, FULL, SINKS, C8, B>);
    if (a.slopes != nullptr || !(sc.scale2 >= FLT_MIN))
      return reinterpret_cast<const void*>(batch_tc_kernel<T, D, 1, PAIR, FULL, SINKS, C8, B>);
    return reinterpret_cast<const void*>(batch_tc_kernel<T, D, 0, PAIR, FULL, SINKS, C8, B>);
  };
  const void* kern = of_mode(std::false_type{});
  if constexpr (std::is_same<T, __nv_bfloat16>::value)  // the failure-path test
    if (a.wait_ns != 0) kern = of_mode(std::true_type{});
  const size_t smem = sizeof(TcSmem<D, PAIR, C8>) + 1024;
  static_assert(sizeof(TcSmem<D, PAIR, C8>) + 1024 <= 227 * 1024, "shared memory of a block");
  if (!set_smem_limit(kern, smem)) return ATTN_ERR_CUDA;
  BatchArgs aa = a;
  aa.item_cost = q_box ? kItemCost : kItemCostRows;
  void* args[] = {&aa, &sc, &tm_k, &tm_v, &tm_v1, &tm_v8, &tm_q, &box_rows, &q_box};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, kern, args) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace
}  // namespace attn
