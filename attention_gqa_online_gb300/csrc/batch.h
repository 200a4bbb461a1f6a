// batch.h -- launch arguments of the batched paged attention and the paged
// append, and the rotary operator.  Not part of the public interface.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/attn_gqa.h"

namespace attn {

// Division by a constant of the launch, for dividends below 2^31: n / d =
// (n + umulhi(n, mul)) >> shift with shift = ceil(log2 d) and mul =
// floor(2^32 (2^shift - d) / d) + 1 (Granlund and Montgomery's round-up form).
struct FastDiv {
  uint32_t d, mul, shift;
};
#ifdef __CUDACC__
__device__ __forceinline__ uint32_t divide(uint32_t n, const FastDiv& f) { return (n + __umulhi(n, f.mul)) >> f.shift; }
#endif
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  while ((1ull << f.shift) < d) ++f.shift;
  f.mul = (uint32_t)((((1ull << f.shift) - d) << 32) / d + 1);
  return f;
}

struct RopeArgs {
  const void* x;
  void* y;
  const uint32_t* positions;  // nullptr: row t is at position t
  const float* table;
  unsigned* status;
  long long x_stride, y_stride;  // elements between rows
  uint32_t rows, table_rows;
  int heads, D, R;
  bool interleaved;
  float sgn;  // 1: turn, -1: turn back
  // Set by launch_rope_apply.
  int units;
  FastDiv per_head, per_row;  // by units, and by units * heads
  bool total_fits31;
};
int launch_rope_apply(RopeArgs a, int dtype, cudaStream_t s);

struct RopeScale {
  int kind;
  double base, factor, orig_max_pos, beta_fast, beta_slow, attn_factor;
};
int launch_rope_table_scaled(float* table, uint32_t max_pos, int R, RopeScale sc, cudaStream_t s);

struct AppendArgs {
  const void* q;  // nullptr with H == 0
  void* q_out;
  const void* k;
  const void* v;
  void* k_pages;
  void* v_pages;
  const uint32_t* block_table;  // [n_seqs][max_blocks]
  const uint32_t* q_start;      // [n_seqs + 1]
  const uint32_t* kv_len;       // [n_seqs]
  const float* table;
  unsigned* status;
  long long q_stride, q_out_stride, k_stride, v_stride, kv_dim;
  uint32_t total_rows, table_rows;
  int n_seqs, H, G, D, R;
  int page_rows, num_pages, max_blocks;
  bool interleaved;
  int units;  // set by launch_append_paged
};
int launch_append_paged(AppendArgs a, int in_dtype, int cache_dtype, cudaStream_t s);

// One record per thread block of the attention grid: the item whose first
// keys the block computed and whose last keys a later block did.
struct BatchSplit {
  int valid;
  int seq, blk, g;  // the item
  int slot0;        // partial slot of this block's piece (the later pieces are in slot 0 of theirs)
  int last;         // block holding the last piece
  int pad[2];
};

struct BatchArgs {
  const void* q;
  const void* k_pages;
  const void* v_pages;
  void* out;
  const uint32_t* block_table;  // [n_seqs][max_blocks]
  const uint32_t* q_start;      // [n_seqs + 1]
  const uint32_t* kv_len;       // [n_seqs]
  const float* slopes;          // [H] or nullptr
  const uint32_t* prefix_len;   // [n_seqs] or nullptr
  unsigned* status;
  float* partial;     // [2 * blocks][rows * (D + 2)]: unnormalised output, then (max, sum) of each row
  BatchSplit* split;  // [blocks]
  // Pieces seen of the item that starts in a block (four counters a multiprocessor), under the call's tag: counts that a
  // call left, because its waits ran out, are older than any later tag.
  unsigned long long* arrived;
  unsigned long long* calls;  // calls begun on this workspace, in units of 2^16 (batch_plan.cuh: begin_call)
  long long q_stride, out_stride, kv_dim;  // elements
  uint32_t total_rows;
  int n_seqs, H, G, D, gs;
  int page_rows, num_pages, max_blocks, capacity;
  int window;  // 0 = none
  float scale, softcap;
  FastDiv by_gs, by_page;  // by gs and page_rows; set by launch_batch_paged
  unsigned wait_ns;        // limit of each wait inside the kernels, 0 = the usual one; set by launch_batch_paged
  int item_cost;           // what an item takes beyond its tiles, in tiles; set by each kernel's launch
};
// Sequences of a batch at most (the plan keeps one count each in shared memory).
constexpr int kMaxBatchSeqs = 16384;
// Positions of a sequence at most: a piece's warps wait for one another for at
// most a second, and 2^24 keys of the slowest score map take about 0.7 s.
constexpr uint64_t kMaxBatchCapacity = 1ull << 24;
// How much L2 fetches around a missed sector of K and V: at most the power of
// two that divides a head's row (its neighbour is another head's, read much
// later by another block).  64 sequences of 8192, 8 kv heads of 64: 229 us with
// 256 bytes, 164 with 128 (6.5 TB/s).
inline int kv_l2_bytes(int head_dim) { return (2 * head_dim) & -(2 * head_dim); }
// Pool rows at most: a box of 256 rows from the first row past the pool still has 31-bit coordinates.
constexpr uint64_t kMaxBatchPool = 0x7fffffffu - 256;
size_t batch_workspace_bytes(int D, int sm_count);
void set_batch_wait_ns(unsigned ns);  // for later launches (the failure-path test)
int launch_batch_paged(BatchArgs a, int dtype, void* workspace, int sm_count, cudaStream_t s);
int launch_batch_mma(const BatchArgs& a, int dtype, int blocks, cudaStream_t s);
int launch_batch_decode(const BatchArgs& a, int dtype, int blocks, int box_rows, cudaStream_t s);
int launch_batch_tc_d64(const BatchArgs& a, int dtype, int blocks, int box_rows, cudaStream_t s);
int launch_batch_tc_d128(const BatchArgs& a, int dtype, int blocks, int box_rows, cudaStream_t s);
int launch_batch_tc_pair(const BatchArgs& a, int dtype, int blocks, int box_rows, cudaStream_t s);
int launch_batch_tc_part64(const BatchArgs& a, int dtype, int blocks, int box_rows, cudaStream_t s);
int launch_batch_tc_part128(const BatchArgs& a, int dtype, int blocks, int box_rows, cudaStream_t s);
int launch_batch_tc_part_pair(const BatchArgs& a, int dtype, int blocks, int box_rows, cudaStream_t s);

}  // namespace attn
