// paged_append.cu -- the new tokens of a ragged batch into a paged cache: K
// turned by its position, V as it is, and (optionally) Q turned for the
// attention that follows, in one launch.
//
// Row i of the token batch belongs to the last sequence s with q_start[s] <= i
// (rows at or past q_start[n_seqs] belong to none and are left alone); its
// position is kv_len[s] - q_start[s + 1] + i, its cache row
// block_table[s][pos / page_rows] * page_rows + pos % page_rows.
//
// The call only moves data (a bf16 row of 32 + 2*8 heads of 128 is 12 KB in,
// 12 KB out): long batches are bound by HBM, single tokens by the chain of
// dependent reads q_start -> block table -> pages, so a row's sequence is
// found by one warp testing 32 starts at a time.
// Four chunks of 2048 rows, 32 + 2*8 heads of 128, fp32 into bf16, move 307 MB in
// 51.4 us, 6.0 TB/s; one token of 64 sequences takes 3.2 us in a graph.
#include "common.cuh"
#include "batch.h"
#include "find_seq.cuh"
#include "rotary.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256;

template <typename TI, typename TO, bool INTER, bool VEC>
__global__ void __launch_bounds__(kThreads) append_paged_kernel(const AppendArgs a, int rows_per_block) {
  __shared__ long long slot_s[8];  // cache row, or -1: the row is skipped
  __shared__ uint32_t pos_s[8];
  const uint32_t row0 = blockIdx.x * (uint32_t)rows_per_block;
  const int nrows = (int)min((uint32_t)rows_per_block, a.total_rows - row0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < nrows) {
    const uint32_t row = row0 + warp;
    const int s = find_seq(a.q_start, a.n_seqs, row);
    long long slot = -1;
    uint32_t p = 0;
    if (s >= 0 && lane == 0) {
      const uint32_t end = a.q_start[s + 1];
      if (row < end) {
        const long long pos = (long long)a.kv_len[s] - (long long)end + (long long)row;
        bool ok = pos >= 0 && pos < (long long)a.page_rows * a.max_blocks && (a.R == 0 || pos < (long long)a.table_rows);
        if (ok) {
          p = (uint32_t)pos;
          const uint32_t page = a.block_table[(long long)s * a.max_blocks + p / (uint32_t)a.page_rows];
          ok = page < (uint32_t)a.num_pages;
          slot = (long long)page * a.page_rows + p % (uint32_t)a.page_rows;
        }
        if (!ok) {
          record_status(a.status, ATTN_ERR_INVALID_ARG);
          slot = -1;
        }
      }
    }
    if (lane == 0) {
      slot_s[warp] = slot;
      pos_s[warp] = p;
    }
  }
  __syncthreads();
  const int vu = VEC ? a.D / 8 : a.D;  // V units per head
  const int nq = a.H * a.units, nk = a.G * a.units, upr = nq + nk + a.G * vu;
  for (int i = threadIdx.x; i < nrows * upr; i += kThreads) {
    const int r = i / upr;
    int u = i - r * upr;
    const long long slot = slot_s[r];
    if (slot < 0) continue;
    const long long row = (long long)row0 + r;
    const float* tab = a.table + (long long)pos_s[r] * a.R;
    if (u < nq) {
      const int h = u / a.units;
      rot::move_unit<TI, TO, INTER, VEC>(static_cast<const TI*>(a.q) + row * a.q_stride + (long long)h * a.D,
                                         static_cast<TO*>(a.q_out) + row * a.q_out_stride + (long long)h * a.D,
                                         u - h * a.units, a.D, a.R, tab, 1.f, true);
    } else if ((u -= nq) < nk) {
      const int h = u / a.units;
      rot::move_unit<TI, TO, INTER, VEC>(static_cast<const TI*>(a.k) + row * a.k_stride + (long long)h * a.D,
                                         static_cast<TO*>(a.k_pages) + slot * a.kv_dim + (long long)h * a.D,
                                         u - h * a.units, a.D, a.R, tab, 1.f, true);
    } else {
      u -= nk;
      const int h = u / vu;
      rot::move_unit<TI, TO, INTER, VEC>(static_cast<const TI*>(a.v) + row * a.v_stride + (long long)h * a.D,
                                         static_cast<TO*>(a.v_pages) + slot * a.kv_dim + (long long)h * a.D,
                                         u - h * vu, a.D, 0, nullptr, 1.f, true);
    }
  }
}

template <typename TI, typename TO>
int launch_t(const AppendArgs& a, bool vec, cudaStream_t s) {
  // Rows a block: one where there are few (64 rows of 32 + 2*8 heads of 128 3.3 us, 5.6 with four), four where many
  // blocks would each find a row's sequence first (32768 rows 146 us with one, 130 with four; of 2*3 heads of 96 56 and
  // 28; at 1024 to 8192 rows of the larger heads alike, of the smaller ones four gain from about 1024 on: 4.8 and 3.5).
  const int rpb = a.total_rows >= 4096 ? 4 : 1;
  const dim3 grid((unsigned)((a.total_rows + rpb - 1) / rpb));
  if (vec) {
    if (a.interleaved)
      append_paged_kernel<TI, TO, true, true><<<grid, kThreads, 0, s>>>(a, rpb);
    else
      append_paged_kernel<TI, TO, false, true><<<grid, kThreads, 0, s>>>(a, rpb);
  } else {
    if (a.interleaved)
      append_paged_kernel<TI, TO, true, false><<<grid, kThreads, 0, s>>>(a, rpb);
    else
      append_paged_kernel<TI, TO, false, false><<<grid, kThreads, 0, s>>>(a, rpb);
  }
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

int launch_append_paged(AppendArgs a, int in_dtype, int cache_dtype, cudaStream_t s) {
  const bool vec = rot::vec_sizes(a.D, a.R, a.interleaved) && aligned16(a.q) && aligned16(a.q_out) && aligned16(a.k) &&
                   aligned16(a.v) && aligned16(a.k_pages) && aligned16(a.v_pages) && aligned16(a.table) &&
                   a.kv_dim % 8 == 0 && a.q_stride % 8 == 0 && a.q_out_stride % 8 == 0 && a.k_stride % 8 == 0 &&
                   a.v_stride % 8 == 0;
  a.units = rot::units_per_head(a.D, a.R, a.interleaved, vec);
  if (in_dtype == ATTN_DT_BF16) return launch_t<__nv_bfloat16, __nv_bfloat16>(a, vec, s);
  if (in_dtype == ATTN_DT_F16) return launch_t<__half, __half>(a, vec, s);
  if (cache_dtype == ATTN_DT_F32) return launch_t<float, float>(a, vec, s);
  if (cache_dtype == ATTN_DT_BF16) return launch_t<float, __nv_bfloat16>(a, vec, s);
  return launch_t<float, __half>(a, vec, s);
}

}  // namespace attn
