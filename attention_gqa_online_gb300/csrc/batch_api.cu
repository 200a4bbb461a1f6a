// batch_api.cu -- the C ABI of the rotary operator and of the batched paged
// calls (declared in include/attn_gqa.h): argument checks and launches.
#include <cmath>
#include <cstdint>

#include "../../include/attn_gqa.h"
#include "batch.h"
#include "common.cuh"
#include "internal.h"

using namespace attn;

namespace {

bool heads_ok(uint32_t H, uint32_t G, uint32_t D) {
  return H >= 1 && G >= 1 && H % G == 0 && D >= 1 && D <= 128 && H <= (1u << 20);
}
bool dtype_ok(int t) { return t == ATTN_DT_F32 || t == ATTN_DT_BF16 || t == ATTN_DT_F16; }
size_t esize(int t) { return t == ATTN_DT_F32 ? 4 : 2; }
bool layout_ok(int l) { return l == ATTN_ROPE_HALF || l == ATTN_ROPE_INTERLEAVED; }
bool paged_ok(uint32_t page_rows, uint32_t num_pages, uint32_t max_blocks) {
  return page_rows >= 1 && num_pages >= 1 && max_blocks >= 1 && (uint64_t)page_rows * max_blocks <= 0x7fffffffu &&
         (uint64_t)page_rows * num_pages <= 0x7fffffffu;
}
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The batched attention over pools of dtype (k_scales nullptr) or of 8-bit codes.
int batch_paged(const void* q, const void* k_pages, const void* v_pages, const uint8_t* k_scales, const uint8_t* v_scales, void* out,
                int dtype, const uint32_t* block_table, const uint32_t* q_start, const uint32_t* kv_len,
                uint32_t total_rows, uint32_t n_seqs, uint32_t n_heads, uint32_t n_kv_heads, uint32_t head_dim,
                uint32_t kv_dim, uint32_t q_stride, uint32_t out_stride, uint32_t page_rows, uint32_t num_pages,
                uint32_t max_blocks, uint32_t scale_rows, float scale, uint32_t window, uint32_t sinks, float softcap,
                const float* alibi_slopes, const uint32_t* prefix_len, void* workspace, size_t workspace_bytes,
                attn_stream_t stream) {
  if (!heads_ok(n_heads, n_kv_heads, head_dim) || !dtype_ok(dtype)) return ATTN_ERR_INVALID_ARG;
  if (!paged_ok(page_rows, num_pages, max_blocks)) return ATTN_ERR_INVALID_ARG;
  if (kv_dim < (uint64_t)n_kv_heads * head_dim || q_stride < (uint64_t)n_heads * head_dim ||
      out_stride < (uint64_t)n_heads * head_dim)
    return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale * 1.5f) || !(softcap >= 0.f) || !std::isfinite(softcap * 1.5f)) return ATTN_ERR_INVALID_ARG;
  if (softcap > 0.f && !std::isfinite(scale / softcap)) return ATTN_ERR_INVALID_ARG;
  if (total_rows == 0 || n_seqs == 0) return ATTN_OK;
  if (q == nullptr || k_pages == nullptr || v_pages == nullptr || out == nullptr || block_table == nullptr ||
      q_start == nullptr || kv_len == nullptr)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(block_table, 4) || !aligned(q_start, 4) || !aligned(kv_len, 4) || !aligned(alibi_slopes, 4) ||
      !aligned(prefix_len, 4))
    return ATTN_ERR_INVALID_ARG;
  if (k_scales != nullptr && (head_dim % 16 != 0 || kv_dim % 16 != 0)) return ATTN_ERR_UNSUPPORTED;
  if (dtype == ATTN_DT_F32 || head_dim % 8 != 0 || kv_dim % 8 != 0 || q_stride % 8 != 0 || out_stride % 8 != 0 ||
      !aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16))
    return ATTN_ERR_UNSUPPORTED;
  if ((uint64_t)total_rows * n_heads > (1u << 30) || n_seqs > (uint32_t)kMaxBatchSeqs ||
      (uint64_t)page_rows * max_blocks > kMaxBatchCapacity || (uint64_t)page_rows * num_pages > kMaxBatchPool)
    return ATTN_ERR_UNSUPPORTED;
  const int sms = device_sm_count();
  if (sms <= 0) return ATTN_ERR_CUDA;
  if (workspace == nullptr || workspace_bytes < batch_workspace_bytes((int)head_dim, sms) || !aligned(workspace, 16))
    return ATTN_ERR_INVALID_ARG;
  BatchArgs a{};
  a.q = q;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.out = out;
  a.block_table = block_table;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.slopes = alibi_slopes;
  a.prefix_len = prefix_len;
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.scale_rows = scale_rows > 0 ? (int)scale_rows : 1;
  a.status = device_status_word();
  if (a.status == nullptr) return ATTN_ERR_CUDA;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.kv_dim = kv_dim;
  a.total_rows = total_rows;
  a.n_seqs = (int)n_seqs;
  a.H = (int)n_heads;
  a.G = (int)n_kv_heads;
  a.D = (int)head_dim;
  a.gs = a.H / a.G;
  a.page_rows = (int)page_rows;
  a.num_pages = (int)num_pages;
  a.max_blocks = (int)max_blocks;
  a.capacity = (int)(page_rows * max_blocks);
  a.window = window > 0x7fffffffu ? 0x7fffffff : (int)window;
  a.sinks = window == 0 ? 0 : sinks > 0x3fffffffu ? 0x3fffffff : (int)sinks;
  a.scale = scale;
  a.softcap = softcap;
  return launch_batch_paged(a, dtype, workspace, sms, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" int attn_rope_table_scaled(float* table, uint32_t max_pos, uint32_t rot_dim, double base,
                                      attn_rope_scaling_t scaling, double factor, uint32_t orig_max_pos,
                                      double beta_fast, double beta_slow, double attn_factor, attn_stream_t stream) {
  if (rot_dim < 2 || rot_dim > 1024 || rot_dim % 2 != 0 || !(base > 1.0) || !std::isfinite(base))
    return ATTN_ERR_INVALID_ARG;
  if ((uint64_t)max_pos * rot_dim > 0x7fffffffu || !std::isfinite(attn_factor)) return ATTN_ERR_INVALID_ARG;
  const int kind = scaling;
  if (kind < ATTN_ROPE_NONE || kind > ATTN_ROPE_BY_PARTS) return ATTN_ERR_INVALID_ARG;
  if (kind != ATTN_ROPE_NONE && !(factor > 0.0 && std::isfinite(factor))) return ATTN_ERR_INVALID_ARG;
  if (kind == ATTN_ROPE_NTK && rot_dim < 4) return ATTN_ERR_INVALID_ARG;
  if (kind == ATTN_ROPE_BY_PARTS &&
      (orig_max_pos == 0 || !std::isfinite(beta_fast) || !std::isfinite(beta_slow) || !(beta_fast > beta_slow)))
    return ATTN_ERR_INVALID_ARG;
  if (max_pos == 0) return ATTN_OK;
  if (table == nullptr || !aligned(table, 4)) return ATTN_ERR_INVALID_ARG;
  const RopeScale sc{kind, base, factor, (double)orig_max_pos, beta_fast, beta_slow, attn_factor};
  return launch_rope_table_scaled(table, max_pos, (int)rot_dim, sc, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int attn_rope_apply(const void* x, void* y, attn_dtype_t dtype, uint32_t rows, uint32_t heads,
                               uint32_t head_dim, uint32_t rot_dim, uint32_t x_stride, uint32_t y_stride,
                               attn_rope_layout_t layout, const uint32_t* positions, const float* table,
                               uint32_t table_rows, int inverse, attn_stream_t stream) {
  if (!dtype_ok(dtype) || !layout_ok(layout)) return ATTN_ERR_INVALID_ARG;
  if (heads == 0 || heads > (1u << 20) || head_dim == 0 || head_dim > 1024) return ATTN_ERR_INVALID_ARG;
  if (rot_dim == 0 || rot_dim % 2 != 0 || rot_dim > head_dim) return ATTN_ERR_INVALID_ARG;
  if (x_stride < (uint64_t)heads * head_dim || y_stride < (uint64_t)heads * head_dim) return ATTN_ERR_INVALID_ARG;
  if (x == y && x_stride != y_stride) return ATTN_ERR_INVALID_ARG;
  if (positions == nullptr && table_rows < rows) return ATTN_ERR_INVALID_ARG;
  if (rows == 0) return ATTN_OK;
  if (x == nullptr || y == nullptr || table == nullptr) return ATTN_ERR_INVALID_ARG;
  if (!aligned(x, esize(dtype)) || !aligned(y, esize(dtype)) || !aligned(table, 4) || !aligned(positions, 4))
    return ATTN_ERR_INVALID_ARG;
  RopeArgs a{};
  a.x = x;
  a.y = y;
  a.positions = positions;
  a.table = table;
  a.status = device_status_word();
  if (a.status == nullptr) return ATTN_ERR_CUDA;
  a.x_stride = x_stride;
  a.y_stride = y_stride;
  a.rows = rows;
  a.table_rows = table_rows;
  a.heads = (int)heads;
  a.D = (int)head_dim;
  a.R = (int)rot_dim;
  a.interleaved = layout == ATTN_ROPE_INTERLEAVED;
  a.sgn = inverse ? -1.f : 1.f;
  return launch_rope_apply(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int attn_append_paged(const void* q, void* q_out, const void* k_new, const void* v_new, attn_dtype_t dtype,
                                 void* k_pages, void* v_pages, attn_dtype_t cache_dtype, const uint32_t* block_table,
                                 const uint32_t* q_start, const uint32_t* kv_len, uint32_t total_rows, uint32_t n_seqs,
                                 uint32_t num_heads, uint32_t num_kv_heads, uint32_t head_dim, uint32_t kv_dim,
                                 uint32_t q_stride, uint32_t q_out_stride, uint32_t k_stride, uint32_t v_stride,
                                 uint32_t page_rows, uint32_t num_pages, uint32_t max_blocks, uint32_t rot_dim,
                                 attn_rope_layout_t layout, const float* table, uint32_t table_rows,
                                 attn_stream_t stream) {
  if (!dtype_ok(dtype) || !dtype_ok(cache_dtype) || !layout_ok(layout)) return ATTN_ERR_INVALID_ARG;
  if (!heads_ok(num_heads > 0 ? num_heads : num_kv_heads, num_kv_heads, head_dim)) return ATTN_ERR_INVALID_ARG;
  if (!paged_ok(page_rows, num_pages, max_blocks)) return ATTN_ERR_INVALID_ARG;
  const uint64_t w = (uint64_t)num_kv_heads * head_dim, wq = (uint64_t)num_heads * head_dim;
  if (kv_dim < w || k_stride < w || v_stride < w) return ATTN_ERR_INVALID_ARG;
  if (num_heads > 0 && (q_stride < wq || q_out_stride < wq)) return ATTN_ERR_INVALID_ARG;
  if (rot_dim % 2 != 0 || rot_dim > head_dim || (rot_dim > 0 && (table == nullptr || table_rows == 0)))
    return ATTN_ERR_INVALID_ARG;
  // (The search of a row's sequence adds to n_seqs in 32 bits.)
  if (total_rows > 0x7fffffffu || n_seqs > (1u << 30)) return ATTN_ERR_INVALID_ARG;
  if (total_rows == 0 || n_seqs == 0) return ATTN_OK;  // (tensors of no rows have no address)
  if ((num_heads == 0) != (q == nullptr) || (num_heads > 0 && q_out == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (k_new == nullptr || v_new == nullptr || k_pages == nullptr || v_pages == nullptr || block_table == nullptr ||
      q_start == nullptr || kv_len == nullptr)
    return ATTN_ERR_INVALID_ARG;
  if (dtype != ATTN_DT_F32 && dtype != cache_dtype) return ATTN_ERR_UNSUPPORTED;
  if (q != nullptr && q == q_out && (q_stride != q_out_stride || dtype != cache_dtype)) return ATTN_ERR_INVALID_ARG;
  const size_t ei = esize(dtype), ec = esize(cache_dtype);
  if (!aligned(q, ei) || !aligned(k_new, ei) || !aligned(v_new, ei) || !aligned(q_out, ec) || !aligned(k_pages, ec) ||
      !aligned(v_pages, ec) || !aligned(table, 4) || !aligned(block_table, 4) || !aligned(q_start, 4) ||
      !aligned(kv_len, 4))
    return ATTN_ERR_INVALID_ARG;
  AppendArgs a{};
  a.q = q;
  a.q_out = q_out;
  a.k = k_new;
  a.v = v_new;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.block_table = block_table;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.table = rot_dim > 0 ? table : nullptr;
  a.status = device_status_word();
  if (a.status == nullptr) return ATTN_ERR_CUDA;
  a.q_stride = num_heads > 0 ? q_stride : 0;
  a.q_out_stride = num_heads > 0 ? q_out_stride : 0;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.kv_dim = kv_dim;
  a.total_rows = total_rows;
  a.table_rows = table_rows;
  a.n_seqs = (int)n_seqs;
  a.H = (int)num_heads;
  a.G = (int)num_kv_heads;
  a.D = (int)head_dim;
  a.R = (int)rot_dim;
  a.page_rows = (int)page_rows;
  a.num_pages = (int)num_pages;
  a.max_blocks = (int)max_blocks;
  a.interleaved = layout == ATTN_ROPE_INTERLEAVED;
  return launch_append_paged(a, dtype, cache_dtype, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t attn_batch_paged_workspace_bytes(uint32_t n_heads, uint32_t n_kv_heads, uint32_t head_dim) {
  if (!heads_ok(n_heads, n_kv_heads, head_dim)) return 0;
  const int sms = device_sm_count();
  return sms > 0 ? batch_workspace_bytes((int)head_dim, sms) : 0;
}

extern "C" int attn_batch_paged(const void* q, const void* k_pages, const void* v_pages, void* out, attn_dtype_t dtype,
                                const uint32_t* block_table, const uint32_t* q_start, const uint32_t* kv_len,
                                uint32_t total_rows, uint32_t n_seqs, uint32_t n_heads, uint32_t n_kv_heads,
                                uint32_t head_dim, uint32_t kv_dim, uint32_t q_stride, uint32_t out_stride,
                                uint32_t page_rows, uint32_t num_pages, uint32_t max_blocks, float scale,
                                uint32_t window, float softcap, const float* alibi_slopes, const uint32_t* prefix_len,
                                void* workspace, size_t workspace_bytes, attn_stream_t stream) {
  return batch_paged(q, k_pages, v_pages, nullptr, nullptr, out, dtype, block_table, q_start, kv_len, total_rows, n_seqs,
                     n_heads, n_kv_heads, head_dim, kv_dim, q_stride, out_stride, page_rows, num_pages, max_blocks, 0,
                     scale, window, 0, softcap, alibi_slopes, prefix_len, workspace, workspace_bytes, stream);
}

extern "C" int attn_batch_paged_sinks(const void* q, const void* k_pages, const void* v_pages, void* out,
                                      attn_dtype_t dtype, const uint32_t* block_table, const uint32_t* q_start,
                                      const uint32_t* kv_len, uint32_t total_rows, uint32_t n_seqs, uint32_t n_heads,
                                      uint32_t n_kv_heads, uint32_t head_dim, uint32_t kv_dim, uint32_t q_stride,
                                      uint32_t out_stride, uint32_t page_rows, uint32_t num_pages, uint32_t max_blocks,
                                      float scale, uint32_t window, float softcap, const float* alibi_slopes,
                                      const uint32_t* prefix_len, void* workspace, size_t workspace_bytes,
                                      uint32_t sinks, attn_stream_t stream) {
  return batch_paged(q, k_pages, v_pages, nullptr, nullptr, out, dtype, block_table, q_start, kv_len, total_rows, n_seqs,
                     n_heads, n_kv_heads, head_dim, kv_dim, q_stride, out_stride, page_rows, num_pages, max_blocks, 0,
                     scale, window, sinks, softcap, alibi_slopes, prefix_len, workspace, workspace_bytes, stream);
}

extern "C" int attn_batch_paged8(const void* q, const void* k_pages, const void* v_pages, const uint8_t* k_scales,
                                 const uint8_t* v_scales, void* out, attn_dtype_t dtype, const uint32_t* block_table,
                                 const uint32_t* q_start, const uint32_t* kv_len, uint32_t total_rows, uint32_t n_seqs,
                                 uint32_t n_heads, uint32_t n_kv_heads, uint32_t head_dim, uint32_t kv_dim,
                                 uint32_t q_stride, uint32_t out_stride, uint32_t page_rows, uint32_t num_pages,
                                 uint32_t max_blocks, uint32_t scale_rows, float scale, uint32_t window, uint32_t sinks,
                                 float softcap, const float* alibi_slopes, const uint32_t* prefix_len, void* workspace,
                                 size_t workspace_bytes, attn_stream_t stream) {
  if (scale_rows == 0 || page_rows % scale_rows != 0) return ATTN_ERR_INVALID_ARG;
  if (total_rows > 0 && n_seqs > 0 && (k_scales == nullptr || v_scales == nullptr)) return ATTN_ERR_INVALID_ARG;
  return batch_paged(q, k_pages, v_pages, k_scales, v_scales, out, dtype, block_table, q_start, kv_len, total_rows,
                     n_seqs, n_heads, n_kv_heads, head_dim, kv_dim, q_stride, out_stride, page_rows, num_pages,
                     max_blocks, scale_rows, scale, window, sinks, softcap, alibi_slopes, prefix_len, workspace,
                     workspace_bytes, stream);
}
