// cache8_api.cu -- the C ABI of the head norms and of the 8-bit paged cache
// (declared in include/attn_gqa.h): argument checks and launches.
#include <cmath>
#include <cstdint>

#include "../../include/attn_gqa.h"
#include "batch.h"
#include "common.cuh"
#include "internal.h"

using namespace attn;

namespace {

bool dtype_ok(int t) { return t == ATTN_DT_F32 || t == ATTN_DT_BF16 || t == ATTN_DT_F16; }
size_t esize(int t) { return t == ATTN_DT_F32 ? 4 : 2; }
bool layout_ok(int l) { return l == ATTN_ROPE_HALF || l == ATTN_ROPE_INTERLEAVED; }
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
// Smaller ones could vanish beside a mean of squares, and rsqrt of a subnormal is not one of fp32's.
bool eps_ok(float eps) { return std::isfinite(eps) && eps >= 1e-30f; }
bool turn_ok(uint32_t rot_dim, uint32_t head_dim, const float* table) {
  return rot_dim % 2 == 0 && rot_dim <= head_dim && (rot_dim == 0 || (table != nullptr && aligned(table, 4)));
}

// Arguments that the forward and the backward share.
int norm_args(NormArgs& a, const void* q, const void* k, void* q_out, void* k_out, const void* q_weight,
              const void* k_weight, int dtype, int w_dtype, uint32_t rows, uint32_t num_heads, uint32_t num_kv_heads,
              uint32_t head_dim, uint32_t q_stride, uint32_t k_stride, uint32_t q_out_stride, uint32_t k_out_stride,
              float eps, uint32_t rot_dim, int layout, const uint32_t* positions, const float* table,
              uint32_t table_rows) {
  if (!dtype_ok(dtype) || !dtype_ok(w_dtype) || !layout_ok(layout) || !eps_ok(eps)) return ATTN_ERR_INVALID_ARG;
  if (num_heads + num_kv_heads == 0 || num_heads > (1u << 20) || num_kv_heads > (1u << 20) || head_dim == 0 ||
      head_dim > 256)
    return ATTN_ERR_INVALID_ARG;
  if (!turn_ok(rot_dim, head_dim, table) || !aligned(positions, 4)) return ATTN_ERR_INVALID_ARG;
  if (rot_dim > 0 && positions == nullptr && table_rows < rows) return ATTN_ERR_INVALID_ARG;
  const uint64_t wq = (uint64_t)num_heads * head_dim, wk = (uint64_t)num_kv_heads * head_dim;
  if (q_stride < wq || q_out_stride < wq || k_stride < wk || k_out_stride < wk) return ATTN_ERR_INVALID_ARG;
  if ((q == q_out && q_stride != q_out_stride && num_heads > 0) ||
      (k == k_out && k_stride != k_out_stride && num_kv_heads > 0))
    return ATTN_ERR_INVALID_ARG;
  const size_t e = esize(dtype), ew = esize(w_dtype);
  if (rows > 0 && num_heads > 0 && (q == nullptr || q_out == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (rows > 0 && num_kv_heads > 0 && (k == nullptr || k_out == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, e) || !aligned(k, e) || !aligned(q_out, e) || !aligned(k_out, e) || !aligned(q_weight, ew) ||
      !aligned(k_weight, ew))
    return ATTN_ERR_INVALID_ARG;
  a.q.x = q;
  a.q.y = q_out;
  a.q.weight = q_weight;
  a.q.x_stride = q_stride;
  a.q.y_stride = q_out_stride;
  a.q.heads = (int)num_heads;
  a.k.x = k;
  a.k.y = k_out;
  a.k.weight = k_weight;
  a.k.x_stride = k_stride;
  a.k.y_stride = k_out_stride;
  a.k.heads = (int)num_kv_heads;
  if (num_heads == 0) a.q = NormTensor{};
  if (num_kv_heads == 0) a.k = NormTensor{};
  a.positions = positions;
  a.table = rot_dim > 0 ? table : nullptr;
  a.rows = rows;
  a.table_rows = table_rows;
  a.D = (int)head_dim;
  a.R = (int)rot_dim;
  a.w_dtype = w_dtype;
  a.interleaved = layout == ATTN_ROPE_INTERLEAVED;
  a.eps = eps;
  return ATTN_OK;
}

// Checks of a batch over an 8-bit cache.
bool cache_ok(uint32_t num_kv_heads, uint32_t head_dim, uint32_t kv_dim, uint32_t page_rows, uint32_t num_pages,
              uint32_t max_blocks, uint32_t scale_rows) {
  return num_kv_heads >= 1 && num_kv_heads <= (1u << 20) && head_dim >= 1 && head_dim <= 128 &&
         kv_dim >= (uint64_t)num_kv_heads * head_dim && page_rows >= 1 && num_pages >= 1 && max_blocks >= 1 &&
         (uint64_t)page_rows * max_blocks <= 0x7fffffffu && (uint64_t)page_rows * num_pages <= 0x7fffffffu &&
         scale_rows >= 1 && page_rows % scale_rows == 0;
}
bool cache_layout_ok(uint32_t head_dim, uint32_t kv_dim, const void* k_pages, const void* v_pages) {
  return head_dim % 16 == 0 && kv_dim % 16 == 0 && aligned(k_pages, 16) && aligned(v_pages, 16);
}

}  // namespace

extern "C" int attn_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, const void* q_weight,
                                 const void* k_weight, attn_dtype_t dtype, attn_dtype_t weight_dtype, uint32_t rows,
                                 uint32_t num_heads, uint32_t num_kv_heads, uint32_t head_dim, uint32_t q_stride,
                                 uint32_t k_stride, uint32_t q_out_stride, uint32_t k_out_stride, float eps,
                                 uint32_t rot_dim, attn_rope_layout_t layout, const uint32_t* positions,
                                 const float* table, uint32_t table_rows, attn_stream_t stream) {
  NormArgs a{};
  const int rc = norm_args(a, q, k, q_out, k_out, q_weight, k_weight, dtype, weight_dtype, rows, num_heads,
                           num_kv_heads, head_dim, q_stride, k_stride, q_out_stride, k_out_stride, eps, rot_dim, layout,
                           positions, table, table_rows);
  if (rc != ATTN_OK || rows == 0) return rc;
  const int sms = device_sm_count();
  a.status = device_status_word();
  if (sms <= 0 || a.status == nullptr) return ATTN_ERR_CUDA;
  return launch_qk_norm(a, dtype, false, sms, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t attn_qk_norm_rope_backward_workspace_bytes(uint32_t head_dim) {
  const int sms = device_sm_count();
  return head_dim >= 1 && head_dim <= 256 && sms > 0 ? qk_norm_workspace_bytes((int)head_dim, sms) : 0;
}

extern "C" int attn_qk_norm_rope_backward(const void* dq, const void* dk, const void* q, const void* k, void* dq_out,
                                          void* dk_out, const void* q_weight, const void* k_weight, void* dq_weight,
                                          void* dk_weight, attn_dtype_t dtype, attn_dtype_t weight_dtype, uint32_t rows,
                                          uint32_t num_heads, uint32_t num_kv_heads, uint32_t head_dim,
                                          uint32_t dq_stride, uint32_t dk_stride, uint32_t q_stride, uint32_t k_stride,
                                          uint32_t dq_out_stride, uint32_t dk_out_stride, float eps, uint32_t rot_dim,
                                          attn_rope_layout_t layout, const uint32_t* positions, const float* table,
                                          uint32_t table_rows, void* workspace, size_t workspace_bytes,
                                          attn_stream_t stream) {
  NormArgs a{};
  const int rc = norm_args(a, q, k, dq_out, dk_out, q_weight, k_weight, dtype, weight_dtype, rows, num_heads,
                           num_kv_heads, head_dim, q_stride, k_stride, dq_out_stride, dk_out_stride, eps, rot_dim,
                           layout, positions, table, table_rows);
  if (rc != ATTN_OK) return rc;
  const size_t e = esize(dtype), ew = esize(weight_dtype);
  if (dq_stride < (uint64_t)num_heads * head_dim || dk_stride < (uint64_t)num_kv_heads * head_dim ||
      (num_heads > 0 && rows > 0 && dq == nullptr) || (num_kv_heads > 0 && rows > 0 && dk == nullptr) ||
      !aligned(dq, e) || !aligned(dk, e) || !aligned(dq_weight, ew) || !aligned(dk_weight, ew) ||
      (num_heads > 0 && dq == dq_out && dq_stride != dq_out_stride) ||
      (num_kv_heads > 0 && dk == dk_out && dk_stride != dk_out_stride))
    return ATTN_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (num_heads > 0) a.q.dy = dq, a.q.dy_stride = dq_stride, a.q.dw = dq_weight;
  if (num_kv_heads > 0) a.k.dy = dk, a.k.dy_stride = dk_stride, a.k.dw = dk_weight;
  // A sum over no rows or no heads.
  if ((rows == 0 || num_heads == 0) && dq_weight != nullptr && cudaMemsetAsync(dq_weight, 0, head_dim * ew, s) != cudaSuccess)
    return ATTN_ERR_CUDA;
  if ((rows == 0 || num_kv_heads == 0) && dk_weight != nullptr && cudaMemsetAsync(dk_weight, 0, head_dim * ew, s) != cudaSuccess)
    return ATTN_ERR_CUDA;
  if (rows == 0) return ATTN_OK;
  const int sms = device_sm_count();
  a.status = device_status_word();
  if (sms <= 0 || a.status == nullptr) return ATTN_ERR_CUDA;
  if ((a.q.dw != nullptr || a.k.dw != nullptr) &&
      (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < qk_norm_workspace_bytes((int)head_dim, sms)))
    return ATTN_ERR_INVALID_ARG;
  a.partial = static_cast<float*>(workspace);
  return launch_qk_norm(a, dtype, true, sms, s);
}

extern "C" int attn_append_paged8(const void* q, void* q_out, const void* k_new, const void* v_new, attn_dtype_t dtype,
                                  attn_dtype_t q_out_dtype, void* k_pages, void* v_pages, uint8_t* k_scales,
                                  uint8_t* v_scales, const uint32_t* block_table, const uint32_t* q_start,
                                  const uint32_t* kv_len, uint32_t total_rows, uint32_t n_seqs, uint32_t num_heads,
                                  uint32_t num_kv_heads, uint32_t head_dim, uint32_t kv_dim, uint32_t q_stride,
                                  uint32_t q_out_stride, uint32_t k_stride, uint32_t v_stride, uint32_t page_rows,
                                  uint32_t num_pages, uint32_t max_blocks, uint32_t scale_rows, const void* q_weight,
                                  const void* k_weight, attn_dtype_t weight_dtype, float eps, uint32_t rot_dim,
                                  attn_rope_layout_t layout, const float* table, uint32_t table_rows,
                                  attn_stream_t stream) {
  if (!dtype_ok(dtype) || !dtype_ok(weight_dtype) || !layout_ok(layout)) return ATTN_ERR_INVALID_ARG;
  if (!cache_ok(num_kv_heads, head_dim, kv_dim, page_rows, num_pages, max_blocks, scale_rows))
    return ATTN_ERR_INVALID_ARG;
  if (num_heads > (1u << 20)) return ATTN_ERR_INVALID_ARG;
  if (num_heads == 0 && q_weight != nullptr) return ATTN_ERR_INVALID_ARG;
  if (num_heads > 0 && q_out_dtype != ATTN_DT_BF16 && q_out_dtype != ATTN_DT_F16) return ATTN_ERR_INVALID_ARG;
  const uint64_t w = (uint64_t)num_kv_heads * head_dim, wq = (uint64_t)num_heads * head_dim;
  if (k_stride < w || v_stride < w || (num_heads > 0 && (q_stride < wq || q_out_stride < wq))) return ATTN_ERR_INVALID_ARG;
  if (!turn_ok(rot_dim, head_dim, table) || (rot_dim > 0 && table_rows == 0)) return ATTN_ERR_INVALID_ARG;
  if ((q_weight != nullptr || k_weight != nullptr) && !eps_ok(eps)) return ATTN_ERR_INVALID_ARG;
  // (The search of a row's sequence adds to n_seqs in 32 bits.)
  if (total_rows > 0x7fffffffu || n_seqs > (1u << 30)) return ATTN_ERR_INVALID_ARG;
  if (total_rows == 0 || n_seqs == 0) return ATTN_OK;  // (tensors of no rows have no address)
  if ((num_heads == 0) != (q == nullptr) || (num_heads > 0 && q_out == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (k_new == nullptr || v_new == nullptr || k_pages == nullptr || v_pages == nullptr || k_scales == nullptr ||
      v_scales == nullptr || block_table == nullptr || q_start == nullptr || kv_len == nullptr)
    return ATTN_ERR_INVALID_ARG;
  if (num_heads > 0 && dtype != ATTN_DT_F32 && dtype != q_out_dtype) return ATTN_ERR_UNSUPPORTED;
  if (q != nullptr && q == q_out && (q_stride != q_out_stride || dtype != q_out_dtype)) return ATTN_ERR_INVALID_ARG;
  const size_t ei = esize(dtype), ew = esize(weight_dtype);
  if (!aligned(q, ei) || !aligned(k_new, ei) || !aligned(v_new, ei) || !aligned(q_out, 2) || !aligned(block_table, 4) ||
      !aligned(q_start, 4) || !aligned(kv_len, 4) || !aligned(q_weight, ew) || !aligned(k_weight, ew))
    return ATTN_ERR_INVALID_ARG;
  if (!cache_layout_ok(head_dim, kv_dim, k_pages, v_pages)) return ATTN_ERR_UNSUPPORTED;
  const int sms = device_sm_count();
  if (sms <= 0) return ATTN_ERR_CUDA;
  Append8Args a{};
  a.q = q;
  a.q_out = q_out;
  a.k = k_new;
  a.v = v_new;
  a.k_pages = static_cast<uint8_t*>(k_pages);
  a.v_pages = static_cast<uint8_t*>(v_pages);
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
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
  a.scale_rows = (int)scale_rows;
  a.w_dtype = weight_dtype;
  a.interleaved = layout == ATTN_ROPE_INTERLEAVED;
  a.eps = eps;
  return launch_append8(a, dtype, q_out_dtype, sms, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int attn_read_paged8(const void* k_pages, const void* v_pages, const uint8_t* k_scales,
                                const uint8_t* v_scales, void* k_out, void* v_out, attn_dtype_t dtype,
                                const uint32_t* block_table, const uint32_t* starts, const uint32_t* first,
                                const uint32_t* kv_len, uint32_t total_rows, uint32_t n_seqs, uint32_t num_kv_heads,
                                uint32_t head_dim, uint32_t kv_dim, uint32_t k_stride, uint32_t v_stride,
                                uint32_t page_rows, uint32_t num_pages, uint32_t max_blocks, uint32_t scale_rows,
                                attn_stream_t stream) {
  if (!dtype_ok(dtype) || !cache_ok(num_kv_heads, head_dim, kv_dim, page_rows, num_pages, max_blocks, scale_rows))
    return ATTN_ERR_INVALID_ARG;
  const uint64_t w = (uint64_t)num_kv_heads * head_dim;
  if (k_stride < w || v_stride < w || total_rows > 0x7fffffffu || n_seqs > (1u << 30)) return ATTN_ERR_INVALID_ARG;
  if (total_rows == 0 || n_seqs == 0) return ATTN_OK;
  if (k_pages == nullptr || v_pages == nullptr || k_scales == nullptr || v_scales == nullptr || k_out == nullptr ||
      v_out == nullptr || block_table == nullptr || starts == nullptr || kv_len == nullptr)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(k_out, esize(dtype)) || !aligned(v_out, esize(dtype)) || !aligned(block_table, 4) ||
      !aligned(starts, 4) || !aligned(first, 4) || !aligned(kv_len, 4))
    return ATTN_ERR_INVALID_ARG;
  if (!cache_layout_ok(head_dim, kv_dim, k_pages, v_pages)) return ATTN_ERR_UNSUPPORTED;
  Read8Args a{};
  a.k_pages = static_cast<const uint8_t*>(k_pages);
  a.v_pages = static_cast<const uint8_t*>(v_pages);
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.k_out = k_out;
  a.v_out = v_out;
  a.block_table = block_table;
  a.starts = starts;
  a.first = first;
  a.kv_len = kv_len;
  a.status = device_status_word();
  if (a.status == nullptr) return ATTN_ERR_CUDA;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.kv_dim = kv_dim;
  a.total_rows = total_rows;
  a.n_seqs = (int)n_seqs;
  a.G = (int)num_kv_heads;
  a.D = (int)head_dim;
  a.page_rows = (int)page_rows;
  a.num_pages = (int)num_pages;
  a.max_blocks = (int)max_blocks;
  a.scale_rows = (int)scale_rows;
  return launch_read8(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}
