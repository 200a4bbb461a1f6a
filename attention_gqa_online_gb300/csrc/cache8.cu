// cache8.cu -- the 8-bit paged cache: the new tokens of a ragged batch written
// into it (K normed and turned on the way, Q too), and ranges of positions read
// back.  The numbers are those of cache8.cuh.
//
// Append.  A scale belongs to scale_rows positions of a kv head, so whoever
// rounds one of them needs the largest magnitude of all.  A team of threads takes
// one block of positions and one kv head of K or V: it reads the block's new rows
// (one a thread stays in registers as fp32, more are read again), finds the
// largest magnitude and with it the scale, and stores the codes.  The first
// block of a sequence may hold older rows; they count by the scale that they have,
// and where the new scale is larger their codes are multiplied and rounded again.
// A block belongs to the team whose chunk of token rows holds the block's first
// new row, so nothing is left to atomics and results do not depend on order.
// Bound by the chain of lookups (sequence, length, page, table row) before each
// row of Q and each block of K and V: 4 chunks of up to 2048 rows, 32 + 2 x 8 heads
// of 128, bf16, 48 us, 3.1 TB/s (0.47 of a copy's rate); one token of 64 sequences
// 4.9 us (in a graph).
//
// Read.  Sixteen codes a thread; bound by the 16- or 32-bit rows it writes: 17
// sequences of up to 8192, 8 heads of 128, to bf16 62 us, 6.1 TB/s (0.92).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "batch.h"
#include "cache8.cuh"
#include "common.cuh"
#include "find_seq.cuh"
#include "internal.h"
#include "norm_rope.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kKeep = 1;  // rows of a thread that stay in registers between the maximum and the codes

// A row of a head in a lane's registers: the pairs of a unit, or (scalar) four columns in a.
template <bool INTER, bool VEC>
struct Held {
  static constexpr int P = VEC ? norm::Unit<INTER>::P : 4;
  float a[P], b[VEC ? P : 1];
};

// What a lane needs of a tensor's rows whatever the row.
template <bool INTER, bool VEC>
struct Head {
  norm::Unit<INTER> u;
  const void* weight;  // nullptr: not normed
  bool turn;
  int lane;       // of the head
  unsigned mask;  // the head's lanes
  __device__ __forceinline__ Head(const Append8Args& a, const void* w, int R_geo, bool t)
      : u(threadIdx.x & (a.lanes - 1), a.D, R_geo), weight(w), turn(t), lane(threadIdx.x & (a.lanes - 1)),
        mask(a.lanes == 32 ? 0xffffffffu : ((1u << a.lanes) - 1u) << (threadIdx.x & 31 & ~(a.lanes - 1))) {}
};

// The row x of a head (its first column), normed and turned; (vector form) as it lies in memory in `raw`.
template <typename TI, bool INTER, bool VEC>
__device__ __forceinline__ void make_row(const Append8Args& a, const TI* x, const norm::Raw<TI, INTER>& raw, uint32_t pos,
                                         const Head<INTER, VEC>& hd, Held<INTER, VEC>& out) {
  const float* tab = a.table + (long long)pos * a.R;
  const float inv_d = 1.f / (float)a.D;
  if constexpr (VEC) {
    constexpr int P = Held<INTER, VEC>::P;
    norm::unpack(raw, out.a, out.b);
    if (hd.weight != nullptr) {
      float wa[P], wb[P];
      norm::load_weight(hd.weight, a.w_dtype, hd.u, wa, wb);
      const float rms = rsqrtf(fmaf(norm::head_sum(norm::squares(hd.u, out.a, out.b), a.lanes, hd.mask), inv_d, a.eps));
#pragma unroll
      for (int i = 0; i < P; ++i) {
        out.a[i] *= rms * wa[i];
        out.b[i] *= rms * wb[i];
      }
    }
    if (hd.turn && hd.u.turned) {  // (others as they are, not + 0 * a column that may hold an infinity)
      float c[P], s[P];
      norm::load_turn(tab, a.R, hd.u, true, c, s);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float va = out.a[i], vb = out.b[i];
        out.a[i] = va * c[i] - vb * s[i];
        out.b[i] = vb * c[i] + va * s[i];
      }
    }
  } else {
    float rms = 1.f;
    if (hd.weight != nullptr) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v = hd.lane + 32 * j < a.D ? rot::to_f32(x[hd.lane + 32 * j]) : 0.f;
        sum = fmaf(v, v, sum);
      }
      rms = rsqrtf(fmaf(norm::head_sum(sum, 32, hd.mask), inv_d, a.eps));
    }
    auto z = [&](int d) {
      const float v = rot::to_f32(x[d]);
      return hd.weight != nullptr ? v * (rms * norm::weight_at(hd.weight, a.w_dtype, d)) : v;
    };
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int d = hd.lane + 32 * j;
      out.a[j] = 0.f;
      if (d < a.D)
        out.a[j] = hd.turn ? norm::turned_column<1>(norm::column_of<INTER>(d, a.R), tab, a.R, true, z) : z(d);
    }
  }
}

template <typename TI, bool INTER, bool VEC>
__device__ __forceinline__ void load_row(const Append8Args& a, const TI* x, uint32_t pos, const Head<INTER, VEC>& hd,
                                         Held<INTER, VEC>& out) {
  norm::Raw<TI, INTER> raw{};
  if constexpr (VEC) norm::load_raw(x, hd.u, raw);
  make_row<TI, INTER, VEC>(a, x, raw, pos, hd, out);
}

// Largest magnitude of a lane's own columns (a NaN leaves it).
template <bool INTER, bool VEC>
__device__ __forceinline__ float held_max(const Held<INTER, VEC>& h, const Head<INTER, VEC>& hd) {
  float m = 0.f, mb = 0.f;
#pragma unroll
  for (int i = 0; i < Held<INTER, VEC>::P; ++i) {
    m = fmaxf(m, fabsf(h.a[i]));
    if constexpr (VEC) mb = fmaxf(mb, fabsf(h.b[i]));
  }
  if constexpr (VEC) m = fmaxf(hd.u.any ? m : 0.f, hd.u.both ? mb : 0.f);
  return m;
}
template <bool INTER, bool VEC>
__device__ __forceinline__ void store_codes(const Held<INTER, VEC>& h, float mul, uint8_t* dst, const Head<INTER, VEC>& hd,
                                            int D) {
  if constexpr (VEC) {
    float v[8];
    auto eight = [&](int c) {
      *reinterpret_cast<uint2*>(dst + c) = make_uint2(c8::from_float4(v[0] * mul, v[1] * mul, v[2] * mul, v[3] * mul),
                                                      c8::from_float4(v[4] * mul, v[5] * mul, v[6] * mul, v[7] * mul));
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = INTER ? (i & 1 ? h.b[i / 2] : h.a[i / 2]) : h.a[i % Held<INTER, VEC>::P];
    if (hd.u.any) eight(hd.u.c0);
    if constexpr (!INTER) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = h.b[i];
      if (hd.u.both) eight(hd.u.c1);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (hd.lane + 32 * j < D) dst[hd.lane + 32 * j] = (uint8_t)c8::from_float2(h.a[j] * mul, 0.f);
  }
}

struct Team {
  int size, id, thread;  // threads of a team, this team of the block, this thread of the team
  int row, rows;         // the thread's first row of a block, and rows at once
  float* red;            // [warps of the block], shared memory
  __device__ __forceinline__ unsigned mask() const {
    return size >= 32 ? 0xffffffffu : ((1u << size) - 1u) << (threadIdx.x & 31 & ~(size - 1));
  }
  __device__ __forceinline__ void sync() const {
    if (size > 32)
      named_barrier(1 + id, size);
    else
      __syncwarp(mask());
  }
  // Largest of m over the team.
  __device__ __forceinline__ float max(float m) const {
    const int w = size < 32 ? size : 32, lane = threadIdx.x & 31;
    for (int d = w >> 1; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(mask(), m, d));
    if (size > 32) {
      const int warp = threadIdx.x >> 5, w0 = id * (size >> 5);
      if (lane == 0) red[warp] = m;
      named_barrier(1 + id, size);
      m = 0.f;
      for (int k = 0; k < (size >> 5); ++k) m = fmaxf(m, red[w0 + k]);
      named_barrier(1 + id, size);  // red may be written again
    }
    return m;
  }
};

// One block of positions of one kv head: token rows [row0, row0 + m) at
// positions pos0 ... of pool page `page`; `held` older rows stand before them.
template <typename TI, bool INTER, bool VEC>
__device__ __forceinline__ void write_block(const Append8Args& a, const Team& t, const TI* src, long long stride,
                                            uint8_t* pages, uint8_t* scales, int h, long long row0, int m,
                                            uint32_t pos0, uint32_t page, int held, const Head<INTER, VEC>& hd) {
  const TI* x = src + row0 * stride + (long long)h * a.D;
  Held<INTER, VEC> kept[kKeep];
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    const int r = t.row + k * t.rows;
    if (r < m) {
      load_row<TI, INTER, VEC>(a, x + r * stride, pos0 + r, hd, kept[k]);
      amax = fmaxf(amax, held_max<INTER, VEC>(kept[k], hd));
    }
  }
  for (int r = t.row + kKeep * t.rows; r < m; r += t.rows) {
    Held<INTER, VEC> v;
    load_row<TI, INTER, VEC>(a, x + r * stride, pos0 + r, hd, v);
    amax = fmaxf(amax, held_max<INTER, VEC>(v, hd));
  }
  const int e_new = c8::exp_for(t.max(amax));
  // (The page is looked at here, so that its lookup and the rows' loads are in flight together.)
  if (page >= (uint32_t)a.num_pages) {
    if (t.thread == 0) record_status(a.status, ATTN_ERR_INVALID_ARG);
    return;
  }
  const long long slot0 = (long long)page * a.page_rows + (pos0 - divide(pos0, a.by_page) * (uint32_t)a.page_rows);
  uint8_t* scale = scales + (long long)divide((uint32_t)slot0, a.by_scale) * a.G + h;
  uint8_t* dst = pages + slot0 * a.kv_dim + (long long)h * a.D;
  int e0 = c8::kMinExp;
  if (held > 0) {
    e0 = c8::exp_of(*scale);
    t.sync();  // all have read it
  }
  const int e = ::max(e0, e_new);
  if (held > 0 && e > e0) {  // the older rows move to the new scale
    const float mul = pow2f(e0 - e);
    const int words = a.D / 4;
    for (int i = t.thread; i < held * words; i += t.size) {
      const int r = i / words;
      uint32_t* p = reinterpret_cast<uint32_t*>(dst - (long long)(held - r) * a.kv_dim) + (i - r * words);
      float v[4];
      c8::to_float4(*p, v);
      *p = c8::from_float4(v[0] * mul, v[1] * mul, v[2] * mul, v[3] * mul);
    }
  }
  if (t.thread == 0) *scale = (uint8_t)(127 + e);
  const float mul = pow2f(-e);
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    const int r = t.row + k * t.rows;
    if (r < m) store_codes<INTER, VEC>(kept[k], mul, dst + (long long)r * a.kv_dim, hd, a.D);
  }
  for (int r = t.row + kKeep * t.rows; r < m; r += t.rows) {
    Held<INTER, VEC> v;
    load_row<TI, INTER, VEC>(a, x + r * stride, pos0 + r, hd, v);
    store_codes<INTER, VEC>(v, mul, dst + (long long)r * a.kv_dim, hd, a.D);
  }
}

// First sequence from s on that ends after row i (q_start ascends).
__device__ __forceinline__ int seq_after(const uint32_t* q_start, int n, int s, uint32_t i) {
  for (int k = 0; k < 4; ++k, ++s)
    if (s >= n || q_start[s + 1] > i) return s;
  int hi = n;
  while (s < hi) {
    const int mid = (s + hi) >> 1;
    if (q_start[mid + 1] > i)
      hi = mid;
    else
      s = mid + 1;
  }
  return s;
}

template <typename TI, typename TQ, bool INTER, bool VEC>
__device__ __forceinline__ void append_q(const Append8Args& a, int block) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long task = (long long)block * kWarps + warp;
  const long long row = task / a.q_splits;
  if (row >= a.total_rows) return;
  const int split = (int)(task - row * a.q_splits);
  const int s = find_seq(a.q_start, a.n_seqs, (uint32_t)row);
  if (s < 0) return;
  const uint32_t end = a.q_start[s + 1];
  if (row >= end) return;
  const long long pos = (long long)a.kv_len[s] - (long long)end + row;
  if (pos < 0 || pos >= (long long)a.page_rows * a.max_blocks || (a.R > 0 && pos >= (long long)a.table_rows) ||
      a.block_table[(long long)s * a.max_blocks + divide((uint32_t)pos, a.by_page)] >= (uint32_t)a.num_pages)
    return;  // (recorded by the row's keys)
  const int at_once = 32 / a.lanes, sub = lane / a.lanes;
  const Head<INTER, VEC> hd(a, a.q_weight, a.R > 0 ? a.R : a.D, a.R > 0);
  const TI* x = static_cast<const TI*>(a.q) + row * a.q_stride;
  TQ* y = static_cast<TQ*>(a.q_out) + row * a.q_out_stride;
  const int step = at_once * a.q_splits;
  if constexpr (VEC) {
    // y_a = r (a w_a c - b w_b s), y_b = r (b w_b c + a w_a s): what does not depend on the head is made once.  The next
    // head's loads are in flight while one is computed.
    constexpr int P = Held<INTER, VEC>::P;
    const norm::Unit<INTER>& u = hd.u;
    norm::Raw<TI, INTER> ahead;
    int h = split * at_once + sub;
    if (h < a.H) norm::load_raw(x + h * a.D, u, ahead);
    float wa[P], wb[P], ac[P], bs[P], bc[P], as[P];
    norm::load_weight(a.q_weight, a.w_dtype, u, wa, wb);
    if (a.R > 0) {
      norm::load_turn(a.table + pos * a.R, a.R, u, true, ac, as);
    } else {  // (u is then that of a head turned as a whole, and there is no table)
#pragma unroll
      for (int i = 0; i < P; ++i) ac[i] = 1.f, as[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      bc[i] = ac[i] * wb[i];
      bs[i] = -as[i] * wb[i];
      ac[i] *= wa[i];
      as[i] *= wa[i];
    }
    const float inv_d = 1.f / (float)a.D;
    const bool turned = a.R > 0 && u.turned;
    for (; h < a.H; h += step) {
      float va[P], vb[P], ya[P], yb[P];
      norm::unpack(ahead, va, vb);
      if (h + step < a.H) norm::load_raw(x + (h + step) * a.D, u, ahead);
      float r = 1.f;
      if (a.q_weight != nullptr)
        r = rsqrtf(fmaf(norm::head_sum(norm::squares(u, va, vb), a.lanes, hd.mask), inv_d, a.eps));
#pragma unroll
      for (int i = 0; i < P; i += 2) {
        const float2 ra = mul2_of(va[i], va[i + 1], r, r), rb = mul2_of(vb[i], vb[i + 1], r, r);
        float2 oa = mul2_of(ra.x, ra.y, ac[i], ac[i + 1]), ob = mul2_of(rb.x, rb.y, bc[i], bc[i + 1]);
        if (turned) {  // (not + 0 * the other column: that may be an infinity)
          oa = fma2_of(rb.x, rb.y, bs[i], bs[i + 1], oa);
          ob = fma2_of(ra.x, ra.y, as[i], as[i + 1], ob);
        }
        ya[i] = oa.x, ya[i + 1] = oa.y;
        yb[i] = ob.x, yb[i + 1] = ob.y;
      }
      norm::store_unit(y + h * a.D, u, ya, yb);
    }
  } else {
    const norm::Raw<TI, INTER> none{};
    for (int h = split * at_once + sub; h < a.H; h += step) {
      Held<INTER, VEC> v;
      make_row<TI, INTER, VEC>(a, x + (long long)h * a.D, none, (uint32_t)pos, hd, v);
      __syncwarp(hd.mask);  // the head's lanes have read it: y may be x
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (hd.lane + 32 * j < a.D) y[(long long)h * a.D + hd.lane + 32 * j] = rot::from_f32<TQ>(v.a[j]);
    }
  }
}

template <typename TI, typename TQ, bool INTER, bool VEC>
__global__ void __launch_bounds__(kThreads, 3) append8_kernel(const Append8Args a) {
  __shared__ float red[kWarps];
  if (blockIdx.x >= (unsigned)a.kv_blocks) {
    append_q<TI, TQ, INTER, VEC>(a, blockIdx.x - a.kv_blocks);
    return;
  }
  Team t;
  t.size = a.team;
  t.id = threadIdx.x / a.team;
  t.thread = threadIdx.x - t.id * a.team;
  t.row = t.thread / a.lanes;
  t.rows = a.team / a.lanes;
  t.red = red;
  const int teams = kThreads / a.team;
  const uint32_t first = blockIdx.x * (uint32_t)teams, item = first + t.id;  // (below 2^31)
  // All lanes of a warp look for the sequence of the warp's first row.
  const long long row_w = (long long)divide(first + (threadIdx.x & ~31) / a.team, a.by_heads) * a.chunk;
  if (row_w >= a.total_rows) return;
  int s = ::max(0, find_seq(a.q_start, a.n_seqs, (uint32_t)row_w));
  const uint32_t chunk = divide(item, a.by_heads);
  if ((long long)chunk * a.chunk >= a.total_rows) return;
  const int which = (int)(item - chunk * 2 * a.G);
  const bool is_v = which >= a.G;
  const int h = is_v ? which - a.G : which;
  uint32_t i = chunk * (uint32_t)a.chunk;
  const uint32_t i_end = (uint32_t)min((long long)a.total_rows, (long long)i + a.chunk);
  const int sr = a.scale_rows;
  while (i < i_end) {
    s = seq_after(a.q_start, a.n_seqs, s, i);
    if (s >= a.n_seqs) break;
    const uint32_t start = a.q_start[s], full_end = a.q_start[s + 1], end = min(full_end, a.total_rows);
    if (i < start) {  // rows of no sequence
      i = start;
      continue;
    }
    const long long pos = (long long)a.kv_len[s] - (long long)full_end + (long long)i;
    if (pos < 0) {  // rows before position 0
      if (t.thread == 0) record_status(a.status, ATTN_ERR_INVALID_ARG);
      i = (uint32_t)min((long long)end, (long long)i - pos);
      continue;
    }
    if (pos >= (long long)a.page_rows * a.max_blocks) {  // and all that follow
      if (t.thread == 0) record_status(a.status, ATTN_ERR_INVALID_ARG);
      i = end;
      continue;
    }
    const uint32_t p = (uint32_t)pos;
    const int in_block = (int)(p - divide(p, a.by_scale) * (uint32_t)sr);
    const int m = (int)min((uint32_t)(sr - in_block), end - i);
    if (in_block != 0 && i != start) {  // the block's first new row is in another chunk
      i += m;
      continue;
    }
    int take = m;
    if (a.R > 0) take = p < a.table_rows ? (int)min((uint32_t)m, a.table_rows - p) : 0;
    if (take < m && t.thread == 0) record_status(a.status, ATTN_ERR_INVALID_ARG);
    if (take > 0) {
      const uint32_t page = a.block_table[(long long)s * a.max_blocks + divide(p, a.by_page)];
      if (is_v)
        write_block<TI, false, VEC>(a, t, static_cast<const TI*>(a.v), a.v_stride, a.v_pages, a.v_scales, h, i, take,
                                    p, page, in_block, Head<false, VEC>(a, nullptr, a.D, false));
      else
        write_block<TI, INTER, VEC>(a, t, static_cast<const TI*>(a.k), a.k_stride, a.k_pages, a.k_scales, h, i, take,
                                    p, page, in_block,
                                    Head<INTER, VEC>(a, a.k_weight, a.R > 0 ? a.R : a.D, a.R > 0));
    }
    i += m;
  }
}

// ---------------------------------------------------------------- read
template <typename T>
__device__ __forceinline__ void store16(T* y, const float (&v)[16], bool vec) {
  if (vec) {
    float a[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] = v[i];
      b[i] = v[8 + i];
    }
    rot::store8<true>(y, a);
    rot::store8<true>(y + 8, b);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = rot::from_f32<T>(v[i]);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) read8_kernel(const Read8Args a) {
  __shared__ long long slot_s[kWarps];  // cache row, -1: zeros, -2: a row of no sequence
  const uint32_t row0 = blockIdx.x * (uint32_t)a.rows_per_block;
  const int nrows = (int)min((uint32_t)a.rows_per_block, a.total_rows - row0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < nrows) {
    const uint32_t row = row0 + warp;
    const int s = find_seq(a.starts, a.n_seqs, row);
    if (lane == 0) {
      long long slot = -2;
      if (s >= 0 && row < a.starts[s + 1]) {
        slot = -1;
        const long long pos = (long long)(a.first != nullptr ? a.first[s] : 0u) + (row - a.starts[s]);
        if (pos < (long long)a.kv_len[s] && pos < (long long)a.page_rows * a.max_blocks) {
          const uint32_t col = divide((uint32_t)pos, a.by_page);
          const uint32_t page = a.block_table[(long long)s * a.max_blocks + col];
          if (page < (uint32_t)a.num_pages)
            slot = (long long)page * a.page_rows + ((uint32_t)pos - col * (uint32_t)a.page_rows);
        }
        if (slot == -1) record_status(a.status, ATTN_ERR_INVALID_ARG);
      }
      slot_s[warp] = slot;
    }
  }
  __syncthreads();
  const int per = a.D / 16, half = a.G * per, upr = 2 * half;  // units of a head, of K, of a row
  T* const k_out = static_cast<T*>(a.k_out);
  T* const v_out = static_cast<T*>(a.v_out);
  for (int i = threadIdx.x; i < nrows * upr; i += kThreads) {
    const int r = i / upr;
    int u = i - r * upr;
    const long long slot = slot_s[r];
    if (slot == -2) continue;
    const bool is_v = u >= half;
    if (is_v) u -= half;
    const int h = u / per;
    float v[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] = 0.f;
    if (slot >= 0) {
      const uint4 c = __ldcs(reinterpret_cast<const uint4*>((is_v ? a.v_pages : a.k_pages) + slot * a.kv_dim + 16 * u));
      const uint8_t b = (is_v ? a.v_scales : a.k_scales)[(long long)divide((uint32_t)slot, a.by_scale) * a.G + h];
      const float mul = pow2f(c8::exp_of(b));
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float f[4];
        c8::to_float4(w[k], f);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * k + e] = f[e] * mul;
      }
    }
    const long long row = (long long)row0 + r;
    if (is_v)
      store16(v_out + row * a.v_stride + 16 * u, v, a.vec);
    else
      store16(k_out + row * a.k_stride + 16 * u, v, a.vec);
  }
}

template <typename TI, typename TQ>
const void* append_kernel_of(bool vec, bool interleaved) {
  if (vec)
    return interleaved ? reinterpret_cast<const void*>(append8_kernel<TI, TQ, true, true>)
                       : reinterpret_cast<const void*>(append8_kernel<TI, TQ, false, true>);
  return interleaved ? reinterpret_cast<const void*>(append8_kernel<TI, TQ, true, false>)
                     : reinterpret_cast<const void*>(append8_kernel<TI, TQ, false, false>);
}
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int pow2_from(long long n) {
  int p = 1;
  while (p < n) p <<= 1;
  return p;
}

}  // namespace

int launch_append8(Append8Args a, int dtype, int q_dtype, int sm_count, cudaStream_t s) {
  a.by_page = fast_div((uint32_t)a.page_rows);
  a.by_scale = fast_div((uint32_t)a.scale_rows);
  if (a.R == 0) a.interleaved = false;
  const int R_geo = a.R > 0 ? a.R : a.D;
  const bool vec = rot::vec_sizes(a.D, R_geo, a.interleaved) && aligned(a.q, 16) && aligned(a.q_out, 16) &&
                   aligned(a.k, 16) && aligned(a.v, 16) && aligned(a.table, 16) && aligned(a.q_weight, 16) &&
                   aligned(a.k_weight, 16) && a.q_stride % 8 == 0 &&
                   a.q_out_stride % 8 == 0 && a.k_stride % 8 == 0 && a.v_stride % 8 == 0;
  a.lanes = vec ? norm::head_lanes(a.D, R_geo, a.interleaved) : 32;
  // A team's rows at once: as many as its block has, by the batch's average; the rest of a block follows in turns.  A chunk
  // is a block's rows, or one row where sequences have about one.  4 x 1800 rows, 16 K and V heads of 128, teams of 1, 2, 4,
  // 8, 16, 32 rows: blocks of 32 positions 134, 78, 50, 50, 54, 61 us, by rows 101, 77, 85, 124, 201, 357; blocks of 64 269,
  // 146, 89, 54, 50, 54; of 1 57, 83 .. 797.  64 x 1 rows: by rows 11 us, by blocks of 16 48; 64 x 4: 11 to 26 and 19 to 38.
  // An uneven batch gets the average's teams: 250 rows among 255 idle sequences 38 us with blocks of 16 and 138 of 64, where
  // teams of 32 by blocks take 13 and 15; 2048 rows among 2000 single tokens 52 and 158 (by rows in teams of 4: 74 and 74).
  const long long avg = a.total_rows / (uint32_t)a.n_seqs;
  const int at_once = pow2_from(avg < 1 ? 1 : avg < a.scale_rows ? avg : a.scale_rows);
  a.team = at_once * a.lanes < kThreads ? at_once * a.lanes : kThreads;
  a.chunk = avg >= 2 ? a.scale_rows : 1;
  const int teams = kThreads / a.team;
  const long long chunks = ((long long)a.total_rows + a.chunk - 1) / a.chunk;
  const long long kv_blocks = (chunks * 2 * a.G + teams - 1) / teams;
  long long q_blocks = 0;
  if (a.H > 0) {
    const int steps = (a.H * a.lanes + 31) / 32;
    a.q_splits = 1;
    while (2 * a.q_splits <= steps && (long long)a.total_rows * a.q_splits < 2ll * kWarps * sm_count) a.q_splits *= 2;
    q_blocks = ((long long)a.total_rows * a.q_splits + kWarps - 1) / kWarps;
  }
  if (chunks * 2 * a.G > 0x7fffff00ll || kv_blocks + q_blocks > 0x7fffffffll) return ATTN_ERR_UNSUPPORTED;
  a.by_heads = fast_div((uint32_t)(2 * a.G));
  a.kv_blocks = (int)kv_blocks;
  const void* kern;
  if (dtype == ATTN_DT_BF16)
    kern = append_kernel_of<__nv_bfloat16, __nv_bfloat16>(vec, a.interleaved);
  else if (dtype == ATTN_DT_F16)
    kern = append_kernel_of<__half, __half>(vec, a.interleaved);
  else if (q_dtype == ATTN_DT_F16)
    kern = append_kernel_of<float, __half>(vec, a.interleaved);
  else
    kern = append_kernel_of<float, __nv_bfloat16>(vec, a.interleaved);
  void* args[] = {&a};
  return cudaLaunchKernel(kern, dim3((unsigned)(kv_blocks + q_blocks)), dim3(kThreads), args, 0, s) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

int launch_read8(Read8Args a, int dtype, cudaStream_t s) {
  a.by_page = fast_div((uint32_t)a.page_rows);
  a.by_scale = fast_div((uint32_t)a.scale_rows);
  a.vec = aligned(a.k_out, 16) && aligned(a.v_out, 16) && a.k_stride % 8 == 0 && a.v_stride % 8 == 0;
  // At 1, 2, 4, 8 rows a block, 8 heads of 128 to bf16: 100 rows 8.9, 8.9, 8.9, 10.9 us, 1000 8.9, 8.9, 10.9, 10.9, 4000 15, 13,
  // 13, 13, 8000 21, 18, 17, 17, 69632 113, 91, 81, 76.
  a.rows_per_block = a.total_rows >= 4096 ? 8 : 1;
  const dim3 grid((a.total_rows + a.rows_per_block - 1) / a.rows_per_block);
  if (dtype == ATTN_DT_BF16)
    read8_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
  else if (dtype == ATTN_DT_F16)
    read8_kernel<__half><<<grid, kThreads, 0, s>>>(a);
  else
    read8_kernel<float><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace attn
