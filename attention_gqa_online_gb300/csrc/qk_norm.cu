// qk_norm.cu -- root-mean-square norm of every query and key head with the
// rotary turn in the same pass, and its backward.
//
//   forward   z = w xh, xh = r x, r = 1 / sqrt(mean(x^2) + eps);  y = R(p) z
//   backward  dz = R(p)^T dy;  dw = sum over rows and heads of dz xh;
//             dx = r (w dz - xh mean(w dz xh))
//
// The backward reads x and makes r anew: one more value a head to keep between
// the passes would save it nothing, as x is read for xh in any case.
//
// A warp takes a row of Q or of K (blocks are divided between the two by their
// heads) and walks its heads, 32 / lanes at a time, the next step's loads in flight,
// with the row's cosines and sines and the weights in registers.  Where rows are
// few, several warps share a row's heads.  dw: each lane sums its columns over all
// its rows and heads in fp32; a block's lanes join in shared memory, blocks in a
// second kernel, always in the same order, so repeated calls give the same bits.
//
// Bound by the loads in flight where rows are many (one head step ahead is 16 KB
// a multiprocessor): 8192 rows of 40 heads of 128, bf16, 39 us, 4.4 TB/s, the
// gradient 53 us, 4.9 TB/s (0.66 and 0.73 of a copy's rate). 4099 rows of 12
// heads of 80, fp32, 32 columns interleaved: gradient 15.5 us, 3.1 TB/s (10 of 16
// lanes have a unit; two launches). 33 rows of 16 heads 2.2 us. All in a graph.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "batch.h"
#include "common.cuh"
#include "internal.h"
#include "norm_rope.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

template <typename T>
struct Rows {
  const T* x;
  const T* dy;
  T* y;
  long long xs, ds, ys;
};
template <typename T>
__device__ __forceinline__ Rows<T> rows_of(const NormTensor& t) {
  return {static_cast<const T*>(t.x), static_cast<const T*>(t.dy), static_cast<T*>(t.y), t.x_stride, t.dy_stride,
          t.y_stride};
}

// Position of a row, and whether the table holds it.
__device__ __forceinline__ bool position_of(const NormArgs& a, uint32_t row, uint32_t* p) {
  *p = a.positions != nullptr ? a.positions[row] : row;
  const bool ok = a.R == 0 || *p < a.table_rows;
  if (!ok && (threadIdx.x & 31) == 0) record_status(a.status, ATTN_ERR_INVALID_ARG);
  return ok;
}

// LANES: of a head, when it is not 0; the case that every lane of them has a unit of 16 columns which turn.
template <typename T, bool INTER, bool BACKWARD, int LANES>
__global__ void __launch_bounds__(kThreads, 2) qk_norm_vec_kernel(const NormArgs a) {
  using U = norm::Unit<INTER>;
  constexpr int P = U::P;
  const bool is_k = blockIdx.x >= (unsigned)a.q_blocks;
  const NormTensor& t = is_k ? a.k : a.q;
  const int block = is_k ? blockIdx.x - a.q_blocks : blockIdx.x, blocks = is_k ? gridDim.x - a.q_blocks : a.q_blocks;
  const Rows<T> r = rows_of<T>(t);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lanes = LANES != 0 ? LANES : a.lanes;
  const int sub = lane / lanes, at_once = 32 / lanes;  // heads of a warp at once
  U u(lane & (lanes - 1), a.D, a.R);
  if constexpr (LANES != 0) u.any = u.both = u.turned = true;
  const long long tasks = (long long)a.rows * t.splits;
  const float inv_d = 1.f / (float)a.D;
  const int step = at_once * t.splits, last = t.heads - 1;
  float wa[P], wb[P], dwa[P], dwb[P];
  norm::load_weight(t.weight, a.w_dtype, u, wa, wb);
  if constexpr (BACKWARD) {
#pragma unroll
    for (int i = 0; i < P; ++i) dwa[i] = dwb[i] = 0.f;
  }
  const long long first = (long long)block * kWarps + warp, stride = (long long)blocks * kWarps;
  auto position_at = [&](long long task) {
    const uint32_t row = (uint32_t)(task >> t.splits_log2);  // (splits is a power of two)
    return a.positions != nullptr && task < tasks ? a.positions[row] : row;
  };
  uint32_t p_ahead = position_at(first);
  for (long long task = first; task < tasks; task += stride) {
    const uint32_t row = (uint32_t)(task >> t.splits_log2);
    const int h0 = ((int)task & (t.splits - 1)) * at_once;
    const T* x = r.x + (long long)row * r.xs;
    const T* dy = BACKWARD ? r.dy + (long long)row * r.ds : nullptr;
    T* y = r.y + (long long)row * r.ys;
    // The next head's loads are in flight while one is computed.  Lanes without a head compute one of zeros
    // (another's infinities, times zero, would make dw NaN).
    norm::Raw<T, INTER> x_ahead, d_ahead;
    auto look = [&](int h) {
      const int at = (h + sub) * a.D;
      if (h + sub > last) {
        x_ahead = d_ahead = norm::Raw<T, INTER>{};
        return;
      }
      norm::load_raw(x + at, u, x_ahead);
      if constexpr (BACKWARD) norm::load_raw(dy + at, u, d_ahead);
    };
    look(h0);
    const uint32_t p = p_ahead;
    p_ahead = position_at(task + stride);
    const bool ok = a.R == 0 || p < a.table_rows;
    if (!ok && lane == 0) record_status(a.status, ATTN_ERR_INVALID_ARG);
    float c[P], s[P];
    norm::load_turn(a.table + (long long)p * a.R, a.R, u, ok, c, s);
    const bool zero = u.turned && !ok;
    // Forward: y_a = r (a w_a c - b w_b s), y_b = r (b w_b c + a w_a s).
    float ac[P], bs[P], bc[P], as[P], ns[P];
    if constexpr (BACKWARD) {
#pragma unroll
      for (int i = 0; i < P; ++i) ns[i] = -s[i];
    }
    if constexpr (!BACKWARD) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        ac[i] = wa[i] * c[i];
        bs[i] = -wb[i] * s[i];
        bc[i] = wb[i] * c[i];
        as[i] = wa[i] * s[i];
      }
    }
    for (int h = h0; h <= last; h += step) {
      float va[P], vb[P];
      norm::unpack(x_ahead, va, vb);
      norm::Raw<T, INTER> d_now;
      if constexpr (BACKWARD) d_now = d_ahead;
      if (h + step <= last) look(h + step);
      const bool mine = h + sub <= last;
      T* to = y + (h + sub) * a.D;
      const float rms = rsqrtf(fmaf(norm::head_sum<LANES>(norm::squares(u, va, vb), lanes, 0xffffffffu), inv_d, a.eps));
      if constexpr (!BACKWARD) {
        float ya[P], yb[P];
#pragma unroll
        for (int i = 0; i < P; i += 2) {
          const float2 ra = mul2_of(va[i], va[i + 1], rms, rms), rb = mul2_of(vb[i], vb[i + 1], rms, rms);
          float2 oa = mul2_of(ra.x, ra.y, ac[i], ac[i + 1]), ob = mul2_of(rb.x, rb.y, bc[i], bc[i + 1]);
          if (u.turned) {  // (not + 0 * the other column: that may be an infinity)
            oa = fma2_of(rb.x, rb.y, bs[i], bs[i + 1], oa);
            ob = fma2_of(ra.x, ra.y, as[i], as[i + 1], ob);
          }
          ya[i] = oa.x, ya[i + 1] = oa.y;
          yb[i] = ob.x, yb[i + 1] = ob.y;
        }
        if (zero) {  // (not 0 * x: that may be NaN)
#pragma unroll
          for (int i = 0; i < P; ++i) ya[i] = yb[i] = 0.f;
        }
        if (mine) norm::store_unit(to, u, ya, yb);
      } else {
        float ga[P], gb[P], da[P], db[P];
        norm::unpack(d_now, da, db);
        if (zero) {
#pragma unroll
          for (int i = 0; i < P; ++i) da[i] = db[i] = 0.f;
        }
        float x0 = 0.f, x1 = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
        for (int i = 0; i < P; i += 2) {
          mul2(va[i], va[i + 1], rms, rms);  // x r
          mul2(vb[i], vb[i + 1], rms, rms);
          // dz_a = dy_a c + dy_b s, dz_b = dy_b c - dy_a s; not turned: dy (not + 0 * the other column, as above)
          float2 za = mul2_of(da[i], da[i + 1], c[i], c[i + 1]), zb = mul2_of(db[i], db[i + 1], c[i], c[i + 1]);
          if (u.turned) {
            za = fma2_of(db[i], db[i + 1], s[i], s[i + 1], za);
            zb = fma2_of(da[i], da[i + 1], ns[i], ns[i + 1], zb);
          }
          // dz x r: into dw, and times w into the mean
          const float2 pa = mul2_of(za.x, za.y, va[i], va[i + 1]), pb = mul2_of(zb.x, zb.y, vb[i], vb[i + 1]);
          fma2_acc(x0, x1, pa.x, pa.y, wa[i], wa[i + 1]);
          fma2_acc(y0, y1, pb.x, pb.y, wb[i], wb[i + 1]);
          add2(dwa[i], dwa[i + 1], pa.x, pa.y);
          add2(dwb[i], dwb[i + 1], pb.x, pb.y);
          const float2 ta = mul2_of(za.x, za.y, wa[i], wa[i + 1]), tb = mul2_of(zb.x, zb.y, wb[i], wb[i + 1]);
          ga[i] = ta.x, ga[i + 1] = ta.y;
          gb[i] = tb.x, gb[i + 1] = tb.y;
        }
        const float dot = -norm::head_sum<LANES>((u.any ? x0 + x1 : 0.f) + (u.both ? y0 + y1 : 0.f), lanes, 0xffffffffu) * inv_d;
#pragma unroll
        for (int i = 0; i < P; i += 2) {
          fma2_acc(ga[i], ga[i + 1], va[i], va[i + 1], dot, dot);
          fma2_acc(gb[i], gb[i + 1], vb[i], vb[i + 1], dot, dot);
          mul2(ga[i], ga[i + 1], rms, rms);
          mul2(gb[i], gb[i + 1], rms, rms);
        }
        if (mine) norm::store_unit(to, u, ga, gb);
      }
    }
  }
  if constexpr (BACKWARD) {
    if (t.dw == nullptr) return;  // (all threads of the block)
    // The block's sum of each column, in the order of its head groups.
    __shared__ float part[kThreads * 2 * P];
    const int groups = kThreads / lanes, group = threadIdx.x / lanes;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (u.any) part[group * a.D + u.c0 + (INTER ? 2 * i : i)] = dwa[i];
      if (u.both) part[group * a.D + (INTER ? u.c0 + 2 * i + 1 : u.c1 + i)] = dwb[i];
    }
    __syncthreads();
    for (int d = threadIdx.x; d < a.D; d += kThreads) {
      float sum = 0.f;
      for (int k = 0; k < groups; ++k) sum += part[k * a.D + d];
      a.partial[(long long)blockIdx.x * a.D + d] = sum;
    }
  }
}

// One warp a head, columns lane, lane + 32, ...
template <typename T, bool INTER, bool BACKWARD>
__global__ void __launch_bounds__(kThreads) qk_norm_scalar_kernel(const NormArgs a) {
  const bool is_k = blockIdx.x >= (unsigned)a.q_blocks;
  const NormTensor& t = is_k ? a.k : a.q;
  const int block = is_k ? blockIdx.x - a.q_blocks : blockIdx.x, blocks = is_k ? gridDim.x - a.q_blocks : a.q_blocks;
  const Rows<T> r = rows_of<T>(t);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float w[norm::kMaxScalar], dw[norm::kMaxScalar];
  norm::Column col[norm::kMaxScalar];
#pragma unroll
  for (int j = 0; j < norm::kMaxScalar; ++j) {
    const int d = lane + 32 * j;
    dw[j] = 0.f;
    w[j] = t.weight != nullptr && d < a.D ? norm::weight_at(t.weight, a.w_dtype, d) : 1.f;
    col[j] = norm::column_of<INTER>(d, a.R);
  }
  const float inv_d = 1.f / (float)a.D;
  const long long tasks = (long long)a.rows * t.heads;
  for (long long task = (long long)block * kWarps + warp; task < tasks; task += (long long)blocks * kWarps) {
    const uint32_t row = (uint32_t)(task / t.heads);
    const int h = (int)(task - (long long)row * t.heads);
    uint32_t p;
    const bool ok = position_of(a, row, &p);
    const float* tab = a.table + (long long)p * a.R;
    const T* x = r.x + (long long)row * r.xs + (long long)h * a.D;
    T* y = r.y + (long long)row * r.ys + (long long)h * a.D;
    float v[norm::kMaxScalar], sum = 0.f;
#pragma unroll
    for (int j = 0; j < norm::kMaxScalar; ++j) {
      v[j] = lane + 32 * j < a.D ? rot::to_f32(x[lane + 32 * j]) : 0.f;
      sum = fmaf(v[j], v[j], sum);
    }
    const float rms = rsqrtf(fmaf(norm::head_sum(sum, 32, 0xffffffffu), inv_d, a.eps));
    if constexpr (BACKWARD) {
      const T* dy = r.dy + (long long)row * r.ds + (long long)h * a.D;
      float g[norm::kMaxScalar], dot = 0.f;
#pragma unroll
      for (int j = 0; j < norm::kMaxScalar; ++j) {
        g[j] = 0.f;
        if (lane + 32 * j < a.D)
          g[j] = norm::turned_column<-1>(col[j], tab, a.R, ok, [&](int d) { return rot::to_f32(dy[d]); });
        v[j] *= rms;
        dw[j] = fmaf(g[j], v[j], dw[j]);
        g[j] *= w[j];
        dot = fmaf(g[j], v[j], dot);
      }
      dot = norm::head_sum(dot, 32, 0xffffffffu) * inv_d;  // (all lanes have read dy: y may be dy)
#pragma unroll
      for (int j = 0; j < norm::kMaxScalar; ++j) v[j] = rms * (g[j] - v[j] * dot);
    } else {
      float z[norm::kMaxScalar];
#pragma unroll
      for (int j = 0; j < norm::kMaxScalar; ++j) {
        z[j] = 0.f;
        if (lane + 32 * j < a.D)
          z[j] = norm::turned_column<1>(col[j], tab, a.R, ok, [&](int d) {
            return rot::to_f32(x[d]) * (rms * (t.weight != nullptr ? norm::weight_at(t.weight, a.w_dtype, d) : 1.f));
          });
      }
#pragma unroll
      for (int j = 0; j < norm::kMaxScalar; ++j) v[j] = z[j];
    }
    __syncwarp();  // every lane has read the row: y may be x
#pragma unroll
    for (int j = 0; j < norm::kMaxScalar; ++j)
      if (lane + 32 * j < a.D) y[lane + 32 * j] = rot::from_f32<T>(v[j]);
  }
  if constexpr (BACKWARD) {
    if (t.dw == nullptr) return;
    __shared__ float part[kWarps][32 * norm::kMaxScalar];
#pragma unroll
    for (int j = 0; j < norm::kMaxScalar; ++j) part[warp][lane + 32 * j] = dw[j];
    __syncthreads();
    for (int d = threadIdx.x; d < a.D; d += kThreads) {
      float sum = 0.f;
      for (int k = 0; k < kWarps; ++k) sum += part[k][d];
      a.partial[(long long)blockIdx.x * a.D + d] = sum;
    }
  }
}

// dw: the blocks' sums, 32 columns a thread block, each of 32 warps every 32nd block, then the warps in order.
__global__ void __launch_bounds__(1024) qk_norm_dw_kernel(const NormArgs a, const int blocks) {
  grid_dependency_wait();
  const NormTensor& t = blockIdx.y ? a.k : a.q;
  if (t.dw == nullptr) return;
  const int b0 = blockIdx.y ? a.q_blocks : 0, b1 = blockIdx.y ? blocks : a.q_blocks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = blockIdx.x * 32 + lane;
  __shared__ float part[32][33];
  float sum = 0.f;
  if (d < a.D)
#pragma unroll 8
    for (int b = b0 + warp; b < b1; b += 32) sum += a.partial[(long long)b * a.D + d];
  part[warp][lane] = sum;
  __syncthreads();
  if (warp != 0 || d >= a.D) return;
  sum = 0.f;
#pragma unroll
  for (int k = 0; k < 32; ++k) sum += part[k][lane];
  if (a.w_dtype == ATTN_DT_F32)
    static_cast<float*>(t.dw)[d] = sum;
  else if (a.w_dtype == ATTN_DT_BF16)
    static_cast<__nv_bfloat16*>(t.dw)[d] = __float2bfloat16_rn(sum);
  else
    static_cast<__half*>(t.dw)[d] = __float2half_rn(sum);
}

template <typename T, bool BACKWARD>
const void* kernel_of(bool vec, bool interleaved, int whole) {
  if (vec && !interleaved && whole == 8) return reinterpret_cast<const void*>(qk_norm_vec_kernel<T, false, BACKWARD, 8>);
  if (vec && !interleaved && whole == 4) return reinterpret_cast<const void*>(qk_norm_vec_kernel<T, false, BACKWARD, 4>);
  if (vec)
    return interleaved ? reinterpret_cast<const void*>(qk_norm_vec_kernel<T, true, BACKWARD, 0>)
                       : reinterpret_cast<const void*>(qk_norm_vec_kernel<T, false, BACKWARD, 0>);
  return interleaved ? reinterpret_cast<const void*>(qk_norm_scalar_kernel<T, true, BACKWARD>)
                     : reinterpret_cast<const void*>(qk_norm_scalar_kernel<T, false, BACKWARD>);
}
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool vec_rows(const NormTensor& t) {
  return aligned16(t.x) && aligned16(t.y) && aligned16(t.dy) && t.x_stride % 8 == 0 && t.y_stride % 8 == 0 &&
         t.dy_stride % 8 == 0;
}
// Thread blocks at most, of both tensors together: two resident on a multiprocessor (in the backward each leaves a row
// of partial sums).
int most_blocks(int sms) { return sms * 2; }

}  // namespace

size_t qk_norm_workspace_bytes(int D, int sm_count) { return (size_t)most_blocks(sm_count) * D * sizeof(float); }

int launch_qk_norm(NormArgs a, int dtype, bool backward, int sm_count, cudaStream_t s) {
  const bool vec = rot::vec_sizes(a.D, a.R, a.interleaved) && vec_rows(a.q) && vec_rows(a.k) &&
                   (a.R == 0 || aligned16(a.table)) && aligned16(a.q.weight) && aligned16(a.k.weight);
  a.lanes = vec ? norm::head_lanes(a.D, a.R, a.interleaved) : 32;
  // Heads of 128 and 64 that turn as a whole (every lane has a whole unit) run on kernels that know it.
  const int whole = a.R == a.D && a.D == 16 * a.lanes ? a.lanes : 0;
  // Blocks stay and take rows in turns, so weights are read once.  A row's heads are split over warps until there are
  // rounds enough for all to end together, and in small calls until no multiprocessor is idle.
  const int most = most_blocks(sm_count);
  const long long rounds = 2ll * most * kWarps;
  long long want[2] = {0, 0};
  NormTensor* t[2] = {&a.q, &a.k};
  for (int i = 0; i < 2; ++i) {
    if (t[i]->heads == 0) continue;
    const int steps = vec ? (t[i]->heads * a.lanes + 31) / 32 : t[i]->heads;
    t[i]->splits = 1;
    t[i]->splits_log2 = 0;
    while (vec && 2 * t[i]->splits <= steps && (long long)a.rows * t[i]->splits < rounds) {
      t[i]->splits *= 2;
      ++t[i]->splits_log2;
    }
    want[i] = ((long long)a.rows * (vec ? t[i]->splits : steps) + kWarps - 1) / kWarps;
    if (want[i] > most) want[i] = most;
  }
  if (want[0] + want[1] > most) {  // in proportion to the heads, at least one each
    int q = (int)((long long)most * a.q.heads / (a.q.heads + a.k.heads));
    if (a.q.heads > 0 && q == 0) q = 1;
    if (a.k.heads > 0 && q == most) q = most - 1;
    if (want[0] > q) want[0] = q;
    if (want[1] > most - want[0]) want[1] = most - want[0];
  }
  a.q_blocks = (int)want[0];
  const int blocks = (int)(want[0] + want[1]);
  const void* kern;
  if (dtype == ATTN_DT_BF16)
    kern = backward ? kernel_of<__nv_bfloat16, true>(vec, a.interleaved, whole) : kernel_of<__nv_bfloat16, false>(vec, a.interleaved, whole);
  else if (dtype == ATTN_DT_F16)
    kern = backward ? kernel_of<__half, true>(vec, a.interleaved, whole) : kernel_of<__half, false>(vec, a.interleaved, whole);
  else
    kern = backward ? kernel_of<float, true>(vec, a.interleaved, whole) : kernel_of<float, false>(vec, a.interleaved, whole);
  void* args[] = {&a};
  if (cudaLaunchKernel(kern, dim3(blocks), dim3(kThreads), args, 0, s) != cudaSuccess) return ATTN_ERR_CUDA;
  if (!backward || (a.q.dw == nullptr && a.k.dw == nullptr)) return ATTN_OK;
  int n = blocks;
  void* args2[] = {&a, &n};
  return launch_pdl(reinterpret_cast<const void*>(qk_norm_dw_kernel), dim3((a.D + 31) / 32, 2), dim3(1024), 0, s,
                    args2) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

}  // namespace attn
