// rope_apply.cu -- rotary positions as an operator of its own, and tables
// whose angles are scaled for contexts longer than the model was trained on.
//
//   y = m R(p) x: of every head, the pairs (i, i + R/2) (half layout) or
//   (2i, 2i + 1) (interleaved), i < R/2, turn by the angle p theta_i; columns
//   >= R pass.  The table row of position p holds m cos and m sin, so the
//   gradient with respect to x is the transposed map: the same call with the
//   sines negated.
//
// Scaled angles (theta_i = base^(-2i/R), f the factor):
//   linear    theta_i / f (positions interpolated)
//   ntk       the base becomes base f^(R/(R-2)): the slowest pair turns f
//             times slower, the fastest as before
//   by parts  theta_i (g_i + (1 - g_i)/f), where g_i rises from 0 to 1 as the
//             pair's turns over the original context, orig theta_i / 2 pi, go
//             from beta_slow to beta_fast
#include <cmath>

#include "common.cuh"
#include "batch.h"
#include "rotary.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256;

// Bound by HBM (each element in and out once; the table's rows, shared by the
// heads, come from L2): 8192 rows of 40 heads of 128, bf16, move 172 MB in 29 us,
// 6.0 TB/s. A unit is 16 or 32 bytes, so a thread's index arithmetic counts: two
// 32-bit multiplications in place of divisions.
template <typename T, bool INTER, bool VEC>
__global__ void __launch_bounds__(kThreads) rope_apply_kernel(const RopeArgs a) {
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.y);
  const uint32_t upr = a.per_row.d;  // units per row
  const long long total = (long long)a.rows * upr;
  const long long stride = (long long)gridDim.x * kThreads;
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < total; i += stride) {
    const uint32_t row = a.total_fits31 ? divide((uint32_t)i, a.per_row) : (uint32_t)(i / upr);
    const uint32_t rem = (uint32_t)(i - (long long)row * upr);
    const uint32_t h = divide(rem, a.per_head), u = rem - h * a.per_head.d;
    const uint32_t pos = a.positions != nullptr ? a.positions[row] : row;
    const bool ok = pos < a.table_rows;
    if (!ok && rem == 0) record_status(a.status, ATTN_ERR_INVALID_ARG);
    rot::move_unit<T, T, INTER, VEC, true>(x + (long long)row * a.x_stride + (long long)h * a.D,
                                     y + (long long)row * a.y_stride + (long long)h * a.D, (int)u, a.D, a.R,
                                     a.table + (long long)(ok ? pos : 0) * a.R, a.sgn, ok);
  }
}

template <typename T>
int launch_t(const RopeArgs& a, bool vec, cudaStream_t s) {
  const long long total = (long long)a.rows * a.units * a.heads;
  const long long blocks = (total + kThreads - 1) / kThreads;
  const dim3 grid((unsigned)(blocks < (1ll << 30) ? blocks : (1ll << 30)));
  if (vec) {
    if (a.interleaved)
      rope_apply_kernel<T, true, true><<<grid, kThreads, 0, s>>>(a);
    else
      rope_apply_kernel<T, false, true><<<grid, kThreads, 0, s>>>(a);
  } else {
    if (a.interleaved)
      rope_apply_kernel<T, true, false><<<grid, kThreads, 0, s>>>(a);
    else
      rope_apply_kernel<T, false, false><<<grid, kThreads, 0, s>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// One thread per pair and eight positions, so that the pair's angle (a power)
// is computed once for them; angles in fp64 (an fp32 angle p theta would be off
// by up to p 2^-24 rad), rounded to fp32 once.
constexpr int kTablePositions = 8;
__global__ void __launch_bounds__(kThreads) rope_table_scaled_kernel(float* table, uint32_t max_pos, int R, RopeScale sc) {
  const int half = R / 2;
  const long long idx = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long p0 = idx / half * kTablePositions;
  if (p0 >= max_pos) return;
  const int i = (int)(idx % half);
  double th = pow(sc.base, -2.0 * (double)i / (double)R);
  if (sc.kind == ATTN_ROPE_LINEAR) {
    th /= sc.factor;
  } else if (sc.kind == ATTN_ROPE_BY_PARTS) {
    const double turns = sc.orig_max_pos * th / 6.283185307179586476925;
    const double g = fmin(1.0, fmax(0.0, (turns - sc.beta_slow) / (sc.beta_fast - sc.beta_slow)));
    th *= g + (1.0 - g) / sc.factor;
  }
  for (long long p = p0; p < p0 + kTablePositions && p < max_pos; ++p) {
    double sn, cs;
    sincos((double)p * th, &sn, &cs);
    table[p * R + i] = (float)(sc.attn_factor * cs);
    table[p * R + half + i] = (float)(sc.attn_factor * sn);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

int launch_rope_apply(RopeArgs a, int dtype, cudaStream_t s) {
  // Whole 16-byte groups where sizes, strides and addresses allow; else one
  // pair a thread.
  const bool vec = rot::vec_sizes(a.D, a.R, a.interleaved) && aligned16(a.x) && aligned16(a.y) && aligned16(a.table) &&
                   a.x_stride % 8 == 0 && a.y_stride % 8 == 0;
  a.units = rot::units_per_head(a.D, a.R, a.interleaved, vec);
  a.per_head = fast_div((uint32_t)a.units);
  a.per_row = fast_div((uint32_t)(a.units * a.heads));
  a.total_fits31 = (long long)a.rows * a.units * a.heads < (1ll << 31);
  switch (dtype) {
    case ATTN_DT_F32: return launch_t<float>(a, vec, s);
    case ATTN_DT_BF16: return launch_t<__nv_bfloat16>(a, vec, s);
    default: return launch_t<__half>(a, vec, s);
  }
}

int launch_rope_table_scaled(float* table, uint32_t max_pos, int R, RopeScale sc, cudaStream_t s) {
  if (sc.kind == ATTN_ROPE_NTK) sc.base *= std::pow(sc.factor, (double)R / (R - 2.0));
  const long long n = ((long long)max_pos + kTablePositions - 1) / kTablePositions * (R / 2);
  rope_table_scaled_kernel<<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(table, max_pos, R, sc);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace attn
