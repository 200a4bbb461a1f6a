// norm_rope.cuh -- one head's row in registers: load, root-mean-square norm,
// rotary turn.  Shared by the head-norm operator and the 8-bit append.
//
//   z = w x / sqrt(mean(x^2) + eps),   y = R(p) z
//
// A head is spread over `lanes` neighbouring lanes (a power of two up to 32).
// Vector form: a lane holds one unit of rotary.cuh: two groups of eight columns
// that turn together (half layout, columns [8u, +8) and [R/2 + 8u, +8)), or one
// group of eight (interleaved pairs, and the columns behind the turned part).
// Scalar form, for sizes, strides or addresses without 16-byte groups: lane l of
// 32 holds columns l, l + 32, ..., and reads the other column of its pair, too.
#pragma once

#include "batch.h"
#include "common.cuh"
#include "rotary.cuh"

namespace attn {
namespace norm {

constexpr int kMaxScalar = 8;  // columns of a lane in the scalar form: heads of up to 256

// Weights of any of the three types, as fp32.
__device__ __forceinline__ float weight_at(const void* w, int dtype, int i) {
  if (dtype == ATTN_DT_F32) return static_cast<const float*>(w)[i];
  if (dtype == ATTN_DT_BF16) return rot::to_f32(static_cast<const __nv_bfloat16*>(w)[i]);
  return rot::to_f32(static_cast<const __half*>(w)[i]);
}

// Where a lane's columns are.
template <bool INTER>
struct Unit {
  bool any, pair;  // columns at all; two groups (half layout)
  bool turned;
  int c0, c1;
  __device__ __forceinline__ Unit(int u, int D, int R) {
    const int nrot = INTER ? R / 8 : R / 16;
    turned = u < nrot;
    pair = !INTER && turned;
    c0 = turned ? 8 * u : R + 8 * (u - nrot);
    c1 = R / 2 + 8 * u;
    any = c0 < D;
  }
};

// Sum over the `lanes` lanes of a head (aligned groups of a warp).  `mask`
// names lanes that call it together, whole groups.
__device__ __forceinline__ float head_sum(float v, int lanes, unsigned mask) {
  for (int d = lanes >> 1; d > 0; d >>= 1) v += __shfl_xor_sync(mask, v, d);
  return v;
}

template <typename T, bool INTER>
__device__ __forceinline__ void load_unit(const T* x, const Unit<INTER>& u, float (&v)[16]) {
  float a[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = b[i] = 0.f;
  if (u.any) rot::load8(x + u.c0, a);
  if (u.pair) rot::load8(x + u.c1, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = a[i];
    v[8 + i] = b[i];
  }
}
template <typename T, bool INTER>
__device__ __forceinline__ void store_unit(T* y, const Unit<INTER>& u, const float (&v)[16]) {
  float a[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = v[i];
    b[i] = v[8 + i];
  }
  if (u.any) rot::store8<true>(y + u.c0, a);
  if (u.pair) rot::store8<true>(y + u.c1, b);
}
template <bool INTER>
__device__ __forceinline__ void load_weight(const void* w, int dtype, const Unit<INTER>& u, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = w != nullptr && u.any ? weight_at(w, dtype, u.c0 + i) : 1.f;
    v[8 + i] = w != nullptr && u.pair ? weight_at(w, dtype, u.c1 + i) : 1.f;
  }
}
// The row's table entries that a lane's unit needs: cos in t[0, 8), sin in
// t[8, 16) (interleaved: four of each).  No turn: cos 1, sin 0.  ok = false (a
// position past the table): zeros.
template <bool INTER>
__device__ __forceinline__ void load_turn(const float* row, int R, const Unit<INTER>& u, bool ok, float (&t)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t[i] = 1.f;
    t[8 + i] = 0.f;
  }
  if (!u.turned) return;
  if (!ok) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = 0.f;
  } else if (INTER) {
    const float4 c = *reinterpret_cast<const float4*>(row + u.c0 / 2);
    const float4 s = *reinterpret_cast<const float4*>(row + R / 2 + u.c0 / 2);
    t[0] = c.x, t[1] = c.y, t[2] = c.z, t[3] = c.w;
    t[8] = s.x, t[9] = s.y, t[10] = s.z, t[11] = s.w;
  } else {
    float c[8], s[8];
    rot::load8_table(row + u.c0, c);
    rot::load8_table(row + R / 2 + u.c0, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t[i] = c[i];
      t[8 + i] = s[i];
    }
  }
}
// v turned (SIGN 1) or turned back (-1) in place.  `zero`: the turned columns
// become zeros, whatever they held.
template <bool INTER, int SIGN>
__device__ __forceinline__ void turn_unit(float (&v)[16], const float (&t)[16], const Unit<INTER>& u, bool zero) {
  if (!u.turned) return;
  if (zero) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
    return;
  }
#pragma unroll
  for (int i = 0; i < (INTER ? 4 : 8); ++i) {
    const int x = INTER ? 2 * i : i, y = INTER ? 2 * i + 1 : 8 + i;
    const float a = v[x], b = v[y], c = t[i], s = SIGN * t[8 + i];
    v[x] = a * c - b * s;
    v[y] = b * c + a * s;
  }
}

// Lanes of a head in the vector form.
inline int head_lanes(int D, int R, bool interleaved) {
  const int units = rot::units_per_head(D, R, interleaved, true);
  int l = 1;
  while (l < units) l <<= 1;
  return l;
}

// ---------------------------------------------------------------- scalar form
struct Column {
  int d, other;  // the column and the one that it turns with (itself: not turned)
  int i;         // pair
  bool first;    // of its pair
};
template <bool INTER>
__device__ __forceinline__ Column column_of(int d, int R) {
  Column c{d, d, 0, true};
  if (d < R) {
    c.i = INTER ? d / 2 : d % (R / 2);
    c.first = INTER ? d % 2 == 0 : d < R / 2;
    c.other = INTER ? d ^ 1 : c.first ? d + R / 2 : d - R / 2;
  }
  return c;
}
// Value of column c of R(+-p) z, where z(d) gives the unturned values.
template <int SIGN, typename F>
__device__ __forceinline__ float turned_column(const Column& c, const float* row, int R, bool ok, F z) {
  if (c.other == c.d) return z(c.d);
  if (!ok) return 0.f;
  const float cs = row[c.i], sn = SIGN * row[R / 2 + c.i];
  return c.first ? z(c.d) * cs - z(c.other) * sn : z(c.d) * cs + z(c.other) * sn;
}

}  // namespace norm
}  // namespace attn
