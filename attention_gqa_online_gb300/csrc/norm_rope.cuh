// norm_rope.cuh -- one head's row in registers: load, root-mean-square norm,
// rotary turn.  Shared by the head-norm operator and the 8-bit append.
//
//   z = w x / sqrt(mean(x^2) + eps),   y = R(p) z
//
// A head is spread over `lanes` neighbouring lanes (a power of two up to 32).
// Vector form: a lane holds one unit of rotary.cuh (16 or 8 columns), as pairs.
// Scalar form, for sizes, strides or addresses without 16-byte groups: lane l of
// 32 holds columns l, l + 32, ..., and reads the other column of its pair, too.
#pragma once

#include <cstring>
#include <type_traits>

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

// A lane's unit: pairs (a, b) of columns that turn together, P of them.  Half layout: columns c0 + i and c1 + i, 8 pairs;
// interleaved: c0 + 2 i and c0 + 2 i + 1, 4 pairs.  Behind the turned part the half layout has eight columns c0 + i and
// b doubles a (c1 = c0); lanes past the head read the first columns, too.  What is read twice counts for nothing.
template <bool INTER>
struct Unit {
  static constexpr int P = INTER ? 4 : 8;
  bool any, both, turned;  // does the lane have columns, does b have its own
  int c0, c1;
  __device__ __forceinline__ Unit(int u, int D, int R) {
    const int nrot = INTER ? R / 8 : R / 16;
    turned = u < nrot;
    c0 = turned ? 8 * u : R + 8 * (u - nrot);
    any = c0 < D;
    if (!any) c0 = 0;
    both = any && (INTER || turned);
    c1 = !INTER && turned ? R / 2 + 8 * u : c0;
  }
};

// Sum over the `lanes` lanes of a head (aligned groups of a warp).  `mask`
// names lanes that call it together, whole groups.
template <int LANES = 0>  // known when it is not 0
__device__ __forceinline__ float head_sum(float v, int lanes, unsigned mask) {
  if constexpr (LANES != 0) {
#pragma unroll
    for (int d = LANES >> 1; d > 0; d >>= 1) v += __shfl_xor_sync(mask, v, d);
  } else {
    for (int d = lanes >> 1; d > 0; d >>= 1) v += __shfl_xor_sync(mask, v, d);
  }
  return v;
}

// A unit as it lies in memory, and its pairs.
template <typename T, bool INTER>
struct Raw {
  uint4 w[(INTER ? 1 : 2) * (sizeof(T) == 4 ? 2 : 1)];
};
template <typename T>
__device__ __forceinline__ uint4 load_stream(const T* p) {
  return sizeof(T) == 4 ? *reinterpret_cast<const uint4*>(p) : __ldcs(reinterpret_cast<const uint4*>(p));
}
template <typename T, bool INTER>
__device__ __forceinline__ void load_raw(const T* x, const Unit<INTER>& u, Raw<T, INTER>& r) {
  if constexpr (sizeof(T) == 4) {
    r.w[0] = load_stream(x + u.c0);
    r.w[1] = load_stream(x + u.c0 + 4);
    if constexpr (!INTER) {
      r.w[2] = load_stream(x + u.c1);
      r.w[3] = load_stream(x + u.c1 + 4);
    }
  } else {
    r.w[0] = load_stream(x + u.c0);
    if constexpr (!INTER) r.w[1] = load_stream(x + u.c1);
  }
}
template <typename T>
__device__ __forceinline__ void unpack8(const uint4* w, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    const uint32_t x[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(x[i]);
  } else {
    const uint32_t x[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        __half2 h;
        memcpy(&h, &x[i], 4);
        const float2 f = __half22float2(h);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      } else {
        v[2 * i] = __uint_as_float(x[i] << 16);
        v[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
      }
    }
  }
}
template <typename T, bool INTER, int P>
__device__ __forceinline__ void unpack(const Raw<T, INTER>& r, float (&a)[P], float (&b)[P]) {
  float v[8];
  unpack8<T>(r.w, v);
  if constexpr (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = v[2 * i];
      b[i] = v[2 * i + 1];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = v[i];
    unpack8<T>(r.w + (sizeof(T) == 4 ? 2 : 1), b);
  }
}
template <typename T, bool INTER, int P>
__device__ __forceinline__ void store_unit(T* y, const Unit<INTER>& u, const float (&a)[P], const float (&b)[P]) {
  if constexpr (INTER) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = a[i];
      v[2 * i + 1] = b[i];
    }
    if (u.any) rot::store8<true>(y + u.c0, v);
  } else {
    if (u.any) rot::store8<true>(y + u.c0, a);
    if (u.both) rot::store8<true>(y + u.c1, b);
  }
}
// The weights (ones without) of a lane's columns.
template <bool INTER, int P>
__device__ __forceinline__ void load_weight(const void* w, int dtype, const Unit<INTER>& u, float (&a)[P], float (&b)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) a[i] = b[i] = 1.f;
  if (w == nullptr) return;
  auto of = [&](auto zero) {
    using W = decltype(zero);
    Raw<W, INTER> r;
    load_raw(static_cast<const W*>(w), u, r);
    unpack(r, a, b);
  };
  if (dtype == ATTN_DT_F32)
    of(float{});
  else if (dtype == ATTN_DT_BF16)
    of(__nv_bfloat16{});
  else
    of(__half{});
}
// Cosines and sines of a lane's pairs.  No turn: 1 and 0.  ok = false (a position past the table): zeros.
template <bool INTER, int P>
__device__ __forceinline__ void load_turn(const float* row, int R, const Unit<INTER>& u, bool ok, float (&c)[P],
                                          float (&s)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    c[i] = u.turned ? 0.f : 1.f;
    s[i] = 0.f;
  }
  if (!u.turned || !ok) return;
  const float* p = row + (INTER ? u.c0 / 2 : u.c0);
#pragma unroll
  for (int i = 0; i < P; i += 4) {
    const float4 x = *reinterpret_cast<const float4*>(p + i), y = *reinterpret_cast<const float4*>(p + R / 2 + i);
    c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
    s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
  }
}
// Sum of the squares of a lane's own columns.
template <bool INTER, int P>
__device__ __forceinline__ float squares(const Unit<INTER>& u, const float (&a)[P], const float (&b)[P]) {
  float x0 = 0.f, x1 = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
  for (int i = 0; i < P; i += 2) {
    fma2_acc(x0, x1, a[i], a[i + 1], a[i], a[i + 1]);
    fma2_acc(y0, y1, b[i], b[i + 1], b[i], b[i + 1]);
  }
  return (u.any ? x0 + x1 : 0.f) + (u.both ? y0 + y1 : 0.f);
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
