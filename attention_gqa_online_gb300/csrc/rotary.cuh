// rotary.cuh -- element access and pair rotation shared by the rotary operator
// and the paged append: groups of eight elements move as 16-byte vectors, and
// all arithmetic is fp32 with one rounding to the stored type at the end.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace attn {
namespace rot {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// Eight consecutive table entries (16-byte aligned).
__device__ __forceinline__ void load8_table(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
// Eight consecutive elements (16-byte aligned) as floats; 16-bit ones, read
// once, with the streaming hint.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const __half* p, float (&v)[8]) {
  const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __half2 h;
    memcpy(&h, &w[i], 4);
    const float2 f = __half22float2(h);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
// STREAM: the streaming hint on 16-bit stores, for results larger than L2 in
// all (8192 rows of 40 heads of 128, bf16, turned: 33 us without hints, 32 with
// that on loads, 29 with both; fp32 gains nothing).
template <bool STREAM>
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
template <bool STREAM>
__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[4]) {
  if (STREAM)
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  else
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <bool STREAM>
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    memcpy(&w[i], &h, 4);
  }
  store_words<STREAM>(p, w);
}
template <bool STREAM>
__device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    memcpy(&w[i], &h, 4);
  }
  store_words<STREAM>(p, w);
}

// One head is cut into units that a thread moves at a time.  Vector units:
// half layout, R/16 units of two 8-element groups (d and d + R/2); interleaved,
// R/8 units of one group (four pairs); then (D - R)/8 groups that only move.
// Scalar units: R/2 pairs, then D - R single elements.
__host__ __device__ inline int units_per_head(int D, int R, bool interleaved, bool vec) {
  if (!vec) return R / 2 + (D - R);
  return (interleaved ? R / 8 : R / 16) + (D - R) / 8;
}
// Sizes for which every unit's groups start on 16 bytes (given aligned rows).
__host__ __device__ inline bool vec_sizes(int D, int R, bool interleaved) {
  return D % 8 == 0 && R % 8 == 0 && (interleaved || R % 16 == 0);
}

// Moves unit u of a head from x to y, turned by the row's table entries (cos
// at tab[i], sin at tab[R/2 + i] of pair i); sgn = -1 turns back.  ok = false
// writes zeros to the turned columns (a position past the table).
template <typename TI, typename TO, bool INTER, bool STREAM>
__device__ __forceinline__ void move_unit_vec(const TI* x, TO* y, int u, int D, int R, const float* tab, float sgn,
                                              bool ok) {
  const int nrot = INTER ? R / 8 : R / 16;
  if (u >= nrot) {  // columns behind the turned part
    float a[8];
    const int d = R + 8 * (u - nrot);
    load8(x + d, a);
    store8<STREAM>(y + d, a);
    return;
  }
  if (!ok) {  // (not 0 * x: x may hold NaN or infinities)
    const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    store8<STREAM>(y + 8 * u, z);
    if (!INTER) store8<STREAM>(y + R / 2 + 8 * u, z);
    return;
  }
  if (INTER) {
    float a[8], o[8];
    load8(x + 8 * u, a);
    const float4 c = *reinterpret_cast<const float4*>(tab + 4 * u);
    const float4 s = *reinterpret_cast<const float4*>(tab + R / 2 + 4 * u);
    const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float sn = sgn * sv[i];
      o[2 * i] = a[2 * i] * cv[i] - a[2 * i + 1] * sn;
      o[2 * i + 1] = a[2 * i + 1] * cv[i] + a[2 * i] * sn;
    }
    store8<STREAM>(y + 8 * u, o);
  } else {
    float a[8], b[8], c[8], s[8];
    load8(x + 8 * u, a);
    load8(x + R / 2 + 8 * u, b);
    load8_table(tab + 8 * u, c);
    load8_table(tab + R / 2 + 8 * u, s);
    float o[8], p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float sn = sgn * s[i];
      o[i] = a[i] * c[i] - b[i] * sn;
      p[i] = b[i] * c[i] + a[i] * sn;
    }
    store8<STREAM>(y + 8 * u, o);
    store8<STREAM>(y + R / 2 + 8 * u, p);
  }
}
template <typename TI, typename TO, bool INTER>
__device__ __forceinline__ void move_unit_scalar(const TI* x, TO* y, int u, int D, int R, const float* tab, float sgn,
                                                 bool ok) {
  if (u >= R / 2) {
    const int d = R + (u - R / 2);
    y[d] = from_f32<TO>(to_f32(x[d]));
    return;
  }
  const int i0 = INTER ? 2 * u : u, i1 = INTER ? 2 * u + 1 : u + R / 2;
  if (!ok) {
    y[i0] = y[i1] = from_f32<TO>(0.f);
    return;
  }
  const float a = to_f32(x[i0]), b = to_f32(x[i1]), c = tab[u], s = sgn * tab[R / 2 + u];
  y[i0] = from_f32<TO>(a * c - b * s);
  y[i1] = from_f32<TO>(b * c + a * s);
}
template <typename TI, typename TO, bool INTER, bool VEC, bool STREAM = false>
__device__ __forceinline__ void move_unit(const TI* x, TO* y, int u, int D, int R, const float* tab, float sgn,
                                          bool ok) {
  if (VEC)
    move_unit_vec<TI, TO, INTER, STREAM>(x, y, u, D, R, tab, sgn, ok);
  else
    move_unit_scalar<TI, TO, INTER>(x, y, u, D, R, tab, sgn, ok);
}

}  // namespace rot
}  // namespace attn
