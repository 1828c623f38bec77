// Groups of a row's values in 8 bits (the definition is kdlayers.h's).
//
// The quotient x / scale is rounded to few bits exactly, ties to even, without
// 64-bit arithmetic: it is computed to within an ulp, the residual's sign
// says on which side the exact quotient lies, and the 24-bit value next to it
// towards zero gets its last bit set if the quotient was not exact ("round to
// odd").  Rounding such a value to any format at least two bits shorter gives
// what rounding the exact quotient gives.
#pragma once

#include "kd_elem.h"

namespace kd {

enum { kRowsNone = 0, kRowsInt8 = 1, kRowsE4m3 = 2 };  // kd_rows_kind

// A group's scale as its values need it.
struct Scale8 {
  float scale;    // as it is stored
  float lift;     // a power of two that keeps the residuals in range
  float s, inv;   // scale lift, and its reciprocal; inv = 0: every q is 0
};

// top: |x|'s largest, as bits (NaN above infinity above every number)
template <int KIND>
__device__ inline Scale8 scale8(uint32_t top) {
  Scale8 r;
  if (top >= 0x7f800000u) return Scale8{__uint_as_float(0x7fc00000u), 0.f, 1.f, 0.f};
  r.scale = __fdiv_rn(__uint_as_float(top), KIND == kRowsInt8 ? 127.f : 448.f);
  r.lift = r.scale < 0x1p-90f ? 0x1p60f : 1.f;
  r.s = r.scale * r.lift;
  r.inv = r.scale > 0.f ? __fdiv_rn(1.f, r.s) : 0.f;
  return r;
}

// x / scale rounded to odd, at most the format's largest in size
template <int KIND>
__device__ inline float odd_quotient(float x, const Scale8& g) {
  x *= g.lift;
  float q = x * g.inv;
  q = fmaf(fmaf(-q, g.s, x), g.inv, q);
  const float r = fmaf(-q, g.s, x);
  uint32_t u = __float_as_uint(q);
  u -= (__float_as_uint(r) ^ u) >> 31;  // |quotient| below |q|: one step down
  u |= 1u;
  q = r == 0.f ? q : __uint_as_float(u);
  const float most = KIND == kRowsInt8 ? 127.f : 448.f;
  return __builtin_amdgcn_fmed3f(q, -most, most);
}

// 8 values of one group
template <int KIND>
__device__ inline uint2 quantize8(const float (&x)[8], const Scale8& g) {
  if (g.inv == 0.f) return uint2{0u, 0u};
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = odd_quotient<KIND>(x[i], g);
  uint32_t w[2] = {0u, 0u};
  if constexpr (KIND == kRowsInt8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i >> 2] |= ((uint32_t)(int)rintf(q[i]) & 0xffu) << (8 * (i & 3));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int v = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
      w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], v, true);
    }
  }
  return uint2{w[0], w[1]};
}

// the values in units of their scale
template <int KIND>
__device__ inline void values8(uint2 w, float (&x)[8]) {
  const uint32_t u[2] = {w.x, w.y};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (KIND == kRowsInt8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 * h + i] = (float)(int8_t)(u[h] >> (8 * i));
    } else {
      const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)u[h], false);
      const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)u[h], true);
      x[4 * h] = a[0];
      x[4 * h + 1] = a[1];
      x[4 * h + 2] = b[0];
      x[4 * h + 3] = b[1];
    }
  }
}

__device__ inline uint32_t top8(const float (&x)[8]) {
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) t = max(t, __float_as_uint(x[i]) & 0x7fffffffu);
  return t;
}

// 8 bytes at any address, n of them
__device__ inline uint2 load_q8(const char* p, int n) {
  uint2 w{0u, 0u};
  if (n >= 8) {
    __builtin_memcpy(&w, p, 8);
    return w;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) (i < 4 ? w.x : w.y) |= (uint32_t)(uint8_t)p[i] << (8 * (i & 3));
  return w;
}
__device__ inline void store_q8(char* p, uint2 w, int n) {
  if (n >= 8) {
    __builtin_memcpy(p, &w, 8);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) p[i] = (char)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
}

}  // namespace kd
