// Groups of a row's values in 8 bits (the definition is kdlayers.h's).
//
// The exact quotient x / scale is rounded, ties to even, without 64-bit
// arithmetic.
//
// 16-bit values (SHORT): of x and the group's largest m, both of 11 bits at
// most, 127 x / m is either the middle of two steps or at least 2^-19 of itself
// away from it (two different products of small integers), and 448 x / m at
// least 2^-16.  x times a reciprocal that is off by less than 2^-20 then falls on
// the right side by itself, and where the middle is hit the exact quotient lies
// on the side to which the scale's own rounding has moved it: the reciprocal is
// that of a scale moved 2^-21 further the same way.  Where the scale is m / 127 or
// m / 448 exactly (one group in 128 or in 7 for bf16), ties are ties: integers go the
// exact way, and for e4m3 the quotient is refined once, which gives a quotient
// of 24 bits or less exactly.
//
// float32 values: x times the scale's reciprocal is off by less than 4 ulps; as
// long as that leaves no doubt on which side of the middle of two steps the
// quotient lies, rounding it is all there is to do.  Where a lane of the wave
// holds a value in doubt, all its values go the exact way.  (For bf16, half of a
// group's largest is in doubt, which took half of the waves the exact way: 16384
// x 4096 to int8 47 us, 35 without it, 8192 x 8192 with layer norm 88 and 73.)
//
// The exact way, integers: the residual of the nearest one says whether it is.
// e4m3: the quotient to within an ulp, the residual's sign, and the 24-bit value
// next to the exact quotient towards zero with its last bit set if that is not
// exact ("round to odd"); rounding such a value to any format at least two bits
// shorter gives what rounding the exact quotient gives.
#pragma once

#include "kd_elem.h"

namespace kd {

enum { kRowsNone = 0, kRowsInt8 = 1, kRowsE4m3 = 2 };  // kd_rows_kind

// A group's scale as its values need it.
struct Scale8 {
  float scale;    // as it is stored
  float lift;     // a power of two that keeps the residuals in range
  float s, inv;   // scale lift, and its reciprocal; inv = 0: every q is 0.  SHORT: of the scale moved
  bool even;      // SHORT: the scale is the largest value over 127 or 448 exactly
};

// top: |x|'s largest, as bits (NaN above infinity above every number).
// The quotient by 127 or 448 is rounded correctly: the residual of the first
// product is exact, the correction's own error is 2^-24 of an ulp, and a
// 24-bit number over 127 or 7 is never nearer than 1/254 ulp to the middle of
// two numbers.  But for scales below the normal range, whose steps are wider:
// 448 of them are as many whole steps as 24 bits hold, so a largest value can lie
// 224 of float32's smallest steps from both neighbours, and its even one is
// taken.  (Only float32 values: those of 16 bits are multiples of 2^16 such steps.
// Over 127, no value lies in the middle.)
template <int KIND, bool SHORT>
__device__ inline Scale8 scale8(uint32_t top) {
  constexpr float most = KIND == kRowsInt8 ? 127.f : 448.f, part = 1.f / most;
  const float x = __uint_as_float(top);
  Scale8 r;
  const float q = x * part;
  r.scale = fmaf(fmaf(-q, most, x), part, q);
  if constexpr (KIND == kRowsE4m3 && !SHORT) {
    const float left = fmaf(-r.scale, most, x);
    const uint32_t u = __float_as_uint(r.scale);
    if (fabsf(left) == 0x1.cp-142f && (u & 1)) r.scale = __uint_as_float(left > 0.f ? u + 1 : u - 1);
  }
  r.lift = r.scale < 0x1p-90f ? 0x1p60f : 1.f;
  r.s = r.scale * r.lift;
  r.even = false;
  if constexpr (SHORT) {
    const float left = fmaf(-r.scale, most, x);  // exact
    r.even = left == 0.f;
    r.s = fmaf(r.s, left > 0.f ? -0x1p-21f : left < 0.f ? 0x1p-21f : 0.f, r.s);
  }
  r.inv = r.scale > 0.f ? __builtin_amdgcn_rcpf(r.s) : 0.f;  // off by an ulp at most
  if (top >= 0x7f800000u) {
    r.scale = __uint_as_float(0x7fc00000u);
    r.s = 1.f;
    r.inv = 0.f;
  }
  return r;
}

// x / scale rounded to odd
__device__ inline float odd_quotient(float x, const Scale8& g) {
  x *= g.lift;
  float q = x * g.inv;
  q = fmaf(fmaf(-q, g.s, x), g.inv, q);
  const float r = fmaf(-q, g.s, x);
  uint32_t u = __float_as_uint(q);
  u -= (__float_as_uint(r) ^ u) >> 31;  // |quotient| below |q|: one step down
  u |= 1u;
  return r == 0.f ? q : __uint_as_float(u);
}

// The integer nearest to x / scale, ties to even: the nearest to a quotient
// that is a few ulps off, moved by one where the residual (exact: x and n s
// agree in all but the last 24 bits) is above half the scale, or half of it
// and n odd.
__device__ inline int nearest_int(float x, const Scale8& g) {
  x *= g.lift;
  const float n = rintf(x * g.inv), r = fmaf(-n, g.s, x), a = fabsf(r), half = 0.5f * g.s;
  int i = (int)n;
  const bool move = a > half || (a == half && (i & 1));
  if (move) i += r > 0.f ? 1 : -1;
  return min(max(i, -127), 127);
}

__device__ inline uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {  // their lowest
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0c0c0400u), __builtin_amdgcn_perm(b, a, 0x0c0c0400u),
                               0x05040100u);
}
__device__ inline uint32_t pack_e4m3(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
}

// 8 values of one group, exactly, whatever its scale
template <int KIND>
__device__ inline uint2 quantize8_exact(const float (&x)[8], const Scale8& g) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (KIND == kRowsInt8) {
      w[h] = pack_bytes(nearest_int(x[4 * h], g), nearest_int(x[4 * h + 1], g), nearest_int(x[4 * h + 2], g),
                        nearest_int(x[4 * h + 3], g));
    } else {
      float q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = __builtin_amdgcn_fmed3f(odd_quotient(x[4 * h + i], g), -448.f, 448.f);
      w[h] = pack_e4m3(q[0], q[1], q[2], q[3]);
    }
  }
  return g.inv == 0.f ? uint2{0u, 0u} : uint2{w[0], w[1]};
}

template <int KIND, bool SHORT>
__device__ inline uint2 quantize8(const float (&x)[8], const Scale8& g) {
  uint2 w;
  if constexpr (SHORT) {
    bool slow = g.lift != 1.f && g.inv != 0.f;
    if constexpr (KIND == kRowsInt8) {
      constexpr float magic = 12582912.f;  // 1.5 2^23: the sum's last bits are the integer
      slow |= g.even;
      float m[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = fmaf(x[i], g.inv, magic);
      w.x = pack_bytes(__float_as_uint(m[0]), __float_as_uint(m[1]), __float_as_uint(m[2]), __float_as_uint(m[3]));
      w.y = pack_bytes(__float_as_uint(m[4]), __float_as_uint(m[5]), __float_as_uint(m[6]), __float_as_uint(m[7]));
    } else {
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = x[i] * g.inv;
      if (__any(g.even)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = fmaf(fmaf(-q[i], g.s, x[i]), g.inv, q[i]);
      }
      w.x = pack_e4m3(q[0], q[1], q[2], q[3]);
      w.y = pack_e4m3(q[4], q[5], q[6], q[7]);
    }
    if (g.inv == 0.f) w = uint2{0u, 0u};
    if (__any(slow)) {
      Scale8 e = g;
      e.s = g.scale * g.lift;
      e.inv = g.inv == 0.f ? 0.f : __builtin_amdgcn_rcpf(e.s);
      w = quantize8_exact<KIND>(x, e);
    }
    return w;
  }
  bool doubt = g.lift != 1.f || g.inv == 0.f;
  if constexpr (KIND == kRowsInt8) {
    // adding 1.5 2^23 rounds to the integer, which then is what the sum's last bits say
    constexpr float magic = 12582912.f;
    float m[8], far = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] = fmaf(x[i], g.inv, magic);
      far = fmaxf(far, fabsf(fmaf(x[i], g.inv, magic - m[i])));
    }
    doubt |= far > 0.5f - 0x1p-15f;  // 4 ulps of 127 are 2^-15
    w.x = pack_bytes(__float_as_uint(m[0]), __float_as_uint(m[1]), __float_as_uint(m[2]), __float_as_uint(m[3]));
    w.y = pack_bytes(__float_as_uint(m[4]), __float_as_uint(m[5]), __float_as_uint(m[6]), __float_as_uint(m[7]));
  } else {
    float q[8];
    uint32_t near = ~0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] = x[i] * g.inv;
      // the 20 bits behind the significand that is kept; below 2^-6 the steps are as wide as above it
      const float a = fabsf(q[i]);
      const uint32_t u = __float_as_uint(a < 0x1p-6f ? a + 0x1p-6f : a);
      near = min(near, (u - 0x80000u + 8u) & 0xfffffu);
    }
    doubt |= near <= 16u;  // within 8 ulps of the middle of two steps
    w.x = pack_e4m3(q[0], q[1], q[2], q[3]);
    w.y = pack_e4m3(q[4], q[5], q[6], q[7]);
  }
  if (__any(doubt)) w = quantize8_exact<KIND>(x, g);
  return w;
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

// 8 bytes at any address, n of them (as load8 and settle8)
template <bool WHOLE = false>
__device__ inline uint2 load_q8(const char* p, int n, bool inner) {
  uint2 w{0u, 0u};
  if constexpr (WHOLE) {
    if (n > 0) __builtin_memcpy(&w, p, 8);
    return w;
  }
  if (n >= 8 || (n > 0 && inner)) {
    __builtin_memcpy(&w, n >= 8 ? p : p - (8 - n), 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) (i < 4 ? w.x : w.y) |= (uint32_t)(uint8_t)p[i] << (8 * (i & 3));
  }
  return w;
}
template <bool WHOLE = false>
__device__ inline void settle_q8(uint2& w, int n, bool inner) {
  if constexpr (WHOLE) return;
  if (n >= 8 || n <= 0 || !inner) return;
  const uint64_t v = ((uint64_t)w.y << 32 | w.x) >> (8 * (8 - n));
  w = uint2{(uint32_t)v, (uint32_t)(v >> 32)};
}
template <bool WHOLE = false>
__device__ inline void store_q8(char* p, uint2 w, int n) {
  if (WHOLE ? n > 0 : n >= 8) {
    __builtin_memcpy(p, &w, 8);
    return;
  }
  if constexpr (WHOLE) return;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) p[i] = (char)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
}

}  // namespace kd
