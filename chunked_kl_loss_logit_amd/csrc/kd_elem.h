// Elements of the three floating types at any element-aligned address, and
// reductions over the lanes of a workgroup.
#pragma once

#include <hip/hip_fp16.h>

#include "kd_gemm.h"

namespace kd {

enum { kTypeF32 = 0, kTypeBf16 = 1, kTypeF16 = 2 };  // KD_F32, KD_BF16, KD_F16

// 16 bytes at any element-aligned address (the hardware takes unaligned
// vector accesses; only those that cross a cache line cost more).
__device__ inline u32x4_t load16(const char* p) {
  u32x4_t v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
__device__ inline void store16(char* p, u32x4_t v) { __builtin_memcpy(p, &v, 16); }

template <int TY>
struct Elem;
template <>
struct Elem<kTypeF32> {
  static constexpr int kBytes = 4;
  __device__ static inline float get(u32x4_t v, int i) { return __uint_as_float(v[i]); }
  __device__ static inline float get1(const char* p) { return *reinterpret_cast<const float*>(p); }
  __device__ static inline void put1(char* p, float x) { *reinterpret_cast<float*>(p) = x; }
};
template <>
struct Elem<kTypeBf16> {
  static constexpr int kBytes = 2;
  __device__ static inline float get(u32x4_t v, int i) {
    return __uint_as_float(i & 1 ? v[i >> 1] & 0xffff0000u : v[i >> 1] << 16);
  }
  __device__ static inline float get1(const char* p) {
    return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
  }
  __device__ static inline void put1(char* p, float x) { *reinterpret_cast<uint16_t*>(p) = (uint16_t)Bf16::cvt(x); }
  __device__ static inline uint32_t pack(float a, float b) { return Bf16::pack2(a, b); }
};
template <>
struct Elem<kTypeF16> {
  static constexpr int kBytes = 2;
  __device__ static inline float get(u32x4_t v, int i) {
    return __half2float(__ushort_as_half((unsigned short)(v[i >> 1] >> (16 * (i & 1)))));
  }
  __device__ static inline float get1(const char* p) { return __half2float(*reinterpret_cast<const __half*>(p)); }
  __device__ static inline void put1(char* p, float x) { *reinterpret_cast<__half*>(p) = __float2half_rn(x); }
  __device__ static inline uint32_t pack(float a, float b) {
    return (uint32_t)__half_as_ushort(__float2half_rn(a)) | ((uint32_t)__half_as_ushort(__float2half_rn(b)) << 16);
  }
};

// ------------------------------------------------------------------ pieces of 8 elements
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// A piece as it lies in memory: 16 bytes, or 32 of float32.
template <int TY>
struct Raw8 {
  u32x4_t v[TY == kTypeF32 ? 2 : 1];
};

// Two values to 16 bits each, to the nearest, ties to even.
template <int TY>
__device__ inline uint32_t pack2x16(float a, float b) {
  if constexpr (TY == kTypeBf16)
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), bf16x2_t));
  else
    return Elem<TY>::pack(a, b);
}

// n of the piece's elements exist (8 or more: all); the others read as 0.
// inner: 8 elements lie before the piece in its row.  A last piece of fewer is
// then loaded as the row's last 8 elements, and settle8 moves its own to their
// place once it is needed: until then nothing waits for the load.
// WHOLE: pieces exist as a whole or not at all.
template <int TY, bool WHOLE = false>
__device__ inline Raw8<TY> load8(const char* p, int n, bool inner) {
  Raw8<TY> r = {};
  if constexpr (WHOLE) {
    if (n > 0) {
      r.v[0] = load16(p);
      if constexpr (TY == kTypeF32) r.v[1] = load16(p + 16);
    }
    return r;
  }
  if (n >= 8 || (n > 0 && inner)) {
    const char* q = n >= 8 ? p : p - (8 - n) * Elem<TY>::kBytes;
    r.v[0] = load16(q);
    if constexpr (TY == kTypeF32) r.v[1] = load16(q + 16);
  } else if (n > 0) {  // a row of fewer than 8
    uint32_t w[TY == kTypeF32 ? 8 : 4] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= n) continue;
      if constexpr (TY == kTypeF32)
        w[i] = *reinterpret_cast<const uint32_t*>(p + 4 * i);
      else
        w[i >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t*>(p + 2 * i) << (16 * (i & 1));
    }
    __builtin_memcpy(&r, w, sizeof r);
  }
  return r;
}
template <int TY, bool WHOLE = false>
__device__ inline void settle8(Raw8<TY>& r, int n, bool inner) {
  if constexpr (WHOLE) return;
  if (n >= 8 || n <= 0 || !inner) return;
  constexpr int W = TY == kTypeF32 ? 8 : 4;
  uint32_t w[W];
  __builtin_memcpy(w, &r, sizeof r);
  const int bits = (8 - n) * Elem<TY>::kBytes * 8;  // down by so many
#pragma unroll
  for (int k = W / 2; k > 0; k >>= 1) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t from = i + k < W ? w[i + k] : 0u;
      w[i] = (bits >> 5) & k ? from : w[i];
    }
  }
  if constexpr (TY != kTypeF32) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t up = i + 1 < W ? w[i + 1] : 0u;
      w[i] = bits & 16 ? (w[i] >> 16) | (up << 16) : w[i];
    }
  }
  __builtin_memcpy(&r, w, sizeof r);
}
template <int TY>
__device__ inline void unpack8(const Raw8<TY>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = Elem<TY>::get(r.v[TY == kTypeF32 ? i >> 2 : 0], TY == kTypeF32 ? i & 3 : i);
}
// The first n of 8 values, rounded to the type.
template <int TY, bool WHOLE = false>
__device__ inline void store8(char* p, const float (&x)[8], int n) {
  if (WHOLE ? n > 0 : n >= 8) {
    if constexpr (TY == kTypeF32) {
#pragma unroll
      for (int i = 0; i < 8; i += 4)
        store16(p + 4 * i, u32x4_t{__float_as_uint(x[i]), __float_as_uint(x[i + 1]), __float_as_uint(x[i + 2]),
                                   __float_as_uint(x[i + 3])});
    } else {
      store16(p, u32x4_t{pack2x16<TY>(x[0], x[1]), pack2x16<TY>(x[2], x[3]), pack2x16<TY>(x[4], x[5]), pack2x16<TY>(x[6], x[7])});
    }
    return;
  }
  if constexpr (WHOLE) return;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) Elem<TY>::put1(p + i * Elem<TY>::kBytes, x[i]);
}

// ------------------------------------------------------------------ reductions
// The value of another lane: of the other one of two, the other pair of four,
// the mirrored one of 8 and of 16 (which holds what the other half holds once
// the halves agree), without going through LDS; 16 and 32 lanes further.
template <int D>
__device__ inline uint32_t other_lane(uint32_t v) {
  if constexpr (D == 1) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xb1, 0xf, 0xf, true);
  else if constexpr (D == 2) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4e, 0xf, 0xf, true);
  else if constexpr (D == 4) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true);
  else if constexpr (D == 8) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, true);
  else if constexpr (D == 16) return (uint32_t)__builtin_amdgcn_ds_swizzle((int)v, 0x401f);
  else return (uint32_t)__shfl_xor((int)v, D);
}
template <int D>
__device__ inline float add_lane(float v) {
  return v + __uint_as_float(other_lane<D>(__float_as_uint(v)));
}
// the largest of each aligned run of `lanes` lanes (4 to 64)
__device__ inline uint32_t wave_max(uint32_t v, int lanes = 64) {
  v = max(v, other_lane<1>(v));
  v = max(v, other_lane<2>(v));
  if (lanes > 4) v = max(v, other_lane<4>(v));
  if (lanes > 8) v = max(v, other_lane<8>(v));
  if (lanes > 16) v = max(v, other_lane<16>(v));
  if (lanes > 32) v = max(v, other_lane<32>(v));
  return v;
}

}  // namespace kd
