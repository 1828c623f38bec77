// One row in the registers of R threads: thread i holds the pieces of 8
// elements i, i + R, .., i + (K - 1) R.  Below R = 256 a workgroup of 256 holds
// several rows, each of a part of a wave, a wave, or two waves; otherwise the
// workgroup is the row's.
#pragma once

#include <type_traits>

#include "kd_elem.h"
#include "kd_rows8.h"

namespace kd {

// Rows of up to kRowMost elements are held in registers, longer ones are read
// again for every pass over them.
constexpr int64_t kRowMost = 16384;

// launch(R, K) of the first of the shapes R x K whose registers hold d
// elements (R K pieces of 8); false if none does.
template <int R, int K>
struct Shape {
  static constexpr int kR = R, kK = K;
};
template <class S, class... More, class F>
inline bool pick_shape(int64_t d, F&& launch) {
  if (d <= (int64_t)8 * S::kR * S::kK) {
    launch(std::integral_constant<int, S::kR>(), std::integral_constant<int, S::kK>());
    return true;
  }
  if constexpr (sizeof...(More) > 0) return pick_shape<More...>(d, launch);
  return false;
}

template <int R>
struct RowTeam {
  static constexpr int kThreads = R < 256 ? 256 : R;
  static constexpr int kRows = kThreads / R;  // rows of a workgroup
  static constexpr int kWaves = R / 64;  // 0: less than one
  // Rows of several waves each in one workgroup: gone through together, as their sums meet at its barriers.
  static constexpr bool kJoint = R > 64 && kRows > 1;
  __device__ static inline int lane() { return threadIdx.x % R; }
  __device__ static inline int slot() { return threadIdx.x / R; }
  __device__ static inline int wave() { return kJoint ? lane() >> 6 : (int)threadIdx.x >> 6; }  // of the row's
  // whether row t, or one beside it that it waits for, is left; and its elements, none behind the last row
  __device__ static inline bool left(int64_t t, int64_t T) { return (kJoint ? t - slot() : t) < T; }
  __device__ static inline int64_t elements(int64_t t, int64_t T, int64_t d) { return !kJoint || t < T ? d : 0; }

  // Sums over the row's threads, each of N values, in the same order every
  // time.  lds: N floats for each wave of the workgroup, free again after the
  // next barrier.
  template <int N>
  __device__ static inline void sum(float (&v)[N], float* lds) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = add_lane<8>(add_lane<4>(add_lane<2>(add_lane<1>(v[i]))));
      if constexpr (R >= 32) v[i] = add_lane<16>(v[i]);
      if constexpr (R >= 64) v[i] = add_lane<32>(v[i]);
    }
    if constexpr (R > 64) {
      const int w = wave();
      if constexpr (kJoint) lds += slot() * N * kWaves;
      __syncthreads();
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) lds[i * kWaves + w] = v[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[i] = 0;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) v[i] += lds[i * kWaves + k];
      }
    }
  }
  __device__ static inline uint32_t most(uint32_t v, uint32_t* lds) {
    v = wave_max(v, R);
    if constexpr (R > 64) {
      if constexpr (kJoint) lds += slot() * kWaves;
      __syncthreads();
      if ((threadIdx.x & 63) == 0) lds[wave()] = v;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kWaves; ++k) v = max(v, lds[k]);
    }
    return v;
  }
};

__device__ inline bool row_valid(const uint8_t* mask, int64_t t) { return !mask || mask[t]; }

template <int TY>
__device__ inline void load_row(const char* row, int64_t d, int p, float (&x)[8]) {
  const int n = (int)(d - 8 * (int64_t)p);
  Raw8<TY> r = load8<TY>(row + (int64_t)p * 8 * Elem<TY>::kBytes, n, p > 0);
  settle8<TY>(r, n, p > 0);
  unpack8<TY>(r, x);
}

// 8 values of a vector whose type is known at run time
__device__ inline void load_any(const char* base, int type, int64_t d, int p, float (&x)[8]) {
  if (type == kTypeF32) load_row<kTypeF32>(base, d, p, x);
  else if (type == kTypeBf16) load_row<kTypeBf16>(base, d, p, x);
  else load_row<kTypeF16>(base, d, p, x);
}
__device__ inline void store_any1(char* base, int type, int64_t i, float v) {
  if (type == kTypeF32) Elem<kTypeF32>::put1(base + 4 * i, v);
  else if (type == kTypeBf16) Elem<kTypeBf16>::put1(base + 2 * i, v);
  else Elem<kTypeF16>::put1(base + 2 * i, v);
}

// launch with the element type as a constant
template <class F>
inline void pick_type(int type, F&& launch) {
  using std::integral_constant;
  if (type == kTypeF32) launch(integral_constant<int, kTypeF32>());
  else if (type == kTypeBf16) launch(integral_constant<int, kTypeBf16>());
  else launch(integral_constant<int, kTypeF16>());
}

}  // namespace kd
