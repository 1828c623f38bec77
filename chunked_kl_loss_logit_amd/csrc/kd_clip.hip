// The global L2 norm of many tensors, and clipping by it.
//
//   n = sqrt(sum x^2) over all elements of all tensors, c = min(1, max / (n + 1e-6)), out = x c
//
// The norm has to be whole before the first element is scaled, so the floor
// is two reads and one write of the gradients.  A block takes kClipBlock
// consecutive elements of one tensor; the tensors of a launch come by value
// in its arguments, so nothing is copied to the device first and the launches
// can be captured.  Squares and sums are in 64 bits (no overflow or underflow
// for any float32 input, and at 2 to 4 bytes per element the memory is still
// what bounds), one partial per block, added in a fixed order.
//
// Measured: 400 M float32 elements, the sum 290 us (5.5 TB/s), the scaling 565
// us (5.7 TB/s; a large copy reaches 5.0); 290 bf16 tensors, 30 M elements,
// into others 57 us in five launches; 6 tensors, 40000 elements, 12 us in one.
#include <hip/hip_fp16.h>

#include "kd_gemm.h"
#include "kd_policy.h"

namespace kd {

namespace {

constexpr int kClipThreads = 512;
enum { kTypeF32 = 0, kTypeBf16 = 1, kTypeF16 = 2 };

template <int NT>
__device__ inline double block_sum(double v) {
  __shared__ double red[NT / 64];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) v += red[i];
  return v;
}

// the tensor that block b covers
__device__ inline int tensor_of(const int32_t* first, int n, int b) {
  int lo = 0, hi = n;  // first index with first > b
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= b) lo = mid + 1; else hi = mid;
  }
  return lo - 1;
}

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

// Elements [b, e) of a tensor (fewer than 2^31) by NT threads: 16-byte pieces, kDeep of a thread's loads in flight at once, then the
// last few elements one by one.
constexpr int kDeep = 4;

template <int TY, int NT>
__device__ inline double sumsq_range(const void* base, long b, long e) {
  using E = Elem<TY>;
  constexpr int N = 16 / E::kBytes;
  const char* p = static_cast<const char*>(base) + b * E::kBytes;
  const int n = (int)(e - b), pieces = n / N;
  double s[2] = {0, 0};
  auto add = [&](u32x4_t v) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const double x = E::get(v, i);
      s[i & 1] = fma(x, x, s[i & 1]);
    }
  };
  int q = threadIdx.x;
  for (; q + (kDeep - 1) * NT < pieces; q += kDeep * NT) {
    u32x4_t v[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) v[k] = load16(p + 16 * (q + k * NT));
#pragma unroll
    for (int k = 0; k < kDeep; ++k) add(v[k]);
  }
  for (; q < pieces; q += NT) add(load16(p + 16 * q));
  const int last = pieces * N + threadIdx.x;
  if (last < n) {
    const double x = E::get1(p + last * E::kBytes);
    s[0] = fma(x, x, s[0]);
  }
  return s[0] + s[1];
}

// One piece of 16 / TI::kBytes elements, scaled, to the output's type: 8, 16 or 32 bytes.
template <int TI, int TO>
__device__ inline void scale_piece(u32x4_t v, char* o, float c) {
  using I = Elem<TI>;
  using O = Elem<TO>;
  constexpr int N = 16 / I::kBytes;
  float x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = I::get(v, i) * c;
  if constexpr (TO == kTypeF32) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      store16(o + 4 * i, u32x4_t{__float_as_uint(x[i]), __float_as_uint(x[i + 1]), __float_as_uint(x[i + 2]),
                                 __float_as_uint(x[i + 3])});
  } else {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N; i += 2) w[i / 2] = O::pack(x[i], x[i + 1]);
    __builtin_memcpy(o, w, sizeof w);
  }
}

template <int TI, int TO, int NT>
__device__ inline void scale_range(const void* base, void* out, long b, long e, float c) {
  using I = Elem<TI>;
  using O = Elem<TO>;
  constexpr int N = 16 / I::kBytes;
  const char* p = static_cast<const char*>(base) + b * I::kBytes;
  char* o = static_cast<char*>(out) + b * O::kBytes;
  const int n = (int)(e - b), pieces = n / N;
  int q = threadIdx.x;
  for (; q + (kDeep - 1) * NT < pieces; q += kDeep * NT) {
    u32x4_t v[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) v[k] = load16(p + 16 * (q + k * NT));
#pragma unroll
    for (int k = 0; k < kDeep; ++k) scale_piece<TI, TO>(v[k], o + N * O::kBytes * (q + k * NT), c);
  }
  for (; q < pieces; q += NT) scale_piece<TI, TO>(load16(p + 16 * q), o + N * O::kBytes * q, c);
  const int last = pieces * N + threadIdx.x;
  if (last < n) O::put1(o + last * O::kBytes, I::get1(p + last * I::kBytes) * c);
}

template <int TI, int NT>
__device__ inline void scale_to(int to, const void* p, void* o, long b, long e, float c) {
  if (to == kTypeF32) scale_range<TI, kTypeF32, NT>(p, o, b, e, c);
  else if (to == kTypeBf16) scale_range<TI, kTypeBf16, NT>(p, o, b, e, c);
  else scale_range<TI, kTypeF16, NT>(p, o, b, e, c);
}

template <int NT>
__device__ inline double sumsq_of(int ty, const void* p, long b, long e) {
  if (ty == kTypeF32) return sumsq_range<kTypeF32, NT>(p, b, e);
  if (ty == kTypeBf16) return sumsq_range<kTypeBf16, NT>(p, b, e);
  return sumsq_range<kTypeF16, NT>(p, b, e);
}

template <int NT>
__device__ inline void scale_of(int ty, int to, const void* p, void* o, long b, long e, float c) {
  if (ty == kTypeF32) scale_to<kTypeF32, NT>(to, p, o, b, e, c);
  else if (ty == kTypeBf16) scale_to<kTypeBf16, NT>(to, p, o, b, e, c);
  else scale_to<kTypeF16, NT>(to, p, o, b, e, c);
}

// min(1, max_norm / (n + 1e-6)); a NaN norm stays NaN, no limit is no limit
__device__ inline float clip_factor(double n, double max_norm) {
  const double r = max_norm / (n + 1e-6);
  return r >= 1.0 || max_norm == INFINITY ? 1.f : (float)r;
}

}  // namespace

__global__ __launch_bounds__(kClipThreads) void sumsq_kernel(SumsqTable t, double* part) {
  const int i = tensor_of(t.first, t.n, blockIdx.x);
  const long b = (long)(blockIdx.x - t.first[i]) * kClipBlock, e = min(b + kClipBlock, (long)t.numel[i]);
  const double s = block_sum<kClipThreads>(sumsq_of<kClipThreads>(t.type[i], t.in[i], b, e));
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// One block of 1024; 4 loads of a thread in flight (12 K partials for 400 M elements).
__global__ __launch_bounds__(1024) void sumsq_total_kernel(const double* part, long n, double* sumsq) {
  double s[4] = {0, 0, 0, 0};
  for (long i = threadIdx.x; i < n; i += 4096)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + 1024 * k < n) s[k] += part[i + 1024 * k];
  const double v = block_sum<1024>((s[0] + s[1]) + (s[2] + s[3]));
  if (threadIdx.x == 0) *sumsq = v;
}

__global__ __launch_bounds__(kClipThreads) void clip_kernel(ClipTable t, const double* sumsq, double max_norm,
                                                            float* norm) {
  const int i = tensor_of(t.first, t.n, blockIdx.x);
  const long b = (long)(blockIdx.x - t.first[i]) * kClipBlock, e = min(b + kClipBlock, (long)t.numel[i]);
  const double n = sqrt(*sumsq);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
  const float c = clip_factor(n, max_norm);
  if (c == 1.f && t.in[i] == t.out[i]) return;
  scale_of<kClipThreads>(t.in_type[i], t.out_type[i], t.in[i], t.out[i], b, e, c);
}

// Few elements in few tensors: norm and clip by one workgroup, the tensors one
// after the other (both sides of the rule at kClipSmallTensors).
__global__ __launch_bounds__(1024) void clip_small_kernel(ClipTable t, double* sumsq, double max_norm, float* norm) {
  double s = 0;
  for (int i = 0; i < t.n; ++i) s += sumsq_of<1024>(t.in_type[i], t.in[i], 0, t.numel[i]);
  s = block_sum<1024>(s);
  const double n = sqrt(s);
  const float c = clip_factor(n, max_norm);
  if (threadIdx.x == 0) {
    *sumsq = s;
    *norm = (float)n;
  }
  for (int i = 0; i < t.n; ++i)
    if (c != 1.f || t.in[i] != t.out[i])
      scale_of<1024>(t.in_type[i], t.out_type[i], t.in[i], t.out[i], 0, t.numel[i], c);
}

__global__ void norm_kernel(const double* sumsq, float* norm) { *norm = (float)sqrt(*sumsq); }

hipError_t launch_sumsq(const SumsqTable& t, double* part, hipStream_t st) {
  hipLaunchKernelGGL(sumsq_kernel, dim3(t.first[t.n]), dim3(kClipThreads), 0, st, t, part);
  return hipGetLastError();
}
hipError_t launch_sumsq_total(const double* part, int64_t n, double* sumsq, hipStream_t st) {
  hipLaunchKernelGGL(sumsq_total_kernel, dim3(1), dim3(1024), 0, st, part, (long)n, sumsq);
  return hipGetLastError();
}
hipError_t launch_clip(const ClipTable& t, const double* sumsq, double max_norm, float* norm, hipStream_t st) {
  hipLaunchKernelGGL(clip_kernel, dim3(t.first[t.n]), dim3(kClipThreads), 0, st, t, sumsq, max_norm, norm);
  return hipGetLastError();
}
hipError_t launch_clip_small(const ClipTable& t, double* sumsq, double max_norm, float* norm, hipStream_t st) {
  hipLaunchKernelGGL(clip_small_kernel, dim3(1), dim3(1024), 0, st, t, sumsq, max_norm, norm);
  return hipGetLastError();
}
hipError_t launch_norm(const double* sumsq, float* norm, hipStream_t st) {
  hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(1), 0, st, sumsq, norm);
  return hipGetLastError();
}

}  // namespace kd
