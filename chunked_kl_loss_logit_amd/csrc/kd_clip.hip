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
#include <hip/hip_fp16.h>

#include "kd_gemm.h"
#include "kd_policy.h"

namespace kd {

namespace {

constexpr int kClipThreads = 256;
enum { kTypeF32 = 0, kTypeBf16 = 1, kTypeF16 = 2 };

__device__ inline double block_sum(double v) {
  __shared__ double red[kClipThreads / 64];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int i = 0; i < kClipThreads / 64; ++i) v += red[i];
  return v;
}

// the tensor that block b covers
__device__ inline int tensor_of(const ClipTable& t, int b) {
  int lo = 0, hi = t.n;  // first index with first > b
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= b) lo = mid + 1; else hi = mid;
  }
  return lo - 1;
}

template <int TY>
__device__ inline float load1(const void* p, long i) {
  if constexpr (TY == kTypeF32) return static_cast<const float*>(p)[i];
  if constexpr (TY == kTypeBf16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  if constexpr (TY == kTypeF16) return __half2float(static_cast<const __half*>(p)[i]);
}
template <int TY>
__device__ inline void store1(void* p, long i, float v) {
  if constexpr (TY == kTypeF32) static_cast<float*>(p)[i] = v;
  if constexpr (TY == kTypeBf16) static_cast<uint16_t*>(p)[i] = (uint16_t)Bf16::cvt(v);
  if constexpr (TY == kTypeF16) static_cast<__half*>(p)[i] = __float2half_rn(v);
}

template <int TY>
__device__ inline double sumsq_range(const void* p, long b, long e) {
  double s = 0;
  for (long i = b + threadIdx.x; i < e; i += kClipThreads) {
    const double x = load1<TY>(p, i);
    s = fma(x, x, s);
  }
  return s;
}

template <int TI, int TO>
__device__ inline void scale_range(const void* p, void* o, long b, long e, float c) {
  for (long i = b + threadIdx.x; i < e; i += kClipThreads) store1<TO>(o, i, load1<TI>(p, i) * c);
}

template <int TI>
__device__ inline void scale_to(int to, const void* p, void* o, long b, long e, float c) {
  if (to == kTypeF32) scale_range<TI, kTypeF32>(p, o, b, e, c);
  else if (to == kTypeBf16) scale_range<TI, kTypeBf16>(p, o, b, e, c);
  else scale_range<TI, kTypeF16>(p, o, b, e, c);
}

}  // namespace

__global__ __launch_bounds__(kClipThreads) void sumsq_kernel(ClipTable t, double* part) {
  const int i = tensor_of(t, blockIdx.x);
  const long b = (long)(blockIdx.x - t.first[i]) * kClipBlock, e = min(b + kClipBlock, (long)t.numel[i]);
  const int ty = t.in_type[i];
  double s;
  if (ty == kTypeF32) s = sumsq_range<kTypeF32>(t.in[i], b, e);
  else if (ty == kTypeBf16) s = sumsq_range<kTypeBf16>(t.in[i], b, e);
  else s = sumsq_range<kTypeF16>(t.in[i], b, e);
  s = block_sum(s);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ __launch_bounds__(kClipThreads) void sumsq_total_kernel(const double* part, long n, double* sumsq) {
  double s = 0;
  for (long i = threadIdx.x; i < n; i += kClipThreads) s += part[i];
  s = block_sum(s);
  if (threadIdx.x == 0) *sumsq = s;
}

__global__ __launch_bounds__(kClipThreads) void clip_kernel(ClipTable t, const double* sumsq, double max_norm) {
  const int i = tensor_of(t, blockIdx.x);
  const long b = (long)(blockIdx.x - t.first[i]) * kClipBlock, e = min(b + kClipBlock, (long)t.numel[i]);
  const double r = max_norm / (sqrt(*sumsq) + 1e-6);
  const float c = r >= 1.0 || max_norm == INFINITY ? 1.f : (float)r;  // a NaN norm stays NaN
  if (c == 1.f && t.in[i] == t.out[i]) return;
  const int ty = t.in_type[i], to = t.out_type[i];
  if (ty == kTypeF32) scale_to<kTypeF32>(to, t.in[i], t.out[i], b, e, c);
  else if (ty == kTypeBf16) scale_to<kTypeBf16>(to, t.in[i], t.out[i], b, e, c);
  else scale_to<kTypeF16>(to, t.in[i], t.out[i], b, e, c);
}

__global__ void norm_kernel(const double* sumsq, float* norm) { *norm = (float)sqrt(*sumsq); }

hipError_t launch_sumsq(const ClipTable& t, double* part, hipStream_t st) {
  hipLaunchKernelGGL(sumsq_kernel, dim3(t.first[t.n]), dim3(kClipThreads), 0, st, t, part);
  return hipGetLastError();
}
hipError_t launch_sumsq_total(const double* part, int64_t n, double* sumsq, hipStream_t st) {
  hipLaunchKernelGGL(sumsq_total_kernel, dim3(1), dim3(kClipThreads), 0, st, part, (long)n, sumsq);
  return hipGetLastError();
}
hipError_t launch_clip(const ClipTable& t, const double* sumsq, double max_norm, hipStream_t st) {
  hipLaunchKernelGGL(clip_kernel, dim3(t.first[t.n]), dim3(kClipThreads), 0, st, t, sumsq, max_norm);
  return hipGetLastError();
}
hipError_t launch_norm(const double* sumsq, float* norm, hipStream_t st) {
  hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(1), 0, st, sumsq, norm);
  return hipGetLastError();
}

}  // namespace kd
