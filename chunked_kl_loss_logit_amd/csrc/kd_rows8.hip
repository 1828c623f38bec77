// Rows in 8 bits and back (kd_rows8.h has the rounding).
//
// Bound by memory: 3 bytes a value of a 16-bit type each way (16384 x 4096 bf16
// in groups of 128 35-41 us to int8, 30 back, part of it from the last-level cache).  A lane holds 8
// consecutive values; a group of 32 to 512 values is then 4 to 64 neighbouring
// lanes of one wave, which find its largest by shuffles.  Where a row is one
// group, it is held in registers as for layer norm.
#include <type_traits>

#include "kd_layers.h"
#include "kd_row.h"

namespace kd {

namespace {
constexpr int kRowsThreads = 256;

// Lanes of a row: the pieces of its groups, to a power of two below a
// workgroup so that rows are told apart by shifts.
struct Lanes {
  int shift;       // log2 of the lanes of a row within a workgroup
  int64_t slabs;   // workgroups of a row
};
Lanes lanes_of(int64_t pieces) {
  Lanes l{0, 1};
  while (l.shift < 8 && (int64_t(1) << l.shift) < pieces) ++l.shift;
  l.slabs = (pieces + kRowsThreads - 1) / kRowsThreads;
  return l;
}
}  // namespace

template <int TY, int KIND>
__global__ __launch_bounds__(kRowsThreads) void quantize_kernel(RowsArgs a, int shift, int slabs) {
  const int lanes = a.group >> 3;
  const int slab = blockIdx.x % slabs;
  const int rows = kRowsThreads >> shift;
  const int p = slab * kRowsThreads + (threadIdx.x & ((1 << shift) - 1));
  const int n = (int)(a.d - 8 * (int64_t)p);
  const int64_t step = (int64_t)(gridDim.x / slabs) * rows;
  for (int64_t t0 = (int64_t)(blockIdx.x / slabs) * rows; t0 < a.T; t0 += step) {
    const int64_t t = t0 + (threadIdx.x >> shift);
    float x[8] = {};
    if (t < a.T) load_row<TY>(a.x + t * a.d * Elem<TY>::kBytes, a.d, p, x);
    const Scale8 g = scale8<KIND, TY != kTypeF32>(wave_max(top8(x), lanes));
    if (t >= a.T || n <= 0) continue;
    store_q8(a.q + t * a.d + 8 * (int64_t)p, quantize8<KIND, TY != kTypeF32>(x, g), n);
    if (p % lanes == 0) a.scale[t * a.groups + p / lanes] = g.scale;
  }
}

template <int TY, int KIND, int R, int K>
__global__ __launch_bounds__(RowTeam<R>::kThreads) void quantize_row_kernel(RowsArgs a) {
  using Team = RowTeam<R>;
  __shared__ uint32_t lds[16];
  const int lane = Team::lane();
  for (int64_t t = (int64_t)blockIdx.x * Team::kRows + Team::slot(); Team::left(t, a.T); t += (int64_t)gridDim.x * Team::kRows) {
    const int64_t d = Team::elements(t, a.T, a.d);
    float x[K][8];
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      load_row<TY>(a.x + t * a.d * Elem<TY>::kBytes, d, lane + k * R, x[k]);
      top = max(top, top8(x[k]));
    }
    const Scale8 g = scale8<KIND, TY != kTypeF32>(Team::most(top, lds));
    if (lane == 0 && d > 0) a.scale[t] = g.scale;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t at = 8 * (int64_t)(lane + k * R);
      if (at < d) store_q8(a.q + t * a.d + at, quantize8<KIND, TY != kTypeF32>(x[k], g), (int)(d - at));
    }
  }
}

template <int TY, int KIND>
__global__ __launch_bounds__(1024) void quantize_long_kernel(RowsArgs a) {
  __shared__ uint32_t lds[16];
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const char* row = a.x + t * a.d * Elem<TY>::kBytes;
    uint32_t top = 0;
    for (int64_t at = 8 * (int64_t)threadIdx.x; at < a.d; at += 8192) {
      float x[8];
      load_row<TY>(row, a.d, (int)(at / 8), x);
      top = max(top, top8(x));
    }
    const Scale8 g = scale8<KIND, TY != kTypeF32>(RowTeam<1024>::most(top, lds));
    if (threadIdx.x == 0) a.scale[t] = g.scale;
    for (int64_t at = 8 * (int64_t)threadIdx.x; at < a.d; at += 8192) {
      float x[8];
      load_row<TY>(row, a.d, (int)(at / 8), x);
      store_q8(a.q + t * a.d + at, quantize8<KIND, TY != kTypeF32>(x, g), (int)(a.d - at));
    }
  }
}

template <int TY, int KIND>
__global__ __launch_bounds__(kRowsThreads) void dequantize_kernel(RowsArgs a, int shift, int slabs) {
  const int slab = blockIdx.x % slabs;
  const int rows = kRowsThreads >> shift;
  const int p = slab * kRowsThreads + (threadIdx.x & ((1 << shift) - 1));
  const int n = (int)(a.d - 8 * (int64_t)p);
  if (n <= 0) return;
  const int64_t step = (int64_t)(gridDim.x / slabs) * rows;
  char* const out = const_cast<char*>(a.x);
  for (int64_t t = (int64_t)(blockIdx.x / slabs) * rows + (threadIdx.x >> shift); t < a.T; t += step) {
    float x[8];
    uint2 q = load_q8(a.q + t * a.d + 8 * (int64_t)p, n, p > 0);
    settle_q8(q, n, p > 0);
    values8<KIND>(q, x);
    const float s = a.scale[t * a.groups + (a.groups == 1 ? 0 : 8 * p / a.group)];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] *= s;
      // the product is rounded to 32 bits, also where the compiler could multiply into 16 bits at once
      asm volatile("" : "+v"(x[i]));
    }
    store8<TY>(out + (t * a.d + 8 * (int64_t)p) * Elem<TY>::kBytes, x, n);
  }
}

namespace {
template <class F>
void with_kind(const RowsArgs& a, F&& f) {
  using std::integral_constant;
  pick_type(a.type, [&](auto ty) {
    if (a.kind == kRowsInt8) f(ty, integral_constant<int, kRowsInt8>());
    else f(ty, integral_constant<int, kRowsE4m3>());
  });
}
dim3 rows_grid(const RowsArgs& a, const Lanes& l) {
  const int64_t rows = kRowsThreads >> l.shift, blocks = (a.T + rows - 1) / rows;
  return dim3((unsigned)(std::min<int64_t>(blocks, std::max<int64_t>(8192 / l.slabs, 1)) * l.slabs));
}
}  // namespace

hipError_t launch_rows_quantize(const RowsArgs& a, hipStream_t st) {
  with_kind(a, [&](auto ty, auto kind) {
    constexpr int TY = decltype(ty)::value, KIND = decltype(kind)::value;
    // a group that is the row, unless a wave's lanes hold it
    if (a.groups == 1) {
      const bool held = pick_shape<Shape<16, 1>, Shape<32, 1>, Shape<64, 1>, Shape<128, 1>, Shape<256, 1>, Shape<512, 1>,
                                   Shape<256, 3>, Shape<512, 2>, Shape<1024, 2>>(a.d, [&](auto r, auto k) {
        constexpr int R = decltype(r)::value, K = decltype(k)::value;
        const int64_t rows = (a.T + RowTeam<R>::kRows - 1) / RowTeam<R>::kRows;
        hipLaunchKernelGGL((quantize_row_kernel<TY, KIND, R, K>), dim3((unsigned)std::min<int64_t>(rows, 8192)),
                           dim3(RowTeam<R>::kThreads), 0, st, a);
      });
      if (!held)
        hipLaunchKernelGGL((quantize_long_kernel<TY, KIND>), dim3((unsigned)std::min<int64_t>(a.T, 512)), dim3(1024), 0,
                           st, a);
      return;
    }
    const Lanes l = lanes_of(a.groups * (a.group / 8));
    hipLaunchKernelGGL((quantize_kernel<TY, KIND>), rows_grid(a, l), dim3(kRowsThreads), 0, st, a, l.shift, (int)l.slabs);
  });
  return hipGetLastError();
}

hipError_t launch_rows_dequantize(const RowsArgs& a, hipStream_t st) {
  with_kind(a, [&](auto ty, auto kind) {
    constexpr int TY = decltype(ty)::value, KIND = decltype(kind)::value;
    const Lanes l = lanes_of((a.d + 7) / 8);
    hipLaunchKernelGGL((dequantize_kernel<TY, KIND>), rows_grid(a, l), dim3(kRowsThreads), 0, st, a, l.shift,
                       (int)l.slabs);
  });
  return hipGetLastError();
}

}  // namespace kd
