// Layer norm.
//
//   mean = sum x / d, r = 1 / sqrt(sum (x - mean)^2 / d + eps), h = (x - mean) r
//   y = h w + b
//
// Bound by memory: x once and y once.  A row stays in its threads' registers
// from the load to the store, the variance is taken around the mean (not as a
// difference of two moments, which loses everything where the mean is large),
// and a workgroup goes over many rows, so that weight and bias are read once
// per workgroup.  Up to 4096 elements one piece of 8 a thread (16384 x 4096 bf16 in
// turn from four inputs 51 us, 268 MB at 5.2 TB/s, with two pieces the same; with its
// copy in 8 bits 67 both ways).  Beyond that three or two, as 16 waves at one
// barrier cost more: 8192 x 8192 with one 55 us, so 51, and with the copy 77 and 73
// (335 MB); 14563 x 4608 69 and 49, 95 and 81.  Narrow rows share a workgroup, by the
// smallest shape that holds them: 67 M values in rows of 136 116 us in whole
// waves, 67 in halves; of 520 in four waves 110, in two 67.
#include <type_traits>

#include "kd_launch.h"
#include "kd_layers.h"
#include "kd_row.h"

// Products and sums are fused where fmaf says so and nowhere else: what a call
// computes does not hang on what else its kernel has to do.
#pragma clang fp contract(off)

namespace kd {

namespace {

constexpr int64_t kNormBlocks = 2048;  // workgroups of the forward pass at most

// ------------------------------------------------------------------ 8-bit copies of a row
// One piece, whose group lies in this wave's neighbouring lanes; d: the row's
// elements, or 0 for a row behind the last one.
template <int TY, int KIND, bool WHOLE>
__device__ inline void keep_piece(const NormArgs& a, int64_t t, int64_t d, int p, const float (&x)[8], uint32_t row_top) {
  const int lanes = a.group >> 3;
  const bool whole = a.groups == 1;
  const Scale8 g = scale8<KIND, TY != kTypeF32>(whole ? row_top : wave_max(top8(x), lanes));
  const int n = (int)(d - 8 * (int64_t)p);
  if (n <= 0) return;
  store_q8<WHOLE>(a.q + t * a.d + 8 * (int64_t)p, quantize8<KIND, TY != kTypeF32>(x, g), n);
  if (whole ? p == 0 : p % lanes == 0) a.scale[t * a.groups + (whole ? 0 : p / lanes)] = g.scale;
}

}  // namespace

// ------------------------------------------------------------------ forward
// The thread's weights and biases: in registers, or in LDS where the 8-bit copy
// takes the registers: with the copy, in registers / in LDS, 16384 x 4096 bf16 106 /
// 67 us, 14563 x 4608 150 / 81, 8192 x 8192 74 / 73; without one 52 / 53, 49 / 58, 51 / 55.
template <bool LDS, int N>
struct Affine {
  float w[N][8], b[N][8];
};
template <int N>
struct Affine<true, N> {};

// Waves a SIMD for which there have to be registers: as many as leave hardly any
// of them in memory.
constexpr int norm_waves(int type, int pieces) {
  if (pieces == 1) return type != kTypeF32 ? 8 : 6;
  return pieces > 2 && type == kTypeF32 ? 3 : 4;
}

// The row's pieces stay in registers as they were loaded, and the next row's
// are loaded while one is worked on.
template <int TY, int KIND, bool WHOLE, int R, int K>
__global__ __launch_bounds__(RowTeam<R>::kThreads, norm_waves(TY, K)) void norm_fwd_kernel(NormArgs a) {
  using Team = RowTeam<R>;
  constexpr bool kLds = KIND != kRowsNone;
  __shared__ float lds[16];
  __shared__ __attribute__((aligned(16))) float affine[2][kLds ? R * K * 8 : 4];
  const int lane = Team::lane();
  Affine<kLds, K> own;
  auto piece = [&](int p, float (&w)[8], float (&b)[8]) {
    if (a.w) load_any(a.w, a.wtype, a.d, p, w);
    if (a.b) load_any(a.b, a.wtype, a.d, p, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!a.w) w[i] = 1.f;
      if (!a.b) b[i] = 0.f;
    }
  };
  if constexpr (kLds) {
    for (int p = threadIdx.x; p < R * K; p += Team::kThreads) {
      float w[8], b[8];
      piece(p, w, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        affine[0][8 * p + i] = w[i];
        affine[1][8 * p + i] = b[i];
      }
    }
    __syncthreads();
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) piece(lane + k * R, own.w[k], own.b[k]);
  }
  const float inv_d = 1.f / (float)a.d;
  const int64_t step = (int64_t)gridDim.x * Team::kRows;
  int64_t t = (int64_t)blockIdx.x * Team::kRows + Team::slot();
  Raw8<TY> r[K], next[K];
  auto load = [&](Raw8<TY> (&to)[K], int64_t row) {  // masked rows and those behind the last one as zeros
    const bool there = row < a.T && row_valid(a.mask, row);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t at = 8 * (int64_t)(lane + k * R);
      to[k] = load8<TY, WHOLE>(a.x + (row * a.d + at) * Elem<TY>::kBytes, there ? (int)(a.d - at) : 0, at > 0);
    }
  };
  load(next, t);
  for (; Team::left(t, a.T); t += step) {
    const int64_t d = Team::elements(t, a.T, a.d);
    const bool valid = d > 0 && row_valid(a.mask, t);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      r[k] = next[k];
      settle8<TY, WHOLE>(r[k], (int)(a.d - 8 * (int64_t)(lane + k * R)), lane + k * R > 0);
    }
    load(next, t + step);
    float s[1] = {0.f};
    float x[8];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      unpack8<TY>(r[k], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += x[i];
    }
    Team::sum(s, lds);
    const float mean = s[0] * inv_d;
    s[0] = 0.f;
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int n = (int)(a.d - 8 * (int64_t)(lane + k * R));
      unpack8<TY>(r[k], x);
      if (WHOLE ? n > 0 : n >= 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float c = x[i] - mean;
          s[0] = fmaf(c, c, s[0]);
        }
      } else if (!WHOLE) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float c = i < n ? x[i] - mean : 0.f;
          s[0] = fmaf(c, c, s[0]);
        }
      }
      if (KIND != kRowsNone && a.groups == 1) top = max(top, top8(x));
    }
    Team::sum(s, lds);
    const float rstd = 1.f / sqrtf(s[0] * inv_d + a.eps);
    if (lane == 0 && d > 0) {
      if (a.mean) a.mean[t] = valid ? mean : 0.f;
      if (a.rstd) a.rstd[t] = valid ? rstd : 0.f;
    }
    if (KIND != kRowsNone && a.groups == 1) top = Team::most(top, reinterpret_cast<uint32_t*>(lds));
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int p = lane + k * R;
      unpack8<TY>(r[k], x);
      if constexpr (KIND != kRowsNone) keep_piece<TY, KIND, WHOLE>(a, t, d, p, x, top);
      if constexpr (kLds) {
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
          const float4 w = *reinterpret_cast<const float4*>(&affine[0][8 * p + h]);
          const float4 b = *reinterpret_cast<const float4*>(&affine[1][8 * p + h]);
          x[h] = fmaf((x[h] - mean) * rstd, w.x, b.x);
          x[h + 1] = fmaf((x[h + 1] - mean) * rstd, w.y, b.y);
          x[h + 2] = fmaf((x[h + 2] - mean) * rstd, w.z, b.z);
          x[h + 3] = fmaf((x[h + 3] - mean) * rstd, w.w, b.w);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fmaf((x[i] - mean) * rstd, own.w[k][i], own.b[k][i]);
      }
      if (!valid) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
      }
      store8<TY, WHOLE>(a.y + (t * a.d + 8 * (int64_t)p) * Elem<TY>::kBytes, x, (int)(d - 8 * (int64_t)p));
    }
  }
}

// Rows that no workgroup's registers hold: read once for each pass over them.
template <int TY>
__global__ __launch_bounds__(1024) void norm_fwd_long_kernel(NormArgs a) {
  using Team = RowTeam<1024>;
  __shared__ float lds[16];
  const int pieces = (int)((a.d + 7) / 8);
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const bool valid = row_valid(a.mask, t);
    const char* row = a.x + t * a.d * Elem<TY>::kBytes;
    auto over = [&](auto&& f) {
      for (int p = threadIdx.x; p < (pieces + 1023) / 1024 * 1024; p += 1024) {
        float x[8] = {};
        if (valid) load_row<TY>(row, a.d, p, x);
        f(p, x, a.d - 8 * (int64_t)p);
      }
    };
    float s[1] = {0.f};
    uint32_t top = 0;
    over([&](int, const float (&x)[8], int64_t) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += x[i];
      top = max(top, top8(x));
    });
    Team::sum(s, lds);
    const float mean = s[0] / (float)a.d;
    s[0] = 0.f;
    over([&](int, const float (&x)[8], int64_t n) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float c = i < n ? x[i] - mean : 0.f;
        s[0] = fmaf(c, c, s[0]);
      }
    });
    Team::sum(s, lds);
    const float rstd = 1.f / sqrtf(s[0] / (float)a.d + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[t] = valid ? mean : 0.f;
      if (a.rstd) a.rstd[t] = valid ? rstd : 0.f;
    }
    if (a.kind && a.groups == 1) top = Team::most(top, reinterpret_cast<uint32_t*>(lds));
    over([&](int p, const float (&x)[8], int64_t n) {
      if (a.kind == kRowsInt8) keep_piece<TY, kRowsInt8, false>(a, t, a.d, p, x, top);
      if (a.kind == kRowsE4m3) keep_piece<TY, kRowsE4m3, false>(a, t, a.d, p, x, top);
      if (n <= 0) return;
      float w[8], b[8], y[8];
      if (a.w) load_any(a.w, a.wtype, a.d, p, w);
      if (a.b) load_any(a.b, a.wtype, a.d, p, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[i] = fmaf((x[i] - mean) * rstd, a.w ? w[i] : 1.f, a.b ? b[i] : 0.f);
        if (!valid) y[i] = 0.f;
      }
      store8<TY>(a.y + (t * a.d + 8 * (int64_t)p) * Elem<TY>::kBytes, y, (int)n);
    });
    __syncthreads();
  }
}

// ------------------------------------------------------------------ launches
hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st) {
  pick_type(a.type, [&](auto ty) {
    constexpr int TY = decltype(ty)::value;
    auto with = [&](auto kind) {
      constexpr int KIND = decltype(kind)::value;
      auto launch = [&](auto r, auto k) {
        constexpr int R = decltype(r)::value, K = decltype(k)::value;
        const int64_t rows = (a.T + RowTeam<R>::kRows - 1) / RowTeam<R>::kRows;
        const dim3 grid((unsigned)std::min<int64_t>(rows, kNormBlocks)), block(RowTeam<R>::kThreads);
        if (a.d % 8 == 0) hipLaunchKernelGGL((norm_fwd_kernel<TY, KIND, true, R, K>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((norm_fwd_kernel<TY, KIND, false, R, K>), grid, block, 0, st, a);
      };
      // by the width alone, so that a row's bits do not hang on how many rows there are
      const bool held = pick_shape<Shape<16, 1>, Shape<32, 1>, Shape<64, 1>, Shape<128, 1>, Shape<256, 1>, Shape<512, 1>,
                                   Shape<256, 3>, Shape<512, 2>, Shape<1024, 2>>(a.d, launch);
      if (!held)
        hipLaunchKernelGGL((norm_fwd_long_kernel<TY>), dim3((unsigned)std::min<int64_t>(a.T, 512)), dim3(1024), 0, st, a);
    };
    using std::integral_constant;
    if (a.kind == kRowsInt8) with(integral_constant<int, kRowsInt8>());
    else if (a.kind == kRowsE4m3) with(integral_constant<int, kRowsE4m3>());
    else with(integral_constant<int, kRowsNone>());
  });
  return hipGetLastError();
}

}  // namespace kd
