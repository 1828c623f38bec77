// Layer norm and its gradients.
//
//   mean = sum x / d, r = 1 / sqrt(sum (x - mean)^2 / d + eps), h = (x - mean) r
//   y = h w + b
//   g = grad w, dx = r (g - sum g / d - h sum (g h) / d), dw = sum_t grad h, db = sum_t grad
//
// Both directions are bound by memory: x once and y once forward, grad, x and
// dx once backward.  A row stays in its threads' registers from the load to
// the store, the variance is taken around the mean (not as a difference of
// two moments, which loses everything where the mean is large), and a
// workgroup goes over many rows, so that weight and bias are read once per
// workgroup.  The sums over rows for dw and db stay in the registers of the
// threads that own those columns; each workgroup leaves one partial row of
// each, which a second kernel adds up in a fixed order.
#include <type_traits>

#include "kd_launch.h"
#include "kd_layers.h"
#include "kd_row.h"

namespace kd {

namespace {

__device__ inline bool row_valid(const uint8_t* mask, int64_t t) { return !mask || mask[t]; }

// ------------------------------------------------------------------ 8-bit copies of a row
// One piece, whose group lies in this wave's neighbouring lanes.
template <int KIND>
__device__ inline void keep_piece(const NormArgs& a, int64_t t, int p, const float (&x)[8], uint32_t row_top) {
  const int lanes = a.group >> 3;
  const bool whole = a.groups == 1;
  const Scale8 g = scale8<KIND>(whole ? row_top : wave_max(top8(x), lanes));
  const int n = (int)(a.d - 8 * (int64_t)p);
  if (n <= 0) return;
  store_q8(a.q + t * a.d + 8 * (int64_t)p, quantize8<KIND>(x, g), n);
  if (whole ? p == 0 : p % lanes == 0) a.scale[t * a.groups + (whole ? 0 : p / lanes)] = g.scale;
}

}  // namespace

// ------------------------------------------------------------------ forward
template <int TY, int R, int K>
__global__ __launch_bounds__(RowTeam<R>::kThreads) void norm_fwd_kernel(NormArgs a) {
  using Team = RowTeam<R>;
  __shared__ float lds[16];
  const int lane = Team::lane();
  float w[K][8], b[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int p = lane + k * R;
    if (a.w) load_any(a.w, a.wtype, a.d, p, w[k]);
    if (a.b) load_any(a.b, a.wtype, a.d, p, b[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!a.w) w[k][i] = 1.f;
      if (!a.b) b[k][i] = 0.f;
    }
  }
  const float inv_d = 1.f / (float)a.d;
  for (int64_t t = (int64_t)blockIdx.x * Team::kRows + Team::slot(); t < a.T; t += (int64_t)gridDim.x * Team::kRows) {
    const bool valid = row_valid(a.mask, t);
    float x[K][8];
    const char* row = a.x + t * a.d * Elem<TY>::kBytes;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (valid) load_row<TY>(row, a.d, lane + k * R, x[k]);
      else
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k][i] = 0.f;
    }
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += x[k][i];
    Team::sum(s, lds);
    const float mean = s[0] * inv_d;
    s[0] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t n = a.d - 8 * (int64_t)(lane + k * R);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float c = i < n ? x[k][i] - mean : 0.f;
        s[0] = fmaf(c, c, s[0]);
      }
    }
    Team::sum(s, lds);
    const float rstd = 1.f / sqrtf(s[0] * inv_d + a.eps);
    if (lane == 0) {
      if (a.mean) a.mean[t] = valid ? mean : 0.f;
      if (a.rstd) a.rstd[t] = valid ? rstd : 0.f;
    }
    uint32_t top = 0;
    if (a.kind && a.groups == 1) {
#pragma unroll
      for (int k = 0; k < K; ++k) top = max(top, top8(x[k]));
      top = Team::most(top, reinterpret_cast<uint32_t*>(lds));
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int p = lane + k * R;
      if (a.kind == kRowsInt8) keep_piece<kRowsInt8>(a, t, p, x[k], top);
      if (a.kind == kRowsE4m3) keep_piece<kRowsE4m3>(a, t, p, x[k], top);
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = valid ? fmaf((x[k][i] - mean) * rstd, w[k][i], b[k][i]) : 0.f;
      store8<TY>(a.y + (t * a.d + 8 * (int64_t)p) * Elem<TY>::kBytes, y, (int)(a.d - 8 * (int64_t)p));
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
      if (a.kind == kRowsInt8) keep_piece<kRowsInt8>(a, t, p, x, top);
      if (a.kind == kRowsE4m3) keep_piece<kRowsE4m3>(a, t, p, x, top);
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

// ------------------------------------------------------------------ backward
namespace {
// piece p of the input of row t: as it is, or from 8 bits
template <int TY, int KIND>
__device__ inline void input_piece(const NormGradArgs& a, int64_t t, int p, float (&x)[8]) {
  if constexpr (KIND == kRowsNone) {
    load_row<TY>(a.x + t * a.d * Elem<TY>::kBytes, a.d, p, x);
  } else {
    const int n = (int)(a.d - 8 * (int64_t)p);
    if (n <= 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
      return;
    }
    const uint2 q = load_q8(a.q + t * a.d + 8 * (int64_t)p, n);
    const float s = a.scale[t * a.groups + (a.groups == 1 ? 0 : 8 * p / a.group)];
    values8<KIND>(q, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= s;
  }
}
}  // namespace

template <int TY, int KIND, int R, int K>
__global__ __launch_bounds__(RowTeam<R>::kThreads) void norm_grad_kernel(NormGradArgs a) {
  using Team = RowTeam<R>;
  __shared__ float lds[2 * 16];
  const int lane = Team::lane();
  float w[K][8], dw[K][8], db[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (a.w) load_any(a.w, a.wtype, a.d, lane + k * R, w[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!a.w) w[k][i] = 1.f;
      dw[k][i] = db[k][i] = 0.f;
    }
  }
  const float inv_d = 1.f / (float)a.d;
  for (int64_t t = (int64_t)blockIdx.x * Team::kRows + Team::slot(); t < a.T; t += (int64_t)gridDim.x * Team::kRows) {
    char* out = a.dx ? a.dx + t * a.d * Elem<TY>::kBytes : nullptr;
    if (!row_valid(a.mask, t)) {
      if (out) {
        const float zero[8] = {};
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int64_t at = 8 * (int64_t)(lane + k * R);
          store8<TY>(out + at * Elem<TY>::kBytes, zero, (int)(a.d - at));
        }
      }
      continue;
    }
    const float mean = a.mean[t], rstd = a.rstd[t];
    float h[K][8], g[K][8];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int p = lane + k * R;
      const int64_t n = a.d - 8 * (int64_t)p;
      input_piece<TY, KIND>(a, t, p, h[k]);
      load_row<TY>(a.grad + t * a.d * Elem<TY>::kBytes, a.d, p, g[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[k][i] = i < n ? (h[k][i] - mean) * rstd : 0.f;
        dw[k][i] = fmaf(g[k][i], h[k][i], dw[k][i]);
        db[k][i] += g[k][i];
        g[k][i] *= w[k][i];
        s[0] += g[k][i];
        s[1] = fmaf(g[k][i], h[k][i], s[1]);
      }
    }
    if (!out) continue;
    Team::sum(s, lds);
    const float c0 = s[0] * inv_d, c1 = s[1] * inv_d;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t at = 8 * (int64_t)(lane + k * R);
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = rstd * (g[k][i] - c0 - h[k][i] * c1);
      store8<TY>(out + at * Elem<TY>::kBytes, o, (int)(a.d - at));
    }
  }
  if (!a.dw && !a.db) return;
  // one partial row of each sum per workgroup; waves that hold a row each are added up first
  if constexpr (Team::kRows > 1) {
    __shared__ float col[Team::kRows][R * 8];
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) col[Team::slot()][lane * 8 + i] = which ? db[k][i] : dw[k][i];
        __syncthreads();
        for (int j = threadIdx.x; j < R * 8; j += Team::kThreads) {
          const int64_t at = (int64_t)k * R * 8 + j;
          float v = 0.f;
#pragma unroll
          for (int r = 0; r < Team::kRows; ++r) v += col[r][j];
          if (at < a.d) a.part[((int64_t)blockIdx.x * 2 + which) * a.d + at] = v;
        }
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t at = 8 * (int64_t)(lane + k * R);
      float* to = a.part + (int64_t)blockIdx.x * 2 * a.d + at;
      store8<kTypeF32>(reinterpret_cast<char*>(to), dw[k], (int)(a.d - at));
      store8<kTypeF32>(reinterpret_cast<char*>(to + a.d), db[k], (int)(a.d - at));
    }
  }
}

// Rows that no workgroup's registers hold; the sums over rows then are kept in
// the workgroup's partial rows, each element by the thread that owns it.
template <int TY, int KIND>
__global__ __launch_bounds__(1024) void norm_grad_long_kernel(NormGradArgs a) {
  using Team = RowTeam<1024>;
  __shared__ float lds[2 * 16];
  const int pieces = (int)((a.d + 7) / 8);
  float* const dw = a.part + (int64_t)blockIdx.x * 2 * a.d;
  float* const db = dw + a.d;
  const float zero[8] = {};
  for (int p = threadIdx.x; p < pieces; p += 1024) {
    store8<kTypeF32>(reinterpret_cast<char*>(dw + 8 * (int64_t)p), zero, (int)(a.d - 8 * (int64_t)p));
    store8<kTypeF32>(reinterpret_cast<char*>(db + 8 * (int64_t)p), zero, (int)(a.d - 8 * (int64_t)p));
  }
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    char* out = a.dx ? a.dx + t * a.d * Elem<TY>::kBytes : nullptr;
    if (!row_valid(a.mask, t)) {
      if (out)
        for (int p = threadIdx.x; p < pieces; p += 1024)
          store8<TY>(out + 8 * (int64_t)p * Elem<TY>::kBytes, zero, (int)(a.d - 8 * (int64_t)p));
      continue;
    }
    const float mean = a.mean[t], rstd = a.rstd[t];
    auto piece = [&](int p, float (&h)[8], float (&g)[8], float (&w)[8]) {
      const int64_t n = a.d - 8 * (int64_t)p;
      input_piece<TY, KIND>(a, t, p, h);
      load_row<TY>(a.grad + t * a.d * Elem<TY>::kBytes, a.d, p, g);
      if (a.w) load_any(a.w, a.wtype, a.d, p, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[i] = i < n ? (h[i] - mean) * rstd : 0.f;
        if (!a.w) w[i] = 1.f;
      }
    };
    float s[2] = {0.f, 0.f};
    for (int p = threadIdx.x; p < pieces; p += 1024) {
      float h[8], g[8], w[8], sw[8], sb[8];
      piece(p, h, g, w);
      const int n = (int)(a.d - 8 * (int64_t)p);
      load_row<kTypeF32>(reinterpret_cast<const char*>(dw), a.d, p, sw);
      load_row<kTypeF32>(reinterpret_cast<const char*>(db), a.d, p, sb);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sw[i] = fmaf(g[i], h[i], sw[i]);
        sb[i] += g[i];
        s[0] = fmaf(g[i], w[i], s[0]);
        s[1] = fmaf(g[i] * w[i], h[i], s[1]);
      }
      store8<kTypeF32>(reinterpret_cast<char*>(dw + 8 * (int64_t)p), sw, n);
      store8<kTypeF32>(reinterpret_cast<char*>(db + 8 * (int64_t)p), sb, n);
    }
    if (!out) continue;
    Team::sum(s, lds);
    const float c0 = s[0] / (float)a.d, c1 = s[1] / (float)a.d;
    for (int p = threadIdx.x; p < pieces; p += 1024) {
      float h[8], g[8], w[8], o[8];
      piece(p, h, g, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = rstd * (g[i] * w[i] - c0 - h[i] * c1);
      store8<TY>(out + 8 * (int64_t)p * Elem<TY>::kBytes, o, (int)(a.d - 8 * (int64_t)p));
    }
  }
}

// dw and db from the workgroups' partial rows: 64 columns a workgroup, the
// partial rows dealt to 16 waves and added up through LDS.
__global__ __launch_bounds__(1024) void norm_sum_kernel(NormGradArgs a) {
  __shared__ float col[16][64];
  const int which = blockIdx.y;
  const int64_t c = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
  const int w = threadIdx.x >> 6;
  float v = 0.f;
  if (c < a.d)
    for (int b = w; b < a.blocks; b += 16) v += a.part[((int64_t)b * 2 + which) * a.d + c];
  col[w][threadIdx.x & 63] = v;
  __syncthreads();
  if (w != 0 || c >= a.d) return;
  v = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) v += col[k][threadIdx.x & 63];
  char* to = which ? a.db : a.dw;
  if (to) store_any1(to, a.wtype, c, v);
}

// ------------------------------------------------------------------ launches
namespace {
// rows that a workgroup holds at once
int64_t team_rows(int64_t d) { return d <= 2048 ? 4 : 1; }
}  // namespace

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st) {
  const int64_t rows = (a.T + team_rows(a.d) - 1) / team_rows(a.d);
  pick_type(a.type, [&](auto ty) {
    constexpr int TY = decltype(ty)::value;
    const bool held = pick_row(a.d, [&](auto r, auto k) {
      constexpr int R = decltype(r)::value, K = decltype(k)::value;
      const dim3 grid((unsigned)std::min<int64_t>(rows, 2048));
      hipLaunchKernelGGL((norm_fwd_kernel<TY, R, K>), grid, dim3(RowTeam<R>::kThreads), 0, st, a);
    });
    if (!held)
      hipLaunchKernelGGL((norm_fwd_long_kernel<TY>), dim3((unsigned)std::min<int64_t>(a.T, 512)), dim3(1024), 0, st, a);
  });
  return hipGetLastError();
}

int norm_grad_blocks(int64_t T, int64_t d) {
  return (int)std::min<int64_t>(std::max<int64_t>((T + team_rows(d) - 1) / team_rows(d), 1), d <= kRowMost ? 512 : 256);
}

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)a.blocks);
  pick_type(a.type, [&](auto ty) {
    constexpr int TY = decltype(ty)::value;
    auto with = [&](auto kind) {
      constexpr int KIND = decltype(kind)::value;
      const bool held = pick_row(a.d, [&](auto r, auto k) {
        constexpr int R = decltype(r)::value, K = decltype(k)::value;
        hipLaunchKernelGGL((norm_grad_kernel<TY, KIND, R, K>), grid, dim3(RowTeam<R>::kThreads), 0, st, a);
      });
      if (!held) hipLaunchKernelGGL((norm_grad_long_kernel<TY, KIND>), grid, dim3(1024), 0, st, a);
    };
    using std::integral_constant;
    if (a.kind == kRowsInt8) with(integral_constant<int, kRowsInt8>());
    else if (a.kind == kRowsE4m3) with(integral_constant<int, kRowsE4m3>());
    else with(integral_constant<int, kRowsNone>());
  });
  return hipGetLastError();
}

hipError_t launch_norm_sum(const NormGradArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)((a.d + 63) / 64), 2), dim3(1024), 0, st, a);
  return hipGetLastError();
}

}  // namespace kd
