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

// Products and sums are fused where fmaf says so and nowhere else: what a call
// computes does not hang on what else its kernel has to do.
#pragma clang fp contract(off)

namespace kd {

namespace {

constexpr int64_t kNormBlocks = 2048;  // workgroups of the forward pass at most

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
// The thread's weights and biases: in registers, or in LDS where the 8-bit copy
// takes the registers (two workgroups of a wide row's 1024 threads then fit a
// CU: 8192 x 8192 with its copy 123 us -> 95; without a copy LDS costs 46 -> 56).
template <bool LDS, int N>
struct Affine {
  float w[N][8], b[N][8];
};
template <int N>
struct Affine<true, N> {};

// The row's pieces stay in registers as they were loaded, and the next row's
// are loaded while one is worked on.
template <int TY, int KIND, int R, int K>
__global__ __launch_bounds__(RowTeam<R>::kThreads, K == 1 ? 8 : 4) void norm_fwd_kernel(NormArgs a) {
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
      to[k] = load8<TY>(a.x + (row * a.d + at) * Elem<TY>::kBytes, there ? (int)(a.d - at) : 0, at > 0);
    }
  };
  load(next, t);
  for (; t < a.T; t += step) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      r[k] = next[k];
      settle8<TY>(r[k], (int)(a.d - 8 * (int64_t)(lane + k * R)), lane + k * R > 0);
    }
    load(next, t + step);
    if (!row_valid(a.mask, t)) {
      if (lane == 0) {
        if (a.mean) a.mean[t] = 0.f;
        if (a.rstd) a.rstd[t] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int p = lane + k * R;
        const float zero[8] = {};
        if constexpr (KIND != kRowsNone) keep_piece<KIND>(a, t, p, zero, 0u);
        store8<TY>(a.y + (t * a.d + 8 * (int64_t)p) * Elem<TY>::kBytes, zero, (int)(a.d - 8 * (int64_t)p));
      }
      continue;
    }
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
      if (n >= 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float c = x[i] - mean;
          s[0] = fmaf(c, c, s[0]);
        }
      } else {
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
    if (lane == 0) {
      if (a.mean) a.mean[t] = mean;
      if (a.rstd) a.rstd[t] = rstd;
    }
    if (KIND != kRowsNone && a.groups == 1) top = Team::most(top, reinterpret_cast<uint32_t*>(lds));
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int p = lane + k * R;
      unpack8<TY>(r[k], x);
      if constexpr (KIND != kRowsNone) keep_piece<KIND>(a, t, p, x, top);
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
      store8<TY>(a.y + (t * a.d + 8 * (int64_t)p) * Elem<TY>::kBytes, x, (int)(a.d - 8 * (int64_t)p));
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
// A piece of the input as it lies in memory: as it is, or 8 bits and a scale.
template <int TY, int KIND>
struct Input {
  Raw8<TY> x;
};
template <int TY>
struct Input<TY, kRowsInt8> {
  uint2 q;
  float scale;
};
template <int TY>
struct Input<TY, kRowsE4m3> {
  uint2 q;
  float scale;
};

// n values of piece p of row t
template <int TY, int KIND>
__device__ inline Input<TY, KIND> load_input(const NormGradArgs& a, int64_t t, int p, int n) {
  Input<TY, KIND> r;
  const int64_t at = t * a.d + 8 * (int64_t)p;
  if constexpr (KIND == kRowsNone) {
    r.x = load8<TY>(a.x + at * Elem<TY>::kBytes, n, p > 0);
  } else {
    r.q = load_q8(a.q + at, n, p > 0);
    r.scale = n > 0 ? a.scale[t * a.groups + (a.groups == 1 ? 0 : 8 * p / a.group)] : 0.f;
  }
  return r;
}
template <int TY, int KIND>
__device__ inline void settle_input(Input<TY, KIND>& r, int p, int n) {
  if constexpr (KIND == kRowsNone) settle8<TY>(r.x, n, p > 0);
  else settle_q8(r.q, n, p > 0);
}
template <int TY, int KIND>
__device__ inline void input_values(const Input<TY, KIND>& r, float (&x)[8]) {
  if constexpr (KIND == kRowsNone) {
    unpack8<TY>(r.x, x);
  } else {
    values8<KIND>(r.q, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= r.scale;
  }
}
}  // namespace

template <int TY, int KIND, int R, int K>
__global__ __launch_bounds__(RowTeam<R>::kThreads, 4) void norm_grad_kernel(NormGradArgs a) {
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
  const int64_t step = (int64_t)gridDim.x * Team::kRows;
  int64_t t = (int64_t)blockIdx.x * Team::kRows + Team::slot();
  Input<TY, KIND> xr[K], xn[K];
  Raw8<TY> gr[K], gn[K];
  float mean = 0.f, rstd = 0.f;
  auto load = [&](int64_t row) {  // masked rows and those behind the last one as zeros
    const bool there = row < a.T && row_valid(a.mask, row);
    mean = there ? a.mean[row] : 0.f;
    rstd = there ? a.rstd[row] : 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int p = lane + k * R;
      const int n = there ? (int)(a.d - 8 * (int64_t)p) : 0;
      xn[k] = load_input<TY, KIND>(a, row, p, n);
      gn[k] = load8<TY>(a.grad + (row * a.d + 8 * (int64_t)p) * Elem<TY>::kBytes, n, p > 0);
    }
  };
  load(t);
  for (; t < a.T; t += step) {
    char* out = a.dx ? a.dx + t * a.d * Elem<TY>::kBytes : nullptr;
    const float m = mean, r = rstd;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int p = lane + k * R, n = (int)(a.d - 8 * (int64_t)p);
      xr[k] = xn[k];
      gr[k] = gn[k];
      settle_input<TY, KIND>(xr[k], p, n);
      settle8<TY>(gr[k], n, p > 0);
    }
    load(t + step);  // the next row, while this one is worked on
    // a piece's h and g from what lies in registers as it was loaded
    auto values = [&](int k, float (&h)[8], float (&g)[8]) {
      const int64_t n = a.d - 8 * (int64_t)(lane + k * R);
      input_values<TY, KIND>(xr[k], h);
      unpack8<TY>(gr[k], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = i < n ? (h[i] - m) * r : 0.f;
    };
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float h[8], g[8];
      values(k, h, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dw[k][i] = fmaf(g[i], h[i], dw[k][i]);
        db[k][i] += g[i];
        const float v = g[i] * w[k][i];
        s[0] += v;
        s[1] = fmaf(v, h[i], s[1]);
      }
    }
    if (!out) continue;
    Team::sum(s, lds);
    const float c0 = s[0] * inv_d, c1 = s[1] * inv_d;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t at = 8 * (int64_t)(lane + k * R);
      float h[8], g[8];
      values(k, h, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = r * fmaf(-h[i], c1, g[i] * w[k][i] - c0);
      store8<TY>(out + at * Elem<TY>::kBytes, g, (int)(a.d - at));
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
      auto in = load_input<TY, KIND>(a, t, p, (int)n);
      settle_input<TY, KIND>(in, p, (int)n);
      input_values<TY, KIND>(in, h);
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
      for (int i = 0; i < 8; ++i) o[i] = rstd * fmaf(-h[i], c1, g[i] * w[i] - c0);
      store8<TY>(out + 8 * (int64_t)p * Elem<TY>::kBytes, o, (int)(a.d - 8 * (int64_t)p));
    }
  }
}

// dw and db from the workgroups' partial rows: 64 columns a workgroup, the
// partial rows dealt to 16 waves, eight loads of a wave in flight, and the
// waves' sums added up through LDS.
__global__ __launch_bounds__(1024) void norm_sum_kernel(NormGradArgs a) {
  __shared__ float col[16][64];
  const int which = blockIdx.y;
  const int64_t c = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
  const int w = threadIdx.x >> 6;
  float v = 0.f;
  if (c < a.d) {
    const float* p = a.part + (int64_t)which * a.d + c;
    for (int b = w; b < a.blocks; b += 128) {
      float q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = b + 16 * j < a.blocks ? p[(int64_t)(b + 16 * j) * 2 * a.d] : 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) v += q[j];
    }
  }
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
hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st) {
  pick_type(a.type, [&](auto ty) {
    constexpr int TY = decltype(ty)::value;
    auto with = [&](auto kind) {
      constexpr int KIND = decltype(kind)::value;
      auto launch = [&](auto r, auto k) {
        constexpr int R = decltype(r)::value, K = decltype(k)::value;
        const int64_t rows = (a.T + RowTeam<R>::kRows - 1) / RowTeam<R>::kRows;
        hipLaunchKernelGGL((norm_fwd_kernel<TY, KIND, R, K>), dim3((unsigned)std::min<int64_t>(rows, kNormBlocks)),
                           dim3(RowTeam<R>::kThreads), 0, st, a);
      };
      // by the width alone, so that a row's bits do not hang on how many rows there are
      const bool held = pick_shape<Shape<64, 1>, Shape<256, 1>, Shape<512, 1>, Shape<1024, 1>, Shape<1024, 2>>(
          a.d, launch);
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

int norm_grad_blocks(int64_t T, int64_t d) {
  const int64_t rows = d <= 512 ? 4 : 1;  // of a workgroup
  return (int)std::min<int64_t>(std::max<int64_t>((T + rows - 1) / rows, 1), d <= kRowMost ? 512 : 256);
}

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)a.blocks);
  pick_type(a.type, [&](auto ty) {
    constexpr int TY = decltype(ty)::value;
    auto with = [&](auto kind) {
      constexpr int KIND = decltype(kind)::value;
      const bool held = pick_shape<Shape<64, 1>, Shape<256, 1>, Shape<512, 1>, Shape<1024, 1>, Shape<1024, 2>>(
          a.d, [&](auto r, auto k) {
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
