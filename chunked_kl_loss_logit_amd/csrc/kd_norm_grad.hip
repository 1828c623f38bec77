// The gradients of layer norm.
//
//   h = (x - mean) r, g = grad w
//   dx = r (g - sum g / d - h sum (g h) / d), dw = sum_t grad h, db = sum_t grad
//
// Bound by memory: grad, x and dx once.  A row stays in its threads' registers
// as it was loaded, and the next one is loaded while it is worked on.  The sums
// over rows for dw and db stay in the registers of the threads that own those
// columns; each workgroup leaves one partial row of each, which a second
// kernel adds up in a fixed order.  16384 x 4096 bf16: 77 us (403 MB, 5.2 TB/s;
// a large copy reaches 5.1) and 5 us for the sums; 8192 x 8192 from 8 bits 76-79.
#include <type_traits>

#include "kd_launch.h"
#include "kd_layers.h"
#include "kd_row.h"

// Products and sums are fused where fmaf says so and nowhere else: what a call
// computes does not hang on what else its kernel has to do.
#pragma clang fp contract(off)

namespace kd {

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
template <int TY, int KIND, bool WHOLE>
__device__ inline Input<TY, KIND> load_input(const NormGradArgs& a, int64_t t, int p, int n) {
  Input<TY, KIND> r;
  const int64_t at = t * a.d + 8 * (int64_t)p;
  if constexpr (KIND == kRowsNone) {
    r.x = load8<TY, WHOLE>(a.x + at * Elem<TY>::kBytes, n, p > 0);
  } else {
    r.q = load_q8<WHOLE>(a.q + at, n, p > 0);
    r.scale = n > 0 ? a.scale[t * a.groups + (a.groups == 1 ? 0 : 8 * p / a.group)] : 0.f;
  }
  return r;
}
template <int TY, int KIND, bool WHOLE>
__device__ inline void settle_input(Input<TY, KIND>& r, int p, int n) {
  if constexpr (KIND == kRowsNone) settle8<TY, WHOLE>(r.x, n, p > 0);
  else settle_q8<WHOLE>(r.q, n, p > 0);
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

template <int TY, int KIND, bool WHOLE, int R, int K>
__global__ __launch_bounds__(RowTeam<R>::kThreads, K > 1 && R == 64 ? 3 : 4) void norm_grad_kernel(NormGradArgs a) {
  using Team = RowTeam<R>;
  // Two pieces a thread: the weights are read again for each row, and with 16 waves to a row they come from LDS and
  // there are no registers for the next row.  7282 x 9216 bf16 with all of it in (spilled) registers 267 us, with the
  // weights from the cache 173, so 106.
  constexpr bool kAhead = K == 1 || R == 64, kLds = K > 1 && R > 64;
  __shared__ __attribute__((aligned(16))) float shared_w[kLds ? R * K * 8 : 4];
  static_assert(!Team::kJoint, "the loop below ends for each row by itself");
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
      if constexpr (kLds) shared_w[8 * (lane + k * R) + i] = w[k][i];
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
      xn[k] = load_input<TY, KIND, WHOLE>(a, row, p, n);
      gn[k] = load8<TY, WHOLE>(a.grad + (row * a.d + 8 * (int64_t)p) * Elem<TY>::kBytes, n, p > 0);
    }
  };
  if constexpr (kAhead) load(t);
  for (; t < a.T; t += step) {
    if constexpr (!kAhead) load(t);
    char* out = a.dx ? a.dx + t * a.d * Elem<TY>::kBytes : nullptr;
    const float m = mean, r = rstd;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int p = lane + k * R, n = (int)(a.d - 8 * (int64_t)p);
      xr[k] = xn[k];
      gr[k] = gn[k];
      settle_input<TY, KIND, WHOLE>(xr[k], p, n);
      settle8<TY, WHOLE>(gr[k], n, p > 0);
    }
    if constexpr (kAhead) load(t + step);  // the next row, while this one is worked on
    auto weights = [&](int k) {
      if constexpr (kLds) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[k][i] = shared_w[8 * (lane + k * R) + i];  // this thread's own
      } else if constexpr (K > 1) {
        if (a.w) load_any(a.w, a.wtype, a.d, lane + k * R, w[k]);
      }
    };
    // a piece's h and g from what lies in registers as it was loaded
    auto values = [&](int k, float (&h)[8], float (&g)[8]) {
      const int64_t n = a.d - 8 * (int64_t)(lane + k * R);
      input_values<TY, KIND>(xr[k], h);
      unpack8<TY>(gr[k], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = (WHOLE ? n > 0 : i < n) ? (h[i] - m) * r : 0.f;
    };
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float h[8], g[8];
      values(k, h, g);
      weights(k);
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
      weights(k);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = r * fmaf(-h[i], c1, g[i] * w[k][i] - c0);
      store8<TY, WHOLE>(out + at * Elem<TY>::kBytes, g, (int)(a.d - at));
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
      auto in = load_input<TY, KIND, false>(a, t, p, (int)n);
      settle_input<TY, KIND, false>(in, p, (int)n);
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

namespace {
// A masked row's dx comes out of the kernel above as 0, since its grad counts as
// 0, unless a weight is not finite: then the masked rows are cleared here.
// (With the mask looked at for each row in that kernel, it took up to a tenth longer: 32768 x 1024 bf16 46 -> 49 us.)
__device__ inline void clear_masked(const NormGradArgs& a) {
  const int pieces = (int)((a.d + 7) / 8);
  uint32_t top = 0;
  for (int p = threadIdx.x; p < pieces; p += 1024) {
    float w[8];
    load_any(a.w, a.wtype, a.d, p, w);
    top = max(top, top8(w));
  }
  if (!__syncthreads_or(top >= 0x7f800000u)) return;
  const int bytes = a.type == kTypeF32 ? 4 : 2;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    if (row_valid(a.mask, t)) continue;
    uint16_t* row = reinterpret_cast<uint16_t*>(a.dx + t * a.d * bytes);
    for (int64_t i = threadIdx.x; i < a.d * bytes / 2; i += 1024) row[i] = 0;
  }
}
}  // namespace

// dw and db from the workgroups' partial rows: 64 columns a workgroup, the
// partial rows dealt to 16 waves, eight loads of a wave in flight, and the
// waves' sums added up through LDS.  first + blockIdx.y: dw, db, the masked rows.
template <bool MASKED>
__global__ __launch_bounds__(1024) void norm_sum_kernel(NormGradArgs a, int first) {
  __shared__ float col[16][64];
  const int which = first + blockIdx.y;
  if (MASKED && which == 2) return clear_masked(a);
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
int norm_grad_blocks(int64_t T, int64_t d) {
  const int64_t rows = d <= 128 ? 16 : d <= 256 ? 8 : d <= 1024 ? 4 : 1;  // of a workgroup
  return (int)std::min<int64_t>(std::max<int64_t>((T + rows - 1) / rows, 1), d <= kRowMost ? 512 : 256);
}

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)a.blocks);
  pick_type(a.type, [&](auto ty) {
    constexpr int TY = decltype(ty)::value;
    auto with = [&](auto kind) {
      constexpr int KIND = decltype(kind)::value;
      const bool held = pick_shape<Shape<16, 1>, Shape<32, 1>, Shape<64, 1>, Shape<64, 2>, Shape<256, 1>, Shape<512, 1>,
                                   Shape<1024, 1>, Shape<1024, 2>>(a.d, [&](auto r, auto k) {
        constexpr int R = decltype(r)::value, K = decltype(k)::value;
        const dim3 block(RowTeam<R>::kThreads);
        if (a.d % 8 == 0) hipLaunchKernelGGL((norm_grad_kernel<TY, KIND, true, R, K>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((norm_grad_kernel<TY, KIND, false, R, K>), grid, block, 0, st, a);
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
  const bool sums = a.dw || a.db, masked = a.dx && a.w && a.mask && a.d <= kRowMost;
  if (!sums && !masked) return hipSuccess;
  const dim3 grid((unsigned)((a.d + 63) / 64), 2 * sums + masked);
  if (masked) hipLaunchKernelGGL((norm_sum_kernel<true>), grid, dim3(1024), 0, st, a, sums ? 0 : 2);
  else hipLaunchKernelGGL((norm_sum_kernel<false>), grid, dim3(1024), 0, st, a, 0);
  return hipGetLastError();
}

}  // namespace kd
