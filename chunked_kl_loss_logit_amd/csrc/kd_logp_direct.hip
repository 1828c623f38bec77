// Token log-probabilities, dZ, dH and dW on the register-fed tiles of
// kd_direct.h: float32 (d and V multiples of 4), and bf16 (of 8) where the 256 x
// 256 ring tiles of kd_logp.hip would leave most of the chip idle or do not
// apply: d not a multiple of 32, V < 256, a head of 4 GiB or more.
//
//   forward  a = W (128 columns), b = H rows      z = W^T H^T, then each row's (m, l, e, x) record per tile
//   dZ       the same product; each row becomes its dZ (row-major)
//   dH       a = W rows (128 of d), b = dZ rows   contraction over the vocabulary
//   dW       a = dZ (128 columns), b = H columns  contraction over the rows
//
// The mathematics is that of kd_logp.hip.  Bounds: a few rows, the read of W
// (each workgroup streams its columns once, 16 KB a wave in flight); many
// rows, float32, the matrix cores (64 instructions of 64 cycles per 64 KB of
// operands).  Measured: forward of 7 rows of 2048 x 32000 bf16 22 us (6.0 TB/s
// of W, half of it from the last-level cache), its dW 34 us (3.9 TB/s written);
// 700 rows of 1024 x 32000 float32, of the 152 TFLOP/s that a large product
// reaches: forward with kept logits 458 us (100 TFLOP/s), dH 427 (107), dW 373
// (123); dZ from the logits 34 us (5.3 TB/s).
#include <type_traits>

#include "kd_direct.h"
#include "kd_policy.h"

namespace kd {

namespace {

constexpr int kDirThreads = 256;

__device__ inline long chunk_rows_of(const RowSet& rs) {
  return rs.rows ? min((long)rs.C, (long)*rs.count - (long)rs.c0) : min((long)rs.C, (long)(rs.T - rs.c0));
}
// The valid rows' blocks of `rows` rows: how many, and this workgroup's place
// among those blocks times `per`, or -1.  Workgroups without work are the last
// of the grid (rows may be masked), so that those with work go round the chip
// evenly: with one row block of four in use by its place in the grid, 33 rows
// of 2048 x 32000 float32 took 250 us, and 75 when it was one of one.
__device__ inline int row_blocks(long M, int rows, int per, int& nrb) {
  nrb = M > 0 ? (int)((M + rows - 1) / rows) : 0;
  const int total = nrb * per;
  return (int)blockIdx.x < total ? xcd_remap(blockIdx.x, total) : -1;
}
__device__ inline long row_at(const RowSet& rs, long i) { return rs.rows ? rs.rows[rs.c0 + i] : rs.c0 + i; }

// over the eight lanes of a row
__device__ inline float row_max(float v) {
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
__device__ inline float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ inline float at4(const float4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

template <int R>
__device__ inline void zero(f32x16_t (&acc)[4][R]) {
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < R; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;
}

// The product of W's columns [n0, n0 + 128) and the chunk's rows [r0, r0 + 32 R),
// the contraction split over the four waves.
template <class E, int R>
__device__ __forceinline__ void logits_tile(const LogpDirectArgs& a, long M, long r0, int n0, f32x16_t (&acc)[4][R]) {
  constexpr int U = 2;
  const int lane = threadIdx.x & 63, m = lane & 31;
  ColsN<E, U> wl;
  // a lane past the last column reads the last four: its results are left out
  wl.init(a.W, a.V * E::kElem, (int)a.d, min(n0 + 4 * m, (int)a.V - 4));
  RowsK<E, R, U> hl;
  hl.K = (int)a.d;
#pragma unroll
  for (int b = 0; b < R; ++b) hl.row(b, a.H + row_at(a.rs, min(r0 + 32 * b + m, M - 1)) * a.d * E::kElem);
  int kb, ke;
  k_range((int)a.d, kDirStep<E, U>, wave_id(), 4, kb, ke);
  zero(acc);
  direct_contract<E, U>(wl, hl, kb, ke, acc);
}

}  // namespace

// A row block of up to 32 R rows: f with as many block columns (1, 2 or 4) as
// its rows fill, so that a short last block costs what its rows do (700 rows
// of a 1024 x 32000 float32 head: forward 525 us without, 468 with).
template <int R, class F>
__device__ __forceinline__ void by_left(long left, F&& f) {
  if constexpr (R > 1) {
    if (left <= 16 * R) {
      by_left<R / 2>(left, f);
      return;
    }
  }
  f(std::integral_constant<int, R>());
}

// ------------------------------------------------------------------ forward
template <class E, int R, bool kEnt>
__device__ __forceinline__ void fwd_tile(const LogpDirectArgs& a, long M, long r0, int tile, float* reg) {
  const int n0 = tile * kDirA;
  const int V = (int)a.V, lane = threadIdx.x & 63;
  const int mine = 8 * wave_id() + (lane >> 3);  // the row of each block this lane will get
  int label[R];  // relative to the tile
#pragma unroll
  for (int b = 0; b < R; ++b) {
    const long i = r0 + 32 * b + mine;
    label[b] = i < M ? (int)((long)a.tokens[row_at(a.rs, i)] - a.v0 - n0) : -1;
  }
  f32x16_t acc[4][R];
  logits_tile<E, R>(a, M, r0, n0, acc);
  float4* part = reinterpret_cast<float4*>(a.part) + (long)tile * a.rs.C + r0;
  const int cols = min(kDirA, V - n0);  // a multiple of 4
  direct_rows<ColsN<E, 2>, R, 4, false>(acc, reg, [&](int b, int m, int q, const float4 (&z)[4]) {
    const int i = 32 * b + m;
    if (a.z && r0 + i < M) {
      float* zr = a.z + (r0 + i) * a.ldz + n0 + 4 * q;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (4 * q + 32 * j < cols) *reinterpret_cast<float4*>(zr + 32 * j) = z[j];
    }
    float mx = -INFINITY, x = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (4 * q + 32 * j >= cols) continue;
      mx = fmaxf(mx, fmaxf(fmaxf(z[j].x, z[j].y), fmaxf(z[j].z, z[j].w)));
      if ((label[b] >> 2) == q + 8 * j) x = at4(z[j], label[b] & 3);
    }
    mx = top_of(row_max(mx), a.c2);
    const float from = subtrahend(mx);
    float l = 0.f, e = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (4 * q + 32 * j >= cols) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float w = fmaf(at4(z[j], k), a.c2, -from), p = fast_exp2(w);
        l += p;
        if constexpr (kEnt) e = fmaf(p, at_least(w), e);
      }
    }
    l = row_sum(l);
    if constexpr (kEnt) e = row_sum(e);
    x = row_sum(x);
    if (q == 0 && r0 + i < M) part[i] = make_float4(mx, l, e, x);
  });
}

template <class E, int R, bool kEnt>
__global__ __launch_bounds__(kDirThreads, R == 4 ? 1 : 2) void logp_direct_fwd_kernel(LogpDirectArgs a) {
  __shared__ __attribute__((aligned(16))) float reg[4 * kDirRegion];
  const long M = chunk_rows_of(a.rs);
  int nrb;
  const int id = row_blocks(M, 32 * R, (int)((a.V + kDirA - 1) / kDirA), nrb);
  if (id < 0) return;
  const long r0 = (long)(id % nrb) * 32 * R;  // row blocks of one W panel run together on one XCD
  by_left<R>(M - r0, [&](auto r) { fwd_tile<E, decltype(r)::value, kEnt>(a, M, r0, id / nrb, reg); });
}

// ------------------------------------------------------------------ dZ
namespace {

// -q (A + B log2 q), and ga more at the token
template <bool kEnt>
__device__ inline float dz_of(float z, float c2, float L2, float A, float B) {
  const float lq = fmaf(z, c2, -L2), q = fast_exp2(lq);
  if constexpr (kEnt) return -q * fmaf(B, at_least(lq), A);
  return -q * A;
}

struct DzConst {
  float L2, A, B, ga;
  int label;
};
__device__ inline DzConst dz_const(const LogpDirectArgs& a, bool rv, long t) {
  DzConst k{0.f, 0.f, 0.f, 0.f, -1};
  if (!rv) return k;
  k.ga = a.g ? a.g[t] * a.inv_tau : 0.f;
  const float gb = a.ge ? a.ge[t] * a.inv_tau : 0.f;
  k.L2 = a.lse[t] * kLog2e;
  k.A = a.ge ? fmaf(gb, a.ent[t], k.ga) : k.ga;
  k.B = gb * kLn2;
  k.label = (int)((long)a.tokens[t] - a.v0);
  return k;
}

// the four columns from c
template <bool kEnt>
__device__ inline float4 dz_four(float4 z, const DzConst& k, float c2, long c) {
  return make_float4(dz_of<kEnt>(z.x, c2, k.L2, k.A, k.B) + (k.label == c ? k.ga : 0.f),
                     dz_of<kEnt>(z.y, c2, k.L2, k.A, k.B) + (k.label == c + 1 ? k.ga : 0.f),
                     dz_of<kEnt>(z.z, c2, k.L2, k.A, k.B) + (k.label == c + 2 ? k.ga : 0.f),
                     dz_of<kEnt>(z.w, c2, k.L2, k.A, k.B) + (k.label == c + 3 ? k.ga : 0.f));
}

// What rounding to bf16 leaves of x (0 of what is not finite).
__device__ inline float rest(float x) {
  const float r = x - __uint_as_float(Bf16::pack2(x, 0.f) << 16);
  return fabsf(r) < INFINITY ? r : 0.f;
}

template <class E>
__device__ inline void store4(char* p, float4 x) {
  if constexpr (E::kElem == 2)
    *reinterpret_cast<uint2*>(p) = make_uint2(Bf16::pack2(x.x, x.y), Bf16::pack2(x.z, x.w));
  else
    *reinterpret_cast<float4*>(p) = x;
}

// A row's x of direct_rows<.., E::kElem == 2, ..>, to the columns from p on, `cols` of them there
template <class E>
__device__ inline void put_row(char* p, int q, int cols, const float4 (&x)[4]) {
  if constexpr (E::kElem == 2) {
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const int c = quad_at<true>(q, j);
      if (c < cols)
        *reinterpret_cast<uint4*>(p + 2 * c) =
            make_uint4(Bf16::pack2(x[j].x, x[j].y), Bf16::pack2(x[j].z, x[j].w), Bf16::pack2(x[j + 1].x, x[j + 1].y),
                       Bf16::pack2(x[j + 1].z, x[j + 1].w));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = quad_at<false>(q, j);
      if (c < cols) *reinterpret_cast<float4*>(p + 4 * c) = x[j];
    }
  }
}
__device__ inline float4 rest4(float4 x) { return make_float4(rest(x.x), rest(x.y), rest(x.z), rest(x.w)); }

}  // namespace

template <class E, int R, bool kEnt>
__device__ __forceinline__ void dz_tile(const LogpDirectArgs& a, long M, long r0, int n0, float* reg) {
  const int V = (int)a.V, lane = threadIdx.x & 63, mine = 8 * wave_id() + (lane >> 3);
  DzConst k[R];
#pragma unroll
  for (int b = 0; b < R; ++b) {
    const long i = r0 + 32 * b + mine;
    k[b] = dz_const(a, i < M, i < M ? row_at(a.rs, i) : 0);
  }
  f32x16_t acc[4][R];
  logits_tile<E, R>(a, M, r0, n0, acc);
  constexpr bool kPairs = E::kElem == 2;
  direct_rows<ColsN<E, 2>, R, 4, kPairs>(acc, reg, [&](int b, int m, int q, const float4 (&z)[4]) {
    const long i = r0 + 32 * b + m;
    float4 o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = i < M ? dz_four<kEnt>(z[j], k[b], a.c2, n0 + quad_at<kPairs>(q, j)) : make_float4(0.f, 0.f, 0.f, 0.f);
    char* p = a.dz + (i * a.ldz + n0) * E::kElem;
    put_row<E>(p, q, V - n0, o);
    if (kPairs && a.lo) {  // what the rounding left
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = rest4(o[j]);
      put_row<E>(p + a.lo, q, V - n0, o);
    }
  });
}

template <class E, int R, bool kEnt>
__global__ __launch_bounds__(kDirThreads, R == 1 ? 2 : 1) void logp_direct_dz_kernel(LogpDirectArgs a) {
  __shared__ __attribute__((aligned(16))) float reg[4 * kDirRegion];
  const long M = chunk_rows_of(a.rs);
  int nrb;
  const int id = row_blocks(M, 32 * R, (int)((a.V + kDirA - 1) / kDirA), nrb);
  if (id < 0) return;
  const long r0 = (long)(id % nrb) * 32 * R;
  by_left<R>(M - r0, [&](auto r) { dz_tile<E, decltype(r)::value, kEnt>(a, M, r0, id / nrb * kDirA, reg); });
}

// From stored logits: a block takes one row and up to kFzCols columns, eight per thread.
constexpr int kFzCols = 2048;
template <class E, bool kEnt>
__global__ __launch_bounds__(256) void logp_direct_dz_from_z_kernel(LogpDirectArgs a) {
  const long M = chunk_rows_of(a.rs);
  const long per = (a.V + kFzCols - 1) / kFzCols, i = blockIdx.x / per;
  if (i >= (M + 31) / 32 * 32) return;
  const DzConst k = dz_const(a, i < M, i < M ? row_at(a.rs, i) : 0);
  const long c0 = (long)(blockIdx.x - i * per) * kFzCols + threadIdx.x * 4;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const long c = c0 + q * (kFzCols / 2);
    if (c >= a.V) break;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < M) o = dz_four<kEnt>(*reinterpret_cast<const float4*>(a.z + i * a.ldz + c), k, a.c2, c);
    char* p = a.dz + (i * a.ldz + c) * E::kElem;
    store4<E>(p, o);
    if (E::kElem == 2 && a.lo) store4<E>(p + a.lo, rest4(o));
  }
}

// ------------------------------------------------------------------ dH
// How the grid is divided among the row blocks there are: as many vocabulary
// ranges as it has room for, at least 1 KB of W's rows each.  A range's part
// holds the row blocks' rows.  (700 valid rows of 777, 1024 x 32000 float32:
// dH from logits 495 us with as many ranges as suit 777 rows, 464 so; 1024 rows,
// half of them masked, of 2048 x 8192 259 and 151.)
struct DirectDh {
  int nrb, S;
  long rows;  // of a part
};
__device__ inline DirectDh direct_dh(long M, int rows, int nda, int grid, int smax) {
  const int nrb = M > 0 ? (int)((M + rows - 1) / rows) : 0;
  return {nrb, max(1, min(nrb > 0 ? grid / (nrb * nda) : 1, smax)), (long)nrb * rows};
}

// Tile: 128 of d x 32 R rows, vocabulary range s of S over the four waves.
// S = 1: dH itself; else the range's float32 part [S][rows][d].  kTwo: 32 rows,
// the second block column their rests, added at the end.
template <class E, int R, class O, bool kTwo = false>
__global__ __launch_bounds__(kDirThreads, 1) void logp_direct_dh_kernel(LogpDirectArgs a, int nda, int smax,
                                                                        float* part, char* dH) {
  constexpr int U = 4;
  __shared__ __attribute__((aligned(16))) float reg[4 * kDirRegion];
  const long M = chunk_rows_of(a.rs);
  constexpr int kRows = kTwo ? 32 : 32 * R;
  const DirectDh sh = direct_dh(M, kRows, nda, gridDim.x, smax);
  int nrb;
  int id = row_blocks(M, kRows, nda * sh.S, nrb);
  if (id < 0) return;
  const long r0 = (long)(id % nrb) * kRows;
  id /= nrb;
  const int d0 = (id % nda) * kDirA, s = id / nda;
  const int lane = threadIdx.x & 63, m = lane & 31, d = (int)a.d;
  RowsK<E, 4, U> wl;
  RowsK<E, R, U> zl;
  wl.K = zl.K = (int)a.V;
#pragma unroll
  for (int f = 0; f < 4; ++f) wl.row(f, a.W + (long)min(d0 + 32 * f + m, d - 1) * a.V * E::kElem);
#pragma unroll
  for (int b = 0; b < R; ++b)
    zl.row(b, a.dz + min(r0 + (kTwo ? m : 32 * b + m), M - 1) * a.ldz * E::kElem + (kTwo && b ? a.lo : 0));
  int kb, ke;
  k_range((int)a.V, kDirStep<E, U>, 4 * s + wave_id(), 4 * sh.S, kb, ke);
  f32x16_t acc[4][R];
  zero(acc);
  direct_contract<E, U>(wl, zl, kb, ke, acc);
  float4 first[4];
  direct_rows<RowsK<E, 4, U>, R, 4, false>(acc, reg, [&](int b, int mm, int q, float4 (&x)[4]) {
    const long i = r0 + (kTwo ? mm : 32 * b + mm);
    if constexpr (kTwo) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (b == 0)
          first[j] = x[j];
        else
          x[j] = make_float4(first[j].x + x[j].x, first[j].y + x[j].y, first[j].z + x[j].z, first[j].w + x[j].w);
      }
      if (b == 0) return;
    }
    if (i >= M) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = d0 + 4 * q + 32 * j;
      if (c >= d) break;
      if (sh.S > 1)
        *reinterpret_cast<float4*>(part + ((long)s * sh.rows + i) * d + c) = x[j];
      else
        store4<O>(dH + (row_at(a.rs, i) * d + c) * O::kElem, x[j]);
    }
  });
}

// dH of a row = its parts in order, four elements per thread
template <class O>
__global__ __launch_bounds__(256) void logp_direct_reduce_kernel(RowSet rs, const float* part, int rows, int nda,
                                                                 int grid, int smax, long d, char* dH) {
  const long q = (long)blockIdx.x * 256 + threadIdx.x, d4 = d / 4;
  const long i = q / d4, j = (q - i * d4) * 4, M = chunk_rows_of(rs);
  if (i >= M) return;
  const DirectDh sh = direct_dh(M, rows, nda, grid, smax);
  if (sh.S == 1) return;  // there already
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < sh.S; ++s) {
    const float4 y = *reinterpret_cast<const float4*>(part + ((long)s * sh.rows + i) * d + j);
    x.x += y.x;
    x.y += y.y;
    x.z += y.z;
    x.w += y.w;
  }
  store4<O>(dH + (row_at(rs, i) * d + j) * O::kElem, x);
}

// ------------------------------------------------------------------ dW
// Tiles of 128 columns of V x 32 F of d.  KS = 4: the rows split over the four
// waves; KS = 1: four tiles side by side in d, all rows each.  F = 2 leaves
// room for a second workgroup on the CU, for few rows, where a tile is little
// more than its stores.
template <class E, int KS, class O, int F>
__global__ __launch_bounds__(kDirThreads, F == 2 ? 2 : 1) void logp_direct_dw_kernel(LogpDirectArgs a, const char* Hc,
                                                                                     int nda, const float* add,
                                                                                     char* out) {
  constexpr int U = E::kElem == 4 || F == 2 ? 1 : 2;  // two chunks would not leave room for the accumulators
  constexpr int kD = 32 * F;
  __shared__ __attribute__((aligned(16))) float reg[4 * kDirRegion];
  const long M = max(0L, chunk_rows_of(a.rs));
  const int id = xcd_remap(blockIdx.x, gridDim.x);
  const int w = wave_id(), lane = threadIdx.x & 63, m = lane & 31;
  const int d0 = ((id % nda) * (KS == 1 ? 4 : 1) + (KS == 1 ? w : 0)) * kD, n0 = id / nda * kDirA;
  const int d = (int)a.d, V = (int)a.V;
  ColsN<E, U> zl;
  ColsN<E, U, F> hl;
  zl.init(a.dz, a.ldz * E::kElem, (int)((M + 31) / 32 * 32), min(n0 + 4 * m, V - 4));  // zero rows behind the last
  hl.init(Hc, (long)d * E::kElem, (int)M, min(d0 + F * m, d - F));
  int kb, ke;
  k_range((int)M, kDirStep<E, U>, KS == 1 ? 0 : w, KS, kb, ke);
  f32x16_t acc[4][F];
  zero(acc);
  for (int plane = a.lo ? 2 : 1;;) {
    direct_contract<E, U>(zl, hl, kb, ke, acc);
    if (--plane == 0) break;
    zl.base += a.lo;
  }
  constexpr bool kPairs = O::kElem == 2;
  direct_rows<ColsN<E, U>, F, KS, kPairs>(acc, reg, [&](int b, int mm, int q, float4 (&x)[4]) {
    const int i = d0 + ColsN<E, U, F>::index(b, mm);
    if (i >= d) return;
    const long at = (long)i * V + n0;
    if (add) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = quad_at<kPairs>(q, j);
        if (n0 + c >= V) break;
        const float4 y = *reinterpret_cast<const float4*>(add + at + c);
        x[j] = make_float4(x[j].x + y.x, x[j].y + y.y, x[j].z + y.z, x[j].w + y.w);
      }
    }
    put_row<O>(out + at * O::kElem, q, V - n0, x);
  });
}

// ------------------------------------------------------------------ rows of the mask
// A block of 256 threads takes kPrepRows rows of the mask: how many valid ones
// come before them (counted anew by every block: at most T bytes), where each
// of its own goes, and the copying, a wave to a row: one launch where counting,
// packing and zeroing apart are three.
constexpr int kPrepRows = 16;

__device__ inline void copy_row(char* to, const char* from, long bytes) {
  for (long q = (threadIdx.x & 63) * 16; q < bytes; q += 1024)
    *reinterpret_cast<u32x4_t*>(to + q) = from ? ld16(from + q) : zero4();
}

__global__ __launch_bounds__(256) void logp_prep_kernel(const uint8_t* mask, long T, int32_t* rows, int32_t* count,
                                                        const char* H, long rowb, long C, char* Hc, char* dH,
                                                        long dhb) {
  __shared__ int red[4];
  __shared__ int pos[kPrepRows];  // compacted position, or -1
  const long t0 = (long)blockIdx.x * kPrepRows;
  int n = 0;
  for (long t = (long)threadIdx.x * 8; t < t0; t += 2048) {  // t0 is a multiple of 16: whole eights
    uint2 v;
    __builtin_memcpy(&v, mask + t, 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) n += ((v.x >> (8 * i) & 255u) != 0) + ((v.y >> (8 * i) & 255u) != 0);
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) n += __shfl_xor(n, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = n;
  __syncthreads();
  const int before = red[0] + red[1] + red[2] + red[3];
  if (threadIdx.x < 64) {
    const long t = t0 + threadIdx.x;
    const bool on = threadIdx.x < kPrepRows && t < T && mask[t] != 0;
    const unsigned long long b = __ballot(on);
    const int at = before + __popcll(b & ((1ull << threadIdx.x) - 1));
    if (threadIdx.x < kPrepRows) pos[threadIdx.x] = on ? at : -1;
    if (on) rows[at] = (int32_t)t;
    if (t0 + kPrepRows >= T && threadIdx.x == 0) *count = before + __popcll(b);
  }
  __syncthreads();
  for (int r = threadIdx.x >> 6; r < kPrepRows; r += 4) {
    const long t = t0 + r;
    if (t >= T) break;
    const int at = pos[r];
    if (at < 0) {
      if (dH) copy_row(dH + t * dhb, nullptr, dhb);
    } else if (Hc && at < C) {
      copy_row(Hc + at * rowb, H + t * rowb, rowb);
    }
  }
}

// The chunk's rows of H one after the other, a wave to a row
__global__ __launch_bounds__(256) void logp_pack_kernel(RowSet rs, const char* H, long rowb, char* Hc) {
  const long i = (long)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (i < chunk_rows_of(rs)) copy_row(Hc + i * rowb, H + row_at(rs, i) * rowb, rowb);
}

hipError_t launch_logp_prep(const uint8_t* mask, int64_t T, int32_t* rows, int32_t* count, const void* H,
                            int64_t row_bytes, int64_t C, void* Hc, void* dH, int64_t dh_row_bytes, hipStream_t st) {
  hipLaunchKernelGGL(logp_prep_kernel, dim3((unsigned)((T + kPrepRows - 1) / kPrepRows)), dim3(256), 0, st, mask,
                     (long)T, rows, count, static_cast<const char*>(H), (long)row_bytes, (long)C,
                     static_cast<char*>(Hc), static_cast<char*>(dH), (long)dh_row_bytes);
  return hipGetLastError();
}

hipError_t launch_logp_pack(const RowSet& rs, const void* H, int64_t row_bytes, void* Hc, hipStream_t st) {
  const int64_t n = rs.C < rs.T - rs.c0 ? rs.C : rs.T - rs.c0;
  hipLaunchKernelGGL(logp_pack_kernel, dim3((unsigned)((n + 3) / 4)), dim3(256), 0, st, rs,
                     static_cast<const char*>(H), (long)row_bytes, static_cast<char*>(Hc));
  return hipGetLastError();
}

// ------------------------------------------------------------------ launches
namespace {

int64_t rows_upto(const RowSet& rs) { return rs.C < rs.T - rs.c0 ? rs.C : rs.T - rs.c0; }
int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

template <class E, int R>
void fwd(const LogpDirectArgs& a, bool entropy, hipStream_t st) {
  const dim3 grid((unsigned)(cdiv(rows_upto(a.rs), 32 * R) * cdiv(a.V, kDirA)));
  if (entropy)
    hipLaunchKernelGGL((logp_direct_fwd_kernel<E, R, true>), grid, dim3(kDirThreads), 0, st, a);
  else
    hipLaunchKernelGGL((logp_direct_fwd_kernel<E, R, false>), grid, dim3(kDirThreads), 0, st, a);
}
template <class E, int R>
void dz(const LogpDirectArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(cdiv(rows_upto(a.rs), 32 * R) * cdiv(a.V, kDirA)));
  if (a.ge)
    hipLaunchKernelGGL((logp_direct_dz_kernel<E, R, true>), grid, dim3(kDirThreads), 0, st, a);
  else
    hipLaunchKernelGGL((logp_direct_dz_kernel<E, R, false>), grid, dim3(kDirThreads), 0, st, a);
}
// Block columns of rows per tile: 1, 2 or 4, no more than hold the rows, and
// fewer where the tiles would not go round the CUs (at 4 a tile's operands are
// used best; forward of float32, us, 1 / 4: 128 rows of 4096 x 4096 73 / 246, of
// 1024 x 32000 123 / 78).
template <class F>
void by_rows(int64_t n, int64_t V, F&& f) {
  const int64_t cols = cdiv(V, kDirA);
  if (n > 64 && cdiv(n, 128) * cols >= 200) f(std::integral_constant<int, 4>());
  else if (n > 32 && cdiv(n, 64) * cols >= 200) f(std::integral_constant<int, 2>());
  else f(std::integral_constant<int, 1>());
}

}  // namespace

hipError_t launch_logp_direct_fwd(int elem, const LogpDirectArgs& a, bool entropy, hipStream_t st) {
  by_rows(rows_upto(a.rs), a.V, [&](auto r) {
    if (elem == 2) fwd<Bf16, decltype(r)::value>(a, entropy, st);
    else fwd<F32, decltype(r)::value>(a, entropy, st);
  });
  return hipGetLastError();
}

hipError_t launch_logp_direct_dz(int elem, const LogpDirectArgs& a, hipStream_t st) {
  by_rows(rows_upto(a.rs), a.V, [&](auto r) {
    if (elem == 2) dz<Bf16, decltype(r)::value>(a, st);
    else dz<F32, decltype(r)::value>(a, st);
  });
  return hipGetLastError();
}

hipError_t launch_logp_direct_dz_from_z(int elem, const LogpDirectArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)cdiv(a.V, kFzCols) * cdiv(rows_upto(a.rs), 32) * 32));
  if (elem == 2 && a.ge)
    hipLaunchKernelGGL((logp_direct_dz_from_z_kernel<Bf16, true>), grid, dim3(256), 0, st, a);
  else if (elem == 2)
    hipLaunchKernelGGL((logp_direct_dz_from_z_kernel<Bf16, false>), grid, dim3(256), 0, st, a);
  else if (a.ge)
    hipLaunchKernelGGL((logp_direct_dz_from_z_kernel<F32, true>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((logp_direct_dz_from_z_kernel<F32, false>), grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_logp_direct_dh(int elem, const LogpDirectArgs& a, int g, float* part, void* dH, int dh_elem,
                                 hipStream_t st) {
  const int64_t n = rows_upto(a.rs);
  const int nda = cdiv(a.d, kDirA), smax = cdiv(a.V * elem, 1024), rows = direct_dh_rows(n);
  const dim3 grid((unsigned)g), block(kDirThreads);
  char* out = static_cast<char*>(dH);
  auto go = [&](auto r) {
    constexpr int R = decltype(r)::value;
    if (elem == 4)
      hipLaunchKernelGGL((logp_direct_dh_kernel<F32, R, F32>), grid, block, 0, st, a, nda, smax, part, out);
    else if (dh_elem == 4)
      hipLaunchKernelGGL((logp_direct_dh_kernel<Bf16, R, F32>), grid, block, 0, st, a, nda, smax, part, out);
    else
      hipLaunchKernelGGL((logp_direct_dh_kernel<Bf16, R, Bf16>), grid, block, 0, st, a, nda, smax, part, out);
  };
  if (a.lo && dh_elem == 4)
    hipLaunchKernelGGL((logp_direct_dh_kernel<Bf16, 2, F32, true>), grid, block, 0, st, a, nda, smax, part, out);
  else if (a.lo)
    hipLaunchKernelGGL((logp_direct_dh_kernel<Bf16, 2, Bf16, true>), grid, block, 0, st, a, nda, smax, part, out);
  else if (rows == 32)
    go(std::integral_constant<int, 1>());
  else
    go(std::integral_constant<int, 2>());
  const dim3 rgrid((unsigned)cdiv(n * (a.d / 4), 256));
  if (dh_elem == 2)
    hipLaunchKernelGGL(logp_direct_reduce_kernel<Bf16>, rgrid, dim3(256), 0, st, a.rs, part, rows, nda, g, smax,
                       (long)a.d, out);
  else
    hipLaunchKernelGGL(logp_direct_reduce_kernel<F32>, rgrid, dim3(256), 0, st, a.rs, part, rows, nda, g, smax,
                       (long)a.d, out);
  return hipGetLastError();
}

hipError_t launch_logp_direct_dw(int elem, const LogpDirectArgs& a, const void* Hc, const float* add32, void* out,
                                 int out_elem, hipStream_t st) {
  // Tiles 64 of d wide up to 64 rows (7 rows of 2048 x 32000 bf16, from logits,
  // 41 us, with tiles of 128 68; 64 rows 44 and 68); else four waves on a tile where there are
  // too few tiles for every wave to have its own.
  const int nv = cdiv(a.V, kDirA), nda = cdiv(a.d, kDirA);
  const bool few = rows_upto(a.rs) <= 64, split = !few && (int64_t)nda * nv < 1024;
  const int n4 = few ? cdiv(a.d, 256) : split ? nda : cdiv(nda, 4);
  const dim3 grid((unsigned)(n4 * nv)), block(kDirThreads);
  const char* h = static_cast<const char*>(Hc);
  char* o = static_cast<char*>(out);
  auto go = [&](auto ks, auto f) {
    constexpr int KS = decltype(ks)::value, F = decltype(f)::value;
    if (elem == 4)
      hipLaunchKernelGGL((logp_direct_dw_kernel<F32, KS, F32, F>), grid, block, 0, st, a, h, n4, add32, o);
    else if (out_elem == 4)
      hipLaunchKernelGGL((logp_direct_dw_kernel<Bf16, KS, F32, F>), grid, block, 0, st, a, h, n4, add32, o);
    else
      hipLaunchKernelGGL((logp_direct_dw_kernel<Bf16, KS, Bf16, F>), grid, block, 0, st, a, h, n4, add32, o);
  };
  using std::integral_constant;
  if (few) go(integral_constant<int, 1>(), integral_constant<int, 2>());
  else if (split) go(integral_constant<int, 4>(), integral_constant<int, 4>());
  else go(integral_constant<int, 1>(), integral_constant<int, 4>());
  return hipGetLastError();
}

}  // namespace kd
