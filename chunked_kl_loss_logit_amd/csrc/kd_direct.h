// Matrix-core tiles fed straight from global memory, without LDS staging.
//
// A wave computes 128 x 32 R outputs, acc[a][b] = sum over k of A(128 a-side
// indices) x B(32 R b-side indices), as 4 x R blocks of 32 x 32; a workgroup
// of four waves either splits one tile's contraction four ways (KS = 4,
// summed through LDS at the end) or holds four tiles (KS = 1).  This is for
// the shapes the 256 x 256 ring tiles leave most of the chip idle on (few
// rows, few columns: here the contraction is spread over four waves and tiles
// are an eighth of the size) and for float32, whose matrix instructions take
// 64 cycles for 4 K products, so that register-direct operands keep up.
//
// Operands, both types, any leading dimension whose rows are 16-byte aligned:
//   RowsK  k-contiguous rows: fragment f, lane l holds index 32 f + l % 32,
//          16-byte chunks of its row.
//   ColsN  n-contiguous (row k holds the indices): lane l holds the four
//          consecutive indices 4 (l % 32) .. + 3, one per fragment, one vector
//          load per k.  bf16 pairs of k are interleaved with v_perm.
// A step is 2 U chunks of k (a chunk: 8 bf16 or 4 float32); lane half h = l /
// 32 takes chunks [U h, U h + U) of both operands, which the matrix
// instruction adds up in whatever order, so each lane reads U chunks in a row.
// Steps are loaded one ahead.  Each operand has its own end of k: past it
// RowsK reads as zero and ColsN repeats its last row, so where both are ColsN
// one of them has to hold zeros up to whole steps.
//
// Afterwards block column b goes through LDS as [32 b-indices][128 a-indices]
// (stride 132 floats: four banks a row, so the 16-byte writes of a half-wave
// spread over all banks), and is read back eight lanes to a row, 16 bytes
// each: 128 contiguous bytes of float32 per row and store.
#pragma once

#include <type_traits>

#include "kd_gemm.h"

namespace kd {

constexpr int kDirA = 128;             // a-side indices of a tile
constexpr int kDirLd = 132;            // LDS row stride, floats
constexpr int kDirRegion = 32 * kDirLd;  // floats of one wave's region

template <class E, int U>
constexpr int kDirStep = 2 * U * E::kEpc;  // k per step

// load() reads a whole step without any condition, load_end() one that may
// reach past K, looking at each chunk or row.
template <class E, int F, int U>
struct RowsK {
  static constexpr bool kColumns = false;
  static constexpr int kFrags = F;
  const char* p[F];  // the lane's rows, at its half's first chunk
  int K;
  u32x4_t r[2][F][U];
  __device__ inline static int index(int f, int m) { return 32 * f + m; }  // of fragment f's row m
  // row: the lane's row of fragment f
  __device__ inline void row(int f, const char* at) { p[f] = at + ((threadIdx.x >> 5) & 1) * 16 * U; }
  __device__ inline void load(int buf, int k) {
    const long at = (long)k * E::kElem;
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int u = 0; u < U; ++u) r[buf][f][u] = ld16(p[f] + at + 16 * u);
  }
  __device__ inline void load_end(int buf, int k) {
    const long at = (long)k * E::kElem;
    const int h = (threadIdx.x >> 5) & 1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kk = k + (U * h + u) * E::kEpc;
      const long back = kk < K ? 0 : (long)(kk - (K - E::kEpc)) * E::kElem;  // to the row's last chunk
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const u32x4_t v = ld16(p[f] + at + 16 * u - back);
        r[buf][f][u] = kk < K ? v : zero4();
      }
    }
  }
  __device__ inline u32x4_t frag(int buf, int f, int u) const { return r[buf][f][u]; }
};

// F consecutive indices to a lane: 4, or 2 where the tile is narrower
template <class E, int U, int F = 4>
struct ColsN {
  static constexpr bool kColumns = true;
  static constexpr int kFrags = F;
  static constexpr int kRows = U * E::kEpc;  // k per half and step
  static constexpr int kWords = F * E::kElem / 4;
  struct __attribute__((aligned(4 * kWords))) Vec {
    uint32_t w[kWords];
  };
  const char* base;  // row 0, uniform
  uint32_t off;      // the lane's indices, in its half's first row
  uint32_t col;      // the lane's indices
  long ld;           // bytes, uniform; 16 rows of it below 4 GB
  int K;
  Vec r[2][kRows];
  __device__ inline static int index(int f, int m) { return F * m + f; }
  // n: the lane's first index (of F that exist)
  __device__ inline void init(const char* b, long ld_, int K_, int n) {
    base = b;
    ld = ld_;
    K = K_;
    col = (uint32_t)n * E::kElem;
    off = col + (uint32_t)(((threadIdx.x >> 5) & 1) * kRows * ld);
  }
  __device__ inline void load(int buf, int k) {
    const char* q = base + (long)k * ld;
#pragma unroll
    for (int s = 0; s < kRows; ++s) r[buf][s] = *reinterpret_cast<const Vec*>(q + s * ld + off);
  }
  __device__ inline void load_end(int buf, int k) {
    const int h = (threadIdx.x >> 5) & 1;
#pragma unroll
    for (int s = 0; s < kRows; ++s)
      r[buf][s] = *reinterpret_cast<const Vec*>(base + (long)max(0, min(k + kRows * h + s, K - 1)) * ld + col);
  }
  // chunk u of index f: 8 bf16 or 4 float32 along k
  __device__ inline u32x4_t frag(int buf, int f, int u) const {
    u32x4_t o;
    if constexpr (E::kElem == 2) {
      const uint32_t sel = f & 1 ? 0x07060302u : 0x05040100u;
#pragma unroll
      for (int w = 0; w < 4; ++w)
        o[w] = __builtin_amdgcn_perm(r[buf][8 * u + 2 * w + 1].w[f >> 1], r[buf][8 * u + 2 * w].w[f >> 1], sel);
    } else {
#pragma unroll
      for (int w = 0; w < 4; ++w) o[w] = r[buf][4 * u + w].w[f];
    }
    return o;
  }
};

// acc += A . B over k in [kb, ke): ke is kb plus whole steps, or the operands'
// end, behind which one of them is zero up to a whole step.
template <class E, int U, class A, class B>
__device__ __forceinline__ void direct_contract(A& a, B& b, int kb, int ke, f32x16_t (&acc)[4][B::kFrags]) {
  constexpr int KS = kDirStep<E, U>;
  auto mma = [&](int buf) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      u32x4_t fb[B::kFrags];
#pragma unroll
      for (int j = 0; j < B::kFrags; ++j) fb[j] = b.frag(buf, j, u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const u32x4_t fa = a.frag(buf, i, u);
#pragma unroll
        for (int j = 0; j < B::kFrags; ++j) E::mma(acc[i][j], fa, fb[j]);
      }
    }
  };
  // pairs of whole steps, the next step's loads out before this one's products
  // (the scheduler would otherwise sink them to their first use); the last
  // prefetch reads a step again, so that every turn has the same loads
  const int end = min(ke, min(a.K, b.K));
  int k = kb;
  if (k + 2 * KS <= end) {
    a.load(0, k);
    b.load(0, k);
    do {
      a.load(1, k + KS);
      b.load(1, k + KS);
      __builtin_amdgcn_sched_barrier(0);
      mma(0);
      __builtin_amdgcn_sched_barrier(0);
      const int next = k + 4 * KS <= end ? k + 2 * KS : k;
      a.load(0, next);
      b.load(0, next);
      __builtin_amdgcn_sched_barrier(0);
      mma(1);
      __builtin_amdgcn_sched_barrier(0);
      k += 2 * KS;
    } while (k + 2 * KS <= end);
  }
  for (; k < ke; k += KS) {  // what is left: up to a pair of steps, the last one short
    a.load_end(0, k);
    b.load_end(0, k);
    mma(0);
  }
}

// part `i` of `parts` of [0, K), in whole units of `unit` k
__device__ inline void k_range(int K, int unit, int i, int parts, int& kb, int& ke) {
  const long n = (K + unit - 1) / unit;
  kb = (int)(n * i / parts) * unit;
  ke = min((int)(n * (i + 1) / parts) * unit, K);
}

// Sums the KS waves' accumulators and hands the tile out: row(b, m, q, x) has
// the sums of b-index B::index(b, m) in x[0 .. 3], four a-indices each, from
// quad_at<kPairs>(q, 0 .. 3) on, with eight lanes (q = 0 .. 7) side by side on
// a row and m differing by lane.  kPairs: x[0], x[1] and x[2], x[3] are eight
// consecutive a-indices, 16 bytes of bf16 (put_row).
// KS = 1: every wave hands out its own tile.  A: the a-side operand's type.
// reg: LDS, 4 regions.
template <bool kPairs>
__device__ inline int quad_at(int q, int j) {
  return 4 * (kPairs ? 2 * q + (j & 1) + 16 * (j >> 1) : q + 8 * j);
}
template <class A, int R, int KS, bool kPairs, class Row>
__device__ __forceinline__ void direct_rows(const f32x16_t (&acc)[4][R], float* reg, Row&& row) {
  const int w = wave_id(), lane = threadIdx.x & 63, h = lane >> 5;
  float* mine = reg + w * kDirRegion + (lane & 31) * kDirLd;
#pragma unroll
  for (int b = 0; b < R; ++b) {
    if (b > 0) __syncthreads();  // the last block's rows have been read
    // register i of block a is a-row 8 (i / 4) + 4 h + i % 4
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      float4 v;
      int at;
      if constexpr (A::kColumns) {  // index 4 m + a: the four blocks' register q side by side
        v = make_float4(acc[0][b][q], acc[1][b][q], acc[2][b][q], acc[3][b][q]);
        at = 4 * (8 * (q >> 2) + 4 * h + (q & 3));
      } else {  // index 32 a + m: four registers of block q / 4 side by side
        const int a = q >> 2, i = 4 * (q & 3);
        v = make_float4(acc[a][b][i], acc[a][b][i + 1], acc[a][b][i + 2], acc[a][b][i + 3]);
        at = 32 * a + 8 * (q & 3) + 4 * h;
      }
      *reinterpret_cast<float4*>(mine + at) = v;
    }
    __syncthreads();
    // eight rows of the block per wave and turn
    for (int t = 0; t < (KS == 1 ? 4 : 1); ++t) {
      const int m = (KS == 1 ? 8 * t : 8 * w) + (lane >> 3), q = lane & 7;
      float4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 y = *reinterpret_cast<const float4*>(reg + (KS == 1 ? w : s) * kDirRegion + m * kDirLd +
                                                            quad_at<kPairs>(q, j));
          x[j].x += y.x;
          x[j].y += y.y;
          x[j].z += y.z;
          x[j].w += y.w;
        }
      row(b, m, q, x);
    }
  }
}

}  // namespace kd
