// Product of 8-bit integers with a scale for each token and channel:
//
//   out[t,v] = sx[t] sw[v] sum_k x[t,k] w[v,k]
//
// Sums are exact in 32-bit integers (d below 2^17), so a split of the
// contraction changes nothing.  Both operands are contiguous along k, in rows
// of bytes; one matrix instruction (32 x 32 x 32) takes 16 bytes a lane of
// each, as the 16-bit one takes 8 elements.
//
// Many rows: 256 x 256 tiles on the direct-to-LDS ring.  x goes through panels
// (kd_dma.h) padded with zeros to whole ring turns, which cancel whatever w's
// rows read past their end.  Few rows or few tiles: w is what has to be read;
// a workgroup takes 64 channels and up to 128 rows, each of its four waves a
// quarter of k, straight from global memory into registers.
#include <type_traits>

#include "kd_dma.h"
#include "kd_launch.h"
#include "kd_layers.h"
#include "kd_row.h"

namespace kd {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

__device__ inline void mma_i8(i32x16_t& acc, u32x4_t a, u32x4_t b) {
  acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), acc, 0, 0,
                                              0);
}

constexpr int kKTurn = kRing * kRowB;  // k of a ring turn

}  // namespace

// ------------------------------------------------------------------ x in panels
__global__ __launch_bounds__(256) void int8_panels_kernel(const char* x, long T, long d, long chunks, char* panels) {
  const long n = T * chunks;
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long)gridDim.x * 256) {
    // four 16-byte chunks of a 64-byte piece are neighbours, then rows, then pieces
    const long c = (i / (4 * T)) * 4 + (i & 3), t = (i >> 2) % T;
    const long byte = c * 16;
    *reinterpret_cast<u32x4_t*>(panels + panel_off(T, t, byte)) = byte < d ? ld16(x + t * d + byte) : zero4();
  }
}

// ------------------------------------------------------------------ tiles
namespace {

template <int NBI>
__device__ inline void stage_i32(const Slots& sl, const i32x16_t (&acc)[4][4]) {
  const int w = wave_id();
  const int lane = opaque((int)threadIdx.x) & 63;
  const StageOff so = stage_offsets(w >> 1, lane);
  float* st = (w & 1) ? st_pair<1>(sl) : st_pair<0>(sl);
#pragma unroll
  for (int mb = 0; mb < 4; ++mb) {
    i32x16_t v = acc[mb][NBI];
    asm volatile("" : "+a"(v));
#pragma unroll
    for (int i = 0; i < 16; ++i)
      st[so.o[((i & 3) >> 1) + 2 * ((i >> 2) & 1)] + mb * 1024 + (i >> 2) * 256 + (i & 3) * 32] = (float)v[i];
  }
}

template <int TO, int NBI>
__device__ inline void store_round(const Slots& sl, const Int8Args& a, const i32x16_t (&acc)[4][4], long row0, long n0) {
  stage_i32<NBI>(sl, acc);
  __syncthreads();
  const int tid = opaque((int)threadIdx.x);
  const int q = tid & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const StPair st = h ? st_pair<1>(sl) : st_pair<0>(sl);
    const long col = n0 + 128 * h + 32 * NBI + 8 * q;
    const int n = (int)min(8L, a.V - col);
    if (n <= 0) continue;
    float sw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sw[i] = i < n ? a.sw[col + i] : 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = (tid >> 2) + 64 * k;
      if (row0 + r >= a.T) break;
      const float sx = a.sx[row0 + r];
      const float4 u = st_read4(st, r, 2 * q), v = st_read4(st, r, 2 * q + 1);
      const float y[8] = {u.x * sx * sw[0], u.y * sx * sw[1], u.z * sx * sw[2], u.w * sx * sw[3],
                          v.x * sx * sw[4], v.y * sx * sw[5], v.z * sx * sw[6], v.w * sx * sw[7]};
      store8<TO>(a.out + ((row0 + r) * a.V + col) * Elem<TO>::kBytes, y, n);
    }
  }
  __syncthreads();
}

}  // namespace

template <int TO>
__global__ __launch_bounds__(kThreads, 1) void int8_tile_kernel(Int8Args a, int nrb, int ncb, int group) {
  KD_DECLARE_SLOTS(sl);
  int rb, cb;
  grouped_coords(xcd_remap(blockIdx.x, gridDim.x), nrb, ncb, group, rb, cb);
  const long row0 = (long)rb * kBM, n0 = (long)cb * 256;
  const long stages = (a.d + kRowB - 1) / kRowB, nst = (stages + kRing - 1) / kRing * kRing;

  DmaRows<256> ra, rw;
  const char* xbase = a.panels + row0 * kRowB;
  ra.init(
      xbase, [&](int i) { return xbase + (row0 + DmaRows<256>::row_of(i) < a.T ? DmaRows<256>::row_of(i) : 0) * (long)kRowB; },
      (uint32_t)(a.T * kRowB));
  const char* wbase = a.w + n0 * a.d;
  rw.init(wbase, [&](int i) { return wbase + (n0 + DmaRows<256>::row_of(i) < a.V ? DmaRows<256>::row_of(i) : 0) * a.d; });
  // the last rows' stages end behind w where d is no multiple of 64: past the range, loads give nothing
  rw.rs = make_rsrc(wbase, min((a.V - n0) * a.d, 0xffffffffL));

  FragReader<256> rd;
  rd.init_rows();
  i32x16_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
  const long w_last = stages - 1;
  ring_contract<DmaRows<256>::kPer * 2, FragsRows<256>>(
      sl, (int)nst,
      [&](long s, char* da, char* db) {
        ra.issue(s, da);
        rw.issue(min(s, w_last), db);
      },
      [&](const char* slot, FragsRows<256>& f) { rd.read_rows(slot, f); },
      [&](const FragsRows<256>& f) {
#pragma unroll
        for (int kg = 0; kg < 2; ++kg)
#pragma unroll
          for (int mb = 0; mb < 4; ++mb)
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) mma_i8(acc[mb][nb], f.a[kg][mb], f.b[kg][nb]);
      });
  store_round<TO, 0>(sl, a, acc, row0, n0);
  store_round<TO, 1>(sl, a, acc, row0, n0);
  store_round<TO, 2>(sl, a, acc, row0, n0);
  store_round<TO, 3>(sl, a, acc, row0, n0);
}

// ------------------------------------------------------------------ few rows
namespace {
constexpr int kFewV = 64;     // channels of a workgroup
constexpr int kFewU = 4;      // 16-byte chunks of a lane and step
constexpr int kFewK = 2 * 16 * kFewU;  // k of a step
}  // namespace

// NB blocks of 32 rows of x
template <int TO, int NB>
__global__ __launch_bounds__(256) void int8_few_kernel(Int8Args a) {
  __shared__ int part[4][32][36];
  const int lane = threadIdx.x & 63, w = wave_id();
  const int m = lane & 31, h = lane >> 5;
  const long v0 = (long)blockIdx.x * kFewV, t0 = (long)blockIdx.y * 32 * NB;
  const char* wp[2];
  const char* xp[NB];
#pragma unroll
  for (int f = 0; f < 2; ++f) wp[f] = a.w + min(v0 + 32 * f + m, (long)a.V - 1) * a.d + h * 16 * kFewU;
#pragma unroll
  for (int f = 0; f < NB; ++f) xp[f] = a.x + min(t0 + 32 * f + m, (long)a.T - 1) * a.d + h * 16 * kFewU;

  const int steps = (int)((a.d + kFewK - 1) / kFewK), whole = (int)(a.d / kFewK);
  const int s0 = steps * w / 4, s1 = steps * (w + 1) / 4;
  u32x4_t rw[2][2][kFewU], rx[2][NB][kFewU];
  auto load = [&](int buf, int s) {
    const long at = (long)s * kFewK;
    if (s < whole) {
#pragma unroll
      for (int u = 0; u < kFewU; ++u) {
#pragma unroll
        for (int f = 0; f < 2; ++f) rw[buf][f][u] = ld16(wp[f] + at + 16 * u);
#pragma unroll
        for (int f = 0; f < NB; ++f) rx[buf][f][u] = ld16(xp[f] + at + 16 * u);
      }
    } else {  // the rows end within the step
#pragma unroll
      for (int u = 0; u < kFewU; ++u) {
        const bool in = at + h * 16 * kFewU + 16 * u < a.d;
#pragma unroll
        for (int f = 0; f < 2; ++f) rw[buf][f][u] = in ? ld16(wp[f] + at + 16 * u) : zero4();
#pragma unroll
        for (int f = 0; f < NB; ++f) rx[buf][f][u] = in ? ld16(xp[f] + at + 16 * u) : zero4();
      }
    }
  };
  i32x16_t acc[2][NB];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
  auto multiply = [&](int buf) {
#pragma unroll
    for (int u = 0; u < kFewU; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) mma_i8(acc[i][j], rw[buf][i][u], rx[buf][j][u]);
  };
  if (s0 < s1) {
    load(0, s0);
    int s = s0;
    for (; s + 2 <= s1; s += 2) {
      load(1, s + 1);
      multiply(0);
      if (s + 2 < s1) load(0, s + 2);
      multiply(1);
    }
    if (s < s1) multiply(0);
  }

  // the waves' sums, block by block: [row of x][channel]
  const int r = threadIdx.x >> 3, c = 4 * (threadIdx.x & 7);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      __syncthreads();
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<i32x4_t*>(&part[w][m][8 * q + 4 * h]) =
            i32x4_t{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
      __syncthreads();
      i32x4_t s = *reinterpret_cast<const i32x4_t*>(&part[0][r][c]);
#pragma unroll
      for (int k = 1; k < 4; ++k) s += *reinterpret_cast<const i32x4_t*>(&part[k][r][c]);
      const long t = t0 + 32 * j + r, v = v0 + 32 * i + c;
      if (t >= a.T || v >= a.V) continue;
      const float sx = a.sx[t];
      char* to = a.out + (t * a.V + v) * Elem<TO>::kBytes;
      float y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = v + e < a.V ? (float)s[e] * sx * a.sw[v + e] : 0.f;
      if (v + 4 <= a.V) {
        if constexpr (TO == kTypeF32) {
          store16(to, u32x4_t{__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3])});
        } else {
          const uint2 o{pack2x16<TO>(y[0], y[1]), pack2x16<TO>(y[2], y[3])};
          __builtin_memcpy(to, &o, 8);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (v + e < a.V) Elem<TO>::put1(to + e * Elem<TO>::kBytes, y[e]);
      }
    }
}

// ------------------------------------------------------------------ launches
bool int8_tiles(int64_t T, int64_t d, int64_t V) {
  return T > 128 && ((T + 255) / 256) * ((V + 255) / 256) >= 128;
}
int64_t int8_panel_bytes(int64_t T, int64_t d) { return T * ((d + kKTurn - 1) / kKTurn * kKTurn); }

hipError_t launch_int8_panels(const Int8Args& a, hipStream_t st) {
  const long chunks = (a.d + kKTurn - 1) / kKTurn * kKTurn / 16;
  const long blocks = std::min<long>((a.T * chunks + 255) / 256, 8192);
  hipLaunchKernelGGL(int8_panels_kernel, dim3((unsigned)blocks), dim3(256), 0, st, a.x, (long)a.T, (long)a.d, chunks,
                     a.panels);
  return hipGetLastError();
}

hipError_t launch_int8_tiles(const Int8Args& a, hipStream_t st) {
  const int nrb = (int)((a.T + 255) / 256), ncb = (int)((a.V + 255) / 256);
  pick_type(a.out_type, [&](auto ty) {
    hipLaunchKernelGGL((int8_tile_kernel<decltype(ty)::value>), dim3((unsigned)(nrb * ncb)), dim3(kThreads), 0, st, a,
                       nrb, ncb, 4);
  });
  return hipGetLastError();
}

hipError_t launch_int8_few(const Int8Args& a, hipStream_t st) {
  pick_type(a.out_type, [&](auto ty) {
    constexpr int TO = decltype(ty)::value;
    auto with = [&](auto nb) {
      constexpr int NB = decltype(nb)::value;
      const dim3 grid((unsigned)((a.V + kFewV - 1) / kFewV), (unsigned)((a.T + 32 * NB - 1) / (32 * NB)));
      hipLaunchKernelGGL((int8_few_kernel<TO, NB>), grid, dim3(256), 0, st, a);
    };
    if (a.T <= 32) with(std::integral_constant<int, 1>());
    else if (a.T <= 64) with(std::integral_constant<int, 2>());
    else with(std::integral_constant<int, 4>());
  });
  return hipGetLastError();
}

}  // namespace kd
