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
// (kd_dma.h) padded with zeros to whole ring turns, which cancel what w's
// stages show twice (kd_int8_place.h).  4001 x 4096 x 128256: 1.90 ms, 2.2 POP/s, the matrix
// pipe busy 65% at the 1.6 GHz that the chip keeps under it, no LDS conflicts.
// Few rows or few tiles: w is what has to be read;
// a workgroup takes 64 channels and up to 128 rows, each of its four waves a
// quarter of k, straight from global memory into registers (few channels: 32
// and eight waves).  4 x 4096 x 32000: 22 us, 131 MB of w at 6 TB/s.
#include <type_traits>

#include "kd_dma.h"
#include "kd_int8_place.h"
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

__device__ inline void mma0_i8(i32x16_t& acc, u32x4_t a, u32x4_t b) {  // into a fresh accumulator
  acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), i32x16_t{},
                                              0, 0, 0);
}

static_assert(kInt8Stage == kRowB && kInt8Turn == kRing * kRowB && kInt8Rows == kBM, "the ring's stages and blocks");

}  // namespace

// ------------------------------------------------------------------ x in panels
__global__ __launch_bounds__(256) void int8_panels_kernel(const char* x, long T, long d, long chunks, char* panels) {
  const long n = T * chunks, rows = int8_panel_rows(T);
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long)gridDim.x * 256) {
    // four 16-byte chunks of a 64-byte piece are neighbours, then rows, then pieces
    const long c = (i / (4 * T)) * 4 + (i & 3), t = (i >> 2) % T;
    const long at = int8_x_at(c >> 2, c & 3, d);
    *reinterpret_cast<u32x4_t*>(panels + panel_off(rows, t, c * 16)) = at >= 0 ? ld16(x + t * d + at) : zero4();
  }
}

// ------------------------------------------------------------------ tiles
namespace {

// Two tiles' scales: sx of 256 rows, sw of 256 columns.
struct ScaleSlots {
  float* f;  // [2][512]
  __device__ inline float* sx(int t) const { return f + (t & 1) * 512; }
  __device__ inline float* sw(int t) const { return f + (t & 1) * 512 + 256; }
};

__device__ inline void dma4(__amdgpu_buffer_rsrc_t rs, uint32_t voff, uint32_t soff, float* lds_wave_base) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (KD_LDS void*)lds_wave_base, 4, (int)voff, (int)soff, 0, 0);
}

// The lane's half of 16 packed columns: lane l holds columns 4 (l / 32) .. + 3
// of both groups of 8, and gets all of group l / 32.
__device__ inline u32x4_t join_halves(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1) {
  const auto p = __builtin_amdgcn_permlane32_swap((int)a0, (int)b0, false, false);
  const auto q = __builtin_amdgcn_permlane32_swap((int)a1, (int)b1, false, false);
  return u32x4_t{(uint32_t)p[0], (uint32_t)q[0], (uint32_t)p[1], (uint32_t)q[1]};
}

// Stores n (at most 16 bytes' worth of) values that lie in v.
template <int TO>
__device__ inline void store_some(char* to, u32x4_t v, long n) {
  constexpr int N = 16 / Elem<TO>::kBytes;
  if (n >= N) {
    store16(to, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < n) {
      if constexpr (TO == kTypeF32) reinterpret_cast<uint32_t*>(to)[i] = v[i];
      else reinterpret_cast<uint16_t*>(to)[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
    }
}

// A wave's quarter of a tile from its accumulators, which hold it transposed
// (mma_frags_t): lane l has row 32 mb + l % 32 and in register i column 32 nb +
// 8 (i / 4) + 4 (l / 32) + i % 4.  No staging in LDS and no barriers: the waves
// go on to the next tile by themselves, whose operands keep landing.
template <int TO>
__device__ inline void store_quarter(const Int8Args& a, const i32x16_t (&acc)[4][4], const float* sx, const float* sw,
                                     long row0, long n0) {
  const int w = wave_id();
  const int lane = opaque((int)threadIdx.x) & 63;
  const int m = lane & 31, h = lane >> 5;
  const int r0 = (w >> 1) * 128, c0 = (w & 1) * 128;
#pragma unroll
  for (int nb = 0; nb < 4; ++nb) {
    float4 s[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) s[q] = *reinterpret_cast<const float4*>(sw + c0 + 32 * nb + 8 * q + 4 * h);
#pragma unroll
    for (int mb = 0; mb < 4; ++mb) {
      const long row = row0 + r0 + 32 * mb + m;
      const float x = sx[r0 + 32 * mb + m];
      i32x16_t v = acc[mb][nb];
      asm volatile("" : "+a"(v));
      float y[16];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        y[4 * q] = (float)v[4 * q] * x * s[q].x;
        y[4 * q + 1] = (float)v[4 * q + 1] * x * s[q].y;
        y[4 * q + 2] = (float)v[4 * q + 2] * x * s[q].z;
        y[4 * q + 3] = (float)v[4 * q + 3] * x * s[q].w;
      }
      const long col = n0 + c0 + 32 * nb;
      char* const to = a.out + (row * a.V + col) * Elem<TO>::kBytes;
      u32x4_t o[4];
      if constexpr (TO == kTypeF32) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          o[q] = u32x4_t{__float_as_uint(y[4 * q]), __float_as_uint(y[4 * q + 1]), __float_as_uint(y[4 * q + 2]),
                         __float_as_uint(y[4 * q + 3])};
      } else {
#pragma unroll
        for (int g = 0; g < 2; ++g)
          o[g] = join_halves(pack2x16<TO>(y[8 * g], y[8 * g + 1]), pack2x16<TO>(y[8 * g + 2], y[8 * g + 3]),
                             pack2x16<TO>(y[8 * g + 4], y[8 * g + 5]), pack2x16<TO>(y[8 * g + 6], y[8 * g + 7]));
      }
      if (row < a.T) {
        if constexpr (TO == kTypeF32) {
#pragma unroll
          for (int q = 0; q < 4; ++q) store_some<TO>(to + 4 * (8 * q + 4 * h), o[q], a.V - col - 8 * q - 4 * h);
        } else {
#pragma unroll
          for (int g = 0; g < 2; ++g) store_some<TO>(to + 2 * (16 * g + 8 * h), o[g], a.V - col - 16 * g - 8 * h);
        }
      }
    }
  }
}

}  // namespace

// Persistent: one workgroup a CU, and one ring that never drains.  XCD x has
// one contiguous range of the tiles (rows grouped, see grouped_coords), its
// workgroups take turns in it, so that what they read at one time shares
// panels of both operands in the XCD's cache.
template <int TO>
__global__ __launch_bounds__(kThreads, 1) void int8_tile_kernel(Int8Args a, int nrb, int ncb, int group) {
  KD_DECLARE_SLOTS(sl);
  const int tiles = nrb * ncb, xcd = blockIdx.x & 7, turn = gridDim.x >> 3;  // the grid is a multiple of 8
  const int begin = (int)((long)tiles * xcd / 8) + (int)(blockIdx.x >> 3), end = (int)((long)tiles * (xcd + 1) / 8);
  const int mine = begin < end ? (end - begin + turn - 1) / turn : 0;
  const long nst = int8_turns(a.d) * kRing, rows = int8_panel_rows(a.T);
  const long panel_bytes = rows * nst * kRowB;

  // what a tile's loads start from; w's rows behind the last one are past its
  // descriptor's range by their vector offset alone
  struct Place {
    long row0, n0;
    __amdgpu_buffer_rsrc_t x, w;
  };
  auto place = [&](int t) {
    int rb, cb;
    grouped_coords(min(begin + t * turn, tiles - 1), nrb, ncb, group, rb, cb);
    Place p;
    p.row0 = (long)rb * kBM;
    p.n0 = (long)cb * 256;
    p.x = make_rsrc(a.panels + p.row0 * kRowB, min(panel_bytes - p.row0 * kRowB, 0xffffffffL));
    p.w = make_rsrc(a.w + p.n0 * a.d, min((a.V - p.n0) * a.d, 0xffffffffL));
    return p;
  };
  const __amdgpu_buffer_rsrc_t rsx = make_rsrc(reinterpret_cast<const char*>(a.sx), a.T * 4);
  const __amdgpu_buffer_rsrc_t rsw = make_rsrc(reinterpret_cast<const char*>(a.sw), min((long)a.V * 4, 0xffffffffL));
  const ScaleSlots scales{sl.ep};
  const uint32_t own = 4 * threadIdx.x;
  auto load_scales = [&](int t, const Place& p) {  // all of the offset where the range is sure to be compared with it
    dma4(rsx, (uint32_t)(p.row0 * 4) + own, 0, scales.sx(t) + 64 * wave_id());
    dma4(rsw, (uint32_t)(p.n0 * 4) + own, 0, scales.sw(t) + 64 * wave_id());
  };

  DmaRows<256> ra, rw;
  ra.init(a.panels, [&](int i) { return a.panels + DmaRows<256>::row_of(i) * (long)kRowB; }, (uint32_t)(rows * kRowB));
  rw.init(a.w, [&](int i) {
    const int m = DmaRows<256>::row_of(i), c = DmaRows<256>::chunk_of(m);
    return a.w + m * a.d + int8_chunk_at(c, a.d) - 16 * c;  // (init adds 16 c)
  });
  FragReader<256> rd;
  rd.init_rows();
  i32x16_t acc[4][4];
  Place now = place(0), next = place(1);
  load_scales(0, now);
  int at = 0;  // the tile of `now`
  ring_run<DmaRows<256>::kPer * 2, FragsRows<256>>(
      sl, mine, (int)nst,
      [&](long t, int s, char* da, char* db) {
        const bool cur = t == at;
        ra.rs = cur ? now.x : next.x;
        rw.rs = cur ? now.w : next.w;
        ra.issue(s, da);
        rw.issue(0, int8_stage_at(s, a.d), db);
      },
      [&](const char* slot, FragsRows<256>& f) { rd.read_rows(slot, f); },
      [&](const FragsRows<256>& f) {
#pragma unroll
        for (int kg = 0; kg < 2; ++kg)
#pragma unroll
          for (int mb = 0; mb < 4; ++mb)
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) mma_i8(acc[mb][nb], f.b[kg][nb], f.a[kg][mb]);
      },
      [&](const FragsRows<256>& f) {
#pragma unroll
        for (int mb = 0; mb < 4; ++mb)
#pragma unroll
          for (int nb = 0; nb < 4; ++nb) mma0_i8(acc[mb][nb], f.b[0][nb], f.a[0][mb]);
#pragma unroll
        for (int mb = 0; mb < 4; ++mb)
#pragma unroll
          for (int nb = 0; nb < 4; ++nb) mma_i8(acc[mb][nb], f.b[1][nb], f.a[1][mb]);
      },
      [&](int t) {
        store_quarter<TO>(a, acc, scales.sx(t), scales.sw(t), now.row0, now.n0);
        now = next;
        at = t + 1;
        next = place(t + 2);
        load_scales(t + 1, now);  // those slots were read last after the tile before this one
      });
}

// ------------------------------------------------------------------ few rows
namespace {
constexpr int kFewU = 4;      // 16-byte chunks of a lane and step
constexpr int kFewK = 2 * 16 * kFewU;  // k of a step
}  // namespace

// NB blocks of 32 rows of x and F of 32 channels a workgroup, W waves that
// split k.
template <int TO, int NB, int F, int W>
__global__ __launch_bounds__(64 * W) void int8_few_kernel(Int8Args a) {
  __shared__ __attribute__((aligned(16))) int part[W][32][36];
  const int lane = threadIdx.x & 63, w = wave_id();
  const int m = lane & 31, h = lane >> 5;
  const long v0 = (long)blockIdx.x * 32 * F, t0 = (long)blockIdx.y * 32 * NB;
  const char* wp[F];
  const char* xp[NB];
#pragma unroll
  for (int f = 0; f < F; ++f) wp[f] = a.w + min(v0 + 32 * f + m, (long)a.V - 1) * a.d + h * 16 * kFewU;
#pragma unroll
  for (int f = 0; f < NB; ++f) xp[f] = a.x + min(t0 + 32 * f + m, (long)a.T - 1) * a.d + h * 16 * kFewU;

  const int steps = (int)((a.d + kFewK - 1) / kFewK), whole = (int)(a.d / kFewK);
  const int s0 = steps * w / W, s1 = steps * (w + 1) / W;
  u32x4_t rw[2][F][kFewU], rx[2][NB][kFewU];
  auto load = [&](int buf, int s) {
    const long at = (long)s * kFewK;
    if (s < whole) {
#pragma unroll
      for (int u = 0; u < kFewU; ++u) {
#pragma unroll
        for (int f = 0; f < F; ++f) rw[buf][f][u] = ld16(wp[f] + at + 16 * u);
#pragma unroll
        for (int f = 0; f < NB; ++f) rx[buf][f][u] = ld16(xp[f] + at + 16 * u);
      }
    } else {  // the rows end within the step
#pragma unroll
      for (int u = 0; u < kFewU; ++u) {
        const bool in = at + h * 16 * kFewU + 16 * u < a.d;
#pragma unroll
        for (int f = 0; f < F; ++f) rw[buf][f][u] = in ? ld16(wp[f] + at + 16 * u) : zero4();
#pragma unroll
        for (int f = 0; f < NB; ++f) rx[buf][f][u] = in ? ld16(xp[f] + at + 16 * u) : zero4();
      }
    }
  };
  i32x16_t acc[F][NB];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
  auto multiply = [&](int buf) {
#pragma unroll
    for (int u = 0; u < kFewU; ++u)
#pragma unroll
      for (int i = 0; i < F; ++i)
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
  const int r = (threadIdx.x >> 3) & 31, c = 4 * (threadIdx.x & 7);
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      __syncthreads();
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<i32x4_t*>(&part[w][m][8 * q + 4 * h]) =
            i32x4_t{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
      __syncthreads();
      if (threadIdx.x >= 256) continue;
      i32x4_t s = *reinterpret_cast<const i32x4_t*>(&part[0][r][c]);
#pragma unroll
      for (int k = 1; k < W; ++k) s += *reinterpret_cast<const i32x4_t*>(&part[k][r][c]);
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
// Rounds of the chip's 256 CUs: a tile takes 46 us at d = 4096, a workgroup of
// the other kernel with 128 rows 28 us, one of them a CU.  Either side, us at
// d = 4096: V 32000, T 96 45 / 51, 128 45 / 58, 512 68 / 222; V 11008, T 128
// 44 / 30, 192 44 / 50, 512 48 / 85; V 4096, T 512 46 / 31, 1024 48 / 57.  Up to
// 64 rows the other kernel has two or three workgroups a CU and waits for w
// only: T 32, V 32000 46 / 27, V 128256 143 / 123; T 64, V 11008 42 / 20, V 32000 45 /
// 36, but V 128256 143 / 160: for the largest heads the border lies a little high.
bool int8_tiles(int64_t T, int64_t d, int64_t V) {
  auto rounds = [](int64_t workgroups) { return (workgroups + 255) / 256; };
  const int64_t tile = rounds(((T + 255) / 256) * ((V + 255) / 256)), few = rounds(((T + 127) / 128) * ((V + 63) / 64));
  return T > 64 && 7 * few > 12 * tile;
}
int64_t int8_panel_bytes(int64_t T, int64_t d) { return int8_panel_rows(T) * int8_turns(d) * kInt8Turn; }

hipError_t launch_int8_panels(const Int8Args& a, hipStream_t st) {
  const long chunks = int8_turns(a.d) * kInt8Turn / 16;
  const long blocks = std::min<long>((a.T * chunks + 255) / 256, 8192);
  hipLaunchKernelGGL(int8_panels_kernel, dim3((unsigned)blocks), dim3(256), 0, st, a.x, (long)a.T, (long)a.d, chunks,
                     a.panels);
  return hipGetLastError();
}

hipError_t launch_int8_tiles(const Int8Args& a, hipStream_t st) {
  const int nrb = (int)((a.T + 255) / 256), ncb = (int)((a.V + 255) / 256);
  pick_type(a.out_type, [&](auto ty) {
    hipLaunchKernelGGL((int8_tile_kernel<decltype(ty)::value>), dim3(256), dim3(kThreads), 0, st, a, nrb, ncb, 4);
  });
  return hipGetLastError();
}

hipError_t launch_int8_few(const Int8Args& a, hipStream_t st) {
  pick_type(a.out_type, [&](auto ty) {
    constexpr int TO = decltype(ty)::value;
    auto with = [&](auto nb, auto f, auto waves) {
      constexpr int NB = decltype(nb)::value, F = decltype(f)::value, W = decltype(waves)::value;
      const dim3 grid((unsigned)((a.V + 32 * F - 1) / (32 * F)), (unsigned)((a.T + 32 * NB - 1) / (32 * NB)));
      hipLaunchKernelGGL((int8_few_kernel<TO, NB, F, W>), grid, dim3(64 * W), 0, st, a);
    };
    using std::integral_constant;
    auto rows = [&](auto f, auto waves) {
      if (a.T <= 32) with(integral_constant<int, 1>(), f, waves);
      else if (a.T <= 64) with(integral_constant<int, 2>(), f, waves);
      else with(integral_constant<int, 4>(), f, waves);
    };
    // Half the channels a workgroup and twice its waves, if one round takes
    // them.  us, so / otherwise: V 4096, T 1 10 / 15, 64 14 / 18, 128 22 / 27; in
    // two rounds V 4096, T 384 44 / 28, V 11008, T 128 44 / 29.
    if ((a.V + 31) / 32 * ((a.T + 127) / 128) <= 256) rows(integral_constant<int, 1>(), integral_constant<int, 8>());
    else rows(integral_constant<int, 2>(), integral_constant<int, 4>());
  });
  return hipGetLastError();
}

}  // namespace kd
