// Token embeddings and their gradient.
//
//   out[t] = scale E[tokens[t]],   dE_v = scale sum_{t: tokens[t] = v} grad[t]
//
// Forward: a copy of rows, or for tied weights a gather of columns.
//
// Backward: rows that meet in one token are added up without atomics.  The
// positions are sorted by token (stable, so in ascending order within one);
// a wave takes a piece of consecutive sorted entries and 512 columns, adds up
// each run of equal tokens in registers and stores it; what it holds of a run
// that goes on in the piece before or after goes to a partial row, and a
// second kernel adds up those of each such run in their order.  The order of
// every sum is that of the positions, cut at multiples of the piece: the same
// bits each time.  A frequent token (the first few take a tenth of a text)
// then costs as many partial rows as it has pieces, spread over the chip.
#include <type_traits>

#include "kd_launch.h"
#include "kd_layers.h"
#include "kd_row.h"

namespace kd {

namespace {

__device__ inline int wave_in_grid() { return blockIdx.x * (blockDim.x >> 6) + wave_id(); }

constexpr int kSlab = 512;  // columns of a wave

}  // namespace

// ------------------------------------------------------------------ forward
template <int TY>
__global__ __launch_bounds__(256) void embed_kernel(EmbedArgs a, int slabs) {
  const int64_t waves = (int64_t)gridDim.x * 4;
  const int lane = threadIdx.x & 63;
  for (int64_t u = wave_in_grid(); u < a.T * slabs; u += waves) {
    const int64_t t = u / slabs;
    const int p = (int)(u - t * slabs) * 64 + lane;
    const int n = (int)(a.d - 8 * (int64_t)p);
    if (n <= 0) continue;
    float x[8];
    if (a.mask && !a.mask[t]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
    } else {
      const int64_t v = a.tokens[t];
      if (v < 0 || v >= a.V) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(0x7fc00000u);
      } else {
        load_row<TY>(a.table + v * a.d * Elem<TY>::kBytes, a.d, p, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= a.scale;
      }
    }
    store8<TY>(a.out + (t * a.d + 8 * (int64_t)p) * Elem<TY>::kBytes, x, n);
  }
}

// Tied: 64 tokens x 64 rows of W a workgroup.  A lane keeps its token and goes
// down the rows; the tile is turned in LDS, so that the output is written in
// runs of 64 elements.
template <int TY>
__global__ __launch_bounds__(256) void embed_tied_kernel(EmbedArgs a, int blocks_t) {
  using E = Elem<TY>;
  __shared__ float tile[64][65];
  const int lane = threadIdx.x & 63, w = wave_id();
  const int64_t t0 = (int64_t)(blockIdx.x % blocks_t) * 64, k0 = (int64_t)(blockIdx.x / blocks_t) * 64;
  const int64_t t = t0 + lane;
  const bool valid = t < a.T && (!a.mask || a.mask[t]);
  const int64_t v = valid ? a.tokens[t] : 0;
  const bool in = valid && v >= 0 && v < a.V;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t k = k0 + w * 16 + i;
    float x = valid ? __uint_as_float(0x7fc00000u) : 0.f;
    if (in && k < a.d) x = E::get1(a.table + (k * a.V + v) * E::kBytes) * a.scale;
    tile[lane][w * 16 + i] = x;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * 8; i += 256) {
    const int64_t to = t0 + (i >> 3), k = k0 + 8 * (i & 7);
    if (to >= a.T || k >= a.d) continue;
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = tile[i >> 3][8 * (i & 7) + j];
    store8<TY>(a.out + (to * a.d + k) * E::kBytes, x, (int)(a.d - k));
  }
}

hipError_t launch_embed(const EmbedArgs& a, hipStream_t st) {
  pick_type(a.type, [&](auto ty) {
    constexpr int TY = decltype(ty)::value;
    if (a.tied) {
      const int64_t bt = (a.T + 63) / 64, bk = (a.d + 63) / 64;
      hipLaunchKernelGGL((embed_tied_kernel<TY>), dim3((unsigned)(bt * bk)), dim3(256), 0, st, a, (int)bt);
    } else {
      const int slabs = (int)((a.d + kSlab - 1) / kSlab);
      const int64_t blocks = (a.T * slabs + 3) / 4;
      hipLaunchKernelGGL((embed_kernel<TY>), dim3((unsigned)std::min<int64_t>(blocks, 1 << 20)), dim3(256), 0, st, a,
                         slabs);
    }
  });
  return hipGetLastError();
}

// ------------------------------------------------------------------ sorting the positions by token
// Least significant digit first, every pass stable.  Within a workgroup wave w
// holds consecutive items, 64 a round; an item's place among the items of its
// digit is the number of such items in earlier waves, earlier rounds and
// earlier lanes.
namespace {

// The lanes that hold the same digit as this one.
template <int BITS>
__device__ inline uint64_t same_digit(uint32_t digit) {
  uint64_t m = ~uint64_t(0);
#pragma unroll
  for (int b = 0; b < BITS; ++b) {
    const bool bit = (digit >> b) & 1;
    const uint64_t set = __ballot(bit);
    m &= bit ? set : ~set;
  }
  return m;
}

// The item's place among those of its digit in this wave so far; `seen` is
// the wave's count of the digit, in LDS.
__device__ inline uint32_t place_in_wave(uint64_t same, volatile uint32_t* seen) {
  const int lane = threadIdx.x & 63;
  const uint32_t before = (uint32_t)__popcll(same & ((uint64_t(1) << lane) - 1));
  const uint32_t had = *seen;
  __builtin_amdgcn_wave_barrier();
  if (before == 0) *seen = had + (uint32_t)__popcll(same);
  __builtin_amdgcn_wave_barrier();
  return had + before;
}

// Exclusive sum over the 1024 threads of a workgroup.
__device__ inline uint32_t block_exclusive(uint32_t v, uint32_t* lds16, uint32_t* total = nullptr) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  uint32_t s = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t up = (uint32_t)__shfl_up((int)s, o);
    if (lane >= o) s += up;
  }
  __syncthreads();
  if (lane == 63) lds16[w] = s;
  __syncthreads();
  uint32_t base = 0, all = 0;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    if (k < w) base += lds16[k];
    all += lds16[k];
  }
  if (total) *total = all;
  return base + s - v;
}

__device__ inline uint32_t key_of(const SortArgs& a, int64_t i) {
  if (a.mask && !a.mask[i]) return (uint32_t)a.V;
  const int64_t v = a.tokens[i];
  return v < 0 || v >= a.V ? (uint32_t)a.V : (uint32_t)v;
}

int bits_of(int64_t V) {  // of the keys 0 .. V
  int b = 1;
  while ((V >> b) != 0) ++b;
  return b;
}

}  // namespace

// Up to kSortSmall tokens in one workgroup: digits of 6 bits, keys and
// positions in LDS between the passes and in registers within one.
template <int ROUNDS>
__global__ __launch_bounds__(1024) void sort_small_kernel(SortArgs a, int bits) {
  __shared__ uint32_t keys[1024 * ROUNDS], poss[1024 * ROUNDS];
  __shared__ uint32_t seen[64 * 16], lds[16];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  uint32_t k[ROUNDS], p[ROUNDS];
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int64_t i = (int64_t)w * 64 * ROUNDS + r * 64 + lane;
    k[r] = i < a.T ? key_of(a, i) : 0xffffffffu;  // behind the last one, and stays there
    p[r] = (uint32_t)i;
  }
  for (int shift = 0; shift < bits; shift += 6) {
    seen[threadIdx.x] = 0;
    __syncthreads();
    uint32_t at[ROUNDS];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      const uint32_t digit = (k[r] >> shift) & 63u;
      at[r] = place_in_wave(same_digit<6>(digit), &seen[digit * 16 + w]);
    }
    __syncthreads();
    const uint32_t base = block_exclusive(seen[threadIdx.x], lds);
    __syncthreads();
    seen[threadIdx.x] = base;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      const uint32_t to = seen[((k[r] >> shift) & 63u) * 16 + w] + at[r];
      keys[to] = k[r];
      poss[to] = p[r];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      const int i = w * 64 * ROUNDS + r * 64 + lane;
      k[r] = keys[i];
      p[r] = poss[i];
    }
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int64_t i = (int64_t)w * 64 * ROUNDS + r * 64 + lane;
    if (i < a.T) {
      a.key[0][i] = k[r];
      a.pos[0][i] = p[r];
    }
  }
}

// More tokens: per pass of 9 bits the workgroups' counts of every digit, their
// sums in the order digit, workgroup, and the items to their places.
namespace {
constexpr int kSortRounds = kSortItems / 1024;
constexpr int kDigitBits = 9;
static_assert(kSortDigits == 1 << kDigitBits, "digits");

__device__ inline void sort_item(const SortArgs& a, int pass, int64_t i, uint32_t& k, uint32_t& p) {
  if (pass == 0) {
    k = key_of(a, i);
    p = (uint32_t)i;
  } else {
    k = a.key[(pass - 1) & 1][i];
    p = a.pos[(pass - 1) & 1][i];
  }
}
}  // namespace

__global__ __launch_bounds__(1024) void sort_count_kernel(SortArgs a, int pass) {
  __shared__ uint32_t n[kSortDigits];
  for (int i = threadIdx.x; i < kSortDigits; i += 1024) n[i] = 0;
  __syncthreads();
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t i = (int64_t)blockIdx.x * kSortItems + r * 1024 + threadIdx.x;
    if (i >= a.T) break;
    uint32_t k, p;
    sort_item(a, pass, i, k, p);
    atomicAdd(&n[(k >> (pass * kDigitBits)) & (kSortDigits - 1)], 1u);  // whole numbers: any order gives the same
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kSortDigits; i += 1024) a.count[(int64_t)i * gridDim.x + blockIdx.x] = n[i];
}

__global__ __launch_bounds__(1024) void sort_scan_kernel(uint32_t* count, int64_t n) {
  __shared__ uint32_t lds[16];
  uint32_t carry = 0;
  for (int64_t i0 = 0; i0 < n; i0 += 8192) {
    const int64_t i = i0 + 8 * (int64_t)threadIdx.x;
    uint32_t v[8], s = 0, all;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = i + j < n ? count[i + j] : 0;
      s += v[j];
    }
    uint32_t at = carry + block_exclusive(s, lds, &all);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (i + j < n) count[i + j] = at;
      at += v[j];
    }
    carry += all;
  }
}

__global__ __launch_bounds__(1024) void sort_scatter_kernel(SortArgs a, int pass) {
  __shared__ uint32_t seen[kSortDigits * 16];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, shift = pass * kDigitBits;
  for (int i = threadIdx.x; i < kSortDigits * 16; i += 1024) seen[i] = 0;
  __syncthreads();
  uint32_t k[kSortRounds], p[kSortRounds], at[kSortRounds];
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t i = (int64_t)blockIdx.x * kSortItems + w * 64 * kSortRounds + r * 64 + lane;
    k[r] = 0xffffffffu;
    p[r] = 0;
    if (i < a.T) sort_item(a, pass, i, k[r], p[r]);
    const uint32_t digit = (k[r] >> shift) & (kSortDigits - 1);
    // items behind the last one count as the highest digit, after all others of this (the last) workgroup
    at[r] = place_in_wave(same_digit<kDigitBits>(digit), &seen[digit * 16 + w]);
  }
  __syncthreads();
  if (threadIdx.x < kSortDigits) {
    uint32_t base = a.count[(int64_t)threadIdx.x * gridDim.x + blockIdx.x];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint32_t n = seen[threadIdx.x * 16 + j];
      seen[threadIdx.x * 16 + j] = base;
      base += n;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t i = (int64_t)blockIdx.x * kSortItems + w * 64 * kSortRounds + r * 64 + lane;
    if (i >= a.T) continue;
    const uint32_t to = seen[((k[r] >> shift) & (kSortDigits - 1)) * 16 + w] + at[r];
    a.key[pass & 1][to] = k[r];
    a.pos[pass & 1][to] = p[r];
  }
}

int sort_passes(int64_t V) { return (bits_of(V) + kDigitBits - 1) / kDigitBits; }
int sort_result(int64_t T, int64_t V) { return T <= kSortSmall ? 0 : (sort_passes(V) - 1) & 1; }

hipError_t launch_sort_small(const SortArgs& a, hipStream_t st) {
  const int bits = bits_of(a.V);
  if (a.T <= 1024) hipLaunchKernelGGL((sort_small_kernel<1>), dim3(1), dim3(1024), 0, st, a, bits);
  else if (a.T <= 4096) hipLaunchKernelGGL((sort_small_kernel<4>), dim3(1), dim3(1024), 0, st, a, bits);
  else hipLaunchKernelGGL((sort_small_kernel<16>), dim3(1), dim3(1024), 0, st, a, bits);
  return hipGetLastError();
}
hipError_t launch_sort_count(const SortArgs& a, int pass, hipStream_t st) {
  hipLaunchKernelGGL(sort_count_kernel, dim3((unsigned)((a.T + kSortItems - 1) / kSortItems)), dim3(1024), 0, st, a, pass);
  return hipGetLastError();
}
hipError_t launch_sort_scan(const SortArgs& a, int, hipStream_t st) {
  const int64_t n = (a.T + kSortItems - 1) / kSortItems * kSortDigits;
  hipLaunchKernelGGL(sort_scan_kernel, dim3(1), dim3(1024), 0, st, a.count, n);
  return hipGetLastError();
}
hipError_t launch_sort_scatter(const SortArgs& a, int pass, hipStream_t st) {
  hipLaunchKernelGGL(sort_scatter_kernel, dim3((unsigned)((a.T + kSortItems - 1) / kSortItems)), dim3(1024), 0, st, a, pass);
  return hipGetLastError();
}

// ------------------------------------------------------------------ gradient
namespace {

__device__ inline float get_any1(const char* base, int type, int64_t i) {
  if (type == kTypeF32) return Elem<kTypeF32>::get1(base + 4 * i);
  if (type == kTypeBf16) return Elem<kTypeBf16>::get1(base + 2 * i);
  return Elem<kTypeF16>::get1(base + 2 * i);
}

// dE_v's piece p from the sum x
__device__ inline void put_sum(const EmbedGradArgs& a, int64_t v, int p, const float (&x)[8]) {
  const int64_t n = a.d - 8 * (int64_t)p;
  if (n <= 0) return;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = x[i] * a.scale;
  if (a.tied) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= n) continue;
      const int64_t at = (8 * (int64_t)p + i) * a.V + v;
      if (a.accumulate) y[i] += get_any1(a.out, a.grad_type, at);
      store_any1(a.out, a.grad_type, at, y[i]);
    }
    return;
  }
  auto put = [&](auto ty) {
    constexpr int G = decltype(ty)::value;
    char* row = a.out + v * a.d * Elem<G>::kBytes;
    if (a.accumulate) {
      float was[8];
      load_row<G>(row, a.d, p, was);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] += was[i];
    }
    store8<G>(row + 8 * (int64_t)p * Elem<G>::kBytes, y, (int)n);
  };
  if (a.grad_type == kTypeF32) put(std::integral_constant<int, kTypeF32>());
  else if (a.grad_type == kTypeBf16) put(std::integral_constant<int, kTypeBf16>());
  else put(std::integral_constant<int, kTypeF16>());
}

__device__ inline void put_part(const EmbedGradArgs& a, int64_t piece, int which, int p, const float (&x)[8]) {
  const int64_t n = a.d - 8 * (int64_t)p;
  if (n <= 0) return;
  store8<kTypeF32>(reinterpret_cast<char*>(a.part + (piece * 2 + which) * a.d + 8 * (int64_t)p), x, (int)n);
}

// the first entry whose key is at least v
__device__ inline int64_t lower_bound(const uint32_t* key, int64_t n, uint32_t v) {
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (key[mid] < v) lo = mid + 1; else hi = mid;
  }
  return lo;
}

constexpr int kFillRows = 16;  // table rows of a wave that writes zeros

__device__ inline uint32_t lane_of(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

}  // namespace

// Waves [0, pieces * slabs) add up, the waves behind them write zeros to the
// table's rows whose tokens do not occur.
template <int TY>
__global__ __launch_bounds__(256) void embed_grad_kernel(EmbedGradArgs a, int64_t pieces, int slabs) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = wave_in_grid();
  if (wave >= pieces * slabs) {
    if (a.tied || a.accumulate) return;
    const int64_t v0 = (wave - pieces * slabs) * kFillRows, v = v0 + lane;
    bool empty = false;
    if (lane < kFillRows && v < a.V) {
      const int64_t i = lower_bound(a.key, a.T, (uint32_t)v);
      empty = i >= a.T || a.key[i] != (uint32_t)v;
    }
    const int64_t bytes = a.d * (a.grad_type == kTypeF32 ? 4 : 2);
    for (uint64_t m = __ballot(empty); m; m &= m - 1) {
      char* row = a.out + (v0 + __builtin_ctzll(m)) * bytes;
      int64_t at = 16 * lane;
      for (; at + 16 <= bytes; at += 1024) store16(row + at, zero4());
      if (at < bytes)
        for (; at < bytes; at += 2) *reinterpret_cast<uint16_t*>(row + at) = 0;
    }
    return;
  }
  const int64_t piece = wave / slabs;
  const int p = (int)(wave - piece * slabs) * 64 + lane;
  const int64_t e0 = piece * a.piece;
  const int ne = (int)min((int64_t)a.piece, a.T - e0);
  // the piece's entries in the lanes, and the keys around it
  const uint32_t keys = lane < ne ? a.key[e0 + lane] : 0xffffffffu;
  const uint32_t poss = lane < ne ? a.pos[e0 + lane] : 0;
  const uint32_t before = e0 > 0 ? a.key[e0 - 1] : 0xffffffffu;
  const uint32_t after = e0 + ne < a.T ? a.key[e0 + ne] : 0xffffffffu;
  float x[8] = {};
  uint32_t v = lane_of(keys, 0);
  bool first = before == v;  // the run began in the piece before
  constexpr int U = 4;
  for (int e = 0; e < ne; e += U) {
    Raw8<TY> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = min(e + u, ne - 1);
      const int64_t t = lane_of(poss, i);
      r[u] = load8<TY>(a.grad + (t * a.d + 8 * (int64_t)p) * Elem<TY>::kBytes,
                       lane_of(keys, i) < (uint32_t)a.V ? (int)(a.d - 8 * (int64_t)p) : 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (e + u >= ne) break;
      const uint32_t k = lane_of(keys, e + u);
      if (k != v) {
        if (first) put_part(a, piece, 0, p, x);
        else put_sum(a, v, p, x);
        first = false;
        v = k;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
      }
      if (v >= (uint32_t)a.V) return;  // only entries that count for nothing from here on
      float y[8];
      unpack8<TY>(r[u], y);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] += y[i];
    }
  }
  if (first) put_part(a, piece, 0, p, x);
  else if (after == v) put_part(a, piece, 1, p, x);
  else put_sum(a, v, p, x);
}

// A wave for each piece in which a run begins that goes on: its partial rows in order.
__global__ __launch_bounds__(256) void embed_join_kernel(EmbedGradArgs a, int64_t pieces, int slabs) {
  const int64_t wave = wave_in_grid();
  const int64_t piece = wave / slabs;
  if (piece + 1 >= pieces) return;
  const int p = (int)(wave - piece * slabs) * 64 + (threadIdx.x & 63);
  const int64_t e0 = piece * a.piece, e1 = e0 + a.piece;
  const uint32_t v = a.key[e1 - 1];
  if (v >= (uint32_t)a.V || a.key[e1] != v) return;              // nothing goes on
  if (e0 > 0 && a.key[e0 - 1] == v) return;                      // it began before
  float x[8], y[8];
  load_row<kTypeF32>(reinterpret_cast<const char*>(a.part + (piece * 2 + 1) * a.d), a.d, p, x);
  const int64_t last = (lower_bound(a.key, a.T, v + 1) - 1) / a.piece;
  for (int64_t j = piece + 1; j <= last; ++j) {
    load_row<kTypeF32>(reinterpret_cast<const char*>(a.part + j * 2 * a.d), a.d, p, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] += y[i];
  }
  put_sum(a, v, p, x);
}

__global__ __launch_bounds__(256) void fill_table_kernel(char* p, int64_t bytes) {
  const int64_t n = bytes / 16, step = (int64_t)gridDim.x * 256;
  const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
  for (int64_t i = i0; i < n; i += step) store16(p + 16 * i, zero4());
  const int64_t tail = 16 * n + 2 * i0;
  if (tail < bytes) *reinterpret_cast<uint16_t*>(p + tail) = 0;
}

int embed_piece(int64_t T) { return T <= kSortSmall ? 16 : 64; }

namespace {
struct GradShape {
  int64_t pieces;
  int slabs;
};
GradShape grad_shape(const EmbedGradArgs& a) {
  return {(a.T + a.piece - 1) / a.piece, (int)((a.d + kSlab - 1) / kSlab)};
}
}  // namespace

hipError_t launch_embed_grad(const EmbedGradArgs& a, hipStream_t st) {
  const GradShape s = grad_shape(a);
  const int64_t fill = a.tied || a.accumulate ? 0 : (a.V + kFillRows - 1) / kFillRows;
  const dim3 grid((unsigned)((s.pieces * s.slabs + fill + 3) / 4));
  pick_type(a.type, [&](auto ty) {
    hipLaunchKernelGGL((embed_grad_kernel<decltype(ty)::value>), grid, dim3(256), 0, st, a, s.pieces, s.slabs);
  });
  return hipGetLastError();
}
hipError_t launch_fill_table(char* p, int64_t bytes, hipStream_t st) {
  const int64_t blocks = std::min<int64_t>(std::max<int64_t>((bytes / 16 + 255) / 256, 1), 8192);
  hipLaunchKernelGGL(fill_table_kernel, dim3((unsigned)blocks), dim3(256), 0, st, p, bytes);
  return hipGetLastError();
}
hipError_t launch_embed_join(const EmbedGradArgs& a, hipStream_t st) {
  const GradShape s = grad_shape(a);
  hipLaunchKernelGGL(embed_join_kernel, dim3((unsigned)((s.pieces * s.slabs + 3) / 4)), dim3(256), 0, st, a, s.pieces,
                     s.slabs);
  return hipGetLastError();
}

}  // namespace kd
