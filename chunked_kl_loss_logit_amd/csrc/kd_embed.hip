// Token embeddings and their gradient.
//
//   out[t] = scale E[tokens[t]],   dE_v = scale sum_{t: tokens[t] = v} grad[t]
//
// Forward: a copy of rows, or for tied weights a gather of columns.  Bound by
// memory: 16384 rows of 2048 bf16 from a table of 128256 17-28 us (134 MB); tied,
// 4096 of 128256 columns of 2048 rows 37 us, from cold lines 44 (tokens as frequent
// as in text: 212 MB of cache lines for 17 MB of elements; spread evenly 94, 459 MB).
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
// For tied weights the runs' sums go to rows of their own first, and a third
// kernel makes them columns of the head's gradient.  Bound by the writes of the
// table's gradient: 16384 x 2048 bf16 into 128256 rows 15 us to sort, 109 for the
// sums and the zeros beside them (592 MB, 5.4 TB/s), 8 to join; tied, 3001 into
// 2048 x 32000 float32 11, 12, 5 and 40 to turn (262 MB at a fill's 6.6 TB/s).
#include <type_traits>

#include "kd_launch.h"
#include "kd_layers.h"
#include "kd_row.h"

namespace kd {

namespace {

__device__ inline int wave_in_grid() { return blockIdx.x * (blockDim.x >> 6) + wave_id(); }

constexpr int kSlab = 512;  // columns of a wave
constexpr int64_t kMostWaves = int64_t(1) << 24;  // of a launch: its threads are counted in 32 bits

}  // namespace

// ------------------------------------------------------------------ forward
// A wave takes kSlabs slabs of a row, all their loads in flight at once.
template <int TY, int SLABS>
__global__ __launch_bounds__(256) void embed_kernel(EmbedArgs a, int units) {
  const int wave = wave_in_grid();
  const int64_t t = wave / units;
  if (t >= a.T) return;
  const int p0 = (wave - (int)t * units) * SLABS * 64 + (threadIdx.x & 63);
  const bool valid = !a.mask || a.mask[t];
  const int64_t v = valid ? a.tokens[t] : -1;
  const bool in = v >= 0 && v < a.V;
  Raw8<TY> r[SLABS];
  if (in) {
    const char* row = a.table + v * a.d * Elem<TY>::kBytes;
#pragma unroll
    for (int i = 0; i < SLABS; ++i) {
      const int64_t at = 8 * (int64_t)(p0 + 64 * i);
      r[i] = load8<TY>(row + at * Elem<TY>::kBytes, (int)(a.d - at), at > 0);
    }
  }
#pragma unroll
  for (int i = 0; i < SLABS; ++i) {
    const int64_t at = 8 * (int64_t)(p0 + 64 * i);
    if (at >= a.d) continue;
    float x[8];
    if (in) {
      settle8<TY>(r[i], (int)(a.d - at), at > 0);
      unpack8<TY>(r[i], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= a.scale;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = valid ? __uint_as_float(0x7fc00000u) : 0.f;
    }
    store8<TY>(a.out + (t * a.d + at) * Elem<TY>::kBytes, x, (int)(a.d - at));
  }
}

// ------------------------------------------------------------------ sorting
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

// The first launch of a sort clears the tokens' marks, workgroup b of n of 1024
// threads its share of them.
__device__ inline void clear_runs(const SortArgs& a, int64_t b, int64_t n) {
  for (int64_t v = b * 4096 + 4 * threadIdx.x; v < a.V; v += n * 4096) {
    if (v + 4 <= a.V)
      *reinterpret_cast<int4*>(a.run_of + v) = int4{-1, -1, -1, -1};
    else
      for (int64_t i = v; i < a.V; ++i) a.run_of[i] = -1;
  }
}

int bits_of(int64_t V) {  // of the keys 0 .. V
  int b = 1;
  while ((V >> b) != 0) ++b;
  return b;
}

}  // namespace

namespace {
// Where an item of a workgroup of 1024 goes when they are ordered by a digit of 6 bits, stable.  seen: 16 x 65.
__device__ inline uint32_t place_in_block(uint32_t digit, uint32_t* seen, uint32_t* lds16) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  seen[w * 65 + lane] = 0;
  __syncthreads();
  const uint32_t at = place_in_wave(same_digit<6>(digit), &seen[w * 65 + digit]);
  __syncthreads();
  uint32_t* const mine = &seen[(threadIdx.x & 15) * 65 + (threadIdx.x >> 4)];  // in the order digit, wave
  const uint32_t base = block_exclusive(*mine, lds16);
  *mine = base;
  __syncthreads();
  return seen[w * 65 + digit] + at;
}
}  // namespace

// ------------------------------------------------------------------ forward, tied weights
// Tied weights: every load takes a cache line for one element, and what limits
// the kernel is how many lines are asked for.  A workgroup takes kTiedT tokens,
// sorts them by the cache line of W's rows that they lie in, and goes down
// ROWS rows: the lanes of a wave then share lines, and neighbouring waves do.
// The elements are turned in LDS and written in runs of ROWS, each to its
// token's row.  Workgroups of the same rows of W run on one XCD.  Up to
// kTiedFew tokens, 64 to a workgroup and unsorted, sorting costs more than it
// saves.  us, unsorted / sorted, cold W, bf16: d 2048, V 128256, T 128 7 / 12, 512 12 /
// 16, 700 16 / 18, 1024 21 / 21, 2048 42 / 37; V 32000, T 512 11 / 14, 1024 20 / 18,
// 2048 34 / 29; d 512, V 32000, T 512 7 / 12, 2048 9 / 13.  (Between 512 and 1024 the
// unsorted one would still be 2 us ahead, at small d beyond that too.)
constexpr int kTiedT = 1024;
constexpr int64_t kTiedFew = 512;

template <int TY, int ROWS>
__global__ __launch_bounds__(kTiedT) void embed_tied_kernel(EmbedArgs a, int blocks_t, int bits) {
  using E = Elem<TY>;
  using Bits = typename std::conditional<E::kBytes == 4, uint32_t, uint16_t>::type;
  constexpr int kLd = ROWS + 4 / E::kBytes;  // rows of words an odd number apart
  __shared__ uint32_t seen[16 * 65], sums[16];
  __shared__ uint32_t order[kTiedT];
  __shared__ __attribute__((aligned(16))) Bits tile[kTiedT * kLd];
  const int logical = xcd_remap(blockIdx.x, gridDim.x);
  const int64_t t0 = (int64_t)(logical % blocks_t) * kTiedT, k0 = (int64_t)(logical / blocks_t) * ROWS;
  constexpr uint32_t kNone = 0xfffffffeu, kOutside = 0xffffffffu;  // masked or behind the last one; no such token
  auto token = [&](int i) -> uint32_t {
    const int64_t t = t0 + i;
    if (t >= a.T || (a.mask && !a.mask[t])) return kNone;
    const int64_t v = a.tokens[t];
    return v < 0 || v >= a.V ? kOutside : (uint32_t)v;
  };
  uint32_t p = threadIdx.x;
  uint32_t line = min(token(p), (uint32_t)a.V) / (128 / E::kBytes);
  for (int shift = 0; shift < bits; shift += 6) {
    const uint32_t digit = (line >> shift) & 63u;
    const uint32_t to = place_in_block(digit, seen, sums);
    order[to] = p | line << 10;
    __syncthreads();
    p = order[threadIdx.x] & 1023u;
    line = order[threadIdx.x] >> 10;
  }
  const uint32_t v = token(p);
  const char* from = a.table + (k0 * a.V + (v < kNone ? v : 0)) * E::kBytes;
  const int rows = (int)min((int64_t)ROWS, a.d - k0);
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    float x = v == kNone ? 0.f : __uint_as_float(0x7fc00000u);
    if (v < kNone && i < rows) x = E::get1(from + i * a.V * E::kBytes) * a.scale;
    E::put1(reinterpret_cast<char*>(&tile[p * kLd + i]), x);
  }
  __syncthreads();
  constexpr int kPer = ROWS / 8;  // pieces of a token's run
  for (int i = threadIdx.x; i < kTiedT * kPer; i += kTiedT) {
    const int row = i / kPer, c = 8 * (i % kPer);
    if (t0 + row >= a.T || c >= rows) continue;
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = E::get1(reinterpret_cast<const char*>(&tile[row * kLd + c + j]));
    store8<TY>(a.out + ((t0 + row) * a.d + k0 + c) * E::kBytes, x, rows - c);
  }
}

constexpr int kFewT = 64, kFewK = 32;

template <int TY>
__global__ __launch_bounds__(256) void embed_tied_few_kernel(EmbedArgs a, int blocks_t) {
  using E = Elem<TY>;
  constexpr int kPer = kFewK / 4;  // rows of a wave
  __shared__ float tile[kFewT][kFewK + 1];
  const int lane = threadIdx.x & 63, w = wave_id();
  const int64_t t0 = (int64_t)(blockIdx.x % blocks_t) * kFewT, k0 = (int64_t)(blockIdx.x / blocks_t) * kFewK;
  const int64_t t = t0 + lane;
  const bool valid = t < a.T && (!a.mask || a.mask[t]);
  const int64_t v = valid ? a.tokens[t] : 0;
  const bool in = valid && v >= 0 && v < a.V;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t k = k0 + w * kPer + i;
    float x = valid ? __uint_as_float(0x7fc00000u) : 0.f;
    if (in && k < a.d) x = E::get1(a.table + (k * a.V + v) * E::kBytes) * a.scale;
    tile[lane][w * kPer + i] = x;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kFewT * kFewK / 8; i += 256) {
    const int row = i / (kFewK / 8), c = 8 * (i % (kFewK / 8));
    const int64_t to = t0 + row, k = k0 + c;
    if (to >= a.T || k >= a.d) continue;
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = tile[row][c + j];
    store8<TY>(a.out + (to * a.d + k) * E::kBytes, x, (int)(a.d - k));
  }
}

hipError_t launch_embed(const EmbedArgs& a, hipStream_t st) {
  pick_type(a.type, [&](auto ty) {
    constexpr int TY = decltype(ty)::value;
    if (a.tied && a.T > kTiedFew) {
      const int64_t bt = (a.T + kTiedT - 1) / kTiedT;
      const int bits = bits_of(a.V / (128 / Elem<TY>::kBytes));
      auto with = [&](auto rows) {
        constexpr int ROWS = decltype(rows)::value;
        const dim3 grid((unsigned)(bt * ((a.d + ROWS - 1) / ROWS)));
        hipLaunchKernelGGL((embed_tied_kernel<TY, ROWS>), grid, dim3(kTiedT), 0, st, a, (int)bt, bits);
      };
      // Longer runs where there are workgroups enough.  us, 32 / 16 rows, cold caches, d 2048: T 16384, V 32000 116 /
      // 128, T 3001 46 / 48, T 700 (64 / 128 workgroups) 36 / 25.
      if (bt * ((a.d + 31) / 32) >= 128) with(std::integral_constant<int, 32>());
      else with(std::integral_constant<int, 16>());
      return;
    }
    if (a.tied) {
      const int64_t bt = (a.T + kFewT - 1) / kFewT, bk = (a.d + kFewK - 1) / kFewK;
      hipLaunchKernelGGL((embed_tied_few_kernel<TY>), dim3((unsigned)(bt * bk)), dim3(256), 0, st, a, (int)bt);
      return;
    }
    auto with = [&](auto n) {
      constexpr int N = decltype(n)::value;
      const int units = (int)((a.d + kSlab * N - 1) / (kSlab * N));
      EmbedArgs some = a;
      for (int64_t t = 0; t < a.T; t += some.T) {
        some.T = std::min(a.T - t, kMostWaves / units);
        some.tokens = a.tokens + t;
        some.mask = a.mask ? a.mask + t : nullptr;
        some.out = a.out + t * a.d * Elem<TY>::kBytes;
        hipLaunchKernelGGL((embed_kernel<TY, N>), dim3((unsigned)((some.T * units + 3) / 4)), dim3(256), 0, st, some, units);
      }
    };
    if (a.T * a.d <= (1 << 20)) with(std::integral_constant<int, 1>());  // waves for the whole chip first
    else with(std::integral_constant<int, 4>());
  });
  return hipGetLastError();
}

// ------------------------------------------------------------------ all tokens by token
// Up to kSortSmall tokens: chunks of 1024, each sorted by one workgroup in LDS
// with digits of 6 bits, and then every entry's place among all chunks by
// binary search in each of them.  (One workgroup for all of 16384 tokens took
// 44 us, the instructions of 16 waves on one CU.)
// Workgroups behind the chunks' clear the marks.
__global__ __launch_bounds__(1024) void sort_chunk_kernel(SortArgs a, int bits, int chunks) {
  __shared__ uint32_t keys[kSortChunk], poss[kSortChunk];
  __shared__ uint32_t seen[16 * 65], lds[16];
  if ((int)blockIdx.x >= chunks) return clear_runs(a, blockIdx.x - chunks, gridDim.x - chunks);
  const int64_t i = (int64_t)blockIdx.x * kSortChunk + threadIdx.x;
  uint32_t k = i < a.T ? key_of(a, i) : 0xffffffffu;  // behind the last one, and stays there
  uint32_t p = (uint32_t)i;
  for (int shift = 0; shift < bits; shift += 6) {
    const uint32_t to = place_in_block((k >> shift) & 63u, seen, lds);
    keys[to] = k;
    poss[to] = p;
    __syncthreads();
    k = keys[threadIdx.x];
    p = poss[threadIdx.x];
  }
  if (i < a.T) {  // one chunk: the result
    a.key[chunks > 1][i] = k;
    a.pos[chunks > 1][i] = p;
  }
}

// 64 entries of one chunk a workgroup, every chunk's keys in LDS; each of the
// four waves searches a quarter of the chunks for all 64.
__global__ __launch_bounds__(256) void sort_rank_kernel(SortArgs a) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t places[4][64];
  const int T = (int)a.T, chunks = (T + kSortChunk - 1) / kSortChunk;
  for (int i = 4 * threadIdx.x; i < T; i += 1024) {
    if (i + 4 <= T)
      *reinterpret_cast<u32x4_t*>(keys + i) = ld16(reinterpret_cast<const char*>(a.key[1] + i));
    else
      for (int j = i; j < T; ++j) keys[j] = a.key[1][j];
  }
  __syncthreads();
  const int lane = threadIdx.x & 63, w = wave_id();
  const int i = min((int)blockIdx.x * 64 + lane, T - 1);
  const int own = (int)blockIdx.x * 64 / kSortChunk;
  const uint32_t k = keys[i];
  uint32_t place = 0;
  constexpr int U = 4;  // chunks searched at once: a step waits for the LDS, not for the others
  for (int c0 = w * U; c0 < chunks; c0 += 4 * U) {
    int lo[U], n[U];  // entries below the bound, of n
    uint32_t v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u;
      lo[u] = 0;
      n[u] = c < chunks && c != own ? min(kSortChunk, T - c * kSortChunk) : 0;
      v[u] = c < own ? k + 1 : k;  // earlier chunks' equal keys come first
    }
#pragma unroll
    for (int step = kSortChunk; step > 0; step >>= 1)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = min((c0 + u) * kSortChunk + lo[u] + step - 1, T - 1);
        if (keys[at] < v[u] && lo[u] + step <= n[u]) lo[u] += step;
      }
#pragma unroll
    for (int u = 0; u < U; ++u) place += (uint32_t)lo[u];
  }
  places[w][lane] = place;
  __syncthreads();
  if (w != 0 || (int)blockIdx.x * 64 + lane >= T) return;
  place = (uint32_t)(i - own * kSortChunk);
#pragma unroll
  for (int j = 0; j < 4; ++j) place += places[j][lane];
  a.key[0][place] = k;
  a.pos[0][place] = a.pos[1][i];
  if (a.run_of && k < (uint32_t)a.V) a.run_of[k] = (int32_t)place;
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
  if (pass == 0 && a.run_of) clear_runs(a, blockIdx.x, gridDim.x);
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

__global__ __launch_bounds__(1024) void sort_scatter_kernel(SortArgs a, int pass, int last) {
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
    if (last && a.run_of && k[r] < (uint32_t)a.V) a.run_of[k[r]] = (int32_t)to;
  }
}

int sort_passes(int64_t V) { return (bits_of(V) + kDigitBits - 1) / kDigitBits; }
int sort_result(int64_t T, int64_t V) { return T <= kSortSmall ? 0 : (sort_passes(V) - 1) & 1; }

hipError_t launch_sort_small(const SortArgs& a, hipStream_t st) {
  const int chunks = (int)((a.T + kSortChunk - 1) / kSortChunk);
  const int64_t clear = a.run_of ? std::min<int64_t>((a.V + 4095) / 4096, 64) : 0;
  hipLaunchKernelGGL(sort_chunk_kernel, dim3((unsigned)(chunks + clear)), dim3(kSortChunk), 0, st, a, bits_of(a.V), chunks);
  if (chunks > 1)
    hipLaunchKernelGGL(sort_rank_kernel, dim3((unsigned)((a.T + 63) / 64)), dim3(256), (unsigned)a.T * 4, st, a);
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
  hipLaunchKernelGGL(sort_scatter_kernel, dim3((unsigned)((a.T + kSortItems - 1) / kSortItems)), dim3(1024), 0, st, a, pass,
                     pass + 1 == sort_passes(a.V));
  return hipGetLastError();
}

// ------------------------------------------------------------------ gradient
namespace {

// Where a run's sum goes: to a row of sums (tied weights), to the table's
// gradient, or on top of it.  (Constants of the kernels: with the choice made
// where the sum is stored, the kernel's code was so long that fetching it took
// a small call 10 us.)
enum { kToSums, kToTable, kOnTable };

// Piece p of the slab of columns from the sum x of the run of token v that
// begins at entry `first`.
template <int SINK, int G>
__device__ inline void put_sum(const EmbedGradArgs& a, int64_t v, int64_t first, int p, const float (&x)[8]) {
  const int64_t n = a.cols - 8 * (int64_t)p;
  if (n <= 0) return;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = x[i] * a.scale;
  if constexpr (SINK == kToSums) {
    store8<kTypeF32>(reinterpret_cast<char*>(a.sums + first * a.cols + 8 * (int64_t)p), y, (int)n);
    if (p == 0) a.run_of[v] = (int32_t)first;
  } else {
    char* row = a.out + v * a.d * Elem<G>::kBytes;
    if constexpr (SINK == kOnTable) {
      float was[8];
      load_row<G>(row, a.d, p, was);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] += was[i];
    }
    store8<G>(row + 8 * (int64_t)p * Elem<G>::kBytes, y, (int)n);
  }
}

// launch(type, sink, gradient's type) as constants
template <class F>
void pick_sink(const EmbedGradArgs& a, F&& launch) {
  using std::integral_constant;
  if (a.tied) return launch(integral_constant<int, kToSums>(), integral_constant<int, kTypeF32>());
  pick_type(a.grad_type, [&](auto g) {
    if (a.accumulate) launch(integral_constant<int, kOnTable>(), g);
    else launch(integral_constant<int, kToTable>(), g);
  });
}

__device__ inline float* part_row(const EmbedGradArgs& a, int64_t piece, int which) {
  return a.part + (piece * 2 + which) * a.cols;
}
__device__ inline void put_part(const EmbedGradArgs& a, int64_t piece, int which, int p, const float (&x)[8]) {
  const int64_t n = a.cols - 8 * (int64_t)p;
  if (n > 0) store8<kTypeF32>(reinterpret_cast<char*>(part_row(a, piece, which) + 8 * (int64_t)p), x, (int)n);
}

// whether a token is among up to kSortChunk sorted ones, which carry no marks
__device__ inline bool occurs(const EmbedGradArgs& a, uint32_t v) {
  int lo = 0, hi = (int)a.T;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.key[mid] < v) lo = mid + 1; else hi = mid;
  }
  return lo < a.T && a.key[lo] == v;
}

__device__ inline uint32_t lane_of(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

}  // namespace

// Waves [0, pieces * slabs) add up, the waves behind them write zeros to the
// table's rows whose tokens do not occur, `fill` rows each.
template <int TY, int SINK, int G>
__global__ __launch_bounds__(256) void embed_grad_kernel(EmbedGradArgs a, int64_t pieces, int slabs, int fill) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = wave_in_grid();
  if (wave >= pieces * slabs) {
    if constexpr (SINK != kToTable) return;
    const int64_t v0 = (wave - pieces * slabs) * fill, v = v0 + lane;
    bool empty = lane < fill && v < a.V;
    if (empty) empty = a.T <= kSortChunk ? !occurs(a, (uint32_t)v) : a.run_of[v] < 0;
    const uint64_t rows = __ballot(empty);
    const int64_t bytes = a.d * Elem<G>::kBytes;
    int per = 64;  // lanes of a row: as many as its 16-byte pieces, to a power of two
    while (per > 1 && 8 * per >= bytes) per >>= 1;
    for (int r = lane / per; r < fill; r += 64 / per) {
      if (!(rows >> r & 1)) continue;
      char* row = a.out + (v0 + r) * bytes;
      int64_t at = 16 * (lane % per);
      for (; at + 16 <= bytes; at += 16 * per) store16(row + at, zero4());
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
  int from = 0;              // where it begins in this one
  constexpr int U = 8;
  for (int e = 0; e < ne; e += U) {
    Raw8<TY> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = min(e + u, ne - 1);
      const int64_t t = lane_of(poss, i);
      r[u] = load8<TY>(a.grad + (t * a.d + a.col0 + 8 * (int64_t)p) * Elem<TY>::kBytes,
                       lane_of(keys, i) < (uint32_t)a.V ? (int)(a.cols - 8 * (int64_t)p) : 0, p > 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (e + u >= ne) break;
      const uint32_t k = lane_of(keys, e + u);
      if (k != v) {
        if (first) put_part(a, piece, 0, p, x);
        else put_sum<SINK, G>(a, v, e0 + from, p, x);
        first = false;
        v = k;
        from = e + u;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
      }
      if (v >= (uint32_t)a.V) return;  // only entries that count for nothing from here on
      float y[8];
      settle8<TY>(r[u], (int)(a.cols - 8 * (int64_t)p), p > 0);
      unpack8<TY>(r[u], y);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] += y[i];
    }
  }
  if (first) put_part(a, piece, 0, p, x);
  else if (after == v) put_part(a, piece, 1, p, x);
  else put_sum<SINK, G>(a, v, e0 + from, p, x);
}

// A workgroup for each piece in which a run begins that goes on, and each
// slab: its partial rows in order, a quarter of them to each wave.
template <int SINK, int G>
__global__ __launch_bounds__(256) void embed_join_kernel(EmbedGradArgs a, int64_t pieces, int slabs) {
  __shared__ float sums[3][64 * 8];
  const int64_t piece = blockIdx.x / slabs;
  const int64_t e0 = piece * a.piece, e1 = e0 + a.piece;
  const int lane = threadIdx.x & 63, w = wave_id();
  const uint32_t v = a.key[e1 - 1], begin = e0 > 0 ? a.key[e0 - 1] : 0xffffffffu;
  if (v >= (uint32_t)a.V || begin == v) return;  // nothing, or it began before
  // the partial rows: this piece's last run, then the first runs of the pieces that begin with the token
  int64_t n = 1;
  for (;;) {
    const int64_t q = piece + n + lane;
    const uint64_t goes_on = __ballot(q < pieces && a.key[min(q * a.piece, a.T - 1)] == v);
    n += goes_on == ~uint64_t(0) ? 64 : __builtin_ctzll(~goes_on);
    if (goes_on != ~uint64_t(0)) break;
  }
  if (n == 1) return;
  const int p = (int)(blockIdx.x - piece * slabs) * 64 + lane;
  float x[8] = {};
  constexpr int U = 4;
  for (int64_t j = n * w / 4, end = n * (w + 1) / 4; j < end; j += U) {
    Raw8<kTypeF32> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t q = piece + min(j + u, n - 1);
      r[u] = load8<kTypeF32>(reinterpret_cast<const char*>(part_row(a, q, q == piece ? 1 : 0) + 8 * (int64_t)p),
                             j + u < end ? (int)(a.cols - 8 * (int64_t)p) : 0, p > 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float y[8];
      settle8<kTypeF32>(r[u], (int)(a.cols - 8 * (int64_t)p), p > 0);
      unpack8<kTypeF32>(r[u], y);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] += y[i];
    }
  }
  if (w > 0)
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[w - 1][i * 64 + lane] = x[i];
  __syncthreads();
  if (w > 0) return;
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] += sums[k][i * 64 + lane];
  int64_t first = e0;
  if constexpr (SINK == kToSums)
    if (begin != v) {  // the run's first entry in the piece
      int lo = 0, hi = a.piece - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.key[e0 + mid] < v) lo = mid + 1; else hi = mid;
      }
      first += lo;
    }
  put_sum<SINK, G>(a, v, first, p, x);
}

// Tied weights: 256 columns x kTurnK rows of the head's gradient a workgroup,
// from the runs' rows of sums, turned in LDS.  The columns whose tokens do not
// occur (most of them) are zeros there from the start.  Without accumulate
// whole rows are written, a kilobyte by each wave at once; with it only the
// columns whose tokens occur are read and written.  A tile of frequent tokens
// has up to 256 runs and is what the call waits for in the end: few rows a
// workgroup, and 16 loads of a thread in flight.
constexpr int kTurnV = 256, kTurnK = 16, kTurnLd = kTurnV + 4;

template <int G>
__global__ __launch_bounds__(256) void embed_turn_kernel(EmbedGradArgs a, int tiles) {
  __shared__ __attribute__((aligned(16))) float tile[kTurnK * kTurnLd];
  __shared__ int first[kTurnV], column[kTurnV], counts[4];
  const int tid = threadIdx.x, lane = tid & 63, w = wave_id();
  const int64_t v0 = (int64_t)(blockIdx.x % tiles) * kTurnV, k0 = (int64_t)(blockIdx.x / tiles) * kTurnK;
  const int rows = (int)min((int64_t)kTurnK, a.cols - k0);
  const int run = v0 + tid < a.V ? a.run_of[v0 + tid] : -1;  // the entry at which the column's run begins
  for (int i = tid; i < kTurnK * kTurnLd / 4; i += 256)
    reinterpret_cast<float4*>(tile)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  const uint64_t here = __ballot(run >= 0);
  if (lane == 0) counts[w] = __popcll(here);
  __syncthreads();
  int n = 0, before = __popcll(here & ((uint64_t(1) << lane) - 1));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < w) before += counts[i];
    n += counts[i];
  }
  if (a.accumulate && n == 0) return;
  if (run >= 0) {
    first[before] = run;
    column[before] = tid;
  }
  __syncthreads();
  const int k = tid % kTurnK;
  const float* const from = a.sums + k0 + min(k, rows - 1);
  constexpr int kStep = 256 / kTurnK;
  for (int j0 = tid / kTurnK; j0 < n; j0 += 16 * kStep) {
    float held[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) held[u] = from[(int64_t)first[min(j0 + u * kStep, n - 1)] * a.cols];
#pragma unroll
    for (int u = 0; u < 16; ++u)
      if (j0 + u * kStep < n) tile[k * kTurnLd + column[j0 + u * kStep]] = held[u];
  }
  __syncthreads();
  char* const out = a.out + ((a.col0 + k0) * a.V + v0) * Elem<G>::kBytes;
  const int64_t ld = a.V * Elem<G>::kBytes;
  if (a.accumulate) {
    if (run >= 0)
#pragma unroll 4
      for (int q = 0; q < rows; ++q) {
        char* to = out + q * ld + tid * Elem<G>::kBytes;
        Elem<G>::put1(to, Elem<G>::get1(to) + tile[q * kTurnLd + tid]);
      }
    return;
  }
  constexpr int kCols = 16 / Elem<G>::kBytes, kLanes = kTurnV / kCols;  // 64 lanes a row, or 32
  const int c = kCols * (tid % kLanes), left = (int)min((int64_t)kCols, a.V - v0 - c);
#pragma unroll
  for (int q = tid / kLanes; q < kTurnK; q += 256 / kLanes) {
    if (q >= rows || left <= 0) continue;
    const float* y = tile + q * kTurnLd + c;
    char* to = out + q * ld + c * Elem<G>::kBytes;
    if (left < kCols) {
      for (int i = 0; i < left; ++i) Elem<G>::put1(to + i * Elem<G>::kBytes, y[i]);
    } else if constexpr (G == kTypeF32) {
      store16(to, *reinterpret_cast<const u32x4_t*>(y));
    } else {
      const float4 p = *reinterpret_cast<const float4*>(y), r = *reinterpret_cast<const float4*>(y + 4);
      store16(to, u32x4_t{pack2x16<G>(p.x, p.y), pack2x16<G>(p.z, p.w), pack2x16<G>(r.x, r.y), pack2x16<G>(r.z, r.w)});
    }
  }
}

__global__ __launch_bounds__(256) void fill_table_kernel(char* p, int64_t bytes) {
  const int64_t n = bytes / 16, step = (int64_t)gridDim.x * 256;
  const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
  for (int64_t i = i0; i < n; i += step) store16(p + 16 * i, zero4());
  const int64_t tail = 16 * n + 2 * i0;
  if (tail < bytes) *reinterpret_cast<uint16_t*>(p + tail) = 0;
}

// Entries of a piece (up to as many tokens need no joining): short ones while
// there are few waves, long ones where the partial rows cost more.  us of the
// gradient, 16 / 64, bf16: V 128256, d 2048, T 4096 117 / 122, 16384 138 / 136, 32768
// 176 / 168, 131072 338 / 310; V 32000, d 512, T 4096 25 / 38, 16384 32 / 42, 32768 51 /
// 57, 65536 92 / 88, 131072 124 / 106.
int embed_piece(int64_t T) { return T <= 16384 ? 16 : 64; }

namespace {
struct GradShape {
  int64_t pieces;
  int slabs;
};
GradShape grad_shape(const EmbedGradArgs& a) {
  return {(a.T + a.piece - 1) / a.piece, (int)((a.cols + kSlab - 1) / kSlab)};
}
}  // namespace

hipError_t launch_embed_grad(const EmbedGradArgs& a, hipStream_t st) {
  const GradShape s = grad_shape(a);
  // table rows of a wave that writes zeros: about one round of the chip's waves (at most a lane each)
  const int fill = a.V >= 16 * kMostWaves ? 64 : (int)std::min<int64_t>(std::max<int64_t>(a.V / 8192, 1), 16);
  const int64_t more = a.tied || a.accumulate ? 0 : (a.V + fill - 1) / fill;
  const dim3 grid((unsigned)((s.pieces * s.slabs + more + 3) / 4));
  pick_type(a.type, [&](auto ty) {
    pick_sink(a, [&](auto sink, auto g) {
      hipLaunchKernelGGL((embed_grad_kernel<decltype(ty)::value, decltype(sink)::value, decltype(g)::value>), grid,
                         dim3(256), 0, st, a, s.pieces, s.slabs, fill);
    });
  });
  return hipGetLastError();
}
hipError_t launch_embed_join(const EmbedGradArgs& a, hipStream_t st) {
  const GradShape s = grad_shape(a);
  if (s.pieces == 1) return hipSuccess;
  pick_sink(a, [&](auto sink, auto g) {
    hipLaunchKernelGGL((embed_join_kernel<decltype(sink)::value, decltype(g)::value>),
                       dim3((unsigned)((s.pieces - 1) * s.slabs)), dim3(256), 0, st, a, s.pieces, s.slabs);
  });
  return hipGetLastError();
}
int64_t embed_turn_cols(int64_t V) { return std::max<int64_t>(kMostWaves / 2 / ((V + kTurnV - 1) / kTurnV), 1) * kTurnK; }
hipError_t launch_embed_turn(const EmbedGradArgs& a, hipStream_t st) {
  pick_type(a.grad_type, [&](auto ty) {
    constexpr int G = decltype(ty)::value;
    const int64_t tiles = (a.V + kTurnV - 1) / kTurnV, blocks = tiles * ((a.cols + kTurnK - 1) / kTurnK);
    hipLaunchKernelGGL((embed_turn_kernel<G>), dim3((unsigned)blocks), dim3(256), 0, st, a, (int)tiles);
  });
  return hipGetLastError();
}
hipError_t launch_fill_table(char* p, int64_t bytes, hipStream_t st) {
  const int64_t blocks = std::min<int64_t>(std::max<int64_t>((bytes / 16 + 255) / 256, 1), 8192);
  hipLaunchKernelGGL(fill_table_kernel, dim3((unsigned)blocks), dim3(256), 0, st, p, bytes);
  return hipGetLastError();
}

}  // namespace kd
