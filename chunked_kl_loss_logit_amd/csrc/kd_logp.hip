// Token log-probabilities through the output head, their entropy and dZ.
//
//   s = z / tau with z = H_t . W, L_t = logsumexp(s), q = softmax(s)
//   logp_t = s[y_t] - L_t           ent_t = L_t - sum_v q_v s_v
//   dZ_t   = (1/tau) (g_t [v = y_t] - q_v (g_t + e_t (ent_t + log q_v)))
//
// Grid: (256 valid rows) x (vocabulary split).  A workgroup walks the
// 256-column tiles of its split; the tile's products are accumulated
// transposed (mma_frags_t), so a lane holds 64 columns of each of four rows
// and both epilogues work in registers.
//   forward: per lane and row a running (m, l, e): m the maximum of y = s
//     log2(e), l = sum 2^(y - m), e = sum 2^(y - m) (y - m).  e is kept
//     relative to the maximum, so the entropy ln2 (log2 l - e / l) is a
//     difference of small numbers whatever the size of the logits.  Moving
//     the maximum by dm <= 0 (old minus new) scales: l' = l 2^dm,
//     e' = (e + dm l) 2^dm.
//   backward: each register becomes its dZ.
// The tile contraction (2 T d V flops) bounds both; without the entropy its
// terms are compiled out.  Measured, T 4096, d 2048, V 128256 (2.15 TFLOP a
// product): forward with the entropy 1.69 ms (1.28 PFLOP/s), with kept logits
// (2.1 GB written) 1.99 ms, dZ 1.79 ms (1.20 PFLOP/s), dZ from kept logits 0.66
// ms (4.8 TB/s), dH 1.60 ms (1.34 PFLOP/s), dW in bf16 1.65 ms (1.30 PFLOP/s);
// a torch product of 8192^3 reaches 1.15 PFLOP/s.
#include <type_traits>

#include "kd_gemm.h"
#include "kd_main.h"
#include "kd_policy.h"

namespace kd {

namespace {

constexpr int kBN = kTileN;
constexpr int kStgBytes = 2048;        // per wave: 32 rows x 64 bytes of dZ, or 16 x 128 of logits
constexpr int kFstWords = 4 * 4 * 64;  // per wave: (m, l, e, x) of 4 rows x 64 lanes

// The ring takes whole tiles only (V >= 256): a last partial tile is shifted
// left to end at V, and its first columns, up to the tile's own lo, were the
// previous tile's.
__device__ inline int tile_n0(int vt, int V) { return min(vt * kBN, V - kBN); }

// The forward product's operands.  The contraction runs over d rounded up to
// whole ring turns (128): the panels of H hold zeros there, and W's stages
// past d (a multiple of 32) read its last one again.
struct LogpMain : DmaNN<kBN> {
  int b_last;
  template <class RowPtr>
  __device__ inline void open(const char* hp, RowPtr&& row, const char* W, long V, long d, long C) {
    init(hp, row, W, V * 2, V, (d + kDmaKMult - 1) / kDmaKMult * kDmaKMult, (uint32_t)(C * kRowB));
    b_last = (int)(d / kDmaKs) - 1;
    b.init(W, LONG_MAX);
  }
  // transposed accumulators of tiles n0(0) .. n0(ntiles - 1)
  template <class N0, class Done>
  __device__ inline void tiles(const Slots& sl, int ntiles, N0&& n0, Done&& done) {
    f32x16_t acc[4][kBN / 64];
    ring_run<kLpw, FragsNN<kBN>>(
        sl, ntiles, nst,
        [&](long t, int s, char* da, char* db) {
          a.issue(s, da);
          b.issue(min(s, b_last), (long)n0((int)t), db);
        },
        [&](const char* slot, FragsNN<kBN>& f) { rd.read_nn(slot, f); },
        [&](const FragsNN<kBN>& f) { mma_frags_t(f, acc); },
        [&](const FragsNN<kBN>& f) { mma_frags_first<true>(f, acc); }, [&](int t) { done(t, acc); });
  }
};

// Byte position of 8 bytes (half hh of 16-byte chunk j) of row r in a wave's
// [32][64 B] staging region: chunk and half XOR-swizzled, so the 32 rows that
// a half-wave writes at once land in distinct bank groups, and so do the
// 4 x 4 chunks a quarter-wave reads back.
__device__ inline int stg8(int r, int j, int hh) {
  return r * 64 + ((j ^ ((r >> 2) & 3)) << 4) + ((hh ^ ((r >> 4) & 1)) << 3);
}

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
__device__ inline uint32_t pk_bf16(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{lo, hi}, bf16x2_t));
}

// (m, l, e) parts of one row over two column sets, merged; m = -inf: nothing yet
template <bool kEnt>
__device__ inline void merge(float& m, float& l, float& e, float om, float ol, float oe) {
  const float M = fmaxf(m, om);
  const float d = m - M, od = om - M;
  const float f = m == -INFINITY ? 0.f : fast_exp2(d), of = om == -INFINITY ? 0.f : fast_exp2(od);
  if constexpr (kEnt)
    e = (m == -INFINITY ? 0.f : f * fmaf(at_least(d), l, e)) + (om == -INFINITY ? 0.f : of * fmaf(at_least(od), ol, oe));
  l = l * f + ol * of;
  m = M;
}

// One row's update from the lane's 64 values of the tile (register i of
// block nb: column base + 32 nb + 8 (i / 4) + 4 h + i % 4).  Columns below lo
// (a multiple of 8) are left out unless kFull.
template <bool kEnt, bool kFull>
__device__ inline void fwd_row(const f32x16_t (&v)[4], float c2, float* st, int label, int base, int lo) {
  const int h = (opaque((int)threadIdx.x) >> 5) & 1;
  float m = st[0], l = st[64];
  auto in = [&](int nb, int i) {
    const int col = base + 32 * nb + 8 * (i >> 2) + 4 * h;
    return kFull || col >= lo;
  };
  float cm = -INFINITY;
#pragma unroll
  for (int nb = 0; nb < 4; ++nb)
#pragma unroll
    for (int i = 0; i < 16; ++i) cm = in(nb, i) ? fmaxf(cm, v[nb][i]) : cm;
  const float cmy = top_of(cm, c2);
  float e = 0.f;
  if constexpr (kEnt) e = st[128];
  if (cmy > m) {
    const float f = fast_exp2(m - cmy);  // 2^(-inf) = 0 while nothing is summed yet
    if constexpr (kEnt) e = l == 0.f ? 0.f : f * fmaf(at_least(m - cmy), l, e);
    l *= f;
    m = cmy;
  }
  float sum = 0.f, es = 0.f;
  const float from = subtrahend(m);
#pragma unroll
  for (int nb = 0; nb < 4; ++nb)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float w = in(nb, i) ? fmaf(v[nb][i], c2, -from) : -256.f;
      const float p = fast_exp2(w);
      sum += p;
      if constexpr (kEnt) es = fmaf(p, at_least(w), es);
    }
  st[0] = m;
  st[64] = l + sum;
  if constexpr (kEnt) st[128] = e + es;
  const int dc = label - base;
  if ((unsigned)dc < 128u && label >= lo && ((dc >> 2) & 1) == h) {
    const int nbl = dc >> 5, at = ((dc >> 3 & 3) << 2) | (dc & 3);
    float z = 0.f;
#pragma unroll
    for (int nb = 0; nb < 4; ++nb)
#pragma unroll
      for (int i = 0; i < 16; ++i) z = nb == nbl && i == at ? v[nb][i] : z;
    st[192] = z;
  }
}

// The raw logits of one 32 x 32 block (the columns from lo on, rows below M),
// fp32, through a wave-private 2 KB LDS region, 16 rows at a time: a store
// instruction then writes 8 rows of 128 contiguous bytes.  Straight from the
// registers it would touch 32 rows of 32 bytes, and the next tile's operand
// loads, which complete in order behind it, wait for four times the requests.
__device__ inline void zout_block(const f32x16_t& v, char* stg, float* zout, long ldz, int brow0, long M, int cb,
                                  int lo) {
  const int lane = opaque((int)threadIdx.x) & 63, h = lane >> 5, r16 = lane & 15;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    if (((lane >> 4) & 1) == p) {
#pragma unroll
      for (int j = 0; j < 4; ++j)  // 16-byte chunk 2 j + h of the row, swizzled against bank conflicts
        *reinterpret_cast<float4*>(stg + r16 * 128 + 16 * ((2 * j + h) ^ (r16 & 7))) =
            make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = 8 * k + (lane >> 3), c = lane & 7;
      const float4 x = *reinterpret_cast<const float4*>(stg + r * 128 + 16 * (c ^ (r & 7)));
      const int row = brow0 + 16 * p + r, col = cb + 4 * c;
      if (row < M && col >= lo) *reinterpret_cast<float4*>(zout + (long)row * ldz + col) = x;
    }
  }
}

}  // namespace

// ------------------------------------------------------------------ forward tiles
template <bool kEnt, bool kOut>
__global__ __launch_bounds__(kThreads, 1) void logp_fwd_kernel(LogpFwdArgs a) {
  __shared__ __attribute__((aligned(16))) char sl_0[kSlotBytes];
  __shared__ __attribute__((aligned(16))) char sl_1[kSlotBytes];
  __shared__ __attribute__((aligned(16))) char sl_2[kSlotBytes];
  __shared__ __attribute__((aligned(16))) char sl_3[kSlotBytes];
  __shared__ float fst_all[4 * kFstWords];
  __shared__ int labk[kBM];
  __shared__ __attribute__((aligned(16))) char stg_all[kOut ? 4 * kStgBytes : 16];
  const Slots sl{sl_0, sl_1, sl_2, sl_3, nullptr};

  const long count = *a.c.count;
  const long M = min(a.C, count - a.c0);  // valid rows of the chunk
  if (M <= 0) return;
  const int nrb = (int)((M + kBM - 1) / kBM), S = ring_splits(M, a.ntiles, a.grid);
  if ((int)blockIdx.x >= nrb * S) return;
  int rb, sp;
  grouped_coords(xcd_remap(blockIdx.x, nrb * S), nrb, S, a.group, rb, sp);
  const int row0 = rb * kBM;
  const int tb = (int)((long)a.ntiles * sp / S);
  const int te = (int)((long)a.ntiles * (sp + 1) / S);
  const int V = (int)a.V;

  LogpMain mainloop;
  mainloop.open(
      a.Hp, [&](int r) -> const char* { return row0 + r < M ? a.Hp + (row0 + r) * kRowB : nullptr; }, a.W, a.V, a.d,
      a.C);

  const int w = wave_id(), wm = w >> 1, wn = w & 1;
  const int lane = (int)threadIdx.x & 63;
  const int trow0 = wm * 128;
  float* fst = fst_all + w * kFstWords;
#pragma unroll
  for (int mb = 0; mb < 4; ++mb) {
    const int ti = row0 + trow0 + mb * 32 + (lane & 31);
    if (wn == 0 && lane < 32)
      labk[trow0 + mb * 32 + lane] = ti < M ? (int)((long)a.tokens[a.c.rows[a.c0 + ti]] - a.v0) : -1;
    fst[mb * 256 + lane] = -INFINITY;
    fst[mb * 256 + 64 + lane] = 0.f;
    fst[mb * 256 + 128 + lane] = 0.f;
    fst[mb * 256 + 192 + lane] = 0.f;
  }

  mainloop.tiles(
      sl, te - tb, [&](int i) { return tile_n0(tb + i, V); },
      [&](int i, const f32x16_t (&acc)[4][4]) {
        const int vt = tb + i, n0 = tile_n0(vt, V), lo = vt * kBN;
        const int base = n0 + wn * 128;
        const int ln = opaque((int)threadIdx.x) & 63;
        const bool full = n0 == lo;
#pragma unroll
        for (int mb = 0; mb < 4; ++mb) {
          float* st = fst + mb * 256 + ln;
          const int label = labk[trow0 + mb * 32 + (ln & 31)];
          if (full)
            fwd_row<kEnt, true>(acc[mb], a.c2, st, label, base, lo);
          else
            fwd_row<kEnt, false>(acc[mb], a.c2, st, label, base, lo);
        }
        if constexpr (kOut) {  // the logits last: a register spilled before them would wait for their stores
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int mb = 0; mb < 4; ++mb)
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) {
              zout_block(acc[mb][nb], stg_all + w * kStgBytes, a.zout, a.ldz, row0 + trow0 + mb * 32, M, base + 32 * nb,
                         lo);
              __builtin_amdgcn_sched_barrier(0);
            }
        }
      });

  // the split's record per row: lane halves, then column halves (wave wn = 1
  // hands its part to wave wn = 0 through slot 0, free after the ring)
  __syncthreads();
  float4* xch = reinterpret_cast<float4*>(sl_0);
#pragma unroll
  for (int mb = 0; mb < 4; ++mb) {
    float m = fst[mb * 256 + lane], l = fst[mb * 256 + 64 + lane], e = fst[mb * 256 + 128 + lane];
    float x = fst[mb * 256 + 192 + lane];
    const float om = __shfl_xor(m, 32), ol = __shfl_xor(l, 32), oe = __shfl_xor(e, 32), ox = __shfl_xor(x, 32);
    if (lane < 32) merge<kEnt>(m, l, e, om, ol, oe);
    x += ox;
    if (wn == 1 && lane < 32) xch[trow0 + mb * 32 + lane] = make_float4(m, l, e, x);
    fst[mb * 256 + lane] = m;
    fst[mb * 256 + 64 + lane] = l;
    fst[mb * 256 + 128 + lane] = e;
    fst[mb * 256 + 192 + lane] = x;
  }
  __syncthreads();
  if (wn == 0 && lane < 32) {
#pragma unroll
    for (int mb = 0; mb < 4; ++mb) {
      const int ti = row0 + trow0 + mb * 32 + lane;
      if (ti >= M) continue;
      float m = fst[mb * 256 + lane], l = fst[mb * 256 + 64 + lane], e = fst[mb * 256 + 128 + lane];
      const float4 o = xch[trow0 + mb * 32 + lane];
      merge<kEnt>(m, l, e, o.x, o.y, o.z);
      float4* dst = reinterpret_cast<float4*>(a.part) + (long)sp * a.C + ti;
      *dst = make_float4(m, l, e, fst[mb * 256 + 192 + lane] + o.w);
    }
  }
}

// ------------------------------------------------------------------ per-row outputs
namespace {

// S records at stride `stride`, merged in order.
__device__ inline float4 merge_records(const float4* pp, int S, long stride) {
  float M = -INFINITY;
  for (int s = 0; s < S; ++s) M = fmaxf(M, pp[s * stride].x);
  float l = 0.f, e = 0.f, x = 0.f;
  for (int s = 0; s < S; ++s) {
    const float4 q = pp[s * stride];
    const float dm = q.x - M, f = exp2f(dm);
    l = fmaf(q.y, f, l);
    if (q.x != -INFINITY) e = fmaf(f, fmaf(at_least(dm), q.y, q.z), e);
    x += q.w;
  }
  return make_float4(M, l, e, x);
}

// logp = ln2 ((y at the token - m) - log2 l): the maximum goes out first, so
// only the small log2 l is subtracted from the row's distance to its maximum.
// (In halves: in base 2 the log-probability of a column masked by the type's
// lowest value passes the 32-bit range, in base e it does not.)  A row of
// nothing but columns below the 32-bit range (l = 0) is NaN.
__device__ inline void finish_row(long t, const float4 r, float c2, const LogpOut& o) {
  const float ll = r.y > 0.f ? log2f(r.y) : NAN;
  o.logp[t] = 2.f * kLn2 * (fmaf(0.5f * r.w, c2, -0.5f * r.x) - 0.5f * ll);
  o.lse[t] = kLn2 * (r.x + ll);
  if (o.entropy) o.entropy[t] = kLn2 * (ll - r.z / r.y);
}

__device__ inline void zero_row(long t, const LogpOut& o) {
  if (o.rec) {
    o.rec[t] = make_float4(0.f, 0.f, 0.f, 0.f);
    return;
  }
  o.logp[t] = 0.f;
  o.lse[t] = 0.f;
  if (o.entropy) o.entropy[t] = 0.f;
}

}  // namespace

// One wave per row of the chunk: lanes merge every 64th record, then each
// other (a row has up to a thousand records; one thread walking them took as
// long as the tiles did for a few rows).  With zero_masked, threads also zero
// the outputs of masked rows.
template <bool kEnt>
__global__ __launch_bounds__(256) void logp_combine_kernel(const float4* part, int S, int grid, RowSet rs, const uint8_t* mask,
                                                           const int32_t* tokens, int V, float c2, LogpOut o,
                                                           int zero_masked) {
  const int lane = threadIdx.x & 63;
  const long j = (long)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (zero_masked && mask != nullptr)
    for (long t = (long)blockIdx.x * 256 + threadIdx.x; t < rs.T; t += (long)gridDim.x * 256)
      if (mask[t] == 0) zero_row(t, o);
  const long M = rs.rows ? min((long)rs.C, (long)*rs.count - (long)rs.c0) : min((long)rs.C, (long)(rs.T - rs.c0));
  if (j >= M) return;
  if (grid > 0) S = ring_splits(M, S, grid);
  float m = -INFINITY, l = 0.f, e = 0.f, x = 0.f;
  for (int s = lane; s < S; s += 64) {
    const float4 q = part[(long)s * rs.C + j];
    merge<kEnt>(m, l, e, q.x, q.y, q.z);
    x += q.w;
  }
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) {
    const float om = __shfl_xor(m, k), ol = __shfl_xor(l, k), oe = __shfl_xor(e, k);
    merge<kEnt>(m, l, e, om, ol, oe);
    x += __shfl_xor(x, k);
  }
  if (lane != 0) return;
  const long t = rs.rows ? rs.rows[rs.c0 + j] : rs.c0 + j;
  if (o.rec) {
    o.rec[t] = make_float4(m, l, e, x);
    return;
  }
  if ((uint32_t)tokens[t] >= (uint32_t)V) x = NAN;  // no such token: loud, not a plausible number
  finish_row(t, make_float4(m, l, e, x), c2, o);
}

hipError_t launch_logp_combine(const float* part, int S, int grid, const RowSet& rs, const uint8_t* mask,
                               const int32_t* tokens, int64_t V, float c2, const LogpOut& o, bool zero_masked,
                               hipStream_t st) {
  const int64_t n = rs.C < rs.T - rs.c0 ? rs.C : rs.T - rs.c0;
  const dim3 blocks((unsigned)((n + 3) / 4));
  const float4* p = reinterpret_cast<const float4*>(part);
  if (o.rec || o.entropy)
    hipLaunchKernelGGL(logp_combine_kernel<true>, blocks, dim3(256), 0, st, p, S, grid, rs, mask, tokens, (int)V, c2, o,
                       zero_masked ? 1 : 0);
  else
    hipLaunchKernelGGL(logp_combine_kernel<false>, blocks, dim3(256), 0, st, p, S, grid, rs, mask, tokens, (int)V, c2, o,
                       zero_masked ? 1 : 0);
  return hipGetLastError();
}

__global__ __launch_bounds__(256) void logp_shard_combine_kernel(const float4* rec, int R, long T, const uint8_t* mask,
                                                                 float c2, LogpOut o) {
  const long t = (long)blockIdx.x * blockDim.x + threadIdx.x;
  if (t >= T) return;
  if (mask != nullptr && mask[t] == 0) {
    zero_row(t, o);
    return;
  }
  finish_row(t, merge_records(rec + t, R, T), c2, o);
}

hipError_t launch_logp_shard_combine(const float4* rec, int R, int64_t T, const uint8_t* mask, float c2,
                                     const LogpOut& o, hipStream_t st) {
  hipLaunchKernelGGL(logp_shard_combine_kernel, dim3((unsigned)((T + 255) / 256)), dim3(256), 0, st, rec, R, (long)T,
                     mask, c2, o);
  return hipGetLastError();
}

// ------------------------------------------------------------------ dZ tiles
namespace {

// What dZ of a row needs: L2 = lse log2(e), A = ga + ge ent, B = ge ln2, ga,
// c2 and the token's column.  Rows past the chunk's valid rows get zeros, c2
// included, so whatever their products hold their dZ is 0.
struct DzRow {
  float4 k;  // (L2, A, B, ga)
  float c2;
  int label;
};
__device__ inline DzRow dz_row(const LogpDzArgs& a, bool rv, long t) {
  DzRow r{make_float4(0.f, 0.f, 0.f, 0.f), 0.f, -1};
  if (!rv) return r;
  const float ga = a.g ? a.g[t] * a.inv_tau : 0.f;
  const float gb = a.ge ? a.ge[t] * a.inv_tau : 0.f;
  r.k = make_float4(a.lse[t] * kLog2e, a.ge ? fmaf(gb, a.ent[t], ga) : ga, gb * kLn2, ga);
  r.c2 = a.c2;
  r.label = (int)((long)a.tokens[t] - a.v0);
  return r;
}
// -q (A + B log2 q)
template <bool kEnt>
__device__ inline float dz_value(float z, const float4 k, float c2) {
  const float lq = fmaf(z, c2, -k.x);
  const float q = fast_exp2(lq);
  if constexpr (kEnt) return -q * fmaf(k.z, at_least(lq), k.y);
  return -q * k.y;
}

// One 32 x 32 block: dZ of the lane's row at its 16 columns, to the chunk's
// panels.  Columns below lo belong to the previous tile and are not stored.
// The block goes through a wave-private 2 KB LDS region (LDS accesses of one
// wave complete in order: no barrier), so that a store instruction writes 16
// consecutive rows of one 64-byte piece.  tail (nullable): the block ends at
// V inside a piece; the columns from V rounded down to 32 on go out again in
// the tail piece (logp_dh_kernel), the others there as zeros.
template <bool kEnt, bool kFull>
__device__ inline void dz_block(const f32x16_t& v, const float4 k, float c2, int label, int cb, int lo, char* stg,
                                char* dz, long C, long brow0, char* tail, int tail0) {
  const int lane = opaque((int)threadIdx.x) & 63, h = lane >> 5, cl = lane & 31;
  float o[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = dz_value<kEnt>(v[i], k, c2);
  const int dc = label - cb;
  if ((unsigned)dc < 32u && ((dc >> 2) & 1) == h) {
    const int at = ((dc >> 3) << 2) | (dc & 3);
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = i == at ? o[i] + k.w : o[i];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint2*>(stg + stg8(cl, j, h)) =
        make_uint2(pk_bf16(o[4 * j], o[4 * j + 1]), pk_bf16(o[4 * j + 2], o[4 * j + 3]));
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    const int r = kk * 16 + (lane >> 2), j = lane & 3;
    const uint4 q = *reinterpret_cast<const uint4*>(stg + r * 64 + ((j ^ ((r >> 2) & 3)) << 4));
    const uint4 x = ((r >> 4) & 1) ? make_uint4(q.z, q.w, q.x, q.y) : q;  // halves stored exchanged
    const int col = cb + 8 * j;
    if (kFull || col >= lo) *reinterpret_cast<uint4*>(dz + panel_off(C, brow0 + r, (long)col * 2)) = x;
    if (!kFull && tail)
      *reinterpret_cast<uint4*>(tail + (brow0 + r) * kRowB + 16 * j) = col >= tail0 ? x : make_uint4(0, 0, 0, 0);
  }
}

}  // namespace

template <bool kEnt>
__global__ __launch_bounds__(kThreads, 1) void logp_dz_kernel(LogpDzArgs a) {
  __shared__ __attribute__((aligned(16))) char sl_0[kSlotBytes];
  __shared__ __attribute__((aligned(16))) char sl_1[kSlotBytes];
  __shared__ __attribute__((aligned(16))) char sl_2[kSlotBytes];
  __shared__ __attribute__((aligned(16))) char sl_3[kSlotBytes];
  __shared__ __attribute__((aligned(16))) char stg_all[4 * kStgBytes];
  __shared__ __attribute__((aligned(16))) float4 rowk[kBM];
  __shared__ __attribute__((aligned(8))) float2 rowc[kBM];
  const Slots sl{sl_0, sl_1, sl_2, sl_3, nullptr};

  const long count = *a.c.count;
  const long M = min(a.C, count - a.c0);
  if (M <= 0) return;
  const int nrb = (int)((M + kBM - 1) / kBM), S = ring_splits(M, a.ntiles, a.grid);
  if ((int)blockIdx.x >= nrb * S) return;
  int rb, sp;
  grouped_coords(xcd_remap(blockIdx.x, nrb * S), nrb, S, a.group, rb, sp);
  const int row0 = rb * kBM;
  const int tb = (int)((long)a.ntiles * sp / S);
  const int te = (int)((long)a.ntiles * (sp + 1) / S);
  const int V = (int)a.V;

  LogpMain mainloop;
  mainloop.open(
      a.Hp, [&](int r) -> const char* { return row0 + r < M ? a.Hp + (row0 + r) * kRowB : nullptr; }, a.W, a.V, a.d,
      a.C);

  {
    const int i = (int)threadIdx.x;
    const bool rv = row0 + i < M;
    const DzRow r = dz_row(a, rv, rv ? a.c.rows[a.c0 + row0 + i] : 0);
    rowk[i] = r.k;
    rowc[i] = make_float2(r.c2, __int_as_float(r.label));
  }
  __syncthreads();
  const int w = wave_id(), wm = w >> 1, wn = w & 1;
  const int trow0 = wm * 128;
  char* stg = stg_all + w * kStgBytes;

  mainloop.tiles(
      sl, te - tb, [&](int i) { return tile_n0(tb + i, V); },
      [&](int i, const f32x16_t (&acc)[4][4]) {
        const int vt = tb + i, n0 = tile_n0(vt, V), lo = vt * kBN;
        const int base = n0 + wn * 128;
        const bool full = n0 == lo;
        const int ln = opaque((int)threadIdx.x) & 31;
#pragma unroll
        for (int mb = 0; mb < 4; ++mb) {
          const float4 k = rowk[trow0 + mb * 32 + ln];
          const float2 cc = rowc[trow0 + mb * 32 + ln];
          const int label = __float_as_int(cc.y);
#pragma unroll
          for (int nb = 0; nb < 4; ++nb) {
            const int cb = base + 32 * nb;
            if (full)
              dz_block<kEnt, true>(acc[mb][nb], k, cc.x, label, cb, lo, stg, a.dz, a.C, row0 + trow0 + mb * 32, nullptr,
                                   0);
            else
              dz_block<kEnt, false>(acc[mb][nb], k, cc.x, label, cb, lo, stg, a.dz, a.C, row0 + trow0 + mb * 32,
                                    V % 32 && cb + 32 == V ? a.dz + a.ldz / 32 * a.C * kRowB : nullptr, V / 32 * 32);
          }
        }
      });
}

// ------------------------------------------------------------------ dZ from stored logits
// A block covers 64 rows and one range of the rows' 64-byte dZ pieces, four
// threads per piece: a wave writes 16 consecutive rows of a piece, a
// contiguous kilobyte of the panels.  Rows past the chunk's valid rows, up
// to the end of the chunk, get zeros.
constexpr int kFzRows = 64, kFzRanges = 64;

template <bool kEnt>
__global__ __launch_bounds__(256) void logp_dz_from_z_kernel(LogpDzArgs a) {
  constexpr int EPT = Bf16::kEpc;
  constexpr int PC = kRowB / 2;  // columns per piece
  const long i = (long)blockIdx.y * kFzRows + (threadIdx.x >> 2);
  const int sub = threadIdx.x & 3;
  const long np = (a.V * 2 + kRowB - 1) / kRowB;
  const long pb = np * blockIdx.x / gridDim.x, pe = np * (blockIdx.x + 1) / gridDim.x;
  const long M = min(a.C, (long)*a.c.count - a.c0);
  const bool rv = i < M;
  const DzRow r = dz_row(a, rv, rv ? a.c.rows[a.c0 + i] : 0);
  const float* zr = a.z + i * a.ldz;
  for (long p = pb; p < pe; ++p) {
    const long v0 = p * PC + sub * EPT;
    if (v0 >= a.V) break;
    float o[EPT];
#pragma unroll
    for (int q = 0; q < EPT; ++q) o[q] = 0.f;
    if (rv) {
#pragma unroll
      for (int e = 0; e < EPT; e += 4) {
        const float4 z4 = *reinterpret_cast<const float4*>(zr + v0 + e);
        o[e + 0] = dz_value<kEnt>(z4.x, r.k, r.c2);
        o[e + 1] = dz_value<kEnt>(z4.y, r.k, r.c2);
        o[e + 2] = dz_value<kEnt>(z4.z, r.k, r.c2);
        o[e + 3] = dz_value<kEnt>(z4.w, r.k, r.c2);
      }
#pragma unroll
      for (int q = 0; q < EPT; ++q) o[q] = (long)r.label == v0 + q ? o[q] + r.k.w : o[q];
    }
    const u32x4_t x = pack16<Bf16>(o);
    *reinterpret_cast<u32x4_t*>(a.dz + panel_off(a.C, i, v0 * 2)) = x;
    if (a.V % 32 && v0 >= a.V - 32) {  // the tail piece: columns V - 32 .. V - 1 (logp_dh_kernel)
      char* tail = a.dz + (a.ldz / 32 * a.C + i) * kRowB;
      *reinterpret_cast<u32x4_t*>(tail + (v0 - (a.V - 32)) * 2) = v0 >= a.V / 32 * 32 ? x : zero4();
    }
  }
}

// ------------------------------------------------------------------ dH
// dz . W^T over the vocabulary: 256 rows x 256 of d, S ranges of whole ring
// turns, each into its own float32 part (summed in order afterwards).  Both
// operands are contiguous along the vocabulary and come 32 columns a stage:
//   stages 0 .. V/32 - 1          dz piece s,          W columns 32 s ..
//   one more where V % 32 != 0    dz's tail piece,     W columns V - 32 .. V - 1
//   to the end of the last turn   zero pieces of dz,   W's first columns
// so W is never read past a row's end; the pieces after dz's own ldz / 32
// hold the tail and the zeros (kDzTailPieces).
namespace {

struct DhMain : DmaNT<256> {
  int full, tail, tail_piece;
  long tail_at;  // bytes to W's last 32 columns
  __device__ inline void tile(const Slots& sl, long s0, long s1, f32x16_t (&acc)[4][4]) {
    zero_acc<4>(acc);
    ring_contract<kLpw, FragsRows<256>>(
        sl, (int)(s1 - s0),
        [&](long s, char* da, char* db) {
          const int t = (int)(s0 + s);
          a.issue((long)(t < full ? t : t - full + tail_piece), da);
          b.issue(0L, t < full ? (long)t * kRowB : t < full + tail ? tail_at : 0L, db);
        },
        [&](const char* slot, FragsRows<256>& f) { rd.read_rows(slot, f); },
        [&](const FragsRows<256>& f) { mma_frags(f, acc); });
  }
};

}  // namespace

// How the grid is divided: whole 256-row blocks of valid rows, 256-wide
// blocks of d, and as many vocabulary ranges as workgroups are left for (the
// mask's rows are only counted here, as for ring_splits).  A range's part
// holds the valid row blocks' rows.
struct DhShape {
  int nrb, S;
  long rows;  // of a part
};
__device__ inline DhShape dh_shape(const LogpDhArgs& a, long M) {
  const int nrb = (int)((M + kBM - 1) / kBM);
  const int ng = (int)((a.V + 32 * kRing - 1) / (32 * kRing));
  const int s = nrb > 0 ? a.grid / (nrb * a.ncb) : 1;
  return {nrb, max(1, min(s, ng)), (long)nrb * kBM};
}

template <bool kTail>
__global__ __launch_bounds__(kThreads, 1) void logp_dh_kernel(LogpDhArgs a) {
  KD_DECLARE_SLOTS(sl);
  const long M = min((long)a.C, (long)*a.count - (long)a.c0);
  if (M <= 0) return;
  const DhShape sh = dh_shape(a, M);
  const int per_split = sh.nrb * a.ncb;
  if ((int)blockIdx.x >= per_split * sh.S) return;
  const int logical = xcd_remap(blockIdx.x, per_split * sh.S);
  const int sp = logical / per_split;
  int rb, cb;
  grouped_coords(logical - sp * per_split, sh.nrb, a.ncb, a.group, rb, cb);
  const long row0 = (long)rb * kBM, n0 = (long)cb * 256;
  std::conditional_t<kTail, DhMain, DmaNT<256>> mainloop;
  mainloop.init(a.dz, [&](int r) -> const char* { return row0 + r < M ? a.dz + (row0 + r) * kRowB : nullptr; },
                a.W, [&](int r) -> const char* { return n0 + r < a.d ? a.W + (n0 + r) * a.V * 2 : nullptr; }, a.V,
                a.C * kRowB);
  if constexpr (kTail) {
    mainloop.full = (int)(a.V / 32);
    mainloop.tail = a.V % 32 ? 1 : 0;
    mainloop.tail_piece = (int)(a.ldz / 32);
    mainloop.tail_at = (a.V - 32) * 2;
  }
  const long ng = (a.V + 32 * kRing - 1) / (32 * kRing);
  f32x16_t acc[4][4];
  mainloop.tile(sl, ng * sp / sh.S * kRing, ng * (sp + 1) / sh.S * kRing, acc);
  float* dst = a.part + (long)sp * sh.rows * a.d;
  const StPair s0 = st_pair<0>(sl), s1 = st_pair<1>(sl);
  auto round = [&](auto nb) {
    constexpr int NBI = decltype(nb)::value;
    stage_block<NBI, 4>(s0, s1, acc);
    __syncthreads();
    rmw_pair_f32(s0, s1, dst, a.d, row0, n0 + NBI * 32, n0 + 128 + NBI * 32, M, a.d, false);
    __syncthreads();
  };
  round(std::integral_constant<int, 0>());
  round(std::integral_constant<int, 1>());
  round(std::integral_constant<int, 2>());
  round(std::integral_constant<int, 3>());
}

// dH of the valid rows = their parts added in order; four elements per thread.
template <int ELEM>
__global__ __launch_bounds__(256) void logp_dh_reduce_kernel(LogpDhArgs a, const int32_t* rows, char* dH) {
  const long M = min((long)a.C, (long)*a.count - (long)a.c0);
  const long q = (long)blockIdx.x * 256 + threadIdx.x, d4 = a.d / 4;
  const long i = q / d4, j = (q - i * d4) * 4;
  if (i >= M) return;
  const DhShape sh = dh_shape(a, M);
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < sh.S; ++s) {
    const float4 y = *reinterpret_cast<const float4*>(a.part + ((long)s * sh.rows + i) * a.d + j);
    x.x += y.x;
    x.y += y.y;
    x.z += y.z;
    x.w += y.w;
  }
  char* p = dH + ((long)rows[a.c0 + i] * a.d + j) * ELEM;
  if constexpr (ELEM == 2)
    *reinterpret_cast<uint2*>(p) = make_uint2(pk_bf16(x.x, x.y), pk_bf16(x.z, x.w));
  else
    *reinterpret_cast<float4*>(p) = x;
}

// ------------------------------------------------------------------ dW in bf16
// H^T . dz over the chunk's rows, one 256 x 256 tile per workgroup, rounded
// once: the transposed accumulators give four consecutive columns per
// register group, the whole tile goes through LDS as bf16 (128 KB, the ring's
// four slots, 64 rows each) and leaves in rows of 512 contiguous bytes.
// 16-byte chunk c of row r sits at c ^ (r % 32), so neither the writes of 32
// rows at once nor the reads of whole rows collide.
__global__ __launch_bounds__(kThreads, 1) void logp_dw_bf16_kernel(DwArgs a, char* out) {
  KD_DECLARE_SLOTS(sl);
  const long M = max(0L, min(a.C, (long)*a.count - a.c0));
  int rb, cb;
  grouped_coords(xcd_remap(blockIdx.x, gridDim.x), a.nrb, a.ncb, a.group, rb, cb);
  const long row0 = (long)rb * kBM, n0 = (long)cb * 256;
  // both buffers hold zeros between M and the end of their last 256-row tile
  const long K = (M + kDmaKMult - 1) / kDmaKMult * kDmaKMult;
  DmaNN<256> mainloop;
  mainloop.init(a.hT, [&](int r) -> const char* { return row0 + r < a.d ? a.hT + (row0 + r) * kRowB : nullptr; },
                a.dz, 0, a.V, K, a.d * kRowB, a.C);
  f32x16_t acc[4][4];
  mainloop.tile<true>(sl, n0, acc);

  const int w = wave_id(), wm = w >> 1, wn = w & 1, lane = threadIdx.x & 63, h = lane >> 5, r32 = lane & 31;
#pragma unroll
  for (int mb = 0; mb < 4; ++mb) {
    char* slot = (wm ? (mb < 2 ? sl.s2 : sl.s3) : (mb < 2 ? sl.s0 : sl.s1)) + ((mb & 1) * 32 + r32) * 512;
#pragma unroll
    for (int nb = 0; nb < 4; ++nb)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int chunk = wn * 16 + nb * 4 + j;  // columns 8 chunk + 4 h ..
        *reinterpret_cast<uint2*>(slot + 16 * (chunk ^ r32) + 8 * h) =
            make_uint2(pk_bf16(acc[mb][nb][4 * j], acc[mb][nb][4 * j + 1]),
                       pk_bf16(acc[mb][nb][4 * j + 2], acc[mb][nb][4 * j + 3]));
      }
  }
  __syncthreads();
  const char* mine = w == 0 ? sl.s0 : w == 1 ? sl.s1 : w == 2 ? sl.s2 : sl.s3;  // rows 64 w ..
  const long col = n0 + 8 * r32;
#pragma unroll 8
  for (int i = 0; i < 32; ++i) {
    const int r = 2 * i + h;
    const long row = row0 + 64 * w + r;
    const u32x4_t x = *reinterpret_cast<const u32x4_t*>(mine + r * 512 + 16 * (r32 ^ (r & 31)));
    if (row < a.d && col < a.V) *reinterpret_cast<u32x4_t*>(out + (row * a.V + col) * 2) = x;
  }
}

__global__ __launch_bounds__(256) void to_bf16_kernel(const float* in, uint16_t* out, long n8) {
  for (long q = (long)blockIdx.x * 256 + threadIdx.x; q < n8; q += (long)gridDim.x * 256) {
    const float4 x = *reinterpret_cast<const float4*>(in + 8 * q), y = *reinterpret_cast<const float4*>(in + 8 * q + 4);
    *reinterpret_cast<uint4*>(out + 8 * q) =
        make_uint4(pk_bf16(x.x, x.y), pk_bf16(x.z, x.w), pk_bf16(y.x, y.y), pk_bf16(y.z, y.w));
  }
}

hipError_t launch_to_bf16(const float* in, void* out, int64_t n, hipStream_t st) {
  const int64_t n8 = n / 8;
  if (n8 == 0) return hipSuccess;
  const int64_t blocks = (n8 + 255) / 256;
  hipLaunchKernelGGL(to_bf16_kernel, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st, in,
                     static_cast<uint16_t*>(out), (long)n8);
  return hipGetLastError();
}

// ------------------------------------------------------------------ launches
bool logp_ring_fits(int elem, int64_t C, int64_t d, int64_t V) {
  const int64_t dp = (d + kDmaKMult - 1) / kDmaKMult * kDmaKMult;
  return elem == 2 && d % kDmaKs == 0 && V >= kBN && fits32(C * dp * 2) && fits32(d * V * 2);
}

hipError_t launch_logp_dh(const LogpDhArgs& a, const int32_t* rows, void* dH, int dh_elem, hipStream_t st) {
  // whole turns of the vocabulary need none of the tail's stage arithmetic (4% of the kernel)
  if (a.V % (32 * kRing))
    hipLaunchKernelGGL(logp_dh_kernel<true>, dim3(a.grid), dim3(kThreads), 0, st, a);
  else
    hipLaunchKernelGGL(logp_dh_kernel<false>, dim3(a.grid), dim3(kThreads), 0, st, a);
  const int64_t n = (a.C < a.T - a.c0 ? a.C : a.T - a.c0) * (a.d / 4);
  const dim3 blocks((unsigned)((n + 255) / 256));
  if (dh_elem == 2)
    hipLaunchKernelGGL(logp_dh_reduce_kernel<2>, blocks, dim3(256), 0, st, a, rows, static_cast<char*>(dH));
  else
    hipLaunchKernelGGL(logp_dh_reduce_kernel<4>, blocks, dim3(256), 0, st, a, rows, static_cast<char*>(dH));
  return hipGetLastError();
}

hipError_t launch_logp_dw_bf16(const DwArgs& a, void* out, hipStream_t st) {
  hipLaunchKernelGGL(logp_dw_bf16_kernel, dim3(a.nrb * a.ncb), dim3(kThreads), 0, st, a, static_cast<char*>(out));
  return hipGetLastError();
}

hipError_t launch_logp_fwd(const LogpFwdArgs& a, bool entropy, hipStream_t st) {
  const dim3 grid(a.grid), block(kThreads);
  if (entropy && a.zout)
    hipLaunchKernelGGL((logp_fwd_kernel<true, true>), grid, block, 0, st, a);
  else if (entropy)
    hipLaunchKernelGGL((logp_fwd_kernel<true, false>), grid, block, 0, st, a);
  else if (a.zout)
    hipLaunchKernelGGL((logp_fwd_kernel<false, true>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((logp_fwd_kernel<false, false>), grid, block, 0, st, a);
  return hipGetLastError();
}

hipError_t launch_logp_dz(const LogpDzArgs& a, hipStream_t st) {
  const dim3 grid(a.grid), block(kThreads);
  if (a.ge)
    hipLaunchKernelGGL(logp_dz_kernel<true>, grid, block, 0, st, a);
  else
    hipLaunchKernelGGL(logp_dz_kernel<false>, grid, block, 0, st, a);
  return hipGetLastError();
}

hipError_t launch_logp_dz_from_z(const LogpDzArgs& a, hipStream_t st) {
  const int64_t pieces = (a.V * 2 + kRowB - 1) / kRowB;
  const dim3 grid((unsigned)(pieces < kFzRanges ? pieces : kFzRanges), (unsigned)(a.C / kFzRows)), block(256);
  if (a.ge)
    hipLaunchKernelGGL(logp_dz_from_z_kernel<true>, grid, block, 0, st, a);
  else
    hipLaunchKernelGGL(logp_dz_from_z_kernel<false>, grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace kd
