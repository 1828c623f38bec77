// Internal interface of the policy- and preference-training operators: token
// log-probabilities through the head, the clipped policy loss, the preference
// loss and gradient clipping.  Every launcher enqueues on the given stream
// and returns the launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kd_launch.h"

namespace kd {

// ---------------------------------------------------------------- token log-probabilities
// The rows of one chunk: valid rows [c0, c0 + C) of T, listed in rows and
// counted in *count, or without a mask (rows null) simply rows c0 + i.
struct RowSet {
  const int32_t* rows;
  const int32_t* count;
  int64_t c0, C, T;
};
// How many vocabulary splits `grid` workgroups give M rows in blocks of 256.
// The valid rows are only counted on the device: a split count chosen for
// all T rows would leave a sixth of the CUs without work where a mask takes
// one of six row blocks, so the kernels divide the grid among the rows there are.
constexpr int kRingMaxSplits = 512;
__host__ __device__ inline int ring_splits(int64_t M, int ntiles, int grid) {
  const int64_t nrb = (M + kTileM - 1) / kTileM;
  int64_t s = nrb > 0 ? grid / nrb : 1;
  s = s < ntiles ? s : ntiles;
  s = s < kRingMaxSplits ? s : kRingMaxSplits;
  return s > 1 ? (int)s : 1;
}

// What a base-2 logit relative to another (an exponent, or the factor of a term
// whose 2^x is 0 there) counts as at least: 2^-256 is 0 in 32 bits, and the
// product of such a 2^x with a column masked by the type's lowest value, whose
// difference passes the 32-bit range, would be 0 times infinity.  (A NaN difference
// stays visible: its 2^x is taken from the value itself.)
__device__ inline float at_least(float x) { return fmaxf(x, -256.f); }
// z c2 of a tile's largest z, which differences are taken from.  Where rounding
// it down leaves more than 1 (beyond 2^24), a step up, so that no difference
// passes 1: a tile of masked columns alone, at -1e30 say, would have sums of
// infinity, which no later maximum scales away.
__device__ inline float top_of(float z, float c2) {
  const float m = z * c2, rest = fmaf(z, c2, -m);  // infinite where m is
  return rest > 1.f && rest < INFINITY ? fmaf(fabsf(m), 0x1p-23f, m) : m;
}
// What is subtracted for a maximum m: below the 32-bit range it is -infinity,
// and there every 2^y is 0.
__device__ inline float subtrahend(float m) { return m == -INFINITY ? 0.f : m; }

// One record per (vocabulary split, row): with y = z log2(e) / tau over the
// split's columns, (m, l, e, x) = (max y, sum 2^(y - m), sum 2^(y - m) (y - m),
// z at the row's token or 0); (-infinity, 0, 0, x) where every y is below the
// 32-bit range.
struct LogpFwdArgs {
  const char* Hp;         // rows [c0, c0 + C) of H in panels of C rows
  const char* W;          // [d][V]
  Compact c;
  const int32_t* tokens;  // [T]
  float* part;            // [S][C][4], row p of a split is compacted row c0 + p
  float* zout;            // nullable: the logits of those rows, fp32 [C][ldz]
  int64_t ldz;
  int64_t c0, C, d, V;
  int32_t v0;             // first column of W in the whole head (tokens are whole-head indices)
  int grid, ntiles;       // workgroups, whole rounds of them (ring_splits)
  int group;
  float c2;               // log2(e) / tau
};
// Whether the ring tiles take a head with chunks of C rows.  Where d is not a
// multiple of 128, Hp's panels hold zeros from d to the next one.
bool logp_ring_fits(int elem, int64_t C, int64_t d, int64_t V);
hipError_t launch_logp_fwd(const LogpFwdArgs& a, bool entropy, hipStream_t st);

// dZ panels of the ring hold kDzTailPieces pieces after their ldz / 32: the
// last 32 columns once more where V is not a multiple of 32 (written with
// dZ), and zeros up to a whole ring turn of dH's contraction.
constexpr int kDzTailPieces = 4;
struct LogpDhArgs {
  const char* dz;  // panels of C rows, the tail pieces included
  const char* W;
  float* part;     // [grid / ncb][256][d] floats
  const int32_t* count;
  int64_t T, c0, C, ldz, d, V;
  int grid, ncb, group;  // workgroups, 256-wide blocks of d
};
// dH of the chunk's valid rows (rows: Compact's list), in elements of dh_elem bytes
hipError_t launch_logp_dh(const LogpDhArgs& a, const int32_t* rows, void* dH, int dh_elem, hipStream_t st);
hipError_t launch_logp_dw_bf16(const DwArgs& a, void* out, hipStream_t st);  // one chunk: out = bf16(H^T dZ)

// Per-row outputs of compacted rows [c0, c0 + C) from the records; with
// zero_masked, also zeroes the outputs of every masked row.  rec != nullptr:
// the merged record itself goes out instead (a vocabulary shard).
struct LogpOut {
  float* logp;
  float* lse;
  float* entropy;  // nullable
  float4* rec;     // nullable
};
// (S records a row, or with grid > 0 ring_splits of S tiles)
hipError_t launch_logp_combine(const float* part, int S, int grid, const RowSet& rs, const uint8_t* mask,
                               const int32_t* tokens, int64_t V, float c2, const LogpOut& o, bool zero_masked,
                               hipStream_t st);
// The same outputs from R shards' records rec [R][T].
hipError_t launch_logp_shard_combine(const float4* rec, int R, int64_t T, const uint8_t* mask, float c2,
                                     const LogpOut& o, hipStream_t st);

// dZ of one chunk: dZ = ga [v = token] - q (ga + ge (ent + log q)), ga = g / tau, ge = grad_entropy / tau.
struct LogpDzArgs {
  const char* Hp;         // rows [c0, c0 + C) of H in panels of C rows (unused with z)
  const char* W;
  const float* z;         // nullable: stored logits [C][ldz] of the chunk
  Compact c;
  const int32_t* tokens;
  const float* lse;
  const float* ent;       // [T], read when ge is set
  const float* g;         // nullable [T]: gradient of the log-probability
  const float* ge;        // nullable [T]: gradient of the entropy
  char* dz;               // [C][ldz] in panels of C rows
  int64_t ldz, c0, C, d, V;
  int32_t v0;
  int grid, ntiles;
  int group;
  float c2, inv_tau;
};
hipError_t launch_logp_dz(const LogpDzArgs& a, hipStream_t st);
hipError_t launch_logp_dz_from_z(const LogpDzArgs& a, hipStream_t st);

// ---------------------------------------------------------------- the same without LDS-staged tiles
// rows and *count from the mask (not null); the first C valid rows of H packed
// into Hc [C][row_bytes] (nullable); masked rows of dH (nullable) zeroed.
hipError_t launch_logp_prep(const uint8_t* mask, int64_t T, int32_t* rows, int32_t* count, const void* H,
                            int64_t row_bytes, int64_t C, void* Hc, void* dH, int64_t dh_row_bytes, hipStream_t st);
// The chunk's rows of H packed into Hc.
hipError_t launch_logp_pack(const RowSet& rs, const void* H, int64_t row_bytes, void* Hc, hipStream_t st);
constexpr int kDirectCols = 128;  // vocabulary columns per tile
struct LogpDirectArgs {
  RowSet rs;
  const char* H;          // [T][d]
  const char* W;          // [d][V]
  const int32_t* tokens;
  int64_t d, V, ldz;
  int32_t v0;
  float c2, inv_tau;
  float* part;            // forward: records [tiles][C][4] as LogpFwdArgs::part
  float* z;               // forward: nullable, logits out [C][ldz]; dz from z: the logits
  const float *lse, *ent, *g, *ge;
  char* dz;               // backward: [C][ldz], row-major; zero rows up to a multiple of 32
  int64_t lo;             // nonzero (chunks of up to 32 rows, bf16): dz's bytes to a second plane, what rounding left
};
hipError_t launch_logp_direct_fwd(int elem, const LogpDirectArgs& a, bool entropy, hipStream_t st);
hipError_t launch_logp_direct_dz(int elem, const LogpDirectArgs& a, hipStream_t st);
hipError_t launch_logp_direct_dz_from_z(int elem, const LogpDirectArgs& a, hipStream_t st);
// dH of the chunk: dz . W^T by `grid` workgroups, the vocabulary in as many ranges as they leave room for, each into
// its part (float32, grid / cdiv(d, 128) blocks of direct_dh_rows rows of d), summed in order
inline int direct_dh_rows(int64_t n) { return n <= 32 ? 32 : 64; }  // rows of a block, of n in the chunk
hipError_t launch_logp_direct_dh(int elem, const LogpDirectArgs& a, int grid, float* part, void* dH, int dh_elem,
                                 hipStream_t st);
// dW of the chunk: sum over its rows of Hc^T dz, plus add32 (nullable), to out (float32 or bf16)
hipError_t launch_logp_direct_dw(int elem, const LogpDirectArgs& a, const void* Hc, const float* add32, void* out,
                                 int out_elem, hipStream_t st);

// out[i] = bf16(in[i]) for i < n, n a multiple of 8, both 16-byte aligned
hipError_t launch_to_bf16(const float* in, void* out, int64_t n, hipStream_t st);

// ---------------------------------------------------------------- clipped policy loss
struct PolicyArgs {
  const float* logp;
  const float* old;
  const float* adv;
  const uint8_t* mask;    // nullable
  const float* ref;       // nullable
  const float* ent;       // nullable
  const int32_t* cu;      // nullable [S+1]
  int32_t T, S;
  int per_sequence, reduction, kl_kind;
  double lo, hi, dual, klw, entw;  // lo, hi: 1 - clip_low, 1 + clip_high
  double* weights;        // [max(S, 1)]
  const float* grad_total;  // nullable: 1
  float* total;           // nullable [1]
  float* stats;           // nullable [6]
  float* grad_logp;       // nullable [T]
  float* grad_ent;        // nullable [T]
  double* part;           // workspace: [policy_blocks(T)][5]
  int32_t* counts;        // workspace: [policy_counts(T, S)]
};
int64_t policy_blocks(int64_t T);
int64_t policy_counts(int64_t T, int64_t S);
// weights (and counts), then loss and / or gradients
hipError_t launch_policy(const PolicyArgs& a, bool make_weights, hipStream_t st);

// ---------------------------------------------------------------- preference loss
struct PrefArgs {
  const float* logp;      // not read by the backward
  const float* ref;       // nullable
  const int32_t* cu;      // [2P+1]
  const uint8_t* mask;    // nullable
  int32_t T, P;
  int kind, average;
  double beta, eps, margin;
  double* sums;           // [2P][2]
  float* loss;            // [P]
  float* rewards;         // [2P]
  const float* grad_loss; // [P]
  float* grad_logp;       // nullable [T]
  double* part;           // workspace: [pref_chunks(T)][4]
};
int64_t pref_chunks(int64_t T);
hipError_t launch_pref(const PrefArgs& a, hipStream_t st);       // sums, loss, rewards, and grad_logp if set
hipError_t launch_pref_grad(const PrefArgs& a, hipStream_t st);  // grad_logp from sums

// ---------------------------------------------------------------- gradient norm and clipping
// One launch's tensors, by value (a table stays within a kernel argument
// segment of 4 KB).  Tensor i is covered by blocks [first[i], first[i + 1]),
// kClipBlock elements each.
constexpr int kClipBlock = 32768;
struct SumsqTable {
  static constexpr int kTensors = 188;
  const void* in[kTensors];
  int64_t numel[kTensors];
  int32_t first[kTensors + 1];
  int32_t n;
  uint8_t type[kTensors];  // KD_F32, KD_BF16, KD_F16
};
struct ClipTable {
  static constexpr int kTensors = 132;
  const void* in[kTensors];
  void* out[kTensors];
  int64_t numel[kTensors];
  int32_t first[kTensors + 1];
  int32_t n;
  uint8_t in_type[kTensors], out_type[kTensors];
};
static_assert(sizeof(SumsqTable) <= 4000 && sizeof(ClipTable) <= 4000, "kernel arguments");
// partial sums of squares, one per block, from part[0] on
hipError_t launch_sumsq(const SumsqTable& t, double* part, hipStream_t st);
hipError_t launch_sumsq_total(const double* part, int64_t n, double* sumsq, hipStream_t st);
// norm (nullable) is written too
hipError_t launch_clip(const ClipTable& t, const double* sumsq, double max_norm, float* norm, hipStream_t st);
hipError_t launch_norm(const double* sumsq, float* norm, hipStream_t st);
// Everything in one workgroup, for at most kClipSmall elements in all, in at
// most kClipSmallTensors tensors, which it walks one after the other.  A call
// that is waited for, us, one launch / three: 32768 float32 elements in 1 tensor
// 27 / 30, in 6 33 / 33, 8 34 / 34, 12 40 / 37, 32 61 / 46, 132 172 / 98; 65536
// in 8 37 / 34.  Called without waiting the host is what counts: 8 tensors 19 /
// 23, 32 31 / 36, 132 88 / 87; in a replayed graph 8 9.5 / 7.4, 132 86 / 7.6.
constexpr int64_t kClipSmall = 65536;
constexpr int kClipSmallTensors = 8;
hipError_t launch_clip_small(const ClipTable& t, double* sumsq, double max_norm, float* norm, hipStream_t st);

}  // namespace kd
