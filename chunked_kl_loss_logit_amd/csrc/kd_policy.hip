// Per-token losses on log-probabilities: the clipped policy loss and the
// preference loss over packed sequences.
//
// Both are a handful of flops on a few streams of 4 bytes per token, so what
// bounds them is the read of those streams and, below a few hundred thousand
// tokens, the launches.  The arithmetic is in 64 bits: at 4 to 24 bytes per
// token it costs nothing next to the memory, decides clip borders exactly as
// the given log-probabilities put them, and leaves one rounding per result.
//
// Sums over sequences of any lengths: a wave takes kChunk consecutive tokens,
// whatever sequences they belong to, so one long sequence is spread over many
// waves and many short ones share one.  A sequence inside one chunk is
// finished there; otherwise the chunk where it starts leaves its part in
// `tail` and every later one in `head`, and a second kernel adds them up in
// order.  No atomics on values: the same call gives the same bits.
//
// Measured: 1048576 tokens in 1000 sequences, forward and backward in one call,
// 30 us (count 6, weights 4, losses and gradients 15 at 1.7 TB/s, statistics
// 4, each behind a launch's 4); 700001 tokens in 384 pairs 23 us (sums 8, pairs
// 5, gradients 8); in one workgroup, 333 tokens 8.6 us and 900 tokens 8.0.
#include <cmath>

#include "kd_gemm.h"
#include "kd_policy.h"

namespace kd {

namespace {

constexpr int kChunk = 512;  // tokens per wave
constexpr int kPerLane = kChunk / 64;

__device__ inline double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ inline int wave_sum(int v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

__device__ inline int cu_at(const int32_t* cu, int i, int T) { return min(max(cu[i], 0), T); }

// The last s of [0, S] with cu[s] <= t, or -1: the sequence of token t when
// it is in [0, S).  (Empty sequences at the same place come before it.)
__device__ inline int seq_of(const int32_t* cu, int S, int t) {
  int b = 0, e = S + 1;  // first index with cu > t
  while (b < e) {
    const int mid = (b + e) >> 1;
    if (cu[mid] <= t) b = mid + 1; else e = mid;
  }
  return b - 1;
}

// The same found by a whole wave (t uniform), 64 entries a step: two
// dependent loads for thousands of sequences where halving takes a dozen.
__device__ inline int seq_of_wave(const int32_t* cu, int S, int t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = S + 1;
  while (true) {
    const int step = (n + 63) / 64;
    const int i = lo + lane * step;
    const bool at_most = lane * step < n && cu[min(i, S)] <= t;
    const int c = __popcll(__ballot(at_most));
    if (c == 0) return lo - 1;  // only where t is before every entry looked at: lo = 0
    lo += (c - 1) * step;
    if (step == 1) return lo;
    n = min(step, S + 1 - lo);
  }
}

// The sequence of this lane's token t, where the wave holds tokens in
// ascending order from t_first to t_last (both uniform, t_last < T).
__device__ inline int seq_of_lane(const int32_t* cu, int S, int t_first, int t_last, int t) {
  int b = seq_of_wave(cu, S, t_first), e = seq_of_wave(cu, S, t_last);
  while (b < e) {  // the last s in [b, e] with cu[s] <= t
    const int mid = (b + e + 1) >> 1;
    if (cu[mid] <= t) b = mid; else e = mid - 1;
  }
  return b;
}

// Chunk c of a wave over sequences cu [S+1]: part(mask of lane's tokens in
// [a, b)) is asked once per sequence that has tokens in the chunk, and
// put(kind, s) tells what the part is: 0 the whole sequence s, 1 its start
// (tail of the chunk), 2 a continuation (head of the chunk).
template <class Part>
__device__ inline void over_sequences(const int32_t* cu, int S, int T, int c, Part&& part) {
  const int t0 = c * kChunk, t1 = min(t0 + kChunk, T);
  for (int s = max(0, seq_of_wave(cu, S, t0)); s < S; ++s) {
    const int a = cu_at(cu, s, T), b = cu_at(cu, s + 1, T);
    if (a >= t1) break;
    if (b <= max(a, t0)) continue;
    part(s, max(a, t0), min(b, t1), a < t0 ? 2 : (b > t1 ? 1 : 0));
  }
}

// Sequence [a, b)'s total from its chunks' parts: whole (one chunk) or
// tail[first] + head[first + 1 .. last], added in order by one lane, or by
// the whole wave where there are many.  Every lane of the wave calls it.
template <class V>
__device__ inline V merge_parts(int a, int b, V whole, const V* head, const V* tail, int stride) {
  V r = V(0);
  int ca = 0, cb = 0;
  if (a < b) {
    ca = a / kChunk;
    cb = (b - 1) / kChunk;
    r = ca == cb ? whole : tail[(long)ca * stride];
  }
  const bool many = cb - ca > 32;
  if (!many)
    for (int c = ca + 1; c <= cb; ++c) r += head[(long)c * stride];
  unsigned long long todo = __ballot(many);
  const int lane = threadIdx.x & 63;
  while (todo) {
    const int l = __ffsll(todo) - 1;
    todo &= todo - 1;
    const int xa = __shfl(ca, l), xb = __shfl(cb, l);
    V v = V(0);
    for (int c = xa + 1 + lane; c <= xb; c += 64) v += head[(long)c * stride];
    v = wave_sum(v);
    if (lane == l) r += v;
  }
  return r;
}

}  // namespace

// ------------------------------------------------------------------ policy: valid tokens and weights
// One wave per chunk: valid tokens per sequence (the whole of [0, T) is the
// one sequence without cu).  cnt: [max(S,1)] whole, then head and tail [chunks].
__global__ __launch_bounds__(256) void policy_count_kernel(PolicyArgs a, int chunks) {
  const int c = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (c >= chunks) return;
  const int n = max(a.S, 1);
  int32_t* head = a.counts + n;
  int32_t* tail = head + chunks;
  const int t0 = c * kChunk, t1 = min(t0 + kChunk, a.T);
  unsigned valid = 0;  // bit j: token t0 + 64 j + lane
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) {
    const int t = t0 + 64 * j + lane;
    if (t < t1 && (a.mask == nullptr || a.mask[t] != 0)) valid |= 1u << j;
  }
  auto count = [&](int x, int y) {
    int k = 0;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      const int t = t0 + 64 * j + lane;
      k += __popcll(__ballot(t >= x && t < y && (valid >> j & 1)));
    }
    return k;
  };
  if (a.cu == nullptr) {
    const int k = count(t0, t1);
    if (lane == 0) head[c] = k;
    return;
  }
  over_sequences(a.cu, a.S, a.T, c, [&](int s, int x, int y, int kind) {
    const int k = count(x, y);
    if (lane == 0) (kind == 0 ? a.counts + s : kind == 1 ? tail + c : head + c)[0] = k;
  });
}

namespace {

// of a valid token in a sequence of k, of `total` in `some` sequences
__device__ inline double policy_weight(int reduction, int k, int total, int some) {
  if (reduction == 1) return total > 0 ? 1.0 / total : 0.0;
  if (reduction == 2) return k > 0 ? 1.0 / ((double)k * some) : 0.0;
  return 1.0;
}

}  // namespace

// One block: every sequence's count, N and S', then the weights.
__global__ __launch_bounds__(1024) void policy_weights_kernel(PolicyArgs a, int chunks) {
  __shared__ int red[2][16];
  const int n = max(a.S, 1);
  const int32_t* head = a.counts + n;
  const int32_t* tail = head + chunks;
  int total = 0, some = 0;
  if (a.cu == nullptr) {
    for (int c = threadIdx.x; c < chunks; c += 1024) total += head[c];
  } else {
    for (int s0 = 0; s0 < a.S; s0 += 1024) {  // whole waves stay together for merge_parts
      const int s = s0 + threadIdx.x;
      const int x = s < a.S ? cu_at(a.cu, s, a.T) : 0, y = s < a.S ? cu_at(a.cu, s + 1, a.T) : 0;
      int k = s < a.S && x < y ? a.counts[s] : 0;
      k = merge_parts<int>(x, y, k, head, tail, 1);
      if (s < a.S) a.counts[s] = k;
      total += k;
      some += k > 0;
    }
  }
  total = wave_sum(total);
  some = wave_sum(some);
  if ((threadIdx.x & 63) == 0) {
    red[0][threadIdx.x >> 6] = total;
    red[1][threadIdx.x >> 6] = some;
  }
  __syncthreads();
  total = some = 0;
  for (int i = 0; i < 16; ++i) {
    total += red[0][i];
    some += red[1][i];
  }
  if (a.stats && threadIdx.x == 0) a.stats[5] = (float)total;
  for (int s = threadIdx.x; s < n; s += 1024) {
    a.weights[s] = policy_weight(a.reduction, a.reduction == 2 ? a.counts[s] : 0, total, some);
  }
}

// ------------------------------------------------------------------ policy: loss and gradients
namespace {

struct Sums {
  double v[5];  // total, policy, kl, entropy, clipped: each weighted
};

// What a token brings, in 32 bits as given.
struct Token {
  float logp, old, adv, ref, ent;
};
struct Grads {
  float logp, ent;
};

// A token of weight w: adds to the sums, returns its gradients.
__device__ inline Grads policy_token(const PolicyArgs& a, const Token& k, double w, double scale, Sums& sum) {
  const double lp = k.logp, A = k.adv;
  const double r = exp(lp - (double)k.old);
  bool cut = (A > 0 && r > a.hi) || (A < 0 && r < a.lo);
  const double rc = fmin(fmax(r, a.lo), a.hi);
  double pg = A == 0 ? 0.0 : -(cut ? rc : r) * A;
  if (a.dual > 0 && A < 0 && r > a.dual) {
    cut = true;
    pg = -a.dual * A;
  }
  double g = cut ? 0.0 : A == 0 ? 0.0 : -A * r;
  double kl = 0.0;
  if (a.ref) {
    const double d = (double)k.ref - lp;
    double dkl;
    if (a.kl_kind == 1) {
      kl = -d;
      dkl = 1.0;
    } else if (a.kl_kind == 2) {
      kl = 0.5 * d * d;
      dkl = -d;
    } else {  // e = exp(d) - 1, exp(d) - 1 - d: by the series where the subtraction would cost digits
      double e, f;
      if (fabs(d) < 0x1p-6) {  // the first term left out, d^7 / 5040, is below 2^-48 of d
        f = d * d * (1.0 / 2 + d * (1.0 / 6 + d * (1.0 / 24 + d * (1.0 / 120 + d * (1.0 / 720)))));
        e = d + f;
      } else {
        e = exp(d) - 1.0;
        f = e - d;
      }
      kl = f;
      dkl = -e;
    }
    if (a.klw != 0) g += a.klw * dkl;  // without weight it is only counted, infinite or not
  }
  const double h = a.ent ? (double)k.ent : 0.0;
  double loss = pg;
  if (a.klw != 0) loss += a.klw * kl;
  if (a.entw != 0) loss -= a.entw * h;
  sum.v[0] += w * loss;
  sum.v[1] += w * pg;
  sum.v[2] += w * kl;
  sum.v[3] += w * h;
  sum.v[4] += cut ? w : 0.0;
  return Grads{(float)(scale * w * g), (float)(-scale * w * a.entw)};
}

// The block's sums to out[0 .. 4]; NW waves
template <int NW, class Put>
__device__ inline void block_sums(const Sums& sum, double (&red)[NW][5], Put&& put) {
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const double v = wave_sum(sum.v[i]);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6][i] = v;
  }
  __syncthreads();
  if (threadIdx.x < 5) {
    double v = 0;
    for (int q = 0; q < NW; ++q) v += red[q][threadIdx.x];
    put((int)threadIdx.x, v);
  }
}

// Four floats from p on (4-byte aligned: the hardware takes unaligned vector accesses), n of them there
__device__ inline float4 load4(const float* p, int n) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (n >= 4)
    __builtin_memcpy(&v, p, 16);
  else {
    v.x = p[0];
    if (n > 1) v.y = p[1];
    if (n > 2) v.z = p[2];
  }
  return v;
}
__device__ inline void store4(float* p, int n, float4 v) {
  if (n >= 4)
    __builtin_memcpy(p, &v, 16);
  else {
    p[0] = v.x;
    if (n > 1) p[1] = v.y;
    if (n > 2) p[2] = v.z;
  }
}
__device__ inline float& at4(float4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Four consecutive tokens of a lane, the wave's tokens being [t_first, t_last];
// weight(s): of a valid token of sequence s.
template <class Weight>
__device__ inline void policy_four(const PolicyArgs& a, int t_first, int t_last, int t0, double scale, Sums& sum,
                                   Weight&& weight) {
  const int n = min(4, a.T - t0), S = max(a.S, 1);
  int s = a.cu ? seq_of_lane(a.cu, a.S, t_first, t_last, min(t0, t_last)) : 0;
  if (n <= 0) return;
  int end = a.cu ? (s < S ? cu_at(a.cu, s + 1, a.T) : a.T) : a.T;
  float4 lp = load4(a.logp + t0, n), old = load4(a.old + t0, n);
  float4 adv = a.per_sequence ? lp : load4(a.adv + t0, n);
  float4 ref = a.ref ? load4(a.ref + t0, n) : lp, ent = a.ent ? load4(a.ent + t0, n) : lp;
  float4 gl = make_float4(0.f, 0.f, 0.f, 0.f), ge = gl;
  double w = s >= 0 && s < S ? weight(s) : 0.0;
  float sa = a.per_sequence && s >= 0 && s < S ? a.adv[s] : 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + i;
    if (i >= n) break;
    if (t >= end) {
      s = seq_of(a.cu, a.S, t);
      end = s < S ? cu_at(a.cu, s + 1, a.T) : a.T;
      w = s >= 0 && s < S ? weight(s) : 0.0;
      sa = a.per_sequence && s >= 0 && s < S ? a.adv[s] : 0.f;
    }
    if (s < 0 || s >= S || (a.mask != nullptr && a.mask[t] == 0)) continue;
    const Token k{at4(lp, i), at4(old, i), a.per_sequence ? sa : at4(adv, i), at4(ref, i), at4(ent, i)};
    const Grads g = policy_token(a, k, w, scale, sum);
    at4(gl, i) = g.logp;
    at4(ge, i) = g.ent;
  }
  if (a.grad_logp) store4(a.grad_logp + t0, n, gl);
  if (a.grad_ent) store4(a.grad_ent + t0, n, ge);
}

}  // namespace

constexpr int kPolicyTokens = 1024;  // per block of 256 threads, 4 consecutive each

int64_t policy_counts(int64_t T, int64_t S) { return (S > 1 ? S : 1) + 2 * ((T + kChunk - 1) / kChunk); }
int64_t policy_blocks(int64_t T) { return (T + kPolicyTokens - 1) / kPolicyTokens; }

__global__ __launch_bounds__(256) void policy_kernel(PolicyArgs a) {
  __shared__ double red[4][5];
  const long tw = (long)blockIdx.x * kPolicyTokens + 256 * (threadIdx.x >> 6);  // the wave's first token
  const double scale = a.grad_total ? (double)*a.grad_total : 1.0;
  Sums sum{};
  if (tw < a.T)
    policy_four(a, (int)tw, (int)min(tw + 255, (long)a.T - 1), (int)tw + 4 * (threadIdx.x & 63), scale, sum,
                [&](int s) { return a.weights[s]; });
  if (a.stats == nullptr) return;
  block_sums<4>(sum, red, [&](int i, double v) { a.part[(long)blockIdx.x * 5 + i] = v; });
}

__global__ __launch_bounds__(256) void policy_stats_kernel(const double* part, long blocks, float* total,
                                                           float* stats) {
  __shared__ double red[4][5];
  Sums sum{};
  for (long b = threadIdx.x; b < blocks; b += 256)
#pragma unroll
    for (int i = 0; i < 5; ++i) sum.v[i] += part[b * 5 + i];
  block_sums<4>(sum, red, [&](int i, double v) {
    stats[i] = (float)v;
    if (total && i == 0) *total = (float)v;
  });
}

// Everything in one workgroup and one launch: counts, weights, loss and
// gradients of at most kSmallTokens tokens in kSmallSeqs sequences (where four
// launches take longer: 4096 tokens 15 us against 16, 512 tokens 8).
constexpr int kSmallTokens = 4096, kSmallSeqs = 2048;

__global__ __launch_bounds__(1024) void policy_small_kernel(PolicyArgs a) {
  __shared__ int cnt[kSmallSeqs];
  __shared__ double red[16][5];
  __shared__ int redi[2][16];
  const int n = max(a.S, 1), tid = threadIdx.x;
  for (int s = tid; s < n; s += 1024) cnt[s] = 0;
  __syncthreads();
  for (int t0 = 0; t0 < a.T; t0 += 1024) {
    const int t = t0 + tid, tw = t0 + (tid & ~63);
    if (tw >= a.T) break;
    const int s = a.cu ? seq_of_lane(a.cu, a.S, tw, min(tw + 63, a.T - 1), min(t, a.T - 1)) : 0;
    if (t < a.T && s >= 0 && s < n && (a.mask == nullptr || a.mask[t] != 0)) atomicAdd(&cnt[s], 1);  // whole numbers
  }
  __syncthreads();
  int total = 0, some = 0;
  for (int s = tid; s < n; s += 1024) {
    total += cnt[s];
    some += cnt[s] > 0;
  }
  total = wave_sum(total);
  some = wave_sum(some);
  if ((tid & 63) == 0) {
    redi[0][tid >> 6] = total;
    redi[1][tid >> 6] = some;
  }
  __syncthreads();
  total = some = 0;
  for (int i = 0; i < 16; ++i) {
    total += redi[0][i];
    some += redi[1][i];
  }
  auto weight = [&](int s) { return policy_weight(a.reduction, cnt[s], total, some); };
  for (int s = tid; s < n; s += 1024) a.weights[s] = weight(s);
  Sums sum{};
  for (int t0 = 256 * (tid >> 6); t0 < a.T; t0 += 4096)
    policy_four(a, t0, min(t0 + 255, a.T - 1), t0 + 4 * (tid & 63), 1.0, sum, weight);
  block_sums<16>(sum, red, [&](int i, double v) {
    a.stats[i] = (float)v;
    if (a.total && i == 0) *a.total = (float)v;
  });
  if (tid == 0) a.stats[5] = (float)total;
}

hipError_t launch_policy(const PolicyArgs& a, bool make_weights, hipStream_t st) {
  const int chunks = (a.T + kChunk - 1) / kChunk;
  if (make_weights && a.T <= kSmallTokens && a.S <= kSmallSeqs) {
    hipLaunchKernelGGL(policy_small_kernel, dim3(1), dim3(1024), 0, st, a);
    return hipGetLastError();
  }
  if (make_weights) {
    if (chunks > 0)
      hipLaunchKernelGGL(policy_count_kernel, dim3((chunks + 3) / 4), dim3(256), 0, st, a, chunks);
    hipLaunchKernelGGL(policy_weights_kernel, dim3(1), dim3(1024), 0, st, a, chunks);
  }
  const int64_t blocks = policy_blocks(a.T);
  if (blocks > 0) hipLaunchKernelGGL(policy_kernel, dim3((unsigned)blocks), dim3(256), 0, st, a);
  if (a.stats) hipLaunchKernelGGL(policy_stats_kernel, dim3(1), dim3(256), 0, st, a.part, (long)blocks,
                                   a.total, a.stats);
  return hipGetLastError();
}

// ------------------------------------------------------------------ preference: sums
// Parts per chunk: [4] doubles, (head sum, head count, tail sum, tail count).
namespace {

__device__ inline void pref_sums(const PrefArgs& a, int c) {
  const int lane = threadIdx.x & 63;
  const int t0 = c * kChunk, t1 = min(t0 + kChunk, a.T);
  double x[kPerLane];
  unsigned valid = 0;
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) {
    const int t = t0 + 64 * j + lane;
    x[j] = 0.0;
    if (t < t1 && (a.mask == nullptr || a.mask[t] != 0)) {
      valid |= 1u << j;
      x[j] = (double)a.logp[t] - (a.ref ? (double)a.ref[t] : 0.0);
    }
  }
  over_sequences(a.cu, 2 * a.P, a.T, c, [&](int s, int lo, int hi, int kind) {
    double sum = 0.0;
    int k = 0;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      const int t = t0 + 64 * j + lane;
      const bool in = t >= lo && t < hi && (valid >> j & 1);
      sum += in ? x[j] : 0.0;
      k += __popcll(__ballot(in));
    }
    sum = wave_sum(sum);
    if (lane == 0) {
      double* o = kind == 0 ? a.sums + 2 * (long)s : a.part + 4 * (long)c + (kind == 1 ? 2 : 0);
      o[0] = sum;
      o[1] = (double)k;
    }
  });
}

struct Pair {
  double loss, dD;  // loss and its derivative by D
};
__device__ inline Pair pair_loss(const PrefArgs& a, double D) {
  const double h = a.beta * D - a.margin;
  if (a.kind == 0) {  // -(1 - e) log s(h) - e log s(-h), s(x) = 1 / (1 + exp(-x))
    const double soft = log1p(exp(-fabs(h)));
    const double q = exp(-fabs(h)) / (1.0 + exp(-fabs(h)));  // s(-|h|)
    const double up = h >= 0 ? q : 1.0 - q;                  // s(-h)
    const double wrong = a.eps == 0 ? 0.0 : a.eps * h;  // no part of an infinite h
    return {soft + (h < 0 ? wrong - h : wrong), a.beta * (a.eps - up)};
  }
  if (a.kind == 1) return {h < 1 ? 1 - h : (h >= 1 ? 0.0 : h), h < 1 ? -a.beta : 0.0};
  const double u = D - 0.5 / a.beta;
  return {u * u, 2 * u};
}
__device__ inline double value_of(const PrefArgs& a, double sum, double n) {
  return a.average ? (n > 0 ? sum / n : 0.0) : sum;
}

}  // namespace

__global__ __launch_bounds__(256) void pref_sums_kernel(PrefArgs a, int chunks) {
  const int c = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (c < chunks) pref_sums(a, c);
}

namespace {

// 32 pairs from p0 on by a wave, lanes 0 .. 31 the chosen sequences and 32 ..
// 63 the rejected ones: their totals, the rewards and the losses.
__device__ inline void pref_pairs(const PrefArgs& a, int p0) {
  const int lane = threadIdx.x & 63, p = p0 + (lane & 31), s = p + (lane >> 5) * a.P;
  const bool in = p < a.P;
  const int x = in ? cu_at(a.cu, s, a.T) : 0, y = in ? cu_at(a.cu, s + 1, a.T) : 0;
  const bool one = x < y && x / kChunk == (y - 1) / kChunk;
  double sum = one ? a.sums[2 * (long)s] : 0.0, n = one ? a.sums[2 * (long)s + 1] : 0.0;
  sum = merge_parts<double>(x, y, sum, a.part, a.part + 2, 4);
  n = merge_parts<double>(x, y, n, a.part + 1, a.part + 3, 4);
  const double v = value_of(a, sum, n);
  const double other = __shfl_xor(v, 32);
  if (!in) return;
  a.sums[2 * (long)s] = sum;
  a.sums[2 * (long)s + 1] = n;
  a.rewards[s] = (float)(a.beta * v);
  if (lane < 32) a.loss[p] = (float)pair_loss(a, v - other).loss;
}

}  // namespace

__global__ __launch_bounds__(64) void pref_loss_kernel(PrefArgs a) { pref_pairs(a, blockIdx.x * 32); }

// ------------------------------------------------------------------ preference: gradient
constexpr int kPrefTokens = 1024;  // per block, 4 consecutive per thread

namespace {

// Four consecutive tokens of a lane, the wave's tokens being [t_first, t_last]
__device__ inline void pref_four(const PrefArgs& a, int t_first, int t_last, int t0) {
  const int S = 2 * a.P, n = min(4, a.T - t0);
  int s = seq_of_lane(a.cu, S, t_first, t_last, min(t0, t_last));
  if (n <= 0) return;
  auto value = [&](int q) {
    if (q < 0 || q >= S) return 0.f;
    const int p = q < a.P ? q : q - a.P;
    const double nc = a.sums[2 * (long)p + 1], nr = a.sums[2 * (long)(p + a.P) + 1];
    const double D = value_of(a, a.sums[2 * (long)p], nc) - value_of(a, a.sums[2 * (long)(p + a.P)], nr);
    const double m = q < a.P ? nc : nr;
    double k = (double)a.grad_loss[p] * pair_loss(a, D).dD;
    if (a.average) k = m > 0 ? k / m : 0.0;
    return (float)(q < a.P ? k : -k);
  };
  float g = value(s);
  int end = s < S ? cu_at(a.cu, s + 1, a.T) : a.T;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + i;
    if (i >= n) break;
    if (t >= end) {
      s = seq_of(a.cu, S, t);
      end = s < S ? cu_at(a.cu, s + 1, a.T) : a.T;
      g = value(s);
    }
    at4(o, i) = a.mask == nullptr || a.mask[t] != 0 ? g : 0.f;
  }
  store4(a.grad_logp + t0, n, o);
}

}  // namespace

__global__ __launch_bounds__(256) void pref_grad_kernel(PrefArgs a) {
  const long tw = (long)blockIdx.x * kPrefTokens + 256 * (threadIdx.x >> 6);
  if (tw < a.T) pref_four(a, (int)tw, (int)min(tw + 255, (long)a.T - 1), (int)tw + 4 * (threadIdx.x & 63));
}

// All of it in one workgroup and one launch, for at most kSmallTokens tokens
// and kSmallPairs pairs; without grad_logp the loss alone.
constexpr int kSmallPairs = 512;

__global__ __launch_bounds__(1024) void pref_small_kernel(PrefArgs a, int chunks) {
  const int w = threadIdx.x >> 6;
  for (int c = w; c < chunks; c += 16) pref_sums(a, c);
  __syncthreads();  // the waves' parts, in global memory, are each other's from here on
  for (int p0 = 32 * w; p0 < a.P; p0 += 512) pref_pairs(a, p0);
  if (a.grad_logp == nullptr) return;
  __syncthreads();
  for (int t0 = 256 * w; t0 < a.T; t0 += 4096) pref_four(a, t0, min(t0 + 255, a.T - 1), t0 + 4 * (threadIdx.x & 63));
}

int64_t pref_chunks(int64_t T) { return (T + kChunk - 1) / kChunk; }

hipError_t launch_pref(const PrefArgs& a, hipStream_t st) {
  const int chunks = (int)pref_chunks(a.T);
  if (a.T <= kSmallTokens && a.P <= kSmallPairs) {
    hipLaunchKernelGGL(pref_small_kernel, dim3(1), dim3(1024), 0, st, a, chunks);
    return hipGetLastError();
  }
  if (chunks > 0) hipLaunchKernelGGL(pref_sums_kernel, dim3((chunks + 3) / 4), dim3(256), 0, st, a, chunks);
  hipLaunchKernelGGL(pref_loss_kernel, dim3((a.P + 31) / 32), dim3(64), 0, st, a);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || a.grad_logp == nullptr ? e : launch_pref_grad(a, st);
}

hipError_t launch_pref_grad(const PrefArgs& a, hipStream_t st) {
  const unsigned blocks = (unsigned)(((int64_t)a.T + kPrefTokens - 1) / kPrefTokens);
  if (blocks > 0) hipLaunchKernelGGL(pref_grad_kernel, dim3(blocks), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace kd
