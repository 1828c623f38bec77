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
// order.  No atomics: the same call gives the same bits.
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

// Chunk c of a wave over sequences cu [S+1]: part(mask of lane's tokens in
// [a, b)) is asked once per sequence that has tokens in the chunk, and
// put(kind, s) tells what the part is: 0 the whole sequence s, 1 its start
// (tail of the chunk), 2 a continuation (head of the chunk).
template <class Part>
__device__ inline void over_sequences(const int32_t* cu, int S, int T, int c, Part&& part) {
  const int t0 = c * kChunk, t1 = min(t0 + kChunk, T);
  for (int s = max(0, seq_of(cu, S, t0)); s < S; ++s) {
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
    double w = 1.0;
    if (a.reduction == 1) w = total > 0 ? 1.0 / total : 0.0;
    if (a.reduction == 2) {
      const int k = a.counts[s];
      w = k > 0 ? 1.0 / ((double)k * some) : 0.0;
    }
    a.weights[s] = w;
  }
}

// ------------------------------------------------------------------ policy: loss and gradients
namespace {

struct Sums {
  double v[5];  // total, policy, kl, entropy, clipped: each weighted
};

// Token t of sequence s (weight w): adds to the sums, writes the gradients.
__device__ inline void policy_token(const PolicyArgs& a, int t, int s, double w, double scale, Sums& sum) {
  const double lp = a.logp[t];
  const double A = a.adv[a.per_sequence ? s : t];
  const double r = exp(lp - (double)a.old[t]);
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
    const double d = (double)a.ref[t] - lp;
    if (a.kl_kind == 1) {
      kl = -d;
      g += a.klw;
    } else if (a.kl_kind == 2) {
      kl = 0.5 * d * d;
      g -= a.klw * d;
    } else {
      const double e = expm1(d);
      kl = e - d;
      g -= a.klw * e;
    }
  }
  const double h = a.ent ? (double)a.ent[t] : 0.0;
  double loss = pg;
  if (a.klw != 0) loss += a.klw * kl;
  if (a.entw != 0) loss -= a.entw * h;
  sum.v[0] += w * loss;
  sum.v[1] += w * pg;
  sum.v[2] += w * kl;
  sum.v[3] += w * h;
  sum.v[4] += cut ? w : 0.0;
  if (a.grad_logp) a.grad_logp[t] = (float)(scale * w * g);
  if (a.grad_ent) a.grad_ent[t] = (float)(-scale * w * a.entw);
}

}  // namespace

constexpr int kPolicyTokens = 1024;  // per block of 256 threads, 4 consecutive each

int64_t policy_counts(int64_t T, int64_t S) { return (S > 1 ? S : 1) + 2 * ((T + kChunk - 1) / kChunk); }
int64_t policy_blocks(int64_t T) { return (T + kPolicyTokens - 1) / kPolicyTokens; }

__global__ __launch_bounds__(256) void policy_kernel(PolicyArgs a) {
  __shared__ double red[4][5];
  const long tb = (long)blockIdx.x * kPolicyTokens + 4 * threadIdx.x;
  const double scale = a.grad_total ? (double)*a.grad_total : 1.0;
  Sums sum{};
  if (tb < a.T) {
    const int t0 = (int)tb;
    int s = a.cu ? seq_of(a.cu, a.S, t0) : 0;
    int end = a.cu ? (s < a.S ? cu_at(a.cu, s + 1, a.T) : a.T) : a.T;
    for (int t = t0; t < min(t0 + 4, a.T); ++t) {
      if (t >= end) {
        s = seq_of(a.cu, a.S, t);
        end = s < a.S ? cu_at(a.cu, s + 1, a.T) : a.T;
      }
      const bool in = s >= 0 && s < max(a.S, 1) && (a.mask == nullptr || a.mask[t] != 0);
      if (in) {
        policy_token(a, t, s, a.weights[s], scale, sum);
      } else {
        if (a.grad_logp) a.grad_logp[t] = 0.f;
        if (a.grad_ent) a.grad_ent[t] = 0.f;
      }
    }
  }
  if (a.stats == nullptr) return;
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const double v = wave_sum(sum.v[i]);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6][i] = v;
  }
  __syncthreads();
  if (threadIdx.x < 5) {
    double v = 0;
    for (int q = 0; q < 4; ++q) v += red[q][threadIdx.x];
    a.part[(long)blockIdx.x * 5 + threadIdx.x] = v;
  }
}

__global__ __launch_bounds__(256) void policy_stats_kernel(const double* part, long blocks, float* total,
                                                           float* stats) {
  __shared__ double red[4][5];
  Sums sum{};
  for (long b = threadIdx.x; b < blocks; b += 256)
#pragma unroll
    for (int i = 0; i < 5; ++i) sum.v[i] += part[b * 5 + i];
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const double v = wave_sum(sum.v[i]);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6][i] = v;
  }
  __syncthreads();
  if (threadIdx.x < 5) {
    double v = 0;
    for (int q = 0; q < 4; ++q) v += red[q][threadIdx.x];
    stats[threadIdx.x] = (float)v;
    if (total && threadIdx.x == 0) *total = (float)v;
  }
}

hipError_t launch_policy(const PolicyArgs& a, bool make_weights, hipStream_t st) {
  const int chunks = (a.T + kChunk - 1) / kChunk;
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
__global__ __launch_bounds__(256) void pref_sums_kernel(PrefArgs a, int chunks) {
  const int c = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (c >= chunks) return;
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

namespace {

struct Pair {
  double loss, dD;  // loss and its derivative by D
};
__device__ inline Pair pair_loss(const PrefArgs& a, double D) {
  const double h = a.beta * D - a.margin;
  if (a.kind == 0) {  // -(1 - e) log s(h) - e log s(-h), s(x) = 1 / (1 + exp(-x))
    const double soft = log1p(exp(-fabs(h)));
    const double q = exp(-fabs(h)) / (1.0 + exp(-fabs(h)));  // s(-|h|)
    const double up = h >= 0 ? q : 1.0 - q;                  // s(-h)
    return {soft + (h >= 0 ? a.eps * h : -(1.0 - a.eps) * h), a.beta * (a.eps - up)};
  }
  if (a.kind == 1) return {h < 1 ? 1 - h : (h >= 1 ? 0.0 : h), h < 1 ? -a.beta : 0.0};
  const double u = D - 0.5 / a.beta;
  return {u * u, 2 * u};
}
__device__ inline double value_of(const PrefArgs& a, double sum, double n) {
  return a.average ? (n > 0 ? sum / n : 0.0) : sum;
}

}  // namespace

// One lane per pair: both sequences' totals, the loss and the rewards.
__global__ __launch_bounds__(256) void pref_loss_kernel(PrefArgs a) {
  const int p = blockIdx.x * 256 + threadIdx.x;
  double v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = p + i * a.P;
    const bool in = p < a.P;
    const int x = in ? cu_at(a.cu, s, a.T) : 0, y = in ? cu_at(a.cu, s + 1, a.T) : 0;
    const bool one = x < y && x / kChunk == (y - 1) / kChunk;
    double sum = one ? a.sums[2 * (long)s] : 0.0, n = one ? a.sums[2 * (long)s + 1] : 0.0;
    sum = merge_parts<double>(x, y, sum, a.part, a.part + 2, 4);
    n = merge_parts<double>(x, y, n, a.part + 1, a.part + 3, 4);
    if (in) {
      a.sums[2 * (long)s] = sum;
      a.sums[2 * (long)s + 1] = n;
      v[i] = value_of(a, sum, n);
      a.rewards[s] = (float)(a.beta * v[i]);
    }
  }
  if (p < a.P) a.loss[p] = (float)pair_loss(a, v[0] - v[1]).loss;
}

// ------------------------------------------------------------------ preference: gradient
constexpr int kPrefTokens = 1024;  // per block, 4 consecutive per thread

__global__ __launch_bounds__(256) void pref_grad_kernel(PrefArgs a) {
  const long tb = (long)blockIdx.x * kPrefTokens + 4 * threadIdx.x;
  if (tb >= a.T) return;
  const int t0 = (int)tb, S = 2 * a.P;
  int end = -1;
  float g = 0.f;
  for (int t = t0; t < min(t0 + 4, a.T); ++t) {
    if (t >= end) {
      const int s = seq_of(a.cu, S, t);
      end = s < S ? cu_at(a.cu, s + 1, a.T) : a.T;
      g = 0.f;
      if (s >= 0 && s < S) {
        const int p = s < a.P ? s : s - a.P;
        const double nc = a.sums[2 * (long)p + 1], nr = a.sums[2 * (long)(p + a.P) + 1];
        const double D = value_of(a, a.sums[2 * (long)p], nc) - value_of(a, a.sums[2 * (long)(p + a.P)], nr);
        const double n = s < a.P ? nc : nr;
        double k = (double)a.grad_loss[p] * pair_loss(a, D).dD;
        if (a.average) k = n > 0 ? k / n : 0.0;
        g = (float)(s < a.P ? k : -k);
      }
    }
    a.grad_logp[t] = a.mask == nullptr || a.mask[t] != 0 ? g : 0.f;
  }
}

int64_t pref_chunks(int64_t T) { return (T + kChunk - 1) / kChunk; }

hipError_t launch_pref_fwd(const PrefArgs& a, hipStream_t st) {
  const int chunks = (int)pref_chunks(a.T);
  if (chunks > 0) hipLaunchKernelGGL(pref_sums_kernel, dim3((chunks + 3) / 4), dim3(256), 0, st, a, chunks);
  hipLaunchKernelGGL(pref_loss_kernel, dim3((a.P + 255) / 256), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_pref_bwd(const PrefArgs& a, hipStream_t st) {
  const unsigned blocks = (unsigned)(((int64_t)a.T + kPrefTokens - 1) / kPrefTokens);
  if (blocks > 0) hipLaunchKernelGGL(pref_grad_kernel, dim3(blocks), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace kd
