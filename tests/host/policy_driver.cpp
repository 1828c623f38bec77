// Host-side checks of kdpolicy.h's argument validation and planning under the
// address and undefined-behaviour sanitizers.  Every call is rejected, or
// sizes a buffer, before its first HIP call.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>
#include <vector>

#include "kdpolicy.h"

namespace {
int failures = 0;
void expect(bool ok, const char* what, int line) {
  if (!ok) {
    std::printf("FAILED line %d: %s (last error: %s)\n", line, what, kd_last_error());
    ++failures;
  }
}
#define EXPECT(x) expect((x), #x, __LINE__)
template <class T>
T* f(uintptr_t off = 0) {
  return reinterpret_cast<T*>(uintptr_t(0x10000) + off);
}
}  // namespace

int main() {
  size_t b = 0;
  for (int64_t T : {int64_t(0), int64_t(1), int64_t(255), int64_t(4097), int64_t(1) << 20, int64_t(INT32_MAX) / 2})
    for (int64_t V : {8, 264, 128256})
      for (int64_t chunk : {int64_t(0), int64_t(1), int64_t(100000), std::numeric_limits<int64_t>::max() / 4}) {
        EXPECT(kd_token_logp_workspace_size(T, 2048, V, KD_BF16, KD_BF16, chunk, &b) == KD_OK);
        EXPECT(kd_token_logp_logits_size(T, V, &b) == KD_OK);
        EXPECT(kd_policy_loss_workspace_size(T, T, &b) == KD_OK);
        EXPECT(kd_preference_loss_workspace_size(T, 1 + T / 8, &b) == KD_OK);
      }
  const int64_t far = std::numeric_limits<int64_t>::max();
  EXPECT(kd_token_logp_workspace_size(far, 2048, 264, KD_BF16, KD_BF16, 0, &b) == KD_ERR_UNSUPPORTED);
  EXPECT(kd_token_logp_workspace_size(8, 2048, 264, KD_BF16, (kd_dtype)9, 0, &b) == KD_ERR_INVALID_ARG);
  EXPECT(kd_policy_loss_workspace_size(far, 1, &b) == KD_ERR_UNSUPPORTED);
  EXPECT(kd_policy_loss_workspace_size(1, far, &b) == KD_ERR_UNSUPPORTED);
  EXPECT(kd_token_logp_shard_combine(f<float>(), far, nullptr, 1.f, 8, f<float>(), f<float>(), nullptr, nullptr) ==
         KD_ERR_UNSUPPORTED);
  EXPECT(kd_token_logp_fwd_shard(f<char>(), f<char>(), f<int32_t>(), nullptr, 1.f, 8, 64, 256, far - 100, KD_BF16,
                                 f<float>(), nullptr, f<char>(), 0, nullptr) == KD_ERR_UNSUPPORTED);
  kd_policy_opts po{};
  po.reduction = (kd_reduction)77;
  po.kl_kind = KD_KL_3;
  EXPECT(kd_policy_loss_fwd(f<float>(), f<float>(), f<float>(), nullptr, &po, 8, nullptr, f<float>(), f<double>(),
                            f<char>(), 0, nullptr) == KD_ERR_INVALID_ARG);
  po.reduction = KD_TOKEN_MEAN;
  EXPECT(kd_policy_loss_fwd(f<float>(), f<float>(), f<float>(), nullptr, &po, 8, nullptr, f<float>(), f<double>(),
                            f<char>(), 0, nullptr) == KD_ERR_WORKSPACE_TOO_SMALL);
  kd_pref_opts pr{};
  pr.kind = (kd_pref_kind)50;
  pr.beta = 0.1;
  EXPECT(kd_preference_loss_fwd(f<float>(), f<int32_t>(), nullptr, &pr, 8, 2, f<float>(), f<float>(), f<double>(),
                                f<char>(), 0, nullptr) == KD_ERR_INVALID_ARG);
  pr.kind = KD_PREF_IPO;
  EXPECT(kd_preference_loss_fwd(f<float>(), f<int32_t>(), nullptr, &pr, 8, 2, f<float>(), f<float>(), f<double>(),
                                f<char>(), 0, nullptr) == KD_ERR_WORKSPACE_TOO_SMALL);
  // many tensors: counts, types, alignment and overlaps
  std::vector<const void*> in;
  std::vector<void*> out;
  std::vector<int64_t> n;
  std::vector<int32_t> ty;
  for (int i = 0; i < 500; ++i) {
    n.push_back(i % 7 ? 100 * i : 0);
    ty.push_back(i % 3);
    in.push_back(i % 7 ? f<char>(uintptr_t(i) << 20) : nullptr);
    out.push_back(i % 7 ? f<char>((uintptr_t(i) << 20) + (1u << 19)) : nullptr);
  }
  EXPECT(kd_grad_norm_workspace_size(n.data(), 500, &b) == KD_OK);
  EXPECT(kd_grad_sumsq(in.data(), n.data(), ty.data(), 500, nullptr, f<char>(), b, nullptr) == KD_ERR_INVALID_ARG);
  EXPECT(kd_grad_clip(in.data(), n.data(), ty.data(), 500, out.data(), ty.data(), nullptr, 1.0, nullptr, nullptr) ==
         KD_ERR_INVALID_ARG);
  out[499] = out[498];
  EXPECT(kd_grad_clip(in.data(), n.data(), ty.data(), 500, out.data(), ty.data(), f<double>(), 1.0, f<float>(),
                      nullptr) == KD_ERR_INVALID_ARG);
  n[3] = far;
  EXPECT(kd_grad_norm_workspace_size(n.data(), 500, &b) == KD_ERR_UNSUPPORTED);
  std::printf("ok: %d failure(s)\n", failures);
  return failures != 0;
}
