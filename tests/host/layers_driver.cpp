// Host-side checks of kdlayers.h's argument validation and planning under the
// address and undefined-behaviour sanitizers.  Every call is rejected, or
// sizes a buffer, before its first HIP call.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>

#include "kdlayers.h"

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
const kd_dtype kHalf = (kd_dtype)KD_F16;
}  // namespace

int main() {
  size_t b = 0;
  const int64_t top = (int64_t(1) << 30) - 1, far = std::numeric_limits<int64_t>::max();
  for (int64_t T : {int64_t(0), int64_t(1), int64_t(255), int64_t(16384), int64_t(16385), top})
    for (int64_t d : {int64_t(1), int64_t(16), int64_t(4096), int64_t(131056), (int64_t(1) << 24) - 1}) {
      for (int64_t V : {int64_t(1), int64_t(300), int64_t(128256), top})
        for (int tied : {0, 1}) EXPECT(kd_embedding_workspace_size(T, V, d, tied, &b) == KD_OK);
      EXPECT(kd_layer_norm_workspace_size(T, d, &b) == KD_OK);
      const kd_status want = d % 16 || d >= (1 << 17) ? KD_ERR_UNSUPPORTED : KD_OK;
      EXPECT(kd_int8_matmul_workspace_size(T, d, 128256, &b) == want);
    }
  for (int64_t bad : {far, std::numeric_limits<int64_t>::min(), int64_t(-1)}) {
    EXPECT(kd_embedding_workspace_size(bad, 10, 8, 1, &b) != KD_OK);
    EXPECT(kd_embedding_workspace_size(10, bad, 8, 0, &b) != KD_OK);
    EXPECT(kd_embedding_workspace_size(10, 10, bad, 1, &b) != KD_OK);
    EXPECT(kd_layer_norm_workspace_size(bad, 8, &b) != KD_OK);
    EXPECT(kd_int8_matmul_workspace_size(bad, 16, 8, &b) != KD_OK);
    EXPECT(kd_int8_matmul_workspace_size(8, 16, bad, &b) != KD_OK);
  }
  EXPECT(kd_layer_norm_workspace_size(8, 8, nullptr) == KD_ERR_INVALID_ARG);

  EXPECT(kd_embedding_fwd(f<int32_t>(), f<void>(), nullptr, NAN, 8, 10, 8, KD_BF16, 0, f<void>(), nullptr) ==
         KD_ERR_INVALID_ARG);
  EXPECT(kd_embedding_fwd(f<int32_t>(), f<void>(1), nullptr, 1.f, 8, 10, 8, kHalf, 1, f<void>(), nullptr) ==
         KD_ERR_ALIGNMENT);
  EXPECT(kd_embedding_bwd(f<void>(), f<int32_t>(), nullptr, 1.f, 8, 10, 8, KD_BF16, KD_F32, 1, 0, f<void>(), f<void>(),
                          8, nullptr) == KD_ERR_WORKSPACE_TOO_SMALL);
  EXPECT(kd_embedding_bwd(nullptr, nullptr, nullptr, 1.f, 0, 10, 8, KD_BF16, KD_F32, 1, 1, f<void>(), nullptr, 0,
                          nullptr) == KD_OK);
  for (int64_t g : {int64_t(1), int64_t(-32), int64_t(33), far})
    EXPECT(kd_rows_quantize(f<void>(), 8, 64, KD_F32, KD_ROWS_INT8, g, f<void>(), f<float>(), nullptr) ==
           KD_ERR_INVALID_ARG);
  EXPECT(kd_rows_dequantize(f<void>(), nullptr, 8, 64, KD_ROWS_E4M3, 0, KD_F32, f<void>(), nullptr) ==
         KD_ERR_INVALID_ARG);
  EXPECT(kd_layer_norm_fwd(f<void>(), nullptr, nullptr, nullptr, -1e-9, 8, 64, KD_F32, KD_F32, f<void>(), nullptr,
                           nullptr, KD_ROWS_NONE, 0, nullptr, nullptr, nullptr) == KD_ERR_INVALID_ARG);
  EXPECT(kd_layer_norm_bwd(f<void>(), f<void>(), nullptr, nullptr, f<float>(), f<float>(), 8, 64, KD_F32, KD_F32,
                           KD_ROWS_NONE, 0, nullptr, nullptr, f<void>(), nullptr, nullptr, f<void>(), 0,
                           nullptr) == KD_ERR_WORKSPACE_TOO_SMALL);
  EXPECT(kd_int8_matmul(f<int8_t>(), f<float>(), f<int8_t>(), f<float>(), 4096, 4096, 32000, KD_BF16, f<void>(),
                        f<void>(), 100, nullptr) == KD_ERR_WORKSPACE_TOO_SMALL);
  EXPECT(kd_int8_matmul(f<int8_t>(8), f<float>(), f<int8_t>(), f<float>(), 4, 4096, 32000, KD_BF16, f<void>(), nullptr,
                        0, nullptr) == KD_ERR_ALIGNMENT);
  std::printf("ok: %d failure(s)\n", failures);
  return failures != 0;
}
