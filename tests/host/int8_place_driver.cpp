// The addresses of the integer product's tiles (kd_int8_place.h), gone through
// on the host: every load of every lane lies inside its array by its whole
// address, or is dropped by its vector offset alone, and the products that the
// stages add up are those of the row, each once.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "kd_int8_place.h"

using namespace kd;

namespace {
int failures = 0;
void expect(bool ok, const char* what, long a, long b, long c, long d) {
  if (!ok && ++failures <= 20) std::printf("FAILED %s: %ld %ld %ld %ld\n", what, a, b, c, d);
}

void contraction(long d) {
  std::vector<int> seen(d / 16, 0);
  for (long s = 0; s < 4 * int8_turns(d); ++s)
    for (long c = 0; c < 4; ++c) {
      const long w = int8_stage_at(s, d) + int8_chunk_at(c, d), x = int8_x_at(s, c, d);
      expect(w >= 0 && w % 16 == 0 && w + 16 <= d, "w's row", d, s, c, w);
      expect(x == -1 || x == w, "x's chunk for w's", d, s, c, x);
      if (x >= 0) ++seen[x / 16];
    }
  for (long k = 0; k < d / 16; ++k) expect(seen[k] == 1, "each chunk once", d, k, seen[k], 0);
}

// One tile of rows [row0, row0 + 256) and channels [n0, n0 + 256).
void tile(long T, long d, long V, long row0, long n0) {
  const long stages = 4 * int8_turns(d), rows = int8_panel_rows(T), x_bytes = rows * stages * 64 - row0 * 64,
             w_bytes = (V - n0) * d;
  for (long m = 0; m < 256; ++m) {
    for (long c = 0; c < 4; ++c)
      for (long s = 0; s < stages; ++s) {
        const long x = m * 64 + 16 * c + s * rows * 64;  // vector and scalar offset
        expect(x >= 0 && x + 16 <= x_bytes, "panels", T, d, m, x);
        const long v = m * d + int8_chunk_at(c, d), u = int8_stage_at(s, d);
        if (n0 + m < V) expect(v + u + 16 <= w_bytes, "w", V, d, m, s);
        else expect(v >= w_bytes, "w's rows behind the last one", V, d, m, s);
      }
  }
}
}  // namespace

int main() {
  for (long d = 16; d <= 4096; d += 16) contraction(d);
  for (long d : {long(131056), long(131008), long(65552)}) contraction(d);
  for (long d : {16L, 32L, 48L, 64L, 80L, 208L, 256L, 272L, 1040L})
    for (long T : {65L, 255L, 256L, 257L, 300L, 511L, 513L})
      for (long V : {1L, 63L, 255L, 256L, 257L, 500L})
        for (long row0 = 0; row0 < T; row0 += 256)
          for (long n0 = 0; n0 < V; n0 += 256) tile(T, d, V, row0, n0);
  std::printf("ok: %d failure(s)\n", failures);
  return failures != 0;
}
