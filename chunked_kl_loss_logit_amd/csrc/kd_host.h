// Host side shared by the C-ABI files: the last error, the profiling record,
// argument checks, workspace carving and the launch shapes of the tile
// kernels.  Every argument check runs on the host before any HIP call, so a
// rejected call enqueues nothing.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <vector>

#include "kd_launch.h"
#include "kdloss.h"

namespace kdh {

inline thread_local std::string g_err;

inline kd_status fail(kd_status s, const std::string& msg) {
  g_err = msg;
  return s;
}

// ------------------------------------------------------------------ profiling
struct ProfEvent {
  const char* name;
  hipEvent_t a, b;
};
inline std::mutex g_prof_mu;
inline bool g_prof_on = false;
inline std::vector<ProfEvent> g_prof_pending;
inline std::vector<std::string> g_prof_names;
inline std::map<std::string, std::pair<int64_t, double>> g_prof_tot;

// Set while a call that may not allocate runs on this thread: its launches
// are not bracketed by events (hipEventCreate allocates).
inline thread_local bool g_no_alloc = false;

// Runs one launcher; while profiling, brackets it with events on `st`.
template <class F>
inline hipError_t run(const char* name, hipStream_t st, F&& launch) {
  if (!g_prof_on || g_no_alloc) return launch();
  hipEvent_t a = nullptr, b = nullptr;
  if (hipEventCreate(&a) != hipSuccess || hipEventCreate(&b) != hipSuccess) return launch();
  (void)hipEventRecord(a, st);
  const hipError_t e = launch();
  (void)hipEventRecord(b, st);
  std::lock_guard<std::mutex> g(g_prof_mu);
  g_prof_pending.push_back({name, a, b});
  return e;
}

inline void prof_fold() {
  std::lock_guard<std::mutex> g(g_prof_mu);
  for (auto& p : g_prof_pending) {
    float ms = 0.f;
    if (hipEventSynchronize(p.b) == hipSuccess && hipEventElapsedTime(&ms, p.a, p.b) == hipSuccess) {
      auto it = g_prof_tot.find(p.name);
      if (it == g_prof_tot.end()) {
        g_prof_names.push_back(p.name);
        it = g_prof_tot.emplace(p.name, std::make_pair(int64_t(0), 0.0)).first;
      }
      it->second.first += 1;
      it->second.second += ms;
    }
    (void)hipEventDestroy(p.a);
    (void)hipEventDestroy(p.b);
  }
  g_prof_pending.clear();
}

// ------------------------------------------------------------------ shapes and checks
constexpr size_t kAlign = 256;
inline size_t up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline int elem_of(kd_dtype dt) { return dt == KD_BF16 ? 2 : 4; }

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline kd_status check_common(int64_t T, int64_t d, int64_t V, kd_dtype dt, float tau) {
  if (dt != KD_F32 && dt != KD_BF16) return fail(KD_ERR_INVALID_ARG, "dtype must be KD_F32 or KD_BF16");
  if (T < 0) return fail(KD_ERR_INVALID_ARG, "T must be >= 0");
  if (d < 1) return fail(KD_ERR_INVALID_ARG, "d must be >= 1");
  if (V < 1) return fail(KD_ERR_INVALID_ARG, "V must be >= 1");
  if (!(tau > 0.f) || !std::isfinite(tau)) return fail(KD_ERR_INVALID_ARG, "tau must be finite and > 0");
  const int64_t epc = dt == KD_BF16 ? 8 : 4;
  if (d % epc) return fail(KD_ERR_UNSUPPORTED, "d must be a multiple of 8 (bf16) or 4 (fp32)");
  if (V % epc) return fail(KD_ERR_UNSUPPORTED, "V must be a multiple of 8 (bf16) or 4 (fp32)");
  if (T > INT32_MAX / 2 || V > INT32_MAX / 2 || d > INT32_MAX / 2)
    return fail(KD_ERR_UNSUPPORTED, "T, d and V must be below 2^30");
  return KD_OK;
}

inline kd_status need(const void* p, const char* name) {
  if (p == nullptr) return fail(KD_ERR_INVALID_ARG, std::string(name) + " is NULL");
  return KD_OK;
}

inline kd_status need_align(const void* p, size_t a, const char* name) {
  if (p != nullptr && !aligned(p, a))
    return fail(KD_ERR_ALIGNMENT, std::string(name) + " must be " + std::to_string(a) + "-byte aligned");
  return KD_OK;
}

#define KD_TRY(x)                   \
  do {                              \
    const kd_status _s = (x);       \
    if (_s != KD_OK) return _s;     \
  } while (0)

#define KD_LAUNCH(name, st, call)                                                              \
  do {                                                                                         \
    const hipError_t _e = run(name, st, [&]() { return (call); });                             \
    if (_e != hipSuccess) return fail(KD_ERR_HIP, std::string(name) + ": " + hipGetErrorString(_e)); \
  } while (0)

// Row blocks per raster group of the tile kernels: consecutive workgroups of
// one XCD share a row block's operand across this many row blocks (grouped_coords).
// Sweeping 1..16 at the 4096 x 3072 x 128256 head moved each kernel by under 4%.
// (dW over all its row blocks in one group ran 1% faster but fetched 60% more
// from HBM, 10.8 instead of 6.8 GB per launch.)
constexpr int kRasterGroup = 4;

// Vocabulary splits of the tile kernels: enough workgroups to fill the CUs,
// and at least 8 so that at large T the workgroups running together read
// several W panels instead of all hammering one.
// Splits of `work` units (vocabulary tiles or stage groups) for `units`
// independent tile rows, at most max_s: the tile kernels run one workgroup
// per CU, so the launch takes ceil(units * S / 256) rounds of ceil(work / S)
// units each, plus about two units per workgroup of fixed cost (ring fill,
// partials); the S with the lowest total wins, ties going to fewer splits.  A
// rule such as ceil(256 / units) overshoots 256 workgroups by a few whenever
// units does not divide 256 (15 row blocks: 270 workgroups, a second round
// for 14 of them).
inline int balanced_splits(int64_t units, int64_t work, int64_t max_s) {
  units = std::max<int64_t>(1, units);
  int best = 1;
  int64_t cost = INT64_MAX;
  for (int64_t s = 1; s <= std::max<int64_t>(1, std::min(max_s, work)); ++s) {
    const int64_t c = cdiv(units * s, 256) * (cdiv(work, s) + 2);
    if (c < cost) {
      cost = c;
      best = (int)s;
    }
  }
  return best;
}

inline int splits_for(int64_t nrb, int64_t ntiles) { return balanced_splits(nrb, ntiles, ntiles); }

// Launch shape of the tile kernels for the chunk of C rows at c0: row blocks
// of the rows it can hold (a last partial chunk gets fewer, and more splits),
// and the splits that fill the GPU with them.  S never exceeds
// max_splits(ntiles), which sizes the per-chunk partial buffers.
struct ChunkShape {
  int nrb, S;
};
inline ChunkShape chunk_shape(int64_t T, int64_t c0, int64_t C, int64_t ntiles) {
  const int nrb = (int)cdiv(std::min(C, T - c0), kd::kTileM);
  return {nrb, splits_for(nrb, ntiles)};
}
inline int64_t max_splits(int64_t ntiles) { return splits_for(1, ntiles); }

// Rows per backward chunk: the request (or the default), at most the rows
// present, rounded up to whole 256-row tiles, and for bf16 at most what keeps
// the chunk's dZ buffer within the 32-bit offsets of the direct-to-LDS loads
// that dH and dW read it with, rounded down to a multiple of the default
// chunk when that is possible (16384 rows at V = 128256: a cap of 65 row
// blocks would launch the tiles in poorly filled rounds).
inline int64_t chunk_of(int64_t T, int64_t V, int elem, int64_t chunk_rows) {
  int64_t C = chunk_rows <= 0 ? KD_DEFAULT_CHUNK_ROWS : chunk_rows;
  C = std::min(C, std::max<int64_t>(T, 1));  // before rounding up, which would pass INT64_MAX
  C = (int64_t)up((size_t)C, 256);
  if (elem == 2) {
    const int64_t ldz = cdiv(V, kd::kTileN) * kd::kTileN;
    int64_t cmax = ((int64_t(1) << 32) - 65537) / (ldz * 2) / 256 * 256;
    if (cmax >= KD_DEFAULT_CHUNK_ROWS) cmax = cmax / KD_DEFAULT_CHUNK_ROWS * KD_DEFAULT_CHUNK_ROWS;
    C = std::min<int64_t>(C, std::max<int64_t>(cmax, 256));
  }
  return C;
}

struct Carver {
  size_t off = 0;
  size_t take(size_t bytes) {
    const size_t o = off;
    off = up(off + bytes, kAlign);
    return o;
  }
};

// Bytes of `rows` rows of row_bytes each in 64-byte panels (a last partial
// piece takes a whole slot).
inline size_t panel_bytes(int64_t rows, int64_t row_bytes) { return (size_t)rows * (size_t)cdiv(row_bytes, 64) * 64; }

// Backward chunk buffers shared by both variants.
struct ChunkPlan {
  int64_t C, ldz;
  int nrb_c, nrb_dh, ncb_dh, S_dh, nrb_dw, ncb_dw;
  size_t o_dz, o_hT, o_dhp, o_hp;  // o_hp: the chunk's rows of H in panels
};

inline ChunkPlan plan_chunk(int64_t T, int64_t d, int64_t V, int elem, int64_t chunk_rows, Carver& cv) {
  ChunkPlan p{};
  p.C = chunk_of(T, V, elem, chunk_rows);
  p.ldz = cdiv(V, kd::kTileN) * kd::kTileN;
  p.nrb_c = (int)(p.C / kd::kTileM);
  p.nrb_dh = p.nrb_c;
  p.ncb_dh = (int)cdiv(d, 256);
  // dH splits the vocabulary (whole groups of four 64-byte stages); at most
  // enough splits for four rounds, which bounds the fp32 partials
  const int64_t units = (int64_t)p.nrb_dh * p.ncb_dh;
  p.S_dh = balanced_splits(units, cdiv(V * elem, 256), std::max<int64_t>(1, cdiv(1024, units)));
  p.nrb_dw = (int)cdiv(d, 256);
  p.ncb_dw = (int)cdiv(V, 256);
  p.o_dz = cv.take((size_t)p.C * p.ldz * elem);
  p.o_hT = cv.take((size_t)d * p.C * elem);
  p.o_dhp = cv.take((size_t)p.S_dh * p.C * d * 4);
  p.o_hp = cv.take(panel_bytes(p.C, d * elem));
  return p;
}

template <class T>
inline T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

inline kd_status check_workspace(const void* ws, size_t have, size_t want) {
  if (want > 0) KD_TRY(need(ws, "workspace"));
  KD_TRY(need_align(ws, kAlign, "workspace"));
  if (have < want)
    return fail(KD_ERR_WORKSPACE_TOO_SMALL,
                "workspace has " + std::to_string(have) + " bytes, needs " + std::to_string(want));
  return KD_OK;
}

// dH and dW of one backward chunk whose dZ sits in the chunk buffer:
// H^T of the chunk's rows, dH split over the vocabulary and reduced in a
// fixed order (into dH's element size dh_elem, 0 = the inputs'), dW stored
// (first chunk) or added in place.
inline kd_status grad_chunk(const void* H, const void* W, void* dH, float* dW, int elem, int64_t d, int64_t V,
                     const kd::Compact& c, const ChunkPlan& ch, char* dz, char* hT, float* dhp, int64_t c0,
                     bool accumulate, hipStream_t st, int dh_elem = 0) {
  KD_LAUNCH("gather_transpose", st, kd::launch_gather_transpose(H, elem, d, c, c0, ch.C, hT, st));
  if (c0 == 0 && kd::dh_direct(elem, V) && V % 128 != 0)  // the dH ring reads the chunk's columns up to ldz
    KD_LAUNCH("fill_zero", st,
              kd::launch_fill_zero(dz + kd::dz_tail_offset(ch.C, V), kd::dz_tail_bytes(ch.C, V, ch.ldz), st));
  kd::DhArgs ha{};
  ha.dz = dz;
  ha.W = static_cast<const char*>(W);
  ha.part = dhp;
  ha.count = c.count;
  ha.c0 = c0;
  ha.C = ch.C;
  ha.ldz = ch.ldz;
  ha.d = d;
  ha.V = V;
  ha.nrb = ch.nrb_dh;
  ha.ncb = ch.ncb_dh;
  ha.group = kRasterGroup;
  ha.S = ch.S_dh;
  KD_LAUNCH("dh_tile", st, kd::launch_dh(elem, ha, st));
  KD_LAUNCH("reduce_dh", st, kd::launch_reduce_dh(dhp, ch.S_dh, ch.C, d, c, c0, dH, dh_elem ? dh_elem : elem, st));
  kd::DwArgs wa{};
  wa.hT = hT;
  wa.dz = dz;
  wa.dW = dW;
  wa.count = c.count;
  wa.c0 = c0;
  wa.C = ch.C;
  wa.ldz = ch.ldz;
  wa.d = d;
  wa.V = V;
  wa.nrb = ch.nrb_dw;
  wa.ncb = ch.ncb_dw;
  wa.group = kRasterGroup;
  wa.accumulate = accumulate;
  KD_LAUNCH("dw_tile", st, kd::launch_dw(elem, wa, st));
  return KD_OK;
}

}  // namespace kdh
