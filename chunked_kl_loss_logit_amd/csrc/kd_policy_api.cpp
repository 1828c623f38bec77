// C-ABI entry points of kdpolicy.h: argument checks, workspace planning and
// the launch sequence of each call.
#include <exception>

#include "kd_host.h"
#include "kd_policy.h"
#include "kdpolicy.h"

using namespace kdh;

namespace {

// ---------------------------------------------------------------- token log-probabilities
// Whether the forward runs on the register-fed tiles (kd_direct.h) rather than the
// 256 x 256 ring tiles: float32, shapes the ring does not take, and bf16
// products too small to fill the ring's rounds of 256 workgroups.  A round
// costs the ring the same however few of its rows and tiles are real; the
// register-fed tiles run at 0.4 of a full round's rate.  Forward, us, ring /
// register-fed: 32 x 4096 x 8192 84 / 31, 64 x 2048 x 128256 152 / 125, 128 x
// 4096 x 32000 87 / 67, 512 x 4096 x 8192 88 / 63; on the other side 128 x 2048
// x 128256 153 / 185, 256 x 4096 x 32000 95 / 124, 1024 x 4096 x 8192 94 / 119.
bool direct_fwd(int64_t T, int64_t d, int64_t V, int elem) {
  const int64_t C = chunk_of(T, V, elem, 0);
  if (!kd::logp_ring_fits(elem, C, d, V)) return true;
  const int64_t rounds = cdiv(cdiv(std::min(T, C), kd::kTileM) * cdiv(V, kd::kTileN), 256);
  return std::min(T, C) * V < rounds * 7000000;
}

// The most rows of row_bytes each, in whole 256-row tiles, that the ring's
// 32-bit offsets reach; 0 where not even one tile's.
int64_t ring_rows(int64_t row_bytes) { return ((int64_t(1) << 32) - 65537) / row_bytes / 256 * 256; }

// Columns of dZ, and what a row of the ring's dZ panels takes with the tail pieces.
int64_t ldz_of(int64_t V) { return cdiv(V, kd::kTileN) * kd::kTileN; }
int64_t ring_dz_bytes(int64_t V) { return (ldz_of(V) + 32 * kd::kDzTailPieces) * 2; }

// The same for the backward, whose products the ring splits better (dH over
// the vocabulary) but pays more launches for: up to 64 rows, and products of
// fewer than 7e9 terms.  Backward, us, recomputing / from kept logits, ring
// against register-fed: 64 x 2048 x 128256 501 / 438, 477 / 368; 1024 x 1024 x
// 4096 102 / 75, 78 / 61; 4096 x 512 x 2048 145 / 126, 113 / 85; on the other
// side 65 x 2048 x 128256 498 / 438, 646 / 476; 700 x 4096 x 4096 165 / 91, 200
// / 137; 512 x 4096 x 8192 187 / 114, 213 / 163.
bool direct_bwd(int64_t T, int64_t d, int64_t V, int elem) {
  const int64_t C = chunk_of(T, V, elem, 0);
  if (!kd::logp_ring_fits(elem, C, d, V) || ring_rows(ring_dz_bytes(V)) == 0) return true;
  const int64_t n = std::min(T, C);
  return n <= 64 || (double)n * d * V < 7e9;
}

struct LogpPlan {
  bool fwd_direct, bwd_direct;
  int ntiles_f, ntiles;  // column tiles of the forward and of the backward's dZ
  int64_t Cf;    // rows per forward chunk
  int64_t C, ldz;  // rows per backward chunk, columns of its dZ
  int grid_dh;  // workgroups of dH
  size_t o_rows, o_count, o_part, o_hp_f, fwd_total;
  size_t o_dz, o_dhp;
  size_t o_hc;        // direct: the chunk's rows of H
  size_t o_hT, o_hp;  // ring: the same transposed and as they are, in panels
  size_t o_dw32, total;  // float32 dW where a bf16 one adds up over chunks
};

// Rows of a ring chunk, however many are asked for: H's panels (dp columns; at
// least the default chunk's rows, logp_ring_fits) and dZ's with the tail pieces
// keep to the ring's reach, dZ's cap in whole default chunks as chunk_of's is.
int64_t ring_chunk(int64_t T, int64_t V, int64_t dp, int64_t chunk_rows) {
  int64_t most = ring_rows(ring_dz_bytes(V));
  if (most >= KD_DEFAULT_CHUNK_ROWS) most = most / KD_DEFAULT_CHUNK_ROWS * KD_DEFAULT_CHUNK_ROWS;
  return std::min({chunk_of(T, V + 32 * kd::kDzTailPieces, 2, chunk_rows), ring_rows(dp * 2), most});
}

LogpPlan plan_logp(int64_t T, int64_t d, int64_t V, int elem, int dw_elem, int64_t chunk_rows) {
  LogpPlan p{};
  p.fwd_direct = direct_fwd(T, d, V, elem);
  p.bwd_direct = direct_bwd(T, d, V, elem);
  p.ntiles_f = (int)cdiv(V, p.fwd_direct ? kd::kDirectCols : kd::kTileN);
  p.ntiles = (int)cdiv(V, kd::kTileN);
  p.Cf = chunk_of(T, V, elem, 0);
  p.ldz = ldz_of(V);
  Carver cv;
  p.o_rows = cv.take((size_t)T * 4);
  p.o_count = cv.take(16);
  Carver fw = cv, bw = cv;  // the two calls' buffers overlap
  const int64_t dp = cdiv(d, 128) * 128;  // the ring's H panels run to whole ring turns of d
  if (p.fwd_direct) {
    p.o_part = fw.take((size_t)p.ntiles_f * p.Cf * 16);
  } else {
    p.o_part = fw.take((size_t)std::min(p.ntiles_f, kd::kRingMaxSplits) * p.Cf * 16);
    p.o_hp_f = fw.take(panel_bytes(p.Cf, dp * elem));
  }
  if (p.bwd_direct) {
    p.C = chunk_of(T, V, elem, chunk_rows);
    // dH's workgroups: for every CU, of vocabulary ranges of at least 1 KB of W's rows
    const int64_t nda = cdiv(d, 128), rows = kd::direct_dh_rows(std::min(p.C, T));
    const int64_t units = cdiv(std::min(p.C, T), rows) * nda;
    const int64_t S = balanced_splits(units, cdiv(V * elem, 1024), std::max<int64_t>(1, cdiv(1024, units)));
    p.grid_dh = (int)up(units * S, 256);
    p.o_dz = bw.take((size_t)p.C * p.ldz * elem);
    p.o_hc = bw.take((size_t)p.C * d * elem);
    p.o_dhp = bw.take((size_t)cdiv(p.grid_dh, nda) * kd::direct_dh_rows(T) * d * 4);
  } else {
    p.C = ring_chunk(T, V, dp, chunk_rows);
    const int64_t ncb = cdiv(d, 256), units = cdiv(std::min(p.C, T), kd::kTileM) * ncb;
    p.grid_dh = (int)up(units * balanced_splits(units, cdiv(V, 128), std::max<int64_t>(1, cdiv(1024, units))), 256);
    p.o_dz = bw.take((size_t)p.C * ring_dz_bytes(V));
    p.o_hT = bw.take((size_t)d * p.C * elem);
    p.o_dhp = bw.take((size_t)cdiv(p.grid_dh, ncb) * 256 * d * 4);
    p.o_hp = bw.take(panel_bytes(p.C, dp * elem));
  }
  p.fwd_total = fw.off;
  p.o_dw32 = bw.take(dw_elem == 2 && p.C < T ? (size_t)d * V * 4 : 0);
  p.total = std::max(fw.off, bw.off);
  return p;
}

kd_status check_dw_type(kd_dtype dt, kd_dtype dw) {
  if (dw != KD_F32 && dw != KD_BF16) return fail(KD_ERR_INVALID_ARG, "dw_dtype must be KD_F32 or KD_BF16");
  if (dw == KD_BF16 && dt != KD_BF16) return fail(KD_ERR_UNSUPPORTED, "a bf16 dW needs bf16 inputs");
  return KD_OK;
}

kd_status check_widths(int64_t T, int64_t d, int64_t V, kd_dtype dt, float tau) {
  KD_TRY(check_common(T, d, V, dt, tau));
  // the register-fed tiles address up to 16 rows of an operand with 32 bits
  if (d >= (1 << 25) || V >= (1 << 25)) return fail(KD_ERR_UNSUPPORTED, "d and V must be below 2^25");
  return KD_OK;
}

kd_status check_v0(int64_t V, int64_t v0) {
  if (v0 < 0) return fail(KD_ERR_INVALID_ARG, "v0 must be >= 0");
  if (v0 > INT32_MAX / 2 - V) return fail(KD_ERR_UNSUPPORTED, "v0 + V must be below 2^30");
  return KD_OK;
}

kd_status check_head(const void* H, const void* W, const int32_t* tokens) {
  KD_TRY(need(H, "H"));
  KD_TRY(need(W, "W"));
  KD_TRY(need(tokens, "tokens"));
  KD_TRY(need_align(H, 16, "H"));
  KD_TRY(need_align(W, 16, "W"));
  KD_TRY(need_align(tokens, 4, "tokens"));
  return KD_OK;
}

// Workgroups of the forward and dZ tiles for the chunk at c0: as many rounds
// of 256 as suit all its rows; the kernels divide them among the valid ones.
int ring_grid(int64_t T, int64_t c0, int64_t C, int64_t ntiles) {
  const ChunkShape sh = chunk_shape(T, c0, C, ntiles);
  return (int)(cdiv((int64_t)sh.nrb * sh.S, 256) * 256);
}

// The chunk's rows of H in panels, with zeros from d to the next multiple of 128.
kd_status head_panels(const void* H, int64_t d, const kd::Compact& c, int64_t c0, int64_t C, char* hp,
                      hipStream_t st) {
  KD_LAUNCH("gather_panels", st, kd::launch_gather_panels(H, d * 2, c, c0, C, hp, st));
  const int64_t dp = cdiv(d, 128) * 128;
  if (dp > d && c0 == 0)  // later chunks find them there
    KD_LAUNCH("fill_zero", st, kd::launch_fill_zero(hp + d / 32 * C * 64, (dp - d) / 32 * C * 64, st));
  return KD_OK;
}

// Whether a bf16 dZ keeps what its rounding leaves in a second plane.  dZ is
// rounded to the type of the products it feeds, as for the other losses; over
// many rows the roundings differ, and dH and dW are off by 0.0023 on average
// where their own rounding to bf16 makes 0.0017.  With few rows one entry of
// dZ, the token's, is most of a row of dH and of a column of dW, and its
// rounding, up to 2^-8, is that of the whole.  Up to 32 rows the products read
// and write W's size whatever dZ holds: a backward of 7 rows of 2048 x 32000
// took 110 us without the second plane and 119 with it.  T counts the masked
// rows too, since the launches are chosen where the mask is not known: 40 rows
// of which 5 are valid do without the plane, at the error of one rounding more.
bool logp_planes(int64_t T, int elem) { return elem == 2 && T <= 32; }

// The valid rows, the masked rows of dH (nullable) zeroed, and up to kPrepMax
// rows the first C of H's packed (Hc nullable): one launch, whose blocks each
// count the mask before them (T^2 / 16 bytes in all); beyond, one block counts
// (forward and backward of 1024 x 256 float32, us, one launch / apart: 777 rows
// 27 + 92 / 28 + 95, 16384 rows 107 + 1026 / 117 + 1049, 65536 rows 347 + 4050 /
// 415 + 4130).
constexpr int64_t kPrepMax = 65536;
kd_status direct_rows(const uint8_t* mask, int64_t T, const kd::Compact& c, const void* H, int64_t row_bytes,
                      int64_t C, char* Hc, void* dH, int64_t dh_row_bytes, hipStream_t st) {
  if (T <= kPrepMax) {
    KD_LAUNCH("logp_prep", st,
              kd::launch_logp_prep(mask, T, c.rows, c.count, H, row_bytes, C, Hc, dH, dh_row_bytes, st));
    return KD_OK;
  }
  KD_LAUNCH("compact", st, kd::launch_compact(mask, T, c, st));
  if (dH) KD_LAUNCH("zero_masked_rows", st, kd::launch_zero_masked_rows(mask, T, dh_row_bytes, dH, st));
  return KD_OK;
}

kd_status logp_fwd(const void* H, const void* W, const int32_t* tokens, const uint8_t* mask, float tau, int64_t T,
                   int64_t d, int64_t V, int64_t v0, kd_dtype dt, const kd::LogpOut& out, bool entropy, float* logits,
                   void* workspace, size_t workspace_bytes, void* stream) {
  const int elem = elem_of(dt);
  const LogpPlan p = plan_logp(T, d, V, elem, 4, 0);
  KD_TRY(check_workspace(workspace, workspace_bytes, p.fwd_total));
  hipStream_t st = static_cast<hipStream_t>(stream);
  const kd::Compact c{at<int32_t>(workspace, p.o_rows), at<int32_t>(workspace, p.o_count)};
  float* part = at<float>(workspace, p.o_part);
  const float c2 = (float)(1.4426950408889634 / (double)tau);
  kd::RowSet rs{c.rows, c.count, 0, p.Cf, T};
  if (p.fwd_direct) {
    if (mask)
      KD_TRY(direct_rows(mask, T, c, H, d * elem, 0, nullptr, nullptr, 0, st));
    else
      rs.rows = rs.count = nullptr;
    kd::LogpDirectArgs a{};
    a.H = static_cast<const char*>(H);
    a.W = static_cast<const char*>(W);
    a.tokens = tokens;
    a.d = d;
    a.V = V;
    a.ldz = p.ldz;
    a.v0 = (int32_t)v0;
    a.c2 = c2;
    a.part = part;
    for (int64_t c0 = 0; c0 < T; c0 += p.Cf) {
      rs.c0 = c0;
      a.rs = rs;
      a.z = logits ? logits + c0 * p.ldz : nullptr;
      KD_LAUNCH("logp_direct_fwd", st, kd::launch_logp_direct_fwd(elem, a, entropy, st));
      KD_LAUNCH("logp_combine", st,
                kd::launch_logp_combine(part, p.ntiles_f, 0, rs, mask, tokens, V, c2, out, c0 == 0, st));
    }
    return KD_OK;
  }
  char* hp = at<char>(workspace, p.o_hp_f);
  KD_LAUNCH("compact", st, kd::launch_compact(mask, T, c, st));
  kd::LogpFwdArgs a{};
  a.Hp = hp;
  a.W = static_cast<const char*>(W);
  a.c = c;
  a.tokens = tokens;
  a.part = part;
  a.ldz = p.ldz;
  a.C = p.Cf;
  a.d = d;
  a.V = V;
  a.v0 = (int32_t)v0;
  a.ntiles = p.ntiles_f;
  a.group = kRasterGroup;
  a.c2 = c2;
  for (int64_t c0 = 0; c0 < T; c0 += p.Cf) {
    const int grid = ring_grid(T, c0, p.Cf, p.ntiles_f);
    KD_TRY(head_panels(H, d, c, c0, p.Cf, hp, st));
    a.c0 = rs.c0 = c0;
    a.zout = logits ? logits + c0 * p.ldz : nullptr;
    a.grid = grid;
    KD_LAUNCH("logp_fwd_tile", st, kd::launch_logp_fwd(a, entropy, st));
    KD_LAUNCH("logp_combine", st,
              kd::launch_logp_combine(part, p.ntiles_f, grid, rs, mask, tokens, V, c2, out, c0 == 0, st));
  }
  return KD_OK;
}

kd_status logp_bwd(const void* H, const void* W, const int32_t* tokens, const uint8_t* mask, float tau, int64_t T,
                   int64_t d, int64_t V, int64_t v0, kd_dtype dt, const float* lse, const float* entropy,
                   const float* logits, const float* g, const float* ge, void* dH, int dh_elem, void* dW,
                   kd_dtype dw_dtype, int64_t chunk_rows, void* workspace, size_t workspace_bytes, void* stream) {
  g_err.clear();
  KD_TRY(check_widths(T, d, V, dt, tau));
  KD_TRY(check_v0(V, v0));
  KD_TRY(check_dw_type(dt, dw_dtype));
  if (chunk_rows < 0) return fail(KD_ERR_INVALID_ARG, "chunk_rows must be >= 0");
  if (!dH && !dW && T > 0) return fail(KD_ERR_INVALID_ARG, "dH and dW are both NULL");
  KD_TRY(need_align(dW, 16, "dW"));
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (T == 0) {
    if (dW) KD_LAUNCH("fill_zero", st, kd::launch_fill_zero(dW, d * V * elem_of(dw_dtype), st));
    return KD_OK;
  }
  KD_TRY(check_head(H, W, tokens));
  KD_TRY(need(lse, "lse"));
  KD_TRY(need_align(dH, 16, "dH"));
  KD_TRY(need_align(lse, 4, "lse"));
  KD_TRY(need_align(g, 4, "grad_logp"));
  KD_TRY(need_align(ge, 4, "grad_entropy"));
  KD_TRY(need_align(entropy, 4, "entropy"));
  KD_TRY(need_align(logits, 16, "logits"));
  if (!g && !ge) return fail(KD_ERR_INVALID_ARG, "grad_logp and grad_entropy are both NULL");
  if (ge) KD_TRY(need(entropy, "entropy (grad_entropy needs it)"));
  const int elem = elem_of(dt);
  const LogpPlan p = plan_logp(T, d, V, elem, elem_of(dw_dtype), chunk_rows);
  KD_TRY(check_workspace(workspace, workspace_bytes, p.total));

  const kd::Compact c{at<int32_t>(workspace, p.o_rows), at<int32_t>(workspace, p.o_count)};
  const float c2 = (float)(1.4426950408889634 / (double)tau), inv_tau = (float)(1.0 / (double)tau);
  if (p.bwd_direct) {
    kd::LogpDirectArgs a{};
    a.H = static_cast<const char*>(H);
    a.W = static_cast<const char*>(W);
    a.tokens = tokens;
    a.d = d;
    a.V = V;
    a.ldz = p.ldz;
    a.v0 = (int32_t)v0;
    a.c2 = c2;
    a.inv_tau = inv_tau;
    a.lse = lse;
    a.ent = entropy;
    a.g = g;
    a.ge = ge;
    a.dz = at<char>(workspace, p.o_dz);
    a.lo = logp_planes(T, elem) ? 128 * p.ldz * elem : 0;  // a chunk has at least 256 rows of room
    float* dw32 = p.C < T ? at<float>(workspace, p.o_dw32) : nullptr;
    for (int64_t c0 = 0; c0 < T; c0 += p.C) {
      a.rs = kd::RowSet{mask ? c.rows : nullptr, c.count, c0, p.C, T};
      const char* hc = a.H + c0 * d * elem;
      if (mask) {
        char* packed = dW ? at<char>(workspace, p.o_hc) : nullptr;
        if (c0 == 0)
          KD_TRY(direct_rows(mask, T, c, H, d * elem, p.C, packed, dH, d * dh_elem, st));
        if (packed && (c0 > 0 || T > kPrepMax))
          KD_LAUNCH("logp_pack", st, kd::launch_logp_pack(a.rs, H, d * elem, packed, st));
        hc = packed;
      }
      if (logits) {
        a.z = const_cast<float*>(logits) + c0 * p.ldz;
        KD_LAUNCH("logp_direct_dz_from_z", st, kd::launch_logp_direct_dz_from_z(elem, a, st));
      } else {
        KD_LAUNCH("logp_direct_dz", st, kd::launch_logp_direct_dz(elem, a, st));
      }
      if (dH)
        KD_LAUNCH("logp_direct_dh", st,
                  kd::launch_logp_direct_dh(elem, a, p.grid_dh, at<float>(workspace, p.o_dhp), dH, dh_elem, st));
      if (!dW) continue;
      // a float32 dW adds up in place; a bf16 one in the workspace, rounded with the last chunk
      const bool f32 = dw_dtype == KD_F32, last = c0 + p.C >= T;
      float* acc = f32 ? static_cast<float*>(dW) : dw32;
      KD_LAUNCH("logp_direct_dw", st,
                kd::launch_logp_direct_dw(elem, a, hc, c0 > 0 ? acc : nullptr, f32 || !last ? acc : dW,
                                          f32 || !last ? 4 : 2, st));
    }
    return KD_OK;
  }
  char* dz = at<char>(workspace, p.o_dz);
  char* hT = at<char>(workspace, p.o_hT);
  char* hp = at<char>(workspace, p.o_hp);
  float* dhp = at<float>(workspace, p.o_dhp);
  const bool dw_direct = dw_dtype == KD_BF16 && p.C >= T;  // one chunk: rounded where it is made
  float* dw32 = dw_dtype == KD_F32 ? static_cast<float*>(dW) : at<float>(workspace, p.o_dw32);
  KD_LAUNCH("compact", st, kd::launch_compact(mask, T, c, st));
  if (dH) KD_LAUNCH("zero_masked_rows", st, kd::launch_zero_masked_rows(mask, T, d * dh_elem, dH, st));
  // dH's last ring turn: zero pieces after dZ's tail piece
  const int64_t stages = cdiv(V, 32), pads = cdiv(stages, 4) * 4 - stages, tail = V % 32 ? 1 : 0;
  if (dH && pads > 0)
    KD_LAUNCH("fill_zero", st, kd::launch_fill_zero(dz + (p.ldz / 32 + tail) * p.C * 64, pads * p.C * 64, st));
  kd::LogpDzArgs a{};
  a.Hp = hp;
  a.W = static_cast<const char*>(W);
  a.c = c;
  a.tokens = tokens;
  a.lse = lse;
  a.ent = entropy;
  a.g = g;
  a.ge = ge;
  a.dz = dz;
  a.ldz = p.ldz;
  a.C = p.C;
  a.d = d;
  a.V = V;
  a.v0 = (int32_t)v0;
  a.ntiles = p.ntiles;
  a.group = kRasterGroup;
  a.c2 = c2;
  a.inv_tau = inv_tau;
  for (int64_t c0 = 0; c0 < T; c0 += p.C) {
    a.c0 = c0;
    if (logits) {
      a.z = logits + c0 * p.ldz;
      KD_LAUNCH("logp_dz_from_z", st, kd::launch_logp_dz_from_z(a, st));
    } else {
      a.grid = ring_grid(T, c0, p.C, p.ntiles);
      KD_TRY(head_panels(H, d, c, c0, p.C, hp, st));
      KD_LAUNCH("logp_dz_tile", st, kd::launch_logp_dz(a, st));
    }
    kd::LogpDhArgs ha{};
    ha.dz = dz;
    ha.W = a.W;
    ha.part = dhp;
    ha.count = c.count;
    ha.T = T;
    ha.c0 = c0;
    ha.C = p.C;
    ha.ldz = p.ldz;
    ha.d = d;
    ha.V = V;
    ha.grid = p.grid_dh;
    ha.ncb = (int)cdiv(d, 256);
    ha.group = kRasterGroup;
    if (dH) KD_LAUNCH("logp_dh_tile", st, kd::launch_logp_dh(ha, c.rows, dH, dh_elem, st));
    if (!dW) continue;
    KD_LAUNCH("gather_transpose", st, kd::launch_gather_transpose(H, elem, d, c, c0, p.C, hT, st));
    kd::DwArgs wa{};
    wa.hT = hT;
    wa.dz = dz;
    wa.dW = dw32;
    wa.count = c.count;
    wa.c0 = c0;
    wa.C = p.C;
    wa.ldz = p.ldz;
    wa.d = d;
    wa.V = V;
    wa.nrb = (int)cdiv(d, 256);
    wa.ncb = (int)cdiv(V, 256);
    wa.group = kRasterGroup;
    wa.accumulate = c0 > 0;
    if (dw_direct)
      KD_LAUNCH("logp_dw_tile", st, kd::launch_logp_dw_bf16(wa, dW, st));
    else
      KD_LAUNCH("dw_tile", st, kd::launch_dw(elem, wa, st));
  }
  if (dW && dw_dtype == KD_BF16 && !dw_direct) KD_LAUNCH("to_bf16", st, kd::launch_to_bf16(dw32, dW, d * V, st));
  return KD_OK;
}

}  // namespace

extern "C" {

kd_status kd_token_logp_logits_size(int64_t T, int64_t V, size_t* bytes) {
  g_err.clear();
  KD_TRY(need(bytes, "bytes"));
  KD_TRY(check_widths(T, 8, V, KD_F32, 1.0f));
  *bytes = (size_t)T * (size_t)ldz_of(V) * 4;
  return KD_OK;
}

kd_status kd_token_logp_fwd_workspace_size(int64_t T, int64_t d, int64_t V, kd_dtype dt, size_t* bytes) {
  g_err.clear();
  KD_TRY(need(bytes, "bytes"));
  KD_TRY(check_widths(T, d, V, dt, 1.0f));
  *bytes = T == 0 ? 0 : plan_logp(T, d, V, elem_of(dt), 4, 0).fwd_total;
  return KD_OK;
}

kd_status kd_token_logp_workspace_size(int64_t T, int64_t d, int64_t V, kd_dtype dt, kd_dtype dw_dtype,
                                       int64_t chunk_rows, size_t* bytes) {
  g_err.clear();
  KD_TRY(need(bytes, "bytes"));
  KD_TRY(check_widths(T, d, V, dt, 1.0f));
  KD_TRY(check_dw_type(dt, dw_dtype));
  if (chunk_rows < 0) return fail(KD_ERR_INVALID_ARG, "chunk_rows must be >= 0");
  *bytes = T == 0 ? 0 : plan_logp(T, d, V, elem_of(dt), elem_of(dw_dtype), chunk_rows).total;
  return KD_OK;
}

kd_status kd_token_logp_fwd(const void* H, const void* W, const int32_t* tokens, const uint8_t* mask, float tau,
                            int64_t T, int64_t d, int64_t V, kd_dtype dt, float* logp, float* lse, float* entropy,
                            float* logits, void* workspace, size_t workspace_bytes, void* stream) {
  g_err.clear();
  KD_TRY(check_widths(T, d, V, dt, tau));
  if (T == 0) return KD_OK;
  KD_TRY(check_head(H, W, tokens));
  KD_TRY(need(logp, "logp"));
  KD_TRY(need(lse, "lse"));
  KD_TRY(need_align(logp, 4, "logp"));
  KD_TRY(need_align(lse, 4, "lse"));
  KD_TRY(need_align(entropy, 4, "entropy"));
  KD_TRY(need_align(logits, 16, "logits"));
  return logp_fwd(H, W, tokens, mask, tau, T, d, V, 0, dt, kd::LogpOut{logp, lse, entropy, nullptr},
                  entropy != nullptr, logits, workspace, workspace_bytes, stream);
}

kd_status kd_token_logp_bwd(const void* H, const void* W, const int32_t* tokens, const uint8_t* mask, float tau,
                            int64_t T, int64_t d, int64_t V, kd_dtype dt, const float* lse, const float* entropy,
                            const float* logits, const float* grad_logp, const float* grad_entropy, void* dH,
                            void* dW, kd_dtype dw_dtype, int64_t chunk_rows, void* workspace, size_t workspace_bytes,
                            void* stream) {
  return logp_bwd(H, W, tokens, mask, tau, T, d, V, 0, dt, lse, entropy, logits, grad_logp, grad_entropy, dH,
                  elem_of(dt), dW, dw_dtype, chunk_rows, workspace, workspace_bytes, stream);
}

kd_status kd_token_logp_fwd_shard(const void* H, const void* W, const int32_t* tokens, const uint8_t* mask, float tau,
                                  int64_t T, int64_t d, int64_t V, int64_t v0, kd_dtype dt, float* rec, float* logits,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  g_err.clear();
  KD_TRY(check_widths(T, d, V, dt, tau));
  KD_TRY(check_v0(V, v0));
  if (T == 0) return KD_OK;
  KD_TRY(check_head(H, W, tokens));
  KD_TRY(need(rec, "rec"));
  KD_TRY(need_align(rec, 16, "rec"));
  KD_TRY(need_align(logits, 16, "logits"));
  return logp_fwd(H, W, tokens, mask, tau, T, d, V, v0, dt,
                  kd::LogpOut{nullptr, nullptr, nullptr, reinterpret_cast<float4*>(rec)}, true, logits, workspace,
                  workspace_bytes, stream);
}

kd_status kd_token_logp_shard_combine(const float* rec, int64_t R, const uint8_t* mask, float tau, int64_t T,
                                      float* logp, float* lse, float* entropy, void* stream) {
  g_err.clear();
  if (T < 0) return fail(KD_ERR_INVALID_ARG, "T must be >= 0");
  if (R < 1) return fail(KD_ERR_INVALID_ARG, "R must be >= 1");
  if (!(tau > 0.f) || !std::isfinite(tau)) return fail(KD_ERR_INVALID_ARG, "tau must be finite and > 0");
  if (T > INT32_MAX / 2 || R > INT32_MAX / std::max<int64_t>(T, 1))
    return fail(KD_ERR_UNSUPPORTED, "R * T must be below 2^31");
  if (T == 0) return KD_OK;
  KD_TRY(need(rec, "rec"));
  KD_TRY(need(logp, "logp"));
  KD_TRY(need(lse, "lse"));
  KD_TRY(need_align(rec, 16, "rec"));
  KD_TRY(need_align(logp, 4, "logp"));
  KD_TRY(need_align(lse, 4, "lse"));
  KD_TRY(need_align(entropy, 4, "entropy"));
  hipStream_t st = static_cast<hipStream_t>(stream);
  KD_LAUNCH("logp_shard_combine", st,
            kd::launch_logp_shard_combine(reinterpret_cast<const float4*>(rec), (int)R, T, mask,
                                          (float)(1.4426950408889634 / (double)tau),
                                          kd::LogpOut{logp, lse, entropy, nullptr}, st));
  return KD_OK;
}

kd_status kd_token_logp_bwd_shard(const void* H, const void* W, const int32_t* tokens, const uint8_t* mask, float tau,
                                  int64_t T, int64_t d, int64_t V, int64_t v0, kd_dtype dt, const float* lse,
                                  const float* entropy, const float* logits, const float* grad_logp,
                                  const float* grad_entropy, float* dH, void* dW, kd_dtype dw_dtype,
                                  int64_t chunk_rows, void* workspace, size_t workspace_bytes, void* stream) {
  return logp_bwd(H, W, tokens, mask, tau, T, d, V, v0, dt, lse, entropy, logits, grad_logp, grad_entropy, dH, 4, dW,
                  dw_dtype, chunk_rows, workspace, workspace_bytes, stream);
}

}  // extern "C"

// ---------------------------------------------------------------- clipped policy loss
namespace {

struct PolicyPlan {
  size_t o_counts, o_part, total;
};
PolicyPlan plan_policy(int64_t T, int64_t S) {
  PolicyPlan p{};
  Carver cv;
  p.o_counts = cv.take((size_t)kd::policy_counts(T, S) * 4);
  p.o_part = cv.take((size_t)kd::policy_blocks(T) * 5 * 8);
  p.total = cv.off;
  return p;
}

kd_status check_tokens(int64_t T, int64_t S) {
  if (T < 0) return fail(KD_ERR_INVALID_ARG, "T must be >= 0");
  if (S < 0) return fail(KD_ERR_INVALID_ARG, "the number of sequences must be >= 0");
  if (T > INT32_MAX / 2 || S > INT32_MAX / 2)
    return fail(KD_ERR_UNSUPPORTED, "tokens and sequences must be below 2^30");
  return KD_OK;
}

kd_status policy_args(const float* logp, const float* old_logp, const float* adv, const uint8_t* mask,
                      const kd_policy_opts* o, int64_t T, kd::PolicyArgs& a) {
  g_err.clear();
  KD_TRY(need(o, "opts"));
  KD_TRY(check_tokens(T, o->S));
  if (o->cu_seqlens != nullptr && o->S < 1) return fail(KD_ERR_INVALID_ARG, "S must be >= 1 with cu_seqlens");
  if (o->cu_seqlens == nullptr && (o->per_sequence || o->reduction == KD_SEQUENCE_MEAN))
    return fail(KD_ERR_INVALID_ARG, "one advantage per sequence and KD_SEQUENCE_MEAN need cu_seqlens");
  if (o->reduction != KD_SUM && o->reduction != KD_TOKEN_MEAN && o->reduction != KD_SEQUENCE_MEAN)
    return fail(KD_ERR_INVALID_ARG, "reduction must be KD_SUM, KD_TOKEN_MEAN or KD_SEQUENCE_MEAN");
  if (o->kl_kind != KD_KL_1 && o->kl_kind != KD_KL_2 && o->kl_kind != KD_KL_3)
    return fail(KD_ERR_INVALID_ARG, "kl_kind must be KD_KL_1, KD_KL_2 or KD_KL_3");
  if (!(o->clip_low >= 0) || !(o->clip_low <= 1)) return fail(KD_ERR_INVALID_ARG, "clip_low must be in [0, 1]");
  if (!(o->clip_high >= 0)) return fail(KD_ERR_INVALID_ARG, "clip_high must be >= 0");
  if (o->dual_clip != 0 && (!(o->dual_clip > 1) || !std::isfinite(o->dual_clip)))
    return fail(KD_ERR_INVALID_ARG, "dual_clip must be 0 or finite and > 1");
  if (!std::isfinite(o->kl_weight) || !std::isfinite(o->entropy_weight))
    return fail(KD_ERR_INVALID_ARG, "kl_weight and entropy_weight must be finite");
  if (T > 0) {
    if (o->kl_weight != 0) KD_TRY(need(o->ref_logp, "ref_logp (kl_weight needs it)"));
    if (o->entropy_weight != 0) KD_TRY(need(o->entropy, "entropy (entropy_weight needs it)"));
    KD_TRY(need(logp, "logp"));
    KD_TRY(need(old_logp, "old_logp"));
    KD_TRY(need(adv, "advantages"));
  }
  KD_TRY(need_align(logp, 4, "logp"));
  KD_TRY(need_align(old_logp, 4, "old_logp"));
  KD_TRY(need_align(adv, 4, "advantages"));
  KD_TRY(need_align(o->ref_logp, 4, "ref_logp"));
  KD_TRY(need_align(o->entropy, 4, "entropy"));
  KD_TRY(need_align(o->cu_seqlens, 4, "cu_seqlens"));
  a = kd::PolicyArgs{};
  a.logp = logp;
  a.old = old_logp;
  a.adv = adv;
  a.mask = mask;
  a.ref = o->ref_logp;
  a.ent = o->entropy;
  a.cu = o->cu_seqlens;
  a.T = (int32_t)T;
  a.S = o->cu_seqlens ? (int32_t)o->S : 0;
  a.per_sequence = o->per_sequence != 0;
  a.reduction = (int)o->reduction;
  a.kl_kind = (int)o->kl_kind;
  a.lo = 1.0 - o->clip_low;
  a.hi = 1.0 + o->clip_high;
  a.dual = o->dual_clip;
  a.klw = o->kl_weight;
  a.entw = o->entropy_weight;
  return KD_OK;
}

kd_status policy_fwd(kd::PolicyArgs& a, float* total, float* stats, double* weights, float* grad_logp, float* grad_entropy,
                     void* workspace, size_t workspace_bytes, void* stream) {
  KD_TRY(need(stats, "stats"));
  KD_TRY(need(weights, "weights"));
  KD_TRY(need_align(stats, 4, "stats"));
  KD_TRY(need_align(total, 4, "total"));
  KD_TRY(need_align(weights, 8, "weights"));
  const PolicyPlan p = plan_policy(a.T, a.S);
  KD_TRY(check_workspace(workspace, workspace_bytes, p.total));
  a.stats = stats;
  a.total = total;
  a.weights = weights;
  a.grad_logp = grad_logp;
  a.grad_ent = grad_entropy;
  a.counts = at<int32_t>(workspace, p.o_counts);
  a.part = at<double>(workspace, p.o_part);
  hipStream_t st = static_cast<hipStream_t>(stream);
  KD_LAUNCH("policy_loss", st, kd::launch_policy(a, true, st));
  return KD_OK;
}

}  // namespace

extern "C" {

kd_status kd_policy_loss_workspace_size(int64_t T, int64_t S, size_t* bytes) {
  g_err.clear();
  KD_TRY(need(bytes, "bytes"));
  KD_TRY(check_tokens(T, S));
  *bytes = plan_policy(T, S).total;
  return KD_OK;
}

kd_status kd_policy_loss_fwd(const float* logp, const float* old_logp, const float* advantages, const uint8_t* mask,
                             const kd_policy_opts* opts, int64_t T, float* total, float* stats, double* weights,
                             void* workspace, size_t workspace_bytes, void* stream) {
  kd::PolicyArgs a;
  KD_TRY(policy_args(logp, old_logp, advantages, mask, opts, T, a));
  return policy_fwd(a, total, stats, weights, nullptr, nullptr, workspace, workspace_bytes, stream);
}

kd_status kd_policy_loss_bwd(const float* logp, const float* old_logp, const float* advantages, const uint8_t* mask,
                             const kd_policy_opts* opts, int64_t T, const double* weights, const float* grad_total,
                             float* grad_logp, float* grad_entropy, void* stream) {
  kd::PolicyArgs a;
  KD_TRY(policy_args(logp, old_logp, advantages, mask, opts, T, a));
  if (T == 0) return KD_OK;
  KD_TRY(need(weights, "weights"));
  KD_TRY(need(grad_total, "grad_total"));
  KD_TRY(need(grad_logp, "grad_logp"));
  KD_TRY(need_align(weights, 8, "weights"));
  KD_TRY(need_align(grad_total, 4, "grad_total"));
  KD_TRY(need_align(grad_logp, 4, "grad_logp"));
  KD_TRY(need_align(grad_entropy, 4, "grad_entropy"));
  a.weights = const_cast<double*>(weights);  // read only: the weights are not made here
  a.grad_total = grad_total;
  a.grad_logp = grad_logp;
  a.grad_ent = grad_entropy;
  hipStream_t st = static_cast<hipStream_t>(stream);
  KD_LAUNCH("policy_grad", st, kd::launch_policy(a, false, st));
  return KD_OK;
}

kd_status kd_policy_loss_fwd_bwd(const float* logp, const float* old_logp, const float* advantages,
                                 const uint8_t* mask, const kd_policy_opts* opts, int64_t T, float* stats,
                                 double* weights, float* grad_logp, float* grad_entropy, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  kd::PolicyArgs a;
  KD_TRY(policy_args(logp, old_logp, advantages, mask, opts, T, a));
  if (T > 0) KD_TRY(need(grad_logp, "grad_logp"));
  KD_TRY(need_align(grad_logp, 4, "grad_logp"));
  KD_TRY(need_align(grad_entropy, 4, "grad_entropy"));
  return policy_fwd(a, nullptr, stats, weights, grad_logp, grad_entropy, workspace, workspace_bytes, stream);
}

}  // extern "C"

// ---------------------------------------------------------------- preference loss
namespace {

kd_status pref_args(const int32_t* cu, const uint8_t* mask, const kd_pref_opts* o, int64_t T, int64_t P,
                    kd::PrefArgs& a) {
  g_err.clear();
  KD_TRY(need(o, "opts"));
  KD_TRY(check_tokens(T, P));
  if (P < 1) return fail(KD_ERR_INVALID_ARG, "P must be >= 1");
  if (P > INT32_MAX / 4) return fail(KD_ERR_UNSUPPORTED, "P must be below 2^29");
  if (o->kind != KD_PREF_SIGMOID && o->kind != KD_PREF_HINGE && o->kind != KD_PREF_IPO)
    return fail(KD_ERR_INVALID_ARG, "kind must be KD_PREF_SIGMOID, KD_PREF_HINGE or KD_PREF_IPO");
  if (!(o->beta > 0) || !std::isfinite(o->beta)) return fail(KD_ERR_INVALID_ARG, "beta must be finite and > 0");
  if (!(o->label_smoothing >= 0) || !(o->label_smoothing < 0.5))
    return fail(KD_ERR_INVALID_ARG, "label_smoothing must be in [0, 1/2)");
  if (o->label_smoothing != 0 && o->kind != KD_PREF_SIGMOID)
    return fail(KD_ERR_UNSUPPORTED, "label_smoothing is for KD_PREF_SIGMOID");
  if (!std::isfinite(o->margin)) return fail(KD_ERR_INVALID_ARG, "margin must be finite");
  if (o->margin != 0 && o->kind == KD_PREF_IPO) return fail(KD_ERR_UNSUPPORTED, "KD_PREF_IPO takes no margin");
  KD_TRY(need(cu, "cu_seqlens"));
  KD_TRY(need_align(cu, 4, "cu_seqlens"));
  KD_TRY(need_align(o->ref_logp, 4, "ref_logp"));
  a = kd::PrefArgs{};
  a.ref = o->ref_logp;
  a.cu = cu;
  a.mask = mask;
  a.T = (int32_t)T;
  a.P = (int32_t)P;
  a.kind = (int)o->kind;
  a.average = o->average != 0;
  a.beta = o->beta;
  a.eps = o->label_smoothing;
  a.margin = o->margin;
  return KD_OK;
}

kd_status pref_fwd_args(const float* logp, float* loss, float* rewards, double* sums, void* workspace,
                        size_t workspace_bytes, kd::PrefArgs& a) {
  if (a.T > 0) KD_TRY(need(logp, "logp"));
  KD_TRY(need(loss, "loss"));
  KD_TRY(need(rewards, "rewards"));
  KD_TRY(need(sums, "sums"));
  KD_TRY(need_align(logp, 4, "logp"));
  KD_TRY(need_align(loss, 4, "loss"));
  KD_TRY(need_align(rewards, 4, "rewards"));
  KD_TRY(need_align(sums, 8, "sums"));
  const size_t want = up((size_t)kd::pref_chunks(a.T) * 32, kAlign);
  KD_TRY(check_workspace(workspace, workspace_bytes, want));
  a.logp = logp;
  a.loss = loss;
  a.rewards = rewards;
  a.sums = sums;
  a.part = at<double>(workspace, 0);
  return KD_OK;
}

kd_status pref_bwd_args(const double* sums, const float* grad_loss, float* grad_logp, kd::PrefArgs& a) {
  KD_TRY(need(sums, "sums"));
  KD_TRY(need(grad_loss, "grad_loss"));
  if (a.T > 0) KD_TRY(need(grad_logp, "grad_logp"));
  KD_TRY(need_align(sums, 8, "sums"));
  KD_TRY(need_align(grad_loss, 4, "grad_loss"));
  KD_TRY(need_align(grad_logp, 4, "grad_logp"));
  a.sums = const_cast<double*>(sums);
  a.grad_loss = grad_loss;
  a.grad_logp = grad_logp;
  return KD_OK;
}

}  // namespace

extern "C" {

kd_status kd_preference_loss_workspace_size(int64_t T, int64_t P, size_t* bytes) {
  g_err.clear();
  KD_TRY(need(bytes, "bytes"));
  KD_TRY(check_tokens(T, P));
  if (P < 1) return fail(KD_ERR_INVALID_ARG, "P must be >= 1");
  *bytes = up((size_t)kd::pref_chunks(T) * 32, kAlign);
  return KD_OK;
}

kd_status kd_preference_loss_fwd(const float* logp, const int32_t* cu_seqlens, const uint8_t* mask,
                                 const kd_pref_opts* opts, int64_t T, int64_t P, float* loss, float* rewards,
                                 double* sums, void* workspace, size_t workspace_bytes, void* stream) {
  kd::PrefArgs a;
  KD_TRY(pref_args(cu_seqlens, mask, opts, T, P, a));
  KD_TRY(pref_fwd_args(logp, loss, rewards, sums, workspace, workspace_bytes, a));
  hipStream_t st = static_cast<hipStream_t>(stream);
  KD_LAUNCH("preference_loss", st, kd::launch_pref(a, st));
  return KD_OK;
}

kd_status kd_preference_loss_bwd(const int32_t* cu_seqlens, const uint8_t* mask, const kd_pref_opts* opts, int64_t T,
                                 int64_t P, const double* sums, const float* grad_loss, float* grad_logp,
                                 void* stream) {
  kd::PrefArgs a;
  KD_TRY(pref_args(cu_seqlens, mask, opts, T, P, a));
  KD_TRY(pref_bwd_args(sums, grad_loss, grad_logp, a));
  hipStream_t st = static_cast<hipStream_t>(stream);
  KD_LAUNCH("preference_grad", st, kd::launch_pref_grad(a, st));
  return KD_OK;
}

kd_status kd_preference_loss_fwd_bwd(const float* logp, const int32_t* cu_seqlens, const uint8_t* mask,
                                     const kd_pref_opts* opts, int64_t T, int64_t P, const float* grad_loss,
                                     float* loss, float* rewards, double* sums, float* grad_logp, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  kd::PrefArgs a;
  KD_TRY(pref_args(cu_seqlens, mask, opts, T, P, a));
  KD_TRY(pref_fwd_args(logp, loss, rewards, sums, workspace, workspace_bytes, a));
  KD_TRY(pref_bwd_args(sums, grad_loss, grad_logp, a));
  hipStream_t st = static_cast<hipStream_t>(stream);
  KD_LAUNCH("preference_loss", st, kd::launch_pref(a, st));
  return KD_OK;
}

}  // extern "C"

// ---------------------------------------------------------------- gradient norm and clipping
namespace {

int64_t clip_blocks(int64_t numel) { return cdiv(numel, kd::kClipBlock); }

kd_status check_counts(const int64_t* numel, int64_t n, int64_t* blocks) {
  if (n < 0) return fail(KD_ERR_INVALID_ARG, "n must be >= 0");
  if (n > 0) KD_TRY(need(numel, "numel"));
  int64_t b = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (numel[i] < 0) return fail(KD_ERR_INVALID_ARG, "numel must be >= 0");
    if (numel[i] <= (int64_t(1) << 44)) b += clip_blocks(numel[i]);
    if (b > INT32_MAX / 2 || numel[i] > (int64_t(1) << 44))
      return fail(KD_ERR_UNSUPPORTED, "too many elements in all");
  }
  *blocks = b;
  return KD_OK;
}

int type_bytes(int32_t t) { return t == KD_F32 ? 4 : t == KD_BF16 || t == KD_F16 ? 2 : 0; }

kd_status check_tensors(const void* const* p, const int64_t* numel, const int32_t* types, int64_t n,
                        const char* name) {
  if (n == 0) return KD_OK;
  KD_TRY(need(p, name));
  KD_TRY(need(types, "types"));
  for (int64_t i = 0; i < n; ++i) {
    const int b = type_bytes(types[i]);
    if (b == 0) return fail(KD_ERR_INVALID_ARG, "a tensor's type must be KD_F32, KD_BF16 or KD_F16");
    if (numel[i] == 0) continue;
    KD_TRY(need(p[i], name));
    KD_TRY(need_align(p[i], b, name));
  }
  return KD_OK;
}

// Outputs may be their own inputs and overlap nothing else.
kd_status check_overlap(const void* const* in, const int32_t* ty, void* const* out, const int32_t* oty,
                        const int64_t* numel, int64_t n) {
  struct Range {
    uintptr_t b, e;
    int64_t i;
    bool out;
  };
  std::vector<Range> r;
  try {
    r.reserve(2 * n);
  } catch (const std::exception&) {  // no exception leaves a C entry
    return fail(KD_ERR_UNSUPPORTED, "too many tensors");
  }
  for (int64_t i = 0; i < n; ++i) {
    if (numel[i] == 0) continue;
    const uintptr_t x = reinterpret_cast<uintptr_t>(in[i]), y = reinterpret_cast<uintptr_t>(out[i]);
    if (x == y && ty[i] != oty[i]) return fail(KD_ERR_INVALID_ARG, "in place needs the same type");
    if (x != y) r.push_back({x, x + (uintptr_t)numel[i] * type_bytes(ty[i]), i, false});
    r.push_back({y, y + (uintptr_t)numel[i] * type_bytes(oty[i]), i, true});
  }
  std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.b < b.b; });
  uintptr_t end_any = 0, end_out = 0;
  for (const Range& x : r) {
    if ((x.out && x.b < end_any) || x.b < end_out)
      return fail(KD_ERR_INVALID_ARG, "an output overlaps another tensor");
    end_any = std::max(end_any, x.e);
    if (x.out) end_out = std::max(end_out, x.e);
  }
  return KD_OK;
}

// The non-empty tensors in tables of at most Table::kTensors: set(table, slot,
// i) fills a slot, f(table, first block of the table) launches it.
template <class Table, class Set, class F>
kd_status over_tables(const int64_t* numel, int64_t n, Set&& set, F&& f) {
  Table t;
  int64_t base = 0;
  t.n = 0;
  t.first[0] = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (numel[i] > 0) {
      set(t, t.n, i);
      t.numel[t.n] = numel[i];
      t.first[t.n + 1] = t.first[t.n] + (int32_t)clip_blocks(numel[i]);
      ++t.n;
    }
    if (t.n > 0 && (t.n == Table::kTensors || i + 1 == n)) {
      KD_TRY(f(t, base));
      base += t.first[t.n];
      t.n = 0;
    }
  }
  return KD_OK;
}

kd_status sumsq_launches(const void* const* grads, const int64_t* numel, const int32_t* dtypes, int64_t n,
                         int64_t blocks, double* sumsq, double* part, hipStream_t st) {
  KD_TRY(over_tables<kd::SumsqTable>(
      numel, n,
      [&](kd::SumsqTable& t, int k, int64_t i) {
        t.in[k] = grads[i];
        t.type[k] = (uint8_t)dtypes[i];
      },
      [&](const kd::SumsqTable& t, int64_t base) {
        KD_LAUNCH("grad_sumsq", st, kd::launch_sumsq(t, part + base, st));
        return KD_OK;
      }));
  KD_LAUNCH("grad_sumsq_total", st, kd::launch_sumsq_total(part, blocks, sumsq, st));
  return KD_OK;
}

kd_status check_clip(const void* const* grads, const int64_t* numel, const int32_t* dtypes, int64_t n,
                     void* const* outs, const int32_t* out_dtypes, const double* sumsq, double max_norm,
                     const float* norm, int64_t* blocks) {
  KD_TRY(check_counts(numel, n, blocks));
  KD_TRY(check_tensors(grads, numel, dtypes, n, "grads"));
  KD_TRY(check_tensors(outs, numel, out_dtypes, n, "outs"));
  if (n > 0) KD_TRY(check_overlap(grads, dtypes, outs, out_dtypes, numel, n));
  if (!(max_norm >= 0)) return fail(KD_ERR_INVALID_ARG, "max_norm must be >= 0");
  KD_TRY(need(sumsq, "sumsq"));
  KD_TRY(need(norm, "norm"));
  KD_TRY(need_align(sumsq, 8, "sumsq"));
  KD_TRY(need_align(norm, 4, "norm"));
  return KD_OK;
}

void set_clip(kd::ClipTable& t, int k, const void* const* grads, const int32_t* dtypes, void* const* outs,
              const int32_t* out_dtypes, int64_t i) {
  t.in[k] = grads[i];
  t.out[k] = outs[i];
  t.in_type[k] = (uint8_t)dtypes[i];
  t.out_type[k] = (uint8_t)out_dtypes[i];
}

kd_status clip_launches(const void* const* grads, const int64_t* numel, const int32_t* dtypes, int64_t n,
                        int64_t blocks, void* const* outs, const int32_t* out_dtypes, const double* sumsq,
                        double max_norm, float* norm, hipStream_t st) {
  if (blocks == 0) KD_LAUNCH("grad_norm", st, kd::launch_norm(sumsq, norm, st));
  return over_tables<kd::ClipTable>(
      numel, n, [&](kd::ClipTable& t, int k, int64_t i) { set_clip(t, k, grads, dtypes, outs, out_dtypes, i); },
      [&](const kd::ClipTable& t, int64_t base) {  // the first launch writes the norm
        KD_LAUNCH("grad_clip", st, kd::launch_clip(t, sumsq, max_norm, base == 0 ? norm : nullptr, st));
        return KD_OK;
      });
}

}  // namespace

extern "C" {

kd_status kd_grad_norm_workspace_size(const int64_t* numel, int64_t n, size_t* bytes) {
  g_err.clear();
  KD_TRY(need(bytes, "bytes"));
  int64_t blocks = 0;
  KD_TRY(check_counts(numel, n, &blocks));
  *bytes = up((size_t)blocks * 8, kAlign);
  return KD_OK;
}

kd_status kd_grad_sumsq(const void* const* grads, const int64_t* numel, const int32_t* dtypes, int64_t n,
                        double* sumsq, void* workspace, size_t workspace_bytes, void* stream) {
  g_err.clear();
  int64_t blocks = 0;
  KD_TRY(check_counts(numel, n, &blocks));
  KD_TRY(check_tensors(grads, numel, dtypes, n, "grads"));
  KD_TRY(need(sumsq, "sumsq"));
  KD_TRY(need_align(sumsq, 8, "sumsq"));
  KD_TRY(check_workspace(workspace, workspace_bytes, up((size_t)blocks * 8, kAlign)));
  return sumsq_launches(grads, numel, dtypes, n, blocks, sumsq, at<double>(workspace, 0),
                        static_cast<hipStream_t>(stream));
}

kd_status kd_grad_clip(const void* const* grads, const int64_t* numel, const int32_t* dtypes, int64_t n,
                       void* const* outs, const int32_t* out_dtypes, const double* sumsq, double max_norm,
                       float* norm, void* stream) {
  g_err.clear();
  int64_t blocks = 0;
  KD_TRY(check_clip(grads, numel, dtypes, n, outs, out_dtypes, sumsq, max_norm, norm, &blocks));
  return clip_launches(grads, numel, dtypes, n, blocks, outs, out_dtypes, sumsq, max_norm, norm,
                       static_cast<hipStream_t>(stream));
}

kd_status kd_grad_clip_norm(const void* const* grads, const int64_t* numel, const int32_t* dtypes, int64_t n,
                            void* const* outs, const int32_t* out_dtypes, double max_norm, double* sumsq,
                            float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  g_err.clear();
  int64_t blocks = 0;
  KD_TRY(check_clip(grads, numel, dtypes, n, outs, out_dtypes, sumsq, max_norm, norm, &blocks));
  KD_TRY(check_workspace(workspace, workspace_bytes, up((size_t)blocks * 8, kAlign)));
  hipStream_t st = static_cast<hipStream_t>(stream);
  int64_t total = 0, some = 0;
  for (int64_t i = 0; i < n; ++i) {
    total += numel[i];  // below 2^46: check_counts bounds the blocks
    some += numel[i] > 0;
  }
  if (blocks > 0 && some <= kd::kClipSmallTensors && total <= kd::kClipSmall)
    return over_tables<kd::ClipTable>(
        numel, n, [&](kd::ClipTable& t, int k, int64_t i) { set_clip(t, k, grads, dtypes, outs, out_dtypes, i); },
        [&](const kd::ClipTable& t, int64_t) {
          KD_LAUNCH("grad_clip_small", st, kd::launch_clip_small(t, sumsq, max_norm, norm, st));
          return KD_OK;
        });
  KD_TRY(sumsq_launches(grads, numel, dtypes, n, blocks, sumsq, at<double>(workspace, 0), st));
  return clip_launches(grads, numel, dtypes, n, blocks, outs, out_dtypes, sumsq, max_norm, norm, st);
}

}  // extern "C"
