// C-ABI layer of kdlayers.h: argument checks, workspace carving and the launch
// sequences.  Every argument check runs on the host before any HIP call, so a
// rejected call enqueues nothing.
#include "kdlayers.h"

#include "kd_host.h"
#include "kd_layers.h"

namespace {

using namespace kdh;

int type_bytes(int t) { return t == KD_F32 ? 4 : t == KD_BF16 || t == KD_F16 ? 2 : 0; }

kd_status check_type(int t, const char* name) {
  if (type_bytes(t) == 0) return fail(KD_ERR_INVALID_ARG, std::string(name) + " must be KD_F32, KD_BF16 or KD_F16");
  return KD_OK;
}

kd_status check_rows(int64_t T, int64_t d) {
  if (T < 0) return fail(KD_ERR_INVALID_ARG, "T must be >= 0");
  if (d < 1) return fail(KD_ERR_INVALID_ARG, "d must be >= 1");
  if (T >= (int64_t(1) << 30)) return fail(KD_ERR_UNSUPPORTED, "T must be below 2^30");
  if (d >= (int64_t(1) << 24)) return fail(KD_ERR_UNSUPPORTED, "d must be below 2^24");
  return KD_OK;
}

kd_status check_vocab(int64_t V) {
  if (V < 1) return fail(KD_ERR_INVALID_ARG, "V must be >= 1");
  if (V >= (int64_t(1) << 30)) return fail(KD_ERR_UNSUPPORTED, "V must be below 2^30");
  return KD_OK;
}

// p is there and aligned to its elements
kd_status need_array(const void* p, size_t elem, const char* name) {
  KD_TRY(need(p, name));
  return need_align(p, elem, name);
}

// ------------------------------------------------------------------ 8-bit rows
kd_status check_kind(int kind, int64_t group) {
  if (kind != KD_ROWS_INT8 && kind != KD_ROWS_E4M3)
    return fail(KD_ERR_INVALID_ARG, "kind must be KD_ROWS_INT8 or KD_ROWS_E4M3");
  if (group != 0 && group != 32 && group != 64 && group != 128 && group != 256 && group != 512)
    return fail(KD_ERR_INVALID_ARG, "group must be 0, 32, 64, 128, 256 or 512");
  return KD_OK;
}
struct Groups {
  int size;
  int64_t n;
};
Groups groups_of(int64_t d, int64_t group) {
  if (group == 0) return {(int)d, 1};
  return {(int)group, cdiv(d, group)};
}

kd_status check_quantized(const void* q, const float* scale, int kind, int64_t group) {
  KD_TRY(check_kind(kind, group));
  KD_TRY(need(q, "q"));
  return need_array(scale, 4, "scale");
}

kd::RowsArgs rows_args(const void* x, const void* q, const float* scale, int64_t T, int64_t d, int dt, int kind,
                       int64_t group) {
  const Groups g = groups_of(d, group);
  kd::RowsArgs a{};
  a.x = static_cast<const char*>(x);
  a.q = static_cast<char*>(const_cast<void*>(q));
  a.scale = const_cast<float*>(scale);
  a.T = T;
  a.d = d;
  a.groups = g.n;
  a.group = g.size;
  a.type = dt;
  a.kind = kind;
  return a;
}

// ------------------------------------------------------------------ embeddings
struct EmbedPlan {
  size_t key[2], pos[2], count, part, sums, run_of, total;
  int64_t cols;  // columns of a slab
};
// A tied head's sums take a row a token: slabs of columns keep them to 1 GiB,
// and the launch that turns them below 2^32 threads.
constexpr int64_t kSumsMost = int64_t(1) << 30;
EmbedPlan plan_embed(int64_t T, int64_t V, int64_t d, bool tied) {
  EmbedPlan p{};
  Carver cv;
  p.cols = d;
  if (tied && T > 0) {
    const int64_t wide = std::max<int64_t>(kSumsMost / (4 * T) / 64 * 64, 64);
    p.cols = std::min({d, wide, kd::embed_turn_cols(V)});
  }
  if (T == 0) return p;
  for (int i = 0; i < 2; ++i) {
    p.key[i] = cv.take((size_t)T * 4);
    p.pos[i] = cv.take((size_t)T * 4);
  }
  if (T > kd::kSortSmall) p.count = cv.take((size_t)cdiv(T, kd::kSortItems) * kd::kSortDigits * 4);
  p.part = cv.take((size_t)cdiv(T, kd::embed_piece(T)) * 2 * p.cols * 4);
  p.run_of = cv.take((size_t)V * 4);
  if (tied) p.sums = cv.take((size_t)T * p.cols * 4);
  p.total = cv.off;
  return p;
}

// ------------------------------------------------------------------ layer norm
kd_status check_norm(const void* weight, const float* mean, const float* rstd, int64_t T, int64_t d, int dt, int wdt) {
  KD_TRY(check_rows(T, d));
  KD_TRY(check_type(dt, "dt"));
  KD_TRY(check_type(wdt, "wdt"));
  if (wdt != dt && wdt != KD_F32) return fail(KD_ERR_UNSUPPORTED, "wdt must be dt or KD_F32");
  KD_TRY(need_align(weight, type_bytes(wdt), "weight"));
  KD_TRY(need_align(mean, 4, "mean"));
  return need_align(rstd, 4, "rstd");
}

size_t norm_bytes(int64_t T, int64_t d) { return up((size_t)kd::norm_grad_blocks(T, d) * 2 * d * 4, kAlign); }

// ------------------------------------------------------------------ 8-bit integers
// Rows of one launch of the tiles: their panels stay below 1 GiB.
int64_t int8_rows(int64_t T, int64_t d) {
  const int64_t most = std::max<int64_t>((int64_t(1) << 30) / kd::int8_panel_bytes(256, d) * 256, 256);
  return std::min(T, most);
}

kd_status check_int8(int64_t T, int64_t d, int64_t V) {
  KD_TRY(check_rows(T, d));
  KD_TRY(check_vocab(V));
  if (d % 16) return fail(KD_ERR_UNSUPPORTED, "d must be a multiple of 16");
  if (d >= (int64_t(1) << 17)) return fail(KD_ERR_UNSUPPORTED, "d must be below 2^17");
  return KD_OK;
}

}  // namespace

extern "C" {

kd_status kd_embedding_fwd(const int32_t* tokens, const void* table, const uint8_t* mask, float scale, int64_t T,
                           int64_t V, int64_t d, kd_dtype dt, int32_t tied, void* out, void* stream) {
  g_err.clear();
  KD_TRY(check_rows(T, d));
  KD_TRY(check_vocab(V));
  KD_TRY(check_type(dt, "dt"));
  if (!std::isfinite(scale)) return fail(KD_ERR_INVALID_ARG, "scale must be finite");
  if (T == 0) return KD_OK;
  KD_TRY(need_array(tokens, 4, "tokens"));
  KD_TRY(need_array(table, type_bytes(dt), "table"));
  KD_TRY(need_array(out, type_bytes(dt), "out"));
  kd::EmbedArgs a{};
  a.tokens = tokens;
  a.table = static_cast<const char*>(table);
  a.mask = mask;
  a.scale = scale;
  a.T = T;
  a.V = V;
  a.d = d;
  a.type = dt;
  a.tied = tied != 0;
  a.out = static_cast<char*>(out);
  hipStream_t st = static_cast<hipStream_t>(stream);
  KD_LAUNCH("embedding", st, kd::launch_embed(a, st));
  return KD_OK;
}

kd_status kd_embedding_workspace_size(int64_t T, int64_t V, int64_t d, int32_t tied, size_t* bytes) {
  g_err.clear();
  KD_TRY(need(bytes, "bytes"));
  KD_TRY(check_rows(T, d));
  KD_TRY(check_vocab(V));
  *bytes = plan_embed(T, V, d, tied != 0).total;
  return KD_OK;
}

kd_status kd_embedding_bwd(const void* grad, const int32_t* tokens, const uint8_t* mask, float scale, int64_t T,
                           int64_t V, int64_t d, kd_dtype dt, kd_dtype grad_dt, int32_t tied, int32_t accumulate,
                           void* grad_table, void* workspace, size_t workspace_bytes, void* stream) {
  g_err.clear();
  KD_TRY(check_rows(T, d));
  KD_TRY(check_vocab(V));
  KD_TRY(check_type(dt, "dt"));
  KD_TRY(check_type(grad_dt, "grad_dt"));
  if (!std::isfinite(scale)) return fail(KD_ERR_INVALID_ARG, "scale must be finite");
  KD_TRY(need_array(grad_table, type_bytes(grad_dt), "grad_table"));
  if (T > 0) {
    KD_TRY(need_array(grad, type_bytes(dt), "grad"));
    KD_TRY(need_array(tokens, 4, "tokens"));
  }
  const EmbedPlan p = plan_embed(T, V, d, tied != 0);
  KD_TRY(check_workspace(workspace, workspace_bytes, p.total));
  hipStream_t st = static_cast<hipStream_t>(stream);
  char* out = static_cast<char*>(grad_table);
  if (T == 0) {
    if (!accumulate) KD_LAUNCH("embedding_fill", st, kd::launch_fill_table(out, V * d * type_bytes(grad_dt), st));
    return KD_OK;
  }

  kd::SortArgs s{};
  s.tokens = tokens;
  s.mask = mask;
  s.T = T;
  s.V = V;
  for (int i = 0; i < 2; ++i) {
    s.key[i] = at<uint32_t>(workspace, p.key[i]);
    s.pos[i] = at<uint32_t>(workspace, p.pos[i]);
  }
  s.count = at<uint32_t>(workspace, p.count);
  // a few tokens' gradient looks for the rows to clear among the tokens themselves
  s.run_of = tied || (T > kd::kSortChunk && !accumulate) ? at<int32_t>(workspace, p.run_of) : nullptr;
  if (T <= kd::kSortSmall) {
    KD_LAUNCH("embedding_sort", st, kd::launch_sort_small(s, st));
  } else {
    for (int pass = 0; pass < kd::sort_passes(V); ++pass) {
      KD_LAUNCH("embedding_sort", st, kd::launch_sort_count(s, pass, st));
      KD_LAUNCH("embedding_sort", st, kd::launch_sort_scan(s, pass, st));
      KD_LAUNCH("embedding_sort", st, kd::launch_sort_scatter(s, pass, st));
    }
  }
  const int r = kd::sort_result(T, V);
  kd::EmbedGradArgs a{};
  a.grad = static_cast<const char*>(grad);
  a.key = s.key[r];
  a.pos = s.pos[r];
  a.scale = scale;
  a.T = T;
  a.V = V;
  a.d = d;
  a.type = dt;
  a.grad_type = grad_dt;
  a.tied = tied != 0;
  a.accumulate = accumulate != 0;
  a.out = out;
  a.part = at<float>(workspace, p.part);
  a.piece = kd::embed_piece(T);
  a.sums = at<float>(workspace, p.sums);
  a.run_of = s.run_of;
  for (a.col0 = 0; a.col0 < d; a.col0 += p.cols) {
    a.cols = std::min(p.cols, d - a.col0);
    KD_LAUNCH("embedding_grad", st, kd::launch_embed_grad(a, st));
    KD_LAUNCH("embedding_join", st, kd::launch_embed_join(a, st));
    if (tied) KD_LAUNCH("embedding_turn", st, kd::launch_embed_turn(a, st));
  }
  return KD_OK;
}

kd_status kd_rows_quantize(const void* x, int64_t T, int64_t d, kd_dtype dt, kd_rows_kind kind, int64_t group, void* q,
                           float* scale, void* stream) {
  g_err.clear();
  KD_TRY(check_rows(T, d));
  KD_TRY(check_type(dt, "dt"));
  KD_TRY(check_kind(kind, group));
  if (T == 0) return KD_OK;
  KD_TRY(need_array(x, type_bytes(dt), "x"));
  KD_TRY(check_quantized(q, scale, kind, group));
  hipStream_t st = static_cast<hipStream_t>(stream);
  KD_LAUNCH("rows_quantize", st, kd::launch_rows_quantize(rows_args(x, q, scale, T, d, dt, kind, group), st));
  return KD_OK;
}

kd_status kd_rows_dequantize(const void* q, const float* scale, int64_t T, int64_t d, kd_rows_kind kind, int64_t group,
                             kd_dtype dt, void* out, void* stream) {
  g_err.clear();
  KD_TRY(check_rows(T, d));
  KD_TRY(check_type(dt, "dt"));
  KD_TRY(check_kind(kind, group));
  if (T == 0) return KD_OK;
  KD_TRY(check_quantized(q, scale, kind, group));
  KD_TRY(need_array(out, type_bytes(dt), "out"));
  hipStream_t st = static_cast<hipStream_t>(stream);
  KD_LAUNCH("rows_dequantize", st, kd::launch_rows_dequantize(rows_args(out, q, scale, T, d, dt, kind, group), st));
  return KD_OK;
}

kd_status kd_layer_norm_fwd(const void* x, const void* weight, const void* bias, const uint8_t* mask, double eps,
                            int64_t T, int64_t d, kd_dtype dt, kd_dtype wdt, void* y, float* mean, float* rstd,
                            kd_rows_kind kind, int64_t group, void* q, float* scale, void* stream) {
  g_err.clear();
  KD_TRY(check_norm(weight, mean, rstd, T, d, dt, wdt));
  KD_TRY(need_align(bias, type_bytes(wdt), "bias"));
  if (!(eps >= 0) || !std::isfinite(eps)) return fail(KD_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (kind != KD_ROWS_NONE) KD_TRY(check_kind(kind, group));
  if (T == 0) return KD_OK;
  KD_TRY(need_array(x, type_bytes(dt), "x"));
  KD_TRY(need_array(y, type_bytes(dt), "y"));
  if (kind != KD_ROWS_NONE) KD_TRY(check_quantized(q, scale, kind, group));
  const Groups g = groups_of(d, group);
  kd::NormArgs a{};
  a.x = static_cast<const char*>(x);
  a.w = static_cast<const char*>(weight);
  a.b = static_cast<const char*>(bias);
  a.mask = mask;
  a.eps = (float)eps;
  a.T = T;
  a.d = d;
  a.type = dt;
  a.wtype = wdt;
  a.y = static_cast<char*>(y);
  a.mean = mean;
  a.rstd = rstd;
  a.kind = kind;
  a.group = g.size;
  a.groups = g.n;
  a.q = static_cast<char*>(q);
  a.scale = scale;
  hipStream_t st = static_cast<hipStream_t>(stream);
  KD_LAUNCH("layer_norm", st, kd::launch_norm_fwd(a, st));
  return KD_OK;
}

kd_status kd_layer_norm_workspace_size(int64_t T, int64_t d, size_t* bytes) {
  g_err.clear();
  KD_TRY(need(bytes, "bytes"));
  KD_TRY(check_rows(T, d));
  *bytes = norm_bytes(T, d);
  return KD_OK;
}

kd_status kd_layer_norm_bwd(const void* grad, const void* x, const void* weight, const uint8_t* mask,
                            const float* mean, const float* rstd, int64_t T, int64_t d, kd_dtype dt, kd_dtype wdt,
                            kd_rows_kind kind, int64_t group, const void* q, const float* scale, void* dx,
                            void* dweight, void* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  g_err.clear();
  KD_TRY(check_norm(weight, mean, rstd, T, d, dt, wdt));
  if (kind != KD_ROWS_NONE) KD_TRY(check_kind(kind, group));
  if (!dx && !dweight && !dbias) return fail(KD_ERR_INVALID_ARG, "dx, dweight and dbias are all NULL");
  KD_TRY(need_align(dx, type_bytes(dt), "dx"));
  KD_TRY(need_align(dweight, type_bytes(wdt), "dweight"));
  KD_TRY(need_align(dbias, type_bytes(wdt), "dbias"));
  if (T > 0) {
    KD_TRY(need_array(grad, type_bytes(dt), "grad"));
    KD_TRY(need(mean, "mean"));
    KD_TRY(need(rstd, "rstd"));
    if (kind == KD_ROWS_NONE) {
      KD_TRY(need_array(x, type_bytes(dt), "x"));
    } else {
      if (x) return fail(KD_ERR_INVALID_ARG, "x must be NULL where q and scale stand for it");
      KD_TRY(check_quantized(q, scale, kind, group));
    }
  }
  KD_TRY(check_workspace(workspace, workspace_bytes, norm_bytes(T, d)));
  if (T == 0 && !dweight && !dbias) return KD_OK;
  const Groups g = groups_of(d, group);
  kd::NormGradArgs a{};
  a.grad = static_cast<const char*>(grad);
  a.x = static_cast<const char*>(x);
  a.w = static_cast<const char*>(weight);
  a.mask = mask;
  a.mean = mean;
  a.rstd = rstd;
  a.T = T;
  a.d = d;
  a.type = dt;
  a.wtype = wdt;
  a.kind = kind;
  a.group = g.size;
  a.groups = g.n;
  a.q = static_cast<const char*>(q);
  a.scale = scale;
  a.dx = static_cast<char*>(dx);
  a.dw = static_cast<char*>(dweight);
  a.db = static_cast<char*>(dbias);
  a.part = at<float>(workspace, 0);
  a.blocks = kd::norm_grad_blocks(T, d);
  hipStream_t st = static_cast<hipStream_t>(stream);
  KD_LAUNCH("layer_norm_grad", st, kd::launch_norm_grad(a, st));
  if (dweight || dbias || (dx && weight && mask)) KD_LAUNCH("layer_norm_sum", st, kd::launch_norm_sum(a, st));
  return KD_OK;
}

kd_status kd_int8_matmul_workspace_size(int64_t T, int64_t d, int64_t V, size_t* bytes) {
  g_err.clear();
  KD_TRY(need(bytes, "bytes"));
  KD_TRY(check_int8(T, d, V));
  *bytes = kd::int8_tiles(T, d, V) ? up((size_t)kd::int8_panel_bytes(int8_rows(T, d), d), kAlign) : 0;
  return KD_OK;
}

kd_status kd_int8_matmul(const int8_t* x, const float* x_scale, const int8_t* w, const float* w_scale, int64_t T,
                         int64_t d, int64_t V, kd_dtype out_dt, void* out, void* workspace, size_t workspace_bytes,
                         void* stream) {
  g_err.clear();
  KD_TRY(check_int8(T, d, V));
  KD_TRY(check_type(out_dt, "out_dt"));
  if (T == 0) return KD_OK;
  KD_TRY(need_array(x, 16, "x"));
  KD_TRY(need_array(w, 16, "w"));
  KD_TRY(need_array(x_scale, 4, "x_scale"));
  KD_TRY(need_array(w_scale, 4, "w_scale"));
  KD_TRY(need_array(out, type_bytes(out_dt), "out"));
  const bool tiles = kd::int8_tiles(T, d, V);
  const int64_t C = int8_rows(T, d);
  KD_TRY(check_workspace(workspace, workspace_bytes, tiles ? up((size_t)kd::int8_panel_bytes(C, d), kAlign) : 0));
  hipStream_t st = static_cast<hipStream_t>(stream);
  kd::Int8Args a{};
  a.w = reinterpret_cast<const char*>(w);
  a.sw = w_scale;
  a.d = d;
  a.V = V;
  a.out_type = out_dt;
  a.panels = at<char>(workspace, 0);
  for (int64_t t = 0; t < T; t += tiles ? C : T) {
    a.x = reinterpret_cast<const char*>(x) + t * d;
    a.sx = x_scale + t;
    a.T = tiles ? std::min(C, T - t) : T;
    a.out = static_cast<char*>(out) + t * V * type_bytes(out_dt);
    if (tiles) {
      KD_LAUNCH("int8_panels", st, kd::launch_int8_panels(a, st));
      KD_LAUNCH("int8_tile", st, kd::launch_int8_tiles(a, st));
    } else {
      KD_LAUNCH("int8_few", st, kd::launch_int8_few(a, st));
    }
  }
  return KD_OK;
}

}  // extern "C"
