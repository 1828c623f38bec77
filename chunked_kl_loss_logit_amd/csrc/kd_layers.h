// Arguments and launchers of the kernels behind kdlayers.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kd {

// ---------------------------------------------------------------- token embeddings
struct EmbedArgs {
  const int32_t* tokens;  // [T]
  const char* table;      // [V,d], or [d,V] if tied
  const uint8_t* mask;    // nullable
  float scale;
  int64_t T, V, d;
  int type;
  bool tied;
  char* out;  // [T,d]
};
hipError_t launch_embed(const EmbedArgs& a, hipStream_t st);

// Sorted entries (key, position) of the tokens; entries that count for nothing have key V and come last.
constexpr int64_t kSortSmall = 32768;  // tokens sorted in chunks of one workgroup each (every chunk's keys in LDS at once)
constexpr int kSortChunk = 1024;
constexpr int kSortItems = 8192;       // tokens of a workgroup otherwise
struct SortArgs {
  const int32_t* tokens;
  const uint8_t* mask;
  int64_t T, V;
  uint32_t* key[2];  // [T] each
  uint32_t* pos[2];
  uint32_t* count;   // [kSortDigits x workgroups], T > kSortSmall only
  int32_t* run_of;   // [V] or nullptr: cleared (-1); beyond kSortChunk tokens an entry of each token is noted
};
constexpr int kSortDigits = 512;
// where the result lies: key[i], pos[i] of the returned index
int sort_result(int64_t T, int64_t V);
int sort_passes(int64_t V);
hipError_t launch_sort_count(const SortArgs& a, int pass, hipStream_t st);
hipError_t launch_sort_scan(const SortArgs& a, int pass, hipStream_t st);
hipError_t launch_sort_scatter(const SortArgs& a, int pass, hipStream_t st);
hipError_t launch_sort_small(const SortArgs& a, hipStream_t st);

struct EmbedGradArgs {
  const char* grad;  // [T,d]
  const uint32_t* key;
  const uint32_t* pos;
  float scale;
  int64_t T, V, d;
  int64_t col0, cols;  // the slab of grad's columns that the call takes (all of them unless tied)
  int type, grad_type;
  bool tied, accumulate;
  char* out;    // the table's gradient
  float* part;  // [pieces][2][cols]: what a piece holds of a token that it shares with the piece before, or after
  int piece;    // entries of a piece
  int32_t* run_of;  // [V]: the sort's; with tied weights in the end each token's first entry, or -1
  float* sums;      // tied only, [T][cols]: the sum of the run that begins at an entry
};
int embed_piece(int64_t T);
hipError_t launch_embed_grad(const EmbedGradArgs& a, hipStream_t st);
hipError_t launch_embed_join(const EmbedGradArgs& a, hipStream_t st);
int64_t embed_turn_cols(int64_t V);  // columns that one launch of it takes
hipError_t launch_embed_turn(const EmbedGradArgs& a, hipStream_t st);
hipError_t launch_fill_table(char* p, int64_t bytes, hipStream_t st);  // zeros, any alignment of 2 bytes

// ---------------------------------------------------------------- rows in 8 bits
struct RowsArgs {
  const char* x;  // quantize: in; dequantize: out
  char* q;
  float* scale;
  int64_t T, d, groups;  // groups of a row
  int group;             // values of a group (d where the row is one)
  int type, kind;
};
hipError_t launch_rows_quantize(const RowsArgs& a, hipStream_t st);
hipError_t launch_rows_dequantize(const RowsArgs& a, hipStream_t st);

// ---------------------------------------------------------------- layer norm
struct NormArgs {
  const char* x;
  const char* w;  // nullable
  const char* b;  // nullable
  const uint8_t* mask;
  float eps;
  int64_t T, d;
  int type, wtype;
  char* y;
  float* mean;
  float* rstd;
  // the row in 8 bits, if kind != 0
  int kind, group;
  int64_t groups;
  char* q;
  float* scale;
};
hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st);

struct NormGradArgs {
  const char* grad;
  const char* x;  // or q and scale
  const char* w;
  const uint8_t* mask;
  const float* mean;
  const float* rstd;
  int64_t T, d;
  int type, wtype;
  int kind, group;
  int64_t groups;
  const char* q;
  const float* scale;
  char* dx;      // nullable
  char* dw;      // nullable
  char* db;      // nullable
  float* part;   // [blocks][2][d]
  int blocks;
};
int norm_grad_blocks(int64_t T, int64_t d);
hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t st);
// dw and db from the partials, and masked rows of dx that weights which are not finite have spoilt
hipError_t launch_norm_sum(const NormGradArgs& a, hipStream_t st);

// ---------------------------------------------------------------- product of 8-bit integers
struct Int8Args {
  const char* x;  // [T,d]
  const char* w;  // [V,d]
  const float* sx;
  const float* sw;
  int64_t T, d, V;
  int out_type;
  char* out;
  char* panels;  // workspace: x in panels of whole row blocks, whole ring turns
};
bool int8_tiles(int64_t T, int64_t d, int64_t V);  // whether the tile kernel takes the call
int64_t int8_panel_bytes(int64_t T, int64_t d);
hipError_t launch_int8_panels(const Int8Args& a, hipStream_t st);
hipError_t launch_int8_tiles(const Int8Args& a, hipStream_t st);
hipError_t launch_int8_few(const Int8Args& a, hipStream_t st);

}  // namespace kd
