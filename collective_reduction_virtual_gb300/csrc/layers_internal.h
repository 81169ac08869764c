// Parameters and kernel selectors of the layer operators (embedding, layer
// norm, 8-bit activations), shared by their host entry points (layers.cpp)
// and kernels.  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include "vcoll_internal.h"

namespace vcoll {

constexpr int kRowThreads = 256;  // threads of a CTA that works on rows

// Accesses per lane in flight in the lookup: 4 of 16 bytes, 8 of fewer.
VCOLL_HD constexpr int lookup_accesses(int A, int E) { return A == E ? 4 : 8; }
struct EmbedParams {
  const void* tokens;
  const void* table;
  void* out;
  int64_t N, V, D;
  int64_t table_ld, out_ld;
  float scale;
  int idx64;
  int64_t pieces;  // of a row, a warp each
};

// The gradient's tokens are sorted by (token, position) with a stable LSD
// radix sort; tokens outside [0, V) sort as V, behind all others.
constexpr int kSortThreads = 1024;
constexpr int kSortMaxBits = 9;  // digit width
// Keys of a CTA where several sort: short lists are cut finer (8192 keys of
// 128000 tokens: 26.5 us a call with tiles of 1024, 27.1 of 2048, 33.0 of 4096;
// 105491 keys: 43.8, 42.7 and 48.8), long ones into no more than 128 tiles,
// since every CTA reads the counts of all (10^6 keys: 158 us with 128, 166 with
// 64 and 224 with 32 tiles).
constexpr int64_t kSortFineTile = 1024, kSortFineMost = 32768;
constexpr int64_t kSortMinTile = 2048;
constexpr int kSortMaxTiles = 128;
constexpr int kPrefetchLines = 4;  // that a lane fetches to L2
constexpr int64_t kFillRows = 2;  // adjacent rows that a warp fills
// Lists that are not sorted: up to kSmallTokens tokens and, since a warp for each
// place and 256 columns reads the list, kSmallWork of tokens squared times these
// tiles.  In place, spread as in text, without and with the sort: 512 tokens of
// 4096 columns 15 and 19 us, 1024 of 1024 14 and 20, 2048 of 256 17 and 23; past
// it 768 of 4096 25 and 20, 2048 of 1024 28 and 22.  One token alone, the worst
// for it: 2048 of 256 28 and 16.
constexpr int kSmallTokens = 2048;
constexpr int64_t kSmallWork = (int64_t)1 << 22;
constexpr int kSmallAlone = 32;    // places of a token that one warp sums alone
constexpr int64_t kJoinAlone = 16;  // partial rows that one warp adds up alone
struct EmbedGradParams {
  const void* tokens;
  const void* grad;
  const void* base;  // NULL: zeros
  void* out;
  uint32_t* key[2];  // ping-pong of the sort: N keys and N positions each
  uint32_t* pos[2];
  uint32_t* cnt;     // digit counts: passes x tiles x 2^bits
  float* part;       // partial rows: chunks x 2 x tiles x (32 * E)
  uint32_t* stamp;   // V positions (vc_embed_count)
  int64_t N, V, D;
  int64_t grad_ld, base_ld, out_ld;
  int64_t sort_tile;  // keys of a tile of the sort
  int64_t chunk;      // places of the sorted list that a warp sums
  int64_t tiles;      // column tiles
  int64_t sum_ctas;   // CTAs that sum
  int64_t fill_begin, fill_end;  // rows that a launch fills where their tokens are absent
  int64_t fill_piece, fill_pieces;  // bytes of a row that a warp fills, and their number
  int fill_each;      // rows of absent tokens that a CTA of the short lists looks after
  int fill_bytes;     // of an access of these: 16, 4 or 2
  int table_es;       // bytes of an element of the table
  int sort_tiles, fill_ctas;  // CTAs of a pass that sort, and that fill
  int64_t row_lines;             // lines of 128 bytes of a row of the gradient
  int64_t line_begin, line_end;  // those that a launch fetches to L2
  int grad_es;
  float scale;
  int idx64;
  int passes, bits, pass;
};

struct NormParams {
  const void* x;       // N x D, or NULL: h comes from codes and scales
  const void* grad;    // backward only
  const void* weight;  // NULL: ones
  const void* bias;    // NULL: zeros
  void* y;             // forward: y; backward: dx (may be NULL)
  float* mean;
  float* rstd;
  int8_t* codes;  // forward: kept 8-bit h (or NULL); backward: where h comes from
  float* scales;
  void* dweight;
  void* dbias;
  float* part;  // backward workspace
  int64_t N, D;
  int64_t x_ld, grad_ld, y_ld, codes_ld;
  float eps;
  int wbf16;  // weight, bias, dweight, dbias are bf16
  int warps;  // that take a row
  int parts;  // partial rows of the gradient (CTAs)
};

// norm_narrow.cuh: rows of a group of lanes in flight.
constexpr int kNarrowRows = 4;
// norm_rows.cuh: warps of a CTA of several teams, and of the largest team.
constexpr int kNormCtaWarps = 8;
constexpr int kNormMaxWarps = 16;
// CTAs of the gradient at most: its partial rows' room in the workspace.
constexpr int kNormMaxCtas = 608;
// Chunks of 32 * E columns that a warp takes: 32 values a lane forward, 16
// backward, where the sums over the rows are in registers too; and at most.
VCOLL_HD constexpr int norm_chunks(int E, bool grad) { return (grad ? 16 : 32) / E; }
VCOLL_HD constexpr int norm_max_chunks(int E, bool grad) { return grad && E == 8 ? 4 : 8; }
// Backward, how many of the two sums over the rows are in shared memory: with
// 32 values a lane registers do not hold them (they spilled: 16384 columns of
// bf16 ran at 2.9 TB/s).
VCOLL_HD constexpr int norm_grad_smem_sums(int R, int E) { return R * E <= 16 ? 0 : E == 8 ? 2 : 1; }
// slots of the ring of rows on their way: 128 to 256 bytes a thread
VCOLL_HD constexpr int norm_stages(int R, int E, bool grad) {
  return grad ? (R <= 2 ? 4 : R * E <= 16 ? 2 : 1) : (R <= 2 ? 4 : 2);
}
// bytes of a thread's slots of one stage of the backward ring
VCOLL_HD constexpr int norm_grad_slot_bytes(int R, int E, bool kept) {
  return R * 16 + (kept ? R * E : R * 16);
}

struct PackParams {
  const void* x;
  void* out;
  const void* weight;
  const void* bias;
  int8_t* codes;
  float* scales;
  int64_t N, D;
  int64_t x_ld, codes_ld;  // x_ld: of x or out
  int64_t pieces;  // of a row, a warp each
  int wbf16;
};
constexpr int kPackChunks = 4;  // chunks that a warp has in flight

// access: elements of an access (a whole 16 bytes of dtype, 2 or 1)
const void* embed_kernel(int dtype, int access);
const void* embed_narrow_kernel(int dtype, int access, int lanes);
const void* embed_sort_kernel();
const void* embed_count_kernel();
const void* embed_scatter_kernel();
enum GradPart { GRAD_SMALL, GRAD_SUM, GRAD_SUM_BASE, GRAD_JOIN };
const void* embed_grad_kernel(int dtype, int table_dtype, int access, GradPart part);
const void* norm_rows_kernel_f32(int access, int chunks, int threads, bool grad, bool kept);
const void* norm_rows_kernel_bf16(int access, int chunks, int threads, bool grad, bool kept);
const void* norm_narrow_kernel_f32(int access, int lanes, bool grad, bool kept);
const void* norm_narrow_kernel_bf16(int access, int lanes, bool grad, bool kept);
const void* norm_wsum_kernel();
const void* norm_wide_kernel(int dtype);
const void* norm_grad_wide_kernel(int dtype);
const void* norm_wgrad_wide_kernel(int dtype);
const void* pack8_kernel(int dtype, int access);
const void* unpack8_kernel(int dtype, int access);
const void* pack8_narrow_kernel(int dtype, int access, int lanes, bool unpack);

}  // namespace vcoll
