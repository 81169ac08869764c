// Host side of the layer operators declared in include/vcoll.h: argument
// checks, choice of kernel and launches.
#include <cuda_runtime.h>

#include <algorithm>

#include "layer_checks.h"

using namespace vcoll;

namespace {

// CTAs for `items` pieces of work of which a CTA does `per` at a time: all of
// them at once, at most `waves` CTAs per SM, each looping over its share.
int grid_for(int64_t items, int64_t per, int waves, int64_t* grid) {
  int sms = 0;
  VCOLL_TRY(device_sms(&sms));
  *grid = std::max<int64_t>(1, std::min<int64_t>(ceil_div(items, per), (int64_t)sms * waves));
  return VCOLL_OK;
}

constexpr int kWarps = kRowThreads / 32;

// Lanes that take a row of D columns where the row is narrow, else 0.
int narrow_lanes(int64_t D, int E) { return D <= 8 * E ? 8 : D <= 16 * E ? 16 : D <= 32 * E ? 32 : 0; }

// kNarrowRows rows for each group of `lanes` lanes.
int launch_narrow(const void* fn, int64_t N, int lanes, void* params, void* stream) {
  return launch_grid(fn, ceil_div(N, (int64_t)kWarps * kNarrowRows * (32 / lanes)), 1, kRowThreads, 0,
                     params, stream);
}

// A warp for each piece of each of N rows.
int launch_pieces(const void* fn, int64_t N, int64_t pieces, void* params, void* stream) {
  const int64_t grid = ceil_div(N, kWarps) > 0x7FFFFFFF / pieces ? 0 : ceil_div(N * pieces, kWarps);
  if (!grid || grid > 0x7FFFFFFF)
    return fail(VCOLL_ERR_UNSUPPORTED, "%lld rows of %lld pieces are too many", (long long)N,
                (long long)pieces);
  return launch_grid(fn, grid, 1, kRowThreads, 0, params, stream);
}

// The widest access, of `most`, 2 or 1 elements, that every row of an operand
// allows (row_access.cuh).  An absent operand allows any.
int access_of(const Operand& o, int most) {
  if (!o.ptr || !o.rows || !o.cols) return most;
  for (int a : {most, 2})
    if ((uint64_t)o.ptr % std::min(16, a * o.es) == 0 && o.cols % a == 0 &&
        (o.rows == 1 || o.ld % a == 0))
      return a;
  return 1;
}

// How a team of warps takes a row of D columns (norm_rows.cuh); 0 chunks: too
// wide for that.
struct NormShape {
  int warps, chunks, threads;
};
NormShape norm_shape(int64_t D, int E, bool grad) {
  const int64_t all = ceil_div(D, 32 * E);
  NormShape s = {1, 0, kNormCtaWarps * 32};
  if (all > (int64_t)kNormMaxWarps * norm_max_chunks(E, grad)) return s;
  s.chunks = 1;
  while (s.chunks < norm_chunks(E, grad) && s.chunks < all) s.chunks *= 2;
  while (ceil_div(all, s.chunks) > kNormMaxWarps) s.chunks *= 2;
  s.warps = (int)ceil_div(all, s.chunks);
  s.threads = s.warps * std::max(1, kNormCtaWarps / s.warps) * 32;
  return s;
}

// Launch of a norm_narrow.cuh kernel: as many CTAs as stay resident, at most
// `most`.  *ctas: how many.
int launch_norm_narrow(const void* fn, int lanes, int64_t most, NormParams* p, void* stream, int* ctas) {
  int sms = 0, fit = 0;
  VCOLL_TRY(device_sms(&sms));
  VCOLL_TRY(device_residency(fn, kRowThreads, 0, &fit));
  const int64_t need = ceil_div(p->N, (int64_t)kWarps * kNarrowRows * (32 / lanes));
  *ctas = (int)std::min(most, std::min<int64_t>(need, (int64_t)sms * fit));
  return launch_grid(fn, *ctas, 1, kRowThreads, 0, p, stream);
}

// Launch of a norm_rows.cuh kernel: as many CTAs as stay resident, at most
// `most`.  *ctas: how many.
int launch_norm_rows(const void* fn, const NormShape& s, size_t smem, int64_t most, NormParams* p,
                     void* stream, int* ctas) {
  if (!fn)
    return fail(VCOLL_ERR_UNSUPPORTED, "no kernel for %d chunks and %d threads", s.chunks, s.threads);
  int sms = 0, fit = 0;
  VCOLL_TRY(device_sms(&sms));
  VCOLL_TRY(device_residency(fn, s.threads, smem, &fit));
  const int64_t need = ceil_div(p->N, s.threads / 32 / s.warps);
  *ctas = (int)std::min(most, std::min<int64_t>(need, (int64_t)sms * fit));
  return launch_grid(fn, *ctas, 1, s.threads, smem, p, stream);
}

// Access of two matrices: fp32 rows are taken in 16 or 4 bytes, bf16 in 16, 4 or 2.
int row_access(int a, int b, int dtype) {
  const int both = std::min(a, b);
  return dtype == VCOLL_F32 && both == 2 ? 1 : both;
}

// Up to this many tokens one CTA sorts (2048: 20 us a call; 4096: 25 us, no
// less than many CTAs take).
constexpr int64_t kSortOneCta = 2048;

// Bytes that are moved for absent rows beside each pass of the sort and beside
// the join, about what the time that these take allows (16384 tokens into 32000
// x 2048 fp32: 70 us with 64 MB, 74 with 48, 77 with 96).
constexpr int64_t kFillPassBytes = 64 << 20;
// Bytes of a row that a warp fills there, where few CTAs have little time, and
// beside the sums (4096 tokens into 32000 x 5120 fp32: 120 us with 4096 and
// 16384, 125 with 8192, 152 with whole rows; 262144 tokens into 128000 x 4096,
// whose sums do most of the filling: 692 us, and 706 with 4096 there, too).
constexpr int64_t kFillPiece = 4096, kFillPieceSums = 16384;
// Bytes of the gradient that are fetched to L2 (129 MB) meanwhile, at most, where
// its rows have kPrefetchRow bytes or more: 65536 x 2048 bf16 into 8000 rows 94
// us without, 90 with 32 MB, 87 with 64 and 89 with 96; 100000 rows of 512 bytes,
// whose sums wait for other things, 45 without and 46 with any.
constexpr int64_t kPrefetchBytes = 64 << 20;
constexpr int64_t kPrefetchRow = 1024;

// Whether the list of the embedding's gradient is short enough not to be sorted:
// a warp for each place and tile reads it.
bool grad_is_short(int64_t N, int64_t D) {
  return N <= kSmallTokens && N * N * ceil_div(D, 256) <= kSmallWork;
}

// The workspace of the embedding's gradient.
struct GradLayout {
  int passes, bits;            // of the sort
  int64_t sort_tile, chunk;
  size_t list, cnt, stamp, part, bytes;  // bytes of one list; offsets; all
};
GradLayout grad_layout(int64_t N, int64_t V, int64_t D) {
  GradLayout L;
  int bits = 1;  // of keys 0 .. V
  while (bits < 31 && (V >> bits)) ++bits;
  L.passes = (int)ceil_div(bits, kSortMaxBits);
  L.bits = (int)ceil_div(bits, L.passes);
  L.sort_tile = std::max(N <= kSortFineMost ? kSortFineTile : kSortMinTile,
                         ceil_div(ceil_div(N, kSortMaxTiles), 32) * 32);
  // Places per warp: enough chunks for two waves of 32 warps on 152 SMs, each
  // of 16 places at least (partial rows are traffic) and 256 at most.
  const int64_t tiles = ceil_div(D, 256);
  L.chunk = std::min<int64_t>(256, std::max<int64_t>(1, ceil_div(N * tiles, 2 * 32 * 152 * 16)) * 16);
  L.list = align256((size_t)N * sizeof(uint32_t));
  L.cnt = 4 * L.list;
  L.stamp = L.cnt;
  if (N > kSortOneCta)
    L.stamp += align256((size_t)L.passes * (size_t)ceil_div(N, L.sort_tile) * sizeof(uint32_t) << L.bits);
  L.part = L.stamp + align256((size_t)V * sizeof(uint32_t));
  // rows of partial sums are padded to whole tiles, of 256 columns at most
  L.bytes = L.part + align256((size_t)ceil_div(N, L.chunk) * 2 * (size_t)tiles * 256 * sizeof(float));
  return L;
}

}  // namespace

extern "C" {

int vcoll_embedding(const void* tokens, int index_type, int64_t N, const void* table,
                    int64_t table_ld, int64_t V, int64_t D, float scale, void* out,
                    int64_t out_ld, int dtype, void* stream) {
  VCOLL_TRY(check_type(dtype, "dtype"));
  if (index_type != VCOLL_I32 && index_type != VCOLL_I64)
    return fail(VCOLL_ERR_INVALID_TYPE, "unknown index type %d", index_type);
  VCOLL_TRY(check_extent(N, "N"));
  VCOLL_TRY(check_extent(V, "V"));
  VCOLL_TRY(check_extent(D, "D", kMaxWidth));
  const int es = elem_size(dtype);
  const Operand ops[] = {
      {"tokens", tokens, D ? N : 0, 1, 1, index_type == VCOLL_I64 ? 8 : 4, false, nullptr},
      {"table", table, N ? V : 0, D, table_ld, es, false, nullptr},
      {"out", out, N, D, out_ld, es, true, nullptr}};
  VCOLL_TRY(check_operands(ops, 3));
  if (!N || !D) return VCOLL_OK;
  EmbedParams p = {};
  p.tokens = tokens;
  p.table = table;
  p.out = out;
  p.N = N;
  p.V = V;
  p.D = D;
  p.table_ld = table_ld;
  p.out_ld = out_ld;
  p.scale = scale;
  p.idx64 = index_type == VCOLL_I64;
  const int E = 16 / es, access = std::min(access_of(ops[1], E), access_of(ops[2], E));
  if (const int lanes = narrow_lanes(D, E))
    return launch_narrow(embed_narrow_kernel(dtype, access, lanes), N, lanes, &p, stream);
  p.pieces = ceil_div(D, lookup_accesses(access, E) * 32 * access);
  return launch_pieces(embed_kernel(dtype, access), N, p.pieces, &p, stream);
}

size_t vcoll_embedding_backward_workspace_bytes(int64_t N, int64_t V, int64_t D) {
  if (N <= 0 || V <= 0 || D <= 0 || N > kMaxExtent || V > kMaxExtent || D > kMaxWidth ||
      grad_is_short(N, D))
    return 0;
  return grad_layout(N, V, D).bytes;
}

int vcoll_embedding_backward(const void* grad, int64_t grad_ld, int dtype, const void* tokens,
                             int index_type, int64_t N, int64_t V, int64_t D, float scale,
                             const void* base, int64_t base_ld, void* table_grad,
                             int64_t table_ld, int table_dtype, void* workspace,
                             size_t workspace_bytes, void* stream) {
  VCOLL_TRY(check_type(dtype, "dtype"));
  VCOLL_TRY(check_type(table_dtype, "table dtype"));
  if (index_type != VCOLL_I32 && index_type != VCOLL_I64)
    return fail(VCOLL_ERR_INVALID_TYPE, "unknown index type %d", index_type);
  VCOLL_TRY(check_extent(N, "N"));
  VCOLL_TRY(check_extent(V, "V"));
  VCOLL_TRY(check_extent(D, "D", kMaxWidth));
  const int es = elem_size(dtype), ts = elem_size(table_dtype);
  const size_t need = vcoll_embedding_backward_workspace_bytes(N, V, D);
  const Operand ops[] = {
      {"tokens", tokens, V && D ? N : 0, 1, 1, index_type == VCOLL_I64 ? 8 : 4, false, nullptr},
      {"grad", grad, V ? N : 0, D, grad_ld, es, false, nullptr},
      {"base", base, base ? V : 0, D, base_ld, ts, false, nullptr},
      {"table_grad", table_grad, V, D, table_ld, ts, true, base},
      {"workspace", workspace, need ? 1 : 0, (int64_t)need, (int64_t)need, 1, true, nullptr}};
  VCOLL_TRY(check_operands(ops, 4));
  VCOLL_TRY(check_workspace(workspace, workspace_bytes, need));
  VCOLL_TRY(check_operands(ops, 5));
  if (!V || !D) return VCOLL_OK;
  const bool in_place = base && base == table_grad;
  if (!N && in_place) return VCOLL_OK;
  EmbedGradParams p = {};
  p.tokens = tokens;
  p.grad = grad;
  p.base = base;
  p.out = table_grad;
  p.N = N;
  p.V = V;
  p.D = D;
  p.grad_ld = grad_ld;
  p.base_ld = base_ld;
  p.out_ld = table_ld;
  p.scale = scale;
  p.idx64 = index_type == VCOLL_I64;
  p.table_es = ts;
  // the fill copies bytes: rows of base and table_grad in pieces of 16, 4 or 2
  p.fill_bytes = std::min(access_of(ops[2], 16 / ts), access_of(ops[3], 16 / ts)) * ts;
  if (p.fill_bytes == 8) p.fill_bytes = 4;
  const int E = 16 / es;
  int access = E;
  for (const Operand* o = ops + 1; o < ops + 4; ++o) access = std::min(access, access_of(*o, E));
  p.tiles = ceil_div(D, 32 * E);
  auto kernel = [&](GradPart part) { return embed_grad_kernel(dtype, table_dtype, access, part); };
  if (grad_is_short(N, D)) {
    p.sum_ctas = ceil_div(N * p.tiles, kWarps);
    // a row for each warp, or eight where there are rows for all SMs
    p.fill_each = ceil_div(V, 8 * kWarps) >= 608 ? 8 * kWarps : kWarps;
    return launch_grid(kernel(GRAD_SMALL), p.sum_ctas + (in_place ? 0 : ceil_div(V, p.fill_each)), 1,
                       kRowThreads, 0, &p, stream);
  }
  const GradLayout L = grad_layout(N, V, D);
  char* ws = (char*)workspace;
  for (int k = 0; k < 2; ++k) {
    p.key[k] = (uint32_t*)(ws + (size_t)(2 * k) * L.list);
    p.pos[k] = (uint32_t*)(ws + (size_t)(2 * k + 1) * L.list);
  }
  p.cnt = (uint32_t*)(ws + L.cnt);
  p.stamp = (uint32_t*)(ws + L.stamp);
  p.part = (float*)(ws + L.part);
  p.passes = L.passes;
  p.bits = L.bits;
  p.sort_tile = L.sort_tile;
  p.chunk = L.chunk;
  p.sum_ctas = ceil_div(ceil_div(N, p.chunk) * p.tiles, kWarps);
  if (p.sum_ctas + ceil_div(ceil_div(V, kFillRows) * ceil_div(D * ts, kFillPiece), kWarps) > 0x7FFFFFFF)
    return fail(VCOLL_ERR_UNSUPPORTED, "%lld rows of %lld columns are too many", (long long)N,
                (long long)D);
  // Rows of absent tokens are filled beside the sort's passes and the join,
  // kFillPassBytes each, the others beside the sums.  In place all of them stay.
  const bool join = N > p.chunk;  // a token may reach a second chunk
  const int64_t share = std::max<int64_t>(1, kFillPassBytes / (D * ts * (base ? 2 : 1)));
  const int64_t early = N <= kSortOneCta ? 0 : std::min(V, p.passes * share);
  const int64_t last = in_place || !join ? V : V - std::min(V - early, share);  // the join's first
  p.fill_end = in_place ? V : 0;  // rows filled so far
  // the next `count` rows, and CTAs of `warps` warps for them
  auto take = [&](int64_t count, int64_t end, int64_t warps, int64_t piece) {
    p.fill_piece = piece;
    p.fill_pieces = ceil_div(D * ts, piece);
    p.fill_begin = p.fill_end;
    p.fill_end = std::min(end, p.fill_begin + count);
    return ceil_div(ceil_div(p.fill_end - p.fill_begin, kFillRows) * p.fill_pieces, warps);
  };
  const size_t smem = ((size_t)1 << kSortMaxBits) * (kSortThreads / 32) * sizeof(uint32_t);
  if (N <= kSortOneCta) {
    VCOLL_TRY(launch_grid(embed_sort_kernel(), 1, 1, kSortThreads, smem, &p, stream));
  } else {
    p.sort_tiles = (int)ceil_div(N, L.sort_tile);
    // where there are no rows to fill yet, or none left, rows of the gradient go
    // to L2; the count takes half a pass's time (16384 x 2048 bf16 into 32000:
    // 69.5 us with nothing beside it, 67.2 with 32 MB, 68.2 with 48)
    p.grad_es = es;
    p.row_lines = ceil_div(D * es, 128);
    const int64_t lines = D * es < kPrefetchRow ? 0 : std::min(N * p.row_lines, kPrefetchBytes / 128);
    auto fetch = [&](int64_t bytes) {
      p.line_begin = p.line_end;
      p.line_end = std::min(lines, p.line_begin + std::max<int64_t>(0, bytes) / 128);
      return ceil_div(p.line_end - p.line_begin, kSortThreads * kPrefetchLines);
    };
    int64_t ahead = fetch(kFillPassBytes / 2);
    VCOLL_TRY(launch_grid(embed_count_kernel(), p.sort_tiles + ahead, 1, kSortThreads, smem, &p, stream));
    for (p.pass = 0; p.pass < p.passes; ++p.pass) {
      p.fill_ctas = (int)take(share, last, kSortThreads / 32, kFillPiece);
      ahead = fetch((share - (p.fill_end - p.fill_begin)) * D * ts);
      VCOLL_TRY(launch_grid(embed_scatter_kernel(), p.sort_tiles + p.fill_ctas + ahead, 1,
                            kSortThreads, smem, &p, stream));
    }
  }
  const int64_t fill = take(V, last, kWarps, kFillPieceSums);
  VCOLL_TRY(launch_grid(kernel(base ? GRAD_SUM_BASE : GRAD_SUM), p.sum_ctas + fill, 1, kRowThreads,
                        0, &p, stream));
  if (!join) return VCOLL_OK;
  const int64_t rest = take(V, V, kWarps, kFillPiece);
  return launch_grid(kernel(GRAD_JOIN), p.sum_ctas + rest, 1, kRowThreads, 0, &p, stream);
}

// x, y (or grad, dx) and the 8-bit operands of the layer norm entry points
static int norm_checks(int64_t N, int64_t D, int dtype, int weight_dtype) {
  VCOLL_TRY(check_type(dtype, "dtype"));
  VCOLL_TRY(check_type(weight_dtype, "weight dtype"));
  VCOLL_TRY(check_extent(N, "N"));
  return check_extent(D, "D", kMaxWidth);
}

static int check_codes(const void* codes, int64_t codes_ld, int64_t N, int64_t D) {
  if (!N || !D) return VCOLL_OK;
  if ((uint64_t)codes % 16 || codes_ld % 16)
    return fail(VCOLL_ERR_INVALID_ARG, "codes and their row stride must be multiples of 16 bytes");
  return VCOLL_OK;
}

// columns of a row of codes that are written
static int64_t codes_cols(int64_t D) { return (D + 15) / 16 * 16; }
static int64_t blocks_of(int64_t D) { return ceil_div(D, VCOLL_CHECKPOINT8_BLOCK); }

static int norm_forward(const void* x, int64_t x_ld, const void* weight, const void* bias,
                        int weight_dtype, int64_t N, int64_t D, float eps, void* y, int64_t y_ld,
                        float* mean, float* rstd, bool keep, int8_t* codes, int64_t codes_ld,
                        float* scales, int dtype, void* stream) {
  VCOLL_TRY(norm_checks(N, D, dtype, weight_dtype));
  const int es = elem_size(dtype), ws = elem_size(weight_dtype);
  const int64_t K = keep ? N : 0, B = blocks_of(D);
  const Operand ops[] = {{"x", x, N, D, x_ld, es, false, nullptr},
                         {"weight", weight, weight && N ? 1 : 0, D, D, ws, false, nullptr},
                         {"bias", bias, bias && N ? 1 : 0, D, D, ws, false, nullptr},
                         {"y", y, N, D, y_ld, es, true, x},
                         {"mean", mean, mean && D ? 1 : 0, N, N, 4, true, nullptr},
                         {"rstd", rstd, rstd && D ? 1 : 0, N, N, 4, true, nullptr},
                         {"codes", codes, K, codes_cols(D), codes_ld, 1, true, nullptr},
                         {"scales", scales, K, B, B, 4, true, nullptr}};
  if (keep) VCOLL_TRY(check_codes(codes, codes_ld, N, D));
  VCOLL_TRY(check_operands(ops, 8));
  if (!N || !D) return VCOLL_OK;
  NormParams p = {};
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.y = y;
  p.mean = mean;
  p.rstd = rstd;
  p.codes = keep ? codes : nullptr;
  p.scales = scales;
  p.N = N;
  p.D = D;
  p.x_ld = x_ld;
  p.y_ld = y_ld;
  p.codes_ld = codes_ld;
  p.eps = eps;
  p.wbf16 = weight_dtype == VCOLL_BF16;
  const int E = 16 / es;
  int access = E, ctas;
  for (int k = 0; k < 4; ++k) access = row_access(access, access_of(ops[k], E), dtype);
  if (const int lanes = narrow_lanes(D, E)) {
    // weight and bias are read once, element by element
    access = row_access(access_of(ops[0], E), access_of(ops[3], E), dtype);
    const void* fn = dtype == VCOLL_F32 ? norm_narrow_kernel_f32(access, lanes, false, keep)
                                        : norm_narrow_kernel_bf16(access, lanes, false, keep);
    return launch_norm_narrow(fn, lanes, kMaxExtent, &p, stream, &ctas);
  }
  const NormShape s = norm_shape(D, E, false);
  if (!s.chunks) {
    int64_t grid;
    VCOLL_TRY(grid_for(N, 1, 32, &grid));
    return launch_grid(norm_wide_kernel(dtype), grid, 1, kRowThreads, 0, &p, stream);
  }
  p.warps = s.warps;
  const void* fn = dtype == VCOLL_F32 ? norm_rows_kernel_f32(access, s.chunks, s.threads, false, keep)
                                      : norm_rows_kernel_bf16(access, s.chunks, s.threads, false, keep);
  // the ring, and two partial sums of 8 bytes a warp
  const size_t smem =
      (size_t)s.threads * 16 * s.chunks * norm_stages(s.chunks, E, false) + s.threads / 2;
  return launch_norm_rows(fn, s, smem, kMaxExtent, &p, stream, &ctas);
}

static int norm_backward(const void* grad, int64_t grad_ld, const void* x, int64_t x_ld,
                         const int8_t* codes, int64_t codes_ld, const float* scales,
                         const float* mean, const float* rstd, const void* weight,
                         int weight_dtype, int64_t N, int64_t D, void* dx, int64_t dx_ld,
                         void* dweight, void* dbias, bool kept, int dtype, void* workspace,
                         size_t workspace_bytes, void* stream) {
  VCOLL_TRY(norm_checks(N, D, dtype, weight_dtype));
  const int es = elem_size(dtype), ws = elem_size(weight_dtype);
  const int64_t K = kept ? N : 0, X = kept ? 0 : N, B = blocks_of(D);
  const bool alias_grad = dx == grad;
  const size_t need = vcoll_layer_norm_workspace_bytes(N, D);
  const Operand ops[] = {
      {"grad", grad, N, D, grad_ld, es, false, nullptr},
      {"x", x, X, D, x_ld, es, false, nullptr},
      {"mean", mean, X && D ? 1 : 0, N, N, 4, false, nullptr},
      {"rstd", rstd, N && D ? 1 : 0, N, N, 4, false, nullptr},
      {"codes", codes, K, D, codes_ld, 1, false, nullptr},
      {"scales", scales, K, B, B, 4, false, nullptr},
      {"weight", weight, weight && N ? 1 : 0, D, D, ws, false, nullptr},
      {"dx", dx, dx ? N : 0, D, dx_ld, es, true, alias_grad ? grad : x},
      {"dweight", dweight, dweight ? 1 : 0, D, D, ws, true, nullptr},
      {"dbias", dbias, dbias ? 1 : 0, D, D, ws, true, nullptr},
      {"workspace", workspace, need ? 1 : 0, (int64_t)need, (int64_t)need, 1, true, nullptr}};
  if (kept) VCOLL_TRY(check_codes(codes, codes_ld, N, D));
  VCOLL_TRY(check_operands(ops, 10));
  VCOLL_TRY(check_workspace(workspace, workspace_bytes, need));
  VCOLL_TRY(check_operands(ops, 11));
  if (!D) return VCOLL_OK;
  NormParams p = {};
  p.x = kept ? nullptr : x;
  p.grad = grad;
  p.weight = weight;
  p.y = dx;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.codes = const_cast<int8_t*>(codes);
  p.scales = const_cast<float*>(scales);
  p.dweight = dweight;
  p.dbias = dbias;
  p.part = (float*)workspace;
  p.N = N;
  p.D = D;
  p.x_ld = x_ld;
  p.grad_ld = grad_ld;
  p.y_ld = dx_ld;
  p.codes_ld = codes_ld;
  p.wbf16 = weight_dtype == VCOLL_BF16;
  const int E = 16 / es;
  const int lanes = narrow_lanes(D, E);
  const NormShape s = norm_shape(D, E, true);
  if (!s.chunks) {
    if (dweight || dbias)
      VCOLL_TRY(launch_grid(norm_wgrad_wide_kernel(dtype), ceil_div(D, 32), 1, kRowThreads, 0, &p, stream));
    if (!dx || !N) return VCOLL_OK;
    int64_t grid;
    VCOLL_TRY(grid_for(N, 1, 32, &grid));
    return launch_grid(norm_grad_wide_kernel(dtype), grid, 1, kRowThreads, 0, &p, stream);
  }
  if (!dx && !dweight && !dbias) return VCOLL_OK;
  if (N) {
    p.part = dweight || dbias ? (float*)workspace : nullptr;
    int access = E;
    for (int k : {0, 1, 7}) access = row_access(access, access_of(ops[k], E), dtype);
    if (lanes) {
      const void* fn = dtype == VCOLL_F32 ? norm_narrow_kernel_f32(access, lanes, true, kept)
                                          : norm_narrow_kernel_bf16(access, lanes, true, kept);
      VCOLL_TRY(launch_norm_narrow(fn, lanes, kNormMaxCtas, &p, stream, &p.parts));
    } else {
      p.warps = s.warps;
      access = row_access(access, access_of(ops[6], E), dtype);
      const void* fn = dtype == VCOLL_F32
                           ? norm_rows_kernel_f32(access, s.chunks, s.threads, true, kept)
                           : norm_rows_kernel_bf16(access, s.chunks, s.threads, true, kept);
      const size_t smem =
          (size_t)s.threads * (norm_stages(s.chunks, E, true) * norm_grad_slot_bytes(s.chunks, E, kept) +
                               norm_grad_smem_sums(s.chunks, E) * s.chunks * E * 4) +
          s.threads / 2;
      VCOLL_TRY(launch_norm_rows(fn, s, smem, kNormMaxCtas, &p, stream, &p.parts));
    }
  }
  if (!dweight && !dbias) return VCOLL_OK;
  return launch_grid(norm_wsum_kernel(), ceil_div(D, 32), 2, 1024, 0, &p, stream);
}

int vcoll_layer_norm(const void* x, int64_t x_ld, const void* weight, const void* bias,
                     int weight_dtype, int64_t N, int64_t D, float eps, void* y, int64_t y_ld,
                     float* mean, float* rstd, int dtype, void* stream) {
  return norm_forward(x, x_ld, weight, bias, weight_dtype, N, D, eps, y, y_ld, mean, rstd, false,
                      nullptr, 0, nullptr, dtype, stream);
}

int vcoll_layer_norm_checkpoint8(const void* x, int64_t x_ld, const void* weight,
                                 const void* bias, int weight_dtype, int64_t N, int64_t D,
                                 float eps, void* y, int64_t y_ld, float* rstd, int8_t* codes,
                                 int64_t codes_ld, float* scales, int dtype, void* stream) {
  return norm_forward(x, x_ld, weight, bias, weight_dtype, N, D, eps, y, y_ld, nullptr, rstd, true,
                      codes, codes_ld, scales, dtype, stream);
}

size_t vcoll_layer_norm_workspace_bytes(int64_t N, int64_t D) {
  // partial rows of the CTAs, for rows that a team holds (in either type)
  if (N <= 0 || D <= 0 || D > kNormMaxWarps * 32 * 32) return 0;
  return (size_t)std::min<int64_t>(N, kNormMaxCtas) * 2 * (size_t)D * sizeof(float);
}

int vcoll_layer_norm_backward(const void* grad, int64_t grad_ld, const void* x, int64_t x_ld,
                              const float* mean, const float* rstd, const void* weight,
                              int weight_dtype, int64_t N, int64_t D, void* dx, int64_t dx_ld,
                              void* dweight, void* dbias, int dtype, void* workspace,
                              size_t workspace_bytes, void* stream) {
  return norm_backward(grad, grad_ld, x, x_ld, nullptr, 0, nullptr, mean, rstd, weight,
                       weight_dtype, N, D, dx, dx_ld, dweight, dbias, false, dtype, workspace,
                       workspace_bytes, stream);
}

int vcoll_layer_norm_backward_checkpoint8(const void* grad, int64_t grad_ld, const int8_t* codes,
                                          int64_t codes_ld, const float* scales,
                                          const float* rstd, const void* weight, int weight_dtype,
                                          int64_t N, int64_t D, void* dx, int64_t dx_ld,
                                          void* dweight, void* dbias, int dtype, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  return norm_backward(grad, grad_ld, nullptr, 0, codes, codes_ld, scales, nullptr, rstd, weight,
                       weight_dtype, N, D, dx, dx_ld, dweight, dbias, true, dtype, workspace,
                       workspace_bytes, stream);
}

int vcoll_checkpoint8(const void* x, int64_t x_ld, int64_t N, int64_t D, int8_t* codes,
                      int64_t codes_ld, float* scales, int dtype, void* stream) {
  VCOLL_TRY(norm_checks(N, D, dtype, VCOLL_F32));
  const int64_t B = blocks_of(D);
  const Operand ops[] = {{"x", x, N, D, x_ld, elem_size(dtype), false, nullptr},
                         {"codes", codes, N, codes_cols(D), codes_ld, 1, true, nullptr},
                         {"scales", scales, N, B, B, 4, true, nullptr}};
  VCOLL_TRY(check_codes(codes, codes_ld, N, D));
  VCOLL_TRY(check_operands(ops, 3));
  if (!N || !D) return VCOLL_OK;
  const int E = 16 / elem_size(dtype);
  PackParams p = {};
  p.x = x;
  p.codes = codes;
  p.scales = scales;
  p.N = N;
  p.D = D;
  p.x_ld = x_ld;
  p.codes_ld = codes_ld;
  const int access = row_access(access_of(ops[0], E), E, dtype);
  if (const int lanes = narrow_lanes(D, E))
    return launch_narrow(pack8_narrow_kernel(dtype, access, lanes, false), N, lanes, &p, stream);
  p.pieces = ceil_div(D, kPackChunks * 32 * E);
  return launch_pieces(pack8_kernel(dtype, access), N, p.pieces, &p, stream);
}

int vcoll_checkpoint8_restore(const int8_t* codes, int64_t codes_ld, const float* scales,
                              const void* weight, const void* bias, int weight_dtype, int64_t N,
                              int64_t D, void* out, int64_t out_ld, int dtype, void* stream) {
  VCOLL_TRY(norm_checks(N, D, dtype, weight_dtype));
  const int ws = elem_size(weight_dtype);
  const int64_t B = blocks_of(D);
  const Operand ops[] = {{"codes", codes, N, D, codes_ld, 1, false, nullptr},
                         {"scales", scales, N, B, B, 4, false, nullptr},
                         {"weight", weight, weight && N ? 1 : 0, D, D, ws, false, nullptr},
                         {"bias", bias, bias && N ? 1 : 0, D, D, ws, false, nullptr},
                         {"out", out, N, D, out_ld, elem_size(dtype), true, nullptr}};
  VCOLL_TRY(check_codes(codes, codes_ld, N, D));
  VCOLL_TRY(check_operands(ops, 5));
  if (!N || !D) return VCOLL_OK;
  const int E = 16 / elem_size(dtype);
  PackParams p = {};
  p.out = out;
  p.weight = weight;
  p.bias = bias;
  p.codes = const_cast<int8_t*>(codes);
  p.scales = const_cast<float*>(scales);
  p.N = N;
  p.D = D;
  p.x_ld = out_ld;
  p.codes_ld = codes_ld;
  p.wbf16 = weight_dtype == VCOLL_BF16;
  int access = row_access(access_of(ops[4], E), E, dtype);
  if (const int lanes = narrow_lanes(D, E))  // weight and bias by single elements
    return launch_narrow(pack8_narrow_kernel(dtype, access, lanes, true), N, lanes, &p, stream);
  for (int k : {2, 3}) access = row_access(access, access_of(ops[k], E), dtype);
  p.pieces = ceil_div(D, kPackChunks * 32 * E);
  return launch_pieces(unpack8_kernel(dtype, access), N, p.pieces, &p, stream);
}

}  // extern "C"
