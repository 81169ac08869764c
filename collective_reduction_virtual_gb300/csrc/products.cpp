// Host side of the products declared in include/vcoll.h (the loss against a
// vocabulary, the gated feed-forward block): argument checks, the workspace's
// layout, pieces of the vocabulary, and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <array>
#include <cmath>

#include "layer_checks.h"
#include "mm_internal.h"

using namespace vcoll;

namespace {

constexpr int64_t kPackBytes = 256 << 20;   // of a piece of the table, laid out
// of the gradient's e for a piece (4096 x 128000 x 4096 bf16: 7.63 ms with 64 MB, 7.39
// with 128, 7.26 with 256 and 7.20 with 512)
constexpr int64_t kErrorBytes = 256 << 20;
// and, where the rows are so many that the narrowest piece of e takes more, of e for a
// block of rows: half of a million fp32 rows of 64 columns would take 6.4 GB at once.
// Blocks of a quarter of this (65536 rows of bf16) cost up to 12 % (65536 x 8000 x 512
// fp32 6.7 ms with all rows at once, 7.5 with four blocks; 131072 x 32000 x 4096 bf16
// 68.1 and 68.4 with two).
constexpr int64_t kBlockBytes = 1 << 30;
constexpr int64_t kPartBytes = 128 << 20;   // of the loss's tiles of a piece
constexpr int kPassThreads = 256;           // of the kernels of mm_parts.cu

// SMs that tiles and splits are planned for: a plan (and with it a workspace and
// the order of the sums) does not depend on the GPU.
constexpr int64_t kPlanSms = 152;

int64_t round_up(int64_t v, int64_t to) { return ceil_div(v, to) * to; }
int parts_of(int dtype) { return dtype == VCOLL_F32 ? 3 : 1; }
// Of the gradients of gate and up.  Rounded to one bf16 they make bf16 results off by
// sqrt(2) times their own rounding (measured 1.37 to 1.43), as those of a program are
// that keeps them in bf16.  That is a mean over n roundings, which chance moves by some
// 1 / sqrt(n): over a hundred by 10 % and more (1.6 was seen), over 8192 by 1 %.  Up to
// there they take two parts and results are off by their own rounding alone (1.00).
// N x D, F in us with two parts and with one: 1 x 1024, 4096 29 and 29; 8 x 1024, 1024
// 27 and 29; 1 x 4096, 8192 102 and 77.  Of more values they would cost 1 x 4096, 11008
// 128 instead of 98, 3001 x 1001, 2671 117 instead of 70.
constexpr int64_t kFineValues = 8192;
int grad_parts(int64_t N, int64_t F, int dtype) { return dtype == VCOLL_F32 ? 3 : N * F <= kFineValues ? 2 : 1; }

// Regions of a workspace, one after the other.
struct Regions {
  size_t bytes = 0;
  size_t take(int64_t n) {
    const size_t at = bytes;
    bytes += align256((size_t)n);
    return at;
  }
};

// A matrix laid out as parts: rows of whole 128-byte lines, which a step of a
// product reads one of.
constexpr int64_t kPackedCols = 64;
int64_t packed_bytes(int64_t rows, int64_t cols, int parts) {
  return rows * round_up(cols, kPackedCols) * 2 * parts;
}

// A product to be planned.
struct Shape {
  int64_t M, N, K;
  int parts;
  bool halves;
  int epilogue;  // cycles that it takes for a column of a tile
};
// Measured on tiles of little depth: 64 columns of bf16 at once, 32 of fp32 (or its
// parts), and those whose rows something is added to, which is waited for.
int epilogue_cycles(int parts, bool add = false) { return add ? 40 : parts > 2 ? 40 : 12; }

// How a launch's products are cut: CTAs that share a tile, and for each product the
// tile's columns, the splits of its sum, and a unit's cycles.
struct Plan {
  int ctas = 1;
  struct {
    int tn = 256, splits = 1;
    double unit = 0;
    size_t bytes = 0;  // of the splits' sums
  } of[2];
  size_t bytes() const { return align256(of[0].bytes) + align256(of[1].bytes); }
};

// Cycles of a step of 64 places: a pair of CTAs sums 256 columns at the tensor
// cores' rate, fewer or one CTA's less well (4096 x 16384 x 2048, bf16: 1930 TFLOP/s
// with 256 columns and 1780 with 128, and 1750, 1520 and 860 by one CTA with 256, 128
// and 64).
double step_cycles(int ctas, int tn) {
  if (ctas == 2) return tn == 256 ? 512 : 280;
  return tn == 256 ? 565 : tn == 128 ? 325 : 290;
}

// The cheapest by a model of cycles.  A step takes the tensor cores' time, or as long
// as its operands take to arrive, at 45 bytes a cycle and SM from memory where one
// row of tiles takes each column once, 3600 for all SMs, and at 80 from L2 where rows
// of tiles share them.  A tile's epilogue goes beside the next tile's sum, but
// for the last one's.  Alone, a product takes whole waves of units; two fill each
// other's last waves to within a unit.
Plan search_plan(const Shape* shape, int count) {
  Plan best;
  double least = -1;
  for (int ctas : {2, 1}) {
    if (ctas == 2 && shape[0].M <= kMmRows && (count == 1 || shape[1].M <= kMmRows)) continue;
    const double slots = kPlanSms / ctas;
    struct Choice {
      int tn, splits;
      double units, unit, join, tail;
      size_t bytes;
    } choice[2][48];
    int choices[2] = {0, 0};
    for (int i = 0; i < count; ++i) {
      const Shape& s = shape[i];
      const int64_t tile_rows = kMmRows * ctas, rows = std::min<int64_t>(s.M, tile_rows);
      const int64_t steps = mm_pairs(s.parts) * ceil_div(s.K, kMmDepth), tiles_m = ceil_div(s.M, tile_rows);
      for (int tn : {256, 128, 64}) {
        if (tn == 64 && (s.halves || ctas == 2)) continue;
        const double tiles = (double)tiles_m * (double)ceil_div(s.N, s.halves ? tn / 2 : tn);
        const double bytes = 128.0 * (double)(std::min<int64_t>(s.M, kMmRows) + tn / ctas);
        for (int k : {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 14, 16}) {
          if (k > 1 && (steps / k < 4 || tiles * k > 8 * kPlanSms)) break;
          const double units = tiles * k, rate = tiles_m > 1 ? 80 : std::min(45.0, 3600 / std::min(units, slots));
          const double step = std::max(step_cycles(ctas, tn), bytes / rate);
          Choice& c = choice[i][choices[i]++];
          const double tail = (double)s.epilogue * tn + 1000;
          c = {tn, k, units, std::max((double)ceil_div(steps, k) * step, k > 1 ? 12.0 * tn : tail) + 200, 0.0, tail, 0};
          if (k > 1) {
            c.bytes = (size_t)units * (size_t)rows * tn * sizeof(float);
            c.join = 2500 + (double)c.bytes * 2 / (10.0 * kPlanSms);
          }
        }
      }
    }
    for (int i = 0; i < choices[0]; ++i) {
      const Choice& a = choice[0][i];
      auto consider = [&](double cost, const Choice* b) {
        if (least >= 0 && cost >= least) return;
        least = cost;
        best.ctas = ctas;
        best.of[0] = {a.tn, a.splits, a.unit, a.bytes};
        if (b) best.of[1] = {b->tn, b->splits, b->unit, b->bytes};
      };
      if (count == 1) {
        consider(std::ceil(a.units / slots) * a.unit + a.tail + a.join, nullptr);
        continue;
      }
      for (int j = 0; j < choices[1]; ++j) {
        const Choice& b = choice[1][j];
        const double work = (a.units * a.unit + b.units * b.unit) / slots;
        consider(std::max(work + 0.5 * std::min(a.unit, b.unit), std::max(a.unit, b.unit)) + std::max(a.tail, b.tail) +
                     std::max(a.join, b.join),
                 &b);
      }
    }
  }
  return best;
}

// A program repeats the sizes of its calls: each thread keeps plans, one in a place
// that the sizes decide.
Plan make_plan(const Shape* shape, int count) {
  struct Kept {
    Shape shape[2];
    int count = 0;
    Plan plan;
  };
  static thread_local Kept kept[256];
  auto same = [](const Shape& a, const Shape& b) {
    return a.M == b.M && a.N == b.N && a.K == b.K && a.parts == b.parts && a.halves == b.halves &&
           a.epilogue == b.epilogue;
  };
  uint64_t place = (uint64_t)count;
  for (int i = 0; i < count; ++i)
    for (const int64_t v : {shape[i].M, shape[i].N, shape[i].K, (int64_t)shape[i].parts + 4 * shape[i].epilogue})
      place = (place ^ (uint64_t)v) * 0x9E3779B97F4A7C15ull;
  Kept& k = kept[place >> 56];
  if (k.count != count || !same(k.shape[0], shape[0]) || (count > 1 && !same(k.shape[1], shape[1]))) {
    for (int i = 0; i < count; ++i) k.shape[i] = shape[i];
    k.plan = search_plan(shape, count);
    k.count = count;
  }
  return k.plan;
}

Plan plan_of(const Shape& a) { return make_plan(&a, 1); }

// Whether the products are those of mm_few.cu, which read fp32 weights where they
// lie.
bool few_rows(int64_t N, int dtype) { return dtype == VCOLL_F32 && N <= kMmFewRows; }
// Splits of the sum of a product with a weight that is taken transposed: one wave of
// two CTAs per SM, of 256 places at least; the join adds them one after the other.
int64_t few_splits(int64_t N, int64_t K) {
  const int64_t fill = 2 * kPlanSms / std::max<int64_t>(1, ceil_div(N, 128));
  return std::max<int64_t>(1, std::min<int64_t>({fill, K / 256, 128}));
}
size_t few_bytes(int64_t M, int64_t N, int64_t K) {
  return (size_t)(ceil_div(N, 128) * few_splits(N, K) * M * 128) * sizeof(float);
}

// Columns of a piece of the vocabulary: `fit` at most, whole tiles, but not fewer than
// a product with them needs to be worth its launches.
constexpr int64_t kLeastPiece = 2048;
int64_t piece_of(int64_t V, int64_t fit) {
  return std::min(V, std::max<int64_t>(kLeastPiece, fit / 256 * 256));
}

// The sizes of the pieces that `all` are cut into: all but the last are alike.
std::array<int64_t, 2> widths_of(int64_t all, int64_t piece) {
  return {piece, piece ? all - (all - 1) / piece * piece : 0};
}

struct LossLayout {
  int64_t piece, pieces;
  size_t x, table, part, state, splits, bytes;
};
LossLayout loss_layout(int64_t N, int64_t V, int64_t D, int dtype, bool direct) {
  const int parts = parts_of(dtype);
  LossLayout L;
  const bool few = few_rows(N, dtype);
  int64_t fit = kPartBytes / (8 * std::max<int64_t>(N, 1)) * 256;
  if (!direct && !few) fit = std::min(fit, kPackBytes / std::max<int64_t>(1, packed_bytes(1, D, parts)));
  L.piece = piece_of(V, fit);
  L.pieces = std::max<int64_t>(1, L.piece ? ceil_div(V, L.piece) : 1);
  Regions r;
  L.x = r.take(direct ? 0 : packed_bytes(N, D, parts));
  L.table = r.take(direct || few ? 0 : packed_bytes(L.piece, D, parts));
  size_t splits = 0;
  int64_t tiles = 0;
  if (few) {
    tiles = ceil_div(L.piece, 64);
  } else {
    for (int64_t w : widths_of(V, L.piece)) {
      const Plan plan = plan_of({N, w, D, parts, false, epilogue_cycles(1)});
      splits = std::max(splits, plan.bytes());
      tiles = std::max(tiles, ceil_div(w, plan.of[0].tn));
    }
  }
  L.part = r.take(2 * tiles * N * (int64_t)sizeof(float2));
  L.splits = r.take((int64_t)splits);
  L.state = r.take(L.pieces > 1 ? N * (int64_t)sizeof(float2) : 0);
  L.bytes = r.bytes;
  return L;
}

// The gradient's e exists for a piece of the vocabulary and a block of rows at a time.
// A block has all rows, or where 2048 columns of them are more than kBlockBytes as many
// as fit: the table's gradient of a piece is then summed over the blocks in fp32.
struct LossGradLayout {
  int64_t piece, pieces, rows, blocks, error_ld;
  size_t scale, x, table, error, accum, table_accum, splits, bytes;
};
LossGradLayout loss_grad_layout(int64_t N, int64_t V, int64_t D, int dtype, bool direct) {
  const int parts = parts_of(dtype);
  LossGradLayout L;
  const bool few = few_rows(N, dtype);
  const int64_t least = std::min<int64_t>(std::max<int64_t>(round_up(V, kPackedCols), 1), kLeastPiece);
  const int64_t most = kBlockBytes / (2 * parts * least) / 256 * 256;
  L.blocks = std::max<int64_t>(1, ceil_div(N, most));
  L.rows = L.blocks > 1 ? round_up(ceil_div(N, L.blocks), 256) : N;
  int64_t fit = kErrorBytes / (2 * parts * std::max<int64_t>(L.rows, 1));
  if (!direct && !few) fit = std::min(fit, kPackBytes / std::max<int64_t>(1, packed_bytes(1, D, parts)));
  L.piece = piece_of(V, fit);
  L.pieces = std::max<int64_t>(1, L.piece ? ceil_div(V, L.piece) : 1);
  L.error_ld = round_up(L.piece, kPackedCols);
  Regions r;
  L.scale = r.take(sizeof(float));
  L.x = r.take(packed_bytes(N, D, parts));
  L.table = r.take(direct || few ? 0 : packed_bytes(L.piece, D, parts));
  L.error = r.take(L.rows * L.error_ld * 2 * parts);
  L.accum = r.take(L.pieces > 1 ? N * round_up(D, 2) * 4 : 0);
  L.table_accum = r.take(L.blocks > 1 ? L.piece * round_up(D, 2) * 4 : 0);
  size_t splits = 0;
  if (few) {
    splits = few_bytes(N, D, L.piece);
  } else {
    for (int64_t w : widths_of(V, L.piece))
      for (int64_t n : widths_of(N, L.rows)) {
        const Shape error = {n, w, D, parts, false, epilogue_cycles(parts)};
        splits = std::max(splits, plan_of(error).bytes());
        for (const bool add : {false, true}) {  // dx, dtable, and both
          const Shape s[2] = {{n, D, w, parts, false, epilogue_cycles(parts, L.pieces > 1)},
                              {w, D, n, parts, false, epilogue_cycles(parts, add)}};
          splits = std::max({splits, plan_of(s[0]).bytes(), plan_of(s[1]).bytes(), make_plan(s, 2).bytes()});
        }
      }
  }
  L.splits = r.take((int64_t)splits);
  L.bytes = r.bytes;
  return L;
}

struct GatedLayout {
  int64_t half;  // backward: gate's columns, a whole number of tiles
  size_t x, w_gate, w_up, grads, splits, bytes;
};
GatedLayout gated_layout(int64_t N, int64_t D, int64_t F, int dtype, bool direct, bool backward) {
  const int parts = parts_of(dtype);
  GatedLayout L;
  L.half = round_up(F, kMmRows);
  Regions r;
  L.x = r.take(direct ? 0 : packed_bytes(N, D, parts));
  const bool few = few_rows(N, dtype);
  L.w_gate = r.take(direct || few ? 0 : packed_bytes(F, D, parts));
  L.w_up = r.take(direct || few ? 0 : packed_bytes(F, D, parts));
  const int fine = grad_parts(N, F, dtype);
  L.grads = r.take(backward ? packed_bytes(N, 2 * L.half, fine > 1 ? 3 : 1) : 0);  // two parts are laid out as three
  size_t splits = 0;
  const int cycles = epilogue_cycles(parts);
  if (few) {
    splits = backward ? few_bytes(N, D, 2 * L.half) : 0;
  } else if (backward) {  // dx; one weight's gradient; both
    const Shape s[3] = {{N, D, 2 * L.half, fine, false, cycles},
                        {F, D, N, fine, false, cycles},
                        {2 * L.half, D, N, fine, false, cycles}};
    const Shape one[2] = {s[0], s[1]}, both[2] = {s[0], s[2]};
    splits = std::max({plan_of(s[0]).bytes(), plan_of(s[1]).bytes(), plan_of(s[2]).bytes(), make_plan(one, 2).bytes(),
                       make_plan(both, 2).bytes()});
  } else {
    splits = plan_of({N, F, D, parts, true, cycles}).bytes();
  }
  L.splits = r.take((int64_t)splits);
  L.bytes = r.bytes;
  return L;
}

constexpr int64_t kMaxStride = (int64_t)1 << 38;  // a tensor map's is below 2^40 bytes

// Whether the products can read the matrix where it lies.
bool lies_direct(const void* p, int64_t rows, int64_t cols, int64_t ld, int dtype) {
  if (!rows || !cols) return true;
  if (dtype != VCOLL_BF16 || (uint64_t)p % 16 || (rows > 1 && (ld % 8 || ld >= kMaxStride)))
    return false;
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return false;
  }
  return a.type == cudaMemoryTypeDevice;
}

MmOperand operand(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t plane = 0) {
  return {p, rows, cols, rows > 1 ? ld : round_up(std::max<int64_t>(cols, 1), 8), plane};
}

bool rows_at_16(const void* p, int64_t rows, int64_t ld, int es) {
  return (uint64_t)p % 16 == 0 && (rows <= 1 || ld * es % 16 == 0);
}

// CTAs of a pass of mm_parts.cu over so many groups of eight values, one a thread:
// CTAs in order keep what is in flight close together in memory (16384 x 11008
// gradients: 353 us, and 390 with eight CTAs per SM that go around).
int64_t pass_blocks(int64_t groups) { return std::min<int64_t>(ceil_div(groups, kPassThreads), 1 << 28); }

// Matrices that are laid out as parts by one launch.
struct Packer {
  MmPackParams p = {};
  int jobs = 0;
  int64_t blocks = 0;

  Packer(int dtype) {
    p.src_f32 = dtype == VCOLL_F32;
    p.parts = parts_of(dtype);
  }
  // The matrix where it lies, or laid out at `to`.  masked: rows whose target is
  // outside [0, V) as zeros.
  int add(const void* src, int64_t rows, int64_t cols, int64_t ld, bool direct, void* to, bool masked,
          MmOperand* o) {
    if (direct) {
      *o = operand(src, rows, cols, ld);
      return VCOLL_OK;
    }
    MmPackJob& j = p.job[jobs];
    j.src = src;
    j.dst = to;
    j.rows = rows;
    j.cols = cols;
    j.src_ld = ld;
    j.dst_ld = round_up(cols, kPackedCols);
    j.plane = rows * j.dst_ld;
    j.masked = masked;
    j.load16 = rows_at_16(src, rows, ld, p.src_f32 ? 4 : 2);
    *o = operand(to, rows, cols, j.dst_ld, j.plane);
    if (!rows || !cols) return VCOLL_OK;
    j.first_block = blocks;
    j.blocks = pass_blocks(rows * ceil_div(cols, 8));
    blocks += j.blocks;
    ++jobs;
    return VCOLL_OK;
  }
  // The parameters, once all matrices are there.
  MmPackParams& params() {
    for (int i = jobs; i < kMmPackJobs; ++i) p.job[i].first_block = INT64_MAX;
    if (!jobs) p.job[0].blocks = 1;
    return p;
  }
  int run(void* stream) {
    const int64_t all = blocks + (p.scale ? 1 : 0);
    return all ? launch_grid(mm_pack_kernel(), all, 1, kPassThreads, 0, &params(), stream) : VCOLL_OK;
  }
};

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                CUtensorMapFloatOOBfill);

// A tensor map of an operand (columns, rows, parts) with boxes of 64 columns and
// `box` rows; what a box reaches outside is read as zeros.
int encode(CUtensorMap* map, const MmOperand& o, int parts, int box) {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      f = nullptr;
    }
    return (EncodeTiled)f;
  }();
  if (!fn) return fail(VCOLL_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
  const cuuint64_t dims[3] = {(cuuint64_t)o.cols, (cuuint64_t)o.rows, (cuuint64_t)parts};
  const cuuint64_t strides[2] = {(cuuint64_t)o.ld * 2, (cuuint64_t)(parts > 1 ? o.plane : o.ld) * 2};
  const cuuint32_t boxes[3] = {kMmDepth, (cuuint32_t)box, 1}, steps[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(o.p), dims, strides,
                        boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(VCOLL_ERR_CUDA, "cuTensorMapEncodeTiled: error %d", (int)r);
  return VCOLL_OK;
}

// Rows that tiles are taken by, column after column: as many as stay in L2 meanwhile
// (kGroupBytes of a), so that b is read once for each group of them.  Where the sums
// are too long for that, 2048 rows make what is in flight about as high as wide.
// 8192 x 128000 x 4096 to the loss, us: 4930 with 1024 rows, 4735 with 2048, 4650 with
// 4096 (this rule's) and 4815 with 8192; sums of 16384 and 22016 places (the block's
// gradient): 3870, 3805 and 3930 with 1024, 2048 and 4096.
constexpr int64_t kGroupBytes = 40 << 20;
int64_t group_rows(int64_t K, int parts) {
  int64_t rows = 2048;
  while (rows < 8192 && 2 * rows * K * 2 * parts <= kGroupBytes) rows *= 2;
  return rows;
}

// Two products fill each other's last waves in one launch.  But their tiles then do
// not run in step, and where both sums are long, more of their operands lies between
// them than L2 holds (16384 rows: 10.6 to 17.4 GB read from memory, apart 7.3 to 12.8): those
// take a launch each, where each has a wave of tiles at least.  The block's gradient,
// us in one launch and in two, N x D, F: 16384 x 4096, 11008 4000 and 3795; 12288 x
// 8192, 16384 8830 and 8340; 9000 x 1024, 8500 521 and 514; with shorter sums, 4096 x
// 4096, 11008 930 and 964.
constexpr int64_t kLongSums = 8192;
bool apart(const MmParams& a, const MmParams& b) {
  const int64_t wave = kPlanSms / 2 * kMmTileN * 2 * kMmRows;
  return std::min(a.K, b.K) >= kLongSums && std::min(a.M * a.N, b.M * b.N) >= wave;
}

// The launch's tiles and their epilogues; partial: the room that the plan's splits
// need.
int products(MmEpilogue epilogue, MmLaunch* all, void* partial, void* stream) {
  const bool b_mn = epilogue == MM_OUT;
  Shape shape[2];
  int which[2], count = 0;
  for (int i = 0; i < 2; ++i) {
    const MmParams& p = all->p[i];
    if (p.M && p.N) {
      const int cycles = epilogue == MM_LSE ? epilogue_cycles(1)
                                            : epilogue_cycles(p.parts, p.accum_in || p.accum_out || p.base);
      shape[count] = {p.M, p.N, p.K, p.parts, p.b_halves != 0, cycles};
      which[count++] = i;
    }
  }
  if (!count) return VCOLL_OK;
  const Plan plan = make_plan(shape, count);
  all->error_word = device_error_symbol();
  if (!all->error_word) return fail(VCOLL_ERR_CUDA, "the device error word has no address");
  int64_t units = 0, join_blocks = 0;
  for (int i = 0; i < count; ++i) {
    MmParams* p = &all->p[which[i]];
    const bool a_mn = which[i] == 1;
    p->tn = plan.of[i].tn;
    p->splits = plan.of[i].splits;
    p->partial = (float*)((char*)partial + (i ? align256(plan.of[0].bytes) : 0));
    p->tile_rows = kMmRows * plan.ctas;
    p->group = (uint32_t)(group_rows(p->K, p->parts) / p->tile_rows);
    const int64_t tiles_m = ceil_div(p->M, p->tile_rows), tiles_n = ceil_div(p->N, p->b_halves ? p->tn / 2 : p->tn);
    if (tiles_m > 0x3FFFFFFF / tiles_n)
      return fail(VCOLL_ERR_UNSUPPORTED, "%lld x %lld tiles are too many", (long long)tiles_m, (long long)tiles_n);
    p->tiles_m = (uint32_t)tiles_m;
    p->tiles_n = (uint32_t)tiles_n;
    p->units = (uint32_t)(tiles_m * tiles_n) * p->splits;
    units += p->units;
    p->warp_rows = 32;
    p->depth = (uint32_t)ceil_div(p->K, kMmDepth);
    p->chunk = p->parts > 2 ? kMmChunkParts : epilogue == MM_LSE ? (p->M > kMmRows ? kMmChunkLoss : kMmChunkFew) : kMmChunkBf16;
    p->a_rows = a_mn || plan.ctas == 2 ? kMmRows : (int)std::min<int64_t>(kMmRows, round_up(p->M, 8));
    all->stage_bytes = std::max(all->stage_bytes, (p->a_rows + p->tn / plan.ctas) * kMmDepth * 2);
    const bool second = p->b[1].p && !p->b_halves;
    if (!second) p->K1 = round_up(p->K, kMmDepth);
    if (p->K) {
      VCOLL_TRY(encode(&p->map_a, p->a, p->parts, a_mn ? kMmDepth : p->a_rows));
      const int box = b_mn ? kMmDepth : p->b_halves ? p->tn / 2 : p->tn / plan.ctas;
      const int parts = p->parts == 3 ? 3 : 1;
      VCOLL_TRY(encode(&p->map_b[0], p->b[0], parts, box));
      if (second || p->b_halves) VCOLL_TRY(encode(&p->map_b[1], p->b[1], parts, box));
    }
    if (p->splits > 1) {
      const int64_t chunks = epilogue == MM_LSE ? 1 : (p->b_halves ? p->tn / 2 : p->tn) / 32;
      p->join_blocks = (uint32_t)ceil_div(tiles_m * tiles_n * std::min<int64_t>(p->M, p->tile_rows) * chunks, 8);
      join_blocks += p->join_blocks;
    }
  }
  all->stages = std::min(kMmMaxStages, kMmStageRoom / all->stage_bytes);
  int sms = 0;
  VCOLL_TRY(device_sms(&sms));
  const uint32_t slots = (uint32_t)std::min<int64_t>(sms / plan.ctas, units), last = all->p[0].units % slots;
  if (count == 2 && last)
    all->ahead = std::min<uint32_t>((uint32_t)std::llround(plan.of[0].unit / plan.of[1].unit),
                                    all->p[1].units / (slots - last));
  VCOLL_TRY(launch_tiles(mm_kernel(epilogue, plan.ctas), (int64_t)plan.ctas * slots, plan.ctas, kMmThreads, kMmSmem,
                         all, stream));
  if (!join_blocks) return VCOLL_OK;
  return launch_grid(mm_join_splits_kernel(epilogue), join_blocks, 1, 256, 0, all, stream);
}

// Products of a few fp32 rows (mm_few.cu); b: fp32 where it lies.
bool wide_rows(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  return cols % 4 == 0 && rows_at_16(p, rows, ld, 4);
}

int few_product(MmEpilogue epilogue, MmLaunch* all, void* partial, void* stream) {
  MmParams* p = &all->p[0];
  if (!p->M || !p->N) return VCOLL_OK;
  const int rows = (int)p->M;
  p->warp_rows = rows;
  const bool second = p->b[1].p != nullptr;
  const bool wide = wide_rows(p->b[0].p, p->b[0].rows, p->b[0].cols, p->b[0].ld) &&
                    (!second || wide_rows(p->b[1].p, p->b[1].rows, p->b[1].cols, p->b[1].ld));
  const void* fn = mm_few_kernel(epilogue, rows, wide);
  if (epilogue != MM_OUT) {
    p->tn = 64;
    p->splits = 1;
    p->tiles_n = (uint32_t)ceil_div(p->N, epilogue == MM_GATED ? 32 : 64);
    return launch_grid(fn, p->tiles_n, 1, kMmFewThreads, 0, all, stream);
  }
  if (!second) p->K1 = p->K;
  p->tn = 128;
  p->splits = (uint32_t)few_splits(p->N, p->K);
  p->partial = (float*)partial;
  p->tile_rows = kMmRows;
  p->tiles_m = p->group = 1;
  p->tiles_n = (uint32_t)ceil_div(p->N, 128);
  p->join_blocks = (uint32_t)ceil_div((int64_t)p->tiles_n * p->M * 4, 8);
  VCOLL_TRY(launch_grid(fn, p->tiles_n, p->splits, kMmFewColThreads, 0, all, stream));
  return launch_grid(mm_join_splits_kernel(MM_OUT), p->join_blocks, 1, 256, 0, all, stream);
}

int few_outer(MmLaunch* all, void* stream) {
  MmParams* p = &all->p[1];
  const int64_t tiles = ceil_div(p->M, 64) * ceil_div(p->N, 128);
  if (!tiles) return VCOLL_OK;
  if (tiles > 0x7FFFFFFF) return fail(VCOLL_ERR_UNSUPPORTED, "%lld tiles are too many", (long long)tiles);
  const int64_t rows = p->M1 ? p->M2 : p->M;
  const bool wide = wide_rows(p->out, rows, p->N, p->out_ld) && (!p->out2 || wide_rows(p->out2, rows, p->N, p->out2_ld)) &&
                    (!p->base || wide_rows(p->base, rows, p->N, p->base_ld));
  return launch_grid(mm_few_outer_kernel(wide), tiles, 1, kMmFewColThreads, 0, all, stream);
}

// The launch's products on the units that suit them.
int run(MmEpilogue epilogue, bool few, MmLaunch* all, void* partial, void* stream) {
  if (!few && apart(all->p[0], all->p[1])) {
    MmLaunch first = *all;
    first.p[1].M = 0;
    all->p[0].M = 0;
    VCOLL_TRY(products(epilogue, &first, partial, stream));
  }
  if (!few) return products(epilogue, all, partial, stream);
  VCOLL_TRY(few_product(epilogue, all, partial, stream));
  return few_outer(all, stream);
}

// Whether two adjacent columns of every row can be moved at once.
bool in_pairs(const void* p, int64_t rows, int64_t ld, int dtype) {
  return (uint64_t)p % (2 * elem_size(dtype)) == 0 && (rows <= 1 || ld % 2 == 0);
}

// Matrices of more values than any memory holds: their bytes fit 64 bits.
constexpr double kMaxValues = 1125899906842624.0;  // 2^50
int check_area(int64_t rows, int64_t cols, const char* what) {
  if ((double)rows * (double)cols > kMaxValues)
    return fail(VCOLL_ERR_UNSUPPORTED, "%s: %lld x %lld values are too many", what, (long long)rows,
                (long long)cols);
  return VCOLL_OK;
}

int check_loss(int dtype, int index_type, int64_t N, int64_t V, int64_t D) {
  VCOLL_TRY(check_type(dtype, "dtype"));
  if (index_type != VCOLL_I32 && index_type != VCOLL_I64)
    return fail(VCOLL_ERR_INVALID_TYPE, "unknown index type %d", index_type);
  VCOLL_TRY(check_extent(N, "N"));
  VCOLL_TRY(check_extent(V, "V"));
  VCOLL_TRY(check_extent(D, "D", kMaxWidth));
  VCOLL_TRY(check_area(N, D, "x"));
  return check_area(V, D, "table");
}

int check_gated(int dtype, int activation, int64_t N, int64_t D, int64_t F) {
  VCOLL_TRY(check_type(dtype, "dtype"));
  if (activation != VCOLL_SILU && activation != VCOLL_GELU && activation != VCOLL_GELU_TANH)
    return fail(VCOLL_ERR_INVALID_OP, "unknown activation %d", activation);
  VCOLL_TRY(check_extent(N, "N"));
  VCOLL_TRY(check_extent(D, "D", kMaxWidth));
  VCOLL_TRY(check_extent(F, "F", kMaxWidth));
  VCOLL_TRY(check_area(N, D, "x"));
  VCOLL_TRY(check_area(N, F, "h"));
  return check_area(F, D, "w_gate");
}

// The workspace is there, is device memory, and overlaps no operand.
int check_room(Operand* ops, int n, void* workspace, size_t bytes, size_t need) {
  VCOLL_TRY(check_operands(ops, n));
  VCOLL_TRY(check_workspace(workspace, bytes, need));
  ops[n] = {"workspace", workspace, need ? 1 : 0, (int64_t)need, (int64_t)need, 1, true, nullptr};
  VCOLL_TRY(check_operands(ops, n + 1));
  if (!need) return VCOLL_OK;
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, workspace) != cudaSuccess) {
    (void)cudaGetLastError();
    a.type = cudaMemoryTypeUnregistered;
  }
  if (a.type != cudaMemoryTypeDevice)
    return fail(VCOLL_ERR_INVALID_ARG, "the workspace is not device memory");
  return VCOLL_OK;
}

}  // namespace

extern "C" {

size_t vcoll_cross_entropy_workspace_bytes(int64_t N, int64_t V, int64_t D, int dtype, int direct) {
  if (check_loss(dtype, VCOLL_I32, N, V, D) || !N) return 0;
  const size_t least = dtype == VCOLL_F32 ? 0 : loss_layout(N, V, D, dtype, true).bytes;
  return dtype == VCOLL_BF16 && direct ? least : std::max(least, loss_layout(N, V, D, dtype, false).bytes);
}

int vcoll_cross_entropy(const void* x, int64_t x_ld, const void* table, int64_t table_ld,
                        const void* targets, int index_type, int64_t N, int64_t V, int64_t D,
                        float* loss, float* lse, int dtype, void* workspace,
                        size_t workspace_bytes, void* stream) {
  VCOLL_TRY(check_loss(dtype, index_type, N, V, D));
  const int es = elem_size(dtype);
  Operand ops[6] = {{"x", x, N, D, x_ld, es, false, nullptr},
                    {"table", table, N ? V : 0, D, table_ld, es, false, nullptr},
                    {"targets", targets, N, 1, 1, index_type == VCOLL_I64 ? 8 : 4, false, nullptr},
                    {"loss", loss, N ? 1 : 0, N, N, 4, true, nullptr},
                    {"lse", lse, N ? 1 : 0, N, N, 4, true, nullptr}};
  VCOLL_TRY(check_operands(ops, 5));
  if (!N) return VCOLL_OK;
  const bool x_direct = lies_direct(x, N, D, x_ld, dtype), t_direct = lies_direct(table, V, D, table_ld, dtype);
  const LossLayout L = loss_layout(N, V, D, dtype, x_direct && t_direct);
  VCOLL_TRY(check_room(ops, 5, workspace, workspace_bytes, L.bytes));
  char* ws = (char*)workspace;
  const bool few = few_rows(N, dtype);
  MmLaunch all = {};
  MmParams& p = all.p[0];
  p.M = N;
  p.K = D;
  p.parts = parts_of(dtype);
  p.targets = targets;
  p.idx64 = index_type == VCOLL_I64;
  p.V = V;
  p.part = (float2*)(ws + L.part);
  p.picked = loss;
  MmJoinParams j = {};
  j.part = p.part;
  j.state = (float2*)(ws + L.state);
  j.targets = targets;
  j.idx64 = p.idx64;
  j.loss = loss;
  j.lse = lse;
  j.N = N;
  j.V = V;
  for (int64_t i = 0; i < L.pieces; ++i) {
    p.token0 = i * L.piece;
    p.N = std::min(L.piece, V - p.token0);
    Packer pack(dtype);
    if (i == 0) VCOLL_TRY(pack.add(x, N, D, x_ld, x_direct, ws + L.x, false, &p.a));
    VCOLL_TRY(pack.add((const char*)table + p.token0 * table_ld * es, p.N, D, table_ld, t_direct || few,
                       ws + L.table, false, &p.b[0]));
    VCOLL_TRY(pack.run(stream));
    VCOLL_TRY(run(MM_LSE, few, &all, ws + L.splits, stream));
    j.tiles = (int64_t)p.tiles_n * (few || p.splits > 1 || p.tn < 128 ? 1 : 2);
    p.join_blocks = 0;
    all.stage_bytes = 0;
    j.first = i == 0;
    j.last = i == L.pieces - 1;
    VCOLL_TRY(launch_grid(mm_join_kernel(), ceil_div(N, 32), 1, kMmJoinThreads, 0, &j, stream));
  }
  return VCOLL_OK;
}

size_t vcoll_cross_entropy_backward_workspace_bytes(int64_t N, int64_t V, int64_t D, int dtype,
                                                    int direct) {
  if (check_loss(dtype, VCOLL_I32, N, V, D)) return 0;
  const size_t least = dtype == VCOLL_F32 ? 0 : loss_grad_layout(N, V, D, dtype, true).bytes;
  return dtype == VCOLL_BF16 && direct ? least
                                       : std::max(least, loss_grad_layout(N, V, D, dtype, false).bytes);
}

int vcoll_cross_entropy_backward(const float* dloss, int64_t dloss_count, const void* x,
                                 int64_t x_ld, const void* table, int64_t table_ld,
                                 const void* targets, int index_type, const float* lse, int64_t N,
                                 int64_t V, int64_t D, void* dx, int64_t dx_ld, const void* base,
                                 int64_t base_ld, void* dtable, int64_t dtable_ld, int dtype,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  VCOLL_TRY(check_loss(dtype, index_type, N, V, D));
  if (dloss_count != N && dloss_count != 1)
    return fail(VCOLL_ERR_INVALID_ARG, "dloss_count = %lld is neither 1 nor N", (long long)dloss_count);
  const int es = elem_size(dtype);
  Operand ops[9] = {{"x", x, N, D, x_ld, es, false, nullptr},
                    {"table", table, N ? V : 0, D, table_ld, es, false, nullptr},
                    {"targets", targets, N, 1, 1, index_type == VCOLL_I64 ? 8 : 4, false, nullptr},
                    {"dloss", dloss, N ? 1 : 0, dloss_count, dloss_count, 4, false, nullptr},
                    {"lse", lse, N ? 1 : 0, N, N, 4, false, nullptr},
                    {"base", base, base && dtable ? V : 0, D, base_ld, es, false, nullptr},
                    {"dx", dx, dx ? N : 0, D, dx_ld, es, true, x},
                    {"dtable", dtable, dtable ? V : 0, D, dtable_ld, es, true, base}};
  VCOLL_TRY(check_operands(ops, 8));
  if (!D || (!dx && !dtable)) return VCOLL_OK;
  if (!N && base && base == dtable) return VCOLL_OK;
  const bool direct = lies_direct(table, N ? V : 0, D, table_ld, dtype);
  const LossGradLayout L = loss_grad_layout(N, V, D, dtype, direct);
  VCOLL_TRY(check_room(ops, 8, workspace, workspace_bytes, L.bytes));
  char* ws = (char*)workspace;
  const int parts = parts_of(dtype), idx64 = index_type == VCOLL_I64;
  const bool few = few_rows(N, dtype);
  float* scale = (float*)(ws + L.scale);
  const int64_t dloss_step = dloss_count == 1 ? 0 : 1, index_bytes = idx64 ? 8 : 4;
  MmOperand all_rows;  // x without the rows that do not count
  for (int64_t i = 0; i < L.pieces; ++i) {
    const int64_t v0 = i * L.piece, width = std::min(L.piece, V - v0);
    MmOperand tokens;
    Packer pack(dtype);
    pack.p.targets = targets;
    pack.p.idx64 = idx64;
    pack.p.V = V;
    if (i == 0) {
      pack.p.dloss = dloss;
      pack.p.dloss_step = dloss_step;
      pack.p.scale = scale;
      pack.p.N = N;
      VCOLL_TRY(pack.add(x, N, D, x_ld, false, ws + L.x, true, &all_rows));
    }
    VCOLL_TRY(pack.add((const char*)table + v0 * table_ld * es, N ? width : 0, D, table_ld, direct || few, ws + L.table,
                       false, &tokens));
    VCOLL_TRY(pack.run(stream));
    float* sums = (float*)(ws + L.table_accum);
    if (L.blocks > 1 && base && dtable) {
      MmWidenParams w = {};
      w.src = (const char*)base + v0 * base_ld * es;
      w.dst = sums;
      w.rows = width;
      w.cols = D;
      w.src_ld = base_ld;
      w.dst_ld = round_up(D, 2);
      w.src_f32 = dtype == VCOLL_F32;
      w.load16 = rows_at_16(w.src, width, base_ld, es);
      w.blocks = pass_blocks(width * ceil_div(D, 8));
      if (width) VCOLL_TRY(launch_grid(mm_widen_kernel(), w.blocks, 1, kPassThreads, 0, &w, stream));
    }
    for (int64_t b = 0; b < L.blocks; ++b) {
      const int64_t n0 = b * L.rows, n = std::min(L.rows, N - n0);
      const MmOperand error = operand(ws + L.error, n, width, L.error_ld, L.rows * L.error_ld);
      MmOperand rows = all_rows;
      rows.p = (const char*)rows.p + n0 * rows.ld * 2;
      rows.rows = n;
      MmLaunch all = {};
      MmParams& p = all.p[0];
      p.a = rows;
      p.b[0] = tokens;
      p.M = n;
      p.N = width;
      p.K = D;
      p.parts = parts;
      p.targets = (const char*)targets + n0 * index_bytes;
      p.idx64 = idx64;
      p.V = V;
      p.token0 = v0;
      p.dloss = dloss + n0 * dloss_step;
      p.dloss_step = dloss_step;
      p.lse = lse + n0;
      p.scale = scale;
      p.error = ws + L.error;
      p.error_ld = L.error_ld;
      p.error_plane = L.rows * L.error_ld;
      VCOLL_TRY(run(MM_ERROR, few, &all, ws + L.splits, stream));
      MmLaunch grads = {};  // of x and of the table
      if (dx) {
        MmParams& q = grads.p[0];
        q.a = error;
        q.b[0] = tokens;
        q.M = n;
        q.N = D;
        q.K = width;
        q.parts = parts;
        q.scale = scale;
        q.out = (char*)dx + n0 * dx_ld * es;
        q.out_pairs = in_pairs(q.out, N, dx_ld, dtype);
        q.out_ld = dx_ld;
        q.out_f32 = dtype == VCOLL_F32;
        q.accum_ld = round_up(D, 2);
        float* so_far = (float*)(ws + L.accum) + n0 * q.accum_ld;
        if (i > 0) q.accum_in = so_far;
        if (i < L.pieces - 1) q.accum_out = so_far;
      }
      if (dtable) {
        MmParams& q = grads.p[1];
        q.a = error;
        q.b[0] = rows;
        q.M = width;
        q.N = D;
        q.K = n;
        q.parts = parts;
        q.scale = scale;
        q.out = (char*)dtable + v0 * dtable_ld * es;
        q.out_ld = dtable_ld;
        q.out_pairs = in_pairs(q.out, V, dtable_ld, dtype);
        q.out_f32 = dtype == VCOLL_F32;
        if (L.blocks == 1 && base) {
          q.base = (const char*)base + v0 * base_ld * es;
          q.base_ld = base_ld;
          q.out_pairs = q.out_pairs && in_pairs(q.base, V, base_ld, dtype);
        }
        if (L.blocks > 1) {
          q.accum_ld = round_up(D, 2);
          q.accum_scaled = 1;
          if (b > 0 || base) q.accum_in = sums;
          if (b < L.blocks - 1) q.accum_out = sums;
        }
      }
      VCOLL_TRY(run(MM_OUT, few, &grads, ws + L.splits, stream));
    }
  }
  return VCOLL_OK;
}

size_t vcoll_gated_ff_workspace_bytes(int64_t N, int64_t D, int64_t F, int dtype, int direct) {
  if (check_gated(dtype, VCOLL_SILU, N, D, F)) return 0;
  return gated_layout(N, D, F, dtype, dtype == VCOLL_BF16 && direct, false).bytes;
}

int vcoll_gated_ff(const void* x, int64_t x_ld, const void* w_gate, int64_t w_gate_ld,
                   const void* w_up, int64_t w_up_ld, int activation, int64_t N, int64_t D,
                   int64_t F, void* h, int64_t h_ld, void* gate, int64_t gate_ld, void* up,
                   int64_t up_ld, int dtype, void* workspace, size_t workspace_bytes,
                   void* stream) {
  VCOLL_TRY(check_gated(dtype, activation, N, D, F));
  const int es = elem_size(dtype);
  const int64_t W = N ? F : 0;
  Operand ops[7] = {{"x", x, F ? N : 0, D, x_ld, es, false, nullptr},
                    {"w_gate", w_gate, W, D, w_gate_ld, es, false, nullptr},
                    {"w_up", w_up, W, D, w_up_ld, es, false, nullptr},
                    {"h", h, N, F, h_ld, es, true, nullptr},
                    {"gate", gate, gate ? N : 0, F, gate_ld, es, true, nullptr},
                    {"up", up, up ? N : 0, F, up_ld, es, true, nullptr}};
  VCOLL_TRY(check_operands(ops, 6));
  if (!N || !F) return VCOLL_OK;
  const bool x_direct = lies_direct(x, N, D, x_ld, dtype), g_direct = lies_direct(w_gate, F, D, w_gate_ld, dtype),
             u_direct = lies_direct(w_up, F, D, w_up_ld, dtype);
  const GatedLayout L = gated_layout(N, D, F, dtype, x_direct && g_direct && u_direct, false);
  VCOLL_TRY(check_room(ops, 6, workspace, workspace_bytes, L.bytes));
  char* ws = (char*)workspace;
  MmLaunch all = {};
  MmParams& p = all.p[0];
  Packer pack(dtype);
  VCOLL_TRY(pack.add(x, N, D, x_ld, x_direct, ws + L.x, false, &p.a));
  const bool few = few_rows(N, dtype);
  VCOLL_TRY(pack.add(w_gate, F, D, w_gate_ld, g_direct || few, ws + L.w_gate, false, &p.b[0]));
  VCOLL_TRY(pack.add(w_up, F, D, w_up_ld, u_direct || few, ws + L.w_up, false, &p.b[1]));
  VCOLL_TRY(pack.run(stream));
  p.M = N;
  p.N = F;
  p.K = D;
  p.parts = parts_of(dtype);
  p.b_halves = 1;
  p.out = h;
  p.out_ld = h_ld;
  p.out_f32 = dtype == VCOLL_F32;
  p.gate = gate;
  p.gate_ld = gate_ld;
  p.up = up;
  p.up_ld = up_ld;
  p.act = activation;
  p.out_pairs = in_pairs(h, N, h_ld, dtype) && (!gate || in_pairs(gate, N, gate_ld, dtype)) &&
                (!up || in_pairs(up, N, up_ld, dtype));
  return run(MM_GATED, few, &all, ws + L.splits, stream);
}

size_t vcoll_gated_ff_backward_workspace_bytes(int64_t N, int64_t D, int64_t F, int dtype,
                                               int direct) {
  if (check_gated(dtype, VCOLL_SILU, N, D, F)) return 0;
  return gated_layout(N, D, F, dtype, dtype == VCOLL_BF16 && direct, true).bytes;
}

int vcoll_gated_ff_backward(const void* dh, int64_t dh_ld, const void* x, int64_t x_ld,
                            const void* w_gate, int64_t w_gate_ld, const void* w_up,
                            int64_t w_up_ld, const void* gate, int64_t gate_ld, const void* up,
                            int64_t up_ld, int activation, int64_t N, int64_t D, int64_t F,
                            void* dx, int64_t dx_ld, void* dw_gate, int64_t dw_gate_ld,
                            void* dw_up, int64_t dw_up_ld, int dtype, void* workspace,
                            size_t workspace_bytes, void* stream) {
  VCOLL_TRY(check_gated(dtype, activation, N, D, F));
  const int es = elem_size(dtype);
  const bool weights = dw_gate || dw_up;
  Operand ops[10] = {{"dh", dh, N, F, dh_ld, es, false, nullptr},
                     {"x", x, weights && F ? N : 0, D, x_ld, es, false, nullptr},
                     {"w_gate", w_gate, dx && N ? F : 0, D, w_gate_ld, es, false, nullptr},
                     {"w_up", w_up, dx && N ? F : 0, D, w_up_ld, es, false, nullptr},
                     {"gate", gate, N, F, gate_ld, es, false, nullptr},
                     {"up", up, N, F, up_ld, es, false, nullptr},
                     {"dx", dx, dx ? N : 0, D, dx_ld, es, true, nullptr},
                     {"dw_gate", dw_gate, dw_gate ? F : 0, D, dw_gate_ld, es, true, nullptr},
                     {"dw_up", dw_up, dw_up ? F : 0, D, dw_up_ld, es, true, nullptr}};
  VCOLL_TRY(check_operands(ops, 9));
  if (!D || (!dx && !weights)) return VCOLL_OK;
  const bool x_direct = !weights || lies_direct(x, F ? N : 0, D, x_ld, dtype),
             g_direct = !dx || lies_direct(w_gate, N ? F : 0, D, w_gate_ld, dtype),
             u_direct = !dx || lies_direct(w_up, N ? F : 0, D, w_up_ld, dtype);
  const GatedLayout L = gated_layout(N, D, F, dtype, x_direct && g_direct && u_direct, true);
  VCOLL_TRY(check_room(ops, 9, workspace, workspace_bytes, L.bytes));
  char* ws = (char*)workspace;
  const int parts = grad_parts(N, F, dtype);
  const MmOperand grads = operand(ws + L.grads, N, 2 * L.half, 2 * L.half, N * 2 * L.half);
  const bool few = few_rows(N, dtype);
  MmOperand rows, gates, ups;
  Packer pack(dtype);
  if (weights) VCOLL_TRY(pack.add(x, F ? N : 0, D, x_ld, x_direct, ws + L.x, false, &rows));
  if (dx) {
    VCOLL_TRY(pack.add(w_gate, N ? F : 0, D, w_gate_ld, g_direct || few, ws + L.w_gate, false, &gates));
    VCOLL_TRY(pack.add(w_up, N ? F : 0, D, w_up_ld, u_direct || few, ws + L.w_up, false, &ups));
  }
  if (N && F) {
    MmGatedGradParams g = {};
    g.dh = dh;
    g.gate = gate;
    g.up = up;
    g.dst = ws + L.grads;
    g.N = N;
    g.F = F;
    g.dh_ld = dh_ld;
    g.gate_ld = gate_ld;
    g.up_ld = up_ld;
    g.dst_ld = 2 * L.half;
    g.half = L.half;
    g.plane = N * 2 * L.half;
    g.f32 = dtype == VCOLL_F32;
    g.parts = parts;
    g.load16 = rows_at_16(dh, N, dh_ld, es) && rows_at_16(gate, N, gate_ld, es) && rows_at_16(up, N, up_ld, es);
    g.blocks = pass_blocks(N * (L.half / 8));
    g.pack = pack.params();
    VCOLL_TRY(launch_grid(mm_gated_grad_kernel(activation), g.blocks + pack.blocks, 1, kPassThreads, 0, &g, stream));
  } else {
    VCOLL_TRY(pack.run(stream));
  }
  MmLaunch all = {};  // dx and the weights' gradients
  if (dx) {
    MmParams& p = all.p[0];
    p.a = grads;
    p.b[0] = gates;
    p.b[1] = ups;
    p.M = N;
    p.N = D;
    p.K = 2 * L.half;
    p.K1 = L.half;
    p.parts = parts;
    p.out = dx;
    p.out_ld = dx_ld;
    p.out_f32 = dtype == VCOLL_F32;
    p.out_pairs = in_pairs(dx, N, dx_ld, dtype);
  }
  if (weights) {  // both as one product, or the one that is wanted
    const bool both = dw_gate && dw_up;
    MmParams& p = all.p[1];
    p.a = grads;
    if (!both) {
      p.a.p = ws + L.grads + (dw_gate ? 0 : (size_t)L.half * 2);
      p.a.cols = L.half;
    }
    p.b[0] = rows;
    p.M = both ? 2 * L.half : F;
    p.N = D;
    p.K = N;
    p.parts = parts;
    p.out = dw_gate ? dw_gate : dw_up;
    p.out_ld = dw_gate ? dw_gate_ld : dw_up_ld;
    p.out_f32 = dtype == VCOLL_F32;
    p.out_pairs = in_pairs(p.out, F, p.out_ld, dtype);
    if (both) {
      p.out2 = dw_up;
      p.out2_ld = dw_up_ld;
      p.M1 = L.half;
      p.M2 = F;
      p.out_pairs = p.out_pairs && in_pairs(dw_up, F, dw_up_ld, dtype);
    }
  }
  return run(MM_OUT, few, &all, ws + L.splits, stream);
}

}  // extern "C"
