// Products of two matrices with the element-wise part of an operator as their
// epilogue (the loss against a vocabulary, the gated feed-forward block):
// parameters shared by the host entry points (products.cpp) and the kernels.
// Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "vcoll_internal.h"

namespace vcoll {

// What a tile of a product becomes.
enum MmEpilogue : int {
  MM_OUT = 0,    // stored, after what it is added to and its scale
  MM_LSE = 1,    // each row's maximum and sum of exponentials, and its target's logit
  MM_ERROR = 2,  // softmax minus one at the target, as bf16 parts
  MM_GATED = 3,  // act(gate) * up, and where they are kept gate and up
};

// An operand in bf16: rows x cols, cols adjacent, rows ld apart.  fp32 values
// stand as three such matrices ("parts", plane elements apart) that add up to
// them.  The product sums over the columns of an operand, or over its rows
// where it is taken transposed.
struct MmOperand {
  const void* p;
  int64_t rows, cols, ld, plane;
};

struct MmParams {
  CUtensorMap map_a, map_b[2];  // of a and b: columns, rows, parts
  MmOperand a, b[2];
  int64_t M, N;   // of a tile space: rows and columns of the result
  int64_t K;      // length of the sum
  int64_t K1;     // the sum's places from here on take b[1] (K: none)
  int parts;      // of each operand: 1, or 3 in six products; 2: of a alone
  uint32_t depth;  // steps of kMmDepth places
  int b_halves;   // the tile's columns are half b[0]'s and half b[1]'s (MM_GATED)
  int tn;         // columns of a tile
  uint32_t tiles_m, tiles_n;
  uint32_t group;     // rows of tiles that are taken column after column
  int tile_rows;      // 128, or 256 of a pair of CTAs
  int warp_rows;      // that a warp's epilogue has at most: 32, or all of a few
  int a_rows;         // of a stage's a: 128, or fewer where M is smaller
  uint32_t chunk;       // steps that the tensor cores sum before the sum is added in registers
  uint32_t splits;      // that a tile's sum is cut into
  uint32_t units;       // tiles times splits
  uint32_t join_blocks;  // CTAs of the splits' join
  float* partial;     // of splits: tiles x splits x min(M, rows of a tile) x tn
  // MM_OUT
  void* out;
  int64_t out_ld;
  void* out2;             // of the rows from M1 on (M1 = 0: none), M2 in each half
  int64_t out2_ld, M1, M2;
  const float* accum_in;  // fp32 sums so far, accum_ld apart
  float* accum_out;       // instead of out
  int64_t accum_ld;
  int accum_scaled;       // the sums so far hold scale (else out applies it); what is added to base begins with it
  const float* scale;     // one value, or NULL
  const void* base;       // of out's type and stride base_ld
  int64_t base_ld;
  int out_f32;
  int out_pairs;          // two adjacent columns can be moved at once
  // MM_LSE, MM_ERROR: column j is token token0 + j of V
  const void* targets;
  const float* dloss;
  int64_t dloss_step;  // 0 or 1
  const float* lse;
  float2* part;        // 2 tiles_n x M: of each half of a tile's columns
  float* picked;       // M: the target's logit
  int64_t token0, V;
  int idx64;
  // MM_ERROR: bf16 parts; MM_GATED: out is h
  void* error;
  int64_t error_ld, error_plane;
  void *gate, *up;
  int64_t gate_ld, up_ld;
  int act;
};

// One launch.  p[0]: the product.  With MM_OUT, which takes b transposed, p[1] is
// another, independent one, which takes a transposed too, and the tiles of both
// fill the GPU together; either may be absent (units 0).  The CTAs (or pairs) take
// p[0]'s units in turn; those that have one fewer of them take `ahead` of p[1]'s
// before all take the rest in turn.
struct MmLaunch {
  MmParams p[2];
  int stages, stage_bytes;
  uint32_t ahead;
  unsigned* error_word;
};

// The six products of three parts that reach an fp32 result's precision, the
// small ones first: parts 0 and 2, 2 and 0, 1 and 1, 0 and 1, 1 and 0, 0 and 0.
VCOLL_HD constexpr int mm_pairs(int parts) { return parts == 3 ? 6 : parts; }
VCOLL_HD constexpr int mm_pair_a(int pairs, int q) { return pairs < 6 ? pairs - 1 - q : (0x010120 >> (4 * q)) & 15; }
VCOLL_HD constexpr int mm_pair_b(int pairs, int q) { return pairs < 6 ? 0 : (0x001102 >> (4 * q)) & 15; }

// Geometry of the tiles.  A CTA has 128 rows of a tile and at most 256 columns;
// one CTA, or two that share their columns' operand, take a tile.  64 places of
// the sum (128 bytes of a row) at a time, in stages of shared memory.
constexpr int kMmRows = 128;
// The tensor cores cut off where they add to an accumulator (its last bit, towards
// zero: a drift, not noise), so a long sum is taken out of them in chunks of steps
// and added in registers.  Relative errors of the loss over 4096 columns: 2.9e-6
// without, 6.9e-7 in chunks of 1024 places, 3.2e-7 of 512, which took 5 % longer; of
// fp32 adders 6.6e-7.
// Rows of one tile wait for memory anyway: their loss takes chunks of 128 places (7 rows
// of 32000 x 4096: 5.3e-8 off in 48 us, 1.2e-7 in chunks of 256, 49.4 us in chunks of 64).
// Of three parts' products only the last and largest is cut, after 256 places: 777 x
// 1001 x 2671 is off by 2.3e-7 (fp32 adders 5.7e-7), after 512 by 4.7e-7 and after 128 by
// 1.3e-7; the smallest gradient of the loss took 87 us, 85.5 and 89, others the same.
// What is rounded to bf16 in the end may drift by 3e-5 in 32768 places, a hundredth
// of that rounding (the gated block of 4096 columns by 4e-6: of its results one in 400
// is rounded to the other neighbour).
constexpr uint32_t kMmChunkLoss = 16, kMmChunkFew = 2, kMmChunkParts = 4, kMmChunkBf16 = 512;
constexpr uint32_t kMmChunkMost = 1 << 16;  // some 20 ms, far below what a wait may take
constexpr int kMmTileN = 256;
constexpr int kMmDepth = 64;
constexpr int kMmStageRoom = 192 * 1024;
constexpr int kMmMaxStages = 12;
constexpr int kMmEpilogueWarps = 8;  // four for the 128 rows, twice: each takes half of the columns
constexpr int kMmThreads = (kMmEpilogueWarps + 2) * 32;
constexpr int kMmPitch = 33;  // words of a row of a warp's block of 32 x 32
constexpr int kMmBlockWords = 32 * kMmPitch;
constexpr int kMmEpilogueBytes = kMmEpilogueWarps * kMmBlockWords * 4;
constexpr int kMmSmem = kMmStageRoom + kMmEpilogueBytes + 512 + 1024;

// A matrix laid out as bf16 parts, masked rows as zeros.
struct MmPackJob {
  const void* src;
  void* dst;
  int64_t rows, cols, src_ld, dst_ld, plane;
  int64_t first_block, blocks;
  int masked;
  int load16;  // rows start at 16-byte boundaries
};
// Up to three matrices; and where targets are given the largest magnitude of
// dloss over the rows that count (block 0).
constexpr int kMmPackJobs = 3;
struct MmPackParams {
  MmPackJob job[kMmPackJobs];
  const void* targets;
  const float* dloss;
  int64_t dloss_step;
  float* scale;  // NULL: not wanted
  int64_t N, V;
  int idx64, src_f32, parts;
};

// A matrix widened to fp32, its rows dst_ld apart.
struct MmWidenParams {
  const void* src;
  float* dst;
  int64_t rows, cols, src_ld, dst_ld;
  int src_f32;
  int load16;  // rows start at 16-byte boundaries
  int64_t blocks;
};

// Joins the tiles' maxima and sums of a piece of the vocabulary to those of
// the pieces before, and after the last gives the loss.
struct MmJoinParams {
  const float2* part;  // tiles x N
  float2* state;       // N: of the pieces before
  const void* targets;
  float *loss, *lse;
  int64_t tiles, N, V;
  int idx64, first, last;
};
constexpr int kMmJoinThreads = 1024;

// The gradients of gate and up, as bf16 parts beside each other.
struct MmGatedGradParams {
  const void *dh, *gate, *up;
  void* dst;
  int64_t N, F, dh_ld, gate_ld, up_ld;
  int64_t dst_ld, half, plane;  // gate's at 0, up's at half
  int f32, parts;
  int load16;  // the rows of dh, gate and up start at 16-byte boundaries
  int64_t blocks;     // CTAs; those after them lay out matrices
  MmPackParams pack;
};

// mm_few.cu: fp32 rows that it takes at most.
constexpr int kMmFewRows = 16;
constexpr int kMmFewThreads = 512;
constexpr int kMmFewColThreads = 256;

// ctas that share a tile: 1 or 2
const void* mm_kernel(MmEpilogue epilogue, int ctas);
const void* mm_join_splits_kernel(MmEpilogue epilogue);
const void* mm_few_kernel(MmEpilogue epilogue, int rows, bool wide);  // MM_OUT: sums for the join
const void* mm_few_outer_kernel(bool wide);
const void* mm_pack_kernel();
const void* mm_widen_kernel();
const void* mm_join_kernel();
const void* mm_gated_grad_kernel(int act);

// Launch of clusters of `cluster` CTAs, one CTA per SM, that take nearly all of
// its shared memory.
int launch_tiles(const void* fn, int64_t grid, int cluster, int threads, size_t smem, void* params,
                 void* stream);

}  // namespace vcoll
