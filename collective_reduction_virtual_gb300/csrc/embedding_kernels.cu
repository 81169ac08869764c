// Embedding lookup and its gradient.
#include "device_common.cuh"
#include "layers_internal.h"
#include "norm_common.cuh"
#include "row_access.cuh"

namespace vcoll {

// A warp takes a piece of a row, all of its accesses in flight: 2 KB in accesses
// of 16 bytes, fewer in narrower ones, so that no lane waits for columns that a
// narrow row does not have.  Bound by HBM: 65536 rows of 4096 bf16 out of 128000,
// 113 us, 6.3 TB/s of rows met and written.
template <typename T, int A>
__global__ void __launch_bounds__(kRowThreads) vc_embed(const __grid_constant__ EmbedParams p) {
  pdl_enter();
  constexpr int G = lookup_accesses(A, kLane<T>);
  const RowPiece piece((int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5), p.pieces);
  if (piece.row >= p.N) return;
  const int64_t t = token_at(p.tokens, p.idx64, piece.row);
  const bool inside = t >= 0 && t < p.V;
  const float scale = inside ? p.scale : 0.0f;  // zeros whatever p.scale is
  const int64_t c0 = piece.piece * (G * 32 * A) + (threadIdx.x & 31) * A;
  const char* from = elem_at<T>(p.table, (inside ? t * p.table_ld : 0) + c0);
  char* to = elem_at<T>(p.out, piece.row * p.out_ld + c0);
  Raw<T, A> r[G];
#pragma unroll
  for (int j = 0; j < G; ++j) {
    if (inside && c0 + j * 32 * A < p.D) r[j].load(elem_at<T>(from, j * 32 * A));
    else r[j].zero();
  }
#pragma unroll
  for (int j = 0; j < G; ++j) {
    if (c0 + j * 32 * A >= p.D) break;
    float f[A];
    r[j].widen(f);
#pragma unroll
    for (int a = 0; a < A; ++a) f[a] = __fmul_rn(f[a], scale);
    Raw<T, A> o;
    o.narrow(f);
    o.store_stream(elem_at<T>(to, j * 32 * A));
  }
}

// Narrow rows, kNarrowRows of each group of G lanes in flight (200000 x 128 bf16:
// 10 us, 5.8 TB/s; a warp per row took 29).
template <typename T, int A, int G>
__global__ void __launch_bounds__(kRowThreads) vc_embed_narrow(const __grid_constant__ EmbedParams p) {
  pdl_enter();
  const Group<T, A, G> g;
  constexpr int E = kLane<T>, U = kNarrowRows, S = 32 / G;
  const int D = (int)p.D;
  const int64_t first = ((int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5)) * (U * S) + g.sub;
  int64_t t[U];
#pragma unroll
  for (int u = 0; u < U; ++u) t[u] = first + u * S < p.N ? token_at(p.tokens, p.idx64, first + u * S) : -1;
  uint4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool inside = t[u] >= 0 && t[u] < p.V;
    raw[u] = g.load(elem_at<T>(p.table, inside ? t[u] * p.table_ld : 0), D, inside);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (first + u * S >= p.N) return;
    const float scale = t[u] >= 0 && t[u] < p.V ? p.scale : 0.0f;  // zeros whatever p.scale is
    float f[E];
    Elem<T>::widen(raw[u], f);
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = __fmul_rn(f[e], scale);
    g.store(elem_at<T>(p.out, (first + u * S) * p.out_ld), D, f);
  }
}

// --------------------------------------------------- rows of absent tokens
// Every token of the list leaves its position in stamp[token] (one of them
// stays, whichever).  A row's token occurs if and only if the position that
// its stamp names holds it, so the stamps need no clearing beforehand: what an
// older call or nobody wrote there does not pass.

namespace {

__device__ __forceinline__ void put_stamp(const EmbedGradParams& p, uint32_t key, uint32_t i) {
  if (key < (uint32_t)p.V) p.stamp[key] = i;
}

// One warp writes base or zeros to the bytes begin .. end - 1 of those of
// kFillRows adjacent rows whose tokens do not occur, eight accesses per lane in
// flight.  BYTES: of an access.
template <int BYTES>
__device__ __forceinline__ void fill_pieces(const EmbedGradParams& p, int64_t v, int64_t begin, int64_t end) {
  using P = Raw<float, BYTES / 4>;
  const char* from = static_cast<const char*>(p.base) + v * p.base_ld * p.table_es;
  char* to = static_cast<char*>(p.out) + v * p.out_ld * p.table_es;
  for (int64_t c0 = begin + (threadIdx.x & 31) * BYTES; c0 < end; c0 += 8 * 32 * BYTES) {
    P r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (p.base && c0 + k * 32 * BYTES < end) r[k].load_stream(from + c0 + k * 32 * BYTES);
      else r[k].zero();
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c0 + k * 32 * BYTES < end) r[k].store_stream(to + c0 + k * 32 * BYTES);
  }
}
// two-byte pieces: rows of bf16 at odd places
__device__ __forceinline__ void fill_halves(const EmbedGradParams& p, int64_t v, int64_t begin, int64_t end) {
  using P = Raw<__nv_bfloat16, 1>;
  const char* from = elem_at<__nv_bfloat16>(p.base, v * p.base_ld);
  char* to = elem_at<__nv_bfloat16>(p.out, v * p.out_ld);
  for (int64_t c0 = begin + (threadIdx.x & 31) * 2; c0 < end; c0 += 8 * 32 * 2) {
    P r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (p.base && c0 + k * 64 < end) r[k].load_stream(from + c0 + k * 64);
      else r[k].zero();
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c0 + k * 64 < end) r[k].store_stream(to + c0 + k * 64);
  }
}

__device__ __forceinline__ void fill_row(const EmbedGradParams& p, int64_t row, int64_t begin, int64_t end) {
  if (p.fill_bytes == 16) fill_pieces<16>(p, row, begin, end);
  else if (p.fill_bytes == 4) fill_pieces<4>(p, row, begin, end);
  else fill_halves(p, row, begin, end);
}

// Unit: p.fill_piece bytes of kFillRows rows from p.fill_begin on.
__device__ __forceinline__ void fill_rows(const EmbedGradParams& p, int64_t unit) {
  const int lane = threadIdx.x & 31;
  const RowPiece at(unit, p.fill_pieces);
  const int64_t first = p.fill_begin + at.row * kFillRows, begin = at.piece * p.fill_piece;
  const int64_t end = min(begin + p.fill_piece, p.D * p.table_es);
  const int64_t v = first + lane;
  bool gone = lane < kFillRows && v < p.fill_end;
  if (gone && p.N) {
    const uint32_t i = p.stamp[v];
    gone = (int64_t)i >= p.N || token_at(p.tokens, p.idx64, i) != v;
  }
  for (uint32_t m = __ballot_sync(~0u, gone); m; m &= m - 1) fill_row(p, first + __ffs(m) - 1, begin, end);
}

}  // namespace

// ------------------------------------------------------ sorting the tokens
// Stable LSD radix sort of the tokens' (key, position) pairs.  A CTA sorts a
// tile of the array by one digit: each warp owns a contiguous part of the
// tile and counts its digits; the counts, scanned over warps and digits, give
// each warp its places; and it walks its part again in order, the lanes of one
// digit taking the next places (match) in lane order.  A pass moves little and is
// bound by its few round trips to L2: the whole gradient of 8 columns, which is
// the sort and three nearly empty launches, takes 20 us for 2048 tokens, 27 for
// 16384 and 62 for 262144 (of 128000).

namespace {

constexpr int kSortWarps = kSortThreads / 32;
constexpr int kStampPiece = 2048, kStampSlots = 8192;
static_assert((kStampPiece + kStampSlots) * 4 <= (1 << kSortMaxBits) * kSortWarps * 4, "shared memory");

__device__ __forceinline__ uint32_t sort_key(const EmbedGradParams& p, int pass, int64_t i) {
  if (pass) return p.key[(pass + 1) & 1][i];
  const int64_t t = token_at(p.tokens, p.idx64, i);
  return t >= 0 && t < p.V ? (uint32_t)t : (uint32_t)p.V;
}

// The part of [lo, hi) that this warp owns.
struct WarpPart {
  int64_t lo, hi;
};
__device__ __forceinline__ WarpPart warp_part(int64_t lo, int64_t hi) {
  const int64_t per = ((hi - lo + kSortWarps - 1) / kSortWarps + 31) & ~(int64_t)31;
  WarpPart w;
  w.lo = lo + (threadIdx.x >> 5) * per;
  w.lo = w.lo < hi ? w.lo : hi;
  w.hi = w.lo + per < hi ? w.lo + per : hi;
  return w;
}

// count[warp][digit] of the warps' parts.
__device__ __forceinline__ void count_digits(const EmbedGradParams& p, int pass, int64_t lo,
                                             int64_t hi, uint32_t* count) {
  const int bins = 1 << p.bits, shift = pass * p.bits;
  for (int b = threadIdx.x; b < bins * kSortWarps; b += kSortThreads) count[b] = 0;
  __syncthreads();
  const WarpPart w = warp_part(lo, hi);
  uint32_t* mine = count + (threadIdx.x >> 5) * bins;
  for (int64_t i = w.lo + (threadIdx.x & 31); i < w.hi; i += 32)
    atomicAdd(&mine[(sort_key(p, pass, i) >> shift) & (bins - 1)], 1u);
  __syncthreads();
}

// Exclusive sum over the threads of the CTA.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* wsum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t u = __shfl_up_sync(~0u, inc, d);
    if (lane >= d) inc += u;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  uint32_t before = lane < warp ? wsum[lane] : 0u;
  before = __reduce_add_sync(~0u, before);
  __syncthreads();
  return before + inc - v;
}

// Turns count[warp][digit] into each warp's first place for each digit;
// thread d holds `first`, the tile's first place for digit d.
__device__ __forceinline__ void place_warps(int bins, uint32_t first, uint32_t* count) {
  if ((int)threadIdx.x < bins)
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t c = count[w * bins + threadIdx.x];
      count[w * bins + threadIdx.x] = first;
      first += c;
    }
  __syncthreads();
}

// Writes the tile's pairs to their places; each(key, place) sees every one.
template <typename F>
__device__ __forceinline__ void scatter_tile(const EmbedGradParams& p, int pass, int64_t lo,
                                             int64_t hi, uint32_t* count, F each) {
  const int bins = 1 << p.bits, shift = pass * p.bits, lane = threadIdx.x & 31;
  const uint32_t* pos = p.pos[(pass + 1) & 1];
  uint32_t* okey = p.key[pass & 1];
  uint32_t* opos = p.pos[pass & 1];
  uint32_t* next = count + (threadIdx.x >> 5) * bins;
  const WarpPart w = warp_part(lo, hi);
  for (int64_t i0 = w.lo; i0 < w.hi; i0 += 32) {
    const int64_t i = i0 + lane;
    const bool in = i < w.hi;
    const uint32_t k = in ? sort_key(p, pass, i) : 0u;
    const uint32_t from = in ? (pass ? pos[i] : (uint32_t)i) : 0u;
    const uint32_t digit = (k >> shift) & (bins - 1);
    const uint32_t same = __match_any_sync(~0u, in ? digit : 0xFFFFFFFFu);
    const uint32_t before = __popc(same & ((1u << lane) - 1));
    const uint32_t at = in ? next[digit] + before : 0u;
    __syncwarp();
    if (in && before == 0) next[digit] += __popc(same);
    __syncwarp();
    if (in) {
      okey[at] = k;
      opos[at] = from;
      each(k, at, from);
    }
  }
}

}  // namespace

// The whole sort in one CTA.
__global__ void __launch_bounds__(kSortThreads) vc_embed_sort(const __grid_constant__ EmbedGradParams p) {
  pdl_enter();
  extern __shared__ uint32_t count[];  // [warp][digit]
  __shared__ uint32_t wsum[kSortWarps];
  const int bins = 1 << p.bits;
  for (int pass = 0; pass < p.passes; ++pass) {
    count_digits(p, pass, 0, p.N, count);
    uint32_t total = 0;
    if ((int)threadIdx.x < bins)
      for (int w = 0; w < kSortWarps; ++w) total += count[w * bins + threadIdx.x];
    place_warps(bins, block_scan(total, wsum), count);
    scatter_tile(p, pass, 0, p.N, count, [&](uint32_t k, uint32_t, uint32_t i) {
      if (pass == 0) put_stamp(p, k, i);
    });
    __syncthreads();
  }
}

// Rows of the gradient on their way to L2 while the sort takes its time: every
// row is read by the sums that follow.  A lane asks for kPrefetchLines lines of
// 128 bytes, those of p.row_lines a row.
__device__ __forceinline__ void prefetch_rows(const EmbedGradParams& p, int64_t cta) {
  const int64_t first = p.line_begin + cta * (kSortThreads * kPrefetchLines) + threadIdx.x;
#pragma unroll
  for (int k = 0; k < kPrefetchLines; ++k) {
    const int64_t line = first + k * kSortThreads;
    if (line >= p.line_end) return;
    const RowPiece at(line, p.row_lines);
    const int64_t byte = min(at.piece * 128, p.D * p.grad_es - 1);
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(p.grad) + at.row * p.grad_ld * p.grad_es + byte));
  }
}

// The sort in one launch per pass, a CTA per tile, after one that counts the
// first digit.  cnt[pass][tile][digit] are the tiles' counts.
__global__ void __launch_bounds__(kSortThreads) vc_embed_count(const __grid_constant__ EmbedGradParams p) {
  pdl_enter();
  extern __shared__ uint32_t count[];
  const int bins = 1 << p.bits;
  if ((int)blockIdx.x >= p.sort_tiles) {
    prefetch_rows(p, (int64_t)blockIdx.x - p.sort_tiles);
    return;
  }
  const int64_t lo = (int64_t)blockIdx.x * p.sort_tile;
  const int64_t hi = lo + p.sort_tile < p.N ? lo + p.sort_tile : p.N;
  const size_t matrix = (size_t)p.sort_tiles * bins;
  for (int b = threadIdx.x; b < bins * (p.passes - 1); b += kSortThreads)
    p.cnt[(size_t)(1 + b / bins) * matrix + (size_t)blockIdx.x * bins + b % bins] = 0;
  // one stamp for each token of a tile's piece: as many stores to a frequent
  // token's stamp as it has places would wait for one another (21 us instead
  // of 6 at 262144 tokens spread as in text)
  uint32_t* skey = count;
  uint32_t* slot = count + kStampPiece;
  for (int64_t i0 = lo; i0 < hi; i0 += kStampPiece) {
    const int n = (int)(hi - i0 < kStampPiece ? hi - i0 : kStampPiece);
    for (int i = threadIdx.x; i < n; i += kSortThreads) {
      const uint32_t k = sort_key(p, 0, i0 + i);
      skey[i] = k;
      slot[k & (kStampSlots - 1)] = i;  // one of those that share the slot stays
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kSortThreads) {
      const uint32_t k = skey[i], in = slot[k & (kStampSlots - 1)];
      if ((int)in == i || skey[in] != k) put_stamp(p, k, (uint32_t)(i0 + i));
    }
    __syncthreads();
  }
  count_digits(p, 0, lo, hi, count);
  if ((int)threadIdx.x < bins) {
    uint32_t total = 0;
    for (int w = 0; w < kSortWarps; ++w) total += count[w * bins + threadIdx.x];
    p.cnt[(size_t)blockIdx.x * bins + threadIdx.x] = total;
  }
}

// One pass: the tile's first place for digit d is what all tiles have below d
// and the tiles before it have at d.  Every CTA sums the matrix of counts for
// itself (it is read from L2), which saves a launch; the next pass's counts
// are collected on the way, each pair's at the tile where it lands.  A pass
// takes a few microseconds and hardly any bandwidth, so CTAs behind the tiles'
// fill rows of absent tokens meanwhile, or fetch rows of the gradient to L2.
__global__ void __launch_bounds__(kSortThreads)
    vc_embed_scatter(const __grid_constant__ EmbedGradParams p) {
  pdl_enter();
  extern __shared__ uint32_t count[];
  __shared__ uint32_t wsum[kSortWarps];
  __shared__ uint32_t sall[kSortThreads], sbefore[kSortThreads];
  const int pass = p.pass, bins = 1 << p.bits, tiles = p.sort_tiles;
  if ((int)blockIdx.x >= tiles + p.fill_ctas) {
    prefetch_rows(p, (int64_t)blockIdx.x - tiles - p.fill_ctas);
    return;
  }
  if ((int)blockIdx.x >= tiles) {
    fill_rows(p, (int64_t)(blockIdx.x - tiles) * kSortWarps + (threadIdx.x >> 5));
    return;
  }
  const uint32_t* cnt = p.cnt + (size_t)pass * tiles * bins;
  const int64_t lo = (int64_t)blockIdx.x * p.sort_tile;
  const int64_t hi = lo + p.sort_tile < p.N ? lo + p.sort_tile : p.N;
  // kSortThreads / bins groups of threads share the tiles
  const int digit = threadIdx.x & (bins - 1), group = threadIdx.x >> p.bits;
  const int groups = kSortThreads >> p.bits;
  uint32_t all = 0, before = 0;
#pragma unroll 16
  for (int t = group; t < tiles; t += groups) {
    const uint32_t c = cnt[(size_t)t * bins + digit];
    all += c;
    before += t < (int)blockIdx.x ? c : 0u;
  }
  sall[threadIdx.x] = all;
  sbefore[threadIdx.x] = before;
  count_digits(p, pass, lo, hi, count);
  all = before = 0;
  if ((int)threadIdx.x < bins)
    for (int g = 0; g < groups; ++g) {
      all += sall[g * bins + threadIdx.x];
      before += sbefore[g * bins + threadIdx.x];
    }
  place_warps(bins, block_scan(all, wsum) + before, count);
  if (pass + 1 < p.passes) {
    uint32_t* next = p.cnt + (size_t)(pass + 1) * tiles * bins;
    const int shift = (pass + 1) * p.bits;
    scatter_tile(p, pass, lo, hi, count, [&](uint32_t k, uint32_t at, uint32_t) {
      atomicAdd(&next[(size_t)(at / (uint32_t)p.sort_tile) * bins + ((k >> shift) & (bins - 1))], 1u);
    });
  } else {
    scatter_tile(p, pass, lo, hi, count, [](uint32_t, uint32_t, uint32_t) {});
  }
}

// --------------------------------------------------- summing the sorted rows
// The sorted list is cut into chunks of p.chunk places, and a warp sums one
// chunk's rows over one tile of 32 * E columns, eight rows' loads in flight.
// A token whose places lie inside the chunk is written at once; the sum of one
// that began in an earlier chunk goes to the chunk's first partial row (fp32),
// of one that goes on in the next to its second, and vc_embed_join adds these
// up in order.  The work is even however the tokens are spread.  Bound by HBM:
// 262144 rows of 4096 bf16 into 128000, spread as in text, 480 us, 5.9 TB/s with
// the fill; rows of odd width, in 4-byte accesses, 4 to 5 TB/s.

namespace {

template <typename T, typename TO, int A>
struct GradTile {
  static constexpr int E = kLane<T>;
  const EmbedGradParams& p;
  int lane;
  int64_t col0;  // first column of the tile

  __device__ __forceinline__ int64_t col(int j) const { return col0 + (j * 32 + lane) * A; }

  // The lane's columns of the row at element `at` of a matrix.  Two-byte pieces,
  // of which there are eight, are loaded without branches: past the row's end a
  // lane takes the last column, whose sum it drops (50021 x 1001 bf16 in place in
  // 49999 rows: 124 us, 226 with branches).
  template <typename M>
  __device__ __forceinline__ void load(const void* rows, int64_t at, Raw<M, A> (&r)[E / A]) const {
    if constexpr (E / A == 8) {
      const int64_t c = min(col(0), p.D - 1);
      const int left = (int)min(p.D - 1 - c, (int64_t)(7 * 32));
      const char* from = elem_at<M>(rows, at + c);
#pragma unroll
      for (int j = 0; j < E / A; ++j) r[j].load_stream(from + min(j * 32, left) * Elem<M>::kBytes);
    } else {
#pragma unroll
      for (int j = 0; j < E / A; ++j) {
        if (col(j) < p.D) r[j].load_stream(elem_at<M>(rows, at + col(j)));
        else r[j].zero();
      }
    }
  }
  // base[v] of the lane's columns, zeros where there is no base
  __device__ __forceinline__ void load_base(int64_t v, Raw<TO, A> (&b)[E / A]) const {
    if (p.base) {
      load<TO>(p.base, v * p.base_ld, b);
    } else {
#pragma unroll
      for (int j = 0; j < E / A; ++j) b[j].zero();
    }
  }
  // table_grad[v] = base[v] + scale * sum
  __device__ __forceinline__ void finish(int64_t v, const float (&sum)[E], const Raw<TO, A> (&b)[E / A]) const {
#pragma unroll
    for (int j = 0; j < E / A; ++j) {
      if (col(j) >= p.D) continue;
      float f[A];
      b[j].widen(f);
#pragma unroll
      for (int a = 0; a < A; ++a)
        f[a] = p.base ? fmaf(sum[j * A + a], p.scale, f[a]) : __fmul_rn(sum[j * A + a], p.scale);
      Raw<TO, A> o;
      o.narrow(f);
      o.store_stream(elem_at<TO>(p.out, v * p.out_ld + col(j)));
    }
  }

  __device__ __forceinline__ float4* partial(int64_t chunk, int slot, int64_t tile) const {
    return reinterpret_cast<float4*>(p.part) + ((chunk * 2 + slot) * p.tiles + tile) * (32 * E / 4) + lane;
  }
  __device__ __forceinline__ void put(float4* at, const float (&sum)[E]) const {
#pragma unroll
    for (int k = 0; k < E; k += 4) at[k * 8] = make_float4(sum[k], sum[k + 1], sum[k + 2], sum[k + 3]);
  }
  __device__ __forceinline__ void add(const float4* at, float (&sum)[E]) const {
#pragma unroll
    for (int k = 0; k < E; k += 4) {
      const float4 v = at[k * 8];
      sum[k] += v.x;
      sum[k + 1] += v.y;
      sum[k + 2] += v.z;
      sum[k + 3] += v.w;
    }
  }
};

}  // namespace

// CTAs that stay on an SM: rows of 16-byte accesses and of two-byte ones take
// more registers (the latter 142 us with four, 124 with three).  With a base,
// whose rows are in flight as well, two-byte ones spill at three, too (about 280
// bytes a thread), and bf16 pairs into fp32 at four (144).
constexpr int grad_ctas(int A, int E) { return A == E || E / A == 8 ? 3 : 4; }

// BASE: there is a base, whose rows are fetched with the rows that end a
// token's sum; half as many rows are in flight then.
template <typename T, typename TO, int A, bool BASE>
__global__ void __launch_bounds__(kRowThreads, grad_ctas(A, kLane<T>))
    vc_embed_grad(const __grid_constant__ EmbedGradParams p) {
  pdl_enter();
  constexpr int E = kLane<T>;
  constexpr int U = BASE || (A == 1 && E == 8) ? 4 : 8;  // rows in flight
  const uint32_t* key = p.key[(p.passes + 1) & 1];
  const uint32_t* pos = p.pos[(p.passes + 1) & 1];
  // the CTAs that fill are spread evenly among those that sum, so that reads
  // and writes mix
  const int64_t fills = (int64_t)gridDim.x - p.sum_ctas;
  const int64_t fill = (int64_t)blockIdx.x * fills / gridDim.x;
  if (((int64_t)blockIdx.x + 1) * fills / gridDim.x != fill) {
    fill_rows(p, fill * (kRowThreads / 32) + (threadIdx.x >> 5));
    return;
  }
  const int64_t unit = ((int64_t)blockIdx.x - fill) * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int64_t chunk = unit / p.tiles, tile = unit % p.tiles;
  const int64_t lo = chunk * p.chunk;
  if (lo >= p.N) return;
  const int64_t hi = lo + p.chunk < p.N ? lo + p.chunk : p.N;
  const GradTile<T, TO, A> g{p, (int)(threadIdx.x & 31), tile * 32 * E};
  const uint32_t none = (uint32_t)p.V;
  // 32 places at a time, one per lane, the next ones loaded ahead; tokens
  // outside the table sort last, so the valid lanes are the first ones
  int64_t at = lo + g.lane;
  uint32_t key_next = at < hi ? key[at] : none, pos_next = at < hi ? pos[at] : 0u;
  const uint32_t first = __shfl_sync(~0u, key_next, 0);
  if (first >= none) return;
  bool began = lo > 0 && key[lo - 1] == first;  // the first token began before this chunk
  const uint32_t after = hi < p.N ? key[hi] : none;  // a token that goes on after it
  float sum[E];
#pragma unroll
  for (int e = 0; e < E; ++e) sum[e] = 0.0f;
  for (int64_t k0 = lo; k0 < hi; k0 += 32) {
    const uint32_t k = key_next, from = pos_next;
    at += 32;
    key_next = at < hi ? key[at] : none;
    pos_next = at < hi ? pos[at] : 0u;
    const int n = __popc(__ballot_sync(~0u, k < none));
    uint32_t next = __shfl_down_sync(~0u, k, 1);
    const uint32_t next32 = __shfl_sync(~0u, key_next, 0);
    if (g.lane == 31) next = next32;
    // places that end a token's sum in this chunk
    const uint32_t ends = __ballot_sync(~0u, k < none && next != k);
#pragma unroll 1
    for (int s = 0; s < n; s += U) {
      Raw<T, A> r[U][E / A];
      Raw<TO, A> b[BASE ? U : 1][E / A];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t row = (int64_t)__shfl_sync(~0u, from, s + u) * p.grad_ld;
        if (s + u < n) {
          g.template load<T>(p.grad, row, r[u]);
        } else {
#pragma unroll
          for (int j = 0; j < E / A; ++j) r[u][j].zero();
        }
      }
      if constexpr (BASE) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t v = __shfl_sync(~0u, k, s + u);
          if (ends >> (s + u) & 1) g.load_base(v, b[u]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < E / A; ++j) b[0][j].zero();
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int j = 0; j < E / A; ++j) {
          float f[A];
          r[u][j].widen(f);
#pragma unroll
          for (int a = 0; a < A; ++a) sum[j * A + a] += f[a];
        }
        if (ends >> (s + u) & 1) {
          const uint32_t v = __shfl_sync(~0u, k, s + u);
          if (began) g.put(g.partial(chunk, 0, tile), sum);
          else if (v == after) g.put(g.partial(chunk, 1, tile), sum);
          else g.finish(v, sum, b[BASE ? u : 0]);
          began = false;
#pragma unroll
          for (int e = 0; e < E; ++e) sum[e] = 0.0f;
        }
      }
    }
    if (n < 32) break;
  }
}

// A warp per (chunk, tile): if a token begins in the chunk and goes on after
// it, its sum is the chunk's second partial row and the first ones of the
// chunks that it reaches.  Tokens over more than kJoinAlone of them are added
// up by all warps of the CTA, each a contiguous part, then in warp order.  Bound
// by a handful of dependent loads, 10 to 20 us cold.
template <typename T, typename TO, int A>
__global__ void __launch_bounds__(kRowThreads) vc_embed_join(const __grid_constant__ EmbedGradParams p) {
  pdl_enter();
  constexpr int E = kLane<T>, NW = kRowThreads / 32;
  __shared__ int64_t last_of[NW];  // the last chunk of the warp's token, -1: nothing to do
  __shared__ float part[NW][32 * E];
  const uint32_t* key = p.key[(p.passes + 1) & 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if ((int64_t)blockIdx.x >= p.sum_ctas) {  // hardly any bandwidth is used here either
    fill_rows(p, ((int64_t)blockIdx.x - p.sum_ctas) * NW + warp);
    return;
  }
  // units a CTA apart: those of one chunk, which a long token makes long, go to
  // different CTAs
  const int64_t unit = (int64_t)warp * p.sum_ctas + blockIdx.x;
  const int64_t chunk = unit / p.tiles, tile = unit % p.tiles;
  const int64_t lo = chunk * p.chunk, hi = lo + p.chunk;
  int64_t last = -1;
  uint32_t v = 0;
  if (hi < p.N) {
    v = key[hi - 1];
    if (v < (uint32_t)p.V && key[hi] == v && !(lo > 0 && key[lo - 1] == v)) {
      // the last chunk that begins inside the token, 32 at a time
      uint32_t reach;
      last = chunk;
      do {
        const int64_t first = (last + 1 + lane) * p.chunk;
        reach = __popc(__ballot_sync(~0u, first < p.N && key[first] == v));
        last += reach;
      } while (reach == 32);
    }
  }
  const GradTile<T, TO, A> g{p, lane, tile * 32 * E};
  if (last >= 0 && last - chunk <= kJoinAlone) {
    float sum[E];
#pragma unroll
    for (int e = 0; e < E; ++e) sum[e] = 0.0f;
    g.add(g.partial(chunk, 1, tile), sum);
    for (int64_t c = chunk + 1; c <= last; ++c) g.add(g.partial(c, 0, tile), sum);
    Raw<TO, A> b[E / A];
    g.load_base(v, b);
    g.finish(v, sum, b);
    last = -1;
  }
  if (lane == 0) last_of[warp] = last;
  __syncthreads();
  for (int w = 0; w < NW; ++w) {
    const int64_t end = last_of[w];
    if (end < 0) continue;  // the same for the whole CTA
    const int64_t u = (int64_t)w * p.sum_ctas + blockIdx.x, from = u / p.tiles, t = u % p.tiles;
    const GradTile<T, TO, A> gw{p, lane, t * 32 * E};
    const int64_t per = (end - from + NW - 1) / NW;
    const int64_t a = from + 1 + warp * per, b = a + per < end + 1 ? a + per : end + 1;
    float sum[E];
#pragma unroll
    for (int e = 0; e < E; ++e) sum[e] = 0.0f;
    if (warp == 0) gw.add(gw.partial(from, 1, t), sum);
#pragma unroll 4
    for (int64_t c = a; c < b; ++c) gw.add(gw.partial(c, 0, t), sum);
#pragma unroll
    for (int e = 0; e < E; ++e) part[warp][e * 32 + lane] = sum[e];
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float s = part[0][e * 32 + lane];
        for (int k = 1; k < NW; ++k) s += part[k][e * 32 + lane];
        sum[e] = s;
      }
      const uint32_t token = key[(from + 1) * p.chunk - 1];
      Raw<TO, A> base[E / A];
      gw.load_base(token, base);
      gw.finish(token, sum, base);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------- short lists
// A short list is not sorted, one launch does all.  A warp per
// (place, tile of columns) reads the list: if an earlier place holds its token
// it has nothing to do, else it sums the rows of the places that hold it, in
// order.  Tokens of more than kSmallAlone places are summed by all warps of the
// CTA, an eighth of the list each, and joined in order.  CTAs behind these fill
// the rows of absent tokens, p.fill_each a CTA.

namespace {

// Adds up the rows of the places lo .. hi - 1 (lo a multiple of 32) that hold v.
template <typename T, typename TO, int A>
__device__ __forceinline__ void sum_places(const GradTile<T, TO, A>& g, const int32_t* list, int lo, int hi,
                                           int32_t v, float (&sum)[kLane<T>]) {
  constexpr int E = kLane<T>, U = A == 1 && E == 8 ? 4 : 8;
#pragma unroll
  for (int e = 0; e < E; ++e) sum[e] = 0.0f;
  for (int i = lo; i < hi; i += 32) {
    uint32_t same = __ballot_sync(~0u, i + g.lane < hi && list[i + g.lane] == v);
    while (same) {
      Raw<T, A> r[U][E / A];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (same) {
          g.template load<T>(g.p.grad, (int64_t)(i + __ffs(same) - 1) * g.p.grad_ld, r[u]);
        } else {
#pragma unroll
          for (int j = 0; j < E / A; ++j) r[u][j].zero();
        }
        same &= same - 1;
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < E / A; ++j) {
          float f[A];
          r[u][j].widen(f);
#pragma unroll
          for (int a = 0; a < A; ++a) sum[j * A + a] += f[a];
        }
    }
  }
}

}  // namespace

template <typename T, typename TO, int A>
__global__ void __launch_bounds__(kRowThreads) vc_embed_grad_small(const __grid_constant__ EmbedGradParams p) {
  pdl_enter();
  constexpr int E = kLane<T>, NW = kRowThreads / 32;
  __shared__ int32_t list[kSmallTokens];  // -1: outside the table
  __shared__ uint32_t met[2];  // of the CTA's rows, those whose tokens occur
  __shared__ int32_t shared_token[NW];  // -1: nothing left for the CTA to do
  __shared__ float part[NW][32 * E];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = (int)p.N;
  const bool fills = (int64_t)blockIdx.x >= p.sum_ctas;
  const int64_t first = ((int64_t)blockIdx.x - p.sum_ctas) * p.fill_each;
  if (threadIdx.x < 2) met[threadIdx.x] = 0u;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kRowThreads) {
    const int64_t t = token_at(p.tokens, p.idx64, i);
    list[i] = t >= 0 && t < p.V ? (int32_t)t : -1;
    if (fills && t >= first && t < first + p.fill_each) atomicOr(&met[(t - first) >> 5], 1u << ((t - first) & 31));
  }
  __syncthreads();
  if (fills) {
    for (int r = warp; r < p.fill_each && first + r < p.V; r += NW)
      if (!(met[r >> 5] >> (r & 31) & 1)) fill_row(p, first + r, 0, p.D * p.table_es);
    return;
  }
  // units a CTA apart: the tiles of a frequent token's place go to different
  // CTAs (512 places of one token, 4096 bf16 columns: 10 us; 56 us when a CTA
  // has eight of its tiles to add up in turn)
  auto unit_of = [&](int w) { return (int64_t)w * p.sum_ctas + blockIdx.x; };
  auto tile_of = [&](int w) { return GradTile<T, TO, A>{p, lane, unit_of(w) % p.tiles * 32 * E}; };
  const int64_t place = unit_of(warp) / p.tiles;
  int32_t v = place < n ? list[place] : -1;
  for (int i = 0; i < place && v >= 0; i += 32)
    if (__ballot_sync(~0u, i + lane < place && list[i + lane] == v)) v = -1;  // an earlier place holds it
  int count = 0;
  if (v >= 0)
    for (int i = (int)place & ~31; i < n; i += 32)
      count += __popc(__ballot_sync(~0u, i + lane < n && list[i + lane] == v));
  float sum[E];
  if (v >= 0 && count <= kSmallAlone) {
    const GradTile<T, TO, A> g = tile_of(warp);
    Raw<TO, A> base[E / A];
    g.load_base(v, base);
    sum_places(g, list, (int)place & ~31, n, v, sum);
    g.finish(v, sum, base);
    v = -1;
  }
  if (lane == 0) shared_token[warp] = v;
  __syncthreads();
  for (int w = 0; w < NW; ++w) {
    v = shared_token[w];
    if (v < 0) continue;  // the same for the whole CTA
    const GradTile<T, TO, A> g = tile_of(w);
    const int per = ((n + NW - 1) / NW + 31) & ~31;
    sum_places(g, list, warp * per, min(n, (warp + 1) * per), v, sum);
#pragma unroll
    for (int e = 0; e < E; ++e) part[warp][e * 32 + lane] = sum[e];
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        for (int k = 1; k < NW; ++k) sum[e] += part[k][e * 32 + lane];
      Raw<TO, A> base[E / A];
      g.load_base(v, base);
      g.finish(v, sum, base);
    }
    __syncthreads();
  }
}

namespace {
template <typename T>
const void* lookup_kernel(int access) {
  return access == kLane<T> ? (const void*)&vc_embed<T, kLane<T>>
         : access == 2      ? (const void*)&vc_embed<T, 2>
                            : (const void*)&vc_embed<T, 1>;
}
}  // namespace
namespace {
template <typename T, int A>
const void* lookup_narrow_kernel(int lanes) {
  return lanes == 8    ? (const void*)&vc_embed_narrow<T, A, 8>
         : lanes == 16 ? (const void*)&vc_embed_narrow<T, A, 16>
                       : (const void*)&vc_embed_narrow<T, A, 32>;
}
template <typename T>
const void* lookup_narrow_kernel(int access, int lanes) {
  return access == kLane<T> ? lookup_narrow_kernel<T, kLane<T>>(lanes)
         : access == 2      ? lookup_narrow_kernel<T, 2>(lanes)
                            : lookup_narrow_kernel<T, 1>(lanes);
}
}  // namespace
const void* embed_narrow_kernel(int dtype, int access, int lanes) {
  return dtype == VCOLL_F32 ? lookup_narrow_kernel<float>(access, lanes)
                            : lookup_narrow_kernel<__nv_bfloat16>(access, lanes);
}
const void* embed_kernel(int dtype, int access) {
  return dtype == VCOLL_F32 ? lookup_kernel<float>(access) : lookup_kernel<__nv_bfloat16>(access);
}
const void* embed_sort_kernel() { return (const void*)&vc_embed_sort; }
const void* embed_count_kernel() { return (const void*)&vc_embed_count; }
const void* embed_scatter_kernel() { return (const void*)&vc_embed_scatter; }

namespace {
template <typename T, typename TO, int A>
const void* grad_kernel(GradPart part) {
  switch (part) {
    case GRAD_SMALL: return (const void*)&vc_embed_grad_small<T, TO, A>;
    case GRAD_SUM: return (const void*)&vc_embed_grad<T, TO, A, false>;
    case GRAD_SUM_BASE: return (const void*)&vc_embed_grad<T, TO, A, true>;
    default: return (const void*)&vc_embed_join<T, TO, A>;
  }
}
template <typename T, typename TO>
const void* grad_kernel(int access, GradPart part) {
  return access == kLane<T> ? grad_kernel<T, TO, kLane<T>>(part)
         : access == 2      ? grad_kernel<T, TO, 2>(part)
                            : grad_kernel<T, TO, 1>(part);
}
}  // namespace

const void* embed_grad_kernel(int dtype, int table_dtype, int access, GradPart part) {
  using B = __nv_bfloat16;
  if (dtype == VCOLL_F32)
    return table_dtype == VCOLL_F32 ? grad_kernel<float, float>(access, part)
                                    : grad_kernel<float, B>(access, part);
  return table_dtype == VCOLL_F32 ? grad_kernel<B, float>(access, part)
                                  : grad_kernel<B, B>(access, part);
}

}  // namespace vcoll
