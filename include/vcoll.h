/*
 * vcoll.h -- C ABI of the virtual-rank collective library for one GB300 GPU.
 *
 * A "virtual rank" is one device buffer.  W ranks live in the HBM of the
 * current CUDA device; the collectives combine them element by element inside
 * single kernel launches.  There is no second GPU, peer access or NCCL.
 *
 * Common conventions for every entry point below
 * ------------------------------------------------
 *  - Pointer arrays (`in`, `out`, `tensors`, `fused`) are HOST arrays of
 *    DEVICE pointers on the current device.  Pinned host memory
 *    (cudaHostAlloc / cudaHostRegister) is accepted too: with unified
 *    addressing its host pointer is a device pointer, and the kernels then
 *    read and write it directly over the CPU-GPU link, which is faster than
 *    staging copies in and out.  Each device pointer must be
 *    aligned to the element size.  Any 16-byte phase works.  Reduce-scatter,
 *    allreduce and allgather use 16-byte vectors whenever their outputs share
 *    a phase (each reduce-scatter output on a grid of its own), realigning
 *    inputs at other phases on the fly; the other entry points when all their
 *    buffers share one.  Otherwise an element-wise path gives the same bits,
 *    more slowly.
 *  - `n` counts elements per rank (int64).  Segment j of an n-element buffer
 *    is [off_j, off_j + len_j) with q = n / W, r = n % W,
 *    off_j = j*q + min(j, r), len_j = q + (j < r): contiguous, the first r
 *    segments one element longer (vcoll_segment computes it).  When W divides
 *    n this is NCCL's layout (block j at j * recvcount).
 *  - Ownership: the caller owns every buffer; the library allocates no device
 *    memory and keeps no pointer after the call returns.
 *  - Streams: `stream` is a cudaStream_t passed as void* (NULL = the legacy
 *    default stream).  Work is enqueued asynchronously on it; nothing
 *    synchronises the host.
 *  - Errors: every call returns a vcoll_status_t.  Argument errors are found
 *    on the host before anything is enqueued.  vcoll_last_error() returns a
 *    thread-local message for the last failure on the calling thread.
 *  - Types: VCOLL_F32 and VCOLL_BF16.  Arithmetic is fp32 for both; bf16
 *    inputs are widened exactly and outputs rounded to nearest even once (a
 *    NaN keeps its sign and top payload bits and is made quiet: the
 *    canonical fp32 NaN becomes 0x7FC0).  Subnormals are kept (no flush to
 *    zero).
 *  - Ops: VCOLL_SUM, VCOLL_MAX, VCOLL_AVG (sum times fl32(1/W), applied once
 *    to the finished sum), VCOLL_MIN, VCOLL_PROD (one fp32 multiply per hop).
 *    max: a NaN operand gives the canonical quiet NaN; +0 wins over -0;
 *    otherwise the larger value.  min: the mirror image (-0 wins over +0).
 *  - Order: with VCOLL_FLAG_RING_ORDER each element of segment j is folded
 *    in ring order -- starting at rank (j+1) mod W, accumulator first, ending
 *    at rank j -- which reproduces the early NCCL ring bit for bit.  Without
 *    it the library uses its fastest order (a pairwise tree for W in
 *    {4, 8, 16}); results then differ from ring order only by float
 *    reassociation.  max and min are the same in every order.
 *  - Special cases: n == 0 returns VCOLL_OK without enqueuing anything;
 *    W == 1 is a device-to-device copy (nothing when in and out coincide).
 *
 * Sources: early NCCL "src/reduce_scatter.cu" (pytorch mirror) for the ring
 * schedule (GetBlock, ReduceScatterKernel) and the error conventions
 * (ncclInvalidType / ncclInvalidOperation, recvcount == 0, nDev == 1);
 * "Distributed primitives" notes for all-reduce / all-gather /
 * reduce-scatter semantics and ring allreduce = reduce-scatter + allgather;
 * Horovod "horovod/common/operations.cc" (PerformOperation, fusion batching in
 * BackgroundThreadLoop) and Apache SINGA "src/io/communicator.cc"
 * (Communicator::fusedSynch) for tensor fusion; MLX PR #3901 ("Add scatter
 * reduce for JACCL") for the latency-bound path at <= 32 KB and the in-place
 * read-before-write rule.
 */
#ifndef VCOLL_H_
#define VCOLL_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define VCOLL_MAX_RANKS 64

typedef enum {
  VCOLL_F32 = 0,
  VCOLL_BF16 = 1,
  VCOLL_F16 = 2 /* IEEE binary16: only as the wire type of vcoll_allreduce_wire */
} vcoll_dtype_t;

typedef enum {
  VCOLL_SUM = 0,
  VCOLL_MAX = 1,
  VCOLL_AVG = 2,
  VCOLL_MIN = 3, /* NCCL FuncMin */
  VCOLL_PROD = 4 /* NCCL FuncProd */
} vcoll_op_t;

typedef enum {
  VCOLL_OK = 0,
  VCOLL_ERR_INVALID_ARG = 1,  /* null pointer, W out of [1, 64], n < 0, misaligned
                                 pointer, or an overlap other than the allowed
                                 in-place forms */
  VCOLL_ERR_INVALID_TYPE = 2, /* dtype not a vcoll_dtype_t (ncclInvalidType) */
  VCOLL_ERR_INVALID_OP = 3,   /* op not a vcoll_op_t (ncclInvalidOperation) */
  VCOLL_ERR_UNSUPPORTED = 4,  /* a valid request this build does not handle */
  VCOLL_ERR_CUDA = 5          /* a CUDA runtime call or launch failed */
} vcoll_status_t;

/* Fold each segment in ring order (bit-exact with the NCCL ring). */
#define VCOLL_FLAG_RING_ORDER 0x1u
/* Force the variant that stages the W input tiles through shared memory with
 * bulk asynchronous copies (TMA), or the variant that loads straight into
 * registers.  Without either flag the library picks by message size.  Both
 * give identical bits.  The staged variant runs on device memory only: when
 * any buffer is pinned host or managed memory (cudaPointerGetAttributes), a
 * staged request runs the direct kernels. */
#define VCOLL_FLAG_STAGED 0x2u
#define VCOLL_FLAG_DIRECT 0x4u

/*
 * Reduce-scatter ("Distributed primitives", section 3; NCCL
 * ncclReduceScatter).  in[u]: n elements of rank u.  out[j]: receives the
 * len_j elements of segment j of the element-wise reduction of all W inputs.
 * In place: out[j] == (char*)in[j] + off_j * elemsize (NCCL's convention) or
 * any out/in pair with the same element mapping; other overlaps are
 * rejected.
 */
int vcoll_reduce_scatter(const void* const* in, void* const* out, int W, int64_t n, int dtype,
                         int op, unsigned flags, void* stream);

/*
 * Allgather ("Distributed primitives", section 2; ring allreduce's second
 * half).  in[j]: the len_j elements of segment j.  out[u]: receives all n
 * elements (segment j at off_j) on every rank u.  op is checked but unused.
 * In place: in[j] == (char*)out[u] + off_j * elemsize for some u.
 */
int vcoll_allgather(const void* const* in, void* const* out, int W, int64_t n, int dtype, int op,
                    unsigned flags, void* stream);

/*
 * Allgather with per-rank sizes (Horovod's allgatherv path: every rank's
 * tensor, first dimensions possibly different, concatenated in rank order on
 * every rank).  in[j]: counts[j] elements (counts: host array of W).
 * out[u]: receives counts[0] + ... + counts[W-1] elements, piece j at
 * counts[0] + ... + counts[j-1].  In place: in[j] == (char*)out[u] + that
 * offset * elemsize.
 */
int vcoll_allgatherv(const void* const* in, const int64_t* counts, void* const* out, int W,
                     int dtype, void* stream);

/*
 * Allreduce ("Distributed primitives", section 1 and ring allreduce =
 * reduce-scatter + allgather; Horovod / SINGA ncclAllReduce call sites).
 * in[u]: n elements; out[u]: n elements, all W outputs receive the same
 * result.  One kernel pass reads the W inputs once and writes the W outputs
 * from registers; its bits equal reduce-scatter followed by allgather.
 * In place: out[u] == in[u] (Horovod's in-place fusion-buffer allreduce).
 */
int vcoll_allreduce(const void* const* in, void* const* out, int W, int64_t n, int dtype, int op,
                    unsigned flags, void* stream);

/*
 * Ring order on a user ring (early NCCL src/reduce_scatter.cu: GetBlock maps
 * a ring position and step to a block through comm->userFromRing, and the
 * schedule comment of ncclReduceScatterWithTypeAndFunc works a 4-GPU ring
 * userFromRing = {1, 2, 0, 3}).  user_from_ring[p] is the rank at ring
 * position p, a permutation of 0 .. W-1 (host array of W ints; NULL: the
 * identity ring, the same as VCOLL_FLAG_RING_ORDER).  Segment j is folded
 * the way the ring reduce-scatter folds block j: it starts with the rank at
 * the ring position after rank j's, takes the following positions' ranks in
 * ring order (accumulator first), and ends at rank j.  The result is written
 * as by vcoll_reduce_scatter / vcoll_allreduce (an allreduce holds the
 * reduce-scatter's segments in every output: its allgather is a bit copy).
 * Arguments, aliasing and errors as vcoll_reduce_scatter / vcoll_allreduce;
 * a user_from_ring that is not a permutation gives VCOLL_ERR_INVALID_ARG.
 * max and min give the same bits in every order.
 */
int vcoll_reduce_scatter_ring(const void* const* in, void* const* out, int W, int64_t n,
                              int dtype, int op, const int* user_from_ring, void* stream);
int vcoll_allreduce_ring(const void* const* in, void* const* out, int W, int64_t n, int dtype,
                         int op, const int* user_from_ring, void* stream);

/*
 * Reduced-precision ("wire") allreduce, Apache SINGA Communicator::synchHalf /
 * fusedSynchHalf: fp32 inputs are converted to the 16-bit wire type (wire =
 * VCOLL_F16 as SINGA's float2half, or VCOLL_BF16), allreduced in that type by
 * the NCCL ring, whose buffers hold wire values so every hop rounds to the
 * wire type, and converted back to fp32 (half2float).  One pass: each
 * element is rounded, folded with a rounding after every op (ring order with
 * VCOLL_FLAG_RING_ORDER, else a pairwise tree), and the widened result is
 * written to the W fp32 outputs.  in[u], out[u]: n fp32 elements.  op: sum or
 * avg (the rounded sum times fl32(1/W), rounded again); max/min/prod give
 * VCOLL_ERR_UNSUPPORTED.  W == 1 is the round trip through the wire type.
 */
int vcoll_allreduce_wire(const void* const* in, void* const* out, int W, int64_t n, int wire, int op,
                         unsigned flags, void* stream);

/*
 * Tensor-fusion batching (Horovod BackgroundThreadLoop): greedy in tensor
 * order; a batch starts with the next tensor (even one above the threshold)
 * and takes the following tensors while the fused byte size stays
 * <= threshold_bytes.  counts[T] (host) are element counts; batch_begin
 * (host, T + 1 ints) receives the first tensor of each batch followed by T;
 * *nbatches the number of batches.  Host only, no GPU work.
 */
int vcoll_fuse_plan(const int64_t* counts, int T, int dtype, int64_t threshold_bytes,
                    int* batch_begin, int* nbatches);

/*
 * Fusion pack (Horovod PerformOperation "memcpy in fusion buffer"; SINGA
 * fusedSynch): fused[u] receives tensors[u*T + t] for t = 0..T-1 back to back,
 * no padding (tensor t at element offset counts[0] + ... + counts[t-1]).
 * tensors: host array of W*T device pointers, rank-major.  counts: host.
 * One kernel launch per up to 64 tensors (fewer when W*T would exceed 1024);
 * no buffer may overlap another.
 */
int vcoll_fuse_pack(const void* const* tensors, const int64_t* counts, int T, void* const* fused,
                    int W, int dtype, void* stream);

/* Fusion unpack: the inverse of vcoll_fuse_pack. */
int vcoll_fuse_unpack(const void* const* fused, const int64_t* counts, int T,
                      void* const* tensors, int W, int dtype, void* stream);

/*
 * Multi-tensor allreduce: Horovod's tensor fusion (PerformOperation: pack into
 * the fusion buffer, ncclAllReduce it in place, unpack; SINGA fusedSynch)
 * without the fusion buffer.  For each rank u the T tensors in[u*T + t] form
 * one virtual buffer of n = counts[0] + ... + counts[T-1] elements (tensor t at
 * offset counts[0] + ... + counts[t-1]); the allreduce of the W virtual
 * buffers is written to out[u*T + t].  The result has the bits of
 * vcoll_fuse_pack -> vcoll_allreduce (in place, same flags) ->
 * vcoll_fuse_unpack of the same batch, but every byte moves once (2*W*n*elemsize
 * instead of 6*W*n*elemsize).  Call it once per batch of vcoll_fuse_plan.
 * in, out: host arrays of W*T device pointers, rank-major; counts: host.  In
 * place: out[e] == in[e].  One launch per up to 64 tensors (fewer when W*T
 * would exceed 768).
 */
int vcoll_allreduce_multi(const void* const* in, void* const* out, const int64_t* counts, int T,
                          int W, int dtype, int op, unsigned flags, void* stream);

/*
 * Tensor-fusion allreduce, planned and executed in one call: the Horovod
 * batches of vcoll_fuse_plan(counts, T, dtype, threshold_bytes) are each
 * allreduced as in vcoll_allreduce_multi (each batch segmented on its own,
 * exactly as its fusion buffer would be), with the pieces of all batches
 * sharing kernel launches.  *nbatches (may be NULL) receives the batch count.
 * Same arguments and aliasing rules as vcoll_allreduce_multi; the bits equal
 * pack -> vcoll_allreduce -> unpack per batch.
 */
int vcoll_fusion_allreduce(const void* const* in, void* const* out, const int64_t* counts, int T,
                           int W, int dtype, int op, unsigned flags, int64_t threshold_bytes,
                           int* nbatches, void* stream);

/*
 * Tensor fusion through fusion buffers, Horovod operations.cc PerformOperation
 * (the NCCL allreduce path): the tensors are planned into the batches of
 * vcoll_fuse_plan(counts, T, dtype, threshold_bytes); for each batch of two or
 * more tensors every rank's tensors are copied back to back into that rank's
 * fusion buffer fused[u] (MEMCPY_IN_FUSION_BUFFER), the W buffers are
 * allreduced in place (NCCL_ALLREDUCE), and the results are copied out to
 * the output tensors (MEMCPY_OUT_FUSION_BUFFER); a batch of one tensor is
 * allreduced straight from its input to its output, as Horovod does with a
 * single entry.  The same fusion buffers serve every batch, in order, on
 * `stream`: the whole pipeline (3 launches per fused batch) runs from one
 * call.  The bits equal vcoll_fusion_allreduce's.
 * in, out: host arrays of W*T device pointers, rank-major; out[e] may equal
 * in[e] (in place), no other tensor may overlap another.  counts: host, T
 * element counts.  fused: host array of W device pointers, each to
 * fused_bytes bytes that overlap no tensor; every batch of two or more
 * tensors must fit (VCOLL_ERR_INVALID_ARG otherwise, before anything is
 * enqueued).  *nbatches (may be NULL) receives the batch count.  Other
 * arguments and errors as vcoll_allreduce.
 */
int vcoll_fusion_allreduce_buffered(const void* const* in, void* const* out,
                                    const int64_t* counts, int T, void* const* fused,
                                    int64_t fused_bytes, int W, int dtype, int op, unsigned flags,
                                    int64_t threshold_bytes, int* nbatches, void* stream);

/*
 * Sparsified allreduce with error feedback (Apache SINGA
 * Communicator::valSparsAllReduce, topK == false, and topKSparsAllReduce,
 * topK == true), fp32.  Per rank u: x = in[u] (+ accum[u] when accum is not
 * NULL).  threshold mode: the entries with |x| > threshold survive (and
 * x != 0); top-K mode: the K = ceil(threshold * n) entries (threshold in
 * [0, 1], computed in fp32 as SINGA does) with the largest values survive,
 * ties broken toward the lower index; values are ordered by their bits (-0
 * just below +0, NaNs beyond the infinities by sign -- with accum, where a
 * NaN comes from the sum in + accum its sign is the GPU's, which IEEE 754
 * leaves open).  With accum, accum[u] becomes x minus
 * the sent values: x elsewhere; where an entry survived, x - x in threshold
 * mode and x - (0 + x) in top-K mode (the sent values are scattered into
 * zeros first): zero for a finite x (-0 for a kept -0 in top-K mode), NaN for
 * an infinite one.  Every out[u]
 * receives the sum of all ranks' survivors, added into zeros rank by rank --
 * what the allgathered sparse lists scattered with cusparseSaxpyi give.
 * nnz (device, W int64, may be NULL) receives each rank's survivor count.
 * workspace: device memory of workspace_bytes bytes, 16-byte aligned, owned
 * by the caller, not kept after the call; calls that share a workspace must
 * not overlap.  Threshold mode needs none.  Top-K needs at least
 * vcoll_sparse_workspace_min_bytes(W, n, 1) (about n/1024 bytes + 8 KiB per
 * rank; smaller gives VCOLL_ERR_INVALID_ARG); vcoll_sparse_workspace_bytes(W,
 * n, 1) (about n bytes + 40 KiB per rank) adds room for candidate lists, which lets the
 * select passes after the first read only the entries above a sampled bound
 * instead of the whole array, and for small K lets the output come from the
 * lists (the same results, about three times as fast at K = 1 % of n; a size
 * in between gives smaller lists, and a rank whose list does not fit falls
 * back to the passes over the whole array).
 * In place: out[u] == in[u].
 */
size_t vcoll_sparse_workspace_bytes(int W, int64_t n, int topk);
size_t vcoll_sparse_workspace_min_bytes(int W, int64_t n, int topk);
int vcoll_sparse_allreduce(const void* const* in, void* const* out, void* const* accum, int W,
                           int64_t n, float threshold, int topk, int64_t* nnz, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * vcoll_sparse_allreduce without a caller workspace, for code that may not
 * allocate device memory (a framework that owns the whole device through its
 * own pool, a callback that must not block on cudaMalloc, a loop that must
 * have every resource in place before it starts).  The top-K working memory
 * is a fixed array inside the library, 1 MiB (VCOLL_SPARSE_NOALLOC_BYTES) on
 * every GPU that loads it, held until the process exits;
 * the call allocates nothing.  Arguments and results are those of
 * vcoll_sparse_allreduce; sizes whose minimum working memory would not fit
 * (vcoll_sparse_workspace_min_bytes(W, n, 1) > the maximum, about n <= 120 Mi
 * elements at W = 8) return VCOLL_ERR_INVALID_ARG with an explanation, and
 * what the array holds beyond that minimum is candidate-list room (enough
 * for the fast path up to a few million entries over all ranks at K = 1 %).  The
 * threshold mode needs no working memory and passes straight through.
 * The first top-K call on a device looks up the array's device address with
 * cudaGetSymbolAddress (again after the device's context changes, as after
 * cudaDeviceReset); make that first call before capturing a stream.
 * All calls share the one array and it keeps the last call's contents (the
 * call clears what must start at zero), so calls that may run at the same
 * time on the GPU -- on different streams, or from different threads --
 * race on it: order them on one stream.
 * The pages have no counterpart of this entry point.
 */
#define VCOLL_SPARSE_NOALLOC_BYTES (1u << 20)
int vcoll_sparse_allreduce_noalloc(const void* const* in, void* const* out, void* const* accum,
                                   int W, int64_t n, float threshold, int topk, int64_t* nnz,
                                   void* stream);

/*
 * Layer operators: the memory-bound ends of a rank's training step, whose
 * weight gradients are what the collectives above reduce.  Each call is one
 * rank's; every gradient output may be a slice of that rank's fusion buffer
 * (any alignment to the element).  The conventions at the top of this file
 * hold, and in addition:
 *  - A matrix of N rows and D columns is a pointer and a row stride `*_ld`
 *    in elements (>= D; rows may be parts of wider rows); its columns are
 *    adjacent.  N and V up to 2^31 - 2, D up to 2^30; offsets are 64-bit.
 *  - Buffers of one call may not overlap, except where a call names an
 *    in-place form; matrices that are different column ranges of the same
 *    wider rows (equal row strides in bytes) do not overlap.
 *  - Sums, means and statistics are fp32; a bf16 output is rounded once (a
 *    computed NaN is the canonical one of the conversion).
 *    The order of every sum is fixed by the sizes, the tokens and the GPU, in
 *    the layer norms also by the alignment and the row strides of the operands
 *    (weight and bias among them), which decide what columns a thread holds.
 *    So a call repeated on the same buffers gives the same bits, but a layer
 *    norm of the same values placed otherwise may differ in the last ones; the
 *    lookup, its gradient and the 8-bit form alone do not.
 *  - `workspace`: device memory of the size the *_workspace_bytes function
 *    gives, 256-byte aligned, contents neither expected nor kept; calls that
 *    share one must not overlap.
 *  - An empty input (N == 0) still writes what its outputs then are (the
 *    gradient of no rows is zero); D == 0 enqueues nothing.
 * The pages have no counterpart of these entry points.
 */

/* Type of a token index. */
typedef enum { VCOLL_I32 = 0, VCOLL_I64 = 1 } vcoll_index_t;

/*
 * Embedding lookup: out[i] = scale * table[tokens[i]] (one fp32 multiply,
 * rounded to dtype), i < N.  table: V x D, out: N x D, both of dtype.  A token
 * outside [0, V) -- padding -- gives a row of zeros.
 */
int vcoll_embedding(const void* tokens, int index_type, int64_t N, const void* table,
                    int64_t table_ld, int64_t V, int64_t D, float scale, void* out,
                    int64_t out_ld, int dtype, void* stream);

/*
 * Its gradient: table_grad[v] = base[v] + scale * (the sum of grad[i] over the
 * i with tokens[i] == v).  Every row of table_grad (V x D, of table_dtype) is
 * written, rows of tokens that do not occur as base or zeros.  base (V x D, of
 * table_dtype) may be NULL (zeros), or table_grad itself with the same row
 * stride: then only the rows of tokens that occur are read and written.
 * Tokens outside [0, V) contribute nothing.  grad: N x D of dtype.  The tokens
 * are brought into order (stably), so each row is summed in the order of i,
 * cut into parts at places that the tokens and the sizes determine.
 */
size_t vcoll_embedding_backward_workspace_bytes(int64_t N, int64_t V, int64_t D);
int vcoll_embedding_backward(const void* grad, int64_t grad_ld, int dtype, const void* tokens,
                             int index_type, int64_t N, int64_t V, int64_t D, float scale,
                             const void* base, int64_t base_ld, void* table_grad,
                             int64_t table_ld, int table_dtype, void* workspace,
                             size_t workspace_bytes, void* stream);

/*
 * Layer norm over the D columns of each row: mean = sum(x) / D,
 * rstd = 1 / sqrt(sum((x - mean)^2) / D + eps), y = (x - mean) * rstd * weight
 * + bias.  x, y: N x D of dtype; in place: y == x with the same row stride.
 * weight, bias: D of weight_dtype, either may be NULL (ones, zeros).  mean,
 * rstd: N fp32 each, kept for the backward pass; either may be NULL.  A row
 * holding an infinity or a NaN is NaN throughout, other rows are not touched
 * by it.
 */
int vcoll_layer_norm(const void* x, int64_t x_ld, const void* weight, const void* bias,
                     int weight_dtype, int64_t N, int64_t D, float eps, void* y, int64_t y_ld,
                     float* mean, float* rstd, int dtype, void* stream);

/*
 * Its gradient.  With h = (x - mean) * rstd and g = grad * weight:
 * dx = rstd * (g - sum(g) / D - h * sum(g * h) / D), dweight = the sum of
 * grad * h over the rows, dbias = the sum of grad over the rows.  grad, x, dx:
 * N x D of dtype; in place: dx == grad or dx == x with the same row stride.
 * weight (NULL: ones), dweight, dbias: D of weight_dtype; dx, dweight and
 * dbias may each be NULL (not wanted).
 */
size_t vcoll_layer_norm_workspace_bytes(int64_t N, int64_t D);
int vcoll_layer_norm_backward(const void* grad, int64_t grad_ld, const void* x, int64_t x_ld,
                              const float* mean, const float* rstd, const void* weight,
                              int weight_dtype, int64_t N, int64_t D, void* dx, int64_t dx_ld,
                              void* dweight, void* dbias, int dtype, void* workspace,
                              size_t workspace_bytes, void* stream);

/*
 * Activations kept in 8 bits between the forward and the backward pass.  Each
 * VCOLL_CHECKPOINT8_BLOCK columns of a row share a scale: with a the block's
 * largest magnitude, scale = a / 127 and code = x * (127 / a) rounded to the
 * nearest integer, ties to even (fp32 divisions and product, each rounded
 * once), standing for code * scale.  A block with a < 2^-100 is kept as zeros
 * (scale 0); one with an infinity or a NaN has scale NaN, so that it reads
 * back as NaN.  codes: N x D int8 at a row stride of codes_ld >= D bytes, a
 * multiple of 16, from a 16-byte aligned address; what lies between D and the
 * next multiple of 16 is written as zeros.  scales: N x
 * ceil(D / VCOLL_CHECKPOINT8_BLOCK) fp32, rows adjacent.  x: N x D of dtype.
 */
#define VCOLL_CHECKPOINT8_BLOCK 128
int vcoll_checkpoint8(const void* x, int64_t x_ld, int64_t N, int64_t D, int8_t* codes,
                      int64_t codes_ld, float* scales, int dtype, void* stream);

/*
 * What the codes stand for: out = code * scale, or code * scale * weight +
 * bias where those are given (D of weight_dtype, either may be NULL).  out:
 * N x D of dtype.
 */
int vcoll_checkpoint8_restore(const int8_t* codes, int64_t codes_ld, const float* scales,
                              const void* weight, const void* bias, int weight_dtype, int64_t N,
                              int64_t D, void* out, int64_t out_ld, int dtype, void* stream);

/*
 * Layer norm that keeps its normalised input h = (x - mean) * rstd in 8 bits
 * on the way (the codes and scales of vcoll_checkpoint8 of h): neither x nor y
 * has to be kept, vcoll_checkpoint8_restore with the weight and bias gives y
 * back.  y is computed from the unrounded h.  Other arguments as
 * vcoll_layer_norm.
 */
int vcoll_layer_norm_checkpoint8(const void* x, int64_t x_ld, const void* weight,
                                 const void* bias, int weight_dtype, int64_t N, int64_t D,
                                 float eps, void* y, int64_t y_ld, float* rstd, int8_t* codes,
                                 int64_t codes_ld, float* scales, int dtype, void* stream);

/* The gradient of vcoll_layer_norm from what vcoll_layer_norm_checkpoint8
 * kept: h is code * scale.  Other arguments as vcoll_layer_norm_backward; in
 * place: dx == grad with the same row stride. */
int vcoll_layer_norm_backward_checkpoint8(const void* grad, int64_t grad_ld, const int8_t* codes,
                                          int64_t codes_ld, const float* scales,
                                          const float* rstd, const void* weight, int weight_dtype,
                                          int64_t N, int64_t D, void* dx, int64_t dx_ld,
                                          void* dweight, void* dbias, int dtype, void* workspace,
                                          size_t workspace_bytes, void* stream);

/*
 * Products of a rank's rows with weights, with the element-wise part of the
 * operator in the product's epilogue: the loss against a vocabulary and the
 * gated feed-forward block.  The conventions of the layer operators hold, and
 * in addition:
 *  - bf16 products are exact and summed in fp32.  fp32 operands are taken as
 *    three bf16 parts each, which together hold their 24 bits, in six products
 *    summed in fp32 (weights that meet 16 rows or fewer as they are); an infinite
 *    fp32 operand may give NaN.
 *  - A bf16 matrix in device memory that starts at a 16-byte boundary, with a
 *    row stride that is a multiple of 8, is read where it lies; any other, and
 *    every fp32 one, is laid out in the workspace first.
 *  - The *_workspace_bytes functions take `direct`: 1 where all the matrices
 *    that the products read (x, table, w_gate, w_up) lie so; 0 always suffices.
 *    The workspace is device memory.
 *  - The order of a sum is fixed by the sizes, the type, the results that are
 *    wanted (dx with or without dtable), whether there is a base, whether the
 *    matrices lie as `direct` says and, of 16 fp32 rows or fewer, whether the
 *    weights' rows are whole 16-byte pieces.  A call repeated on the same
 *    buffers gives the same bits; a call that differs in one of these may
 *    differ in a result's last bits.
 */

/*
 * Softmax cross entropy of N rows against a table of V tokens, without keeping
 * the logits z = x * table^T: lse[i] = log(sum over v of exp(z[i][v])), loss[i]
 * = lse[i] - z[i][targets[i]].  A target outside [0, V) -- padding -- has loss
 * 0.  x: N x D, table: V x D, both of dtype; loss, lse: N fp32.  V == 0: lse is
 * -infinity.  D == 0: the logits are zeros.  A logit that overflows to +infinity
 * gives lse +infinity, and the loss +infinity to other targets of its row.
 */
size_t vcoll_cross_entropy_workspace_bytes(int64_t N, int64_t V, int64_t D, int dtype, int direct);
int vcoll_cross_entropy(const void* x, int64_t x_ld, const void* table, int64_t table_ld,
                        const void* targets, int index_type, int64_t N, int64_t V, int64_t D,
                        float* loss, float* lse, int dtype, void* workspace,
                        size_t workspace_bytes, void* stream);

/*
 * Its gradient.  With e[i][v] = dloss[i] * (exp(z[i][v] - lse[i]) - (v ==
 * targets[i])), and e[i] zeros where the target is outside [0, V) (whatever
 * that row of x, its dloss and its lse hold): dx = e * table, dtable = base +
 * e^T * x.  The logits are computed again, a piece of the vocabulary at a time.
 * dloss: N fp32, or one for all rows (dloss_count N or 1).  base (V x D of
 * dtype) may be NULL (zeros), or dtable itself with the same row stride; dx may
 * be x with the same row stride.  dx and dtable may each be NULL (not wanted).
 * With bf16 operands e is rounded to bf16 for the products, relative to the
 * largest magnitude of dloss over the rows that count.
 */
size_t vcoll_cross_entropy_backward_workspace_bytes(int64_t N, int64_t V, int64_t D, int dtype,
                                                    int direct);
int vcoll_cross_entropy_backward(const float* dloss, int64_t dloss_count, const void* x,
                                 int64_t x_ld, const void* table, int64_t table_ld,
                                 const void* targets, int index_type, const float* lse, int64_t N,
                                 int64_t V, int64_t D, void* dx, int64_t dx_ld, const void* base,
                                 int64_t base_ld, void* dtable, int64_t dtable_ld, int dtype,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* Activation of a gated block: g / (1 + exp(-g)); g * Phi(g) with the normal
 * distribution function Phi; g * (1 + tanh(sqrt(2 / pi) * (g + 0.044715 *
 * g^3))) / 2.  At an infinite g the activation and its derivative are their
 * limits. */
typedef enum { VCOLL_SILU = 0, VCOLL_GELU = 1, VCOLL_GELU_TANH = 2 } vcoll_activation_t;

/*
 * Gated feed-forward block: gate = x * w_gate^T, up = x * w_up^T, h =
 * act(gate) * up, computed from the unrounded gate and up.  x: N x D, w_gate,
 * w_up: F x D, h, gate, up: N x F, all of dtype.  gate and up are kept for the
 * backward pass; either may be NULL.  D == 0: zeros.
 */
size_t vcoll_gated_ff_workspace_bytes(int64_t N, int64_t D, int64_t F, int dtype, int direct);
int vcoll_gated_ff(const void* x, int64_t x_ld, const void* w_gate, int64_t w_gate_ld,
                   const void* w_up, int64_t w_up_ld, int activation, int64_t N, int64_t D,
                   int64_t F, void* h, int64_t h_ld, void* gate, int64_t gate_ld, void* up,
                   int64_t up_ld, int dtype, void* workspace, size_t workspace_bytes,
                   void* stream);

/*
 * Its gradient from the kept gate and up: dgate = dh * up * act'(gate), dup =
 * dh * act(gate), dx = dgate * w_gate + dup * w_up, dw_gate = dgate^T * x,
 * dw_up = dup^T * x.  With bf16 operands dgate and dup are rounded to bf16 for
 * the products, or where N * F is 8192 or less to twice its bits.  dx, dw_gate
 * and dw_up may each be NULL (not wanted).
 */
size_t vcoll_gated_ff_backward_workspace_bytes(int64_t N, int64_t D, int64_t F, int dtype,
                                               int direct);
int vcoll_gated_ff_backward(const void* dh, int64_t dh_ld, const void* x, int64_t x_ld,
                            const void* w_gate, int64_t w_gate_ld, const void* w_up,
                            int64_t w_up_ld, const void* gate, int64_t gate_ld, const void* up,
                            int64_t up_ld, int activation, int64_t N, int64_t D, int64_t F,
                            void* dx, int64_t dx_ld, void* dw_gate, int64_t dw_gate_ld,
                            void* dw_up, int64_t dw_up_ld, int dtype, void* workspace,
                            size_t workspace_bytes, void* stream);

/* Device-side error bits, OR-ed into one word per device by the kernels.
 * The staged kernels and the products bound every wait on their shared-memory
 * barriers (2 s of wall-clock time); a wait that gives up records
 * VCOLL_DEVICE_ERR_TIMEOUT and the kernel returns early (its outputs are then
 * incomplete). */
#define VCOLL_DEVICE_ERR_TIMEOUT 0x1u

/* Reads the current device's error word into *flags (and resets it when
 * clear != 0).  Synchronous: waits for all work on the device to finish. */
int vcoll_device_errors(unsigned* flags, int clear);

/* Diagnostics for the bounded waits: launches one thread that waits on a
 * shared-memory barrier nothing ever arrives at; the wait gives up after
 * limit_us microseconds (1 .. 10^6) and records VCOLL_DEVICE_ERR_TIMEOUT in
 * the device error word, and the kernel returns -- the device stays usable.
 * Read the word with vcoll_device_errors.  Asynchronous on `stream`. */
int vcoll_selftest_wait_timeout(unsigned limit_us, void* stream);

/* Segment j of an n-element buffer over W ranks (host only). */
int vcoll_segment(int64_t n, int W, int j, int64_t* off, int64_t* len);

/* Static description of a status code. */
const char* vcoll_status_string(int status);

/* Thread-local detail of the last failing call on this thread ("" if none). */
const char* vcoll_last_error(void);

/* Library version, major * 10000 + minor * 100 + patch. */
int vcoll_version(void);

#ifdef __cplusplus
}
#endif

#endif /* VCOLL_H_ */
