/*
 * dt.h -- C ABI of libdt: DTensor-style tensor-parallel linears and layout
 * transforms on one GB300 (sm_103a).
 *
 * Every mesh rank is a LOGICAL shard: all P ranks' local tensors ("slots")
 * live in the HBM of one GPU, and what a multi-GPU framework does with
 * collectives is done here by one kernel over all slots.
 *
 * Sources (page title and section):
 *  - Hyper-Parallel DTensor API (MindSpore hyper-parallel pull request 121):
 *    DeviceMesh / placements / layout, distribute_tensor, redistribute,
 *    reduce_partial, full_tensor, shape, local_shape.
 *  - DTorch user guide, "Module parallel", section 3 (Linear implementation
 *    walkthrough): tp_dim, tp_shard_type, weight/bias placements and the
 *    input placement checks; section 2: EmbeddingWithReplicateOutput.
 *  - Model parallelism (wineandchord), "Tensor Parallel": Y_i = X W_i
 *    (column), Y = sum_i X_i W_i (row), weights stored [in, out].
 *  - nanotron tutorial ch. 5, sections 5.1 and 5.5: ALL_REDUCE and
 *    REDUCE_SCATTER modes of the row-parallel linear.
 *
 * Conventions for every entry point
 *  - Pointers named "device" are CUDA device pointers on the current GPU;
 *    everything else (descriptors, slot arrays, stride arrays, output
 *    scalars) is host memory that is read during the call only.
 *  - The caller owns all device memory: inputs, outputs and workspaces.  The
 *    library allocates no device memory, on any call.  A linear's workspace
 *    (its size from the *_workspace_size query of that call) holds the
 *    split tail's scratch: where the tensor-core GEMM's last wave would
 *    leave CTA pairs idle, the remaining tiles' K range is divided over all
 *    pairs and the pieces' fp32 partials meet in the workspace.  A call given
 *    no workspace, or one too small, runs every tile whole: same results up
 *    to fp32 summation order, slower where the split pays.  The workspace's
 *    contents between calls are the caller's (the library zeroes what it
 *    needs zeroed on the call's stream); calls whose kernels may overlap on
 *    the GPU need separate workspaces.
 *  - The library keeps host-side caches (TMA descriptors; launch plans keyed
 *    by the operands' layouts, slot pointers, strides, workspace and stream,
 *    so a repeated call skips planning) and, made once and kept, per device
 *    one auxiliary stream with two events (a redistribute call with both
 *    copies and Partial reductions runs the reductions there, forked from
 *    and joined back to the caller's stream).  dt_clear_cache() drops the
 *    caches.
 *  - Environment switches, read once per process:
 *      DT_GEMM_SPLIT=0     turns the split tail off; =2 splits every last
 *                          wave the finishing can take, whether or not the
 *                          cost model expects a gain (to compare schedules);
 *      DT_GEMM_BANDS=m,n   fixes the GEMM tile order's band height and block
 *                          width (in 256 x 256 tiles) instead of the host's
 *                          choice, to compare orders.
 *    Test hooks exercise the bounded-wait exit without a fault:
 *      DT_GEMM_WAIT_LIMIT_MS=n  bounds every GEMM barrier wait at n ms
 *                               (1..10000; default 2000);
 *      DT_GEMM_STARVE=1         makes the GEMM producers issue no copies,
 *                               so every wait runs out and the launch
 *                               reports DT_DEV_ERR_TIMEOUT.
 *      DT_RD_WAIT_LIMIT_MS=n,   the same two hooks for the bulk (TMA) copy
 *      DT_RD_STARVE=1           kernel of dt_redistribute;
 *      DT_KV4_WAIT_LIMIT_MS=n,  and for dt_tp_kv4_attention, whose copies
 *      DT_KV4_STARVE=m          stay short of what is awaited from the m-th
 *                               step of each CTA (tile of each warp) on.
 *  - Compute calls are asynchronous on the given stream (a cudaStream_t;
 *    NULL = the legacy default stream).  Their return value covers the checks
 *    done on the host before any launch; on any error nothing is launched.
 *  - Errors found on the GPU are OR-ed, as DT_DEV_* bits, into the int32 at
 *    device address d_status (read it after synchronising).  Kernels never
 *    trap.  d_status may be NULL: the bits then go to a status word inside
 *    the library, read and cleared by dt_read_device_status().
 *  - Inputs and outputs must not overlap.
 *  - Empty tensors are valid operands.  A slot with no elements may have a
 *    NULL pointer and any strides.  A call with nothing to write (no tokens,
 *    no output columns) returns DT_OK without launching or calling CUDA.  A
 *    linear whose inner dim K is 0 writes its bias, or zeros.
 *  - dt_last_error() returns a human-readable reason for the last non-OK
 *    status returned on the calling thread.
 */
#ifndef DT_H_
#define DT_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Exported symbols keep default visibility even when the library is built
 * with -fvisibility=hidden. */
#if defined(__GNUC__)
#define DT_API __attribute__((visibility("default")))
#else
#define DT_API
#endif

#define DT_MAX_MESH_DIMS 4
#define DT_MAX_TENSOR_DIMS 4
#define DT_MAX_SLOTS 64

/* CUDA stream handle; the same type as cudaStream_t / CUstream. */
typedef struct CUstream_st* dt_stream_t;

typedef enum dt_status {
  DT_OK = 0,
  DT_ERR_INVALID_ARG = 1,  /* null pointer, bad enum, bad count */
  DT_ERR_SHAPE = 2,        /* shapes of the operands do not agree */
  DT_ERR_PLACEMENT = 3,    /* placement breaks the layer's rule (the DTorch
                              guide's `assert input.check_placement(...)`) */
  DT_ERR_UNSUPPORTED = 4,  /* legal in principle, not provided (e.g. Shard -> Partial) */
  DT_ERR_ALIGNMENT = 5,    /* pointer or stride alignment the kernel needs */
  DT_ERR_CUDA = 6,         /* a CUDA runtime or driver call failed */
  DT_ERR_CAPACITY = 7      /* more slots, tasks or groups than one call plans, or a
                              linear dimension at or above 2^31 - 512 (the GEMM
                              kernels' coordinates are 32-bit) */
} dt_status;

/* Bits OR-ed into *d_status by kernels. */
#define DT_DEV_ERR_INDEX 0x1   /* an embedding id was outside [0, vocab): its row was zero-filled */
#define DT_DEV_ERR_TIMEOUT 0x2 /* a bounded wait (GEMM or bulk copy kernel) gave up; its outputs are not valid */

typedef enum dt_dtype { DT_BF16 = 0, DT_FP32 = 1, DT_INT32 = 2 } dt_dtype;

/* Placement kinds (Hyper-Parallel DTensor API, placement-type table). */
typedef enum dt_pkind { DT_REPLICATE = 0, DT_SHARD = 1, DT_PARTIAL = 2 } dt_pkind;
/* Partial reductions.  SUM adds the partial values in rank order in fp32;
 * AVG divides that sum once (fp32, correctly rounded) by the number of
 * partial values; MAX keeps the largest in rank order.  bf16 results are
 * rounded once at the end.  All Partial dims of one layout use one op. */
typedef enum dt_reduce_op { DT_SUM = 0, DT_AVG = 1, DT_MAX = 2 } dt_reduce_op;

/* Row-parallel output modes (nanotron 5.1; DTorch RowParallelLinear keeps Partial). */
typedef enum dt_tp_mode {
  DT_TP_PARTIAL = 0,        /* output Partial() on tp: P materialised partial products */
  DT_TP_ALL_REDUCE = 1,     /* output Replicate() on tp: the summed product */
  DT_TP_REDUCE_SCATTER = 2  /* output Shard(0) on tp: each slot keeps a block of rows */
} dt_tp_mode;

typedef struct dt_placement {
  int32_t kind; /* dt_pkind */
  int32_t dim;  /* tensor dim for DT_SHARD; negative counts from the end */
  int32_t op;   /* dt_reduce_op for DT_PARTIAL */
} dt_placement;

/*
 * A global tensor's distribution over a logical mesh.
 *  - Ranks are numbered row-major over mesh_shape (last mesh dim fastest), as
 *    in the printed distribute_tensor example (ranks 0,1 hold rows 0-1).
 *  - A Shard splits a dim torch.chunk-style: width ceil(n/p), trailing parts
 *    may be short or empty.  Two mesh dims sharding one tensor dim nest in
 *    mesh-dim order.
 *  - Slots: with materialize_replicas == 0, ranks that differ only in their
 *    Replicate coordinates share ONE slot.  Slots are numbered row-major
 *    over the non-Replicate mesh dims.  With materialize_replicas != 0,
 *    slot == rank.
 */
typedef struct dt_layout {
  int32_t mesh_ndim;
  int32_t mesh_shape[DT_MAX_MESH_DIMS];
  dt_placement placements[DT_MAX_MESH_DIMS];
  int32_t ndim;
  int64_t gshape[DT_MAX_TENSOR_DIMS];
  int32_t dtype; /* dt_dtype */
  int32_t materialize_replicas;
} dt_layout;

/*
 * A distributed tensor: a layout plus one device pointer per slot.
 * slots[s] points at slot s's local tensor (local shape from
 * dt_layout_slot_box); it may be NULL only when that slot is empty.
 * strides: NULL for contiguous row-major slots, else a host array of
 * nslots * layout.ndim element strides (slot-major).
 */
typedef struct dt_dtensor {
  dt_layout layout;
  int32_t nslots;
  void* const* slots;
  const int64_t* strides;
} dt_dtensor;

/* ---- host-only layout queries (Hyper-Parallel DTensor API: Layout, shape, local_shape) ---- */

/* Number of slots of a layout.  Errors: DT_ERR_INVALID_ARG on a malformed layout. */
DT_API dt_status dt_layout_nslots(const dt_layout* layout, int32_t* nslots);

/* Slot holding rank `rank`'s local tensor. */
DT_API dt_status dt_layout_slot_of_rank(const dt_layout* layout, int32_t rank, int32_t* slot);

/* Local shape and global offset (layout.ndim entries each) of slot `slot`. */
DT_API dt_status dt_layout_slot_box(const dt_layout* layout, int32_t slot, int64_t* local_shape,
                             int64_t* global_offset);

/* ---- data movement ---- */

/*
 * redistribute(): move `src` to `dst` placements on the same mesh and global
 * shape (Hyper-Parallel DTensor API: redistribute, reduce_partial,
 * full_tensor, distribute_tensor).  The transitions are
 *   Shard(a) -> Shard(b)  (all-to-all),  Shard -> Replicate (all-gather),
 *   Replicate -> Shard (slicing),  Partial -> Replicate (all-reduce),
 *   Partial -> Shard (reduce-scatter),  Replicate -> Partial (coordinate 0
 *   keeps the value, the others get zeros), Partial -> Partial (kept).
 * Partial sums add the partial values of an element in rank order in fp32
 * and round a bf16 result once, to nearest even: results are bit-exact and
 * independent of the launch shape.  Shard -> Partial returns
 * DT_ERR_UNSUPPORTED; dtypes must match; int32 supports no Partial.
 * Copies whose rows are all 16-byte aligned on both sides run on the bulk
 * (TMA) copy engine, the others on a warp copy kernel; only the bulk kernel
 * waits (bounded), and a wait that gives up sets DT_DEV_ERR_TIMEOUT in
 * *d_status (NULL: the library's status word).
 */
DT_API dt_status dt_redistribute(const dt_dtensor* src, const dt_dtensor* dst, int32_t* d_status,
                          dt_stream_t stream);

/*
 * n independent redistributes, src[i] -> dst[i], each with the rules and
 * results of dt_redistribute.  The pages move one tensor per call; this
 * batched form (no counterpart there) packs the copies of all n pairs into
 * one kernel launch and their Partial reductions into one more, as far as a
 * launch's parameter block holds (128 source and 128 destination slots, 192
 * boxes, 256 partial references), and starts further launches beyond that.
 * Pairs may differ in mesh, shape, dtype and reduce op; a launch holds one
 * dtype (and, for reductions, one op), so each further dtype or op adds a
 * launch.  All tensors of a call live on one device (that of the first
 * non-empty destination slot, where the kernels run).  No dst[i] may
 * overlap any src[j] or another dst[j] of the same call: the pairs run
 * concurrently.  Every pair is checked before anything launches; an error
 * names the pair and nothing runs.  n == 0 is a no-op.
 */
DT_API dt_status dt_redistribute_batch(int32_t n, const dt_dtensor* src, const dt_dtensor* dst,
                                int32_t* d_status, dt_stream_t stream);

/*
 * EmbeddingWithReplicateOutput (DTorch guide, section 2): table Shard(1) on
 * tp (slot i holds [vocab, d_i] bf16 or fp32, d_i from the torch.chunk split
 * of the embedding dim), ids int32 Replicate on tp, out Replicate on tp with
 * shape ids.shape + [dim].  out[t, o_i:o_i+d_i] = table_i[ids[t], :]; an id
 * outside [0, vocab) zero-fills that row and sets DT_DEV_ERR_INDEX.
 * Other mesh dims must be Replicate for all three.  With no tokens (or an
 * empty embedding dim) the call returns DT_OK without launching; a table of
 * no rows with tokens to gather is refused with DT_ERR_SHAPE.
 */
DT_API dt_status dt_tp_embedding(const dt_dtensor* ids, const dt_dtensor* table, const dt_dtensor* out,
                          int32_t tp_mesh_dim, int32_t* d_status, dt_stream_t stream);

/* ---- linears (weights stored [in, out] as in the wineandchord reference) ----
 *
 * Every linear takes `workspace` / `workspace_bytes`: NULL (size ignored) or
 * caller-owned device memory, 256-byte aligned, of any size.  With at least
 * the bytes its *_workspace_size query reports, the call splits the tensor-
 * core GEMM's last wave where that pays (see the ownership convention
 * above); with less it runs every tile whole.  The queries take the call's
 * operands (host descriptors only, nothing is read from the device), check
 * them as the call would, and answer for the CURRENT device, whose number
 * of co-resident CTA pairs decides the split; without a CUDA device they
 * return DT_ERR_CUDA.
 * bf16 operands whose row pitch is not a multiple of 16 bytes, or whose base
 * is not 16-byte aligned (the shards of a dim that torch.chunk splits
 * unevenly, e.g. 8190 columns over 4), cannot be read by TMA.  With enough
 * workspace (the query counts it) the call copies each such operand into
 * the workspace with a padded pitch and runs on the tensor cores; with less
 * it runs on a CUDA-core kernel, an order of magnitude slower, and
 * dt_cuda_core_gemm_count() counts the launch.  fp32 linears always run on
 * the CUDA-core kernel and need no workspace (0 bytes).
 */

/*
 * ColumnParallelLinear: Y_i = X W_i (+ b_i) for every tp shard i, all shards
 * in one launch (wineandchord "Column parallel"; DTorch tp_shard_type "col").
 *   x    [..., K] Replicate on tp            (bf16 or fp32)
 *   w    [K, N]   Shard(1) on tp             (same dtype as x)
 *   bias [N]      Shard(0) on tp, or NULL    (bf16 or fp32)
 *   y    [..., N] Shard(-1) on tp            (bf16 or fp32; fp32 accumulate)
 * On other mesh dims w and bias must be Replicate and x, y must agree.
 * tp_mesh_dim < 0 means no TP (ReplicateParallelLinear).  Leading dims of x
 * and y are flattened and must be collapsible with unit inner stride.
 * bf16 operands run on the tcgen05 tensor-core GEMM (operands whose pitch
 * TMA cannot describe through a padded copy in the workspace, see above);
 * fp32 runs on a CUDA-core kernel.
 */
DT_API dt_status dt_column_parallel_linear(const dt_dtensor* x, const dt_dtensor* w, const dt_dtensor* bias,
                                    const dt_dtensor* y, int32_t tp_mesh_dim, void* workspace,
                                    size_t workspace_bytes, int32_t* d_status, dt_stream_t stream);

/*
 * Several column-parallel linears that share one input (e.g. fused q/k/v),
 * in ONE launch: y[j] = column_parallel(x, w[j], bias[j]) for j < n.
 * w, y: arrays of n descriptors; bias: NULL or an array of n descriptors
 * whose entries may have nslots == 0 for "no bias".
 */
DT_API dt_status dt_column_parallel_linear_multi(const dt_dtensor* x, int32_t n, const dt_dtensor* w,
                                          const dt_dtensor* bias, const dt_dtensor* y,
                                          int32_t tp_mesh_dim, void* workspace, size_t workspace_bytes,
                                          int32_t* d_status, dt_stream_t stream);

/* Workspace bytes of dt_column_parallel_linear(_multi) on these operands
 * (n = 1 for the single form; the bias does not change it). */
DT_API dt_status dt_column_parallel_linear_workspace_size(const dt_dtensor* x, int32_t n, const dt_dtensor* w,
                                                          const dt_dtensor* y, int32_t tp_mesh_dim,
                                                          size_t* bytes);

/*
 * RowParallelLinear: Y = sum_i X_i W_i (+ b) (wineandchord "Row parallel";
 * DTorch tp_shard_type "row"; nanotron TensorParallelRowLinear).
 *   x    [..., K] Shard(-1) on tp
 *   w    [K, N]   Shard(0) on tp
 *   bias [N]      Replicate, or NULL; added ONCE (DTorch keeps the row bias
 *                 Partial so the shards' biases sum to one bias)
 *   y    mode DT_TP_ALL_REDUCE:     [..., N] Replicate on tp
 *        mode DT_TP_REDUCE_SCATTER: [..., N] Shard(0) on tp
 *        mode DT_TP_PARTIAL:        [..., N] Partial on tp (bias on part 0)
 * For ALL_REDUCE and REDUCE_SCATTER the sum over shards is fused into the
 * fp32 tensor-core accumulator: no partial product is written to memory.
 */
DT_API dt_status dt_row_parallel_linear(const dt_dtensor* x, const dt_dtensor* w, const dt_dtensor* bias,
                                 const dt_dtensor* y, int32_t mode, int32_t tp_mesh_dim, void* workspace,
                                 size_t workspace_bytes, int32_t* d_status, dt_stream_t stream);

/* Workspace bytes of dt_row_parallel_linear on these operands. */
DT_API dt_status dt_row_parallel_linear_workspace_size(const dt_dtensor* x, const dt_dtensor* w, const dt_dtensor* y,
                                                       int32_t mode, int32_t tp_mesh_dim, size_t* bytes);

/*
 * Llama-style TP MLP (nanotron 5.1: the MLP follows the attention's
 * column/row pattern):
 *   H_i = bf16( SiLU(X Wg_i) * (X Wu_i) )     gate/up column-parallel, one launch,
 *                                            two accumulators per tile, SiLU in fp32
 *   Y   = row_parallel(H, Wd, mode)           down projection
 * x [M, K] Replicate, w_gate/w_up [K, F] Shard(1), w_down [F, N] Shard(0),
 * y per `mode` as in dt_row_parallel_linear.  All bf16 (y bf16 or fp32).
 * workspace: caller-owned device memory, 256-byte aligned.  It receives H
 * at its start, as one [M, F] bf16 row-major tensor per distinct x slot
 * (shard i = the columns of chunk i; blocks 256-byte aligned), which the
 * call needs (DT_ERR_INVALID_ARG when the workspace is smaller); the bytes
 * after H are the two GEMMs' split-tail scratch, as for the linears.
 * dt_tp_mlp_workspace_size reports H plus that scratch for the current
 * device (DT_ERR_CUDA without one).
 */
DT_API dt_status dt_tp_mlp_workspace_size(const dt_dtensor* x, const dt_dtensor* w_gate, const dt_dtensor* w_up,
                                          const dt_dtensor* w_down, const dt_dtensor* y, int32_t mode,
                                          int32_t tp_mesh_dim, size_t* bytes);
DT_API dt_status dt_tp_mlp(const dt_dtensor* x, const dt_dtensor* w_gate, const dt_dtensor* w_up,
                    const dt_dtensor* w_down, const dt_dtensor* y, int32_t mode, int32_t tp_mesh_dim,
                    void* workspace, size_t workspace_bytes, int32_t* d_status, dt_stream_t stream);

/*
 * The TP MLP for callers that cannot allocate device memory at call time
 * (for example a serving loop that must not allocate once running, or host
 * code that does not own the device allocator).  Same operands, results and
 * errors as dt_tp_mlp, but H lives in a buffer built into the library: a
 * device array of DT_TP_MLP_STATIC_WORKSPACE_BYTES that every GPU which
 * loads the library holds until the process exits.  This entry point has no
 * counterpart in the pages; it exists for such callers only.
 *  - It allocates nothing (no cudaMalloc, no allocator of any library), and
 *    it runs every GEMM tile whole (it has no split-tail scratch).
 *  - Problems whose H (the [M, F] bf16 blocks described for dt_tp_mlp)
 *    exceeds the array are rejected with DT_ERR_CAPACITY.
 *  - The first call on a device looks up the array's device address on that
 *    device (cudaGetSymbolAddress).  CUDA loads the library's device code
 *    lazily, so that first call is also when the device reserves the
 *    array, and it fails with DT_ERR_CUDA if the device has no room left.
 *    Make the first call on each device at start-up, before memory is
 *    committed elsewhere and before any stream capture.
 *  - All calls share the one array: calls whose kernels overlap on the GPU
 *    (different streams, or different host threads) race on H.  H is fully
 *    rewritten by every call, so nothing needs clearing in between.
 */
#define DT_TP_MLP_STATIC_WORKSPACE_BYTES (32 * 1024 * 1024)
DT_API dt_status dt_tp_mlp_static_workspace(const dt_dtensor* x, const dt_dtensor* w_gate, const dt_dtensor* w_up,
                                            const dt_dtensor* w_down, const dt_dtensor* y, int32_t mode,
                                            int32_t tp_mesh_dim, int32_t* d_status, dt_stream_t stream);

/* ---- between the q/k/v projections and the o projection ----
 *
 * These operators take activations as the column-parallel q/k/v projections
 * leave them: [..., H * head_dim], Shard(-1) on tp (every shard holding whole
 * heads, else DT_ERR_SHAPE) or Replicate on tp (tp_mesh_dim < 0: Replicate
 * everywhere), Replicate on the other mesh dims, leading dims collapsible to
 * one token dim, unit inner stride.  bf16 or fp32; all arithmetic is fp32 and
 * each result is rounded once.  All heads of all shards run in one launch.
 * Outputs must not have materialised replicas.  Tokens (in attention times
 * query heads per kv head) number less than 2^31 - 2^16 (DT_ERR_CAPACITY).
 */

/*
 * Norms of queries and keys for each head, with the position rotation:
 *   z = x / sqrt(mean(x^2) + eps) * weight       (per token and head)
 *   y = z with its first R channels rotated by the angles of row
 *       positions[t] of cos_sin
 *   q, k       [..., Hq * head_dim], [..., Hk * head_dim]; k may be NULL
 *   q_weight, k_weight  [head_dim] Replicate, bf16 or fp32; NULL: no norm
 *   cos_sin    fp32 [rows, R] Replicate: R/2 cosines, then R/2 sines; R even,
 *              at most head_dim; NULL (with positions NULL): no rotation
 *   positions  int32 Replicate, one per token; a position outside
 *              [0, rows) zero-fills its token's outputs and sets
 *              DT_DEV_ERR_INDEX
 *   interleaved  0: channel i is paired with i + R/2; else 2i with 2i + 1
 *   q_out, k_out  shape and dtype of q and k
 * head_dim 2 .. 1024.  Heads of a multiple of 16 channels (rotations too) on
 * 16-byte boundaries run on a vector kernel, all others on a kernel of one
 * element per lane.
 */
DT_API dt_status dt_tp_qk_norm_rope(const dt_dtensor* q, const dt_dtensor* k, const dt_dtensor* q_weight,
                                    const dt_dtensor* k_weight, const dt_dtensor* cos_sin,
                                    const dt_dtensor* positions, const dt_dtensor* q_out, const dt_dtensor* k_out,
                                    int32_t head_dim, float eps, int32_t interleaved, int32_t tp_mesh_dim,
                                    int32_t* d_status, dt_stream_t stream);

/*
 * Its gradients: from dq_out, dk_out (gradients of q_out, k_out) and the
 * forward's inputs,
 *   dq, dk                 gradients of q and k (shape and dtype of q, k)
 *   dq_weight, dk_weight   [head_dim] Replicate, bf16 or fp32: summed over all
 *                          tokens and the heads of all shards, in an order
 *                          fixed by the shapes (the same inputs give the same
 *                          bits); given exactly where the weight is
 * Tokens whose position is out of range get dq = dk = 0 and add nothing.
 * workspace: 256-byte aligned device memory of the queried size for the
 * weights' partial sums (not needed without weights).
 */
DT_API dt_status dt_tp_qk_norm_rope_backward(const dt_dtensor* dq_out, const dt_dtensor* dk_out, const dt_dtensor* q,
                                             const dt_dtensor* k, const dt_dtensor* q_weight,
                                             const dt_dtensor* k_weight, const dt_dtensor* cos_sin,
                                             const dt_dtensor* positions, const dt_dtensor* dq, const dt_dtensor* dk,
                                             const dt_dtensor* dq_weight, const dt_dtensor* dk_weight,
                                             int32_t head_dim, float eps, int32_t interleaved, int32_t tp_mesh_dim,
                                             void* workspace, size_t workspace_bytes, int32_t* d_status,
                                             dt_stream_t stream);
DT_API dt_status dt_tp_qk_norm_rope_backward_workspace_size(int32_t head_dim, size_t* bytes);

/*
 * The paged cache of keys and values in 4 bits: int32
 * [pages, kv heads, page_size, words], Shard(1) on tp (or Replicate), with
 * words = dt_kv4_record_words(head_dim, group); head_dim 64, 128 or 256 in
 * groups of 32 or 64 channels.  The record of one token and kv head:
 *   head_dim/8 words      key codes, nibble i of word w = channel 8 w + i
 *   head_dim/8 words      value codes
 *   head_dim/group words  key parameters, one per group: bf16 step in the
 *                         low half, bf16 minimum in the high half
 *   head_dim/group words  value parameters
 *   padding to a multiple of 4 words
 * A code c stands for minimum + c * step.  Page and head strides are free
 * (multiples of 16 bytes); the records of a page and head are contiguous.
 *
 * The batch, shared by dt_tp_kv4_append and dt_tp_kv4_attention, all int32
 * and Replicate:
 *   page_table [batch, n]     page of keys [i * page_size, (i + 1) * page_size)
 *   kv_lens    [batch]        keys of each sequence, the new tokens included
 *   q_starts   [batch + 1]    rows [q_starts[b], q_starts[b + 1]) of the
 *                             activations are sequence b's new tokens; NULL:
 *                             the same number for each sequence
 * They are read on the device, at the call's turn in its stream: a captured
 * graph replays with new lengths and pages.  New token i of n is key number
 * kv_len - n + i, which is also its position.  Lengths beyond the page table
 * are clamped to it, entries of the page table that are used but are no page
 * are skipped; both set DT_DEV_ERR_INDEX.  Rows of no sequence are not
 * written.
 */
DT_API dt_status dt_kv4_record_words(int32_t head_dim, int32_t group, int32_t* words);

/*
 * Append: the new tokens' keys (rotated) and values into the cache, and the
 * rotated queries into q_out.
 *   k, v       [..., Hkv * head_dim], Hkv = the cache's heads
 *   cos_sin    as in dt_tp_qk_norm_rope, R a multiple of 16; NULL: no
 *              rotation (keys that are rotated already)
 *   q, q_out   [..., Hq * head_dim] or both NULL
 *   k_stored, v_stored  shape and dtype of k, or both NULL: the keys and
 *              values as the cache now holds them, for a prompt whose own
 *              tokens attend to each other outside the cache
 * Per group of a rotated key or a value, in fp32, each operation rounded on
 * its own:
 *   minimum = bf16(min), step = bf16((max - min) * fp32(1/15)),
 *   code = clamp(rint((x - minimum) * (1 / step)), 0, 15)
 * A step below the least normal fp32 number gives codes 0; a group with a
 * value, minimum or step that is not finite is held as NaN.  Tokens whose
 * position lies outside cos_sin are not stored and get zeros in q_out.
 * Rows of k, v, q and the outputs must be 16-byte aligned (DT_ERR_ALIGNMENT).
 */
DT_API dt_status dt_tp_kv4_append(const dt_dtensor* k, const dt_dtensor* v, const dt_dtensor* cache,
                                  const dt_dtensor* page_table, const dt_dtensor* kv_lens, const dt_dtensor* q_starts,
                                  const dt_dtensor* cos_sin, const dt_dtensor* q, const dt_dtensor* q_out,
                                  const dt_dtensor* k_stored, const dt_dtensor* v_stored, int32_t head_dim,
                                  int32_t group, int32_t interleaved, int32_t tp_mesh_dim, int32_t* d_status,
                                  dt_stream_t stream);

/*
 * Attention of each sequence's new tokens over its keys in the cache:
 *   out = softmax(scale * q K^T + mask) V, query head h on kv head h / (Hq / Hkv)
 *   q     [..., Hq * head_dim], Hq a multiple of the cache's heads
 *   out   shape and dtype of q
 *   lse   fp32 [..., Hq], sharded like q's heads, or NULL: the logarithm of
 *         the softmax's denominator (natural, scale included)
 *   causal  0: every key of the sequence; else keys at or before the query's
 *         position; window > 0 (causal only): of those the last `window`
 * A query that sees no key gets out = 0 and lse = -inf.  Whatever the hidden
 * keys, or places of the pages beyond a sequence's length, hold (infinities
 * and NaN too) does not reach the result.  One limit: what fits numbers into
 * fp16 is a power of two for a block of queries (with few rows 8 or 16 of
 * them; with 64 rows or more per sequence and kv head 256).  A key that some
 * queries of a block see and others do not, with finite numbers more than
 * 2^16 times those of the others' keys, takes bits from the others.
 * The softmax and all sums are fp32.  For bf16 activations the products take
 * fp16 operands (11 bits), scaled by powers of two into fp16's range: queries,
 * probabilities times value steps, and with many rows the cache's numbers.
 * For fp32 activations each is three bf16 parts (24 bits).
 * A value group held as NaN makes the results that see it NaN: its channels,
 * and with 64 (query, head) rows per sequence and kv head or more the whole
 * head's (there also for a group whose minimum + 15 steps is beyond fp32).
 * At most 32768 query heads.
 * workspace: 256-byte aligned device memory of the queried size, which
 * depends on the current device; its contents between calls are the
 * caller's.  Waits for copies are bounded (DT_DEV_ERR_TIMEOUT).
 */
DT_API dt_status dt_tp_kv4_attention(const dt_dtensor* q, const dt_dtensor* cache, const dt_dtensor* page_table,
                                     const dt_dtensor* kv_lens, const dt_dtensor* q_starts, const dt_dtensor* out,
                                     const dt_dtensor* lse, int32_t head_dim, int32_t group, float scale,
                                     int32_t causal, int32_t window, int32_t tp_mesh_dim, void* workspace,
                                     size_t workspace_bytes, int32_t* d_status, dt_stream_t stream);
DT_API dt_status dt_tp_kv4_attention_workspace_size(const dt_dtensor* q, const dt_dtensor* cache,
                                                    const dt_dtensor* page_table, int32_t head_dim, int32_t group,
                                                    int32_t tp_mesh_dim, size_t* bytes);

/* ---- between blocks ----
 *
 * Operands of rows: [..., channels], each on its own Replicate or Shard(0) on
 * every mesh dim (so a call may gather or scatter tokens on its way), leading
 * dims collapsible to one token dim, unit inner stride, fewer than 2^31 - 2^16
 * tokens (DT_ERR_CAPACITY).  All arithmetic is fp32 and each result is rounded
 * once.  Outputs must not have materialised replicas.
 */

/*
 * What lies between a block's output and the next block's input, in one pass:
 *   s = x, its parts added in rank order when x is Partial(sum) on tp
 *   u = s / sqrt(mean(s^2) + eps) * post_weight          (norm after the block)
 *   f = keep ? u * gate / (1 - dropout) : 0
 *   h = residual_scale * residual + f
 *   y = h / sqrt(mean(h^2) + eps) * pre_weight           (norm before the next)
 *   x           bf16 or fp32; may be Partial(sum) on tp
 *   residual    x's shape; bf16 or fp32 (fp32 when x is); NULL: none
 *   post_weight [channels] Replicate, bf16 or fp32; NULL: no norm of x
 *   gate        [channels] or [..., channels] Replicate, bf16 or fp32; its rows
 *               divide the tokens, each for as many consecutive ones; NULL: none
 *   pre_weight  [channels] Replicate, given exactly when y is
 *   rng         int32 [4] Replicate, needed with dropout > 0 and read on the
 *               device: a captured graph replays with new ones
 *   h           dtype of the residual (without one bf16 or fp32, fp32 when x
 *               is); NULL: not written
 *   y           dtype of x
 * y comes from h before its rounding.  Element i = token * channels + channel
 * is kept when word i % 4 of Philox4x32-10 at the counter (i / 4 in 64 bits,
 * rng[2], rng[3]) under the key (rng[0], rng[1]) is at least
 * floor(dropout * 2^32): the mask depends on the element alone, not on the
 * layout, and is not stored.  Without post_weight, what a dropped element of x
 * holds reaches nothing.  With eps 0 a row of zeros gives NaN.
 * h may be the residual itself, and y x itself (the same slots and strides).
 */
DT_API dt_status dt_tp_block_norm(const dt_dtensor* x, const dt_dtensor* residual, const dt_dtensor* post_weight,
                                  const dt_dtensor* gate, const dt_dtensor* pre_weight, const dt_dtensor* rng,
                                  const dt_dtensor* h, const dt_dtensor* y, float eps, float residual_scale,
                                  float dropout, int32_t tp_mesh_dim, int32_t* d_status, dt_stream_t stream);

/*
 * Its gradients, from dh and dy (gradients of h and y, of their dtypes; dh may
 * be NULL, dy is given exactly when pre_weight is) and the forward's inputs
 * with the same rng:
 *   dx         shape and dtype of x, Replicate or Shard(0) (every part of a
 *              Partial x has this gradient); NULL: not written
 *   dresidual  dtype of the residual; NULL: not written
 *   dpost_weight, dgate, dpre_weight   shapes of their operands, bf16 or fp32,
 *              given exactly when these are; summed over tokens in an order
 *              fixed by the shapes (the same inputs give the same bits)
 * dx may be x or dy itself, dresidual the residual or dh itself (the same slots
 * and strides).
 * workspace: 256-byte aligned device memory of the queried size (gate_rows 0
 * without a gate) for the sums over tokens; not needed without weights.
 */
DT_API dt_status dt_tp_block_norm_backward(const dt_dtensor* dh, const dt_dtensor* dy, const dt_dtensor* x,
                                           const dt_dtensor* residual, const dt_dtensor* post_weight,
                                           const dt_dtensor* gate, const dt_dtensor* pre_weight, const dt_dtensor* rng,
                                           const dt_dtensor* dx, const dt_dtensor* dresidual,
                                           const dt_dtensor* dpost_weight, const dt_dtensor* dgate,
                                           const dt_dtensor* dpre_weight, float eps, float residual_scale, float dropout,
                                           int32_t tp_mesh_dim, void* workspace, size_t workspace_bytes,
                                           int32_t* d_status, dt_stream_t stream);
DT_API dt_status dt_tp_block_norm_backward_workspace_size(int64_t tokens, int64_t channels, int64_t gate_rows,
                                                          size_t* bytes);

/* ---- behind the head ---- */

/*
 * Log probabilities over a sharded vocabulary, without gathering the logits:
 *   l = log_softmax(scale * logits)
 *   logits        [..., V] bf16 or fp32, Shard(-1) (as a column-parallel head
 *                 leaves them) or Replicate on tp, Replicate on the other mesh
 *                 dims, leading dims collapsible, unit inner stride
 *   ids           int32 [...] or [..., C], C at most 64, Replicate
 *   logprobs      fp32, shape of ids: l at the given ids (both NULL: none)
 *   lse           fp32 [...]: log of the sum of exp(scale * logits); or NULL
 *   entropy       fp32 [...]: -sum exp(l) l; or NULL
 *   top_ids, top_logprobs   int32 and fp32 [..., k], k at most 32: the k largest
 *                 logits, largest first, ties to the lowest id; or both NULL
 * All small tensors are Replicate and contiguous.  scale 2^-20 .. 2^20; with
 * alternatives V is at most 2^24, or 2^21 of 2^28 tokens (DT_ERR_CAPACITY).  An id that is
 * ignore_index gives 0; another one outside [0, V) gives 0 and sets
 * DT_DEV_ERR_INDEX.  Logits may have any finite size (what is beyond fp32 in a
 * result is an infinity); those of -inf have probability 0, a row of nothing else
 * gives lse = -inf, entropy 0 and log probabilities -inf.  A row with NaN or
 * +inf gives NaN (in the order of the alternatives NaN is above all).
 */
DT_API dt_status dt_tp_log_probs(const dt_dtensor* logits, const dt_dtensor* ids, const dt_dtensor* logprobs,
                                 const dt_dtensor* lse, const dt_dtensor* entropy, const dt_dtensor* top_logprobs,
                                 const dt_dtensor* top_ids, float scale, int32_t ignore_index, int32_t tp_mesh_dim,
                                 int32_t* d_status, dt_stream_t stream);

/*
 * The gradient with respect to the logits, from dlogprobs (fp32, shape of ids;
 * both NULL: none), dentropy (fp32 [...]; NULL: none) and what the forward
 * returned (lse; entropy where dentropy is given):
 *   dlogits  shape, dtype and placement of logits; it may be logits itself
 *            (the same slots and strides)
 * Ids that were given twice add up; those that gave 0 above add nothing.  A row
 * whose gradients are all 0, and one whose lse is -inf, get 0 whatever its
 * logits hold.  Probabilities are exp(scale * logits - lse), of an lse in fp32:
 * accurate while |scale * logits| of the likely ones is small against 2^24, where
 * lse's last place is 1; beyond they are off by a factor and may overflow.
 */
DT_API dt_status dt_tp_log_probs_backward(const dt_dtensor* dlogprobs, const dt_dtensor* dentropy,
                                          const dt_dtensor* logits, const dt_dtensor* ids, const dt_dtensor* lse,
                                          const dt_dtensor* entropy, const dt_dtensor* dlogits, float scale,
                                          int32_t ignore_index, int32_t tp_mesh_dim, int32_t* d_status,
                                          dt_stream_t stream);

/* ---- utilities ---- */

/* Static description of a status code. */
DT_API const char* dt_status_string(dt_status status);

/* Reason for the last non-OK status on this thread ("" if none). */
DT_API const char* dt_last_error(void);

/* Copy the library's own device status word (used when d_status == NULL)
 * to *bits and, if clear != 0, reset it.  Synchronous on the current device. */
DT_API dt_status dt_read_device_status(int32_t* bits, int32_t clear);

/* Drop the host-side caches (TMA descriptors, launch plans).  Not to be
 * called while another thread launches. */
DT_API dt_status dt_clear_cache(void);

/* Number of kernels this library has launched in this process so far
 * (every successful launch on any stream counts once). */
DT_API uint64_t dt_launch_count(void);

/* Of those, the launches of the CUDA-core GEMM: linears whose operands are
 * fp32 or whose bf16 pitches or bases TMA cannot describe (row pitch not a
 * multiple of 16 bytes, base not 16-byte aligned) run there, an order of
 * magnitude slower than the tensor cores. */
DT_API uint64_t dt_cuda_core_gemm_count(void);

/* Library version, as major * 10000 + minor * 100 + patch. */
DT_API int32_t dt_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DT_H_ */
