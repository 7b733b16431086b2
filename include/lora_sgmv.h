/*
 * lora_sgmv.h -- C ABI of the GB300 (sm_103a) segmented gather matrix-vector
 * (SGMV) LoRA library.
 *
 * The library adds, for every token row t routed to an adapter slot s,
 *     y_t += B_s . (A_s . x_t)
 * to a projection's base output y ("vLLM LoRA 实现深度解析", section 1: the
 * forward pass h = W0 x + (alpha/r) B A x with the scale folded into B;
 * section 6: output += lora_b_stacked[slot] . lora_a_stacked[slot] . x).
 *
 * Routing follows the triple of the "max.pipelines.lora.LoRAManagerV3" API
 * page (get_lora_graph_inputs): lora_ids and grouped_offsets live on the
 * device, end on the host.  Rows at or past `end` (base requests, which the
 * sort puts last) are never read or written.  Within [0, end) every kernel
 * writes only the rows of the group it is working on; the tensor-core
 * kernels for long groups load whole 128-row boxes of x and y, so they may
 * READ rows of neighbouring groups (never rows at or past `end`: their
 * tensor maps end there).
 *
 * Conventions for every entry point:
 *   - Every buffer is owned by the caller.  No entry point allocates or frees
 *     device memory, and none keeps a pointer after it returns.
 *   - Device work is enqueued on `stream` (a cudaStream_t; NULL is the legacy
 *     default stream) and is asynchronous; host arrays passed in may be reused
 *     as soon as the call returns.
 *   - Arguments are validated on the host before anything is launched; on any
 *     error nothing is launched and the error code is returned.
 *   - The device-side routing arrays are checked by the kernels themselves
 *     (slot range, monotone offsets, first offset 0, last offset == end).  A
 *     violation makes that launch skip ALL of its work, leaves y untouched and
 *     records a flag that lora_get_device_status() returns.
 *   - A CUDA launch failure returns LORA_ERR_CUDA.
 *   - Entry points are thread-safe as far as CUDA itself is; two calls that
 *     write the same y concurrently on different streams race.
 */
#ifndef LORA_SGMV_H
#define LORA_SGMV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t, without pulling in the CUDA headers. */
typedef struct CUstream_st* lora_stream_t;

typedef enum {
  LORA_OK = 0,
  LORA_ERR_NULL = 1,          /* a required pointer is NULL */
  LORA_ERR_SHAPE = 2,         /* a count, size or stride is out of range */
  LORA_ERR_RANK = 3,          /* adapter rank r > max_lora_rank, or r < 0 */
  LORA_ERR_SLOT_RANGE = 4,    /* a slot id < -1 (requests) or >= max_num_loras */
  LORA_ERR_ROUTING = 5,       /* routing triple inconsistent (num_groups, end) */
  LORA_ERR_DTYPE = 6,         /* unknown storage type */
  LORA_ERR_ALIGN = 7,         /* pointer/stride alignment required by the call */
  LORA_ERR_WORKSPACE = 8,     /* workspace NULL or smaller than lora_workspace_bytes() */
  LORA_ERR_CUDA = 9,          /* a CUDA runtime call or kernel launch failed */
  LORA_ERR_TOO_MANY_GROUPS = 10, /* num_groups > max_num_loras ("No free lora slots") */
  LORA_ERR_NO_PAGES = 11       /* not enough free cache pages (lora_pages_append) */
} lora_status_t;

/* Storage type of x, y and the A/B stacks of one problem. */
typedef enum { LORA_DTYPE_F32 = 0, LORA_DTYPE_BF16 = 1 } lora_dtype_t;

/* Flags of the device status word (lora_get_device_status). */
#define LORA_DEV_BAD_SLOT 1u     /* lora_ids[g] outside [0, max_num_loras) */
#define LORA_DEV_BAD_OFFSETS 2u  /* grouped_offsets[0] != 0 or a decreasing offset */
#define LORA_DEV_BAD_END 4u      /* grouped_offsets[num_groups] != end */
#define LORA_DEV_TIMEOUT 8u      /* a kernel gave up (after ~1 s) waiting for its own copies */
#define LORA_DEV_BAD_ROW 16u     /* a token_rows entry outside [0, num_tokens) */
#define LORA_DEV_BAD_PAGE 32u    /* a block-table page or a cache row outside the cache */
#define LORA_DEV_BAD_LENGTH 64u  /* a sequence length below 0 or past its block table */

#define LORA_MAX_SLICES 3

/*
 * One projection slice of a problem.  A and B are the per-slot stacks of the
 * "vLLM LoRA 实现深度解析" page, section 9 (memory layout):
 *   A: slot s block at A + s*A_slot_stride, shape [max_lora_rank, in_dim],
 *      row-major, row stride in_dim (elements).
 *   B: slot s block at B + s*B_slot_stride, shape [out_dim, max_lora_rank],
 *      row-major, row stride max_lora_rank.
 *   y: row t of this slice's output at y + t*y_row_stride, out_dim elements.
 * Strides are in elements.  Fused q/k/v ("MAX max.pipelines.lora 模块解析",
 * load pipeline, QKV fusion: A concatenated on the rank dimension, B on the
 * output dimension) is pure pointer arithmetic on one fused stack:
 *   slice j: A = A_fused + j*R*in_dim, A_slot_stride = n*R*in_dim,
 *            B = B_fused + off_j*R,   B_slot_stride = O*R,
 *            y = y_fused + off_j,      y_row_stride  = O,
 * so slice j's B multiplies only rank columns [jR, (j+1)R) of the
 * intermediate.  Per-projection (unfused) q/k/v is three slices with their
 * own stacks.
 */
typedef struct {
  const void* A;
  int64_t A_slot_stride;
  const void* B;
  int64_t B_slot_stride;
  int32_t out_dim;
  void* y;
  int64_t y_row_stride;
  /* Optional LoRA bias ("MAX max.pipelines.lora 模块解析", LoRA types: BIAS, the
   * bias attached to B; "vLLM LoRA 实现深度解析" section 8, --enable-lora-bias):
   * slot s's vector of out_dim values at bias + s*bias_slot_stride, storage
   * type, added unscaled to every routed row (inside the one rounding).
   * NULL: no bias. */
  const void* bias;
  int64_t bias_slot_stride;
} lora_slice_t;

/*
 * One LoRA problem: a projection input x[num_tokens, in_dim] (row stride
 * x_row_stride elements, rows in sorted-batch order) and 1..3 slices sharing
 * it.  max_num_loras (S) and max_lora_rank (R) are the stack sizes.
 */
typedef struct {
  lora_dtype_t dtype;
  int32_t num_tokens;
  int32_t in_dim;
  int32_t max_num_loras;
  int32_t max_lora_rank;
  const void* x;
  int64_t x_row_stride;
  int32_t num_slices;
  lora_slice_t slices[LORA_MAX_SLICES];
  /* Optional DEVICE int32 [max_num_loras]: the true rank r_s of each slot
   * (0..max_lora_rank), a hint that lets the kernels skip the zero padding:
   * rank columns from ceil16(r_s) on (A rows, B columns) are then never read
   * and contribute nothing; columns [r_s, ceil16(r_s)) must still be zero, as
   * lora_set_slot writes them.  NULL: every slot uses max_lora_rank. */
  const int32_t* slot_ranks;
} lora_problem_t;

/*
 * The routing triple ("max.pipelines.lora.LoRAManagerV3",
 * get_lora_graph_inputs): lora_ids[num_groups] and
 * grouped_offsets[num_groups + 1] are DEVICE int32 arrays; num_groups and end
 * are host values.  Group g covers sorted-batch rows
 * [grouped_offsets[g], grouped_offsets[g+1]) and uses slot lora_ids[g].
 * num_groups == 0 or end == 0 is a valid no-op.  num_groups > max_num_loras
 * returns LORA_ERR_TOO_MANY_GROUPS (a batch needs a slot per group: "No free
 * lora slots", "vLLM LoRA 实现深度解析" section 5.3); other inconsistent host
 * values (end < 0, end > num_tokens, end > 0 with no group) LORA_ERR_ROUTING.
 * The same slot may appear in two groups (each group uses its slot); the
 * routing builder never produces that.
 */
typedef struct {
  const int32_t* lora_ids;
  const int32_t* grouped_offsets;
  int32_t num_groups;
  int32_t end;
  /* Optional, DEVICE int32 [end]: token_rows[i] is the row of x and y that
   * holds the i-th routed token of the sorted order, for batches that are not
   * physically sorted (the per-token slot mapping of "vLLM LoRA 实现深度解析"
   * section 6, whose kernels walk tokens sorted by adapter).  NULL: row i is
   * row i (the sorted batch of the MAX page).  Entries must be distinct and in
   * [0, num_tokens); an entry outside that range makes the launch skip the
   * tiles containing it and raises LORA_DEV_BAD_ROW.  Long gathered groups
   * run on the tcgen05 kernels too (x rows gathered with 16-byte copies, y
   * rows read and written in place); lora_base_gemm_apply refuses token_rows. */
  const int32_t* token_rows;
  /* Optional HOST int32 [num_groups + 1]: the same values as
   * grouped_offsets, read by the call itself (not by the kernels).  With it
   * lora_sgmv_apply picks the kernels per group: groups of at least
   * LORA_TC_MIN_ROWS routed rows on the tensor-core (tcgen05) kernels, the
   * others on the mma.sync kernels, both in the same call.  NULL: one choice
   * per call, from the average group length (end / num_groups).  When given
   * it is checked on the host (entry 0 is 0, entries non-decreasing, entry
   * num_groups equals end; else LORA_ERR_ROUTING). */
  const int32_t* host_grouped_offsets;
  /* Optional HOST int32 [num_groups]: the same values as lora_ids; used only
   * together with host_grouped_offsets (alone: LORA_ERR_NULL), each entry in
   * [0, max_num_loras) (else LORA_ERR_SLOT_RANGE).  With both host copies,
   * lora_sgmv_apply gives its mma.sync shrink a table of its tiles (up to
   * 128 tiles of 64 rows) as a launch parameter: each CTA knows its slot and
   * rows without reading the device triple.  The expand still reads the
   * device triple and checks it against a 64-bit digest of the host copies
   * (SplitMix64 terms per group, summed): a difference raises
   * LORA_DEV_BAD_OFFSETS and the expand skips its work, leaving y as it was
   * (a difference that leaves the digest unchanged goes unseen; for unequal
   * triples that is a chance of about 2^-64).  A CUDA graph that captures the
   * call replays the captured copies: recapture after changing the triple. */
  const int32_t* host_lora_ids;
} lora_routing_t;

/* Routed rows from which a group counts as long (tcgen05 tiles) when the
 * kernels are picked per group. */
#define LORA_TC_MIN_ROWS 64

/*
 * lora_build_routing -- HOST ONLY.  Sort + group ("max.pipelines.lora.
 * LoRAManagerV3", sort_lora_batch and get_lora_graph_inputs).
 *
 * Input: num_requests requests in arrival order, request i on slot
 * req_slot[i] (-1 = base model, else 0..max_num_loras-1) with
 * req_num_tokens[i] >= 0 token rows.
 * Output (caller-allocated host arrays):
 *   perm[num_requests]               sorted order: perm[i] is the arrival index
 *                                    of the i-th request of the sorted batch.
 *                                    Ascending slot, stable, base last.
 *   lora_ids[max_num_loras]          slot of each group (first *num_groups used)
 *   grouped_offsets[max_num_loras+1] first row of each group; entry
 *                                    [*num_groups] equals *end
 *   *num_groups, *end (LoRA-routed rows), *total_tokens (all rows).
 * Consecutive same-slot requests form one group; the walk stops at the first
 * base request.  A zero-token request still opens its slot's group.
 * Errors: LORA_ERR_SHAPE (num_requests < 0, max_num_loras < 1, a negative
 * token count, total rows > INT32_MAX), LORA_ERR_SLOT_RANGE, LORA_ERR_NULL.
 * Outputs are unspecified on error.
 */
lora_status_t lora_build_routing(int32_t num_requests, const int32_t* req_slot,
                                 const int32_t* req_num_tokens, int32_t max_num_loras,
                                 int32_t* perm, int32_t* lora_ids, int32_t* grouped_offsets,
                                 int32_t* num_groups, int32_t* end, int32_t* total_tokens);

/*
 * lora_build_token_rows -- HOST ONLY.  For a batch whose rows are in ARRIVAL
 * order (request i owns rows [start_i, start_i + req_num_tokens[i]), start
 * the running sum in arrival order), write the row of every routed token in
 * the sorted order produced by lora_build_routing: token_rows[0, end) lists
 * the rows of request perm[0], then perm[1], ..., stopping after `end` rows.
 * Pass it (uploaded) as lora_routing_t.token_rows.
 * Errors: LORA_ERR_NULL, LORA_ERR_SHAPE (negative counts, a perm entry out of
 * range, end larger than the rows of the batch).
 */
lora_status_t lora_build_token_rows(int32_t num_requests, const int32_t* req_num_tokens,
                                    const int32_t* perm, int32_t end, int32_t* token_rows);

/*
 * lora_set_slot -- load-time preparation of one adapter slot for one slice
 * ("MAX max.pipelines.lora 模块解析", load pipeline: scale pre-multiplied into
 * B, rank padding, dtype unification; "vLLM LoRA 实现深度解析" section 1,
 * scale alpha/r or alpha/sqrt(r) with rsLoRA, and section 5.3 set_lora).
 *
 * Writes slot `slot` of slice `slice` of the stacks described by `problem`
 * (the stacks must be writable device memory):
 *   A[slot, k, i] = A_raw[k, i]                        for k < r, else 0
 *   B[slot, o, k] = rne(fp32(B_raw[o, k]) * scale)     for k < r, else 0
 * where scale = fp32(lora_alpha / r), or fp32(lora_alpha / sqrt(r)) when
 * use_rslora != 0, computed in double on the host; the product is formed in
 * fp32 and rounded once (round to nearest even) to problem->dtype.
 * A_raw [r, in_dim] and B_raw [out_dim, r] are contiguous DEVICE arrays of
 * raw_dtype (fp32 or bf16).  r == 0 zeroes the slot (A_raw/B_raw may be NULL).
 * Errors: LORA_ERR_RANK (r < 0 or r > max_lora_rank), LORA_ERR_SLOT_RANGE,
 * LORA_ERR_SHAPE (slice out of range, bad dims), LORA_ERR_NULL, LORA_ERR_DTYPE.
 */
lora_status_t lora_set_slot(const lora_problem_t* problem, int32_t slice, int32_t slot, int32_t r,
                            double lora_alpha, int32_t use_rslora, const void* A_raw,
                            const void* B_raw, lora_dtype_t raw_dtype, lora_stream_t stream);

/*
 * lora_set_slot_bias -- load-time preparation of slot `slot`'s bias for slice
 * `slice`: bias[slot, o] = cast(bias_raw[o]) (round to nearest even), or zero
 * when bias_raw is NULL.  bias_raw is a contiguous DEVICE array of out_dim
 * values of raw_dtype.  The slice's bias pointer must be set.
 * Errors: LORA_ERR_NULL (no bias stack), LORA_ERR_SLOT_RANGE, LORA_ERR_SHAPE,
 * LORA_ERR_DTYPE.
 */
lora_status_t lora_set_slot_bias(const lora_problem_t* problem, int32_t slice, int32_t slot,
                                 const void* bias_raw, lora_dtype_t raw_dtype, lora_stream_t stream);

/*
 * lora_shrink -- u[t, j*R + k] = sum_i A_j[lora_ids[g], k, i] * x[t, i] for
 * every routed row t < end (group g), slice j, k < R.  u is a DEVICE fp32
 * array [end, num_slices*R] (row stride num_slices*R), fully overwritten.
 * Products of the stored values are exact; sums are fp32.
 */
lora_status_t lora_shrink(const lora_problem_t* problem, const lora_routing_t* routing, float* u,
                          lora_stream_t stream);

/*
 * lora_expand -- boundary-aware expand: y_j[t, o] = rn(y_j[t, o] +
 * bias_j[s, o] + sum_k B_j[s, o, k] * u[t, j*R + k]) with s = lora_ids[g]
 * (bias only when the slice has one) for routed rows t < end only,
 * with one rounding to the storage type.  u as produced by lora_shrink.
 * Accumulation is fp32.  On the bf16 tensor-core path u enters the product as
 * two bf16 terms (u = hi + lo, 16 significant bits, the split is exact);
 * elsewhere it enters as fp32.
 */
lora_status_t lora_expand(const lora_problem_t* problem, const lora_routing_t* routing,
                          const float* u, lora_stream_t stream);

/*
 * Bytes of device workspace lora_sgmv_apply needs for `end` routed rows: for
 * max_lora_rank 64 or 128 the packed intermediate of the tensor-core path
 * ((max_num_loras + end / 128) tiles x n*R x 512 bytes), then room for the
 * fp32 intermediate (up to 16 partial planes of end x n*R); both are live
 * when the kernels are picked per group.  Depends on shapes only.
 */
size_t lora_workspace_bytes(const lora_problem_t* problem, int32_t end);

/*
 * lora_sgmv_apply -- shrink then expand in one call; the intermediate lives in
 * `workspace` (DEVICE, >= lora_workspace_bytes(problem, end) bytes, 16-byte
 * aligned, contents on entry ignored): fp32 partial planes, or, on the
 * tensor-core path (bf16, rank 64 or 128, long groups), u already split into
 * bf16 hi + lo terms and laid out as the expand's operand per 128-row tile.
 * The expand is launched as a programmatic dependent of the shrink, so its
 * weight and y loads overlap the shrink.  With the routing's host copy of
 * the offsets (host_grouped_offsets), a batch mixing long and short groups
 * runs both kernel families in the one call, each on its own groups.  Two
 * calls whose kernels may overlap on the GPU need two workspaces.
 */
lora_status_t lora_sgmv_apply(const lora_problem_t* problem, const lora_routing_t* routing,
                              void* workspace, size_t workspace_bytes, lora_stream_t stream);

/*
 * lora_sgmv_apply_noalloc -- lora_sgmv_apply for callers that cannot allocate
 * device memory.  The pages have no counterpart to this entry point.
 *
 * Some callers cannot call cudaMalloc: plug-ins living inside a host
 * framework that owns every device allocation (and gives them none), or
 * latency-critical loops where an allocation could stall or fail.  This call
 * takes no workspace argument and allocates nothing; the fp32 intermediate
 * lives in a fixed array of LORA_NOALLOC_MAX_WORKSPACE_BYTES compiled into the
 * library (every GPU that loads the library holds it until the process exits).
 *
 * Same problem, routing, results and errors as lora_sgmv_apply, plus:
 *   - LORA_ERR_WORKSPACE if the fp32 intermediate, end x n*R x 4 bytes
 *     rounded up to 256, exceeds LORA_NOALLOC_MAX_WORKSPACE_BYTES (use
 *     lora_sgmv_apply with your own workspace for such batches).
 *   - The first call on a device looks up the array's device address (with
 *     that device current) and caches it; LORA_ERR_CUDA if the lookup fails.
 *     Make that first call before any stream capture.
 *   - Every call on a device shares the one array and leaves its own
 *     intermediate in it.  Nothing has to start at zero (each call writes
 *     every value it later reads), but calls whose GPU work overlaps -- on
 *     different streams, or from different threads -- race on the array.
 *     Serialize them (one stream, or events).
 */
#define LORA_NOALLOC_MAX_WORKSPACE_BYTES (16u * 1024u * 1024u)
lora_status_t lora_sgmv_apply_noalloc(const lora_problem_t* problem, const lora_routing_t* routing,
                                      lora_stream_t stream);

/* Base projection weight of one slice: W0 [out_dim, in_dim] in the
 * problem's storage type, row o at W0 + o * row_stride (elements). */
typedef struct {
  const void* W0;
  int64_t row_stride;
} lora_base_weight_t;

/*
 * lora_base_gemm_apply -- the LoRA delta fused into the base projection
 * ("vLLM LoRA 实现深度解析" section 1: h = W0 x + (alpha/r) B A x, the scale
 * folded into B):
 *   y_j[t, o] = rn( sum_i W0_j[o, i] x[t, i]
 *                   + [t < end] (bias_j[s, o] + sum_k B_j[s, o, k] u[t, j*R + k]) )
 * for EVERY row t < num_tokens and every slice j (s: the slot of t's group;
 * base rows get the base product alone), with one rounding to the storage
 * type.  y is written, never read: the delta joins the base product in the
 * accumulator instead of a read-modify-write of y.  base[num_slices] gives
 * each slice's W0 (DEVICE).  The shrink writes u into `workspace` as for
 * lora_sgmv_apply (same size; NULL allowed when
 * num_groups or end is 0).  Rows must be in sorted order: token_rows is
 * refused (LORA_ERR_SHAPE).
 * Kernels: bf16 fast-path shapes (16-byte aligned W0, row stride a multiple
 * of 8) run a tcgen05 GEMM whose K loop ends with the delta as extra K
 * steps (u = hi + lo as bf16 terms against the slot's B block, per group
 * overlapping a 128-row tile); other shapes a generic kernel.
 * Errors: as lora_sgmv_apply, plus LORA_ERR_NULL (base or a W0 missing),
 * LORA_ERR_SHAPE (a row stride below in_dim, token_rows given).
 */
lora_status_t lora_base_gemm_apply(const lora_problem_t* problem, const lora_routing_t* routing,
                                   const lora_base_weight_t* base, void* workspace, size_t workspace_bytes,
                                   lora_stream_t stream);

/*
 * 4-bit base projection weight of one slice, W0 [out_dim, in_dim]:
 *   W0[o, i] = scales[o, i / group_size] * (code[o, i] - zeros[o, i / group_size])
 * code[o, i], 0..15, is the low half of byte q[o*q_row_stride + i / 2] for an
 * even i and its high half for an odd one; scales has the problem's storage
 * type (row stride in elements), zeros bytes of 0..255 (NULL: 8 everywhere).
 * A row has ceil(in_dim / group_size) groups, the last one maybe short; a
 * group_size of in_dim or more is one group a row.
 */
typedef struct {
  const uint8_t* q;
  int64_t q_row_stride;
  const void* scales;
  int64_t scale_row_stride;
  const uint8_t* zeros;
  int64_t zero_row_stride;
  int32_t group_size;
} lora_q4_weight_t;

/*
 * lora_base_q4_apply -- lora_base_gemm_apply on 4-bit base weights, for the
 * few rows of a decode or verification step (any number is taken; W0 is
 * unpacked anew for every 32 rows of a small batch, every 128 of a large one):
 *   y_j[t, o] = rn( sum_i W0_j[o, i] x[t, i]
 *                   + [t < end] (bias_j[s, o] + sum_k B_j[s, o, k] u[t, j*R + k]) )
 * for every row t < num_tokens, y written and never read, one rounding.  A
 * weight is never rounded to the storage type: codes less their zero are exact
 * in the products, a group's sum is fp32 and takes its scale there.
 * base[num_slices] gives each slice's W0 (DEVICE).  workspace as for
 * lora_base_gemm_apply; token_rows is refused likewise.
 * Kernels: bf16 with in_dim a multiple of 32, R up to 256, group sizes of a
 * multiple of 32 (or one group a row), x and q on 16-byte boundaries with rows
 * of such strides, and scales that fit shared memory (some 1000 groups a row)
 * run on the tensor cores, large batches in groups of a multiple of 64 on
 * tcgen05; others on a generic kernel.  An infinity or NaN in a row of x or in
 * a slot's B stays with the rows concerned.
 * Errors: as lora_base_gemm_apply (LORA_ERR_SHAPE also for a group_size < 1 or
 * row strides below the row's bytes or groups; LORA_ERR_ALIGN for scales off
 * their element's boundary).
 */
lora_status_t lora_base_q4_apply(const lora_problem_t* problem, const lora_routing_t* routing,
                                 const lora_q4_weight_t* base, void* workspace, size_t workspace_bytes,
                                 lora_stream_t stream);

/* ==========================================================================
 * Attention between the projections: what a served layer does with the
 * q/k/v rows that lora_sgmv_apply or lora_base_gemm_apply leaves, before the
 * o_proj call.  The pages have no counterpart; the conventions at the top of
 * this file hold (caller-owned buffers, host validation before any launch,
 * device arrays checked by the kernels, the status word).
 * ========================================================================== */

/* Widest head of the calls below. */
#define LORA_MAX_HEAD_DIM 256

/* A [rows, heads, head_dim] view: element (r, h, d) at
 * data + r*row_stride + h*head_stride + d (strides in elements).  The q part
 * of a fused q/k/v output y is {y, y_row_stride, head_dim}, its k part
 * {y + n_heads*head_dim, y_row_stride, head_dim}. */
typedef struct {
  void* data;
  int64_t row_stride;
  int64_t head_stride;
} lora_heads_t;

/*
 * One layer's paged key/value cache.  Element (page p, token o of the page,
 * head h, d) of K is k[p*page_stride + o*token_stride + h*head_stride + d]
 * (elements), V the same from v.  Token-major pages ([pages, page_size,
 * heads, head_dim]) and head-major ones ([pages, heads, page_size, head_dim])
 * are both such views, as is one pool that holds K and V side by side.  The
 * strides may leave gaps but no two elements may share an address
 * (LORA_ERR_SHAPE).  "Cache row" c is token c % page_size of page
 * c / page_size; num_pages * page_size is at most INT32_MAX.  Offsets are
 * formed in 64 bits.
 */
typedef struct {
  lora_dtype_t dtype;
  int32_t num_pages;
  int32_t page_size;
  int32_t num_kv_heads;
  int32_t head_dim;
  void* k;
  void* v;
  int64_t page_stride;
  int64_t token_stride;
  int64_t head_stride;
} lora_kv_cache_t;

/* How the frequencies of lora_build_rope are scaled for long contexts. */
typedef enum {
  LORA_ROPE_NONE = 0,
  LORA_ROPE_LINEAR = 1,  /* position interpolation: f / factor */
  LORA_ROPE_NTK = 2,     /* base theta * factor^(D / (D - 2)), D = rotary_dim >= 4 */
  LORA_ROPE_PARTS = 3    /* by parts: g f + (1 - g) f / factor with
                            g = clamp((n - low_turns) / (high_turns - low_turns), 0, 1),
                            n = original_max_positions * f / (2 pi), the turns the
                            pair makes over the original context */
} lora_rope_scaling_t;

/*
 * lora_build_rope -- HOST ONLY.  The frequency of each rotated pair i <
 * rotary_dim / 2, f_i = theta^(-2 i / rotary_dim) radians per position (or
 * frequencies[i], when that HOST array of rotary_dim / 2 values is given),
 * scaled, as a 64-bit fixed-point fraction of a turn:
 *   turns[i] = floor(frac(f_i / (2 pi)) * 2^64).
 * position * turns[i] modulo 2^64 is then the angle's fractional turn with
 * no range reduction; the entry's own rounding, that of a double (2^-55 of a
 * turn), is all that grows with the position.  Upload it for
 * lora_rope_t.turns.  Errors: LORA_ERR_SHAPE (rotary_dim odd, < 2 or >
 * LORA_MAX_HEAD_DIM; theta or factor not positive and finite; NTK with
 * frequencies given or rotary_dim < 4; PARTS with original_max_positions < 1
 * or high_turns <= low_turns; a frequency, or the NTK base, that is not finite
 * as given or as scaled; an unknown scaling), LORA_ERR_NULL.
 */
lora_status_t lora_build_rope(int32_t rotary_dim, double theta, lora_rope_scaling_t scaling, double factor,
                              int32_t original_max_positions, double low_turns, double high_turns,
                              const double* frequencies, uint64_t* turns);

/* Which two elements of a head form pair i of the rotation. */
typedef enum {
  LORA_ROPE_HALVES = 0,     /* i and i + rotary_dim / 2 */
  LORA_ROPE_INTERLEAVED = 1 /* 2 i and 2 i + 1 */
} lora_rope_layout_t;

/* One lora_rope_append call; every pointer is DEVICE memory. */
typedef struct {
  lora_dtype_t dtype;    /* q, k, v, their outputs, the norm weights and the cache */
  int32_t num_tokens;
  int32_t num_heads;     /* query heads, 0: no q */
  int32_t num_kv_heads;  /* key (and value) heads, 0: no k */
  int32_t head_dim;
  int32_t rotary_dim;    /* first rotary_dim elements of a head rotate (even, 0..head_dim) */
  lora_rope_layout_t layout;
  float attention_scale; /* factor on the rotated elements (YaRN's sqrt(1/t)); 1 normally */
  float eps;             /* of the norms */
  const uint64_t* turns;     /* [rotary_dim / 2], lora_build_rope */
  const int32_t* positions;  /* [num_tokens], any sign */
  lora_heads_t q, k, v;      /* inputs; v only with cache rows */
  lora_heads_t q_out;        /* may be q itself */
  lora_heads_t k_out;        /* optional (data NULL: none); may be k itself */
  const void* q_weight;      /* optional [head_dim]: RMS norm of each query head */
  const void* k_weight;      /* optional [head_dim]: RMS norm of each key head */
  const int32_t* cache_rows; /* optional [num_tokens]: cache row of each token, -1: none */
} lora_rope_t;

/*
 * lora_rope_append -- one pass over the q/k/v rows of a batch.  For every
 * token and head, in fp32 with one rounding to the storage type:
 *   n = x * rsqrt(mean(x^2) + eps) * weight     (over head_dim; weight given)
 *   pair i of the rotated part: (a, b) -> s (a cos - b sin, a sin + b cos)
 * with s = attention_scale and the angle position * f_i; elements from
 * rotary_dim on are n unchanged.  q goes to q_out, k to k_out (if given) and
 * to cache row cache_rows[t] of K, v unchanged to the same row of V.  Cache
 * rows must be distinct; a row below -1 or past the cache is not stored and
 * raises LORA_DEV_BAD_PAGE.  cache may be NULL exactly when cache_rows is.
 * q_out (k_out) may be q (k) itself, with the same strides, but must not
 * overlap the inputs otherwise.  num_tokens == 0 is a valid no-op.
 * Errors: LORA_ERR_NULL, LORA_ERR_DTYPE (an unknown type, a cache of another),
 * LORA_ERR_SHAPE (sizes, a negative input stride, output strides that let two
 * elements share an address, a cache whose heads or head_dim differ),
 * LORA_ERR_ALIGN (a pointer that is not on its element's boundary).
 */
lora_status_t lora_rope_append(const lora_rope_t* rope, const lora_kv_cache_t* cache, lora_stream_t stream);

/* One lora_paged_attention call; every pointer is DEVICE memory. */
typedef struct {
  int32_t num_seqs;   /* rows of q and out */
  int32_t num_heads;  /* a multiple of the cache's num_kv_heads: head h reads key/value head
                         h / (num_heads / num_kv_heads) */
  lora_heads_t q;     /* the cache's type */
  lora_heads_t out;   /* the cache's type; may be q itself */
  const int32_t* block_tables; /* row b lists the pages of sequence b in order */
  int64_t table_stride;        /* entries from one row to the next */
  int32_t max_pages;           /* entries of a row */
  const int32_t* lengths;      /* [num_seqs]: cached tokens, the new one's included */
  float scale;                 /* of the scores, usually 1 / sqrt(head_dim) */
  float* lse;                  /* optional [num_seqs, num_heads]: log of the scores' exponential sum */
} lora_attention_t;

/*
 * lora_attention_workspace_bytes -- DEVICE workspace of lora_paged_attention:
 * the partial results of contexts that several CTAs share.  Depends on
 * shapes only; 0 for arguments that the call would refuse.
 */
size_t lora_attention_workspace_bytes(const lora_attention_t* attention, const lora_kv_cache_t* cache);

/*
 * lora_paged_attention -- attention of one new token per sequence to its
 * cached tokens: out_h = sum_j p_j v_j / sum_j p_j, p_j = exp(scale q_h . k_j),
 * over j < lengths[b].  A sequence of length 0 (a padding entry of a batch)
 * gives out = 0 and lse = -inf, as does a row whose every score is -inf.
 * Scores, softmax sums and the output's accumulation are fp32; on the bf16
 * tensor-core path (pages of a multiple of 8 tokens, rows of cache and q on
 * 16-byte boundaries) the probabilities enter the product with V as three
 * bf16 terms, whose sum has fp32's 24 bits.  Cached values past a sequence's
 * end and block-table entries past its last page are never used.  A length
 * below 0 or above max_pages * page_size raises LORA_DEV_BAD_LENGTH, a used
 * page id outside the cache LORA_DEV_BAD_PAGE; that sequence's rows of out and
 * lse are left as they were, the others are computed.  The cached tokens are
 * shared out evenly over the GPU whatever the lengths; the same lengths, with
 * tables of the same width on the same GPU, give the same bits.
 * workspace: >= lora_attention_workspace_bytes, 16-byte aligned, contents on
 * entry ignored; two calls that may overlap need two.
 * Errors: LORA_ERR_NULL, LORA_ERR_DTYPE, LORA_ERR_SHAPE, LORA_ERR_WORKSPACE,
 * LORA_ERR_ALIGN.
 */
lora_status_t lora_paged_attention(const lora_attention_t* attention, const lora_kv_cache_t* cache,
                                   void* workspace, size_t workspace_bytes, lora_stream_t stream);

/* Most 64-bit words of a tree mask row. */
#define LORA_MAX_MASK_WORDS 16

/*
 * lora_build_tree -- HOST ONLY.  The mask and depth of each node of a tree of
 * drafted tokens: parents[i] in [-1, i) (-1: the node hangs on the context's
 * end).  masks[i * mask_words + w], bit j: node 64 w + j is i itself or one of
 * its ancestors.  depths[i]: ancestors of i, so the token's position is the
 * context's length plus depths[i].  Either output may be NULL.  Errors:
 * LORA_ERR_NULL, LORA_ERR_SHAPE (num_nodes < 0, a parent out of range,
 * mask_words not in [1, LORA_MAX_MASK_WORDS] or too few for num_nodes).
 */
lora_status_t lora_build_tree(int32_t num_nodes, const int32_t* parents, int32_t mask_words, uint64_t* masks,
                              int32_t* depths);

/* One lora_tree_attention call; every pointer is DEVICE memory.  Sequence b
 * has the rows row_offsets[b] to row_offsets[b + 1] - 1 of q and out, one for
 * each of its drafted tokens, whose keys and values are the last tokens of its
 * lengths[b] cached ones, in the same order.  What is cached before them is
 * its context. */
typedef struct {
  int32_t num_seqs;
  int32_t num_rows;   /* rows of q, out, masks and lse; those behind the last sequence's are left as they were */
  int32_t num_heads;  /* a multiple of the cache's num_kv_heads */
  lora_heads_t q;     /* the cache's type */
  lora_heads_t out;   /* the cache's type; may be q itself */
  const int32_t* block_tables; /* row b lists the pages of sequence b in order */
  int64_t table_stride;
  int32_t max_pages;
  const int32_t* lengths;     /* [num_seqs]: cached tokens, the drafted ones included */
  const int32_t* row_offsets; /* [num_seqs + 1], not decreasing, within [0, num_rows] */
  const uint64_t* masks;      /* [num_rows, mask_words]: bit j of a row names drafted token j of its sequence;
                                 NULL: a chain, row i sees drafted tokens 0..i */
  int32_t mask_words;         /* 1..LORA_MAX_MASK_WORDS; not read without masks */
  float scale;
  float* lse;                 /* optional [num_rows, num_heads] */
} lora_tree_attention_t;

/* DEVICE workspace of lora_tree_attention.  Depends on shapes only; 0 for
 * arguments that the call would refuse. */
size_t lora_tree_attention_workspace_bytes(const lora_tree_attention_t* attention, const lora_kv_cache_t* cache);

/*
 * lora_tree_attention -- attention of the drafted tokens of each sequence to
 * its context and to the drafted tokens that each one's mask names:
 * out_h = sum_j p_j v_j / sum_j p_j, p_j = exp(scale q_h . k_j) over what the
 * row sees.  Mask bits of tokens that the sequence does not have are ignored.
 * A row that sees nothing, or whose every score is -inf, gives out = 0 and
 * lse = -inf.  What a row does not see has no part in it, be it infinite or
 * NaN.  Scores, softmax sums and the output's accumulation are fp32; on the
 * tensor-core path (bf16; rows of cache, q and out on 16-byte boundaries) the
 * probabilities enter the product with V with fp32's 24 bits, as three bf16
 * terms.  An infinite value that a row sees with a probability of 0 in fp32 may
 * make its column NaN.  A sequence without rows reads nothing.  A length below
 * the sequence's rows or above max_pages * page_size, or more rows than the
 * masks have bits, raises LORA_DEV_BAD_LENGTH, a used page id outside the cache LORA_DEV_BAD_PAGE; that
 * sequence's rows of out and lse are left as they were, the others are
 * computed.  Row offsets that decrease or leave [0, num_rows] raise
 * LORA_DEV_BAD_OFFSETS and nothing is computed.  The same arguments give the
 * same bits on the same GPU.
 * workspace: >= lora_tree_attention_workspace_bytes, 16-byte aligned, contents
 * on entry ignored; two calls that may overlap need two.
 * Errors: LORA_ERR_NULL, LORA_ERR_DTYPE, LORA_ERR_SHAPE, LORA_ERR_WORKSPACE,
 * LORA_ERR_ALIGN.
 */
lora_status_t lora_tree_attention(const lora_tree_attention_t* attention, const lora_kv_cache_t* cache,
                                  void* workspace, size_t workspace_bytes, lora_stream_t stream);

/* Most entries of a path of lora_kv_keep_rows. */
#define LORA_MAX_KEPT 1024

/* One lora_kv_keep_rows call; every pointer is DEVICE memory.  block_tables,
 * lengths and row_offsets as in lora_tree_attention_t. */
typedef struct {
  int32_t num_seqs;
  const int32_t* block_tables;
  int64_t table_stride;
  int32_t max_pages;
  const int32_t* lengths;
  const int32_t* row_offsets;
  const int32_t* path;  /* [num_seqs, max_kept]: the drafted tokens to keep, ascending; -1 ends a row */
  int64_t path_stride;
  int32_t max_kept;     /* 0..LORA_MAX_KEPT */
  int32_t* new_lengths; /* optional [num_seqs]: context + kept tokens; must not overlap lengths */
} lora_keep_t;

/*
 * lora_kv_keep_rows -- after a verification: in every one of num_caches caches
 * (the layers of a model: same geometry and type) the K and V of drafted token
 * path[b][k] of sequence b become those of its cached token context + k, for
 * every k before the row's first -1, as if all were read before any is
 * written.  The sequence then has new_lengths[b] tokens; what its pages hold
 * behind them is unspecified (lora_pages_trim gives the pages back).  Copies
 * are exact, gaps between strided rows are not touched.  Pages that are
 * written must not be shared (lora_pages_append saw to that).  A sequence
 * without drafted tokens keeps its length, which is not looked at.  Another's
 * length that lora_tree_attention would refuse, or offsets that are negative or
 * decrease, raise LORA_DEV_BAD_LENGTH, a path
 * that does not ascend or names a token that the sequence does not have
 * LORA_DEV_BAD_ROW, a used page outside the cache LORA_DEV_BAD_PAGE; that
 * sequence and its new length are left as they were.
 * No tensor may be listed twice or overlap another.
 * Errors: LORA_ERR_NULL, LORA_ERR_DTYPE, LORA_ERR_SHAPE (also a K or V listed
 * twice), LORA_ERR_ALIGN, LORA_ERR_WORKSPACE (no host memory to check a long
 * list).
 */
lora_status_t lora_kv_keep_rows(const lora_kv_cache_t* caches, int32_t num_caches, const lora_keep_t* keep,
                                lora_stream_t stream);

/*
 * lora_kv_copy_pages -- K and V of page dst[i] become those of page src[i],
 * for every i < num_copies and every one of num_caches caches (the layers of
 * a model: same geometry and type, else LORA_ERR_SHAPE).  src and dst are
 * HOST arrays, read by the call.  A source may repeat (one page to many
 * forks); a destination may not, nor be a source as well: the copies have no
 * order among themselves (LORA_ERR_SHAPE, as for a page outside the caches).
 * Gaps between strided rows are not touched.  Copies are exact, whatever the
 * values.  Errors also: LORA_ERR_NULL, LORA_ERR_DTYPE, LORA_ERR_ALIGN,
 * LORA_ERR_WORKSPACE (no host memory to check a long list).
 */
lora_status_t lora_kv_copy_pages(const lora_kv_cache_t* caches, int32_t num_caches, const int32_t* src,
                                 const int32_t* dst, int32_t num_copies, lora_stream_t stream);

/*
 * Which page holds what: HOST bookkeeping of one cache's pages, in arrays
 * that the caller owns.  Pages are counted by reference, so forked sequences
 * share them; a shared page that is only partly filled is copied before
 * either sequence writes to it (copy on write).  The calls below change these
 * arrays alone; they return the page copies to run with lora_kv_copy_pages,
 * enqueued before the rows are written.  On an error nothing is changed.
 * Not thread-safe on one set of arrays.
 */
typedef struct {
  int32_t num_pages;
  int32_t page_size;
  int32_t max_seqs;
  int32_t max_pages;   /* of one sequence */
  int32_t* tables;     /* [max_seqs, max_pages] block tables; -1 past a sequence's last page */
  int32_t* lengths;    /* [max_seqs] tokens; 0: not in use */
  int32_t* refs;       /* [num_pages] sequences that hold the page */
  int32_t* free_pages; /* [num_pages] stack of free pages, the next one at num_free - 1 */
  int32_t num_free;
} lora_pages_t;

/* Every page free, every sequence empty.  LORA_ERR_NULL; LORA_ERR_SHAPE (a
 * size < 1, num_pages * page_size > INT32_MAX). */
lora_status_t lora_pages_init(lora_pages_t* pages);

/*
 * num_tokens >= 0 more tokens of sequence seq: takes pages as needed and
 * writes the cache row of each new token to rows[num_tokens] (NULL allowed
 * when num_tokens is 0).  *copy_src / *copy_dst: a page copy to run first, or
 * -1 (at most one: the sequence's last page, when shared and partly filled).
 * LORA_ERR_SHAPE: seq out of range, a negative count, more than max_pages
 * pages.  LORA_ERR_NO_PAGES: not enough free pages.
 */
lora_status_t lora_pages_append(lora_pages_t* pages, int32_t seq, int32_t num_tokens, int32_t* rows,
                                int32_t* copy_src, int32_t* copy_dst);

/* The empty sequence child becomes the first num_tokens of parent, sharing
 * its pages.  LORA_ERR_SHAPE: a sequence out of range, child not empty,
 * num_tokens < 0 or above the parent's. */
lora_status_t lora_pages_fork(lora_pages_t* pages, int32_t parent, int32_t child, int32_t num_tokens);

/* Keeps the first num_tokens of seq (0: the sequence ends) and gives the pages
 * behind them back.  LORA_ERR_SHAPE: seq or num_tokens out of range. */
lora_status_t lora_pages_trim(lora_pages_t* pages, int32_t seq, int32_t num_tokens);

/*
 * Moves every page in use below the count of pages in use and rewrites the
 * block tables: src[i] -> dst[i] for i < *num_copies are the copies to run
 * (src and dst hold up to num_pages / 2 entries; no page is in both lists).
 */
lora_status_t lora_pages_compact(lora_pages_t* pages, int32_t* src, int32_t* dst, int32_t* num_copies);

/*
 * lora_get_device_status -- reads and clears, in one atomic exchange ordered
 * after the work already on `stream`, the device status word of the current
 * device (an OR of LORA_DEV_* flags from every launch since the last read,
 * on any stream), then synchronizes `stream` and returns the flags.  A flag
 * raised by a kernel on another stream is never lost: it is either returned
 * by this call or kept for the next.  Returns LORA_ERR_CUDA if the exchange,
 * the copy or the synchronization fails.
 */
lora_status_t lora_get_device_status(lora_stream_t stream, uint32_t* flags);

/*
 * Kernel families (bits of lora_last_call_path).  The pages have no
 * counterpart; this is an introspection aid for tests and profiling.
 */
#define LORA_PATH_GENERIC_SHRINK 0x1u  /* one warp per u element (fp32, odd shapes) */
#define LORA_PATH_GENERIC_EXPAND 0x2u  /* one thread per y element */
#define LORA_PATH_MMA_SHRINK 0x4u      /* mma.sync shrink (short groups) */
#define LORA_PATH_MMA_EXPAND 0x8u      /* mma.sync expand (short groups) */
#define LORA_PATH_TC_SHRINK 0x10u      /* tcgen05 + TMA shrink (long groups) */
#define LORA_PATH_TC_EXPAND 0x20u      /* persistent tcgen05 + TMA expand (long groups) */
#define LORA_PATH_PREP 0x80u           /* load-time slot / bias preparation */
#define LORA_PATH_BASE_GEMM 0x100u     /* base projection GEMM with the delta as K tail */
#define LORA_PATH_ROPE 0x200u          /* norm + rotation + cache append, 16-byte accesses */
#define LORA_PATH_GENERIC_ROPE 0x400u  /* the same, element by element (odd shapes) */
#define LORA_PATH_MMA_ATTENTION 0x800u /* paged attention on mma.sync (bf16) */
#define LORA_PATH_GENERIC_ATTENTION 0x1000u /* paged attention in fp32 arithmetic */
#define LORA_PATH_JOIN 0x2000u         /* join of the contexts that CTAs shared */
#define LORA_PATH_PAGES 0x4000u        /* page copies */
#define LORA_PATH_MMA_Q4 0x8000u       /* 4-bit base projection on mma.sync */
#define LORA_PATH_GENERIC_Q4 0x10000u  /* 4-bit base projection in fp32 arithmetic */
#define LORA_PATH_TC_TREE 0x20000u     /* tree attention on tcgen05 (bf16) */
#define LORA_PATH_GENERIC_TREE 0x40000u /* tree attention in fp32 arithmetic */
#define LORA_PATH_KEEP 0x80000u        /* kept cache rows */
#define LORA_PATH_TC_Q4 0x100000u      /* 4-bit base projection on tcgen05 */

/*
 * lora_last_call_path -- the OR of LORA_PATH_* bits of the kernels launched
 * by the most recent entry-point call made on the calling host thread (0 if
 * it launched nothing: a no-op, or an error before any launch), and, when
 * num_launches is not NULL, how many kernels that call launched.  Host only;
 * reads thread-local state, no CUDA call.
 */
uint32_t lora_last_call_path(uint32_t* num_launches);

/*
 * lora_selftest_wait_timeout -- exercises the failure path of the pipelined
 * kernels without faulting the GPU (no counterpart on the pages).  One thread
 * waits on a fresh shared-memory barrier that nothing completes, gives up
 * after `polls` polls of mbarrier.try_wait (bounded), sets LORA_DEV_TIMEOUT
 * in the device status word and exits; the context stays usable.  Read the
 * flag with lora_get_device_status.  Returns LORA_ERR_CUDA if the launch
 * fails.
 */
lora_status_t lora_selftest_wait_timeout(uint32_t polls, lora_stream_t stream);

/* Static, human-readable name of a status code. */
const char* lora_status_string(lora_status_t status);

#ifdef __cplusplus
}
#endif

#endif /* LORA_SGMV_H */
