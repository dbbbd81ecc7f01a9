/*
 * sgmv.h -- C ABI of libsgmv.so, Punica's SGMV multi-LoRA hot path on one
 * NVIDIA GB300 (sm_103a).
 *
 * SGMV (Segmented Gather Matrix-Vector multiplication) adds each request's
 * LoRA delta to its rows of a batch in which contiguous row segments use
 * different adapters:
 *
 *     Y[row(p), :] += scale * (X[row(p), :] . A[idx[s]]) . B[idx[s]]
 *         for every sorted position p in segment s = [seg_ptr[s], seg_ptr[s+1])
 *
 * Pages this interface follows (cited by title and section):
 *   [Article] "Punica: when LoRA fine-tuned models need multi-tenant serving"
 *             (omica.com.cn):
 *               §2.1 the LoRA part of a layer is x.A.B, A [H1, r], B [r, H2];
 *               §2.2 SGMV = a segmented gather of A_i out of one stack of all
 *                    adapters with v_i = x_i.A_i ("shrink"), then v_i.B_i with
 *                    all B_i stacked the same way ("expand");
 *               §5.1 the batch builder groups requests by LoRA id;
 *               §5.2 a wrong rank or shape shows up as illegal memory access.
 *   [Review]  "Punica: Multi-Tenant LoRA Serving" (nubint.ai review),
 *             "Proposed method": the kernel works on segmented inputs and
 *             outputs so that different LoRA models share one batch.
 *   [Q&A]     "How to deploy several LoRA adapters without reloading the base
 *             model (Punica, S-LoRA)?" (aivaro.ru):
 *               §3.1 each request computes x = x + (x @ A) @ B;
 *               §3.2 adapter weights sit in one contiguous buffer and the
 *                    kernel selects them by index (segmented gather/scatter);
 *                    the kernel accepts any rank r without recompiling.
 *
 * Layouts (all row-major, all tensors in device memory unless stated):
 *   x  [T][H1]    f16 or bf16           batch input rows
 *   A  [L][H1][r] same type as x        stacked adapter "A" matrices
 *   B  [L][r][H2] same type as x        stacked adapter "B" matrices
 *   y  [T][H2]    f16, bf16 or f32      output rows, updated in place
 *   v  [T][r]     f32                   shrink result, by sorted position
 *   perm    int32 [T] or NULL           physical row of sorted position p;
 *                                       NULL means position p is row p
 *   seg_ptr int32 [S+1]                 segment bounds in sorted positions,
 *                                       non-decreasing, inside [0, T]
 *   idx     int32 [S]                   adapter of each segment, in [-1, L);
 *                                       -1 = no adapter (rows left unchanged)
 * Empty segments are allowed; adjacent segments may share an adapter; rows
 * outside [seg_ptr[0], seg_ptr[S]) are neither read nor written.  perm must
 * be one-to-one on the covered positions.
 *
 * Requirements checked on the host (status returned, nothing launched):
 *   pointers non-NULL where used and 16-byte aligned; H1 and H2 multiples of
 *   8 and >= 8; 1 <= r <= 128; T >= 0; L >= 1; dtypes as above.  seg_ptr_host,
 *   when given, is checked for bounds and order.
 * Checked on the device (the bad segment or row is skipped and the sticky
 * device error word is set; read it with sgmv_get_device_error):
 *   idx outside [-1, L) -> SGMV_ERR_BAD_INDEX; a segment outside [0, T] or
 *   with end < start -> SGMV_ERR_BAD_SEGMENTS; perm entry outside [0, T) ->
 *   SGMV_ERR_BAD_INDEX.  No kernel traps or asserts; every wait in a kernel is
 *   bounded and reports SGMV_ERR_TIMEOUT if it runs out.
 *
 * Ownership and execution: the caller owns every buffer; the library never
 * allocates device memory.  Calls are asynchronous on `stream` (a
 * cudaStream_t, NULL = legacy default stream), take no locks and keep no
 * state except the device error word.  The device addresses of the library's
 * own device variables (the error word, the scratch of sgmv_apply_noalloc)
 * are looked up once per device and kept: after cudaDeviceReset, or any other
 * teardown of a device's primary context, the library must not be used again
 * on that device in the same process.  Kernels are launched with
 * programmatic dependent launch: a kernel may start while the previous
 * kernel on the stream finishes, and before it waits for that kernel it
 * reads only A, B, row_adapter and the segment metadata.  So those inputs must
 * not be written by the SGMV kernel launched just before on the same stream
 * (x and y may be: they are read only after the wait).
 */
#ifndef SGMV_H
#define SGMV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SGMV_OK = 0,
    SGMV_ERR_INVALID_ARG = 1,   /* NULL pointer, size out of range, bad dtype */
    SGMV_ERR_UNSUPPORTED = 2,   /* valid but outside what the library handles */
    SGMV_ERR_ALIGNMENT = 3,     /* pointer not 16-byte aligned, H1/H2 % 8 != 0 */
    SGMV_ERR_BAD_INDEX = 4,     /* adapter id or perm entry out of range */
    SGMV_ERR_CUDA = 5,          /* a CUDA runtime call failed */
    SGMV_ERR_WORKSPACE = 6,     /* workspace smaller than sgmv_workspace_bytes */
    SGMV_ERR_TIMEOUT = 7,       /* a bounded wait inside a kernel ran out */
    SGMV_ERR_BAD_SEGMENTS = 8   /* seg_ptr out of [0, T] or decreasing */
} sgmv_status;

typedef enum {
    SGMV_F16 = 0,
    SGMV_BF16 = 1,
    SGMV_F32 = 2,               /* output y; logits */
    SGMV_E4M3 = 3               /* caches of sgmv_cache_commit */
} sgmv_dtype;

/* Human-readable name of a status code (static string, never NULL). */
const char *sgmv_status_string(int status);

/* Detail of the last SGMV_ERR_CUDA returned on the calling thread (which CUDA
 * call failed and its error string); empty if none.  Thread-local storage
 * owned by the library, valid until the thread's next failing call. */
const char *sgmv_last_error_string(void);

/* Number of kernels the calling thread's last sgmv_shrink / sgmv_expand /
 * sgmv_apply / sgmv_build_segments_device call launched (0 when it returned
 * before launching anything). */
int sgmv_last_launch_count(void);

/* Upper bound on the number of segments that grouping T rows over L adapters
 * (ids -1..L-1) can produce: min(T, L + 1).  Size seg_ptr (bound + 1) and idx
 * (bound) with it for sgmv_build_segments_device. */
int32_t sgmv_max_segments(int32_t T, int32_t L);

/*
 * Group a batch's rows by adapter id, on the host ([Article] §5.1; [Review]
 * "Proposed method").  Stable: ascending id with -1 first, original row order
 * within an id, one segment per id that occurs.
 *   row_adapter  host int32 [T], ids in [-1, L)
 *   perm         host int32 [T]      out: physical row of each sorted position
 *   seg_ptr      host int32 [T + 1]  out: S + 1 entries used
 *   idx          host int32 [T]      out: S entries used
 *   S            host int32 [1]      out: number of segments
 * Returns SGMV_ERR_BAD_INDEX if an id is out of range (outputs undefined).
 */
int sgmv_build_segments(const int32_t *row_adapter, int32_t T, int32_t L,
                        int32_t *perm, int32_t *seg_ptr, int32_t *idx,
                        int32_t *S);

/*
 * The same grouping on the device, one small kernel, no host synchronisation.
 * All pointers are device pointers.  seg_ptr must hold
 * sgmv_max_segments(T, L) + 1 entries and idx sgmv_max_segments(T, L): past
 * the real segment count the kernel writes empty segments (seg_ptr = T,
 * idx = -1), so the arrays can be passed to the SGMV calls with
 * S = sgmv_max_segments(T, L).  *S receives the real count.  An id out of
 * range is grouped as -1 and sets SGMV_ERR_BAD_INDEX in the device error
 * word.  Requires L <= 32767.
 */
int sgmv_build_segments_device(const int32_t *row_adapter, int32_t T, int32_t L,
                               int32_t *perm, int32_t *seg_ptr, int32_t *idx,
                               int32_t *S, void *stream);

/*
 * Bytes of device workspace that lets sgmv_apply use its tensor-core path for
 * long segments: v for T rows as two 16-bit halves, plus 256 bytes for a
 * counter the tensor-core kernels use to share out the last part of the
 * work.  Calls that run at the same time need separate workspaces.
 * sgmv_apply also accepts workspace == NULL with workspace_bytes == 0 and
 * then runs every segment on the CUDA-core path.
 */
size_t sgmv_workspace_bytes(int32_t T, int32_t H1, int32_t H2, int32_t r);

/*
 * Shrink, the first SGMV step ([Article] §2.2):
 *   v[p][k] = sum_h x[row(p)][h] * A[idx[s]][h][k]    (fp32 accumulation)
 * v rows of segments with idx = -1 are set to 0; other rows of v are not
 * written.  seg_ptr_host (host int32 [S+1] copy of seg_ptr, or NULL) lets the
 * host size the launch exactly; without it the launch is sized by a bound.
 */
int sgmv_shrink(float *v, const void *x, const void *A, int in_dtype,
                const int32_t *perm, const int32_t *seg_ptr, const int32_t *idx,
                int32_t S, const int32_t *seg_ptr_host, int32_t T, int32_t L,
                int32_t H1, int32_t r, void *stream);

/*
 * Expand, the second SGMV step ([Article] §2.2), accumulated into y
 * ([Q&A] §3.1):
 *   y[row(p)][j] = round(y[row(p)][j] + scale * sum_k v[p][k] * B[idx[s]][k][j])
 * computed in fp32 and rounded once (to nearest even) to y's type.
 */
int sgmv_expand(void *y, int y_dtype, const float *v, const void *B, int in_dtype,
                float scale, const int32_t *perm, const int32_t *seg_ptr,
                const int32_t *idx, int32_t S, const int32_t *seg_ptr_host,
                int32_t T, int32_t L, int32_t H2, int32_t r, void *stream);

/*
 * Shrink and expand in one call: y += scale * (x . A[idx]) . B[idx] per
 * segment, with v kept on chip (never written to device memory) on the
 * CUDA-core path.  Segments of at least 64 rows use the tensor-core path when
 * a workspace of sgmv_workspace_bytes() is given (it holds v for those rows).
 * Result equals sgmv_shrink followed by sgmv_expand up to fp32 summation
 * order.
 */
int sgmv_apply(void *y, int y_dtype, const void *x, const void *A, const void *B,
               int in_dtype, float scale, const int32_t *perm,
               const int32_t *seg_ptr, const int32_t *idx, int32_t S,
               const int32_t *seg_ptr_host, int32_t T, int32_t L, int32_t H1,
               int32_t H2, int32_t r, void *workspace, size_t workspace_bytes,
               void *stream);

/*
 * Grouping and update in one call, from the batch's row -> adapter ids: the
 * whole hot path (group rows by adapter, gather x, shrink, expand, scatter
 * into y) for a batch whose rows arrive in any order.
 *   row_adapter  device int32 [T], ids in [-1, L) (-1 = no adapter)
 *   perm, seg_ptr, idx, S   device int32 arrays as for
 *                sgmv_build_segments_device, receiving the grouping so later
 *                calls on the same batch (other layers and projections) can
 *                pass it to sgmv_apply; all four NULL or all four set.
 * For T <= 64 rows this is a single kernel: every CTA groups the rows
 * itself, so no metadata is read from device memory (the arrays, if given,
 * are still written).  Otherwise it runs the grouping kernel into the caller's arrays
 * (then required: SGMV_ERR_INVALID_ARG if NULL) followed by sgmv_apply.  An id
 * out of range is treated as -1 and reported as SGMV_ERR_BAD_INDEX in the
 * device error word.
 */
int sgmv_apply_rows(void *y, int y_dtype, const void *x, const void *A, const void *B,
                    int in_dtype, float scale, const int32_t *row_adapter, int32_t T, int32_t L,
                    int32_t H1, int32_t H2, int32_t r, int32_t *perm, int32_t *seg_ptr,
                    int32_t *idx, int32_t *S, void *workspace, size_t workspace_bytes,
                    void *stream);

/*
 * sgmv_apply for callers that cannot allocate device memory: the pages
 * describing SGMV have no counterpart of this call.  It is for code that may
 * not call cudaMalloc where it runs SGMV -- a plugin that only gets the
 * buffers its host engine planned at start-up, a serving loop that forbids
 * allocation after warm-up, or code running while a CUDA graph is captured.
 * Arguments and results are those of sgmv_apply, without the workspace: the
 * scratch for the tensor-core path is a fixed 4 MiB array inside the
 * library's device image, held by every GPU that loads the library until the
 * process exits.  Only problems that can reach the tensor-core path (r = 64
 * or 128 and T >= 64) use it; those whose sgmv_workspace_bytes(T, H1, H2, r)
 * exceeds 4 MiB are refused with SGMV_ERR_WORKSPACE before anything is
 * launched.  Every other problem runs on the CUDA cores without scratch,
 * whatever its size.  The first such call on a device looks the array's
 * device address up (cudaGetSymbolAddress, no allocation); make that first
 * call before any stream capture.  All calls share the one array and it keeps
 * the last call's contents (nothing in it has to start at zero), so calls
 * that overlap on the GPU -- on different streams, or from different threads
 * -- race on it.
 */
int sgmv_apply_noalloc(void *y, int y_dtype, const void *x, const void *A, const void *B,
                       int in_dtype, float scale, const int32_t *perm, const int32_t *seg_ptr,
                       const int32_t *idx, int32_t S, const int32_t *seg_ptr_host, int32_t T,
                       int32_t L, int32_t H1, int32_t H2, int32_t r, void *stream);

/*
 * Bytes of device workspace sgmv_fused_linear_lora needs: v [T][r] fp32, the
 * pair table and the 16-bit v tiles of the adapter terms (at most T tiles of
 * [16][64] elements, two per pair for r > 32), and an fp32 scratch area for
 * the partial sums of tiles split across a cluster (at most 8 x
 * ceil(H2 / 128) x round32(T) x 128 floats); each part 256-byte aligned.
 */
size_t sgmv_fused_workspace_bytes(int32_t T, int32_t H2, int32_t r);

/*
 * The whole LoRA layer in one pass over its weights: the base linear layer and
 * the SGMV update together ([Article] §2.1: a LoRA layer computes
 * y = xW + xAB; [Q&A] §3.2, "Fused Kernel": the LoRA transform is merged into
 * the base model's linear layer so that memory is read fewer times):
 *   y[t][j] = round( sum_h x[t][h] * W[h][j]
 *                    + scale * sum_k v[p][k] * B[idx[s]][k][j] )
 *   with v[p] = x[t] . A[idx[s]], for physical row t = perm[p] of position p
 *   in segment s with idx[s] >= 0; rows in no segment with an adapter get
 *   the base product alone.
 * Every row t in [0, T) of y is overwritten (y is the layer's output; it must
 * not overlap x, W, A or B); the sums are fp32 and y is rounded once.
 *   W  [H1][H2]  device, in_dtype (f16 / bf16), row-major
 *   x, A, B, perm, seg_ptr, idx, S, L, r as for sgmv_apply; y as for
 *   sgmv_apply but written, not updated.
 *   workspace  device, >= sgmv_fused_workspace_bytes(T, H2, r) bytes, 16-byte
 *              aligned (holds v, its tiles and partial sums between the kernels).
 * Decode batches: 1 <= T <= 128 rows and r <= 64 (SGMV_ERR_UNSUPPORTED
 * otherwise).  Three kernels on `stream` (one when S == 0): the CUDA-core
 * shrink writes v; a small kernel lays scale * v out as block-diagonal 16-bit
 * tiles (each value as a high and a low half); a tensor-core kernel streams W
 * and the adapters' B slices once and makes every element of y, base and
 * adapter terms in one fp32 accumulation.  Errors as for sgmv_apply (host checks, device error
 * word).
 */
int sgmv_fused_linear_lora(void *y, int y_dtype, const void *x, const void *W, const void *A,
                           const void *B, int in_dtype, float scale, const int32_t *perm,
                           const int32_t *seg_ptr, const int32_t *idx, int32_t S, int32_t T,
                           int32_t L, int32_t H1, int32_t H2, int32_t r, void *workspace,
                           size_t workspace_bytes, void *stream);

/*
 * sgmv_apply for P problems at once (1 <= P <= 4) that share the rows, the
 * segments and the shapes but have their own x, A, B and y: the projections
 * of one layer that read the same rows, q / k / v, or gate / up ([Article]
 * §2.1: a LoRA pair A, B sits beside a weight matrix W; §3.2: the pairs are
 * injected into the model's linear layers, e.g. each layer's attention q
 * projection; §2.2 for the operation).  y[k] += scale * (x[k] . A[k][idx]) . B[k][idx], every
 * argument otherwise as for sgmv_apply (host arrays of P device pointers for
 * y, x, A, B; x[k] may all be the same pointer, the y[k] must not overlap
 * one another: the problems' updates run at the same time).  The P problems run as one
 * launch of the streaming CUDA-core kernel when r <= 64, r % 4 == 0 and the
 * batch is large enough for one-CTA clusters (T > 76 on 152 SMs; each CTA
 * walks several (problem, tile) units), with each row's arithmetic exactly
 * that of P separate sgmv_apply calls without a workspace (the same bits);
 * otherwise it makes those P calls.  P = 1 is allowed: a serving loop that
 * sends all its calls here runs a single kernel.
 * No workspace, nothing allocated.  Errors: SGMV_ERR_INVALID_ARG for P out
 * of range or null arrays or pointers, then as sgmv_apply; when the problems
 * run as P calls and call k fails, problems 0 .. k-1 are already queued on
 * `stream` and k .. P-1 are not.
 */
int sgmv_apply_multi(int32_t P, void *const *y, int y_dtype, const void *const *x,
                     const void *const *A, const void *const *B, int in_dtype, float scale,
                     const int32_t *perm, const int32_t *seg_ptr, const int32_t *idx, int32_t S,
                     const int32_t *seg_ptr_host, int32_t T, int32_t L, int32_t H1, int32_t H2,
                     int32_t r, void *stream);

/*
 * Loads one adapter into slot `slot` of the stacked pools: A_src [H1][r] into
 * A_pool[slot] and B_src [r][H2] into B_pool[slot], as two asynchronous copies
 * on `stream`.  Page: [Review] "Punica: Multi-Tenant LoRA Serving" (nubint.ai
 * review), "Proposed method" and findings: LoRA weights are loaded on demand,
 * in milliseconds, instead of keeping every adapter resident.
 *   A_pool  [L][H1][r]  device, in_dtype        stacked "A" matrices
 *   B_pool  [L][r][H2]  device, in_dtype        stacked "B" matrices
 *   A_src, B_src        host or device memory, in_dtype, contiguous; from
 *                       page-locked host memory the copies overlap with
 *                       kernels on other streams and return at once
 * Nothing is allocated.  The caller orders the copies before the SGMV calls
 * that read the slot (an event on `stream`) and must not overwrite a slot that
 * an SGMV call in flight still reads.  Errors: SGMV_ERR_INVALID_ARG for null
 * pointers, slot outside [0, L), non-positive sizes or an input type other
 * than f16 / bf16; SGMV_ERR_CUDA if a copy cannot be enqueued.
 */
int sgmv_load_adapter(void *A_pool, void *B_pool, int in_dtype, int32_t slot, const void *A_src,
                      const void *B_src, int32_t L, int32_t H1, int32_t H2, int32_t r,
                      void *stream);

/*
 * Up to 512 copies dst[i] <- src[i] (bytes[i] bytes each) on `stream`, for
 * loading every piece of an adapter at once (same page and passage as
 * sgmv_load_adapter: one Llama-2-7B adapter is 448 pieces).  Every copy whose
 * source and destination the current device reads directly (its own device
 * memory, or page-locked host memory), both 16-byte aligned, with bytes[i] a
 * multiple of 16, is moved by ONE kernel launch: the SMs read the sources
 * (page-locked host memory over the CPU-GPU link) and write the destinations.
 * Each other copy is enqueued as its own asynchronous copy-engine transfer on
 * `stream`.  All copies are ordered after earlier work on `stream`.
 *   n          number of copies, 0 <= n <= 512 (0: nothing happens)
 *   dst, src   host arrays of n pointers (host or device addresses); the
 *              ranges must not overlap one another
 *   bytes      host array of n sizes; a zero size skips its copy (its
 *              pointers may then be null)
 *   max_ctas   most CTAs of the kernel; 0 = four per SM.  A small cap leaves
 *              SMs to kernels that run at the same time on other streams.
 * The arrays are read before the call returns; the copied memory must stay
 * valid until the copies complete.  Nothing is allocated.  Errors:
 * SGMV_ERR_INVALID_ARG for n outside [0, 512], negative max_ctas, null arrays
 * or a null pointer with a non-zero size; SGMV_ERR_CUDA if a copy or the
 * launch cannot be enqueued (then some copies may have been enqueued).
 * sgmv_last_launch_count() is 1 if the kernel was launched, else 0.
 */
int sgmv_copy_gather(int32_t n, void *const *dst, const void *const *src, const uint64_t *bytes,
                     int32_t max_ctas, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Speculative decoding over a paged KV cache: what a step of a multi-LoRA model
 * runs between its projections.  (No counterpart on the pages, which leave
 * attention and the cache to the serving engine.)
 *
 *   sgmv_rope            rotary positions of q and k, k and v appended to the cache
 *   sgmv_tree_attention  attention of every sequence's drafted tokens over the cache
 *   sgmv_tree_verify     which drafted tokens the target distribution accepts
 *   sgmv_cache_commit    the accepted tokens' k and v moved to their final places
 *
 * Shared conventions.  The batch has T rows (tokens); sequence b owns the rows
 * [tree_ptr[b], tree_ptr[b+1]), its "nodes" 0, 1, ....  parents[row] is the
 * node's parent within its sequence: an earlier node, -1 for a node whose only
 * ancestors are the tokens already in the cache, or -2 for a padding row.
 * parents == NULL makes every sequence a chain (node i's parent is i - 1).  A
 * sequence has at most SGMV_TREE_MAX_NODES nodes; empty sequences are allowed.
 *
 * The cache holds token position j of sequence b in page block_table[b][j /
 * block_size], at offset j % block_size.  Positions 0 .. prefix_lens[b] - 1
 * are the context; node i sits at position prefix_lens[b] + i.  k_cache and
 * v_cache have the same strides (in elements; the last dimension is
 * contiguous), any block_size >= 1, and may be views of one array in either
 * order of pages, tokens and heads.  Nothing is assumed about slots that hold no token.
 *
 * Arguments travel in a struct, which is read before the call returns.  All
 * pointers are device pointers unless stated; f16 / bf16 data must be 16-byte
 * aligned and its strides multiples of 8 elements, int32 and fp32 data 4-byte
 * aligned (SGMV_ERR_ALIGNMENT); the stride of a dimension of one entry does not matter.
 * Metadata is checked on the device: a sequence with bad tree_ptr or too many
 * nodes is skipped (SGMV_ERR_BAD_SEGMENTS in the device error word), and a
 * parent, slot, token or path entry out of range is left out, a page out of
 * range spoils its own sequence alone (SGMV_ERR_BAD_INDEX).  Calls are asynchronous, allocate nothing, and read
 * their inputs only after the previous kernel on the stream has finished.
 */
#define SGMV_TREE_MAX_NODES 256

/*
 * Rotary positions.  The first 2 * pairs columns of every head of q and k turn
 * pairwise by the angle positions[t] * inv_freq[i]:
 *   out_a = scale * (x_a cos - x_b sin),  out_b = scale * (x_a sin + x_b cos)
 * with (a, b) = (i, i + pairs), or (2i, 2i + 1) if interleaved; the other
 * columns are copied.  inverse != 0 turns by the negative angle: applied to
 * the gradients of the outputs it gives the gradients of the inputs.  scale
 * is the magnitude factor of long-context scalings (1 without).  The angle is
 * reduced in 64-bit fixed point, so positions of any size are as accurate as
 * small ones; sums are fp32 and rounded once.
 *   q [T][Hq][D], k and v [T][Hk][D]  any token and head strides; q or k may
 *     be NULL (with Hq or Hk = 0).  q_out / k_out may equal q / k (in place)
 *     but must not overlap them otherwise.  k_out may be NULL when k_cache is given.
 *   positions int32 [T]; inv_freq HOST double [pairs], 0 <= 2 pairs <= D
 *   k_cache, v_cache, slots: all NULL, or the rotated k and the unchanged v of
 *     row t are also written to slot slots[t] (page * block_size + offset;
 *     -1 = not appended).  v_cache needs v.  Slots must be distinct.
 * D a multiple of 8, at most 256 (SGMV_ERR_UNSUPPORTED beyond).
 */
typedef struct {
    void *q_out;
    const void *q;
    void *k_out;
    const void *k;
    const void *v;
    void *k_cache;
    void *v_cache;
    const int32_t *positions;
    const int32_t *slots;
    const double *inv_freq;
    int64_t q_out_token, q_out_head, q_token, q_head;
    int64_t k_out_token, k_out_head, k_token, k_head, v_token, v_head;
    int64_t cache_block, cache_token, cache_head;
    int32_t T, Hq, Hk, D, pairs, num_blocks, block_size, dtype, interleaved, inverse;
    float scale;
} sgmv_rope_args;
int sgmv_rope(const sgmv_rope_args *args, void *stream);

/*
 * Inverse frequencies of rotary positions, on the host: inv_freq[i] =
 * base^(-2i / (2 pairs)), i < pairs, then stretched for contexts of `factor`
 * times the `trained` length: a pair that turns at least `fast` times over
 * the trained length is kept, one that turns at most `slow` times is divided
 * by factor, with a linear ramp between (slow < fast).  factor = 1 leaves them
 * as they are; slow = fast = INFINITY divides every pair (linear position
 * interpolation).
 */
int sgmv_rope_frequencies(double *inv_freq, int32_t pairs, double base, double factor,
                          double trained, double slow, double fast);

/*
 * Attention of the drafted tokens over the cache:
 *   out[t][h] = sum_j p_j v_j,  p = softmax_j(scale * q[t][h] . k_j)
 * over the context of t's sequence, t's ancestors and t itself; k_j and v_j
 * of head h / (Hq / Hkv).  What a row does not see has no influence on it,
 * infinities and NaN included.  A row that sees nothing (padding) gets 0 and
 * lse -inf.  The sequences' nodes must have been appended to the cache.
 *   q, out [T][Hq][D]; lse fp32 [T][Hq] contiguous or NULL: log of the sum of
 *     exp(scale * score); block_table int32 [B][max_blocks], row stride
 *     table_row; prefix_lens int32 [B]; tree_ptr int32 [B+1]
 *   scale: multiplied onto the scores (usually D^-1/2)
 *   workspace: sgmv_tree_attention_workspace_bytes() bytes, 256-byte aligned;
 *     what it holds does not matter.  Calls that run at the same time need
 *     separate ones.  No batch of at most T rows and B sequences needs more
 *     than the bytes of T and B (21 MB at most).
 * Hq a multiple of Hkv, D a multiple of 8 up to 256.  Heads of more than 128
 * columns run on the CUDA cores, a CTA per row and query head over the whole
 * context: right, but for short contexts and few rows (32 rows over up to 4096
 * tokens, 32 heads of 256: 1.3 ms; of 128: 0.17).  Scores, softmax and sums
 * are fp32; the weights p are rounded to the inputs' type for the tensor
 * cores, the output once.  out must not overlap the inputs.  Rows in no
 * sequence are not written.
 */
typedef struct {
    void *out;
    const void *q;
    const void *k_cache;
    const void *v_cache;
    float *lse;
    const int32_t *block_table;
    const int32_t *prefix_lens;
    const int32_t *tree_ptr;
    const int32_t *parents;
    void *workspace;
    uint64_t workspace_bytes;
    int64_t out_token, out_head, q_token, q_head;
    int64_t cache_block, cache_token, cache_head, table_row;
    int32_t T, B, Hq, Hkv, D, num_blocks, block_size, max_blocks, dtype;
    float scale;
} sgmv_tree_attention_args;
size_t sgmv_tree_attention_workspace_bytes(int32_t T, int32_t B, int32_t Hq, int32_t Hkv,
                                           int32_t D);
int sgmv_tree_attention(const sgmv_tree_attention_args *args, void *stream);

/*
 * Verification of drafted tokens (speculative sampling on a tree), from given
 * random numbers.  Node 0 of a sequence is its last token, already accepted;
 * tokens[row] is each node's token; target[row] the model's distribution
 * after the node, draft[row] the distribution its children were drawn from
 * (independent draws), or draft == NULL for children proposed without one.
 * From node 0 on, the children of the last accepted node are tried in order:
 *   child c is accepted if  u_accept[c] * q(token) * W < w(token),
 * else the rest of the distribution shrinks:  w = max(w - q W, 0), W = sum w
 * (without a draft: q = 1 at the token, so w(token) = 0).  w starts as the
 * target's weights with W = 1 at every accepted node.  When no child is left,
 * `token` is drawn from w by inverting its running sum at u_sample[b]; if w
 * is zero everywhere, from the target itself, and -1 if that is zero too.
 * The accepted tokens and the drawn one follow the target's distribution.
 * Weights are whole multiples of 2^-38 (probabilities are clamped to [0, 1];
 * NaN counts as 0), so sums are exact and results do not depend on the order
 * of summation; products are single fp32 multiplications.
 *   target, draft fp32 [T][V], rows target_row / draft_row elements apart, 4-byte aligned
 *   u_accept fp32 [T], u_sample fp32 [B], in [0, 1)
 *   count int32 [B]: accepted nodes, node 0 among them (0 for an empty sequence)
 *   path int32 [B][max_path]: their node numbers, -1 beyond; the walk stops
 *     when it is full.  token int32 [B].
 */
typedef struct {
    const float *target;
    const float *draft;
    const int32_t *tokens;
    const int32_t *parents;
    const int32_t *tree_ptr;
    const float *u_accept;
    const float *u_sample;
    int32_t *count;
    int32_t *path;
    int32_t *token;
    int64_t target_row, draft_row;
    int32_t T, B, V, max_path;
} sgmv_tree_verify_args;
int sgmv_tree_verify(const sgmv_tree_verify_args *args, void *stream);

/*
 * Moves the accepted nodes' k and v to their final places in the cache (f16,
 * bf16, or e4m3 with D and the strides multiples of 16), in place: position
 * prefix_lens[b] + d takes what position prefix_lens[b] + path[b][d] held, for
 * d < count[b].  path rows ascend (as
 * sgmv_tree_verify writes them).  Afterwards the sequence's context is
 * prefix_lens[b] + count[b] long.  layers > 1 moves the same tokens in that
 * many caches, cache_layer elements apart.
 */
typedef struct {
    void *k_cache;
    void *v_cache;
    const int32_t *block_table;
    const int32_t *prefix_lens;
    const int32_t *path;
    const int32_t *count;
    int64_t cache_layer, cache_block, cache_token, cache_head, table_row;
    int32_t layers, B, Hkv, D, num_blocks, block_size, max_blocks, max_path, dtype;
} sgmv_cache_commit_args;
int sgmv_cache_commit(const sgmv_cache_commit_args *args, void *stream);

/*
 * ---------------------------------------------------------------------------
 * A decoding step of models with normalised heads, with an 8-bit cache, and the
 * sampling of its tokens.  The conventions are those above.
 *
 *   sgmv_norm_rope        norms of q and k per head, rotary positions, append
 *   sgmv_norm_rope_grad   their gradient
 *   sgmv_quant_attention  tree attention over an e4m3 cache
 *   sgmv_sample           temperature, top-k, top-p and min-p
 *
 * An e4m3 cache holds 8-bit values (sign, 4 bits of exponent, 3 of mantissa; up to
 * 448), in multiples of one positive fp32 scale per KV head for k and one for v:
 * k_scale, v_scale [Hk].  Written, a value is divided by its scale (as a product
 * with the fp32 reciprocal), limited to +-448 and rounded to nearest even, once; NaN
 * stays NaN.  D and the cache's strides are multiples of 16 (SGMV_ERR_ALIGNMENT).
 * Heads of up to 256 columns are written and moved (sgmv_norm_rope,
 * sgmv_cache_commit), of up to 128 read (sgmv_quant_attention).
 */

/*
 * Norms, rotary positions and append in one pass:
 *   y = R(positions[t]) (w * x / sqrt(mean(x^2) + eps))
 * for every head x of q with w = q_weight and of k with w = k_weight ([D], of q's
 * type; NULL: that tensor is not normalised, x alone is rotated), R as in sgmv_rope
 * (rope.scale included).  y is rounded once, to q_out, to k_out, and to the cache
 * with v beside it: to q's type if k_scale and v_scale are NULL, else to e4m3.
 * `rope` is as for sgmv_rope, with inverse = 0; its caches are of the type just
 * said.  Squares are summed in fp32, and so must not pass its range (3.4e38).  eps > 0.
 * T * (Hq + 2 Hk) up to 2^30 (SGMV_ERR_UNSUPPORTED beyond).
 */
typedef struct {
    sgmv_rope_args rope;
    const void *q_weight;
    const void *k_weight;
    const float *k_scale;
    const float *v_scale;
    float eps;
} sgmv_norm_rope_args;
int sgmv_norm_rope(const sgmv_norm_rope_args *args, void *stream);

/*
 * Gradients of the inputs of sgmv_norm_rope from those of q_out and k_out: with
 * g = scale R^T dy, r = 1 / sqrt(mean(x^2) + eps), h = w * g,
 *   dx = r (h - r^2 x mean(h * x)),   dw = sum over rows and heads of g * r x
 * (dx = g for a tensor without a weight).  q, k, dq_out, dk_out, dq, dk [T][heads][D]
 * of any token and head strides, dq and dk apart from all inputs and from each other
 * (SGMV_ERR_INVALID_ARG for the same address); q or k may be left out (Hq or Hk = 0), and
 * is not read without its weight; T * (Hq + Hk) up to 2^30.  dq_weight, dk_weight fp32 [D],
 * written (not added to); given exactly where the weight is.  Sums are fp32, joined in fp64
 * in a fixed order: the same result in every run.
 *   workspace: sgmv_norm_rope_grad_workspace_bytes(D) bytes, 16-byte aligned; what it
 *     holds does not matter.  Calls that run at the same time need separate ones.
 */
typedef struct {
    void *dq;
    void *dk;
    const void *dq_out;
    const void *dk_out;
    const void *q;
    const void *k;
    const void *q_weight;
    const void *k_weight;
    float *dq_weight;
    float *dk_weight;
    const int32_t *positions;
    const double *inv_freq;
    void *workspace;
    uint64_t workspace_bytes;
    int64_t dq_token, dq_head, dk_token, dk_head, dq_out_token, dq_out_head;
    int64_t dk_out_token, dk_out_head, q_token, q_head, k_token, k_head;
    int32_t T, Hq, Hk, D, pairs, dtype, interleaved;
    float scale, eps;
} sgmv_norm_rope_grad_args;
size_t sgmv_norm_rope_grad_workspace_bytes(int32_t D);
int sgmv_norm_rope_grad(const sgmv_norm_rope_grad_args *args, void *stream);

/*
 * sgmv_tree_attention over an e4m3 cache: out = v_scale[h] softmax(scale *
 * k_scale[h] * q K^T) V, with K and V as stored.  `attention` is as there, its caches
 * of e4m3; D a multiple of 16, at most 128 (SGMV_ERR_UNSUPPORTED beyond).  Masks, padding,
 * lse and values that are no numbers as there.  The products' operands are f16: K and V
 * exactly; queries of bf16 too, a row at a time by a power of two (a value loses 2^-39 of its
 * row's largest at most); the weights rounded to f16, the output to q's type.
 */
typedef struct {
    sgmv_tree_attention_args attention;
    const float *k_scale;
    const float *v_scale;
} sgmv_quant_attention_args;
size_t sgmv_quant_attention_workspace_bytes(int32_t T, int32_t B, int32_t Hq, int32_t Hkv,
                                            int32_t D);
int sgmv_quant_attention(const sgmv_quant_attention_args *args, void *stream);

/*
 * The next token of every row of logits [T][V] (f16, bf16 or fp32), from given
 * random numbers.  Weights are whole numbers,
 *   w_i = floor(2^38 exp((l_i - max l) / temperature))   (to a few units),
 * and tokens are ranked by logit, ties by index, the lowest first.  Kept are
 *   the first top_k                                (top_k <= 0 or >= V: all),
 *   of those, as many of the first as it takes for their weights to reach
 *     top_p of their sum, one at least            (top_p >= 1: all),
 *   of those, the ones with w_i >= min_p 2^38      (min_p <= 0: all).
 * The token is the first, by index, at which the running sum of the kept weights
 * passes u of their sum; probs receives the kept weights over their sum, zero for
 * the others: the distribution for sgmv_tree_verify.  temperature <= 0 or NaN, top_k = 1, or top_p <= 0
 * or NaN: the likeliest token alone.  top_p and u count in multiples of 2^-24 (rounded
 * down), limited to [0, 1].  NaN logits count as -inf, which is never drawn, others are limited
 * to +-2^126; a row with no logit above -inf gives token -1 and zeros.  Sums are exact: the
 * result does not depend on the order of summation.
 *   temperature, top_p, min_p fp32 [T], top_k int32 [T]; each may be NULL: then
 *     temperature_all, ... hold for every row
 *   u fp32 [T], token int32 [T]: both or neither; probs fp32 [T][V], or NULL
 *   logits_row, probs_row: elements between rows; logits aligned to its type
 * probs must not overlap logits (SGMV_ERR_INVALID_ARG for the same address).  V up to 2^24, T to 2^27 (SGMV_ERR_UNSUPPORTED beyond).
 */
typedef struct {
    const void *logits;
    const float *u;
    const float *temperature;
    const int32_t *top_k;
    const float *top_p;
    const float *min_p;
    int32_t *token;
    float *probs;
    int64_t logits_row, probs_row;
    int32_t T, V, dtype, top_k_all;
    float temperature_all, top_p_all, min_p_all;
} sgmv_sample_args;
int sgmv_sample(const sgmv_sample_args *args, void *stream);

/*
 * Diagnostics (no counterpart on the pages).
 *
 * sgmv_read_floor: the floor of a decode-sized SGMV launch on this GPU.  Reads
 * `bytes` (a multiple of 16) of device memory at `src` (16-byte aligned) and
 * nothing else, spread evenly over the grid, cluster size, ring depth and
 * copy size that the streaming kernel gets from sgmv_apply_rows for a batch
 * of T rows over L adapters with these dimensions, types and rank (the
 * one-launch grouped form up to 64 rows; sgmv_apply on the device grouping
 * otherwise).  Pass the batch's algorithmic bytes to time what merely
 * bringing them on chip costs with that launch shape.  *ctas and *cluster
 * (each may be NULL) receive the grid's CTA count and cluster size.
 * SGMV_ERR_UNSUPPORTED when the streaming kernel does not apply (r not a
 * multiple of 4, or above 64).  Asynchronous on `stream`; writes nothing.
 */
int sgmv_read_floor(const void *src, size_t bytes, int32_t T, int32_t L, int32_t H1, int32_t H2,
                    int32_t r, int in_dtype, int y_dtype, int32_t *ctas, int32_t *cluster,
                    void *stream);

/*
 * sgmv_debug_inject_wait_timeout: for tests of the device-side timeout path.
 * While enabled (non-zero) on the calling thread, every streaming-kernel
 * launch it makes takes the timeout path at each compute thread's first wait
 * for a staged chunk, as if that wait had run out: SGMV_ERR_TIMEOUT is set in
 * the device error word, the chunk is then awaited with the full limit (so
 * the kernel still ends normally, with every copy landed) and the thread
 * writes no y.  Launches of the tree attention for heads of up to 128 columns
 * (and of sgmv_quant_attention) take theirs in one role of each CTA, given by the value: 1 the walk along
 * the work, 2 the loading of K and V, 3 the matrix products, 4 the softmax;
 * the status is the same, and the call writes no output.  Other kernels are
 * unaffected.  Returns SGMV_OK.
 */
int sgmv_debug_inject_wait_timeout(int enable);

/*
 * Synchronises `stream`, then reads and clears the current device's sticky
 * error word.  Returns SGMV_OK if no kernel reported an error since the last
 * read, else the first status code reported (SGMV_ERR_BAD_INDEX,
 * SGMV_ERR_BAD_SEGMENTS or SGMV_ERR_TIMEOUT), or SGMV_ERR_CUDA if the
 * synchronisation itself failed.
 */
int sgmv_get_device_error(void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SGMV_H */
