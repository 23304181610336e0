/*
 * wl.h: C ABI of the fused reconstruct-and-project linear for AMD MI355X (gfx950).
 *
 * The operation ("In-kernel reconstruction" page, introduction: the
 * reconstruction formula and its per-element expansion):
 *
 *     y[t,o] = s[o] * sum_i W0[o,i] * x[t,i]  +  sum_k U[o,k] * sum_i V[i,k] * x[t,i]
 *
 * i.e. y = s (.) (W0 x) + U (V^T x), computed without ever forming the dense
 * weight diag(s) W0 + U V^T in memory.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Memory.    Every tensor pointer is a DEVICE pointer on the current HIP device.
 *            The caller allocates and owns every buffer, including the
 *            workspace; the library never allocates or frees memory. What
 *            carries from call to call lives in the caller's workspace (its
 *            sync area, below); the library's own global state is two
 *            process-wide switches for tests and measurements (wl_testing.h).
 * Layout.    All tensors are row-major and contiguous:
 *              W0 [d_out][d_in]   s fp32 [d_out]
 *              U  [d_out][r]      V [d_in][r]
 *              x  [T][d_in]       y [T][d_out]
 *            (the index roles of the per-element expansion; the GEMM form on
 *            the same page, "The GEMM path", multiplies x by W0 transposed, by
 *            V, and the result by U transposed).
 * Dtypes.    A theta's `dtype` sets the element type of its W0, U, V and of
 *            the call's x, y (and of the MLP's h and of W_eff): WL_DTYPE_BF16
 *            or WL_DTYPE_F32 (the custom op "also supports float32", "In-kernel
 *            reconstruction", the custom-op path). s is fp32 in both. The
 *            thetas of one fused call share one dtype. A zero-filled theta is
 *            bf16.
 * Alignment. W0, U, V, x, y and W_eff must be 16-byte aligned, s 4-byte
 *            aligned, the workspace 256-byte aligned. d_in must be a multiple
 *            of 8 (rows are read in 16-byte pieces).
 * Limits.    0 <= r <= 64; d_in, d_out >= 1; T >= 0 (T == 0 is a no-op that
 *            returns WL_OK, and x, y may then be NULL). Sizes are int32 and
 *            every tensor must hold fewer than 2^31 elements.
 * Numerics.  Products accumulate in fp32; the epilogue s[o]*m + U[o,:].vtx is
 *            fp32; a bf16 y is rounded once, round-to-nearest-even ("In-kernel
 *            reconstruction", "The custom-op path": every implementation
 *            accumulates in float32 and casts back to the output dtype); an
 *            fp32 y is the fp32 result. The bf16 matrix-core regime feeds
 *            vtx = V^T x to the matrix cores as a bf16 head plus a bf16
 *            remainder. Results are deterministic from run to
 *            run (no floating-point atomics) but not bit-exact against other
 *            summation orders ("Serve and generate with weightless", "Set the
 *            fast path on NVIDIA": parity is logit parity, not bit equality).
 * Streams.   Every call only enqueues work on `hip_stream` (a hipStream_t;
 *            NULL = the default stream) and returns; errors that happen on the
 *            device surface at the caller's next synchronization.
 * Workspace. Operations that take `ws` need at least wl_workspace_bytes(...)
 *            bytes of device memory. For wl_linear, wl_qkv_fused and
 *            wl_mlp_fused its first WL_SYNC_BYTES bytes are a sync area:
 *            ticket counters and generation-tagged 64-bit words by which the
 *            workgroups of one decode launch hand each other V^T x and partial
 *            outputs ("In-kernel reconstruction", the custom-op path: V^T x
 *            formed once and shared). Before a workspace's first use, and after
 *            anything other than these calls has written its first
 *            WL_SYNC_BYTES, the caller runs wl_workspace_init on it (a kernel,
 *            so it may be captured in a graph); the calls keep the area
 *            consistent from then on. Bytes 4088 to 4095 of the area count
 *            (int64) the decode workgroups that stopped waiting and computed
 *            V^T x themselves (a diagnostic; the result is the same). The rest
 *            of the workspace is scratch whose contents on entry do not matter.
 *            Calls that can run at the same time (different streams) must not
 *            share a workspace.
 * Errors.    Every argument is checked on the host before anything is
 *            enqueued; a fused operation checks all of its thetas first, so an
 *            invalid argument never leaves a partial launch.
 *              WL_ERR_INVALID_ARG  null or misaligned pointer, bad size or
 *                                  shape mismatch, output overlapping an input
 *                                  or the workspace
 *              WL_ERR_UNSUPPORTED  r > 64, or a dtype other than the two
 *              WL_ERR_WORKSPACE    ws_bytes below the required size
 *              WL_ERR_HIP          a kernel launch failed
 *            No call aborts, throws or prints (set the environment variable
 *            WL_LOG to log the regime chosen and every failure to stderr).
 *            wl_last_error() describes the last failure on the calling thread.
 * Devices.   One device per call; nothing here shards across GPUs ("Serve and
 *            generate with weightless", "Supported encodings and devices": the
 *            pages' implementation runs on a single device as well).
 */
#ifndef WL_H
#define WL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define WL_ABI_VERSION 6

/* Bytes at the start of a projection workspace that hold the sync area. */
#define WL_SYNC_BYTES 9764864
/* Bytes of the static workspace of wl_linear_static, per device. */
#define WL_STATIC_SCRATCH_BYTES 33554432

typedef enum {
    WL_OK = 0,
    WL_ERR_INVALID_ARG = 1,
    WL_ERR_UNSUPPORTED = 2,
    WL_ERR_HIP = 3,
    WL_ERR_WORKSPACE = 4
} wl_status;

/* One projection's theta bundle ("Serve and generate with weightless",
 * introduction: a shared block W0 per band of layers, a per-row scale s and a
 * low-rank delta U, V of rank r). Several thetas may point at the same W0
 * (band sharing). The library only reads through these pointers. */
/* Element types of W0, U, V, x, y. */
enum { WL_DTYPE_BF16 = 0, WL_DTYPE_F32 = 1 };

typedef struct {
    const void  *W0;   /* dtype [d_out][d_in]                                  */
    const float *s;    /* fp32 [d_out]; NULL means every s[o] is 1              */
    const void  *U;    /* dtype [d_out][r]; ignored (may be NULL) when r == 0   */
    const void  *V;    /* dtype [d_in][r];  ignored (may be NULL) when r == 0   */
    int32_t d_in, d_out, r;
    int32_t dtype;     /* WL_DTYPE_BF16 (0) or WL_DTYPE_F32 (1)                 */
} wl_theta;

/* Operation codes for wl_workspace_bytes. */
enum { WL_OP_LINEAR = 0, WL_OP_QKV = 1, WL_OP_MLP = 2 };

/* Bytes of workspace `op` needs for these thetas at T tokens:
 *   WL_OP_LINEAR: th[0]                      (n_th == 1)
 *   WL_OP_QKV:    th[0..2] = Q, K, V         (n_th == 3)
 *   WL_OP_MLP:    th[0..2] = gate, up, down  (n_th == 3)
 * Returns 0 for invalid arguments (the matching call then fails with the
 * specific status). The value is a multiple of 256 and grows with T. */
size_t wl_workspace_bytes(int32_t op, const wl_theta *const *th, int32_t n_th, int32_t T);

/* The reconstruct-and-project linear ("In-kernel reconstruction",
 * introduction: reconstruction formula and per-element expansion).
 *   th    one theta bundle
 *   x     dtype [T][th->d_in]
 *   y     dtype [T][th->d_out] (written; must not overlap any input)
 *   T     tokens (rows of x)
 *   ws    workspace, ws_bytes >= wl_workspace_bytes(WL_OP_LINEAR, &th, 1, T)
 * With th->r == 0 and th->s == NULL this is the dense product y = x W0^T: the
 * comparator of the precompute-outside path ("Serve and generate with
 * weightless", "Set the fast path on NVIDIA") when W0 is a materialized W_eff. */
wl_status wl_linear(const wl_theta *th, const void *x, void *y, int32_t T,
                    void *ws, size_t ws_bytes, void *hip_stream);

/* wl_linear without a workspace argument, for callers that cannot allocate
 * device memory: code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc. Arguments, result and errors as wl_linear; the
 * workspace is a static device array of WL_STATIC_SCRATCH_BYTES that the
 * library holds on each device it runs on until the process ends. The call
 * allocates nothing. Its first call on a device looks the array up and
 * enqueues on hip_stream a fill kernel that clears the array's sync area,
 * ahead of its own kernels. Every call on a device shares that device's array
 * and the array keeps the last call's contents, so calls that overlap on one
 * device (other streams, other host threads) race and must be serialized by
 * the caller; wl_linear with workspaces of its own does not share it. A call
 * whose workspace would exceed WL_STATIC_SCRATCH_BYTES (the decode and
 * few-token kernels of the Gemma-3 shapes fit; long prefill passes may not)
 * fails with WL_ERR_WORKSPACE before launching anything. */
wl_status wl_linear_static(const wl_theta *th, const void *x, void *y, int32_t T, void *hip_stream);

/* Q/K/V fusion ("In-kernel reconstruction", "Q/K/V fusion"): the three
 * attention projections that read the same x, computed in one pass over the
 * concatenated W0 rows, each child with its own V^T x (a block-diagonal U).
 *   q, k, v   thetas with equal d_in and dtype; ranks, scales and d_out may differ
 *   x         dtype [T][d_in]
 *   y_qkv     dtype [T][q->d_out + k->d_out + v->d_out], columns Q | K | V
 *   ws        ws_bytes >= wl_workspace_bytes(WL_OP_QKV, {q, k, v}, 3, T)
 * Each child's columns equal wl_linear of that child to within rounding. */
wl_status wl_qkv_fused(const wl_theta *q, const wl_theta *k, const wl_theta *v,
                       const void *x, void *y_qkv, int32_t T,
                       void *ws, size_t ws_bytes, void *hip_stream);

/* Fused MLP ("In-kernel reconstruction", "The custom-op path": the fused MLP
 * op runs gate, up, the activation and down as one operation):
 *   g = linear(gate, x), u = linear(up, x)       (fp32, not rounded)
 *   h = round(gelu_tanh(g) * u)                  (rounded once to the dtype:
 *                                                 bf16 RNE, or the fp32 value)
 *   y = linear(down, h)
 * with gelu_tanh(z) = 0.5 z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))).
 * Shapes: gate.d_in == up.d_in (= d_model), gate.d_out == up.d_out ==
 * down.d_in (= d_ff), one dtype; x dtype [T][d_model], y dtype [T][down.d_out].
 * h lives in the workspace:
 *   ws_bytes >= wl_workspace_bytes(WL_OP_MLP, {gate, up, down}, 3, T). */
wl_status wl_mlp_fused(const wl_theta *gate, const wl_theta *up, const wl_theta *down,
                       const void *x, void *y, int32_t T,
                       void *ws, size_t ws_bytes, void *hip_stream);

/* The effective weight of the precompute-outside path ("Serve and generate
 * with weightless", "Set the fast path on NVIDIA"):
 *   W_eff[o,i] = round( s[o] * W0[o,i] + sum_k U[o,k] * V[i,k] )
 * W_eff: th->dtype [th->d_out][th->d_in] (bf16: rounded once, RNE; fp32: the
 * fp32 result), written; must not overlap any input.
 * Needs no workspace. */
wl_status wl_materialize_weff(const wl_theta *th, void *W_eff, void *hip_stream);

/* The effective weight of the precompute-outside path ("Serve and generate
 * with weightless", "Set the fast path on NVIDIA") for n projections (a
 * layer's seven, say): wl_materialize_weff for each, in one launch per eight
 * of them instead of one each; the same values, bit for bit.
 * th[j], W_eff[j] for j < n as in wl_materialize_weff, all thetas of one
 * dtype (fp32: one launch per projection); no W_eff may overlap another or
 * any theta's tensors. Every argument is checked before anything is
 * launched. n = 0: nothing to do. Needs no workspace. */
wl_status wl_materialize_weff_batch(const wl_theta *const *th, void *const *W_eff, int32_t n, void *hip_stream);

/* Decode steps ("Throughput" page, "Versus vanilla MAX": at batch 1 a step's
 * dispatches, not its arithmetic, dominate; "Serve and generate with
 * weightless", "Current limits": shared-W0 (G = 1) configurations). A step is a
 * fixed list of wl_linear / wl_qkv_fused / wl_mlp_fused calls that the library
 * records once into a HIP graph and launches with one call.
 *   op   WL_OP_LINEAR (th[0]), WL_OP_QKV (th = Q, K, V) or WL_OP_MLP (th =
 *        gate, up, down); unused th entries are ignored
 *   x, y, T   as in the op's own call (QKV: y is [T][dq + dk + dv]) */
typedef struct {
    int32_t op;
    const wl_theta *th[3];
    const void *x;
    void *y;
    int32_t T;
} wl_call;

/* wl_step_create flag: launch the calls that share their first theta's W0 back
 * to back (groups in order of first appearance, given order within a group),
 * so that a W0 shared by several layers (G = 1) is read while it is still in
 * the caches. Allowed only when no call reads or overwrites another call's
 * output (else WL_ERR_INVALID_ARG); results are the same as in given order. */
enum { WL_STEP_GROUP_SHARED_W0 = 1 };

typedef struct wl_step_s *wl_step;

/* Workspace bytes of a step: the largest of its calls' wl_workspace_bytes
 * (the calls run one after another on one workspace). 0 for invalid calls. */
size_t wl_step_workspace_bytes(const wl_call *calls, int32_t n_calls);

/* Records the calls (1 <= n_calls <= 65536) into a HIP graph, in the given
 * order or as WL_STEP_GROUP_SHARED_W0 regroups them, each exactly as its own
 * entry point would launch it (the regime switch is read now), and
 * instantiates it. Every call is checked as by its own entry point, before
 * anything runs; on an error no step is made and the message names the call.
 * The theta structs and the call array are read only here; the device buffers
 * they and x, y, ws point at must stay allocated while the step exists, and
 * their contents are read or written at each launch (new x values between
 * launches are used). ws: ws_bytes >= wl_step_workspace_bytes, 256-byte
 * aligned, prepared by wl_workspace_init; it may be shared with other calls
 * and steps that never overlap this step's launches. Creating a step makes
 * host-side objects (a capture stream, the graph); launching allocates
 * nothing. A call may read an earlier call's output (given order only). */
wl_status wl_step_create(const wl_call *calls, int32_t n_calls, int32_t flags, void *ws, size_t ws_bytes,
                         wl_step *step);

/* One launch of the step's graph on hip_stream (every call, in order). Two
 * launches of one step, or of steps sharing a workspace, must not overlap:
 * they share the workspace. */
wl_status wl_step_launch(wl_step step, void *hip_stream);

/* Frees the step's graph. NULL is accepted. The caller makes sure no launch
 * of the step is still running (for example by synchronizing its stream). */
wl_status wl_step_destroy(wl_step step);

/* ---------------------------------------------------------------------------
 * The rest of a decoder layer, between the projections: norms with a block's
 * residual, rotary positions, a paged cache of keys and values, attention over
 * it. Conventions as above (device pointers, caller's buffers, checks on the
 * host before anything is enqueued, one rounding of every result, no atomics),
 * with these additions:
 *   - `dtype` (WL_DTYPE_BF16 or WL_DTYPE_F32) is the type of every tensor whose
 *     type is not stated.
 *   - Rows may be strided: `ld...` is the distance of two tokens' rows in
 *     elements, so that Q, K and V can lie side by side as wl_qkv_fused leaves
 *     them. It is a multiple of 8 and at least the row's width.
 *   - An output may be exactly one of its call's inputs where that is stated
 *     (same pointer, same ld); any other overlap is WL_ERR_INVALID_ARG.
 *   - T is at most 2^24.
 *   - Index arrays (positions, sequences, slots, lengths, page table) are device
 *     int32, read when the work runs, so a recorded step follows them. The host
 *     cannot check them; the kernels do, as stated at each operation, and never
 *     read or write outside the tensors whatever they hold.
 * Serving only: these operations have no gradients (a rotation by the negated
 * positions is the rotation's transpose).
 */

/* Norms around a block, fused with its gate and its residual:
 *   p  = post ? rms(y) (post + offset) : y       the norm behind the block
 *   x' = res_scale x + branch_scale gate p       the residual stream
 *   n  = rms(x') (pre + offset)                  the norm before the next block
 *   rms(z) = z / sqrt(mean_i z_i^2 + eps)
 * n is formed from the unrounded x'. y == NULL: no block (x' = res_scale x).
 *   x, y          [T][d]; y may be NULL
 *   post, pre     [d]; NULL means no post norm / every weight pre + offset is 1
 *   gate          [d] with gate_ld 0, or [T] rows gate_ld apart; NULL means 1
 *   x_out, n_out  [T][d]; either may be NULL, not both; each may be x or y
 * d: a multiple of 8, at most 32768. offset is 1 where weights are stored as
 * w - 1, else 0. Sums are fp32. */
typedef struct {
    const void *x, *y, *post, *pre, *gate;
    void *x_out, *n_out;
    int32_t T, d, gate_ld, dtype;
    float eps, offset, res_scale, branch_scale;
} wl_norm_args;
wl_status wl_norm_residual(const wl_norm_args *a, void *hip_stream);

/* Rotary positions. The first `rot` elements of a head are rot/2 pairs: (e,
 * e + rot/2) in the half style, (2e, 2e+1) in the interleaved one. Pair e of a
 * token at position p becomes
 *   (a, b) -> scale (a cos t - b sin t, a sin t + b cos t),  t = p freq[e]
 * the rest of the head is kept. t is formed and reduced to one turn in fp64, so
 * far positions cost no accuracy; the turn itself is fp32.
 *   freq   device fp64 [rot/2], radians per position, 8-byte aligned
 *   pos    device int32 [T] (negative ones allowed)
 *   rot    a multiple of 8, 8 <= rot <= d */
enum { WL_ROPE_HALF = 0, WL_ROPE_INTERLEAVED = 1 };
typedef struct {
    const double *freq;
    const int32_t *pos;
    int32_t rot, style;
    float scale;
} wl_rotary;

/* Frequencies of wl_rotary for `rot` rotated elements, on the host:
 *   WL_ROPE_PLAIN   f_e = base^(-2e/rot)
 *   WL_ROPE_LINEAR  f_e / factor (positions interpolated)
 *   WL_ROPE_BASE    base replaced by base factor^(rot/(rot-2)): the slowest pair
 *                   turns `factor` times slower, the fastest as before
 *   WL_ROPE_PARTS   by parts: with n_e = original f_e / (2 pi) turns over the
 *                   original context and g = clamp((n_e - slow)/(fast - slow), 0, 1),
 *                   f_e (g + (1 - g)/factor); *scale = 0.1 ln(factor) + 1
 *                   (*scale is 1 in the others)
 * freq: host fp64 [rot/2], written. base > 1, factor >= 1, original > 0,
 * fast > slow (the last three in WL_ROPE_PARTS only); rot as in wl_rotary, and
 * above 2 pairs in WL_ROPE_BASE. */
enum { WL_ROPE_PLAIN = 0, WL_ROPE_LINEAR = 1, WL_ROPE_BASE = 2, WL_ROPE_PARTS = 3 };
wl_status wl_rope_frequencies(int32_t rot, double base, int32_t scaling, double factor, double original,
                              double slow, double fast, double *freq, float *scale);

/* Q and K rotated (and normalised per head first, where weights are given):
 *   head -> rotary( q_weight ? rms(head) (q_weight + offset) : head )
 *   q, q_out  [T] rows of n_q heads of d; q_out may be q
 *   k, k_out  [T] rows of n_k heads of d; k_out may be k
 *   q_weight, k_weight  [d] or NULL
 *   rotary    NULL: no rotation (per-head norm only)
 * n_q >= 0, n_k >= 0, not both 0 (pointers of an empty side are ignored);
 * d: a multiple of 8, at most 256. */
typedef struct {
    const void *q, *k, *q_weight, *k_weight;
    void *q_out, *k_out;
    const wl_rotary *rotary;
    int32_t T, n_q, n_k, d, ldq, ldk, ldq_out, ldk_out, dtype;
    float eps, offset;
} wl_rope_args;
wl_status wl_rope(const wl_rope_args *a, void *hip_stream);

/* A paged cache of keys and values.
 *   k, v     [n_pages][n_kv][page][d] of the format's type, 16-byte aligned
 *   k_scale, v_scale  fp32 [n_pages][n_kv][page], 16-byte aligned, in the
 *            quantised formats (ignored in the others)
 *   table    device int32 [n_seq][max_pages]: the page that holds slots
 *            [i page, (i+1) page) of a sequence. A page number outside
 *            [0, n_pages) is no page: nothing is written to or read from it.
 * Formats: WL_CACHE_BF16, WL_CACHE_F32, and one byte per element with one scale
 * per token and head, most = the row's largest magnitude:
 *   WL_CACHE_INT8  scale = most / 127, code = round(127 x / most)
 *   WL_CACHE_E4M3  scale = most / 448, code = e4m3(448 x / most)  (OCP, finite)
 * to nearest even; a row of zeros has scale 0, and a row with an infinity or a
 * NaN reads back as NaN. dtype bf16 goes with bf16, int8 and e4m3 caches, dtype
 * f32 with f32, int8 and e4m3 ones (else WL_ERR_UNSUPPORTED).
 * page: a power of two from 16 to 1024; d: a multiple of 16, at most 256. The
 * pools may hold more than 2^31 elements. */
enum { WL_CACHE_BF16 = 0, WL_CACHE_F32 = 1, WL_CACHE_INT8 = 2, WL_CACHE_E4M3 = 3 };
typedef struct {
    void *k, *v;
    float *k_scale, *v_scale;
    const int32_t *table;
    int32_t n_pages, page, n_kv, d, n_seq, max_pages, format;
} wl_cache;

/* Writes tokens into the cache, with wl_rope's norm and rotation of K, and of Q
 * beside it, in the same launch. K is stored as rounded once from the fp32
 * rotated value, V as it is.
 *   k, v   [T] rows of cache->n_kv heads of cache->d
 *   seq    device int32 [T]: the sequence of each token. A token whose seq is
 *          outside [0, n_seq) is skipped: nothing of it is written, q_out neither.
 *   slot   device int32 [T]: its place in the sequence. A slot outside
 *          [0, max_pages page) or without a page: K and V are not written.
 *   q, q_out  [T] rows of n_q heads, q_out may be q; n_q == 0: no Q
 *   rotary    NULL: no rotation. Its pos may be NULL: the slots are the positions
 *   q_weight, k_weight, eps, offset  as in wl_rope
 * Two tokens of one call with the same seq and slot: either may be stored, whole
 * elements of both may be mixed. */
typedef struct {
    const wl_cache *cache;
    const void *k, *v, *q, *q_weight, *k_weight;
    void *q_out;
    const int32_t *seq, *slot;
    const wl_rotary *rotary;
    int32_t T, n_q, ldk, ldv, ldq, ldq_out, dtype;
    float eps, offset;
} wl_cache_write_args;
wl_status wl_cache_write(const wl_cache_write_args *a, void *hip_stream);

/* Reads tokens back: k_out, v_out [T] rows of n_kv heads of d, as dtype. A token
 * whose seq, slot or page is invalid (as in wl_cache_write) leaves its rows as
 * they were. k_out or v_out may be NULL. */
typedef struct {
    const wl_cache *cache;
    const int32_t *seq, *slot;
    void *k_out, *v_out;
    int32_t T, ldk, ldv, dtype;
} wl_cache_read_args;
wl_status wl_cache_read(const wl_cache_read_args *a, void *hip_stream);

/* Attention of new tokens over the cache, which holds them already:
 *   o = sum_j w_j v_j,  w = softmax_j( scale q . k_j )  over the visible keys j
 * for every query head h, with key/value head h / (n_q / n_kv).
 *   q, o      [T] rows of n_q heads of cache->d (o may be q)
 *   q_start   device int32 [n_seq + 1]: rows [q_start[s], q_start[s+1]) of q are
 *             sequence s's, rows outside every sequence are left as they were
 *   kv_len    device int32 [n_seq]: keys of the sequence, the new tokens' last.
 *             Query i of m has its own key in slot kv_len - m + i.
 *   max_q, max_kv  (max_kv <= 2^30) the largest q_start[s+1] - q_start[s] and kv_len[s]: these fix
 *             the launch. Queries beyond max_q get no result, keys beyond max_kv
 *             (or beyond max_pages page) are not seen.
 *   mask      WL_ATTN_CAUSAL  query i sees the slots up to its own
 *             WL_ATTN_TREE    every slot before the new tokens, and new token j
 *                             where bit j % 32 of tree[row][j / 32] is set
 *             WL_ATTN_FULL    every slot below kv_len
 *   tree      device [T][tree_words] (WL_ATTN_TREE only)
 *   window    0, or how many positions back a query sees: of a query at position
 *             p, slots above p - window (in WL_ATTN_TREE the mask alone decides
 *             over new tokens; not in WL_ATTN_FULL)
 *   q_pos     device int32 [T]: the queries' positions for the window in
 *             WL_ATTN_TREE; NULL means their slots
 * A query that sees no key, or whose every score is -inf, gives zeros. A key
 * that a query does not see has no influence on it, whatever it holds; the same
 * goes for slots from kv_len on. n_q is a multiple of n_kv.
 * Products of bf16 tensors run on the matrix cores with fp32 sums. For the
 * second product a weight (times its key's v_scale, in the quantised formats) is
 * rounded to bf16 (2^-8 of it at most), with the remainder as a second bf16 (then
 * 2^-16) where a call is small: with rows = min(max_q, T) n_q / n_kv, rows <= 64 or
 * n_seq n_kv ceil(rows / 64) <= 32. Without the remainder, a bf16 cache's weights
 * are summed as rounded too. dtype f32 is fp32 throughout.
 * max_kv does not change what is rounded; the order of the fp32 sums follows the
 * division of the keys, which depends on max_kv and on all sequences' lengths, so
 * that a query's last bits may differ with the batch it is in.
 *   ws   ws_bytes >= wl_attention_workspace_bytes(a), prepared as the other
 *        operations' (its first WL_SYNC_BYTES are not touched, so that one
 *        workspace serves a whole layer); NULL is accepted where that is 0 */
enum { WL_ATTN_CAUSAL = 0, WL_ATTN_TREE = 1, WL_ATTN_FULL = 2 };
typedef struct {
    const wl_cache *cache;
    const void *q;
    void *o;
    const int32_t *q_start, *kv_len;
    const uint32_t *tree;
    const int32_t *q_pos;
    int32_t T, n_q, ldq, ldo, max_q, max_kv, mask, window, tree_words, dtype;
    float scale;
} wl_attention_args;
/* 0 for invalid arguments too (the call then says which). */
size_t wl_attention_workspace_bytes(const wl_attention_args *a);
wl_status wl_attention(const wl_attention_args *a, void *ws, size_t ws_bytes, void *hip_stream);

/* Steps of whole layers: wl_step_create for a list that mixes projection calls
 * with the operations above, so that a decode step of a model is one graph.
 *   op    WL_OP_LINEAR, WL_OP_QKV, WL_OP_MLP: args is a wl_call (whose op says
 *         the same); the others: args is the operation's argument struct
 * Launched and destroyed as any step; positions, slots, lengths, page tables are
 * read at each launch, max_q and max_kv are fixed here (give the largest that
 * the step will meet). Every operation is checked as by its own entry point. */
enum { WL_OP_NORM = 3, WL_OP_ROPE = 4, WL_OP_CACHE_WRITE = 5, WL_OP_CACHE_READ = 6, WL_OP_ATTENTION = 7 };
typedef struct {
    int32_t op;
    const void *args;
} wl_step_op;
size_t wl_step_ops_workspace_bytes(const wl_step_op *ops, int32_t n_ops);
wl_status wl_step_create_ops(const wl_step_op *ops, int32_t n_ops, void *ws, size_t ws_bytes, wl_step *step);

/* Size of a set of theta bundles against the dense weights they replace
 * ("What weightless inference costs", "Compression": the ratio of the theta
 * bundle, W0 + s + U + V across every layer and family, to the original
 * projection weights). For th[0 .. n_th):
 *   *bundle_bytes = e d_out d_in once per distinct W0 pointer
 *                   + per theta: 4 d_out (when s is not NULL) + e r (d_out + d_in)
 *   *dense_bytes  = per theta: e d_out d_in (the weight it stands for)
 * with e = 2 for bf16 thetas and 4 for fp32 ones.
 * Thetas that share a W0 pointer must share its shape and dtype (else
 * WL_ERR_INVALID_ARG). Host only: reads the structs, never the tensors. */
wl_status wl_bundle_size(const wl_theta *const *th, int32_t n_th,
                         size_t *bundle_bytes, size_t *dense_bytes);

/* Reconstruction fidelity ("What weightless inference costs", "Reconstruction
 * fidelity"): result[0] = ||W - R||_F / ||W||_F, accumulated in fp64 (the
 * differences and squares of bf16 values are exact there), in a fixed order
 * that depends on n only.
 *   W, R    bf16 [n] device tensors, 16-byte aligned: e.g. an original weight
 *           and the W_eff of wl_materialize_weff
 *   n       elements, 1 <= n < 2^40
 *   result  device pointer to one double, 8-byte aligned, written
 *   ws      workspace, ws_bytes >= wl_rel_frob_workspace_bytes(n)
 * When ||W||_F is 0 the result is 0 if R equals W and +inf otherwise. */
size_t wl_rel_frob_workspace_bytes(int64_t n);
wl_status wl_relative_frobenius_error(const void *W, const void *R, int64_t n, double *result,
                                      void *ws, size_t ws_bytes, void *hip_stream);

/* Prepares a projection workspace: clears its sync area (the first
 * WL_SYNC_BYTES) with a kernel enqueued on hip_stream. Needed once before the
 * workspace's first use by wl_linear, wl_qkv_fused or wl_mlp_fused, and again
 * after anything else has written that area (the calls write it with
 * generation-tagged words that are never reset; a tag left by foreign data
 * could make a later call take a stale value). ws must be 256-byte aligned and
 * ws_bytes >= WL_SYNC_BYTES (else WL_ERR_INVALID_ARG / WL_ERR_WORKSPACE). */
wl_status wl_workspace_init(void *ws, size_t ws_bytes, void *hip_stream);

/* WL_SYNC_BYTES of the built library. */
size_t wl_sync_bytes(void);

/* Static description of a status code. */
const char *wl_status_str(wl_status status);

/* Message describing the last non-WL_OK return on the calling thread ("" after
 * a success). The pointer stays valid until the thread's next library call. */
const char *wl_last_error(void);

/* WL_ABI_VERSION of the built library. */
int32_t wl_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* WL_H */
