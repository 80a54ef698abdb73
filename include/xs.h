/*
 * xs.h - C ABI of libxs: non-causal attention fused with the post-attention
 * Ulysses All-to-All layout, for one GB300 (sm_103a).
 *
 * Source of the operations: "X-Stage: An Overlooked Pipeline Stage for
 * Communication-Computation Overlap in DiT Inference" (arXiv 2607.23264).
 *  - Abstract: for Ulysses sequence-parallel attention, the post-attention
 *    All-to-All is fused tile by tile into FlashAttention, so that the owner of
 *    an output tile issues its stores itself and resumes computation, with no
 *    dedicated communication warp or SM; compared against serial execution
 *    (FlashAttention, then the All-to-All) and FlashAttention alone.
 *  - Figure 5 (d)-(e): FlashAttention produces each head partition's output and
 *    the post-attention All-to-All restores the original sequence partition.
 *  - Figure 1 / Figure 7: the stores of one output tile drain while the next
 *    mainloop computes (the piggybacked FlashAttention-A2A pipeline).
 *
 * What every attention entry point computes, per batch b and head h:
 *     o[b][h][n][:] = softmax_j( q[b][h][n][:] . k[b][h][j][:] / sqrt(d) ) v[b][h][j][:]
 * over all N keys (non-causal, no mask, no dropout), fp32 accumulation, output
 * rounded to bf16 (round to nearest even).
 *
 * The layout ("shards"): destination p (0 <= p < P) receives the contiguous
 * sequence block [p*N/P, (p+1)*N/P) of every head:
 *     shard_p[b][i][h][c] = o[b][h][p*(N/P) + i][c],   0 <= i < N/P.
 * On one GPU the P destinations are P separate device buffers.
 *
 * Conventions shared by all calls
 *  - Element type: every buffer is bf16 (2 bytes), in device memory.
 *  - q, k, v, o: [B][H][N][d], contiguous (d fastest).
 *  - shard p: [B][N/P][H][d], contiguous; out_shards is a HOST array of P
 *    device pointers, read during the call (the array may be freed afterwards).
 *  - Ownership: the caller owns every buffer. The library allocates no device
 *    memory; it keeps only a device status word (see xs_last_device_status)
 *    and the fixed scratch array of xs_attn_serial_noalloc. An optional
 *    caller-owned workspace (xs_set_workspace) enables a balanced schedule.
 *  - Asynchrony: each call only enqueues work on `stream` (a cudaStream_t; NULL
 *    means the legacy default stream) and returns without synchronising. Launch
 *    errors are reported as XS_ERR_CUDA. Kernel-side waits are bounded: a wait
 *    that runs out records XS_ERR_TIMEOUT in the status word and the kernel
 *    returns, leaving the context usable.
 *  - Aliasing: inputs, outputs and shards must not overlap.
 *  - Threads: calls on different streams are independent.
 *  - Validation, in this order, before any device work:
 *      XS_ERR_INVALID     a NULL pointer (also any NULL shard), B, N or H < 0,
 *                         P not in [1, 8], N % P != 0,
 *                         store_tile not in {1, 2, 4, 8};
 *      XS_ERR_UNSUPPORTED d not in {64, 128, 256}, N % 128 != 0, d = 256
 *                         with store_tile != 8 (at d = 256 every finished tile
 *                         is stored at once: a deferred tile does not fit on
 *                         chip beside the K/V ring), or B*H*N >= 2^31 (the
 *                         kernels address rows with 32-bit coordinates);
 *      XS_ERR_ALIGN       a pointer that is not 16-byte aligned.
 *    B == 0, H == 0 or N == 0 is an empty problem: the call validates its
 *    other arguments and returns XS_OK without launching anything.
 */
#ifndef XS_H
#define XS_H

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  XS_OK = 0,
  XS_ERR_INVALID = 1,
  XS_ERR_UNSUPPORTED = 2,
  XS_ERR_ALIGN = 3,
  XS_ERR_CUDA = 4,
  XS_ERR_TIMEOUT = 5
} xs_status;

/* Fused attention + shard layout (abstract: tile-granular fusion of the
 * post-attention All-to-All with FlashAttention; Figure 7). One persistent
 * kernel (d = 64 and 128: two query tiles per CTA; d = 256: one query tile per
 * CTA with its scores double-buffered on chip). Each finished 128-row output
 * tile is staged on chip and written into the P shards by the warps that own
 * it, in bursts of `store_tile` 16-row slabs interleaved with the KV
 * iterations of that warp group's next tile (store_tile = 8, or a tile with no
 * next tile on its SM: the whole tile right after it is finished).
 * The result does not depend on store_tile.
 *   q, k, v     [B][H][N][d] bf16, device.
 *   out_shards  host array of P device pointers, shard p [B][N/P][H][d] bf16.
 *   store_tile  1, 2, 4 or 8 slabs per burst (8 only at d = 256). */
xs_status xs_attn_fused(const void *q, const void *k, const void *v,
                        void *const *out_shards, int B, int N, int H, int d,
                        int P, int store_tile, void *stream);

/* Flags of xs_attn_fused_ex. */
#define XS_FLAG_COMPLETION_COUPLED 1

/* xs_attn_fused with two experiment controls for the residual-slope test
 * (Pith review of X-Stage, "If this is right": the completion-coupled model,
 * where the issuer is blocked until its stores are visible, predicts a
 * residual over FlashAttention alone that grows linearly with sequence length,
 * while X-Stage predicts a flat one; Figure 11 caption: relative
 * sender-visible residual E_res(M)/T_FA; referee summary: per-tile
 * remote-store span distributions).
 *   flags  0, or XS_FLAG_COMPLETION_COUPLED: after issuing a finished tile's
 *          stores the issuing thread waits until they have completed before
 *          its warp group resumes (requires store_tile 8).
 *   spans  NULL, or a device buffer of 2*B*H*(N/128) unsigned 64-bit values,
 *          all zero on entry (8-byte aligned): for output tile
 *          t = (b*H + h)*(N/128) + n/128, spans[2t] and spans[2t + 1] receive
 *          the %globaltimer (ns) at which its first slab was issued and at which
 *          the last of its issuing warps was released.
 * Output bytes are identical to xs_attn_fused. Other flag bits, or the
 * coupled flag with store_tile != 8: XS_ERR_INVALID. */
xs_status xs_attn_fused_ex(const void *q, const void *k, const void *v,
                           void *const *out_shards, int B, int N, int H, int d,
                           int P, int store_tile, int flags,
                           unsigned long long *spans, void *stream);

/* Attention alone (the FlashAttention-alone time the abstract compares the
 * fused kernel with): same kernel, output written head-major to
 * o [B][H][N][d] bf16 (device). */
xs_status xs_attn(const void *q, const void *k, const void *v, void *o, int B,
                  int N, int H, int d, void *stream);

/* The layout alone (the separate post-attention All-to-All of serial
 * execution, Figure 5 (e)), as a bit-exact copy kernel:
 * o [B][H][N][d] -> shards. Any 16-bit payload is copied unchanged. */
xs_status xs_scatter(const void *o, void *const *out_shards, int B, int N,
                     int H, int d, int P, void *stream);

/* Serial execution (abstract: the baseline of the sender-visible speedup):
 * xs_attn into the caller's o_scratch [B][H][N][d] bf16, then xs_scatter into
 * the shards, two launches on `stream`. o_scratch holds o afterwards. */
xs_status xs_attn_serial(const void *q, const void *k, const void *v,
                         void *o_scratch, void *const *out_shards, int B, int N,
                         int H, int d, int P, void *stream);

/* Ulysses sequence-parallel attention with BOTH All-to-Alls fused (Figure 5:
 * QKV projection and the pre-attention All-to-All turn sequence-partitioned
 * tokens into head partitions (a)-(c); FlashAttention and the post-attention
 * All-to-All produce the output and restore the sequence partition (d)-(e)).
 * The inputs stay in the sequence partition: q_shards[p], k_shards[p],
 * v_shards[p] (host arrays of P device pointers) are [B][N/P][H_total][d] bf16,
 * the tokens [p*N/P, (p+1)*N/P) of every head, as each rank holds them after
 * the QKV projection. The call computes attention over all N tokens for the
 * heads [h0, h0 + H) only (the head partition one rank owns after the
 * pre-attention All-to-All), reading its Q/K/V tiles straight from the
 * sequence shards, and stores output row n of head h0 + h into
 * out_shards[n / (N/P)][b][n % (N/P)][h0 + h][:] (destinations [B][N/P][H_total][d]),
 * the owner of each tile issuing the stores as in xs_attn_fused. On one GPU,
 * h0 = 0 and H = H_total does the whole layer; P calls with
 * h0 = r*H_total/P, H = H_total/P do rank r's share each.
 * Validation as xs_attn_fused, plus: XS_ERR_INVALID for NULL arrays or
 * entries, H_total < 1, h0 < 0, H < 0 or h0 + H > H_total;
 * XS_ERR_UNSUPPORTED unless N/P is a multiple of 128 (a 128-row tile never
 * straddles two input shards); XS_ERR_ALIGN for unaligned shard pointers.
 * H == 0 is an empty call. Heads outside [h0, h0 + H) of the destinations are
 * not touched. */
xs_status xs_attn_ulysses(const void *const *q_shards, const void *const *k_shards,
                          const void *const *v_shards, void *const *out_shards, int B,
                          int N, int H_total, int h0, int H, int d, int P,
                          int store_tile, void *stream);

/* Store-burst probe for the Burst-Gap model (Pith review of X-Stage, "What
 * carries the argument" and "What would settle it": zero-gap periodic bursts
 * give the drain rate R, a recovered large-gap plateau the backpressure-free
 * issue time T_iss^0, the isolated-burst knee the outstanding capacity Q;
 * Figure 3 caption). Local form: the stores go to this GPU's own memory.
 * K producer CTAs (128 threads each) each issue n_bursts bursts of burst_bytes
 * into fresh memory, separated by gap_ns nanoseconds without stores. For
 * producer c and burst b, times[2*(c*n_bursts + b)] and [.. + 1] receive the
 * %globaltimer values (ns) at which the CTA started issuing the burst and at
 * which every store had been issued.
 *   dst       device buffer of dst_bytes >= K*n_bursts*burst_bytes (16-byte aligned)
 *   times     device buffer of 2*K*n_bursts unsigned 64-bit values (8-byte aligned)
 *   mode      0: posted st.global.v4 from all threads; 1: TMA bulk copies from
 *             shared memory, span ending when their source has been read
 *   XS_ERR_INVALID for NULL pointers, K not in [1, 1024], n_bursts < 1,
 *   burst_bytes not a positive multiple of 2048, gap_ns > 1e9, a bad mode or a
 *   too small dst; XS_ERR_ALIGN for misaligned pointers. */
xs_status xs_store_burst_probe(void *dst, unsigned long long dst_bytes, int K,
                               unsigned long long burst_bytes, int n_bursts,
                               unsigned long long gap_ns, int mode,
                               unsigned long long *times, void *stream);

/* Size of the scratch array that xs_attn_serial_noalloc uses: 32 MiB. */
#define XS_NOALLOC_SCRATCH_BYTES (32ull << 20)

/* Serial execution without a caller-supplied intermediate buffer, for callers
 * that cannot allocate device memory (for example code embedded in a host
 * framework that owns all device memory through its own allocator or a fixed
 * memory plan, or loops where a cudaMalloc would synchronise the device).
 * The paper has no counterpart to this entry point; it only changes where the
 * intermediate o of xs_attn_serial lives.
 * Same arguments, results and validation as xs_attn_serial minus o_scratch:
 * the intermediate o [B][H][N][d] bf16 lives in one array of
 * XS_NOALLOC_SCRATCH_BYTES compiled into the library, which every GPU that
 * loads the library holds until the process exits. Nothing is allocated:
 * no cudaMalloc, cudaFree or allocating library call.
 *   - XS_ERR_INVALID if B*H*N*d*2 bytes exceed XS_NOALLOC_SCRATCH_BYTES
 *     (checked first, factor by factor so no product wraps, before any device
 *     work).
 *   - Every call looks up the array's device address on the current device
 *     (a symbol lookup, no allocation), so a device reset that reloads the
 *     library's device code cannot leave a stale address in use. The first
 *     call on a device may load that code: make it before any stream capture.
 *   - Every call on a device shares the one array and leaves the last call's o
 *     in it (each call overwrites all of the o it reads, so nothing needs
 *     clearing). Calls that overlap on the GPU (different streams, or
 *     different host threads without ordering) race on the array. */
xs_status xs_attn_serial_noalloc(const void *q, const void *k, const void *v,
                                 void *const *out_shards, int B, int N, int H,
                                 int d, int P, void *stream);

/* Balanced schedule with a workspace (a scheduling aid of this implementation;
 * the paper has no counterpart). The attention kernel runs one persistent CTA
 * per SM. Without a workspace each CTA takes whole units (a head and a pair of
 * 128-row query tiles) in turn, so when the units do not divide evenly over
 * the SMs the last wave leaves SMs idle. With a workspace the launch may
 * instead give every CTA an equal contiguous range of the (unit, 128-key tile)
 * iterations (a "stream-K" schedule): a unit cut by a range boundary is
 * computed in pieces on consecutive CTAs, each piece leaves its partial result
 * (unnormalised output rows, running maximum, row sum; fp32) in the workspace,
 * and the CTA finishing a unit's last piece merges the pieces with the
 * online-softmax rescaling identity and stores the output tile as usual (into
 * o, or into the shards). The library chooses per launch, from the shape and
 * the SM count, whichever schedule its cost model finds shorter. Results agree
 * with the whole-unit schedule within fp32 rounding of the merge (they are not
 * bit-identical to it) and are identical from launch to launch.
 *
 * XS_WORKSPACE_HEADER_BYTES: the first bytes of a workspace hold per-unit
 * counters that must be zero before a launch; the launches leave them zero. */
#define XS_WORKSPACE_HEADER_BYTES 16384ull

/* Registers (ws != NULL) or removes (ws == NULL) the caller's device workspace
 * for the current device. Later attention launches on that device (every entry
 * point above that computes attention) use it when the balanced schedule is
 * shorter and `bytes` suffice; otherwise they take whole units. The caller
 * keeps ownership and must keep the buffer alive until it removes it.
 *   ws     device memory, 256-byte aligned (XS_ERR_ALIGN otherwise)
 *   bytes  >= XS_WORKSPACE_HEADER_BYTES (XS_ERR_INVALID otherwise)
 * The call zeroes the header on `stream` and synchronises it (XS_ERR_CUDA on
 * failure). Launches that use one workspace must not overlap on the GPU
 * (different streams without ordering race on it). After a launch reported
 * XS_ERR_TIMEOUT (xs_last_device_status), register the workspace again to
 * re-zero its counters. */
xs_status xs_set_workspace(void *ws, unsigned long long bytes, void *stream);

/* For an attention launch of this shape on the current device with an
 * unlimited workspace: *bytes = the workspace it would use and *cut = 1 if it
 * would take the balanced schedule (*bytes = 0 and *cut = 0 for whole units).
 * cut may be NULL. XS_ERR_INVALID for a NULL bytes or B, N, H < 0;
 * XS_ERR_UNSUPPORTED for d not in {64, 128, 256} or N % 128 != 0; XS_ERR_CUDA if
 * the device cannot be queried. */
xs_status xs_workspace_bytes(int B, int N, int H, int d, unsigned long long *bytes, int *cut);

/* Element types of the calls that take more than bf16. */
#define XS_BF16 0
#define XS_FP16 1
#define XS_FP32 2

/* One tensor of an xs_rope call: `heads` heads of rows of d contiguous values on
 * both sides, strides in elements (batch, token, head). */
typedef struct {
  const void *x;           /* input, device */
  void *y;                 /* output, device; x itself for an update in place */
  const float *weight;     /* [d] fp32 (device): RMS-norm the row first; NULL: no norm */
  long long x_stride[3];   /* batch, token, head; 0 repeats one row */
  long long y_stride[3];
  int heads;
  int rotate;              /* 0: the row keeps its position (v, or text tokens) */
} xs_rope_tensor;

/* Flag of xs_rope: column 2i pairs with 2i + 1; without it column i of the
 * rotated part pairs with i + rot/2. */
#define XS_ROPE_ADJACENT 1

/* Rotary positions with several axes (time, height, width of an image or video
 * token), with the per-head RMS norm of q and k that goes before them: the step
 * between the QKV projection and attention (Figure 5 (a)-(c): sequence-partitioned
 * tokens become head partitions; the figure does not show positions, this call is
 * this library's). Up to three tensors (q, k, v) in one launch, typically from the
 * projection's token-major [B][N][heads][d] to the head-major [B][heads][N][d] of
 * the attention calls, or in place in the sequence shards that xs_attn_ulysses
 * reads. Per row, in fp32, rounded once at the end:
 *     x <- x / sqrt(mean(x^2) + eps) * weight            where weight is given
 *     (x_a, x_b) <- (x_a cos t - x_b sin t, x_b cos t + x_a sin t),  t = pos[axis] * f
 * for every pair of the first rot = sum(axis_dims) columns of a rotated tensor; the
 * other columns stay. The norm holds for rows of any finite values (squares past fp32's
 * range included); a row of zeros stays one, with eps = 0 too. Pair i (in the order of
 * the axes) has frequency freqs[i] and belongs to the axis whose axis_dims[a]/2 pairs
 * hold it. t modulo a turn is off by 2^-25 of a turn at most, for every 32-bit position
 * and every frequency; negated positions undo a rotation.
 *   pos               int32 (device), token n of batch entry b at
 *                     pos + b*pos_batch_stride + n*n_axes; stride 0 shares one list
 *   axis_dims, freqs  HOST arrays (n_axes entries; rot/2 radians per step), read
 *                     during the call
 *   in_type, out_type XS_BF16, XS_FP16 or XS_FP32; equal, or out_type XS_BF16
 * Outputs must not overlap each other or another tensor's input.
 * XS_ERR_INVALID for NULL pointers (weight, and the pointers of a tensor of no heads,
 * aside), n_tensors not in [1, 3], negative sizes or strides, n_axes not in [1, 4], an
 * axis width that is odd, below 2 or past d, eps negative or not finite, a frequency
 * that is not finite, unknown flags or types, output rows that overlap (a stride below d
 * over more than one row), or x == y with other strides or another type.
 * XS_ERR_UNSUPPORTED for d not a multiple of 8 in [8, 256], pairs i, i + rot/2 with rot
 * not a multiple of 8, other type pairs, a frequency of 2^64 or more, B*N >= 2^31 or
 * more than 65535 heads. XS_ERR_ALIGN unless x, y and weight are 16-byte aligned and
 * every stride over more than one row is a multiple of 16 bytes. The strides of a tensor
 * without rows are not looked at.
 * Empty problems return XS_OK. */
xs_status xs_rope(const xs_rope_tensor *tensors, int n_tensors, const int *pos,
                  long long pos_batch_stride, const int *axis_dims, int n_axes,
                  const double *freqs, int B, int N, int d, float eps, int flags,
                  int in_type, int out_type, void *stream);

/* Operands of differential attention. q [B][H][Nq][d], k and v [B][H_kv][Nk][d] bf16
 * (device), rows of d contiguous values, strides in elements (batch, head, row);
 * head h reads k/v head h / (H / H_kv). */
typedef struct {
  const void *q, *k, *v;
  long long q_stride[3], k_stride[3], v_stride[3];
  const float *lambda;        /* [H] fp32 (device): the second map's weight, per head */
  const float *norm_weight;   /* [d] fp32 (device), or NULL: no norm */
  const int *kv_len;          /* [B] int32 (device), or NULL: Nk keys everywhere */
  float scale;                /* of the scores; 1/sqrt(d/2) is the usual one */
  float eps, out_scale;       /* of the norm; a factor on the result */
  int B, H, H_kv, Nq, Nk, d;
} xs_diff_args;

/* Differential attention (this library's own addition beside xs_attn: same element
 * type, head dimensions and output layouts). A head's d columns hold two maps,
 * q = [q1 | q2] and k = [k1 | k2] of d/2 columns each, over one v of d columns:
 *     x = (softmax(q1 k1^T * scale) - lambda[h] softmax(q2 k2^T * scale)) v
 *     o = x / sqrt(mean(x^2) + eps) * norm_weight * out_scale
 * (norm_weight NULL: o = x * out_scale), both softmaxes over the first kv_len[b] keys
 * (taken into [0, Nk]; what lies behind them is not used, NaN and infinity included),
 * non-causal. A batch entry without keys gives zeros, a map whose scores of a row are
 * all -inf (they overflowed) gives 0 there, and a row x of zeros stays one under the
 * norm, with eps = 0 too; the norm holds for rows x of any finite values (squares past
 * fp32's range included). Scores times scale are taken below 2^30 in magnitude (beyond
 * it fp32 no longer holds a weight's exponent, and a row may come out as zeros or not
 * a number). fp32 accumulation and statistics, softmax weights
 * rounded to bf16 for the product with v, output rounded to bf16. Outputs must not
 * overlap each other or an input.
 * lambda is taken as it is: a model computes it once from its learned vectors, for
 * example exp(a1.b1) - exp(a2.b2) + lambda_init, with out_scale = 1 - lambda_init.
 * Nq, Nk: any size, also 1 (one new token against a long sequence); not multiples of
 * 128 either.
 *   o, o_stride  [B][H][Nq][d] bf16 (device), strides in elements (batch, head, row)
 *   out_shards   host array of P device pointers, shard p [B][Nq/P][H][d] bf16, as in
 *                xs_attn_fused; the CTA that finishes a row stores it in its shard
 *   ws           caller-owned device memory, 256-byte aligned, whose first
 *                XS_WORKSPACE_HEADER_BYTES are zero before the first call (each call
 *                leaves them zero), or NULL. With xs_diff_workspace_bytes of it a
 *                launch may cut units into ranges of keys over all SMs (few queries,
 *                a last wave that is not full, ragged lengths); with less it takes
 *                whole units. At d = 256 a CTA also keeps the first map's rows in it
 *                (fp32, 128 KB for 128 queries) while the second map's are computed:
 *                with less than XS_WORKSPACE_HEADER_BYTES + 1024 * min(128, Nq rounded
 *                up to 8) bytes a norm is refused, with places for fewer CTAs than SMs
 *                fewer SMs work under a norm; without one a call may run both maps at
 *                once on each half of v's columns (their scores computed twice), which
 *                needs no workspace, and takes what should end first. Calls that
 *                share one workspace must not overlap on the GPU. After a timeout
 *                (xs_last_device_status) zero the header again.
 * Results are the same from launch to launch on one GPU model; they differ in fp32
 * rounding between workspace and none.
 * XS_ERR_INVALID for NULL args, q, lambda, output or (Nk > 0) k, v; negative sizes;
 * H not a multiple of H_kv; scale not positive and finite, eps negative or not finite,
 * out_scale not finite; P not in [1, 8], Nq % P != 0; a stride below d over more than
 * one row (rows that overlap or repeat); ws NULL with ws_bytes > 0; too small a
 * workspace at d = 256 with a norm. XS_ERR_UNSUPPORTED for d not in {64, 128, 256} or
 * more than 2^31 - 1 tiles of 128 queries. XS_ERR_ALIGN for q, k, v, norm_weight or an
 * output that is not 16-byte aligned, strides over more than one row that are not
 * multiples of 8, or a ws that is not 256-byte aligned. Empty problems return XS_OK. */
xs_status xs_diff_attn(const xs_diff_args *args, void *o, const long long *o_stride,
                       void *ws, unsigned long long ws_bytes, void *stream);
xs_status xs_diff_attn_fused(const xs_diff_args *args, void *const *out_shards, int P,
                             void *ws, unsigned long long ws_bytes, void *stream);

/* *bytes = the workspace with which a call of this shape on the current device (norm:
 * 1 if it has a norm weight) can take every schedule. XS_ERR_INVALID for a NULL bytes
 * or negative sizes, XS_ERR_UNSUPPORTED for d not in {64, 128, 256}, XS_ERR_CUDA if
 * the device cannot be queried. */
xs_status xs_diff_workspace_bytes(int B, int H, int Nq, int Nk, int d, int norm,
                                  unsigned long long *bytes);

/* A quantised key/value cache: pages of rows (one token, one k/v head, d values) in
 * e4m3, each row with a power of two as its scale. Row i of head h of a page is
 * page * H_kv * page_size + h * page_size + i; its values are code * 2^(byte - 127),
 * codes in k or v at row * d, the byte in k_scale or v_scale at row. A byte of 255
 * makes the whole row NaN, the codes 0x7f and 0xff are NaN under any byte. xs_cache_write
 * gives bytes from 7 to 246 and 255; under bytes from 247 to 254 what is past the largest
 * bf16 counts as an infinity in bf16 outputs and among values under attention, and may
 * do so among keys. The caller owns all four arrays (device). */
typedef struct {
  void *k, *v;                         /* [n_pages][H_kv][page_size][d] e4m3 */
  unsigned char *k_scale, *v_scale;    /* [n_pages][H_kv][page_size] */
  int n_pages, H_kv, page_size, d;     /* page_size: a power of two in [16, 1024] */
} xs_cache;

/* One list of pages for each request: place i of request b is row i % page_size of page
 * pages[b * stride + i / page_size]. Lists may share pages. */
typedef struct {
  const int *pages;   /* device */
  long long stride;   /* entries between requests; 0: one list for all */
  int count;          /* entries of a list */
} xs_pages;

/* Quantises rows into a cache (this library's own addition: history that later steps of
 * attention read, kept in half the memory of bf16). Token n < lens[b] of request b goes to
 * place start[b] + n:
 *     e = the least integer with max|x| <= 448 * 2^e, within [-120, 119] (0 for zeros),
 *     codes = e4m3(x * 2^-e), to nearest even, at most 448; byte = e + 127.
 * A row with a NaN or an infinity gets the byte 255. Nothing else of the cache changes:
 * tokens from lens[b] on, and those whose place no page holds (negative, past the list, or
 * a page that is not in [0, n_pages)), are not stored. What a place holds that two tokens of
 * one call go to is not specified (columns and scale may be of different ones).
 *   k, v, strides   [B][H_kv][N][d] of in_type (device), rows of d contiguous values,
 *                   strides in elements (batch, head, token)
 *   start           [B] int32 (device), or NULL: 0
 *   lens            [B] int32 (device), taken into [0, N], or NULL: N
 * XS_ERR_INVALID for NULL cache, lists, k, v, strides or arrays of the cache (with
 * pages), negative sizes or strides, page_size < 1 or an unknown type; XS_ERR_UNSUPPORTED
 * for d not a multiple of 16 in [16, 256], a page_size that is not a power of two in
 * [16, 1024] or H_kv * N >= 2^31; XS_ERR_ALIGN unless k, v and the cache's arrays are
 * 16-byte aligned and every stride over more than one row is a multiple of 16 bytes.
 * Empty problems return XS_OK. */
xs_status xs_cache_write(const xs_cache *cache, const void *k, const void *v,
                         const long long *k_stride, const long long *v_stride,
                         const xs_pages *pages, const int *start, const int *lens, int B,
                         int N, int in_type, void *stream);

/* The rows that a cache stands for, back: arguments and refusals as xs_cache_write, with
 * the outputs k and v of out_type (strides of at least d over more than one row). Values
 * are exact in bf16 and fp32 and rounded to nearest even in fp16. Tokens from lens[b] on
 * are left as they were; those whose place no page holds become NaN. Outputs must not
 * overlap each other or the cache. */
xs_status xs_cache_read(const xs_cache *cache, void *k, void *v, const long long *k_stride,
                        const long long *v_stride, const xs_pages *pages, const int *start,
                        const int *lens, int B, int N, int out_type, void *stream);

/* Operands of attention over a shared prefix. The prefix's keys and values lie in tensors
 * (prefix_k not NULL) or in the pages of `cache` that prefix_pages lists (one list); the
 * requests' own ones in tensors (k not NULL) or in pages of the same cache. Tensors are
 * bf16 (device), rows of d contiguous values, strides in elements. Head h reads k/v head
 * h / (H / H_kv). */
typedef struct {
  const void *q;                        /* [B][H][Nq][d] */
  const void *prefix_k, *prefix_v;      /* [H_kv][Np][d] */
  const void *k, *v;                    /* [B][H_kv][Nk][d] */
  const int *kv_len;                    /* [B] int32 (device), or NULL: Nk own keys everywhere */
  long long q_stride[3];                /* batch, head, row; k and v alike */
  long long prefix_k_stride[2], prefix_v_stride[2];   /* head, row */
  long long k_stride[3], v_stride[3];
  xs_pages prefix_pages, pages;
  xs_cache cache;                       /* not looked at where nothing lies in it */
  float scale;                          /* of the scores; 1/sqrt(d) is the usual one */
  int B, H, H_kv, Nq, Np, Nk, d;        /* Np: keys of the prefix; Nk: own keys at most */
} xs_prefix_args;

/* Attention of a batch of requests that share a prefix (this library's own addition beside
 * xs_attn: same element type and output layouts; several candidates of one prompt, guidance
 * branches, continuations of one history):
 *     o[b][h] = softmax(q[b][h] [K | K_b]^T * scale) [V | V_b]
 * K, V the prefix's Np keys and values of the head, K_b, V_b the first kv_len[b] of the
 * request's own (taken into [0, Nk]; what lies behind them is not used, NaN and infinity
 * included), non-causal. The prefix's keys are read once for a whole tile of queries,
 * whichever requests and heads of one k/v head they belong to. A request without any key
 * gives zeros. fp32 accumulation and statistics, softmax weights rounded to bf16 for the
 * product with v, output rounded to bf16; cached keys and values count as they are. A query
 * that meets cached keys may be taken in two 8-bit parts: exact for values down to 2^-13 of its
 * largest magnitude, to within 2^-21 of that below. A NaN or infinity in a query, or among
 * the keys and values that count, makes NaN of whole rows (or of what the formula gives) of the
 * requests that see it, and touches no other request; a row whose scores are all -inf (they
 * overflowed) gives zeros. Scores times scale are taken below 2^30 in magnitude (beyond it
 * fp32 no longer holds a weight's exponent, and a row may come out as zeros or not a number).
 * A cached key whose place no page holds counts as NaN. Outputs must not overlap each other or an input. Nq, Np, Nk: any size, also 0
 * or 1.
 *   o, o_stride  [B][H][Nq][d] bf16 (device), strides in elements (batch, head, row)
 *   out_shards   host array of P device pointers, shard p [B][Nq/P][H][d] bf16, as in
 *                xs_attn_fused; the warps that finish a row store it in its shard
 *   ws           caller-owned device memory, 256-byte aligned, of any content, or NULL. With
 *                xs_prefix_workspace_bytes of it a launch may cut units into ranges of keys over
 *                all SMs (few queries, a last wave that is not full); with less it takes whole
 *                units. Calls that share one workspace must not overlap on the GPU.
 * Results are the same from launch to launch on one GPU model; they differ in fp32
 * rounding between workspace and none.
 * XS_ERR_INVALID for NULL args, q, output or a NULL of a part that has keys; negative sizes;
 * H not a multiple of H_kv; a cache whose H_kv or d differ; scale not positive and finite;
 * P not in [1, 8], Nq % P != 0; a stride below d over more than one row; ws NULL with
 * ws_bytes > 0. XS_ERR_UNSUPPORTED for d not in {64, 128}, a page_size as in xs_cache_write,
 * a length past 2^29, or 2^31 and more rows of a k/v head or tiles of 128 of them.
 * XS_ERR_ALIGN for a tensor that is not 16-byte aligned, strides over more than one row that
 * are not multiples of 8, or a ws that is not 256-byte aligned. Empty problems return XS_OK. */
xs_status xs_prefix_attn(const xs_prefix_args *args, void *o, const long long *o_stride,
                         void *ws, unsigned long long ws_bytes, void *stream);
xs_status xs_prefix_attn_fused(const xs_prefix_args *args, void *const *out_shards, int P,
                               void *ws, unsigned long long ws_bytes, void *stream);

/* Flags of xs_prefix_workspace_bytes: which part lies in the cache. */
#define XS_PREFIX_CACHED 1
#define XS_OWN_CACHED 2

/* *bytes = the workspace with which a call of this shape on the current device can take
 * every schedule. With more than 128 queries for each k/v head (of all requests and of the
 * heads that share it) that includes room for the cached keys and values in bf16, which such
 * a call reads back first; with less a call reads them as they are, more slowly then.
 * XS_ERR_INVALID for a NULL bytes, negative sizes, other flags or H not a multiple of H_kv,
 * XS_ERR_UNSUPPORTED for d not in {64, 128}, XS_ERR_CUDA if the device cannot be queried. */
xs_status xs_prefix_workspace_bytes(int B, int H, int H_kv, int Nq, int Np, int Nk, int d,
                                    int cached, unsigned long long *bytes);

/* Static English text for a status code; never NULL. */
const char *xs_status_string(xs_status s);

/* Synchronises `stream`, then reads and clears the library's device status
 * word for the current device: XS_ERR_TIMEOUT if a kernel's bounded wait ran
 * out since the last call, XS_ERR_CUDA if the synchronisation failed, else
 * XS_OK. For tests and debugging; the attention calls never block on it. */
xs_status xs_last_device_status(void *stream);

/* Sets the limit, in nanoseconds, after which a kernel's on-chip wait gives up
 * (default 2e9 = 2 s; 0 restores the default). Applies to later launches from
 * this process. Returns the previous limit. */
unsigned long long xs_set_wait_limit_ns(unsigned long long limit_ns);

/* Self-test of the bounded wait: launches one CTA that waits on an on-chip
 * barrier that nothing ever signals, with the current wait limit. The wait
 * must run out, record XS_ERR_TIMEOUT in the status word and return. Read the
 * outcome with xs_last_device_status. */
xs_status xs_selftest_bounded_wait(void *stream);

/* Self-test of the softmax's two exponential paths: for i < n (device fp32
 * buffers), out_poly[i] = 2^x[i] as the attention kernel's polynomial computes
 * it on the FMA pipe for a share of each row (range reduction x = n + f,
 * degree-3 minimax polynomial for 2^f, n added to the exponent; arguments below
 * -126 raised to -126), out_mufu[i] = 2^x[i] from the MUFU unit (ex2.approx,
 * subnormal results flushed to zero). For tests comparing the two against each
 * other and against an error bound. XS_ERR_INVALID for NULL pointers or n < 0. */
xs_status xs_selftest_exp2(const float *x, float *out_poly, float *out_mufu, int n, void *stream);

/* ABI version of this header (1). */
int xs_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* XS_H */
