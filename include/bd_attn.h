/*
 * bd_attn.h -- C ABI of the B200 (sm_100a) block-diffusion attention library
 * (libbdattn.so).
 *
 * Two operations, both exact masked softmax attention with a natural-log
 * log-sum-exp side output:
 *
 *   bd_attn_fwd     training / prefill form over the sequence [x_t ; x_0].
 *   bd_attn_decode  block-decode form: a block of b noisy queries over a
 *                   clean KV cache plus the block itself.
 *
 * Conventions shared by every entry point
 *   - All tensor arguments are DEVICE pointers owned by the caller, contiguous
 *     row-major, 16-byte aligned.  bf16 tensors are IEEE bfloat16 bit patterns.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *     stream) and return right after the launch.  They never synchronise the
 *     host, never allocate (except bd_attn_decode with workspace == NULL, see
 *     there) and never free.
 *   - No exception or abort crosses the ABI: every error is a bd_status.
 *     Argument errors are detected on the host before anything is launched;
 *     nothing is written to any output in that case.
 *   - Grouped-query attention: q-head h reads kv-head h / (Hq / Hkv).
 *   - lse is ln( sum over visible keys of exp(scale * q.k) ).
 */
#ifndef BD_ATTN_H
#define BD_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st; /* cudaStream_t is `struct CUstream_st *` */

#if defined(__GNUC__)
#define BD_API __attribute__((visibility("default")))
#else
#define BD_API
#endif

typedef enum {
    BD_OK = 0,
    BD_ERR_INVALID_ARG = 1,     /* null/misaligned pointer, bad size or mode */
    BD_ERR_UNSUPPORTED = 2,     /* valid request this build does not handle */
    BD_ERR_CUDA = 3,            /* a CUDA runtime/driver call failed */
    BD_ERR_DEVICE_TIMEOUT = 4   /* a bounded device wait ran out, a
                                   device-side range check failed, or two
                                   launches shared a work counter pair */
} bd_status;

/*
 * Training / prefill block-diffusion attention.
 *
 * Defines: the three-part mask of "Nemotron-Labs-Diffusion-8B-Base 3x decoding
 * speed-up" (doido.pw), section 1 "Block Diffusion Attention" -- block
 * diagonal M_BD, offset block-causal M_OBC, block-causal M_BC -- read with the
 * BDLM objective of "LLaDA2.0-Uni" (discuss.pytorch.kr), section "Training
 * objective and loss function", eq. L_BDLM, which predicts x_{0,k} from
 * x_{0,<k} and x_{t,k} with K = L_total / L_B blocks.
 *
 * Each (batch, head) slice is a sequence of N = 2L rows: rows 0..L-1 are the
 * noisy tokens x_t, rows L..2L-1 the clean tokens x_0, each half cut into L/b
 * blocks of b rows.  A noisy row of block k sees the noisy rows of block k
 * (bidirectionally) and the clean rows of blocks < k; a clean row of block k
 * sees the clean rows of blocks <= k; no row sees a noisy row of another
 * block, and clean rows see no noisy row.
 *
 *   q    [B, Hq,  2L, d] bf16      (read)
 *   k, v [B, Hkv, 2L, d] bf16      (read)
 *   out  [B, Hq,  2L, d] bf16      (written: softmax(scale q k^T) v, rounded
 *                                   to nearest even)
 *   lse  [B, Hq,  2L]    fp32      (written)
 *   scale: softmax scale applied to q.k (typically 1/sqrt(d)); finite, > 0.
 *
 * Errors: BD_ERR_INVALID_ARG for a null or non-16-byte-aligned pointer, any
 * size <= 0, Hq % Hkv != 0, L % b != 0, or a non-finite/non-positive scale;
 * BD_ERR_UNSUPPORTED for d not in {32, 64, 128}; BD_ERR_CUDA if the launch
 * fails.
 *
 * Kernels: every head dim runs on the tcgen05 / TMA kernels (d = 64 and 32
 * on tiles read zero-extended to 128 columns).
 *
 * Concurrency: the launch is one persistent CTA per SM that takes
 * its work items from one of 64 counter pairs in device memory, chosen
 * round-robin when the call is made (and so fixed inside a captured CUDA
 * graph) and reset by the launch's last CTA.  Launches sharing a pair must
 * not overlap in time: keep fewer than 64 calls in flight per device, and do
 * not run two replays of one captured graph at the same time.  Each CTA
 * counts itself into the pair before its first fetch; a count beyond the
 * launch's own CTAs means such an overlap, and the device status word then
 * records BD_ERR_DEVICE_TIMEOUT (the outputs of the overlapping launches are
 * unreliable).
 */
BD_API bd_status bd_attn_fwd(const void *q, const void *k, const void *v, void *out,
                      float *lse, int B, int Hq, int Hkv, int L, int b, int d,
                      float scale, struct CUstream_st *stream);

/*
 * Backward of the training / prefill block-diffusion attention.
 *
 * Defines: the gradient that the BDLM training objective of "LLaDA2.0-Uni"
 * (discuss.pytorch.kr), section "Training objective and loss function", eq.
 * L_BDLM, sends through the attention of bd_attn_fwd (same mask, same
 * layouts).  For every visible (query i, key j) pair of one head, with
 * P_ij = exp(scale q_i.k_j - lse_i) and D_i = dout_i . out_i:
 *     dv_j = sum_i P_ij dout_i,
 *     dS_ij = P_ij (dout_i . v_j - D_i),
 *     dq_i = scale sum_j dS_ij k_j,   dk_j = scale sum_i dS_ij q_i;
 * the q-heads of a GQA group add into their kv-head's dk and dv.  The lse
 * side output of the forward is treated as a constant (no gradient into it).
 *
 *   q, out, dout [B, Hq,  2L, d] bf16   (read; out and lse as written by
 *   lse          [B, Hq,  2L]    fp32    bd_attn_fwd for these q, k, v)
 *   k, v         [B, Hkv, 2L, d] bf16   (read)
 *   dq           [B, Hq,  2L, d] bf16   (written)
 *   dk, dv       [B, Hkv, 2L, d] bf16   (written)
 *   workspace    DEVICE scratch of bd_attn_bwd_workspace_bytes(B, Hq, L)
 *                bytes, 256-byte aligned (per-row D and lse * log2 e)
 *
 * Three kernels on `stream`: a per-row pass, a dK/dV pass over key tiles and
 * a dQ pass over query tiles; nothing is allocated and no atomics are used,
 * so results are deterministic.  Concurrency as for bd_attn_fwd (each pass
 * takes one of the 64 scheduling counter pairs).
 *
 * Errors: as bd_attn_fwd, plus BD_ERR_INVALID_ARG for a null or misaligned
 * workspace or one smaller than required; BD_ERR_UNSUPPORTED for d != 128.
 */
BD_API bd_status bd_attn_bwd(const void *q, const void *k, const void *v,
                             const void *out, const float *lse,
                             const void *dout, void *dq, void *dk, void *dv,
                             int B, int Hq, int Hkv, int L, int b, int d,
                             float scale, struct CUstream_st *stream,
                             void *workspace, size_t workspace_bytes);

/* Bytes of scratch bd_attn_bwd needs (0 on bad sizes).  Host only. */
BD_API size_t bd_attn_bwd_workspace_bytes(int B, int Hq, int L);

/*
 * Block-decode block-diffusion attention.
 *
 * Defines: a block of b noisy queries attends to the cached clean prefix and
 * to its own block, bidirectionally while denoising a draft and causally when
 * verifying it against the same cache: "Nemotron-Labs-Diffusion-8B-Base 3x
 * decoding speed-up", section 2 "Linear Speculative Decoding";
 * "Nemotron-Labs-Diffusion-VLM-8B", section "Multi-mode decoding";
 * "Nemotron-Labs-Diffusion-3B", section "What it is" (guess a run of tokens
 * and check them in the same cache memory).
 *
 * The caller has already written the block's own K/V into the caches at
 * positions cache_len[i] .. cache_len[i]+b-1; cache_len counts the clean
 * prefix only.  Block row j of sequence i sees cache positions
 * 0 .. cache_len[i]-1 and block positions cache_len[i]+j' for every j' < b
 * (intra_block_mode 0, bidirectional denoise) or every j' <= j
 * (intra_block_mode 1, causal verify).  intra_block_mode 2 is cross-attention
 * only: the b rows are the canvas of an encoder-decoder model and see the
 * encoder's cache positions 0 .. cache_len[i]-1 and nothing of themselves
 * ("DiffusionGemma" pipeline page of the diffusers docs, introduction and
 * pipeline class description: a bidirectional decoder cross-attends to the
 * KV cache a causal encoder wrote, to denoise a canvas of canvas_length
 * tokens); with cache_len[i] = 0 such rows see nothing and get out = 0,
 * lse = -inf.  Softmax scale is 1/sqrt(d).
 *
 *   q_blk            [B, Hq, b, d]        bf16 (read)
 *   k_cache, v_cache [B, Hkv, S_cap, d]   bf16 (read; rows beyond
 *                                               cache_len[i]+b never read)
 *   cache_len        [B] int32, DEVICE memory (read on the device only, so
 *                    the call never waits for the host and can be captured in
 *                    a CUDA graph)
 *   out              [B, Hq, b, d]        bf16 (written)
 *   lse              [B, Hq, b]           fp32 (written)
 *   S_cap            row capacity of the caches (>= b in modes 0 and 1)
 *   workspace        device scratch of at least
 *                    bd_attn_decode_workspace_bytes(B, Hq, Hkv, b, d, S_cap)
 *                    bytes (19.6 MB, the same for every size: the partial
 *                    results of at most two cut units per persistent CTA),
 *                    256-byte aligned; its contents on entry do not matter.
 *                    NULL makes the library use an internal buffer of the
 *                    current device, allocated by the first such call (so
 *                    that call must not be inside a stream capture) and
 *                    never freed, so graphs captured with it stay valid.
 *                    Every NULL-workspace call on a device shares that
 *                    buffer: calls whose kernels may overlap on the GPU (two
 *                    streams without ordering between them) race on it and
 *                    give wrong results -- order them, or
 *                    pass each stream its own workspace.
 *
 * Errors: BD_ERR_INVALID_ARG for a null or misaligned pointer, any size <= 0,
 * Hq % Hkv != 0, S_cap < b in modes 0 and 1, intra_block_mode not 0/1/2, or
 * a workspace smaller than required; BD_ERR_UNSUPPORTED for d not in {32,
 * 64, 128}, B Hkv > 65535 or B Hq b > 2^31 - 1; BD_ERR_CUDA if the launch (or
 * the internal workspace allocation) fails.  A cache_len[i] outside [0, S_cap - b] (modes 0 and 1) or [0, S_cap]
 * (mode 2) is caught on the device: that sequence's rows are written as NaN
 * with lse NaN, and the device status word (see bd_attn_get_device_status)
 * records BD_ERR_DEVICE_TIMEOUT.
 */
BD_API bd_status bd_attn_decode(const void *q_blk, const void *k_cache,
                         const void *v_cache, const int32_t *cache_len,
                         void *out, float *lse, int B, int Hq, int Hkv, int b,
                         int d, int intra_block_mode,
                         struct CUstream_st *stream, int S_cap,
                         void *workspace, size_t workspace_bytes);

/* Size of the fixed scratch array bd_attn_decode_noalloc works in. */
#define BD_ATTN_NOALLOC_SCRATCH_BYTES (32u << 20)

/*
 * Block decode that never allocates device memory (no counterpart on the
 * source pages; it exists for callers that cannot allocate).
 *
 * Some callers cannot call cudaMalloc at the point where they decode: a
 * serving loop whose device memory is owned entirely by another allocator
 * (a framework's caching allocator, a fixed memory budget), code running
 * inside a stream capture where allocation is not allowed, or real-time code
 * that forbids allocation after start-up.  This call computes exactly what
 * bd_attn_decode computes, with the same arguments, layouts and errors, but
 * takes no workspace: its scratch (bd_attn_decode_workspace_bytes, 19.6 MB
 * for every size) lives in a fixed array of BD_ATTN_NOALLOC_SCRATCH_BYTES
 * bytes compiled into the library's device code.  Every GPU on which the
 * library's kernels are loaded holds that array until the process exits.
 *
 * - The first call on a device looks up the array's device address (with
 *   that device current) and caches it; make that first call before any
 *   stream capture.
 * - The array holds the scratch of every size (checked when the library is
 *   built); a size whose scratch exceeded it would be rejected with
 *   BD_ERR_UNSUPPORTED before anything is launched.
 * - All calls share the one array and it keeps whatever the last call left
 *   there; nothing in it needs to start at zero.  Calls whose kernels overlap
 *   on the GPU (for example on two streams without ordering between them)
 *   race on the array and give wrong results: order them on one stream or
 *   with events.
 * - It calls no cudaMalloc, cudaFree or other allocating routine.
 */
BD_API bd_status bd_attn_decode_noalloc(const void *q_blk, const void *k_cache,
                                        const void *v_cache,
                                        const int32_t *cache_len, void *out,
                                        float *lse, int B, int Hq, int Hkv,
                                        int b, int d, int intra_block_mode,
                                        struct CUstream_st *stream, int S_cap);

/*
 * Speculative decoding: accepted prefix length.
 *
 * Defines: "Nemotron-Labs-Diffusion-8B-Base 3x decoding speed-up", section 2
 * "Linear Speculative Decoding": a block drafted with bidirectional attention
 * is validated with causal attention and its longest matching prefix is
 * accepted.
 *
 *   draft, target  [B, b] int32 tokens, DEVICE memory (read): the drafted
 *                  block and the verifier's token for each block position
 *   n_accept       [B] int32, DEVICE memory (written): the length of the
 *                  longest prefix j = 0 .. n-1 with draft[i][j] == target[i][j]
 *
 * Errors: BD_ERR_INVALID_ARG for a null or non-4-byte-aligned pointer or a
 * size <= 0; BD_ERR_CUDA if the launch fails.
 */
BD_API bd_status bd_spec_accept(const int32_t *draft, const int32_t *target,
                                int32_t *n_accept, int B, int b,
                                struct CUstream_st *stream);

/*
 * Append accepted rows to the KV cache and advance its length, on the device.
 *
 * Defines: the "update the KV cache" step of linear speculative decoding,
 * "Nemotron-Labs-Diffusion-8B-Base 3x decoding speed-up", section 2.
 *
 *   k_cache, v_cache  [B, Hkv, S_cap, d] bf16 (read and written in place)
 *   cache_len         [B] int32, DEVICE memory (read, then advanced by
 *                     n_new[i])
 *   k_new, v_new      [B, Hkv, b, d] bf16 (read): the block's K/V; rows
 *                     0 .. n_new[i]-1 are copied to cache positions
 *                     cache_len[i] .. cache_len[i]+n_new[i]-1.  Both NULL:
 *                     the rows are already there (the usual case: the block's
 *                     K/V were written at the cache tail before the causal
 *                     verification), so only the length advances.
 *   n_new             [B] int32, DEVICE memory (read), e.g. from
 *                     bd_spec_accept
 *
 * Nothing is allocated; the call can be captured in a CUDA graph.  A
 * sequence with n_new[i] outside [0, b] or cache_len[i] + n_new[i] > S_cap is
 * left untouched and the device status word records BD_ERR_DEVICE_TIMEOUT.
 * Errors: BD_ERR_INVALID_ARG for a null pointer (k_new and v_new must be both
 * NULL or both set), a misaligned pointer or a size <= 0;
 * BD_ERR_UNSUPPORTED for d not in {32, 64, 128}; BD_ERR_CUDA if the launch
 * fails.
 */
BD_API bd_status bd_cache_append(void *k_cache, void *v_cache, int32_t *cache_len,
                                 const void *k_new, const void *v_new,
                                 const int32_t *n_new, int B, int Hkv, int b,
                                 int d, int S_cap, struct CUstream_st *stream);

/*
 * Crop the KV cache to at most max_len positions: cache_len[i] =
 * min(cache_len[i], max_len), on the device (the cache rows stay where they
 * are).  Defines: "Nemotron-Labs-Diffusion-8B-Base 3x decoding speed-up",
 * section "KV cache strategy" (the cache is cropped to a maximum length
 * during generation).  cache_len: [B] int32 in DEVICE memory.
 * Errors: BD_ERR_INVALID_ARG for a null or misaligned pointer, B <= 0 or
 * max_len < 0; BD_ERR_CUDA if the launch fails.
 */
BD_API bd_status bd_cache_crop(int32_t *cache_len, int B, int max_len,
                               struct CUstream_st *stream);

/*
 * Sparse prefix retention (SPRINT): prune the cached prefix once at the start
 * of a block.
 *
 * Defines: "LLaDA2.0-Uni" (discuss.pytorch.kr), section "SPRINT: training-free
 * inference acceleration", paragraph "Sparse Prefix Retention".  Each prefix
 * position p < cache_len[i] gets the score
 *     s_p = alpha * I_p + (1 - alpha) * conf[i][p],
 *     I_p = |k_p|_2 / mean over the prefix of |k_j|_2,
 * where |k_p|_2 is the norm of position p's key over all kv-heads and dims
 * of this cache (0 for all p if that mean is 0), and conf is the caller's
 * top-1 softmax confidence.  Each modality (modality[i][p] == 0: text, else
 * image) with n prefix positions keeps floor(r * n + 1/2) of them, r =
 * keep_text or keep_image: those with the highest score, ties to the lower
 * position.  The page uses alpha = 0.5, keep_image = 0.8, keep_text = 1.0.
 * The kept positions, in their original order, become the new prefix.
 * Scores are computed in double precision.
 *
 *   k_cache, v_cache  [B, Hkv, S_cap, d] bf16 (read)
 *   cache_len         [B] int32, DEVICE (read)
 *   conf              [B, S_cap] fp32, DEVICE (read; entries < cache_len[i])
 *   modality          [B, S_cap] uint8, DEVICE (read; entries < cache_len[i])
 *   k_out, v_out      [B, Hkv, S_cap, d] bf16 (written: rows 0 ..
 *                     new_len[i]-1 are the kept rows; later rows untouched).
 *                     Must not overlap the input caches.
 *   kept              [B, S_cap] int32, DEVICE (written: kept positions in
 *                     increasing order, then -1)
 *   new_len           [B] int32, DEVICE (written; the prefix length to pass to
 *                     bd_attn_decode as cache_len afterwards)
 *   score             [B, S_cap] fp64, DEVICE (written for p < cache_len[i])
 *                     or NULL
 *   workspace         DEVICE scratch of bd_sprint_workspace_bytes(B, S_cap)
 *                     bytes, 256-byte aligned
 *
 * Errors: BD_ERR_INVALID_ARG for a null (other than score) or misaligned
 * pointer, a size <= 0, alpha or a keep ratio outside [0, 1], aliasing
 * outputs, or a short workspace; BD_ERR_UNSUPPORTED for d not in {32, 64,
 * 128} or S_cap > 65536; BD_ERR_CUDA if a launch fails.  A cache_len[i]
 * outside [0, S_cap] gives new_len[i] = 0 and records BD_ERR_DEVICE_TIMEOUT
 * in the device status word.
 */
BD_API bd_status bd_sprint_prune(const void *k_cache, const void *v_cache,
                                 const int32_t *cache_len, const float *conf,
                                 const uint8_t *modality, float alpha,
                                 float keep_text, float keep_image,
                                 void *k_out, void *v_out, int32_t *kept,
                                 int32_t *new_len, double *score, int B,
                                 int Hkv, int d, int S_cap,
                                 struct CUstream_st *stream, void *workspace,
                                 size_t workspace_bytes);

/* Bytes of scratch bd_sprint_prune needs (0 on bad sizes).  Host only. */
BD_API size_t bd_sprint_workspace_bytes(int B, int S_cap);

/*
 * The serving step over a KV cache in 8 bits.
 *
 * The pages decode over a cache in the model's own type; the calls below have
 * no counterpart on them.  They are the operators that a step of block
 * decoding (bd_attn_decode) is made of when the cache is held in 8 bits:
 * rotary positions, quantising rows as they are written, attention over the
 * codes, verification by sampling.  bd_cache_crop works on such a cache as it
 * is; for bd_sprint_prune read the prefix back, prune it and append the kept
 * rows to an emptied cache.
 *
 * The cache in 8 bits
 *   k_cache, v_cache  [B, Hkv, S_cap, d] e4m3 codes (1 sign, 4 exponent, 3
 *                     mantissa bits, no infinity, largest value 448)
 *   k_scale, v_scale  [B, Hkv, ceil(S_cap / group)] fp32: one scale for every
 *                     `group` consecutive positions of a kv-head; a position's
 *                     values are its codes times its group's scale
 *                     (an infinity where fp32 does not hold the product)
 *   group             16, 32, 64 or 128
 * bd_cache_append_q8 writes powers of two between 2^-64 and 2^120 as scales.
 * The reading calls take any scale from 2^-100 to 2^120 in the groups that
 * hold visible positions (bd_attn_decode_q8 works with both the scale and its
 * inverse); codes and scales behind them are never used, whatever they hold.
 */

/* Scalings of bd_rope_table. */
#define BD_ROPE_PLAIN 0
#define BD_ROPE_LINEAR 1
#define BD_ROPE_NTK 2
#define BD_ROPE_YARN 3

/*
 * Frequencies of rotary positions (host arithmetic; needs no GPU).
 *
 * f_i = base^(-2 i / rot_dim) radians a position for pair i, and for contexts
 * `factor` times longer than the trained one:
 *   BD_ROPE_LINEAR  f_i / factor (position interpolation);
 *   BD_ROPE_NTK     base * factor^(rot_dim / (rot_dim - 2)) for base;
 *   BD_ROPE_YARN    f_i / factor (1 - w) + f_i w with w = (turns - beta_slow) /
 *                   (beta_fast - beta_slow) clamped to [0, 1], turns =
 *                   trained_len f_i / 2 pi (the "NTK-by-parts" rule of Peng et
 *                   al., "YaRN", section 3.2), and mscale = 0.1 ln(factor) + 1.
 *                   The ramp w is linear in the turns, as in the paper.  Models
 *                   trained with a ramp linear in the pair's index i, between two
 *                   bounds, need a table of their own: bd_rope takes any inv_freq.
 *
 *   inv_freq  [rot_dim / 2] fp64, HOST memory (written)
 *   mscale    HOST memory (written): 1 but for BD_ROPE_YARN
 *
 * Errors: BD_ERR_INVALID_ARG for a null pointer, rot_dim <= 0 or odd (<= 2
 * with BD_ROPE_NTK), base not above 1 and finite, an unknown scaling, factor
 * not in [1, inf) where it is used, and for BD_ROPE_YARN trained_len <= 0 or
 * not 0 <= beta_slow < beta_fast < inf.
 */
BD_API bd_status bd_rope_table(double *inv_freq, float *mscale, int rot_dim,
                               double base, int scaling, double factor,
                               int trained_len, double beta_fast, double beta_slow);

/*
 * Rotary positions of queries and keys, or the gradient through them.
 *
 * Row r of sequence i has the position positions[i][r], or start[i] + r mod
 * period (start NULL: 0).  The training form's [x_t ; x_0] has N = 2L and
 * period = L: a noisy token stands where its clean one does.  A decoded block
 * has N = period = b and start = cache_len.  With t = position * inv_freq[j],
 * the pair (x_a, x_b) of every head becomes
 *     (mscale (x_a cos t - x_b sin t), mscale (x_b cos t + x_a sin t)),
 * (a, b) = (j, j + rot_dim/2), or (2j, 2j + 1) if interleaved; dims from
 * rot_dim on are copied.  adjoint = 1 takes -t: it maps the gradients of
 * q_out and k_out to those of q and k (with mscale 1 it is the inverse).
 * Angles are reduced in fp64, so positions may be as large as int32 holds.
 *
 *   q, q_out   [B, Hq,  N, d] bf16   (read, written)
 *   k, k_out   [B, Hkv, N, d] bf16   (both NULL with Hkv = 0: queries alone)
 *              q_out may be q, and k_out may be k; no other overlap
 *   inv_freq   [rot_dim / 2] fp64, DEVICE
 *   start      [B] int32, DEVICE, or NULL
 *   positions  [B, N] int32, DEVICE, or NULL; not together with start
 *
 * Errors: BD_ERR_INVALID_ARG for a null (other than the above) or misaligned
 * pointer, a size or period <= 0, rot_dim > d, a non-finite mscale, flags not
 * 0/1, or aliased outputs; BD_ERR_UNSUPPORTED for d not in {32, 64, 128} or
 * rot_dim not a multiple of 16; BD_ERR_CUDA if the launch fails.
 */
BD_API bd_status bd_rope(const void *q, const void *k, void *q_out, void *k_out,
                         const double *inv_freq, const int32_t *start,
                         const int32_t *positions, int B, int Hq, int Hkv,
                         int N, int d, int rot_dim, int period,
                         int interleaved, float mscale, int adjoint,
                         struct CUstream_st *stream);

/*
 * Quantise rows into the cache in 8 bits at its tail.
 *
 * Rows 0 .. n_new[i]-1 of k_new, v_new go to positions cache_len[i] ..
 * cache_len[i]+n_new[i]-1.  Every group that takes a row gets the scale s =
 * 2^max(-64, k), k the smallest with |x| <= 448 * 2^k over the finite values
 * of the rows that it then holds (the new ones, and those below cache_len[i]),
 * and all of those rows the codes rne(x / s): +-inf becomes +-448, NaN stays
 * NaN.  At the largest scale, 2^120, codes are at most +-240: 256 2^120 would be
 * an infinity in fp32 and bf16.
 * Rows that stay are requantised from the values that they have.  Where the old
 * scale is one that this call wrote, that is exact for values of 2^-6 s and more
 * (and for 0); smaller ones are rounded to a multiple of 2^-9 s.  What is lost
 * stays lost: a large row costs the rows before it in its group precision for
 * good, also as a draft that the next write replaces.  Positions from
 * cache_len[i]+n_new[i] on keep their codes, and groups that take no row keep
 * their scales; positions behind the rows in a written group lose their value.
 *
 *   cache_len      [B] int32, DEVICE (read; advanced by n_new[i] if advance)
 *   k_new, v_new   [B, Hkv, b, d] bf16 (read).  Both NULL, with advance = 1:
 *                  the rows are already there, only the length advances.
 *   n_new          [B] int32, DEVICE (read), or NULL: b rows each
 *   advance        0: the rows are a draft behind the prefix, to be attended
 *                  to (modes 0 and 1 of bd_attn_decode_q8) and overwritten;
 *                  1: they join the prefix
 *
 * One kernel, and one more to advance.  Nothing is allocated; the call can be
 * captured in a CUDA graph.  A sequence with n_new[i] outside [0, b], a
 * negative length or cache_len[i] + n_new[i] > S_cap is left untouched and the
 * device status word records BD_ERR_DEVICE_TIMEOUT.
 * Errors: BD_ERR_INVALID_ARG for a null or misaligned pointer (16 bytes for
 * codes and rows, 4 for the rest), codes or scales of K and V in one buffer, a
 * size <= 0, only one of k_new and v_new, or nothing to do;
 * BD_ERR_UNSUPPORTED for d not in {32, 64, 128}, another group, B > 65535,
 * Hkv > 32767 or S_cap or b > 2^30; BD_ERR_CUDA if a launch fails.
 */
BD_API bd_status bd_cache_append_q8(void *k_cache, void *v_cache, float *k_scale,
                                    float *v_scale, int32_t *cache_len,
                                    const void *k_new, const void *v_new,
                                    const int32_t *n_new, int B, int Hkv, int b,
                                    int d, int S_cap, int group, int advance,
                                    struct CUstream_st *stream);

/*
 * Read the cache in 8 bits back: rows 0 .. cache_len[i]-1 of k_out, v_out
 * [B, Hkv, S_cap, d] bf16 become codes times scale, rounded to nearest even
 * (exact for the scales that bd_cache_append_q8 writes); later rows are left
 * as they are.  A cache_len[i] outside [0, S_cap] leaves that sequence's rows
 * and records BD_ERR_DEVICE_TIMEOUT in the device status word.
 * Errors: as bd_cache_append_q8, plus BD_ERR_INVALID_ARG for aliased outputs.
 */
BD_API bd_status bd_cache_read_q8(const void *k_cache, const void *v_cache,
                                  const float *k_scale, const float *v_scale,
                                  const int32_t *cache_len, void *k_out,
                                  void *v_out, int B, int Hkv, int d, int S_cap,
                                  int group, struct CUstream_st *stream);

/*
 * Block decode over the cache in 8 bits: what bd_attn_decode computes, with
 * the keys and values codes times scale.  Same masks and modes, same q_blk,
 * out, lse, cache_len and workspace; the block's own rows are in the cache at
 * cache_len[i] .. cache_len[i]+b-1 in modes 0 and 1 (bd_cache_append_q8 with
 * advance = 0).  Codes of positions that no row of the block sees are not
 * used, NaN codes among them; in mode 1 a NaN value in one of the block's own
 * V rows reaches every row of the block.  A query row with an infinity or a
 * NaN gives NaN.  Queries may be as small as bf16's smallest normal value; the
 * largest |q| |k| / sqrt(d) of a row has to fit fp32.
 *
 * What is held in fewer than 32 bits on the way: a query value below 2^-10 of
 * its row's largest is off by at most 2^-17 of that (none is where a kv-head's
 * rows are few); the weights p that multiply V by 2^-11 of themselves, or, where
 * p s (s: V's scale) is below 2^-17 of the row's largest such product, by 2^-28
 * of that product, over s.  So out is off by at most 2^-11 sum p |v|, n 2^-28
 * 448 max p s over n visible keys, and its rounding to bf16: for a million keys
 * the second is 2^-8 of 448 max p s.  Sums and lse are fp32.
 *
 * Errors: as bd_attn_decode and, for the cache, bd_cache_append_q8.
 */
BD_API bd_status bd_attn_decode_q8(const void *q_blk, const void *k_cache,
                                   const void *v_cache, const float *k_scale,
                                   const float *v_scale, const int32_t *cache_len,
                                   void *out, float *lse, int B, int Hq, int Hkv,
                                   int b, int d, int intra_block_mode,
                                   struct CUstream_st *stream, int S_cap,
                                   int group, void *workspace,
                                   size_t workspace_bytes);

/*
 * Verify drafted tokens against the target's probabilities, with the random
 * numbers given: speculative sampling, where bd_spec_accept compares tokens.
 *
 * Position j of sequence i is accepted while u q(x) < p(x): x = draft[i][j],
 * q and p its probabilities in rows j of draft_prob[i] and target_prob[i], u =
 * u_accept[i][j]; decided exactly (the product in fp64).  n_accept[i] = n, the
 * number of positions before the first refusal.  next_token[i] is drawn from
 * the weights max(p_n - q_n, 0) of row n, or from p_n if they are all 0, or if
 * every position was accepted (n = n_draft[i]): the lowest t whose running sum
 * w_0 + .. + w_t exceeds u_sample[i] times the sum of all (sums in fp64; the
 * last t with a weight if rounding leaves none).  A weight that is NaN counts
 * as 0; without any mass next_token[i] is -1.
 *
 *   draft        [B, b] int32, DEVICE
 *   draft_prob   [B, b, V] fp32, DEVICE, or NULL: the draft was not sampled,
 *                q is 1 at the drafted token and 0 elsewhere
 *   target_prob  [B, b + 1, V] fp32, DEVICE
 *   u_accept     [B, b] fp32, u_sample [B] fp32, DEVICE, in [0, 1)
 *   n_draft      [B] int32, DEVICE, drafted positions, or NULL: b each
 *   n_accept, next_token  [B] int32, DEVICE (written); one of them may be
 *                n_draft, the counts replaced in place.  No other overlap with
 *                one another or an input
 *
 * A sequence with n_draft[i] outside [0, b] or a drafted token outside [0, V)
 * gets n_accept 0 and next_token -1, and the device status word records
 * BD_ERR_DEVICE_TIMEOUT.  Errors: BD_ERR_INVALID_ARG for a null or misaligned
 * pointer, a size <= 0 or outputs that overlap one another or an input but
 * as above; BD_ERR_UNSUPPORTED for V > 4194304 or B > 268435455; BD_ERR_CUDA
 * if the launch fails.
 */
BD_API bd_status bd_spec_verify(const int32_t *draft, const float *draft_prob,
                                const float *target_prob, const float *u_accept,
                                const float *u_sample, const int32_t *n_draft,
                                int32_t *n_accept, int32_t *next_token, int B,
                                int b, int V, struct CUstream_st *stream);

/* Bytes of scratch bd_attn_decode needs for these sizes (0 on bad sizes).
 * Pure host arithmetic; needs no GPU. */
BD_API size_t bd_attn_decode_workspace_bytes(int B, int Hq, int Hkv, int b, int d,
                                      int S_cap);

/* Synchronises `stream`, then returns and clears the device status word of
 * the current device: BD_OK, or BD_ERR_DEVICE_TIMEOUT if a kernel gave up a
 * bounded wait, rejected a device-resident size, or found its work counter
 * pair in use by another launch since the last call;
 * BD_ERR_CUDA if the synchronisation itself failed. */
BD_API bd_status bd_attn_get_device_status(struct CUstream_st *stream);

/* Static, NUL-terminated description of a status code. */
BD_API const char *bd_attn_status_string(bd_status status);

#ifdef __cplusplus
}
#endif

#endif /* BD_ATTN_H */
