/*
 * gdn.h -- C ABI of the Gated DeltaNet (GDN) prompt-prefill library for one
 * NVIDIA GB300 GPU (sm_103a).
 *
 * The path has three stages, after the three kernels the pages benchmark
 * ("Round 30 Track C Audit: gdn_pre, gdn_post, and gdn_scanr_4", sections 1
 * and 2: gdn_pre, the gdn_scan_r recurrence and gdn_post, timed separately
 * and as one pre+scan+post total over 36 layers):
 *
 *   gdn_pre   width-4 causal depthwise conv over the packed q|k|v channels
 *             with a carried 3-token history, SiLU, L2 normalisation of every
 *             q and k head (eps), and the per-(token, value head) gates
 *             lam = log g = -exp(A_log) * softplus(a + dt_bias),
 *             beta = sigmoid(b).
 *   gdn_scan  the gated delta rule, per value head h with key head
 *             h / (hv/hk) and fp32 state S in R^{dk x dv}:
 *               S <- g S;  u = beta (v - S^T k);  S <- S + k u^T;
 *               o = S^T q / sqrt(dk).
 *   gdn_post  y = o / sqrt(mean(o^2) + eps) * gamma * SiLU(z), fp16 or fp32.
 *   gdn_layer the three stages back to back on one stream.
 *   gdn_step  one decode step (a single token per sequence) through all three.
 *
 * Conventions shared by every entry point
 * ----------------------------------------
 *  - Every array pointer is a DEVICE pointer (memory of the current CUDA
 *    device), owned by the caller, dense and row-major in the layout stated.
 *    The library allocates no device memory and keeps no pointer after the
 *    call returns; the work runs asynchronously on `stream` (NULL = legacy
 *    default stream), so buffers must stay valid until the stream reaches it.
 *  - fp16 arrays are IEEE binary16 bit patterns (uint16_t).
 *  - Shapes: hk key heads, hv value heads (hv a multiple of hk), dk = dv =
 *    128, C = 2*hk*dk + hv*dv packed channels ordered q (hk heads) | k (hk
 *    heads) | v (hv heads).  T = total tokens of a packed variable-length
 *    batch of n_seq sequences; sequence s owns tokens
 *    [cu_seqlens[s], cu_seqlens[s+1]).  cu_seqlens is a DEVICE int32 array of
 *    n_seq+1 entries, non-decreasing, cu_seqlens[0] = 0,
 *    cu_seqlens[n_seq] = T (not read on the host; a violation is undefined).
 *    Zero-length sequences are allowed: their history and state pass
 *    through unchanged.
 *  - Every pointer must be 16-byte aligned.
 *  - Errors: argument problems are detected on the host before anything is
 *    launched and return a status with nothing enqueued.  A failed launch
 *    returns GDN_ERR_CUDA (the CUDA error string is kept for
 *    gdn_last_error_string).  Asynchronous faults surface at the caller's
 *    next synchronisation, as with any CUDA library, and, without one, through
 *    gdn_last_async_error once any CUDA call of the process has observed them.
 *  - Thread safety: calls may be made from several host threads on
 *    different streams; they share no mutable state except the last-error
 *    string, which is per host thread.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st; /* cudaStream_t is `struct CUstream_st *` */

#if defined(__GNUC__)
#define GDN_API __attribute__((visibility("default")))
#else
#define GDN_API
#endif

typedef enum gdn_status {
    GDN_OK = 0,
    GDN_ERR_INVALID_ARG = 1, /* null pointer, negative size, overlap, bad value */
    GDN_ERR_UNSUPPORTED = 2, /* shape outside what the kernels implement       */
    GDN_ERR_ALIGNMENT = 3,   /* a pointer is not 16-byte aligned               */
    GDN_ERR_WORKSPACE = 4,   /* workspace missing or smaller than required     */
    GDN_ERR_CUDA = 5,        /* a CUDA runtime call or launch failed            */
    GDN_ERR_TIMEOUT = 6      /* a bounded wait inside a kernel expired: that
                                call's outputs are invalid (gdn_*_check)        */
} gdn_status;

/* Model shape.  Implemented: dk == dv == 128, 1 <= hk, hv % hk == 0,
 * hv <= 4096, eps > 0 (the pages' layer: hk=16, hv=48, eps=1e-6 -- "round 10
 * track b: gdn vectorization and scan", source and execution). */
typedef struct gdn_dims {
    int32_t hk;  /* key (and query) heads                              */
    int32_t hv;  /* value heads                                        */
    int32_t dk;  /* key head dimension (128)                           */
    int32_t dv;  /* value head dimension (128)                         */
    float eps;   /* epsilon of the L2 norms and of the RMSNorm         */
} gdn_dims;

/* Human-readable name of a status code (static storage). */
GDN_API const char* gdn_status_string(gdn_status s);

/* Detail of the last non-OK status returned on this host thread. */
GDN_API const char* gdn_last_error_string(void);

/*
 * gdn_last_async_error -- the sticky CUDA error: GDN_ERR_CUDA once the library
 * has seen an error that leaves the CUDA context unusable (a kernel that
 * faulted: illegal address or instruction, misaligned address, launch
 * failure or timeout, device assert, uncorrectable ECC), else GDN_OK.  The
 * error is seen either by one of the library's own calls (every later launch
 * or copy in a faulted context returns it) or, at this call, through the
 * CUDA runtime's last-error state.  Does not synchronise, enqueues nothing and
 * clears nothing: once set it stays set for the life of the process, as the
 * context's fault does.  The detail goes to gdn_last_error_string.
 */
GDN_API gdn_status gdn_last_async_error(void);

/*
 * gdn_pre -- stage 1 ("Round 30 Track C Audit", section 1, gdn_pre: the
 * 4-tap conv loop, the history write at the last token, the per-key-head
 * q/k sum-of-squares reductions; "round 10 track b", variants: each conv
 * output is four multiply-adds in tap order, history kept channel by
 * channel).
 *
 * In:  qkv      fp16 [T][C]             raw projections, q | k | v
 *      conv_w   fp32 [C][4]             taps; tap 3 multiplies the current
 *                                       token, tap 0 the token 3 back
 *      hist_in  fp16 [n_seq][C][3]      the 3 inputs before each sequence,
 *                                       oldest first
 *      a, b     fp16 [T][hv]            gate pre-activations
 *      A_log, dt_bias fp32 [hv]
 * Out: hist_out fp16 [n_seq][C][3]      last 3 inputs of each sequence
 *                                       (old history shifted in when the
 *                                       sequence is shorter than 3); bit
 *                                       copies, never rounded.  May be the
 *                                       same buffer as hist_in: the new
 *                                       history is then written by a second
 *                                       launch, after every read of the old
 *                                       one.  Any other overlap is rejected.
 *      qn, kn   fp32 [T][hk][dk]        SiLU(conv) / sqrt(|.|^2 + eps)
 *      vc       fp32 [T][hv][dv]        SiLU(conv) of the v channels
 *      glog     fp32 [T][hv]            lam = log g (<= 0)
 *      beta     fp32 [T][hv]            sigmoid(b)
 */
GDN_API gdn_status gdn_pre(const gdn_dims* dims, int32_t n_seq, int32_t total_tokens,
                   const int32_t* cu_seqlens, const uint16_t* qkv, const float* conv_w,
                   const uint16_t* hist_in, uint16_t* hist_out, const uint16_t* a,
                   const uint16_t* b, const float* A_log, const float* dt_bias, float* qn,
                   float* kn, float* vc, float* glog, float* beta, struct CUstream_st* stream);

/* Workspace bytes gdn_scan needs for this batch shape (0 is a valid answer). */
GDN_API size_t gdn_scan_workspace_bytes(const gdn_dims* dims, int32_t n_seq, int32_t total_tokens);

/*
 * gdn_scan -- stage 2, the gated delta-rule recurrence ("Round 30 Track C
 * Audit", section 1: gdn_scan_r keeps the fp32 state on chip, decays and
 * updates it per token and forms the k and q products against it).
 * Computed chunk-wise (64 tokens), exact in exact arithmetic.
 *
 * In:  qn, kn   fp32 [T][hk][dk]        unit-norm q and k (as gdn_pre writes)
 *      vc       fp32 [T][hv][dv]
 *      glog     fp32 [T][hv]            log-decay, <= 0 (-inf allowed: g = 0)
 *      beta     fp32 [T][hv]
 *      S_in     fp32 [n_seq][hv][dk][dv]  state before each sequence
 * Out: S_out    fp32 [n_seq][hv][dk][dv]  state after each sequence; may be
 *                                       the same buffer as S_in
 *      o        fp32 [T][hv][dv]        S^T q / sqrt(dk) after each token
 * workspace: device scratch of at least gdn_scan_workspace_bytes() bytes
 *            (may be NULL when that is 0); contents on entry are ignored.
 * Stream capture: a call may be captured into a CUDA graph.  Nothing it
 * enqueues depends on host state that changes from call to call, so each
 * replay of the graph is a complete scan of what the captured buffers then
 * hold.  Calls sharing one workspace must not overlap on the GPU.
 */
GDN_API gdn_status gdn_scan(const gdn_dims* dims, int32_t n_seq, int32_t total_tokens,
                    const int32_t* cu_seqlens, const float* qn, const float* kn,
                    const float* vc, const float* glog, const float* beta, const float* S_in,
                    float* S_out, float* o, void* workspace, size_t workspace_bytes,
                    struct CUstream_st* stream);

/*
 * gdn_post -- stage 3, gated RMSNorm ("Round 30 Track C Audit", section 1,
 * gdn_post: per-head sum-of-squares reduction and the f32 output switch;
 * "opus_r25_gdn -- round 25 track A", shipped: the sigmoid gate and gamma).
 *
 * In:  o        fp32 [T][hv][dv]
 *      z        fp16 [T][hv][dv]
 *      gamma    fp32 [dv]               shared by all heads
 * Out: y        fp16 [T][hv][dv] when out_f32 == 0, else fp32 [T][hv][dv]
 */
GDN_API gdn_status gdn_post(const gdn_dims* dims, int32_t total_tokens, const float* o,
                    const uint16_t* z, const float* gamma, int32_t out_f32, void* y,
                    struct CUstream_st* stream);

/*
 * gdn_scan_noalloc -- gdn_scan for callers that cannot allocate device
 * memory.  The paper has no counterpart to this entry point.
 *
 * Some callers have no device allocator to hand to the library: a host
 * program that links this C ABI directly and has no workspace buffer to
 * give, or a service that forbids device allocations after start-up.  For
 * them this entry point runs the same scan with its scratch in a
 * fixed-size array that the library owns (GDN_SCAN_NOALLOC_MAX_BYTES, held
 * on every device that loads the library until the process exits).  The
 * caller still passes every input and output, exactly as for gdn_scan.
 *
 * - Allocates nothing: no cudaMalloc, cudaFree or allocating library call.
 * - The first call on each device looks up that device's copy of the array
 *   (with the device current) and caches it; make that first call before
 *   any stream capture.
 * - Batches whose scan scratch (gdn_scan_workspace_bytes) exceeds
 *   GDN_SCAN_NOALLOC_MAX_BYTES are rejected with GDN_ERR_UNSUPPORTED and a
 *   message naming the limit; nothing is enqueued.
 * - All calls on a device share the one array and it keeps the last call's
 *   contents (the part that must start at zero is cleared by every call):
 *   calls whose work overlaps on the GPU -- different streams, or several
 *   host threads -- race on it.  Serialise them, e.g. on one stream.
 * - The array's device address is looked up again on every call made outside
 *   stream capture (so a device reset, after which the library's module is
 *   loaded afresh, is picked up); under capture the address from the last
 *   call outside capture is used.
 */
#define GDN_SCAN_NOALLOC_MAX_BYTES ((size_t)64 << 20)
GDN_API gdn_status gdn_scan_noalloc(const gdn_dims* dims, int32_t n_seq, int32_t total_tokens,
                                    const int32_t* cu_seqlens, const float* qn, const float* kn,
                                    const float* vc, const float* glog, const float* beta,
                                    const float* S_in, float* S_out, float* o,
                                    struct CUstream_st* stream);

/*
 * gdn_scan_noalloc_check -- the failure report of the last gdn_scan_noalloc on
 * the current device (as gdn_scan_check for an ordinary workspace: its
 * record is the first word of the library's own scratch array, whose address
 * the caller never holds).  Enqueues a 4-byte device-to-host copy on `stream`,
 * SYNCHRONISES it and returns GDN_OK or GDN_ERR_TIMEOUT; GDN_ERR_INVALID_ARG
 * if gdn_scan_noalloc has not run on this device yet.
 */
GDN_API gdn_status gdn_scan_noalloc_check(struct CUstream_st* stream);

/* Workspace bytes gdn_layer needs: the stage tensors vc, glog, beta, o plus
 * the scan's own workspace, each 256-byte aligned (q and k go from the pre
 * stage straight into the scan's operand images there: no qn / kn). */
GDN_API size_t gdn_layer_workspace_bytes(const gdn_dims* dims, int32_t n_seq, int32_t total_tokens);

/*
 * gdn_layer -- the whole prefill layer: gdn_pre, gdn_scan and gdn_post on
 * `stream`, the stage tensors kept in `workspace` (the pages time the three
 * stages back to back as one pre+scan+post total, "Round 30 Track C Audit",
 * section 2).  Arguments as in the three stage calls.  S_out may equal S_in
 * and hist_out may equal hist_in (partial overlaps are rejected).  May be
 * captured into a CUDA graph, as gdn_scan.
 */
GDN_API gdn_status gdn_layer(const gdn_dims* dims, int32_t n_seq, int32_t total_tokens,
                     const int32_t* cu_seqlens, const uint16_t* qkv, const float* conv_w,
                     const uint16_t* hist_in, uint16_t* hist_out, const uint16_t* a,
                     const uint16_t* b, const uint16_t* z, const float* A_log,
                     const float* dt_bias, const float* gamma, const float* S_in, float* S_out,
                     int32_t out_f32, void* y, void* workspace, size_t workspace_bytes,
                     struct CUstream_st* stream);

/*
 * gdn_scan_fast / gdn_layer_fast -- the same computations with every
 * tensor-core product of the scan taken in one pass on bf16 operands (fp32
 * accumulation, fp32 state) instead of the split hi/lo passes: a third of
 * the MMA instructions, traded for accuracy.  Arguments, workspaces, layouts
 * and errors exactly as gdn_scan / gdn_layer.  The error against the fp64
 * reference is bounded by bf16 rounding of K, Q, the state and the chunk
 * intermediates rather than by the 1e-4 of the split path; the tests state the
 * bound they check.
 */
GDN_API gdn_status gdn_scan_fast(const gdn_dims* dims, int32_t n_seq, int32_t total_tokens,
                                 const int32_t* cu_seqlens, const float* qn, const float* kn,
                                 const float* vc, const float* glog, const float* beta,
                                 const float* S_in, float* S_out, float* o, void* workspace,
                                 size_t workspace_bytes, struct CUstream_st* stream);
GDN_API gdn_status gdn_layer_fast(const gdn_dims* dims, int32_t n_seq, int32_t total_tokens,
                                  const int32_t* cu_seqlens, const uint16_t* qkv, const float* conv_w,
                                  const uint16_t* hist_in, uint16_t* hist_out, const uint16_t* a,
                                  const uint16_t* b, const uint16_t* z, const float* A_log,
                                  const float* dt_bias, const float* gamma, const float* S_in,
                                  float* S_out, int32_t out_f32, void* y, void* workspace,
                                  size_t workspace_bytes, struct CUstream_st* stream);

/*
 * Failure reports of the scan.  Every wait inside the scan kernels is
 * bounded (about two seconds); one that expires makes its CTA record an
 * error in the scan workspace, release what it holds and stop, so the CUDA
 * context stays usable but the call's outputs are invalid.  These functions
 * read that record for the last gdn_scan (or gdn_layer) that used the
 * workspace: they enqueue a 4-byte device-to-host copy on `stream`,
 * SYNCHRONISE the stream and return GDN_OK or GDN_ERR_TIMEOUT (GDN_ERR_CUDA if
 * the copy fails).  gdn_layer_check takes the layer's shape to find the scan
 * part of the layer workspace.
 */
GDN_API gdn_status gdn_scan_check(const void* workspace, struct CUstream_st* stream);
GDN_API gdn_status gdn_layer_check(const gdn_dims* dims, int32_t n_seq, int32_t total_tokens,
                                   const void* workspace, struct CUstream_st* stream);

/*
 * gdn_step -- one decode step: a single new token for each of n_seq
 * sequences through the whole layer (pre, the recurrence for that token, and
 * post), fused into one launch.  Per token it computes exactly what gdn_layer
 * computes for a batch in which every sequence holds one token: the
 * token-sequential recurrence of "Round 30 Track C Audit: gdn_pre, gdn_post,
 * and gdn_scanr_4", section 1 (gdn_scan_r's per-token decay, delta update and
 * k/q products against the fp32 state), with that section's pre and post
 * arithmetic for the token.
 *
 * In:  qkv      fp16 [n_seq][C]         the token's raw projections, q | k | v
 *      conv_w   fp32 [C][4]             as for gdn_pre
 *      hist_in  fp16 [n_seq][C][3]      the 3 inputs before the token, oldest first
 *      a, b     fp16 [n_seq][hv]        gate pre-activations
 *      z        fp16 [n_seq][hv][dv]    output gate
 *      A_log, dt_bias fp32 [hv];  gamma fp32 [dv]
 *      S_in     fp32 [n_seq][hv][dk][dv]  state before the token
 * Out: hist_out fp16 [n_seq][C][3]      history after the token (slots 1, 2 of
 *                                       hist_in, then the token); bit copies.
 *                                       Must not overlap any input.
 *      S_out    fp32 [n_seq][hv][dk][dv]  state after the token; may be the same
 *                                       buffer as S_in (not a partial overlap)
 *      y        fp16 [n_seq][hv][dv] when out_f32 == 0, else fp32
 * No workspace.  n_seq == 0 is a no-op.  Errors as for the other entry points.
 */
GDN_API gdn_status gdn_step(const gdn_dims* dims, int32_t n_seq, const uint16_t* qkv, const float* conv_w,
                            const uint16_t* hist_in, uint16_t* hist_out, const uint16_t* a,
                            const uint16_t* b, const uint16_t* z, const float* A_log,
                            const float* dt_bias, const float* gamma, const float* S_in, float* S_out,
                            int32_t out_f32, void* y, struct CUstream_st* stream);

/* ------------------------------------------------------------------------
 * Attention layers between GDN layers: an 8-bit paged cache of keys and
 * values, the append that fills it, the attention that reads it, and the
 * check of drafted tokens.  The pages have no counterpart to these.
 * ------------------------------------------------------------------------ */

/* activation type of q, k, v and the attention's output; fp32 is for the
 * residual stream of gdn_block_norm alone */
typedef enum gdn_dtype { GDN_FP16 = 0, GDN_BF16 = 1, GDN_FP32 = 2 } gdn_dtype;

/* what a cache byte holds: a two's complement integer in [-127, 127], or a
 * 4-bit-exponent, 3-bit-mantissa float (largest value 448, no infinities) */
typedef enum gdn_kv_format { GDN_KV_INT8 = 0, GDN_KV_E4M3 = 1 } gdn_kv_format;

/*
 * gdn_kv_cache -- one layer's pool of pages.  A page holds page_tokens
 * consecutive positions of one sequence for every kv head; which page holds
 * which positions is the page table's affair:
 *   page_table  int32 [n_seq] rows of max_pages entries, page_table_stride
 *               entries apart: entry j of row s is the pool page of positions
 *               [j * page_tokens, (j + 1) * page_tokens) of sequence s.
 * A value is its code times the scale of its (page, head), one scale for k and
 * one for v.  Scales are 0 (every value 0), a power of two, or NaN (a value
 * that was not finite was stored: everything read from that page and head is
 * NaN, until an append starts at or in front of the first such position; the
 * NaN's bits say what the append needs to know for that, so scales are to be
 * copied as bits).  Fresh pages need no initialisation: the call that stores a
 * page's first position ignores what the page held.
 */
typedef struct gdn_kv_cache {
    int32_t heads;       /* kv heads, 1..1024                              */
    int32_t head_dim;    /* 64 or 128                                      */
    int32_t page_tokens; /* 16, 32, 64 or 128                              */
    int32_t n_pages;     /* pages in the pool                              */
    int32_t format;      /* gdn_kv_format                                  */
    uint8_t* k;          /* [n_pages][heads][page_tokens][head_dim]        */
    uint8_t* v;          /* [n_pages][heads][page_tokens][head_dim]        */
    float* k_scale;      /* [n_pages][heads]                               */
    float* v_scale;      /* [n_pages][heads]                               */
} gdn_kv_cache;

/*
 * gdn_kv_append -- stores the new tokens' keys and values, rotating keys (and
 * queries) by their positions on the way.
 *
 * Token i of sequence s has position past[s] + i, past[s] being the tokens
 * that the sequence already holds.
 *
 * In:  past     int32 [n_seq] (device)
 *      q        [T][hq][head_dim], k, v [T][heads][head_dim] of `dtype`; tokens
 *               are q_stride, k_stride, v_stride elements apart (multiples of
 *               8: the three may be slices of one packed projection, or lie
 *               further apart; arrays that span more than 2^58 elements are
 *               refused).  q may be NULL (hq 0): only k and v are stored.
 *      cos, sin fp32 [n_pos][rot_dim / 2], the rotation of each position
 *               (positions past the table take its last row); NULL with
 *               rot_dim 0 for none.  rot_dim: a multiple of 16 up to head_dim;
 *               the channels behind it are left as they are.  Channel pairs
 *               (a, b) are (j, j + rot_dim/2) when interleaved == 0, (2j, 2j + 1)
 *               when 1, and turn to (a c - b s, b c + a s), each product and sum
 *               rounded to fp32.
 * Out: q_out    [T][hq][head_dim] dense, of `dtype`; overlaps no input
 *      the cache: with x the rotated k (or v) in fp32, a page and head's scale
 *      becomes the larger of its own and the smallest power of two (at least
 *      2^-100) not below max|x| / 127 (int8) or max|x| / 448 (e4m3) over its new
 *      tokens, its own counting as 0 when this call stores the page's first
 *      position.  New codes are x / scale to nearest even; where the scale grew,
 *      the codes of the page's earlier positions are divided by the growth and
 *      rounded again.  The error of a value is therefore below one code step
 *      of its page, however its page was filled.
 * A position that is negative, past the table row or whose entry is outside
 * [0, n_pages) is not stored (its query is still rotated).  Going back to an
 * earlier length needs no call: append again from there.  What was stored
 * behind that length and is given up leaves one mark, on the page that the
 * length ends in: a larger value among it has grown the page's scale, which
 * does not fall again, so the page's kept values have been rounded to the
 * coarser steps.  Values that are not finite leave none: they count as 0 in
 * max|x|, and the page's other codes are what they would be without them.  Two
 * sequences of one call must not store into the same page.
 */
GDN_API gdn_status gdn_kv_append(const gdn_kv_cache* cache, int32_t dtype, int32_t n_seq,
                                 int32_t total_tokens, const int32_t* cu_seqlens, const int32_t* past,
                                 const int32_t* page_table, int64_t page_table_stride,
                                 int32_t max_pages, int32_t hq, const uint16_t* q, int64_t q_stride,
                                 const uint16_t* k, int64_t k_stride, const uint16_t* v,
                                 int64_t v_stride, const float* cos, const float* sin,
                                 int32_t rot_dim, int32_t n_pos, int32_t interleaved,
                                 uint16_t* q_out, struct CUstream_st* stream);

/* Workspace bytes gdn_kv_attn needs for this batch shape (0 for one that it
 * refuses): parts of outputs, some 16 MB at head_dim 128, and where the batch
 * can hold a sequence of more than 96 query rows per kv head, 40 MB more and
 * unpacked copies of such sequences' caches, 4 bytes per code byte up to 2 GB
 * (sequences that find no room are attended to without). */
GDN_API size_t gdn_kv_attn_workspace_bytes(const gdn_kv_cache* cache, int32_t n_seq,
                                           int32_t total_tokens, int32_t hq, int32_t max_pages);

/*
 * gdn_kv_attn -- causal attention of the new tokens over the cache (after
 * their own gdn_kv_append): for query head h and its kv head h / (hq / heads),
 *   y = sum_j softmax_j(softmax_scale * q . k_j) v_j   over positions
 *   j <= past[s] + i.
 * A position whose table entry is outside [0, n_pages), or past the table row,
 * is not seen; a token that sees none (past[s] + i < 0, say, for an idle slot
 * of a captured batch) gives zeros.  A query that is not finite gives NaN.
 *
 * In:  q        [T][hq][head_dim] of `dtype`, tokens q_stride elements apart (a
 *               multiple of 8); hq a multiple of heads, at most 64 per kv head
 * Out: y        [T][hq][head_dim] dense, of `dtype`
 * workspace: device scratch of at least gdn_kv_attn_workspace_bytes() bytes;
 *            contents on entry are ignored.  Calls sharing one must not overlap
 *            on the GPU.
 * Scores, softmax statistics and sums are fp32, exponentials the hardware's;
 * the softmax weights are rounded to fp16 for their product with v (11 bits, in
 * steps of 2^-31 of the largest weight below).  A call may be captured into a CUDA
 * graph; the lengths in `past` may change between replays.
 */
GDN_API gdn_status gdn_kv_attn(const gdn_kv_cache* cache, int32_t dtype, int32_t n_seq,
                               int32_t total_tokens, const int32_t* cu_seqlens, const int32_t* past,
                               const int32_t* page_table, int64_t page_table_stride,
                               int32_t max_pages, int32_t hq, const uint16_t* q, int64_t q_stride,
                               float softmax_scale, uint16_t* y, void* workspace,
                               size_t workspace_bytes, struct CUstream_st* stream);

/*
 * gdn_kv_attn_check -- the failure report of the last gdn_kv_attn on this
 * workspace: every wait inside its kernels is bounded (about two seconds), and
 * one that expires ends its CTA and is recorded, as for the scan.  Enqueues a
 * 4-byte device-to-host copy on `stream`, SYNCHRONISES it and returns GDN_OK or
 * GDN_ERR_TIMEOUT (that call's outputs are invalid).
 */
GDN_API gdn_status gdn_kv_attn_check(const void* workspace, struct CUstream_st* stream);

/*
 * gdn_draft_verify -- accepts or replaces drafted tokens so that the tokens
 * kept are distributed as the target's.
 *
 * Sequence s has n_draft[s] drafts (n_draft NULL: max_draft; clamped to
 * [0, max_draft]), drawn from the rows q; row i of p is the target's
 * distribution at draft i, row n_draft[s] the one after the last draft.
 *   accepted[s] = the number of leading drafts i with u[s][i] q_i(x_i) < p_i(x_i)
 *                 (fp32 product; a draft outside [0, vocab) is not accepted)
 *   next[s]     = the token after them: the first index whose running sum of
 *                 weights exceeds floor(u[s][max_draft] W), W the sum of all.
 *                 The weight of a token is floor(min(max(x, 0), 1) 2^43), NaN
 *                 counting as 0, with x = p - q (fp32) at the first draft not
 *                 accepted, x = p after the last draft.  If W = 0, x = p; if W is
 *                 still 0, next[s] = -1.
 * The sums are of whole numbers, so the result does not depend on their order.
 *
 * In:  p        fp32 [n_seq][max_draft + 1] rows of vocab, p_stride apart
 *      q        fp32 [n_seq][max_draft] rows of vocab, q_stride apart
 *               (NULL when max_draft is 0)
 *      draft    int32 [n_seq][max_draft];  n_draft int32 [n_seq] or NULL
 *      u        fp32 [n_seq][max_draft + 1], uniform in [0, 1)
 * Out: accepted, next  int32 [n_seq]
 * vocab: 1..2^19.  These arrays need 4-byte alignment only.
 */
GDN_API gdn_status gdn_draft_verify(int32_t n_seq, int32_t max_draft, int32_t vocab, const float* p,
                                    int64_t p_stride, const float* q, int64_t q_stride,
                                    const int32_t* draft, const int32_t* n_draft, const float* u,
                                    int32_t* accepted, int32_t* next, struct CUstream_st* stream);

/*
 * gdn_kv_remap -- the page table of a batch's next step from that of its last:
 * rows forked, cut, dropped and grown in one call, with their pages shared
 * where they can be.  Row r of the new table
 *   keeps   the first keep[r] tokens of row parent[r] of the old table (r itself
 *           to go on; another's to fork it; keep[r] = 0 or a parent outside
 *           [0, n_old): nothing), that is its first ceil(keep[r] / page_tokens)
 *           entries;
 *   gets    room for need[r] tokens: new pages up to
 *           ceil(need[r] / page_tokens) entries (never fewer than it keeps).
 * Pages that no row of the new table keeps are free, whoever had them.  A row
 * with need[r] > keep[r] whose kept tokens end inside a page will write into
 * that page.  Where another row keeps the page too it takes a new page in its
 * place and the pair is listed for gdn_kv_copy; of rows that all write into the
 * page the lowest keeps it.  (A row that keeps a page without writing into it
 * never loses it.)  New pages go to the rows in order, a row's copy first, then
 * its other entries in order, and are the free pages in order.
 * If there are too few, the last to ask get none: their entries are -1 (what
 * is appended there is not stored), and info says how many.
 *
 * In:  page_table  int32 [n_old] rows of max_pages entries, page_table_stride
 *                  apart; an entry outside [0, n_pages) names no page and is
 *                  kept as -1 (nothing is copied for it)
 *      parent, keep, need  int32 [n_rows]; lengths below 0 count as 0, and
 *                  past the row's end as its end
 * Out: table_out   int32 [n_rows] rows of max_pages entries, table_out_stride
 *                  apart, -1 behind what a row has; overlaps no input
 *      copy_from, copy_to  int32 [n_rows]: the page that row r's last kept
 *                  page is to be copied from and to, or -1.  A page that is
 *                  copied from is never copied to, so gdn_kv_copy may follow
 *                  at once, and the append behind it.
 *      info        int32 [2]: pages that the new table names, and pages that
 *                  were wanted and not there
 * Nothing is kept between calls: what a row does not name is free.  To hold
 * pages for later (a shared prompt, say) keep a row for them.
 * page_tokens as in gdn_kv_cache; n_pages up to 2^28; n_rows, n_rows *
 * max_pages, max_pages * page_tokens and the tables' strides up to 2^30.  The
 * int32 arrays need 4-byte alignment only.  workspace: at least
 * gdn_kv_remap_workspace_bytes() bytes (0 for a shape that is refused); contents
 * on entry are ignored, calls sharing one must not overlap on the GPU.  May be
 * captured into a CUDA graph.
 */
GDN_API size_t gdn_kv_remap_workspace_bytes(int32_t n_pages, int32_t n_rows, int32_t max_pages);
GDN_API gdn_status gdn_kv_remap(int32_t page_tokens, int32_t n_pages, int32_t max_pages, int32_t n_old,
                                const int32_t* page_table, int64_t page_table_stride, int32_t n_rows,
                                const int32_t* parent, const int32_t* keep, const int32_t* need,
                                int32_t* table_out, int64_t table_out_stride, int32_t* copy_from,
                                int32_t* copy_to, int32_t* info, void* workspace, size_t workspace_bytes,
                                struct CUstream_st* stream);

/*
 * gdn_kv_compact -- renames pages so that those in use are the pool's first
 * ones: with U pages named by the table, those at or behind U move, in order, to
 * the free ones in front of U, in order.
 *
 * In:  page_table  int32 [n_rows] rows of max_pages entries, page_table_stride
 *                  apart; entries outside [0, n_pages) name no page
 * Out: table_out   the same with the new names, -1 where an entry names no
 *                  page; table_out_stride apart; may be page_table itself with
 *                  the same stride, else overlaps it nowhere
 *      copy_from, copy_to  int32 [n_pages / 2]: the moves, -1 behind them.  No
 *                  page is in both lists: gdn_kv_copy may follow at once.
 *      info        int32 [2]: U, and the number of moves
 * Limits, alignment, workspace and capture as for gdn_kv_remap.
 */
GDN_API size_t gdn_kv_compact_workspace_bytes(int32_t n_pages);
GDN_API gdn_status gdn_kv_compact(int32_t n_pages, int32_t max_pages, int32_t n_rows, const int32_t* page_table,
                                  int64_t page_table_stride, int32_t* table_out, int64_t table_out_stride,
                                  int32_t* copy_from, int32_t* copy_to, int32_t* info, void* workspace,
                                  size_t workspace_bytes, struct CUstream_st* stream);

/*
 * gdn_kv_copy -- copies pages (codes and scales, as bits) within the caches of
 * all layers that share a page table: page copy_from[i] to copy_to[i] for
 * i < n, in each cache.  A pair with an index outside [0, n_pages), or twice
 * the same, is passed over.  A page may be copied from more than once; a page
 * that is copied to is in the lists once (twice, or as a source too: its
 * contents are then some mixture of the pages named).
 *
 * In:  caches      host array of n_caches caches (up to 1024) with the same heads,
 *                  head_dim, page_tokens, n_pages and format, none overlapping
 *                  another
 *      copy_from, copy_to  int32 [n] (device, 4-byte aligned), n up to 2^30
 */
GDN_API gdn_status gdn_kv_copy(const gdn_kv_cache* caches, int32_t n_caches, int32_t n, const int32_t* copy_from,
                               const int32_t* copy_to, struct CUstream_st* stream);

/* ------------------------------------------------------------------------
 * Around the layers, for a server of many requests: the residual stream
 * between blocks, and adapters beside the projections.  The pages have no
 * counterpart to these.
 * ------------------------------------------------------------------------ */

/* what a block's output is multiplied with: nothing, the gate as it is, its
 * sigmoid, or gate * sigmoid(gate) */
typedef enum gdn_gate { GDN_GATE_NONE = 0, GDN_GATE_LINEAR = 1, GDN_GATE_SIGMOID = 2, GDN_GATE_SILU = 3 } gdn_gate;

/*
 * gdn_block_norm -- a block's output joins the residual stream, which is
 * normalised for the next block:
 *   u  = y, or y / sqrt(mean(y^2) + eps) * post_weight where that is given
 *   x' = x + scale * act(gate) * u          (act(gate) = 1 for GDN_GATE_NONE)
 *   h  = x' / sqrt(mean(x'^2) + eps) * pre_weight
 * token by token over `width` channels, in fp32 throughout: x' and h are each
 * rounded once, h from x' before its rounding.
 *
 * In:  x       [T][width] of x_dtype: `dtype`, or GDN_FP32
 *      y       [T][width] of `dtype` (GDN_FP16 or GDN_BF16), or NULL: x' = x
 *              (in front of the first block; gate, post_weight and x_out NULL)
 *      gate    [T][width] of `dtype`; gate_stride 0: one row for all tokens;
 *              NULL with GDN_GATE_NONE
 *      post_weight, pre_weight  fp32 [width]; post_weight NULL: y is taken as
 *              it is; pre_weight NULL with h NULL
 *      Tokens are x_stride, y_stride, gate_stride elements apart (multiples of
 *      8 up to 2^30; y may be a slice of a wider row).
 * Out: x_out   [T][width] dense, of x_dtype; NULL: x' is not wanted (behind the
 *              last block).  May be x itself where x_stride == width; overlaps
 *              nothing else.
 *      h       [T][width] dense, of `dtype`, or NULL: not wanted (not both)
 * width: a multiple of 8 up to 16384.  eps > 0.  Squares are summed in fp32, so
 * rows with values beyond 1e19 have a norm of infinity.
 */
GDN_API gdn_status gdn_block_norm(int32_t x_dtype, int32_t dtype, int32_t total_tokens, int32_t width,
                                  const void* x, int64_t x_stride, const uint16_t* y, int64_t y_stride,
                                  const uint16_t* gate, int64_t gate_stride, int32_t gate_kind,
                                  float scale, const float* post_weight, const float* pre_weight,
                                  float eps, void* x_out, uint16_t* h, struct CUstream_st* stream);

/*
 * gdn_adapter_add -- the low-rank adapter of each sequence added to the output
 * of a projection that all share: for token t of sequence s, a = ids[s],
 *   h     = down[a] x[t]                      (ranks[a] values)
 *   y_out[t] = y[t] + scales[a] * up[a]^T h
 * A sequence whose id is outside [0, n_adapters), or whose adapter's rank is 0,
 * has none: y_out = y.
 *
 * In:  ids     int32 [n_seq] (device)
 *      ranks   int32 [n_adapters], clamped to [0, rank], or NULL: all `rank`.
 *              What down and up hold behind an adapter's rank is not read.
 *      down    [n_adapters][rank][d_in], up [n_adapters][rank][d_out], of `dtype`
 *      scales  fp32 [n_adapters]
 *      x       [T][d_in], y [T][d_out] of `dtype` (GDN_FP16 or GDN_BF16); tokens
 *              are x_stride, y_stride elements apart (multiples of 8 up to 2^30:
 *              y may be the q slice of a packed projection, say)
 * Out: y_out   [T][d_out] of `dtype`, y_out_stride apart; may be y itself with
 *              the same stride, else overlaps no input
 * rank: a multiple of 8 up to 128; d_in, d_out: multiples of 8 up to 65536;
 * n_adapters up to 2^20.  ids, ranks and scales need 4-byte alignment only.
 * Sums are fp32, and y_out is rounded once.  h enters its product in fp32, or, in
 * tiles of many tokens, in two pieces of the weights' type: 17 bits or more in
 * bf16; 22 in fp16, or 2^-39 of the token's largest.  So the last bits in fp32 of
 * what is added may differ with the batch that a token comes in.  Values of x and
 * of the weights that are not finite reach the tokens, and the channels, that
 * their products reach (an infinity in `up` as infinity or NaN).
 * workspace: device scratch of at least gdn_adapter_workspace_bytes() bytes (0
 * for a shape that is refused, and for no tokens); contents on entry are
 * ignored, calls sharing one must not overlap on the GPU.  May be captured into
 * a CUDA graph; ids and lengths may change between replays.
 */
GDN_API size_t gdn_adapter_workspace_bytes(int32_t n_seq, int32_t total_tokens, int32_t rank, int32_t d_in);
GDN_API gdn_status gdn_adapter_add(int32_t dtype, int32_t n_seq, int32_t total_tokens, const int32_t* cu_seqlens,
                                   const int32_t* ids, int32_t n_adapters, int32_t rank, const int32_t* ranks,
                                   const uint16_t* down, const uint16_t* up, const float* scales, int32_t d_in,
                                   const uint16_t* x, int64_t x_stride, int32_t d_out, const uint16_t* y,
                                   int64_t y_stride, uint16_t* y_out, int64_t y_out_stride, void* workspace,
                                   size_t workspace_bytes, struct CUstream_st* stream);

/*
 * gdn_adapter_check -- the failure report of the last gdn_adapter_add with
 * tokens on this workspace: every wait inside its kernels is bounded, and one
 * that expires is recorded (that call's outputs are invalid).  Enqueues a small
 * device-to-host copy on `stream`, SYNCHRONISES it and returns GDN_OK or
 * GDN_ERR_TIMEOUT.
 */
GDN_API gdn_status gdn_adapter_check(const void* workspace, struct CUstream_st* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
