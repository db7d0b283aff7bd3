/*
 * jattn.h — C ABI of libjattn: MM-DiT joint self-attention with QK-RMSNorm,
 * forward and backward, on one NVIDIA GB300 (sm_103a).
 *
 * The operation (re-diffusion README — "architecture flowchart": inside each
 * DiT layer the caption-stream and image-stream Q/K/V are concatenated as
 * [c; x] and one multi-head self-attention runs over the joint sequence;
 * "design notes" table, row "QK norm": RMSNorm on Q and on K; "attention fix"
 * section: scaled-dot-product attention over the same [B, H, N, d] Q/K/V
 * layout, without materialising the B x H x N x N score matrix):
 *
 *   r(x)   = (mean_c x_c^2 + eps)^(-1/2),  eps = 1e-6          (per row)
 *   q_hat  = bf16(gq * q * r(q)),  k_hat = bf16(gk * k * r(k))
 *   S      = q_hat k_hat^T / sqrt(d)                           (per b, h)
 *   LSE_i  = ln sum_j exp(S_ij),   O = exp(S - LSE) V
 *
 * Layout.  q, k, v, out, dout, dq, dk, dv are contiguous row-major
 * [B, H, N, d] bfloat16 (stored as uint16_t bit patterns), N = N_txt + N_img
 * with the N_txt caption rows first, then the N_img image rows.  lse is
 * [B, H, N] float32, natural log.  gq, gk, dgq, dgk are [d] float32, one gain
 * vector shared by all heads.  No mask, dropout or causality: N_txt and N_img
 * only define N and the row order.
 *
 * Pointers.  Every array pointer is a DEVICE pointer (CUDA global memory),
 * 16-byte aligned.  `stream` is a cudaStream_t passed as void* (NULL = the
 * legacy default stream); all work is enqueued on it and the call returns
 * without synchronising.  The caller owns every buffer.  The library
 * allocates its scratch memory per call, stream-ordered on `stream`
 * (cudaMallocAsync / cudaFreeAsync), and keeps no state between calls.
 *
 * Errors.  Every entry point returns a jattn_status and never aborts or
 * prints.  Arguments are validated before anything is enqueued; a non-OK
 * status from validation means nothing ran.  JATTN_ERR_CUDA reports a failed
 * launch or allocation.  The kernels' internal waits are bounded: a wait
 * that gives up ends the kernel early and jattn_last_device_error() then
 * reports it (it synchronises `stream`).  Asynchronous faults surface, as
 * usual in CUDA, at the caller's next synchronisation.
 */
#ifndef JATTN_H
#define JATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t jattn_bf16; /* bfloat16 bit pattern */

typedef enum {
  JATTN_OK = 0,
  JATTN_ERR_INVALID_ARG = 1, /* null pointer, B/H/d <= 0, N_img/N_txt < 0, N < 1, size overflow */
  JATTN_ERR_UNSUPPORTED = 2, /* d not in {64, 128}; projections and token rows: C not a multiple of 8 (8-bit tokens:
                                of 16; token rows: or above JATTN_MAX_WIDTH), rank not as jattn_qkv_norm_lora says */
  JATTN_ERR_MISALIGNED = 3,  /* a pointer is not 16-byte aligned */
  JATTN_ERR_ALIAS = 4,       /* an output buffer overlaps an input or another output */
  JATTN_ERR_CUDA = 5,        /* a CUDA launch or allocation failed */
  JATTN_ERR_TIMEOUT = 6,     /* a device-side bounded wait gave up (reported by jattn_last_device_error) */
  JATTN_ERR_SCRATCH_LIMIT = 7 /* jattn_fwd_noalloc: the problem needs more scratch than its fixed array holds */
} jattn_status;

/*
 * Forward.  Computes out = softmax(q_hat k_hat^T / sqrt(d)) v and lse (the
 * natural-log row log-sum-exp of the scaled scores) for every (b, h).
 *   q, k, v : [B, H, N, d] bf16, read only.
 *   gq, gk  : [d] float32 RMSNorm gains for q and k, read only.
 *   B, H    : batch size and heads (>= 1).
 *   N_img   : image-token rows, N_txt: caption-token rows (>= 0 each,
 *             N = N_img + N_txt >= 1).
 *   d       : head dimension, 64 or 128.
 *   out     : [B, H, N, d] bf16, overwritten.
 *   lse     : [B, H, N] float32, overwritten.
 * Limits: B*H*N*d < 2^31.
 */
int jattn_fwd(const jattn_bf16* q, const jattn_bf16* k, const jattn_bf16* v, const float* gq, const float* gk,
              int B, int H, int N_img, int N_txt, int d, jattn_bf16* out, float* lse, void* stream);

/*
 * Backward.  Given the forward's inputs, its outputs (out, lse) and the
 * upstream gradient dout, computes the gradients of L = sum(dout * out):
 *   dq, dk, dv : [B, H, N, d] bf16, overwritten.
 *   dgq, dgk   : [d] float32, overwritten (summed over all b, h, n).
 * The bf16 rounding of q_hat/k_hat is treated as the identity.  The
 * normalised q_hat/k_hat are recomputed from q, k (nothing is cached from
 * the forward call; jattn_fwd_train / jattn_bwd_train below keep them).  dk, dv and dgk are always summed in a fixed order and
 * repeat bit for bit.  dq is accumulated in float32 across key tiles: by
 * default with reduce-adds in arrival order, so that dq and dgq (a sum over
 * dq's accumulator) may differ in the last bits between runs; with
 * jattn_set_deterministic(1), in a fixed order, so that all five gradients
 * repeat bit for bit (on the same GPU model and CTA cap).
 */
int jattn_bwd(const jattn_bf16* q, const jattn_bf16* k, const jattn_bf16* v, const float* gq, const float* gk,
              const jattn_bf16* out, const float* lse, const jattn_bf16* dout, jattn_bf16* dq, jattn_bf16* dk,
              jattn_bf16* dv, float* dgq, float* dgk, int B, int H, int N_img, int N_txt, int d, void* stream);

/*
 * Packed variable-length forward and backward: one call over sequences of
 * different lengths, each attending only within itself.  This is for batches
 * that mix resolutions, for example images from different aspect-ratio buckets
 * with their captions.  The re-diffusion README's training-data paragraph
 * describes the aspect-bucketed export, and its roadmap lists multi-resolution
 * training.
 *   Layout: [H, T, d] bf16 with T = cu_seqlens[n_seqs].  Head h holds T rows,
 *           and sequence s is rows cu_seqlens[s] .. cu_seqlens[s+1]-1 of every
 *           head.  This is the [B, H, N, d] layout with B = 1 and the
 *           sequences concatenated along N; each sequence lists its caption
 *           rows and image rows in any order.
 *   cu_seqlens: HOST array of n_seqs + 1 ints, cu_seqlens[0] = 0, strictly
 *           increasing (every sequence has at least one row); read during
 *           the call only.
 *   n_seqs: 1 .. JATTN_MAX_SEQS.
 *   lse   : [H, T] float32.
 *   The other arguments and every status are those of jattn_fwd / jattn_bwd.
 *   An invalid cu_seqlens gives JATTN_ERR_INVALID_ARG; n_seqs above
 *   JATTN_MAX_SEQS gives JATTN_ERR_UNSUPPORTED.  H*T*d < 2^31.
 * dgq and dgk sum over every sequence, head and row.
 */
#define JATTN_MAX_SEQS 256
int jattn_fwd_varlen(const jattn_bf16* q, const jattn_bf16* k, const jattn_bf16* v, const float* gq, const float* gk,
                     const int* cu_seqlens, int n_seqs, int H, int d, jattn_bf16* out, float* lse, void* stream);
int jattn_bwd_varlen(const jattn_bf16* q, const jattn_bf16* k, const jattn_bf16* v, const float* gq, const float* gk,
                     const jattn_bf16* out, const float* lse, const jattn_bf16* dout, jattn_bf16* dq, jattn_bf16* dk,
                     jattn_bf16* dv, float* dgq, float* dgk, const int* cu_seqlens, int n_seqs, int H, int d,
                     void* stream);

/*
 * Training pair: a forward that keeps the normalised q_hat, k_hat and the
 * rows' 1/rms r(q), r(k) in a caller buffer `saved`, and a backward that
 * reads them there instead of recomputing them (the autograd practice of
 * saving an op's activations for its backward).  Results are those of
 * jattn_fwd / jattn_bwd with the same arguments, bit for bit where those
 * repeat bit for bit.
 *   saved : DEVICE buffer of jattn_saved_bytes(...) bytes (16-byte aligned),
 *           written by the forward and used by the backward, which must be
 *           given the same q, k, gq, gk and shape; its layout is private.
 *           It may not overlap any other argument.  It also holds the
 *           backward's fp32 dQ accumulator, which the forward zeroes while it
 *           runs (with HBM bandwidth its attention kernel leaves idle) so
 *           that the backward need not; a backward that finds it not zeroed
 *           by a forward since the last backward (a second backward on the
 *           same buffer, or a buffer no forward has filled) zeroes it itself,
 *           so any number of backward calls per forward stay correct.
 *           Size: 2 B*H*N*d*2 + B*H*N*d*4 + 2 B*H*N*4 bytes plus alignment.
 * jattn_saved_bytes returns 0 for a shape the calls would reject.  The other
 * arguments and every status are those of jattn_fwd / jattn_bwd (and of
 * their varlen forms); a null `saved` gives JATTN_ERR_INVALID_ARG.
 */
size_t jattn_saved_bytes(int B, int H, int N_img, int N_txt, int d);
size_t jattn_saved_bytes_varlen(const int* cu_seqlens, int n_seqs, int H, int d);
int jattn_fwd_train(const jattn_bf16* q, const jattn_bf16* k, const jattn_bf16* v, const float* gq, const float* gk,
                    int B, int H, int N_img, int N_txt, int d, jattn_bf16* out, float* lse, void* saved,
                    void* stream);
int jattn_bwd_train(const jattn_bf16* q, const jattn_bf16* k, const jattn_bf16* v, const float* gq, const float* gk,
                    const jattn_bf16* out, const float* lse, const jattn_bf16* dout, void* saved,
                    jattn_bf16* dq, jattn_bf16* dk, jattn_bf16* dv, float* dgq, float* dgk, int B, int H, int N_img,
                    int N_txt, int d, void* stream);
int jattn_fwd_train_varlen(const jattn_bf16* q, const jattn_bf16* k, const jattn_bf16* v, const float* gq,
                           const float* gk, const int* cu_seqlens, int n_seqs, int H, int d, jattn_bf16* out,
                           float* lse, void* saved, void* stream);
int jattn_bwd_train_varlen(const jattn_bf16* q, const jattn_bf16* k, const jattn_bf16* v, const float* gq,
                           const float* gk, const jattn_bf16* out, const float* lse, const jattn_bf16* dout,
                           void* saved, jattn_bf16* dq, jattn_bf16* dk, jattn_bf16* dv, float* dgq, float* dgk,
                           const int* cu_seqlens, int n_seqs, int H, int d, void* stream);

/*
 * QKV projection with QK-RMSNorm in its epilogue (re-diffusion README,
 * "architecture flowchart": each stream's tokens are projected to Q, K, V
 * with that stream's own weights, the streams are concatenated along the
 * token axis and Q, K are RMS-normalised before the attention; "design notes"
 * table, row "QK norm").  One call computes, for both streams,
 *
 *   Y = bf16(X W^T + b)           fp32 accumulation, bias added in fp32,
 *                                 then one rounding to bf16
 *   q, k, v = the Y columns of each head, written into the joint layout
 *   q_hat, k_hat, 1/rms of every q and k row, as jattn_fwd_train keeps them
 *
 * so that jattn_fwd_saved can start the attention from q_hat / k_hat and
 * jattn_bwd_train can run the backward, with no normalisation pass of their
 * own.  Results are those of projecting, then calling jattn_fwd_train on the
 * projected q, k, v: q_hat, k_hat bit for bit (both correctly rounded), the
 * 1/rms values to fp32 rounding.
 *   x_img  : [B, N_img, C] bf16 image-stream tokens (rows N_txt .. N - 1)
 *   w_img  : [3 H d, C] bf16 image-stream weight, row-major like a linear
 *            layer's weight: rows h d .. h d + d - 1 give head h of q, rows
 *            H d + h d .. of k, rows 2 H d + h d .. of v
 *   b_img  : [3 H d] float32 bias, or NULL for none
 *   x_txt, w_txt, b_txt : the caption stream's, likewise (rows 0 .. N_txt - 1);
 *            a stream with no rows may pass NULL tokens and weight
 *   gq, gk : [d] float32 gains
 *   C      : model width, a multiple of 8 (else JATTN_ERR_UNSUPPORTED)
 *   q, k, v: [B, H, N, d] outputs (the layout above)
 *   saved  : jattn_saved_bytes(B, H, N_img, N_txt, d) bytes, written as a
 *            training forward writes it
 * Every pointer is a 16-byte aligned DEVICE pointer (q, k, v and saved at
 * 32-byte boundaries are written 3 to 25 % faster); outputs may not overlap
 * inputs or each other (JATTN_ERR_ALIAS).  The [B, H, N, d] layout only (no
 * varlen form).  Sizes: 3 H d C, B N_img C and B N_txt C below 2^31.
 *
 * jattn_fwd_saved is the attention forward of a training pair whose q_hat /
 * k_hat are already in `saved` (from jattn_qkv_norm, or from jattn_fwd_train
 * with the same shape): out and lse as jattn_fwd computes them from the q, k
 * that gave those q_hat / k_hat.  It launches the attention kernel only (which
 * also zeroes the buffer's dQ accumulator, as jattn_fwd_train does).
 */
int jattn_qkv_norm(const jattn_bf16* x_img, const jattn_bf16* w_img, const float* b_img, const jattn_bf16* x_txt,
                   const jattn_bf16* w_txt, const float* b_txt, const float* gq, const float* gk, int B, int H,
                   int N_img, int N_txt, int d, int C, jattn_bf16* q, jattn_bf16* k, jattn_bf16* v, void* saved,
                   void* stream);
int jattn_fwd_saved(const jattn_bf16* v, int B, int H, int N_img, int N_txt, int d, jattn_bf16* out, float* lse,
                    void* saved, void* stream);

/*
 * Token rows: the residual's addition with RMSNorm over the model width, and
 * rows in 8 bits with scales.  (The steps before the QKV projection; the pages
 * name no code for them.)  For T rows of C values, row-major and contiguous:
 *
 *   h = bf16(x + res)                       (without res: h is x)
 *   r = (mean_c h_c^2 + eps)^(-1/2)         fp32
 *   z = g * h * r                           fp32
 *   y = bf16(z), or 8 bits: m = max(max_c |z_c|, 2^-80), s = m / 448 (fp32),
 *                           y8 = e4m3(448 z / m), the real quotient in fp32 first
 *
 * e4m3 is 1 sign, 4 exponent and 3 mantissa bits, largest finite value 448,
 * one byte a value; a row stands for s * y8.  The sum of squares is fp32: a
 * row whose sum passes the fp32 range comes out as zeros.  A row with
 * a NaN comes out as NaN (jattn_quant_rows: the NaN values stay NaN and do not
 * enter the row's maximum); 8-bit rows with an infinite z read NaN.
 *   x     : [T, C] bf16
 *   res   : [T, C] bf16 or NULL
 *   g     : [C] float32
 *   T, C  : T >= 1 rows; C a multiple of 8, at most JATTN_MAX_WIDTH (else
 *           JATTN_ERR_UNSUPPORTED).  T * C may pass 2^31.
 *   eps   : > 0 and finite
 *   h     : [T, C] bf16, overwritten; it may be res itself (the residual
 *           stream updated in place), and is NULL exactly if res is
 *   y, y8 : [T, C] bf16, or bytes
 *   s     : [T] float32
 *   r     : [T] float32, or NULL when no backward will run
 * jattn_quant_rows does the last step alone on z = x (weights once when they
 * are loaded, or tokens that another norm made).
 *
 * jattn_add_norm_bwd: with n = h r and u = g dy, for the gradients dy of y and
 * dh of h (or NULL: none),
 *
 *   dx = dh + r (u - n mean_c(u n)),    dg = sum_t dy n
 *
 * dx [T, C] bf16 is the gradient of x and of res alike, and may be dh itself;
 * dg [C] float32 is summed in a fixed order that T and C alone set, so both
 * repeat bit for bit.  h and r are the forward's (without res, h is x).
 *   work  : jattn_add_norm_bwd_bytes(T, C) bytes, contents of no meaning
 *           before or after; calls that overlap on the GPU need one each.
 * jattn_add_norm_bwd_bytes returns 0 for sizes the call would reject.
 */
#define JATTN_MAX_WIDTH 16384
int jattn_add_norm(const jattn_bf16* x, const jattn_bf16* res, const float* g, int T, int C, float eps,
                   jattn_bf16* h, jattn_bf16* y, float* r, void* stream);
int jattn_add_norm_fp8(const jattn_bf16* x, const jattn_bf16* res, const float* g, int T, int C, float eps,
                       jattn_bf16* h, uint8_t* y8, float* s, float* r, void* stream);
int jattn_quant_rows(const jattn_bf16* x, int T, int C, uint8_t* x8, float* s, void* stream);
size_t jattn_add_norm_bwd_bytes(int T, int C);
int jattn_add_norm_bwd(const jattn_bf16* dy, const jattn_bf16* dh, const jattn_bf16* h, const float* r,
                       const float* g, int T, int C, jattn_bf16* dx, float* dg, void* work, void* stream);

/*
 * The projection from 8-bit tokens and weights (serving; 8-bit tokens carry
 * no gradient).  jattn_qkv_norm with rows in e4m3 and their fp32 scales, as
 * jattn_add_norm_fp8 and jattn_quant_rows write them:
 *
 *   Y = bf16((sum_c x8_tc w8_oc) sx_t sw_o + b_o)   fp32, in this order
 *
 *   x_img, x_txt   : [B, N_img, C] and [B, N_txt, C] bytes
 *   sx_img, sx_txt : [B, N_img] and [B, N_txt] float32
 *   w_img, w_txt   : [3 H d, C] bytes
 *   sw_img, sw_txt : [3 H d] float32
 *   C              : a multiple of 16 (else JATTN_ERR_UNSUPPORTED)
 * Everything else is jattn_qkv_norm's.
 */
int jattn_qkv_norm_fp8(const uint8_t* x_img, const float* sx_img, const uint8_t* w_img, const float* sw_img,
                       const float* b_img, const uint8_t* x_txt, const float* sx_txt, const uint8_t* w_txt,
                       const float* sw_txt, const float* b_txt, const float* gq, const float* gk, int B, int H,
                       int N_img, int N_txt, int d, int C, jattn_bf16* q, jattn_bf16* k, jattn_bf16* v, void* saved,
                       void* stream);

/*
 * The projection with low-rank adapters of the batch items' own (serving
 * many requests, each with its adapter, in one batch).  For item b with a =
 * index[b], per stream and part p of (q, k, v):
 *
 *   U_p = scale[a] X A_ap^T                         fp32, kept in full
 *   Y_p = bf16(X W_p^T + U_p B_ap^T + b_p)          fp32 accumulation, one rounding
 *
 * and for an item whose index is outside 0 .. n_adapters - 1, jattn_qkv_norm's
 * Y.  The rest (heads, joint layout, q_hat, k_hat, 1/rms in `saved`) is
 * jattn_qkv_norm's.
 *   down_img, down_txt : [n_adapters, 3 rank, C] bf16, rows p rank .. p rank +
 *                        rank - 1 of adapter a are A_ap
 *   up_img, up_txt     : [n_adapters, 3 H d, rank] bf16, rows p H d .. of
 *                        adapter a are B_ap; a stream may have neither (both
 *                        NULL): no adapters there
 *   scale              : [n_adapters] float32
 *   index              : [B] int32, read on the device by each call (a captured
 *                        graph replays with what it then holds); any value is
 *                        allowed, and any items may share an adapter
 *   n_adapters         : >= 1
 *   rank               : a multiple of 8, 8 .. JATTN_MAX_RANK (else
 *                        JATTN_ERR_UNSUPPORTED); adapters of lower rank are
 *                        padded with zeros by the caller
 *   work               : jattn_qkv_norm_lora_bytes(...) bytes for U, contents of
 *                        no meaning before or after; calls that overlap on the
 *                        GPU need one each
 * A tile of 128 or 256 tokens takes each different adapter among its items in
 * turn, wherever in the tile they lie.
 * jattn_qkv_norm_lora_bytes returns 0 for sizes the call would reject.
 */
#define JATTN_MAX_RANK 128
size_t jattn_qkv_norm_lora_bytes(int B, int H, int N_img, int N_txt, int d, int rank);
int jattn_qkv_norm_lora(const jattn_bf16* x_img, const jattn_bf16* w_img, const float* b_img,
                        const jattn_bf16* x_txt, const jattn_bf16* w_txt, const float* b_txt, const float* gq,
                        const float* gk, const jattn_bf16* down_img, const jattn_bf16* up_img,
                        const jattn_bf16* down_txt, const jattn_bf16* up_txt, const float* scale, const int* index,
                        int n_adapters, int rank, int B, int H, int N_img, int N_txt, int d, int C, jattn_bf16* q,
                        jattn_bf16* k, jattn_bf16* v, void* saved, void* work, void* stream);

/*
 * Forward without any device allocation.  (No counterpart on the pages: an
 * integration entry point.)  Same arguments, layout and results as jattn_fwd,
 * but the scratch it needs (the normalised q_hat and k_hat, 2 * 2 * B*H*N*d
 * bytes, each part 256-byte aligned) lives in one fixed file-scope device
 * array of JATTN_NOALLOC_SCRATCH_BYTES (64 MiB) instead of a per-call
 * cudaMallocAsync.  It calls no cudaMalloc / cudaFree / allocating library
 * routine.
 *
 * Who needs it: callers that cannot let a library allocate device memory, such
 * as a serving process that reserves nearly all of HBM for its own pool up
 * front (a library allocation would then fail mid-step), or a launch sequence
 * that must never block on or recover from an allocator call.
 *
 * Rules:
 *  - Problems needing more than the array (B*H*N*d > 16,777,216 = 2^24 at these
 *    alignments, e.g. the 768 px / d = 128 workload) return
 *    JATTN_ERR_SCRATCH_LIMIT before anything is enqueued.
 *  - The first call on each device looks up the array's device address
 *    (cudaGetSymbolAddress, with that device current) and caches it; make
 *    that first call before any stream capture.
 *  - Every call, on any stream, shares the one array, which keeps the last
 *    call's contents.  Nothing in it needs clearing (the norm kernel writes
 *    every element it is later read back from), but calls that overlap on the
 *    GPU (for example on two streams at once) race on it: serialise them.
 *  - Every GPU that loads this library holds the array until the process
 *    exits.
 */
#define JATTN_NOALLOC_SCRATCH_BYTES (64u * 1024u * 1024u)
int jattn_fwd_noalloc(const jattn_bf16* q, const jattn_bf16* k, const jattn_bf16* v, const float* gq, const float* gk,
                      int B, int H, int N_img, int N_txt, int d, jattn_bf16* out, float* lse, void* stream);

/*
 * Synchronises `stream` and returns JATTN_ERR_TIMEOUT if any kernel launched
 * by this library on the current device since the previous call gave up a
 * bounded wait, JATTN_ERR_CUDA if the synchronisation itself failed, else
 * JATTN_OK.  Clears the recorded device error.
 */
int jattn_last_device_error(void* stream);

/*
 * Self-test of the bounded-wait path (no counterpart on the pages: failure
 * detection).  Enqueues on `stream` a one-thread kernel that waits on an
 * mbarrier nothing ever arrives at.  The wait is the one every attention
 * kernel uses: it gives up after its limit (about 1 s), records the device
 * error and returns, so the context stays usable.  The next
 * jattn_last_device_error(stream) then returns JATTN_ERR_TIMEOUT.  Returns
 * JATTN_OK, or JATTN_ERR_CUDA if the launch failed.
 */
int jattn_selftest_wait_timeout(void* stream);

/*
 * Kernel timing (off by default; no counterpart on the pages: measurement
 * support).  While enabled, every kernel launch made by the library
 * on the calling thread's device is bracketed by two CUDA events recorded on
 * the caller's stream.  jattn_profile_read synchronises on those events and
 * adds, for one kernel kind, the number of launches and their summed
 * event-to-event milliseconds since the last jattn_profile_reset.
 */
typedef enum {
  JATTN_KERNEL_QK_NORM_FWD = 0,  /* RMSNorm of q and k (forward) */
  JATTN_KERNEL_ATTN_FWD = 1,     /* tensor-core attention forward */
  JATTN_KERNEL_BWD_PREP = 2,     /* norm recompute + rowsum(dO*O) + dq accumulator clear */
  JATTN_KERNEL_ATTN_BWD = 3,     /* tensor-core attention backward (+ K-norm backward) */
  JATTN_KERNEL_Q_NORM_BWD = 4,   /* Q-norm backward from the dq accumulator, and the gain gradients */
  JATTN_KERNEL_QKV_NORM = 5,     /* QKV projection of both streams with the QK-RMSNorm epilogue */
  JATTN_KERNEL_COUNT = 6
} jattn_kernel_kind;

/* Kinds of the token-row kernels, numbered apart from the attention path's
 * (jattn_profile_read and jattn_kernel_name take both). */
typedef enum {
  JATTN_TOKEN_KERNEL_FIRST = 16,
  JATTN_KERNEL_ADD_NORM = 16,      /* residual + RMSNorm, either output */
  JATTN_KERNEL_ADD_NORM_BWD = 17,  /* its backward: dx and partial sums of dg */
  JATTN_KERNEL_ADD_NORM_DG = 18,   /* dg from the partial sums */
  JATTN_KERNEL_QUANT_ROWS = 19,    /* rows to 8 bits */
  JATTN_KERNEL_LORA_DOWN = 20,     /* the adapters' first product (the projections themselves: QKV_NORM) */
  JATTN_TOKEN_KERNEL_END = 21
} jattn_token_kernel_kind;

int jattn_profile_enable(int on);
int jattn_profile_reset(void);
int jattn_profile_read(int kind, int* launches, double* total_ms);
const char* jattn_kernel_name(int kind);

/*
 * Deterministic backward (off by default; no counterpart on the pages).
 * With on != 0, later jattn_bwd / jattn_bwd_varlen calls from any thread add
 * the key tiles' contributions to each query tile's float32 dq accumulator in
 * a fixed order (the first is stored, each later one is added only after the
 * one before it has completed), so that dq and dgq repeat bit for bit.  The
 * order costs time: contributions wait on one another across CTAs (bounded
 * waits: a stalled wait ends the kernel and jattn_last_device_error reports
 * JATTN_ERR_TIMEOUT).  Every CTA of the launch must be able to run at the
 * same time as the others (see jattn_set_sm_limit).  Returns JATTN_OK.
 */
int jattn_set_deterministic(int on);

/*
 * Caps the number of CTAs the persistent attention kernels launch, and so the
 * SMs they occupy, at max_sms (0 = every SM of the device, the default); for
 * sharing the GPU with concurrent work, and for exercising the kernels' work
 * schedules on small problems.  It applies to later calls from any thread.
 * In the deterministic mode the backward picks its dQ order from it.  A cap
 * above the SMs the process may use (for example under an MPS thread limit)
 * can make the deterministic backward's cross-CTA waits give up
 * (JATTN_ERR_TIMEOUT).  Returns JATTN_ERR_INVALID_ARG for a negative cap.
 * (No counterpart on the pages.)
 */
int jattn_set_sm_limit(int max_sms);

/* Static description of a status code (never NULL). */
const char* jattn_status_string(int status);

/* Human-readable detail of the last failing CUDA call or driver step seen
 * by an entry point on the calling thread (never NULL). */
const char* jattn_last_error_message(void);

/* Library version, major*10000 + minor*100 + patch. */
int jattn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* JATTN_H */
