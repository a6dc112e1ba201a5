/* sffn.h -- predictor-guided, neuron-aware sparse FFN for one MI355X (gfx950).
 *
 * C ABI of libsffn.so. Every entry point takes plain pointers and sizes; all
 * tensor pointers are DEVICE pointers owned by the caller, and the library
 * never allocates device memory. Calls enqueue work on `stream` (a
 * hipStream_t, NULL = the null stream) and return at once; results are valid
 * once the stream has reached them. No call synchronises the device, so a
 * sequence of calls can be captured into a HIP graph.
 *
 * The operation follows the PowerInfer pages:
 *   - "Online stage: neuron-aware inference engine" and "Adaptive sparsity
 *     predictors" (Turkish article): a small per-layer predictor runs on every
 *     token, marks the neurons that will be active, and the engine skips the
 *     rest;
 *   - "Neuron-aware operator" (same article): the sparse operators work on
 *     individual rows and columns of the weight matrices, never a dense copy;
 *   - "Neuron placement and management" (same article): neurons are stored in
 *     a chosen order and a table maps each back to its original position;
 *   - summary bullets and "Limitations/FAQ" (Indonesian digest): ReLU-family
 *     FFNs (ReLU, ReGLU, squared ReLU); "Quantization": INT4 Q4_0 weights.
 *
 * Notation. D = d_model, F = d_ffn (neurons), r = predictor rank, B = tokens
 * of one call (1 for decode; B > 1 computes every token over the union of the
 * per-token masks). "Stored order" is the caller's neuron order (a
 * permutation of the original one); the library never sees the permutation:
 * every per-neuron array (rows of P2, W_gate, W_up, W_down^T, b, c) must be
 * given in the same stored order, and the caller maps ids back.
 *
 * Layouts (row-major, contiguous):
 *   x        [B, D] fp32           token inputs
 *   P1       [r, D] fp16           predictor first factor
 *   P2       [F, r] fp16           predictor second factor (stored order)
 *   c        [F]    fp32 or NULL   predictor bias
 *   W_gate   [F, D] fp16           ReGLU gate rows (stored order), b_gate [F] fp32
 *   W_up     [F, D] fp16           up rows, b_up [F] fp32 (ReLU)
 *   W_downT  [F, D] fp16           W_down transposed: row k = column k of W_down
 *   mask     [ceil(F/64)] uint64   bit (k % 64) of word k / 64 = stored neuron k active
 *   y        [B, D] fp32
 * Q4_0 matrices (sffn_q4): blocks of 32 consecutive weights along d_model in
 * every neuron row, w = (q - 8) * s with q in 0..15:
 *   q  [F, D/2] uint8: for block j of a row, bytes 16j..16j+15; byte i holds
 *      element 32j+i in its low nibble and element 32j+16+i in its high nibble
 *   s  [F, D/32] fp16 scale of each block.
 *
 * Alignment: every tensor pointer 16-byte aligned; the workspace 256-byte
 * aligned. Limits: 1 <= B <= 64; 8 <= D <= 16384 with D % 8 == 0 (D % 32 == 0
 * for Q4_0); 1 <= F <= 1<<22; 8 <= r <= 1024 with r % 8 == 0; B * r <= 32768;
 * every weight matrix and the B x F activations below 2 GiB.
 *
 * Batches. B == 1 (decode) and B == 2 with 2 * D <= 16384 run the decode
 * kernels (vector ALU, x staged once per block); so do B in {4, 8} with
 * B * D <= 16384 when F > 32768. Every other B > 1 runs the union kernels on
 * the matrix cores ("Neuron-aware operator": each active row is read once for
 * the whole batch); these compact the whole mask inside one workgroup and
 * take F <= 32768 in sffn_forward / sffn_forward_q4. With fp16 weights and
 * up to 8 tokens the fp32 inputs and activations enter the matrix cores as
 * two fp16 halves (x = hi + lo), so those results match the decode kernels'
 * to within fp32 rounding; larger batches, and Q4_0 weights, take each as one
 * fp16 value after a per-token power-of-two scaling (relative 2^-11 per
 * value, inside the output tolerance the parity tests hold).
 *
 * Workspace (sffn_workspace_size bytes, 256-byte parts, caller-owned, no
 * state kept between calls): activations a [F, B] fp32 (for B == 1 at least
 * 4 KiB: sffn_decode keeps its per-block decision bitmaps there); for B > 1 the
 * normalised inputs [B, D]; partial sums of y, [256, D] fp32 for B == 1 (one
 * per block of the fused kernel) or [16, B, D] for B > 1 (row splits; the
 * union predictor also keeps its partial h there); for B > 1 the partial
 * pre-activations of the k-split union row kernel, [KS, 2, F, B] fp32 (KS = 8,
 * 4 or 2 shares for 7-8, 9-16 and 17-32 tokens, none otherwise), the union
 * row kernel's token operands (room for two fp16 planes of ceil(D/32) x
 * ceil(B/16) KiB, then 16 fp32 per 16 tokens) and its largest |a| per row
 * tile and token; the predictor's h [B, r] fp32 last. One workspace may serve
 * the predict and
 * forward calls of a layer in turn on one stream; calls that overlap in time
 * need separate workspaces.
 *
 * Errors: arguments are checked on the host before anything is enqueued; a
 * failed check returns its status and leaves the stream untouched. A failed
 * launch returns SFFN_ERR_HIP. sffn_last_error() gives the detail text of the
 * calling thread's last failure. No exception crosses the ABI.
 */
#ifndef SFFN_H
#define SFFN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SFFN_OK = 0,
  SFFN_ERR_NULL = 1,       /* a required pointer is NULL                      */
  SFFN_ERR_SHAPE = 2,      /* B, D, F or r outside the limits above            */
  SFFN_ERR_ALIGN = 3,      /* a pointer is not aligned as required             */
  SFFN_ERR_WORKSPACE = 4,  /* workspace smaller than sffn_workspace_size()     */
  SFFN_ERR_ACT = 5,        /* unknown activation, or operands it needs missing */
  SFFN_ERR_ARG = 6,        /* other bad argument (threshold outside (0, 1))    */
  SFFN_ERR_HIP = 7         /* the HIP runtime reported an error                */
} sffn_status;

typedef enum {
  SFFN_ACT_RELU = 0,   /* a_k = max(0, W_up[k] x + b_up[k])                        */
  SFFN_ACT_REGLU = 1,  /* a_k = max(0, W_gate[k] x + b_gate[k]) * (W_up[k] x)      */
  SFFN_ACT_SQRELU = 2  /* a_k = max(0, W_up[k] x + b_up[k])^2  (squared ReLU; operands as for RELU) */
} sffn_act;

/* One Q4_0 matrix (device pointers, layout above). */
typedef struct {
  const uint8_t* q;
  const void* s;
} sffn_q4;

/* Text of a status code (static storage). */
const char* sffn_status_string(int status);

/* Detail of the calling thread's last failure ("" if none). */
const char* sffn_last_error(void);

/* Bytes of workspace that sffn_predict / sffn_forward / sffn_forward_q4 need for these sizes. */
size_t sffn_workspace_size(int B, int D, int F, int r);

/* Number of 64-bit mask words for F neurons: ceil(F / 64). */
int sffn_mask_words(int F);

/* Which kernels sffn_forward (q4 = 0) or sffn_forward_q4 (q4 = 1) runs for these sizes:
 *   SFFN_PATH_FUSED (B == 1, F <= 32768, and D <= 5120 for fp16 ReGLU, D <= 8192 for fp16 ReLU and for Q4_0):
 *     one kernel gathers the gate/up rows, applies the activation and accumulates the W_downT rows into
 *     per-block partial sums of y; a second kernel adds the partials in fixed order (timing ids SFFN_K_ROWS and
 *     SFFN_K_COLS);
 *   SFFN_PATH_DECODE (other B == 1; B == 2 with 2 * D <= 16384; B in {4, 8} with B * D <= 16384 and
 *     F > 32768): row gather + activation, then the column gather;
 *   SFFN_PATH_UNION (every other B): matrix-core kernels over the union mask.
 * Returns -1 for an unknown activation. */
enum { SFFN_PATH_DECODE = 0, SFFN_PATH_FUSED = 1, SFFN_PATH_UNION = 2 };
int sffn_forward_path(int act, int q4, int B, int D, int F);

/* Activation predictor ("Adaptive sparsity predictors"; "Online stage").
 *   h[b, :] = P1 xn[b, :]                     (fp32 accumulate; h is never rounded)
 *   z[b, k] = P2[k, :] h[b, :] + c[k]         (c = NULL means 0)
 *   neuron k active  <=>  sigmoid(z[b, k]) > t for some token b
 *                    <=>  z[b, k] > ln(t / (1 - t))  (decided in logit space)
 * xn = x, or, if x_norm != 0, xn[b, :] = (x[b, :] - m) / sqrt(v + 1e-6) with m the mean and v the
 * (population) variance of x[b, :] -- the parameter-free normalisation between stacked layers, applied as the
 * input is loaded.
 * Outputs: mask (every word written, bits >= F zero); logits [B, F] fp32 if
 * non-NULL. Uses the workspace. Two kernels for B <= 8 (h, then z; a normalised input is normalised as it is
 * loaded); for B > 8 three (partial h over shares of d, their sum, z), after a normalisation pass with x_norm. */
int sffn_predict(const void* P1, const void* P2, const float* c, const float* x, int x_norm, int B, int D, int F,
                 int r, float t, uint64_t* mask, float* logits, void* ws, size_t ws_bytes, void* stream);

/* sffn_predict with an always-active prefix ("Neuron placement and management", Turkish article: neurons are
 * stored in a chosen order, here hottest first). Stored neurons 0 .. n_hot-1 are set in the mask whatever the
 * predictor would say, and their rows of P2 and entries of c are never read (P2 and c must still span all F
 * rows; only rows >= n_hot are loaded). Their logits, if requested, are written as +infinity. Every other
 * neuron is decided exactly as by sffn_predict, which is this call with n_hot = 0. SFFN_ERR_ARG if n_hot is
 * outside 0..F. */
int sffn_predict_hot(const void* P1, const void* P2, const float* c, const float* x, int x_norm, int B, int D, int F,
                     int r, float t, int n_hot, uint64_t* mask, float* logits, void* ws, size_t ws_bytes,
                     void* stream);

/* Neuron-aware sparse FFN over the neurons set in `mask` ("Neuron-aware operator").
 *   compaction: active[0 .. n) = ascending stored ids of the set bits, *n_active = n
 *   a[b, j]  = act(row active[j] of W_gate / W_up, xn[b, :])   (only active rows are read)
 *   y[b, :]  = sum_j a[b, j] * W_downT[active[j], :]          (only active rows are read)
 * xn as in sffn_predict. W_gate / b_gate are used (and required) for REGLU only;
 * RELU and SQRELU read W_up and b_up; b_up may be NULL (0). active [F] int32 and n_active [1] int32 are device
 * outputs; y [B, D] is overwritten. Uses the workspace. Two kernels; the union kernels add a sum of the row-split partials (and a normalisation pass for x_norm). */
int sffn_forward(int act, const void* W_gate, const float* b_gate, const void* W_up, const float* b_up,
                 const void* W_downT, const float* x, int x_norm, int B, int D, int F, const uint64_t* mask,
                 int32_t* active, int32_t* n_active, float* y, void* ws, size_t ws_bytes, void* stream);

/* sffn_forward with Q4_0 weights ("Quantization": INT4 Q4_0); weights are
 * dequantised in registers, w = (q - 8) * s exactly in fp32. */
int sffn_forward_q4(int act, sffn_q4 W_gate, const float* b_gate, sffn_q4 W_up, const float* b_up, sffn_q4 W_downT,
                    const float* x, int x_norm, int B, int D, int F, const uint64_t* mask, int32_t* active,
                    int32_t* n_active, float* y, void* ws, size_t ws_bytes, void* stream);

/* One decode step of one layer for a single token: sffn_predict_hot (n_hot = 0: sffn_predict) followed by
 * sffn_forward, with the same operands, outputs and results ("Adaptive sparsity predictors" and "Neuron-aware
 * operator", Turkish article). mask, active, n_active, y and logits (if non-NULL) are written as the two calls
 * would write them. Where sffn_decode_path says SFFN_DECODE_FOLDED, the predictor's second stage runs inside
 * the row gather: each of the 256 workgroups decides the neurons it owns (stored neurons k with k % 256 equal to
 * its index) and gathers the active ones at once, so the layer takes three kernels instead of four and one
 * dependent round trip less; the mask and the ascending ids are assembled while the partial sums of y are added.
 * Otherwise the two calls run as they are. fp16 weights only (the Q4_0 forward keeps its separate calls). Uses
 * the workspace of sffn_workspace_size(1, D, F, r). Errors as sffn_predict and sffn_forward. */
enum { SFFN_DECODE_SEPARATE = 0, SFFN_DECODE_FOLDED = 1 };
int sffn_decode_path(int act, int q4, int D, int F, int r);   /* -1 for an unknown activation */
int sffn_decode(int act, const void* P1, const void* P2, const float* c, float t, int n_hot, const void* W_gate,
                const float* b_gate, const void* W_up, const float* b_up, const void* W_downT, const float* x,
                int x_norm, int D, int F, int r, uint64_t* mask, int32_t* active, int32_t* n_active, float* y,
                float* logits, void* ws, size_t ws_bytes, void* stream);

/* sffn_decode without a workspace argument, for callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc. Same operands, outputs and results as
 * sffn_decode. Its workspace is a scratch array of sffn_noalloc_scratch_bytes() bytes (16 MiB) in the library's
 * own device memory: one per GPU, allocated when the library is loaded on that GPU and held until the process
 * ends. The call allocates nothing. Sizes whose workspace (sffn_workspace_size(1, D, F, r)) exceeds the scratch
 * return SFFN_ERR_WORKSPACE before anything is enqueued (D = 8192, F = 32768, r = 1024 need 8.1 MiB). Every call
 * on one GPU shares that GPU's scratch, which keeps the last call's contents (no call needs them): calls that
 * overlap in time on one GPU (several streams or host threads) race on it and must be serialised by the caller.
 * The first call on a device looks up the scratch's address there (SFFN_ERR_HIP if that fails). */
size_t sffn_noalloc_scratch_bytes(void);
int sffn_decode_noalloc(int act, const void* P1, const void* P2, const float* c, float t, int n_hot,
                        const void* W_gate, const float* b_gate, const void* W_up, const float* b_up,
                        const void* W_downT, const float* x, int x_norm, int D, int F, int r, uint64_t* mask,
                        int32_t* active, int32_t* n_active, float* y, float* logits, void* stream);

/* Per-launch timing of one kernel (profiling aid; not needed for computing).
 * kernel: SFFN_K_PRED_H (P1 x), SFFN_K_PRED_Z (P2 h + c, threshold, mask), SFFN_K_ROWS (compaction + W_gate /
 * W_up row gather + activation), SFFN_K_COLS (W_downT column gather; in the union path the row-split down
 * projection, not the sum of its partials). In a folded sffn_decode the folded kernel (predictor stage 2 + row
 * gather) is SFFN_K_ROWS and the sum of partials with the mask assembly SFFN_K_COLS.
 * Between sffn_profile_begin and sffn_profile_end, every launch of that kernel made by the calling thread, up
 * to max_launches of them, is issued with a pair of HIP events that take the kernel's own start and end
 * timestamps (hipExtLaunchKernelGGL): the kernel's time on the device, without host-side queueing. The events
 * are created by sffn_profile_begin (host call; launches under graph capture are not timed: profile eager
 * calls). sffn_profile_end waits for the last event, writes the elapsed milliseconds of the launches to
 * ms[0 .. min(count, max)) and returns the count (negative status on error). Returns SFFN_ERR_ARG for a bad
 * kernel id or max_launches < 1. */
enum { SFFN_K_PRED_H = 0, SFFN_K_PRED_Z = 1, SFFN_K_ROWS = 2, SFFN_K_COLS = 3 };
int sffn_profile_begin(int kernel, int max_launches);
int sffn_profile_end(float* ms, int max);

/* ---------------------------------------------------------------------------------------------------------------
 * The attention half of a layer: residual norm, paged K/V cache, attention of new tokens over it. Errors, streams and
 * checks as above; the stream belongs to the current device.
 *
 * Element types. 16-bit tensors (queries, new K / V, outputs) are SFFN_F16 or SFFN_BF16. A cache holds the same
 * 16-bit type, or 8-bit codes (SFFN_I8, SFFN_E4M3: OCP e4m3) with one fp32 scale per token and head:
 *   scale = fp32(max|x| / top), top = 127 or 448;  code = x / scale rounded to nearest, ties to even (of the exact
 *   quotient);  value = code * scale.
 * Rows whose scale would be below 2^-60 are stored as zeros with scale 0; a row that holds an infinity or NaN is
 * stored with scale NaN and codes 0. sffn_kv_read takes any scale; sffn_attn takes V scales that are NaN, 0 (with codes 0) or
 * finite and at least 2^-60, as they are stored. */
typedef enum { SFFN_F32 = 0, SFFN_F16 = 1, SFFN_BF16 = 2, SFFN_I8 = 3, SFFN_E4M3 = 4 } sffn_type;

/* One layer's cache (device pointers, contiguous): k, v [n_pages, n_kv_heads, page, head_dim], and for 8-bit types
 * k_scale, v_scale [n_pages, n_kv_heads, page] fp32 (else ignored). page: a power of two, 16 .. 1024. head_dim: a
 * multiple of 8 (16 for 8-bit types), 16 .. 256. n_pages * n_kv_heads * page < 2^31; n_kv_heads <= 65535. */
typedef struct {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int type, n_pages, page, n_kv_heads, head_dim;
} sffn_kv;

/* The sequences of a call (device pointers to int32). Rows cu[s] .. cu[s + 1] - 1 of the call's token tensors (T rows
 * in all; cu [S + 1] ascends from 0) are the newest tokens of sequence s, whose cache holds kv_len[s] tokens with
 * them: the i-th of n stands at position kv_len[s] - n + i. Position p lies in slot p % page of page
 * table[s * table_stride + p / page]; a table row holds max_pages entries. Rows at and behind cu[S] belong to no
 * sequence: they are not written, and what they hold has no effect. The arrays are read on the device, so they are not checked on the
 * host; whatever they hold, no access leaves the given tensors: a position outside the table row or a page id
 * outside 0 .. n_pages - 1 holds no token (not written, not read, not seen). New tokens keep their positions there: of a
 * sequence that has run past its table row the last ones are not held, and see what the row holds. kv_len counts up to
 * 2^30 + 2^24. Tokens before a sequence's first (kv_len[s] < n) see nothing. 1 <= S <= 65535, 0 <= T <= 2^24 (T = 0: nothing is done), max_pages * page <= 2^30. */
typedef struct {
  const int32_t* cu;
  const int32_t* kv_len;
  const int32_t* table;
  int S, T, max_pages, table_stride;
} sffn_seqs;

/* New tokens' K and V into the cache. k, v: [T, n_kv_heads, head_dim] of a 16-bit `type` (the cache's own if that has
 * 16 bits), tokens k_stride and v_stride elements apart (multiples of 8, at least n_kv_heads * head_dim, so columns
 * of a fused Q/K/V product serve as they are). T * n_kv_heads * head_dim, the last rounded up to 32, 64, 128 or 256,
 * < 2^36. Two tokens of one call that share a slot (sequences whose tables
 * share the page that is written) leave it undefined. One kernel. */
int sffn_kv_write(sffn_kv cache, sffn_seqs seqs, int type, const void* k, int64_t k_stride, const void* v,
                  int64_t v_stride, void* stream);

/* The other way: the rows named by seqs (cu[s + 1] - cu[s] = kv_len[s] takes whole sequences) as contiguous K and V,
 * code * scale rounded once to `type`; a 16-bit cache is copied. Limits as above. Rows whose position holds no token stay as they
 * were. One kernel. */
int sffn_kv_read(sffn_kv cache, sffn_seqs seqs, int type, void* k, int64_t k_stride, void* v, int64_t v_stride,
                 void* stream);

/* Attention of the new tokens over the cache, which holds them already (sffn_kv_write first):
 *   out[t, h, :] = sum_j softmax_j(scale * q[t, h, :] . K[j, h', :]) V[j, h', :],   h' = h / (Hq / n_kv_heads)
 * over the positions j that token t at position p sees: j <= p, j < kv_len, and if window > 0 also j > p - window or
 * j < sinks (a sliding window beside which the first `sinks` tokens stay visible). A token that sees nothing gets
 * zeros. What lies in places a token does not see, infinities and NaN (of an 8-bit cache: NaN scales, and e4m3's NaN codes,
 * which no write stores) included, has no effect on it.
 * q [T, Hq, head_dim] of a 16-bit `type` (the cache's own if that has 16 bits), out likewise, tokens q_stride and
 * out_stride elements apart (multiples of 8). lse [T, Hq] fp32 or NULL: the natural logarithm of the softmax's sum
 * (-infinity for a token that sees nothing). Scores, sums and accumulators are fp32; the weights enter the second
 * product as 16-bit values of the cache's type (fp16 over 8-bit caches; those under 2^-21 of a token's largest, times the
 * scales there, are off by up to 2^-32 of it), and 8-bit codes enter both products exactly. Over an 8-bit cache the V scales
 * that one token sees lie within 2^80 of each other (beyond it the sum loses the part of those with small ones), and bf16
 * queries enter the first product rounded to steps of 2^-38 of the largest finite element among the rows of a workgroup (of
 * 2^-150 where that one is below 2^-112).
 * max_q: at least the largest number of new tokens of one sequence (tokens past it are not computed and their rows
 * stay as they were). max_kv: about the largest kv_len; it decides only over how many workgroups a sequence's keys
 * are spread. Up to 32 rows max_q * Hq / n_kv_heads (64 for head_dim <= 64, 16 for head_dim > 128) run the few-row kernel
 * (SFFN_ATTN_FEW), more run the tile kernel (SFFN_ATTN_MANY); where keys are spread a second kernel joins the parts
 * in a fixed order, so the same call gives the same bits. The workspace needs sffn_attn_workspace_size bytes of
 * the same sizes (0: none needed, ws may be NULL); it holds nothing between calls, and calls that overlap in time
 * need separate ones. Hq * T < 2^31; for the tile kernel Hq * T / 128 + n_kv_heads * min(S, T) < 2^24. */
enum { SFFN_ATTN_FEW = 0, SFFN_ATTN_MANY = 1 };
int sffn_attn_path(int Hq, int n_kv_heads, int head_dim, int max_q);   /* -1 for bad sizes */
size_t sffn_attn_workspace_size(int T, int S, int Hq, int n_kv_heads, int head_dim, int max_q, int max_kv, int window,
                                int sinks);
int sffn_attn(sffn_kv cache, sffn_seqs seqs, int type, const void* q, int64_t q_stride, int Hq, int max_q, int max_kv,
              float scale, int window, int sinks, void* out, int64_t out_stride, float* lse, void* ws, size_t ws_bytes,
              void* stream);

/* Root-mean-square norm with the residual's addition:
 *   h = x + res (fp32; h = x if res is NULL);  res_out = h rounded to res_type (if non-NULL; may be res itself,
 *                                                           with its stride)
 *   y = h / sqrt(mean(h^2) + eps) * w          (from the unrounded h)
 * x, res, res_out [T, D] of SFFN_F32 / F16 / BF16 (res and res_out of one type), w [D] fp32 or NULL (1), y [T, D] of
 * any type; 8-bit y is codes with y_scale [T] fp32 as in the cache, per row and without its lower limit, computed in
 * 64 bits from h on. Row strides in elements, multiples of 8, at least D. D as elsewhere:
 * 8 <= D <= 16384, D % 8 == 0. eps >= 0. y overlaps no input. 0 <= T <= 2^24. One kernel for each 2^21 rows. */
int sffn_add_rmsnorm(int x_type, const void* x, int64_t x_stride, int res_type, const void* res, int64_t res_stride,
                     const float* w, double eps, int T, int D, int y_type, void* y, int64_t y_stride, float* y_scale,
                     void* res_out, int64_t res_out_stride, void* stream);

/* ---------------------------------------------------------------------------------------------------------------
 * What joins the attention half: 8-bit products for its projections, norms and rotation of queries and keys, and a cache that
 * keeps the tokens that attention goes to. Errors, streams and checks as above.
 *
 * Blocks of 128 columns as e4m3 codes: rows = 1 gives every row of x [T, D] (F32, F16 or BF16) one fp32 scale for each 128 of
 * its columns (activations), rows = 128 one for each 128 x 128 block (weights); the last blocks may be smaller.
 *   scale = fp32(max|x| / 448);  code = x / scale rounded to nearest, ties to even (of the exact quotient)
 * A scale below 2^-60 becomes 0 with codes 0; a block that holds an infinity or NaN gets the scale NaN and codes 0.
 * y [T, D] codes, scale [ceil(T / rows), ceil(D / 128)]. Row strides in elements, multiples of 8, at least D. 8 <= D <= 65536,
 * D % 8 == 0; 0 <= T <= 2^24. y overlaps no input. One kernel. */
int sffn_quant128(int x_type, const void* x, int64_t x_stride, int T, int D, int rows, void* y, int64_t y_stride,
                  float* scale, void* stream);

/* Product of two such matrices:
 *   out[t, n] = sum_kb a_scale[t, kb] b_scale[n / 128, kb] * sum_{k in kb} a[t, k] b[n, k]
 * a [T, K] codes with a_scale [T, ceil(K / 128)], b [N, K] codes with b_scale [ceil(N / 128), ceil(K / 128)] (scales contiguous),
 * out [T, N] of F32, F16 or BF16, rounded once. The sums over a block are fp32 (codes widened exactly to fp16 products) up to 64
 * tokens and for fp32 results; 16-bit results of more tokens take the 8-bit matrix instruction, which drops of each 8 products what
 * lies 2^-13 under the largest one's leading bit (of independent terms about a tenth of fp16's rounding of the result; more where
 * large products cancel: fp32 results keep it whatever the number of tokens). Blocks are scaled and added in fp32, so the product of a block's two scales, and its sum times that, have to
 * stay in fp32's range. e4m3's NaN codes and NaN scales make NaN of the results
 * that they enter. K % 16 == 0, 16 <= K <= 65536; N % 8 == 0, 8 <= N <= 2^22; 0 <= T <= 2^24; strides of a and b multiples of
 * 16, at least K, at most 2^22; of out a multiple of 8, at least N. out overlaps no input. The workspace needs
 * sffn_mm_workspace_size bytes of the same sizes (0: none, ws may be NULL), holds nothing between calls, and calls that overlap
 * in time need separate ones. The same call gives the same bits. ceil(T / 128) * ceil(N / 128) < 2^24. */
size_t sffn_mm_workspace_size(int T, int N, int K);
int sffn_mm_e4m3(const void* a, int64_t a_stride, const float* a_scale, const void* b, int64_t b_stride, const float* b_scale,
                 int T, int N, int K, int out_type, void* out, int64_t out_stride, void* ws, size_t ws_bytes, void* stream);

/* Root-mean-square norm of every head of the queries and keys, then the rotation by their positions, in one pass:
 *   h = x / sqrt(mean(x^2) + eps) * w           (norm != 0; over a head's elements; w_q, w_k [head_dim] fp32 or NULL (1). Else h = x.)
 *   y_a = h_a cos f - h_b sin f,  y_b = h_b cos f + h_a sin f,  f = position * freq[i]
 * for the pairs i < rot / 2 of a head's first rot elements: (a, b) = (i, i + rot / 2), or (2 i, 2 i + 1) if `interleaved`; the
 * elements behind stay h. freq [rot / 2] fp32 (finite; not read if rot = 0). The i-th of a sequence's n new tokens (cu as in
 * sffn_seqs) is at position seq_len[s] - n + i: seq_len is kv_len, or what the sequence counts where tokens were evicted. Angles
 * are reduced in 64 bits, the rest is fp32, rounded once.
 * q, q_out [T, Hq, head_dim] and k, k_out [T, n_kv_heads, head_dim] of a 16-bit `type` (k and k_out NULL: queries alone); strides as
 * elsewhere, between tokens, multiples of 8. An output may be its input, with its stride, and overlaps nothing else. Rows at and
 * behind cu[S] are not written. head_dim % 8 == 0, 8 <= head_dim <= 256; rot % 8 == 0, 0 <= rot <= head_dim; Hq, n_kv_heads <=
 * 65535; S, T as elsewhere. One kernel (one for each 2^22 tokens). */
int sffn_qk_norm_rope(int type, const int32_t* cu, const int32_t* seq_len, int S, int T, const void* q, int64_t q_stride, int Hq,
                      const void* k, int64_t k_stride, int n_kv_heads, int head_dim, int norm, const float* w_q, const float* w_k,
                      double eps, const float* freq, int rot, int interleaved, void* q_out, int64_t q_out_stride, void* k_out,
                      int64_t k_out_stride, void* stream);

/* Attention weight of the cached tokens, accumulated: after sffn_attn, with its q, cache, sequences, scale, window and sinks and
 * the lse that it wrote,
 *   mass_out[s, h, j] = (j is a new token's slot ? 0 : mass[s, h, j]) + sum over rows that see j of exp(scale * q . K[j, h] - lse)
 * over the new tokens and the query heads that share K/V head h, for the slots j < min(kv_len[s], what the table row holds, W) of
 * the sequences that have new tokens; everything else stays as it was. New tokens' slots get pos[s, h, j] = the token's position
 * in the sequence, as in sffn_qk_norm_rope. mass, mass_out (which may be mass), pos [S, n_kv_heads, W], contiguous. Rows whose lse
 * is -infinity, and rows past max_q tokens of a sequence, add nothing. What lies in places that a token does not see has no
 * effect. Sums are fp32 in a fixed order: the same call gives the same bits. bf16 queries over an 8-bit cache enter the product
 * as in sffn_attn, or as they are. max_kv is a hint as there, of the workspace's size (sffn_attn_mass_workspace_size bytes of the same
 * sizes; 0: none needed). S * n_kv_heads < 2^22, S * n_kv_heads * W < 2^31. One kernel, or two where a long prompt's rows are shared out. */
size_t sffn_attn_mass_workspace_size(int S, int Hq, int n_kv_heads, int head_dim, int max_q, int max_kv, int W);
int sffn_attn_mass(sffn_kv cache, sffn_seqs seqs, const int32_t* seq_len, int type, const void* q, int64_t q_stride, int Hq,
                   int max_q, int max_kv, float scale, int window, int sinks, const float* lse, const float* mass, float* mass_out,
                   int32_t* pos, int W, void* ws, size_t ws_bytes, void* stream);

/* Eviction: every sequence that holds more than `keep` tokens (of the first W, in its table row) is cut down to `keep` of them,
 * for each K/V head its own: those whose position is below `sinks` or at least seq_len[s] - recent, then those with the largest
 * mass, ties to the lowest slot (a mass that is negative or NaN counts as 0; slots in pages outside the cache go first). Kept
 * tokens in slots at and behind `keep` move, in order, into the given-up slots below it, in order; the others stay where they are.
 * src [S, n_kv_heads, keep] int32: the slot that each of the first `keep` slots' tokens stood in (its own where nothing moved).
 * Moved are K, V, their scales, mass and pos: mass_out and pos_out [S, n_kv_heads, W] get the first min(kv_len, keep) slots (they
 * may be mass and pos themselves), kv_len_out[s] = keep where tokens were evicted, else kv_len[s] (it may be kv_len, but not
 * seq_len, nor kv_len where seq_len is kv_len too: the sequence would forget how long it is). Pages wholly
 * behind the new length are free. Slots are no longer in the order of positions afterwards: attention sees every slot below a
 * new token's whatever its position, but a sliding window would count slots. The pages of the sequences must be their own (not
 * shared between rows of the table). A move into a page outside the cache loses the token. sinks, recent >= 0, sinks + recent <= keep;
 * 1 <= keep <= W; S, n_kv_heads and W as in sffn_attn_mass. cache: its 16-bit type or 8-bit as elsewhere. Limits of cache and table as in sffn_kv_write.
 * The workspace needs sffn_kv_evict_workspace_size bytes. Two kernels up to W = 8192, five above. */
size_t sffn_kv_evict_workspace_size(int S, int n_kv_heads, int W, int keep);
int sffn_kv_evict(sffn_kv cache, const int32_t* kv_len, const int32_t* seq_len, const int32_t* table, int S, int max_pages,
                  int table_stride, const float* mass, const int32_t* pos, int W, int keep, int sinks, int recent, int32_t* src,
                  float* mass_out, int32_t* pos_out, int32_t* kv_len_out, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SFFN_H */
