/*
 * qd.h — C ABI of libqd.so: the token-decode step of a Qwen3-style GQA
 * transformer on one GB300 (sm_103a).
 *
 * Sources (page title, section):
 *   [KL-DEC]  "GPU Kernel Lab" README, "Decode integration": the order of one
 *             decode step (fixed token/position buffers, projections, Q/K
 *             RMSNorm + RoPE + direct K/V cache write, GQA split-KV attention,
 *             residual + RMSNorm, gate/up GEMV + SwiGLU, residual + next
 *             RMSNorm, LM-head GEMV + argmax + token/position update, CUDA
 *             graph replay).
 *   [KL-FUN]  "GPU Kernel Lab" README, "Fundamental kernels": Qwen-exact RMSNorm
 *             cast order, RoPE pair rotation, SwiGLU, stable softmax,
 *             warp-reduced decode GEMV, split-KV decode attention.
 *   [CD-GEMV] "qwen3-8b-rtx4080-cutedsl" README, "Decode GEMV path".
 *   [CD-ATT]  "qwen3-8b-rtx4080-cutedsl" README, "GQA + QK-Norm" and
 *             "Split-KV decode attention".
 *   [CD-ROPE] "qwen3-8b-rtx4080-cutedsl" README, "RoPE vectorized kernel" and
 *             "L2 persistence" (the RoPE frequency table).
 *   [CD-GRAPH] "qwen3-8b-rtx4080-cutedsl" README, "CUDA graphs".
 *   [EQ-SPEED] "emit_qwen38_generate" rustdoc, "Where the speed comes from":
 *             one GEMV per shared activation (concatenated rows), one graph per
 *             token with the token and position advanced on device, residual +
 *             RMSNorm + activation re-quantisation fused, Q8_0 lanes (deq).
 *   [KL-PAGED] "GPU Kernel Lab" README, "Measured final results" / "Serving
 *             system": K/V in fixed physical pages read through a page table.
 *
 * Conventions shared by every call:
 *   - Return value: QD_OK (0) or a negative QD_ERR_* code; qd_last_error()
 *     returns a thread-local message for the last failure of this thread.
 *   - All tensor pointers are DEVICE pointers owned by the caller, unless a
 *     parameter says "host". Pointers must be 16-byte aligned.
 *   - Every call is asynchronous on the given cudaStream_t (0 = legacy default
 *     stream); none synchronises the host, allocates memory or reads device
 *     memory on the host, except qd_check_device_error and the qd_graph_* calls
 *     documented as such. Arguments are validated on the host before any launch;
 *     on an error nothing is launched.
 *   - Matrices are row-major. bf16 = IEEE bfloat16, f16 = IEEE binary16, f32 =
 *     binary32. "Rows" are output features, "cols" the reduction dimension.
 *   - Device-side range faults (a page id outside the cache, a position past
 *     the cache capacity, an all-NaN logit row, a full out_tokens buffer) do not
 *     trap: the kernel skips the access and sets a sticky error word that
 *     qd_check_device_error reports.
 */
#ifndef QD_H
#define QD_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
  QD_OK = 0,
  QD_ERR_INVALID_ARG = -1,
  QD_ERR_UNSUPPORTED = -2,
  QD_ERR_CUDA = -3,
  QD_ERR_WORKSPACE = -4,
  QD_ERR_DEVICE = -5, /* a sticky device-side range fault was recorded */
};

/* device error word bits (qd_check_device_error) */
enum {
  QD_DEVERR_PAGE = 1,      /* page id >= n_pages or logical page >= max_pages */
  QD_DEVERR_POS = 2,       /* position >= cache capacity */
  QD_DEVERR_NAN = 4,       /* an all-NaN logit row in argmax */
  QD_DEVERR_STEPS = 8,     /* step >= max_steps in argmax_advance */
  QD_DEVERR_TIMEOUT = 16,  /* a bounded wait on an asynchronous copy gave up */
  QD_DEVERR_CACHE = 32,    /* a page operation that could not be carried out whole (nothing changed) */
};

/* Weight formats: BF16; Q8_0 (32-wide int8 blocks with an fp16 scale); INT4 (W4A16: */
/* 4-bit codes with one fp16 scale per output row, see qd_gemv_w4).                  */
typedef enum { QD_W_BF16 = 0, QD_W_Q8_0 = 1, QD_W_INT4 = 2 } qd_wtype;
/* Q8_0 activation lanes ([EQ-SPEED] ``deq``): F32 = dequantising lane,
 * I8 = activation re-quantised per 32-block to int8 (dp4a lane). */
typedef enum { QD_ACT_F32 = 0, QD_ACT_I8 = 1 } qd_act;

const char* qd_last_error(void);
int qd_version(void);

/* ------------------------------------------------------------------------ */
/* Weight-streaming GEMV, BF16 weights ([CD-GEMV], [KL-FUN] "warp-reduced     */
/* decode GEMV", [EQ-SPEED] item 1).                                          */
/*   y[b, r] = sum_c W[r, c] * x[b, c]      b < batch, r < rows, c < cols      */
/* W: bf16 [rows, cols]. x: bf16 [batch, cols] (x_is_f32 = 0) or f32            */
/* [batch, cols] (x_is_f32 = 1; the kernel rounds x to bf16 first). y: f32      */
/* [batch, rows]. Accumulation in f32, deterministic order.                   */
/* batch 1: CUDA-core ring GEMV (cols % 8 == 0). batch 2..8 with bf16 x and     */
/* cols % 32 == 0: the weight-streaming GEMV with its multiply-add on mma.sync   */
/* (each weight read once for all rows); otherwise batch <= 8 runs the CUDA-core */
/* GEMV (QD_SMALLB_IMPL=simt forces it). batch >= 9: the product is a dense     */
/* contraction and runs on the tcgen05 tensor cores ("qwen3-8b-rtx4080-         */
/* cutedsl" README, "Baseline tiled GEMM"), one CTA per 128 rows x 64 batch     */
/* rows; above 128 batch rows (a prompt's tokens, for prefill) a persistent     */
/* kernel, one CTA per SM over 128 x 256 tiles (QD_GEMM_WIDE=tiles: one CTA per */
/* tile). Needs bf16 x and cols % 64 == 0.                                      */
int qd_gemv_bf16(const void* W, int rows, int cols, const void* x, int x_is_f32,
                 float* y, int batch, cudaStream_t stream);

/* ------------------------------------------------------------------------ */
/* Q8_0 GEMV, both lanes ([EQ-SPEED] ``deq``).                                 */
/* W = f32(d[r, c/32]) * qs[r, c]; qs: int8 [rows, cols]; d: f16 [rows, cols/32]. */
/* act == QD_ACT_F32: y[r] = sum_b f32(d[r,b]) * sum_i qs[r,32b+i] * x_f32[32b+i] */
/* act == QD_ACT_I8:  y[r] = sum_b f32(d[r,b]) * f32(x_d[b]) * (int32 block dot  */
/*                    of qs and x_q), the int32 dot exact.                      */
/* Unused activation pointers may be NULL. Limits: cols % 32 == 0.             */
int qd_gemv_q8_0(const int8_t* qs, const void* d_f16, int rows, int cols,
                 const float* x_f32, const int8_t* x_q, const void* x_d_f16,
                 qd_act act, float* y, cudaStream_t stream);

/* ------------------------------------------------------------------------ */
/* Batched Q8_0 projection on the tcgen05 tensor cores ("qwen3-8b-rtx4080-     */
/* cutedsl" README, "Baseline tiled GEMM"; Q8_0 blocks per [EQ-SPEED]):          */
/*   y[b, r] = sum_c bf16(f32(d[r, c/32]) * qs[r, c]) * x[b, c]                  */
/* Each weight is widened on chip to bf16 (the product is exact in binary32,     */
/* then one round to nearest even) and the contraction runs as bf16 MMA with f32 */
/* accumulation. qs: int8 [rows, cols]; d: f16 [rows, cols/32]; x: bf16          */
/* [batch, cols]; y: f32 [batch, rows]. workspace: NULL (no K split) or device   */
/* scratch of qd_gemm_workspace_bytes(rows, cols, QD_W_Q8_0) bytes, zero-filled  */
/* before its first use (each call leaves it zero-filled); with it, grids that   */
/* do not fill the SMs split K and sum the partials in split order.              */
/* Limits: cols % 256 == 0, batch >= 1 (above 64: 64-row tiles, no K split and   */
/* the workspace unused), every pointer 16-byte aligned.                         */
size_t qd_gemm_workspace_bytes(int rows, int cols, qd_wtype wtype);
int qd_gemm_q8_0(const int8_t* qs, const void* d_f16, int rows, int cols, const void* x_bf16,
                 int batch, float* y, void* workspace, size_t workspace_bytes,
                 cudaStream_t stream);

/* ------------------------------------------------------------------------ */
/* W4A16 GEMV ("GPU Kernel Lab" README, "Quantization experiments": W4A16 decode */
/* GEMV, packed INT4 LM head with local top-k, per-output-channel weight          */
/* quantization; "qwen3-8b-rtx4080-cutedsl" README, "W4A16 dequant-fused GEMM").   */
/* W: uint8 [rows, cols/2], each byte two offset-binary nibbles u = q + 8 (q in    */
/* [-8, 7]), the even column in the low nibble; d: f16 [rows], one scale per row:  */
/* w[r, c] = f32(d[r]) * q[r, c].  y[r] = sum_c w[r, c] * x[c] with x bf16 [cols];  */
/* y f32 [rows]; batch 1, f32 accumulation. Limits: cols % 32 == 0, cols <= 16384; */
/* W and x 16-byte aligned, d 2-byte aligned.                                      */
int qd_gemv_w4(const uint8_t* W, const void* d_f16, int rows, int cols, const void* x_bf16, float* y,
               cudaStream_t stream);
/* The same with a workspace: with cols % 256 == 0 the product runs on the tcgen05  */
/* tensor cores (each weight code widened to bf16 in tensor memory, the activation */
/* as the other operand), and a matrix whose 128-row tiles underfill the SMs      */
/* splits K across CTAs, adding the partials in split order. workspace: NULL (no  */
/* split; what qd_gemv_w4 does) or zero-filled device scratch of                  */
/* qd_gemv_w4_workspace_bytes(rows, cols) bytes (0: no split), left zero-filled.  */
size_t qd_gemv_w4_workspace_bytes(int rows, int cols);
int qd_gemv_w4_ex(const uint8_t* W, const void* d_f16, int rows, int cols, const void* x_bf16, float* y,
                  void* workspace, size_t workspace_bytes, cudaStream_t stream);
/* The INT4 LM-head form: y as qd_gemv_w4 (the logits), and the top k rows of y     */
/* (value descending, the lower row first among equal values, NaN never chosen):  */
/* topk_ids int32 [k] (-1 past the non-NaN rows), topk_vals f32 [k]. Each CTA picks */
/* the top k of its rows; the last CTA merges them. 1 <= k <= 16. workspace:        */
/* zero-filled device scratch of qd_w4_topk_workspace_bytes() bytes, left zero.   */
size_t qd_w4_topk_workspace_bytes(void);
int qd_gemv_w4_topk(const uint8_t* W, const void* d_f16, int rows, int cols, const void* x_bf16, int k,
                    float* y, int32_t* topk_ids, float* topk_vals, void* workspace, size_t workspace_bytes,
                    cudaStream_t stream);

/* Activation re-quantisation per 32-block ([EQ-SPEED] item 3): amax = max|x|,  */
/* d = amax / 127, q = round-half-away(x * (1/d)) in IEEE binary32 (0 if d = 0), */
/* d stored as f16 (round to nearest even). x: f32 [n]; x_q: int8 [n];            */
/* x_d: f16 [n/32]. Limits: n % 32 == 0.                                        */
int qd_quantize_q8_0(const float* x, int n, int8_t* x_q, void* x_d_f16, cudaStream_t stream);

/* ------------------------------------------------------------------------ */
/* GQA split-KV decode attention over a paged cache ([CD-ATT], [KL-FUN],       */
/* [KL-PAGED]).                                                               */
/*   out[b, h, :] = sum_{t < seq_lens[b]} softmax_t(scale * q[b,h,:].K_b[t,g,:]) */
/*                  * V_b[t, g, :],   g = h / (n_q_heads / n_kv_heads)          */
/* q: f32 [batch, n_q_heads, head_dim]. k_pages, v_pages: bf16                  */
/* [n_pages, n_kv_heads, page_size, head_dim]; logical token t of sequence b    */
/* lives in page page_table[b * max_pages + t / page_size], slot t % page_size. */
/* page_table: int32 [batch, max_pages]. seq_lens: int32 [batch] (device).      */
/* out: f32 [batch, n_q_heads, head_dim]. workspace: device scratch of at least  */
/* qd_attn_workspace_bytes(...) bytes, zero-filled before its first use (the   */
/* call leaves it zero-filled again). seq_lens[b] == 0 gives out = 0.           */
/* Limits: head_dim == 128, n_q_heads % n_kv_heads == 0, n_q_heads/n_kv_heads   */
/* <= 8, page_size >= 1, seq_lens[b] <= max_pages * page_size.                  */
size_t qd_attn_workspace_bytes(int batch, int n_q_heads, int n_kv_heads, int max_ctx);
int qd_attn_decode_paged(const float* q, const void* k_pages, const void* v_pages,
                         const int32_t* page_table, const int32_t* seq_lens, int batch,
                         int n_q_heads, int n_kv_heads, int head_dim, int page_size,
                         int max_pages, int n_pages, float scale, float* out,
                         void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Allocation-free variant of qd_attn_decode_paged. (The pages describe no    */
/* such call; it exists for callers that cannot allocate device memory:       */
/* hosts whose device memory is reserved up front by their own pool, plugins  */
/* handed only input and output buffers, and latency-critical loops where     */
/* cudaMalloc/cudaFree would add an implicit device synchronisation.)          */
/* Same arguments, layouts and result as qd_attn_decode_paged, without the    */
/* workspace: the split-KV scratch is a static 8 MiB device array inside the  */
/* library, held by every GPU that loads it until the process exits. Shapes   */
/* whose workspace (qd_attn_workspace_bytes) exceeds 8 MiB are rejected with  */
/* QD_ERR_WORKSPACE. The call allocates nothing; it clears the scratch's      */
/* ticket counters with cudaMemsetAsync on `stream` before the launch. The    */
/* first call on each device looks up the array's device address            */
/* (cudaGetSymbolAddress) with that device current; make that first call     */
/* before any stream capture. All calls share the one array, which keeps the  */
/* last call's contents: calls that overlap on the GPU (for example on two     */
/* streams) race on it and must be serialised by the caller.                 */
int qd_attn_decode_paged_noalloc(const float* q, const void* k_pages, const void* v_pages,
                                 const int32_t* page_table, const int32_t* seq_lens, int batch,
                                 int n_q_heads, int n_kv_heads, int head_dim, int page_size,
                                 int max_pages, int n_pages, float scale, float* out,
                                 cudaStream_t stream);

/* ------------------------------------------------------------------------ */
/* Attention over the packed rows of several prompts (the batched form of       */
/* qd_prefill's attention; [KL-FUN], [KL-PAGED]). Sequence b owns the rows        */
/* cu_rows[b] .. cu_rows[b + 1) of q; its keys, the rows' own included, are        */
/* already in the cache, seq_lens[b] of them. Row j of its n rows is the token at  */
/* position seq_lens[b] - n + j and sees that position and all before:            */
/*   out[r, h, :] = sum_{t <= seq_lens[b] - n + j} softmax_t(scale * q[r,h,:].K_b[t,g,:]) */
/*                  * V_b[t, g, :],   g = h / (n_q_heads / n_kv_heads)               */
/* A row before position 0 (seq_lens[b] < n) sees nothing and gives 0 (a row that    */
/* sees keys whose scores are all -inf gives NaN, as its softmax does). Rows of q  */
/* outside every sequence have no effect, and out is left as it was there.        */
/* q: [n_rows, n_q_heads, head_dim], q_stride elements from one row to the next    */
/* (>= n_q_heads * head_dim, a multiple of 16 bytes: q may be part of the QKV       */
/* projection's rows); q_is_f32 = 1: q and out f32 (q and the softmax weights       */
/* enter the bf16 matrix products in three parts, 24 bits), 0: both bf16 (the weights  */
/* rounded to bf16, sums and softmax statistics in f32). out: [n_rows, n_q_heads,   */
/* head_dim], contiguous, apart from q. Caches and page_table as in qd_attn_decode_paged; */
/* cu_rows: int32 [batch + 1], ascending from >= 0 to <= n_rows; seq_lens: int32      */
/* [batch] (both device). Keys a row does not see have no effect on it, NaN and       */
/* infinities included. Errors on the device (QD_DEVERR_POS: cu_rows not ascending     */
/* or past n_rows, which leaves all of out; a length past the table, which leaves the   */
/* sequence's rows). A NaN that a row sees reaches it, however small its weight; an infinity in V  */
/* gives that infinity, one in K a score of it (q_is_f32 = 1: NaN, since q enters in parts).        */
/* workspace: device scratch of qd_attn_prompt_workspace_bytes() bytes for the current device,          */
/* its first QD_ATTN_WORKSPACE_HEAD bytes zero-filled before its first use (each call leaves it         */
/* ready for the next, but for one that ends with QD_DEVERR_TIMEOUT: zero-fill it again);   */
/* two calls that overlap on the GPU need two.                                              */
/* Limits: head_dim == 128, n_q_heads / n_kv_heads in {1, 2, 4, 8}, batch <= 1024,      */
/* n_rows <= 2^20; the blocks of 128 q rows (a row and a q head of one kv head) by 128 keys   */
/* that the call computes fewer than 2^31 (else QD_DEVERR_POS, and out is left as it was).    */
#define QD_ATTN_WORKSPACE_HEAD 8192
size_t qd_attn_prompt_workspace_bytes(void);
int qd_attn_prompt(const void* q, int q_is_f32, int64_t q_stride, const void* k_pages, const void* v_pages,
                   const int32_t* page_table, const int32_t* cu_rows, const int32_t* seq_lens, int batch,
                   int n_rows, int n_q_heads, int n_kv_heads, int head_dim, int page_size, int max_pages,
                   int n_pages, float scale, void* out, void* workspace, size_t workspace_bytes,
                   cudaStream_t stream);

/* Attention of packed rows over a window: qd_attn_prompt in which the row at token p sees the     */
/* tokens t <= p with t > p - window or t < n_sinks (the first tokens of the cache stay visible);    */
/* a page of which no row of the sequence sees a token is not read, and its entry in page_table may  */
/* name none. window >= 1 (2147483647: every token), n_sinks >= 0, else QD_ERR_INVALID_ARG; both may   */
/* hide nothing. The other arguments, limits, errors and the workspace (which serves either call)       */
/* are qd_attn_prompt's; so is what a row before position 0 gives, and a row that sees NaN or            */
/* infinities.                                                                                          */
int qd_attn_prompt_window(const void* q, int q_is_f32, int64_t q_stride, const void* k_pages, const void* v_pages,
                          const int32_t* page_table, const int32_t* cu_rows, const int32_t* seq_lens, int batch,
                          int n_rows, int n_q_heads, int n_kv_heads, int head_dim, int page_size, int max_pages,
                          int n_pages, float scale, int window, int n_sinks, void* out, void* workspace,
                          size_t workspace_bytes, cudaStream_t stream);

/* Decode attention of sequences that share prefixes: the result of qd_attn_decode_paged for      */
/* sequences whose page tables name the same pages at their start (qd_pages_fork), each shared     */
/* page read once for all of them. Where that would spare less than 80 MB of re-reading in the     */
/* whole call, over all groups (QD_SHARED_MIN_MB, read at every call, sets another limit; 0:       */
/* always share), each sequence reads its own table's pages, which is then faster.                 */
/* Group i holds the sequences cu_seqs[i] .. cu_seqs[i + 1); their first shared_lens[i] tokens     */
/* lie in the pages of the group's first sequence's row (a sequence shorter than that sees its     */
/* own seq_lens tokens of them). Sequences outside every group are left as they were.              */
/* shared_lens[i] may be 0 and need not be a multiple of page_size. Arguments as in                */
/* qd_attn_prompt with one row per sequence: q, out [batch, n_q_heads, head_dim]; page_table       */
/* [batch, max_pages], seq_lens [batch]; cu_seqs: int32 [n_groups + 1], ascending; shared_lens:    */
/* int32 [n_groups] (both device). seq_lens[b] == 0 gives out = 0.                                 */
/* A visible NaN reaches the row, as in qd_attn_prompt; so does an infinity in V, or NaN in its    */
/* place; one in K gives a score of it (q_is_f32 = 1: NaN, since q enters in parts). After an      */
/* error that leaves rows unwritten in qd_attn_prompt, out is undefined there.                     */
/* workspace: qd_attn_shared_workspace_bytes(...) bytes for the current device, its head           */
/* zero-filled before its first use, as in qd_attn_prompt (whose calls it can serve as well).      */
/* Limits: as qd_attn_prompt, n_groups <= 1024, batch <= 65535.                                 */
size_t qd_attn_shared_workspace_bytes(int batch, int n_q_heads, int n_kv_heads);
int qd_attn_decode_shared(const void* q, int q_is_f32, int64_t q_stride, const void* k_pages, const void* v_pages,
                          const int32_t* page_table, const int32_t* seq_lens, const int32_t* cu_seqs,
                          const int32_t* shared_lens, int n_groups, int batch, int n_q_heads, int n_kv_heads,
                          int head_dim, int page_size, int max_pages, int n_pages, float scale, void* out,
                          void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Decode attention over a window: the row of sequence b, at token p = seq_lens[b] - 1, sees the    */
/* tokens t <= p with t > p - window or t < n_sinks (the first tokens of the cache stay visible);      */
/* nothing else is read, NaN included. window >= 1 (2147483647: every token), n_sinks >= 0. q and out    */
/* [batch, n_q_heads, head_dim], the other arguments, limits and errors as in qd_attn_decode_shared       */
/* (q_is_f32 = 0: the softmax weights enter the products in two bf16 parts). seq_lens[b] == 0 gives out    */
/* = 0; a length past the table sets QD_DEVERR_POS and leaves the sequence as it was.                      */
/* key_weights: f32 [batch, n_kv_heads, max_pages * page_size], or NULL. To key_weights[b, g, t] of each     */
/* visible token t is added its softmax weight, summed over the q heads of kv head g: attention that keys     */
/* have drawn, which qd_pages_evict goes by. Deterministic. A visible NaN makes all of its row's weights NaN.   */
/* workspace: qd_attn_decode_window_workspace_bytes(batch, heads, max_keys) bytes, max_keys = min(window +        */
/* n_sinks, max_pages * page_size) with key_weights and 0 without (more is fine); its first                       */
/* QD_ATTN_WINDOW_HEAD bytes zero-filled before its first use, each call leaves them zero; two calls that           */
/* overlap on the GPU need two.                                                                                    */
#define QD_ATTN_WINDOW_HEAD 16384
size_t qd_attn_decode_window_workspace_bytes(int batch, int n_q_heads, int n_kv_heads, int64_t max_keys);
int qd_attn_decode_window(const void* q, int q_is_f32, int64_t q_stride, const void* k_pages, const void* v_pages,
                          const int32_t* page_table, const int32_t* seq_lens, int batch, int n_q_heads,
                          int n_kv_heads, int head_dim, int page_size, int max_pages, int n_pages, float scale,
                          int window, int n_sinks, float* key_weights, void* out, void* workspace,
                          size_t workspace_bytes, cudaStream_t stream);

/* The attention that packed rows give to each key: to key_weights[b, g, t] (f32 [batch, n_kv_heads,    */
/* max_pages * page_size]) is added the softmax weight of token t, summed over the last `last` rows of    */
/* sequence b (0: all of its rows) and the q heads of kv head g. Rows, windows, limits and errors as in     */
/* qd_attn_prompt_window, whose rows' attention it is (q and cache as there, V not needed); q_is_f32 = 1:     */
/* q enters the products in three bf16 parts. Deterministic. A visible NaN makes all of its row's weights     */
/* NaN; keys that no counted row sees keep their sums. workspace: qd_attn_key_weights_workspace_bytes(...)      */
/* bytes, which serve either type of q (..._for: of one type; a bf16 q needs about a third: q's row tiles in one     */
/* part instead of three), its first QD_ATTN_WEIGHTS_HEAD bytes zero-filled                                         */
/* before its first use (each call leaves them zero, but for one that ends with QD_DEVERR_TIMEOUT: zero-fill       */
/* them again); two calls that overlap on the GPU need two.                                                        */
#define QD_ATTN_WEIGHTS_HEAD 16384
size_t qd_attn_key_weights_workspace_bytes(int batch, int n_rows, int n_q_heads, int n_kv_heads, int last);
size_t qd_attn_key_weights_workspace_bytes_for(int q_is_f32, int batch, int n_rows, int n_q_heads, int n_kv_heads,
                                               int last);
int qd_attn_key_weights(const void* q, int q_is_f32, int64_t q_stride, const void* k_pages, const int32_t* page_table,
                        const int32_t* cu_rows, const int32_t* seq_lens, int batch, int n_rows, int n_q_heads,
                        int n_kv_heads, int head_dim, int page_size, int max_pages, int n_pages, float scale, int last,
                        int window, int n_sinks, float* key_weights, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream);

/* ------------------------------------------------------------------------ */
/* Packed rows into the cache: what stands between the QKV projection of several sequences'   */
/* rows and the attention over them. Row r is [n_q_heads; n_kv_heads; n_kv_heads] heads of 128  */
/* (q, k, v as in w_qkv). Each q and k head is normed and rotated,                              */
/*   y = w * x / sqrt(mean(x^2) + eps),  y'[i] = y[i] c_i - y[i + 64] s_i,                      */
/*   y'[i + 64] = y[i + 64] c_i + y[i] s_i,  (c_i, s_i) = rope_table[positions[axes[i], r], i], i < 64; */
/* q goes to q_out, k and v in bf16 to the row's cache slot: row j of sequence b's n rows          */
/* (cu_rows, as in qd_attn_prompt) at token seq_lens[b] - n + j. cast_bf16 = 1 rounds to bf16 after    */
/* the division and after the weight too, as the decode step and qd_prefill of a BF16 model do.        */
/* qkv: f32 (qkv_is_f32 = 1) or bf16, rows qkv_stride elements apart (a multiple of 16 bytes);         */
/* q_norm, k_norm: bf16 [128]; rope_table: f32 [rope_max_pos, 64, 2] (qd_rope_table_init);               */
/* positions: int32 [n_axes, n_rows] (device), or NULL: each row's cache slot; axes: HOST uint8 [64], the  */
/* position axis of each frequency (time, height, width of image tokens, in sections or in any other      */
/* order), NULL where n_axes is 1; q_out: f32 or bf16 [n_rows, n_q_heads, 128], apart from qkv; pages,       */
/* page_table, seq_lens as in qd_attn_prompt, the pages of all rows in the table.                            */
/* Rows outside every sequence are left as they were. A row whose slot or position lies outside the            */
/* cache or the table is left too and sets QD_DEVERR_POS; one whose page does not exist gives q alone and       */
/* sets QD_DEVERR_PAGE. cu_rows not ascending or past n_rows: QD_DEVERR_POS, and which rows are written is          */
/* undefined. Needs no workspace. Limits: head_dim == 128, batch, heads <= 1024, n_rows <= 2^20, n_axes <= 4.        */
int qd_qk_norm_rope(const void* qkv, int qkv_is_f32, int64_t qkv_stride, const void* q_norm, const void* k_norm,
                    float eps, int cast_bf16, const float* rope_table, int rope_max_pos, const int32_t* positions,
                    int n_axes, const uint8_t* axes, const int32_t* page_table, const int32_t* cu_rows,
                    const int32_t* seq_lens, int batch, int n_rows, int n_q_heads, int n_kv_heads, int head_dim,
                    int page_size, int max_pages, int n_pages, void* q_out, int out_is_f32, void* k_pages,
                    void* v_pages, cudaStream_t stream);

/* ------------------------------------------------------------------------ */
/* Page operations on the K/V cache ([KL-PAGED]: fixed physical pages behind a      */
/* page table). The state is in device memory, owned by the caller:                 */
/*   page_table int32 [max_seqs, max_pages]: the pages of each sequence in order,     */
/*     -1 past its last;  seq_lens int32 [max_seqs]: its tokens;                        */
/*   refs int32 [n_pages]: how many page-table entries name the page (0: free).          */
/* New pages are the lowest free ids, taken in sequence order, so a call's result           */
/* follows from its arguments alone. A call that cannot be carried out whole changes         */
/* nothing and sets QD_DEVERR_CACHE. A table entry within a sequence's length that names no      */
/* page of the cache (the state is broken) sets QD_DEVERR_PAGE where a call meets it: qd_pages_fork  */
/* copies it as it is, qd_pages_trim drops it, qd_pages_compact leaves it, and each does the rest;     */
/* qd_pages_extend, whose tokens would go to it, changes nothing.                                       */
/* k_cache, v_cache: host arrays of n_layers device pointers, each [n_pages,                  */
/* n_kv_heads, page_size, head_dim] bf16. workspace: qd_pages_workspace_bytes(cache)            */
/* bytes, zero-filled before its first use. 4-byte alignment for the int32 arrays.              */
/* Limits: head_dim % 8 == 0, max_seqs <= 2048, max_pages * page_size <= 2^30; n_pages <= 2^30     */
/* for all but qd_pages_copy.                                                                     */
typedef struct {
  void* const* k_cache;
  void* const* v_cache;
  int n_layers, n_kv_heads, page_size, head_dim, n_pages;
  int32_t* page_table;
  int32_t* seq_lens;
  int32_t* refs;
  int max_seqs, max_pages;
  void* workspace;
  size_t workspace_bytes;
} qd_page_cache;
size_t qd_pages_workspace_bytes(const qd_page_cache* cache);
/* K and V of page src[i] to page dst[i], i < n, in every layer (src, dst: int32 [n],     */
/* device). A pair with a negative id is skipped. No page may be a destination twice, or    */
/* both a source and a destination of different pairs (the contents of those pages would     */
/* depend on the order of the copies). Uses neither the state nor the workspace.              */
int qd_pages_copy(const qd_page_cache* cache, const int32_t* src, const int32_t* dst, int n, cudaStream_t stream);
/* Sequence children[i] becomes a copy of sequence parents[i] (as it was before the         */
/* call), i < n (int32 [n], device): the page-table row and the length; every page is        */
/* shared, the partly filled last one too (qd_pages_extend gives the writer its own).         */
/* Children must be empty (length 0) and named once, and not be their own parent.             */
int qd_pages_fork(const qd_page_cache* cache, const int32_t* parents, const int32_t* children, int n,
                  cudaStream_t stream);
/* Room for n_new[s] more tokens (int32 [max_seqs], device; <= 0: none): seq_lens[s] +=         */
/* n_new[s], new pages for them, and where the sequence's partly filled last page is shared       */
/* a copy of that page (of the sequences that are extended in one call, the last one in         */
/* sequence order keeps the page if nobody else names it). The tokens' K/V are the caller's    */
/* to write (the decode step, qd_prefill).                                                    */
int qd_pages_extend(const qd_page_cache* cache, const int32_t* n_new, cudaStream_t stream);
/* Sequence s cut to new_lens[s] tokens (int32 [max_seqs], device; negative or not below          */
/* its length: unchanged; 0 frees it): pages past the new length lose a reference.                 */
int qd_pages_trim(const qd_page_cache* cache, const int32_t* new_lens, cudaStream_t stream);
/* Moves the pages in use to the ids 0 .. n_live - 1 (those above go, in ascending order, to      */
/* the free ids below), with the page tables and counts; n_live: int32 [1], device.                */
int qd_pages_compact(const qd_page_cache* cache, int32_t* n_live, cudaStream_t stream);
/* Cuts sequence s to keep[s] tokens (int32 [max_seqs], device; negative or not below its length:   */
/* unchanged; 0 frees it), each layer and kv head choosing its own: the first n_sinks, the last      */
/* n_recent, and of those between the ones of the largest key_weights (the lower token first among     */
/* equals; NaN counts as -infinity), keep[s] in all (fewer of the last, then of the first, where       */
/* keep[s] is below their number). The kept tokens' K and V move down in their order to tokens 0 ..     */
/* keep[s] - 1, and so do their weights, past which zeros follow up to the old length; pages past the    */
/* new length lose a reference as in qd_pages_trim. A token's place is then no longer its position: new     */
/* ones are written with explicit positions (qd_qk_norm_rope).                                             */
/* key_weights: f32 [n_layers, max_seqs, n_kv_heads, max_pages * page_size], device (each layer's part        */
/* filled by qd_attn_decode_window and qd_attn_key_weights; they go by sequence and token, so the other page     */
/* calls leave them: after a trim or before a slot's next sequence zero the tokens behind its length, for a      */
/* fork copy the parent's). A page that may be written (one with a token between the first ones that stay         */
/* and the new length) and that others share (qd_pages_fork), or a length past the table, changes nothing and     */
/* sets QD_DEVERR_CACHE; so does a table entry that names no page (with QD_DEVERR_PAGE).                          */
/* Limits: head_dim <= 256, n_pages * n_kv_heads * page_size < 2^31.                                               */
int qd_pages_evict(const qd_page_cache* cache, float* key_weights, const int32_t* keep, int n_sinks, int n_recent,
                   cudaStream_t stream);

/* ------------------------------------------------------------------------ */
/* Greedy argmax + on-device advance ([KL-DEC] "LM-head GEMV + argmax +        */
/* token/position update"; [EQ-SPEED] item 2).                                  */
/* For each b < batch: t = lowest index of the maximum of logits[b, :vocab]     */
/* (NaN never wins; an all-NaN row gives 0 and sets QD_DEVERR_NAN);             */
/* out_tokens[b * max_steps + step[b]] = t (if step[b] < max_steps, else        */
/* QD_DEVERR_STEPS); tok[b] = t; pos[b] += 1; step[b] += 1.                      */
/* workspace: zero-filled scratch of qd_argmax_workspace_bytes(batch) bytes.    */
size_t qd_argmax_workspace_bytes(int batch);
int qd_argmax_advance(const float* logits, int vocab, int batch, int32_t* tok, int32_t* pos,
                      int32_t* step, int32_t* out_tokens, int max_steps, void* workspace,
                      size_t workspace_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------ */
/* RoPE cos/sin table ([CD-ROPE]): table[p, i] = (cos(p * f_i), sin(p * f_i)),  */
/* f_i = theta^(-2i/head_dim), i < head_dim/2, p < max_pos; angles evaluated in  */
/* binary64 on the device, stored as f32 pairs. table: f32 [max_pos, head_dim/2, 2]. */
int qd_rope_table_init(float* table, int max_pos, int head_dim, float theta, cudaStream_t stream);

/* ------------------------------------------------------------------------ */
/* Layers and the whole decode step.                                         */
typedef struct {
  int hidden, n_q_heads, n_kv_heads, head_dim, ffn;
  float rms_eps, rope_theta;
  qd_wtype wtype;
  qd_act act; /* Q8_0 models only */
} qd_layer_dims;

/* Row order ([EQ-SPEED] item 1): w_qkv = [q rows (Hq*D); k rows (Hkv*D);       */
/* v rows (Hkv*D)] x hidden; w_o = hidden x (Hq*D); w_gu = [gate rows (ffn);     */
/* up rows (ffn)] x hidden; w_down = hidden x ffn. BF16: bf16 matrices, s_* NULL. */
/* Q8_0: int8 matrices plus f16 scales [rows, cols/32]. INT4: packed matrices    */
/* [rows, cols/2] (as qd_gemv_w4) plus f16 scales [rows]. Norm weights: bf16.     */
typedef struct {
  const void *w_qkv, *w_o, *w_gu, *w_down;
  const void *s_qkv, *s_o, *s_gu, *s_down;
  const void *ln_in, *ln_post, *q_norm, *k_norm;
} qd_layer_weights;

typedef struct qd_layer qd_layer; /* opaque: dims + pointers, no tensor data */

/* Validates and records dims and pointers (host memory only; the weights stay */
/* owned by the caller and must outlive the handle).                          */
int qd_create_layer(const qd_layer_dims* dims, const qd_layer_weights* w, qd_layer** out);
int qd_destroy_layer(qd_layer* layer);

/* One decode token for `batch` sequences ([KL-DEC]):                          */
/*   res = embed[tok]; per layer: xn = RMSNorm(res; ln_in) (Qwen cast order);  */
/*   [q;k;v] = W_qkv xn; q,k = RoPE_pos(RMSNorm_head(q; q_norm / k; k_norm));    */
/*   K/V cache slot pos = (k, v) in bf16; o = GQA attention over slots 0..pos;  */
/*   res += W_o bf16(o); xn = RMSNorm(res; ln_post); [g;u] = W_gu xn;           */
/*   res += W_down bf16(silu(g) * u); then logits = W_lm RMSNorm(res; final_norm) */
/*   and argmax_advance (tok, pos, step, out_tokens updated on the device).     */
/* k_cache / v_cache: arrays (host memory) of n_layers device pointers, each    */
/* bf16 [n_pages, n_kv_heads, page_size, head_dim]. A contiguous cache is one   */
/* page of max_ctx tokens per sequence (page_size = max_ctx, page_table[b] = b). */
/* tok, pos, step: int32 [batch] device; out_tokens: int32 [batch, max_steps].   */
/* rope_table: from qd_rope_table_init with max_pos >= every position reached.  */
/* logits: f32 [batch, vocab] device output. workspace: device scratch of        */
/* qd_step_workspace_bytes(args) bytes, zero-filled before first use.           */
/* BF16 layers: batch 1 runs the ring GEMV path. Batch 2..8 with a bf16 LM head  */
/* and hidden, n_q_heads * head_dim, ffn multiples of 32 runs every projection   */
/* on the mma.sync weight-streaming GEMV (five launches per layer, RMSNorm and   */
/* SwiGLU fused). Batch 9..64 (and 3..8 with QD_SMALLB_IMPL=tc, from           */
/* QD_TC_MIN_BATCH, default 3) runs every projection as a tcgen05 GEMM over the  */
/* batch when those dims are multiples of 64; otherwise batch <= 8 runs the      */
/* CUDA-core GEMV path (batch 2: K <= 12288).                                    */
/* Q8_0 layers: batch 1 runs the                                                 */
/* Q8_0 GEMV lanes (act, lm_act); 2..64 runs the tcgen05 GEMMs with the weights  */
/* widened to bf16 as in qd_gemm_q8_0 (act and lm_act unused; dims % 256 == 0,   */
/* scales 16-byte aligned). INT4 layers: batch 1, the W4A16 GEMVs with bf16      */
/* activations (dims % 32 == 0, <= 16384).                                       */
/* LM head: lm_wtype QD_W_INT4 with lm_head_scales = the per-row f16 scales is an */
/* INT4 head (batch 1): its GEMV also picks the top_k tokens (0: only the argmax)  */
/* into topk_ids / topk_vals [top_k] and advances the step itself. Otherwise the  */
/* head is Q8_0 when lm_head_scales is set, else bf16, followed by argmax_advance. */
typedef struct {
  const qd_layer* const* layers;
  int n_layers;
  const void* embed;           /* bf16 [vocab, hidden] */
  const void* final_norm;      /* bf16 [hidden] */
  const void* lm_head;         /* bf16 [vocab, hidden], or int8 for a Q8_0 head */
  const void* lm_head_scales;  /* f16 [vocab, hidden/32] for a Q8_0 head, else NULL */
  qd_act lm_act;               /* Q8_0 head lane */
  int vocab;
  void* const* k_cache;
  void* const* v_cache;
  const int32_t* page_table;
  int page_size, max_pages, n_pages;
  const float* rope_table;
  int rope_max_pos;
  int32_t *tok, *pos, *step, *out_tokens;
  int max_steps;
  int batch;
  float* logits;
  void* workspace;
  size_t workspace_bytes;
  qd_wtype lm_wtype;   /* QD_W_INT4 for an INT4 head (see above) */
  int top_k;           /* INT4 head: 0..16 tokens into topk_ids / topk_vals */
  int32_t* topk_ids;
  float* topk_vals;
} qd_step_args;

size_t qd_step_workspace_bytes(const qd_step_args* args);
int qd_decode_step(const qd_step_args* args, cudaStream_t stream);

/* Whole-step CUDA graph ([CD-GRAPH], [EQ-SPEED] item 2): captures
 * `steps_per_launch` consecutive qd_decode_step calls (the token and position
 * advance on the device, so replays need no host round trip) on `stream`, and
 * instantiates the graph. Capture happens on the calling thread; the args
 * (pointers and sizes) are frozen into the graph. qd_graph_launch replays it on
 * `stream`. qd_graph_create synchronises nothing but must not be called while
 * `stream` is already capturing. */
typedef struct qd_graph qd_graph;
int qd_graph_create(const qd_step_args* args, int steps_per_launch, cudaStream_t stream,
                    qd_graph** out);
int qd_graph_launch(qd_graph* g, cudaStream_t stream);
int qd_graph_destroy(qd_graph* g);

/* ------------------------------------------------------------------------ */
/* Speculative verify ("qwen3-8b-rtx4080-cutedsl" README, "Speculative          */
/* decoding": a draft proposes tokens and the target model checks k of them in  */
/* one forward pass that reuses the weight bytes already streamed). For the one */
/* sequence of `args` (batch 1): the k input tokens are tok[0] (the last token   */
/* emitted) and draft[0 .. k-2], at positions pos[0] .. pos[0] + k - 1. They run  */
/* as k rows of one pass: every projection streams its weights once for the k   */
/* rows (bf16: the mma.sync GEMV when the dims are multiples of 32; Q8_0, or     */
/* QD_SMALLB_IMPL=tc: tcgen05 GEMMs); the                                        */
/* k new K/V rows are written to the cache first, and row i attends to positions */
/* 0 .. pos[0] + i (causal among the drafted tokens).                           */
/* Outputs: logits f32 [k, vocab] (device, 16-byte aligned); target int32 [k]:   */
/* the argmax of each row (the model's token after input i, as in               */
/* qd_argmax_advance); n_accept int32 [1]: m = the number of leading drafts with  */
/* draft[i] == target[i] (0 <= m <= k - 1). The state advances on the device:     */
/* out_tokens[step .. step + m] = draft[0 .. m - 1], target[m]; tok = target[m];  */
/* pos += m + 1; step += m + 1. Cache rows past pos[0] + m hold the rejected      */
/* drafts' K/V until a later step overwrites them.                               */
/* draft: int32 [k - 1] device (may be NULL when k == 1). 1 <= k <= 8. The       */
/* projections' K must be multiples of 32 (bf16 on the mma.sync GEMV), 64 (bf16 */
/* on tcgen05) or 256 (Q8_0, whose weights are                                   */
/* widened on chip as in qd_gemm_q8_0). workspace: args->workspace of at least    */
/* qd_verify_workspace_bytes(args, k) bytes, zero-filled before first use; the   */
/* pass's scratch follows the first qd_step_workspace_bytes(args) bytes (the      */
/* decode step's, left untouched), so passes and decode steps may alternate.     */
size_t qd_verify_workspace_bytes(const qd_step_args* args, int k);
int qd_verify_step(const qd_step_args* args, const int32_t* draft, int k, float* logits, int32_t* target,
                   int32_t* n_accept, cudaStream_t stream);

/* Sampled verification of drafted tokens, beside qd_verify_step's greedy rule, for a    */
/* batch: sequence b has n = n_draft[b] drafts (n_draft NULL: k - 1 each) draft[b, i]     */
/* drawn from draft_probs[b, i, :]; target_probs[b, i, :] is the target's distribution     */
/* after draft i - 1. Draft i is accepted while                                             */
/*   u[b, i] * draft_probs[b, i, draft[b, i]] < target_probs[b, i, draft[b, i]];             */
/* with m accepted, the next token t is the least index whose running sum of r passes         */
/* u[b, k - 1] times the sum of r, r = max(target_probs[b, m, :] - draft_probs[b, m, :], 0)    */
/* if m < n (target_probs[b, m, :] if that is zero everywhere), r = target_probs[b, n, :] if    */
/* m == n. Entries of r that are not finite count as 0; a row without mass gives 0 and sets       */
/* QD_DEVERR_NAN; a draft outside the vocabulary is rejected; n_draft outside 0 .. k - 1 is        */
/* clamped and sets QD_DEVERR_POS. The border is met to 2^-39 of the sum (2^-43      */
/* measured). The state advances as in                                                             */
/* qd_verify_step: n_accept[b] = m; out_tokens[b, step ..] = the m drafts, t; tok = t;               */
/* pos += m + 1; step += m + 1 (past max_steps: QD_DEVERR_STEPS).                                    */
/* target_probs: f32, row (b, i) at (b * k + i) * target_stride; draft_probs: f32, row (b, i) at       */
/* (b * (k - 1) + i) * draft_stride (may be NULL with draft when k == 1); draft: int32 [batch,          */
/* k - 1]; u: f32 [batch, k] in [0, 1); n_accept: int32 [batch]; all device. workspace:                  */
/* qd_verify_sample_workspace_bytes(batch) bytes, the first 4 * batch of them zero-filled before its      */
/* first use (for calls of several sizes: of the largest batch). Limits:                                */
/* 1 <= k <= 1024, vocab <= 4194304, batch <= 65535.                                                     */
size_t qd_verify_sample_workspace_bytes(int batch);
int qd_verify_sample(const float* target_probs, int64_t target_stride, const float* draft_probs,
                     int64_t draft_stride, const int32_t* draft, const int32_t* n_draft, const float* u, int vocab,
                     int batch, int k, int32_t* tok, int32_t* pos, int32_t* step, int32_t* out_tokens,
                     int max_steps, int32_t* n_accept, void* workspace, size_t workspace_bytes,
                     cudaStream_t stream);

/* ------------------------------------------------------------------------ */
/* Prefill ("qwen3-8b-rtx4080-cutedsl" README, "Flash Attention 2" and           */
/* "Baseline tiled GEMM": the prompt is processed as one batch of rows with      */
/* tiled attention that never forms the full score matrix). For the one sequence */
/* of `args` (batch 1): tokens int32 [n_tokens] (device) sit at positions         */
/* pos[0] .. pos[0] + n_tokens - 1. Every layer runs over all rows at once: the   */
/* projections are tcgen05 GEMMs over 64- or 256-token tiles (Q8_0 weights above */
/* 128 rows widened to bf16 once per projection, bf16(f32(d) q), into the        */
/* workspace first), the rows' K/V are                                           */
/* written to the cache first, and row i attends causally to positions 0 ..       */
/* pos[0] + i (the keys already cached included) on tcgen05 (QD_PREFILL_ATTN=mma: */
/* the mma.sync kernel). The workspace includes a packed copy of the kv heads'    */
/* keys up to the cache capacity (and, for Q8_0 above 128 rows, the bf16 copy of */
/* the largest projection). The last row alone goes through the final            */
/* norm and the LM head: logits f32 [vocab] (device, 16-byte aligned). The state  */
/* then advances as one decode step from the last row: tok = argmax (first index */
/* among equal maxima), out_tokens[step] = tok, pos += n_tokens, step += 1.      */
/* Position errors (pos[0] + n_tokens past the cache or the RoPE table) set      */
/* QD_DEVERR_POS. 1 <= n_tokens <= 32768; BF16 or Q8_0 weights (K multiples of 64 */
/* or 256 as in qd_verify_step). workspace: args->workspace of at least           */
/* qd_prefill_workspace_bytes(args, n_tokens) bytes, zero-filled before first use; */
/* as in qd_verify_step, the decode step's part of it is left untouched.          */
size_t qd_prefill_workspace_bytes(const qd_step_args* args, int n_tokens);
int qd_prefill(const qd_step_args* args, const int32_t* tokens, int n_tokens, float* logits, cudaStream_t stream);

/* Reads and clears the sticky device error word (synchronises `stream`).      */
/* *bits receives a mask of QD_DEVERR_*. Returns QD_OK or QD_ERR_CUDA.           */
int qd_check_device_error(cudaStream_t stream, int* bits);

/* Number of kernel launches one qd_decode_step call issues for these args.    */
int qd_step_launch_count(const qd_step_args* args);

/* ------------------------------------------------------------------------ */
/* Test-only exports (make the bit-exactness claims directly checkable).      */
/* qd_debug_q8_block_dots runs the production Q8_0 GEMV of the i8 lane          */
/* (qd_gemv_q8_0 with act = QD_ACT_I8 and x_q, x_d given: the same dispatch and  */
/* kernels as the decode step's Q8_0 GEMVs) in a form that also stores each      */
/* int32 block dot it forms: dots[r, b] = sum_i qs[r, 32b+i] * x_q[32b+i],        */
/* int32 [rows, cols/32]; y: f32 [rows], the GEMV result.                        */
int qd_debug_q8_block_dots(const int8_t* qs, const void* d_f16, int rows, int cols, const int8_t* x_q,
                           const void* x_d_f16, int32_t* dots, float* y, cudaStream_t stream);
/* idx[b, t] = page_table[b*max_pages + t/page_size]*page_size + t%page_size for */
/* t < n_tokens: the physical token slot the attention kernels read, through    */
/* the same device function they use. A page id outside [0, n_pages) gives      */
/* idx = -1 and sets QD_DEVERR_PAGE (the attention kernels read page 0 there).  */
int qd_debug_paged_indices(const int32_t* page_table, int batch, int max_pages,
                           int page_size, int n_pages, int n_tokens, int32_t* idx,
                           cudaStream_t stream);
/* The timeout path of the kernels' bounded waits: one thread arms an mbarrier   */
/* for bytes no copy will deliver (none is issued) and waits on it for limit_us  */
/* microseconds (1 .. 1000000); the wait gives up, sets QD_DEVERR_TIMEOUT and the */
/* kernel returns, leaving the context usable. Asynchronous on `stream`.          */
int qd_debug_wait_timeout(int limit_us, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* QD_H */
