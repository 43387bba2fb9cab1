/*
 * attn_gb300.h -- C ABI of the GB300 (sm_103a) IO-aware attention forward library.
 *
 * The operation is scaled dot-product attention, O = softmax(scale * Q K^T) V, computed row by
 * row over the keys each query may see, together with the per-row log-sum-exp of the scaled
 * scores (CS336 Lecture 5 notes, section 6.1 for the definition; section 6.2 for the fused,
 * tiled, online-softmax forward that never writes the score matrix to HBM and keeps only m and l
 * "merged into a logsumexp"; CS336 GPU/attention notes, "Online softmax 回顾", for the merge).
 *
 * Conventions shared by every entry point:
 *   - All tensor pointers are DEVICE pointers owned by the caller.  No call allocates device
 *     memory (the fused kernel uses on-chip shared and tensor memory only; the unfused
 *     comparison path uses a caller-provided workspace).  The one piece of device memory the
 *     library holds is a file-scope array of ATTN_NOALLOC_SCRATCH_BYTES (64 MiB), the scratch of
 *     attn_fwd_unfused_noalloc, which every GPU that loads the library keeps until exit.
 *   - Element types: q, k, v, o are bfloat16 (passed as void*); lse is float32;
 *     cu_seqlens is int32.
 *   - Dense layout (cu_seqlens == NULL): q, k, v, o are [B, H, N, d] contiguous, d innermost;
 *     lse is [B, H, N].
 *   - Packed variable-length layout (cu_seqlens != NULL): B is the number of sequences and N is
 *     the total token count T = cu_seqlens[B] (passed by the host, which never reads device
 *     memory); q, k, v, o are [H, T, d] and lse is [H, T].  Sequence s owns rows
 *     cu_seqlens[s] .. cu_seqlens[s+1]-1 of every head and attends only to itself.
 *     cu_seqlens must be non-decreasing with cu_seqlens[0] = 0 and cu_seqlens[B] = N; a
 *     violation is the caller's error and gives undefined output (never an out-of-bounds write
 *     outside [0, N) rows of o and lse).  Zero-length sequences are allowed and write nothing.
 *   - causal != 0 keeps key j for query i iff j <= i, positions counted from the start of each
 *     sequence.
 *   - scale multiplies the scores before the softmax (1/sqrt(d) for the usual attention); it must
 *     be finite and > 0.  lse is the natural-log log-sum-exp of the scaled scores.
 *   - d must be 64 or 128.  Pointers must be 16-byte aligned.
 *   - B, H, N >= 0; if any of them is 0 there is nothing to compute and the call returns
 *     ATTN_OK without touching the pointers.
 *   - Work is enqueued on `stream` (a cudaStream_t, 0 = legacy default stream) and runs
 *     asynchronously.  The return value covers host-side validation and the launch; a device-side
 *     failure (a pipeline wait that timed out) is reported by attn_get_last_device_error().
 *   - On any non-zero return the contents of o and lse are unspecified.
 *   - Entry points are thread-safe as long as concurrent calls use different output buffers.
 */
#ifndef ATTN_GB300_H
#define ATTN_GB300_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define ATTN_API __attribute__((visibility("default")))
#else
#define ATTN_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ATTN_OK = 0,
  ATTN_ERR_NULL = -1,        /* a required pointer is NULL                                  */
  ATTN_ERR_HEAD_DIM = -2,    /* d is not 64 or 128                                          */
  ATTN_ERR_SHAPE = -3,       /* a negative size, or sizes whose products overflow the kernel */
  ATTN_ERR_ALIGN = -4,       /* a tensor pointer is not 16-byte aligned                     */
  ATTN_ERR_LAUNCH = -5,      /* a CUDA call failed while preparing or launching the kernel  */
  ATTN_ERR_DEVICE = -6,      /* the current device is not an sm_103 (GB300-class) GPU       */
  ATTN_ERR_SCALE = -7,       /* scale is not finite or not > 0                              */
  ATTN_ERR_WORKSPACE = -8,   /* workspace NULL, unaligned or smaller than required          */
  ATTN_ERR_UNSUPPORTED = -9, /* an argument combination this entry point does not support   */
  ATTN_ERR_SCRATCH_LIMIT = -10 /* the problem needs more than the built-in scratch (no-alloc) */
} attn_status;

/*
 * Fused forward (the hot path).  One kernel launch: each CTA keeps a 128-row tile of Q on chip,
 * streams 128-row tiles of K and V through TMA-fed shared memory, computes S = Q K^T with tcgen05
 * tensor-core MMAs into tensor memory, applies the online softmax (running row max m and sum l,
 * exp2 of log2(e)-prescaled scores, rescaling of the O accumulator) and accumulates P V on the
 * tensor cores, then writes O = acc / l in bf16 and lse = m + ln l in fp32.  The N x N score
 * matrix never reaches HBM; causal tiles above the diagonal are skipped.
 *   q, k, v : bf16 inputs (read only)          o   : bf16 output, same layout as q
 *   lse     : fp32 output                      cu_seqlens : NULL (dense) or int32[B+1] (packed;
 *                                                           a prefix sum from 0 to N, else the
 *                                                           status word reports kind 2)
 *   B, H, N, d, causal, scale : as described above; stream : cudaStream_t
 * Returns an attn_status.
 */
ATTN_API int attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
             const int32_t* cu_seqlens, int B, int H, int N, int d, int causal, float scale,
             void* stream);

/*
 * Grouped-query / multi-query forward (CS336 Lecture 5 notes, section 6.3: several query heads
 * share one K/V head).  As attn_fwd, except that k and v have H_kv heads and query head h reads
 * K/V head h / (H / H_kv):
 *   dense : q, o [B, H, N, d]; k, v [B, H_kv, N, d]; lse [B, H, N]
 *   packed: q, o [H, T, d];    k, v [H_kv, T, d];    lse [H, T]
 * H_kv must divide H (H_kv = H is attn_fwd; H_kv = 1 is multi-query attention), else
 * ATTN_ERR_SHAPE.  Returns an attn_status.
 */
ATTN_API int attn_fwd_gqa(const void* q, const void* k, const void* v, void* o, float* lse,
                          const int32_t* cu_seqlens, int B, int H, int H_kv, int N, int d,
                          int causal, float scale, void* stream);

/*
 * Split-KV forward for problems with few query tiles (small B * H): the key/value sequence of
 * every pair of query tiles is cut into num_splits contiguous slices, each computed by its own
 * CTA (head dim 64) or cluster of two CTAs (head dim 128), so that more SMs share the work (sequence-dimension parallelism, CS336 Lecture 5 notes, section 6.3).
 * Each slice leaves its unnormalised output, its reference row maximum and its row sums in
 * `workspace`; a second kernel on `stream` merges the slices with the block merge of the CS336
 * GPU/attention notes, "Online softmax 回顾" (M = max of the slice maxima, each slice weighted by
 * exp(m_s - M), O = sum of weighted outputs / sum of weighted sums, lse = M + ln(weighted sum)).
 * Dense layout only: q, k, v, o [B, H, N, d] bf16, lse [B, H, N] fp32, as attn_fwd.
 *   num_splits : slices per query pair, at most 32 and at most the number of 128-key tiles
 *                (larger values are lowered).  <= 0 lets the library choose: the count that
 *                minimises (waves of units) x (key tiles per slice + 2), the smallest on ties,
 *                where a wave is 152 units at d = 64 and 76 (two SMs each) at d = 128.
 *                When the count is 1 this is attn_fwd and the workspace is not touched.
 *   workspace  : caller-owned device buffer of at least
 *                attn_fwd_splitkv_workspace_bytes(B, H, N, d, num_splits) bytes, 256-byte
 *                aligned, else ATTN_ERR_WORKSPACE; its contents on return are unspecified.
 * Returns an attn_status (argument checks as attn_fwd).
 */
ATTN_API int attn_fwd_splitkv(const void* q, const void* k, const void* v, void* o, float* lse,
                              int B, int H, int N, int d, int causal, float scale, int num_splits,
                              void* workspace, size_t workspace_bytes, void* stream);

/*
 * The slice count attn_fwd_splitkv uses for these sizes and num_splits (0 for invalid sizes or
 * a head dim other than 64 and 128).
 */
ATTN_API int attn_fwd_splitkv_slices(int B, int H, int N, int d, int num_splits);

/*
 * Workspace bytes attn_fwd_splitkv needs: with S the slice count it will use, an fp32 partial
 * output [S][B*H*N][d] followed by two fp32 planes [2][S][B*H*N] (slice max in log2 units, the
 * row sum), each region rounded up to 256 bytes.
 * Returns 0 when S is 1 (no workspace needed) or the sizes are invalid.
 */
ATTN_API size_t attn_fwd_splitkv_workspace_bytes(int B, int H, int N, int d, int num_splits);

/*
 * Backward pass (dQ, dK, dV) of the fused forward.  Nothing N x N is read or kept: S and P are
 * rebuilt tile by tile from the logsumexp the forward saved (CS336 Lecture 5 notes, section 6.2,
 * "反向传播怎么办"), and the gradients follow from the definition by the chain rule:
 * dV = P^T dO, dP = dO V^T, dS = P * (dP - D) with D_i = dO_i . O_i, dQ = scale dS K,
 * dK = scale dS^T Q.  Two kernel launches on `stream`: a row pass (D and lse * log2 e into the
 * workspace), then one grid whose first CTAs run the dK/dV pass (one CTA per 128-key tile) and
 * the rest the dQ pass (one CTA per 128-query tile); every output element is written once
 * (deterministic, no atomics).
 * Dense layout only:
 *   q, k, v, o, dout : bf16 [B, H, N, d] (o is the forward's output, dout the gradient of the loss
 *                      with respect to it)         lse : fp32 [B, H, N], the forward's lse output
 *   dq, dk, dv       : bf16 [B, H, N, d] outputs
 *   causal, scale    : as in the forward call that produced o and lse
 *   workspace        : caller-owned device buffer of at least attn_bwd_workspace_bytes(B,H,N,d)
 *                      bytes, 256-byte aligned; contents on return unspecified
 * Every tensor pointer must be 16-byte aligned (ATTN_ERR_ALIGN) and non-NULL (ATTN_ERR_NULL);
 * other checks as attn_fwd.  Returns an attn_status.
 */
ATTN_API int attn_bwd(const void* q, const void* k, const void* v, const void* o,
                      const float* lse, const void* dout, void* dq, void* dk, void* dv, int B,
                      int H, int N, int d, int causal, float scale, void* workspace,
                      size_t workspace_bytes, void* stream);

/*
 * Backward pass of grouped-query / multi-query attention (CS336 Lecture 5 notes, section 6.3):
 * as attn_bwd, except that k, v, dk and dv have H_kv heads ([B, H_kv, N, d]) and query head h
 * reads K/V head h / (H / H_kv).  A K/V head's gradients are the sums over the query heads that
 * share it: the dK/dV pass runs one CTA per (K/V head, key tile) that visits the query tiles of
 * all of them, so the sums accumulate in tensor memory and each element is still written once.
 * H_kv must divide H, else ATTN_ERR_SHAPE.  The workspace is attn_bwd_workspace_bytes(B,H,N,d).
 */
ATTN_API int attn_bwd_gqa(const void* q, const void* k, const void* v, const void* o,
                          const float* lse, const void* dout, void* dq, void* dk, void* dv,
                          int B, int H, int H_kv, int N, int d, int causal, float scale,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward pass on a packed batch of variable-length sequences (the layout of attn_fwd with
 * cu_seqlens): q, o, dout, dq [H, T, d]; k, v, dk, dv [H_kv, T, d]; lse [H, T]; cu_seqlens
 * int32[B + 1] on the device, B = number of sequences, T = total rows.  Sequences are independent;
 * grouped-query heads as attn_bwd_gqa (H_kv = H for multi-head).  The tile passes run one CTA per
 * (head, 128-row tile of a sequence), found by a scan of cu_seqlens; offsets are clamped into
 * [0, T].  workspace: attn_bwd_varlen_workspace_bytes(B, H, T, d) bytes, 256-byte aligned.
 * cu_seqlens NULL: ATTN_ERR_NULL.  Returns an attn_status.
 */
ATTN_API int attn_bwd_varlen(const void* q, const void* k, const void* v, const void* o,
                             const float* lse, const void* dout, void* dq, void* dk, void* dv,
                             const int32_t* cu_seqlens, int B, int H, int H_kv, int T, int d,
                             int causal, float scale, void* workspace, size_t workspace_bytes,
                             void* stream);

/*
 * Workspace bytes attn_bwd_varlen needs: two fp32 planes of H * 128 * (ceil(T/128) + B) rows,
 * each rounded up to 256 bytes.  Returns 0 for invalid sizes.
 */
ATTN_API size_t attn_bwd_varlen_workspace_bytes(int B, int H, int T, int d);

/*
 * Workspace bytes attn_bwd needs: two fp32 planes of B * H * Npad values (Npad = N rounded up to
 * 128), each rounded up to 256 bytes.  Returns 0 for invalid sizes.
 */
ATTN_API size_t attn_bwd_workspace_bytes(int B, int H, int N, int d);

/*
 * Per-tile E4M3 quantization (the FP8 format of CS336 Lecture 5 notes, section 3.1: 1 sign,
 * 4 exponent, 3 mantissa bits, largest magnitude 448; per-tile scaling).  For every tile of 128
 * rows of a head of the bf16 tensor x [B, H, N, d] (d = 64 or 128):
 *   scale = amax / 448 in fp32 (1 for an all-zero tile), written to scales[(b*H + h)*T + t]
 *   (T = ceil(N/128)); code = E4M3 round-to-nearest-even of x / scale rounded to nearest fp32
 *   (the IEEE quotient, which the kernel forms from the tile's reciprocal with one correction;
 *   attn_selftest_fp8_quotients checks every input), saturating at +-448, the sign bit kept for
 *   values that round to zero.
 *   transpose = 0: codes [B, H, N, d] (N*d bytes per head)
 *   transpose = 1: codes [B, H, d, Npad] with Npad = 128*T, padding codes 0 (the V operand of
 *                  attn_fwd_fp8)
 * x and codes must be 16-byte aligned, scales 4-byte aligned.  Returns an attn_status.
 */
ATTN_API int attn_quantize_fp8(const void* x, void* codes, float* scales, int B, int H, int N,
                               int d, int transpose, void* stream);

/*
 * FP8 fused forward (FlashAttention-3's FP8 path, CS336 Lecture 5 notes, section 6.3), head dim
 * 128, dense layout.  Inputs are E4M3 codes with per-tile fp32 scales as attn_quantize_fp8
 * writes them: q8, k8 [B, H, N, 128] (transpose = 0), vt8 [B, H, 128, Npad] (transpose = 1); the
 * value of an input element is code x its tile's scale.  S = Q K^T runs on kind::f8f6f4 tensor
 * cores; the probabilities enter P V as E4M3 codes of P * 48 * sv_j / max(sv) (V's tile scales
 * folded in; P <= 8 against a reference maximum that trails the row maximum by at most 3 in log2
 * units); O (bf16) and lse (fp32, natural log of the scaled scores' normaliser) as attn_fwd.
 * d other than 128: ATTN_ERR_HEAD_DIM.  Returns an attn_status.
 */
ATTN_API int attn_fwd_fp8(const void* q8, const float* sq, const void* k8, const float* sk,
                          const void* vt8, const float* sv, void* o, float* lse, int B, int H,
                          int N, int d, int causal, float scale, void* stream);

/*
 * A paged key-value cache (the paged cache of CS336 Lecture 5 notes, section 6.3).  K and V are each
 * num_pages pages of H_kv heads of page_size rows of d elements; row r of page p and K/V head h
 * starts at element p * page_stride + (h * page_size + r) * d.  A token's place is its slot,
 * page * page_size + row.  Passed by address; the struct itself is host memory, read during the call.
 *   k, v             : device pointers, 16-byte aligned; bf16, or E4M3 codes
 *   k_scale, v_scale : E4M3 only (else ignored): fp32 [num_pages, H_kv, page_size], contiguous,
 *                      16-byte aligned: the value of an element is its code x its row's scale (of
 *                      any size and sign; the rows of a request may differ in it by any factor)
 *   page_stride      : elements from one page to the next, of k and of v (>= H_kv * page_size * d;
 *                      a multiple of 16 bytes), so k and v may be interleaved page by page
 *   page_size        : 16, 32, 64, 128 or 256
 *   dtype            : ATTN_CACHE_BF16 or ATTN_CACHE_E4M3
 * A malformed cache is ATTN_ERR_SHAPE (sizes, strides), ATTN_ERR_NULL, ATTN_ERR_ALIGN or
 * ATTN_ERR_UNSUPPORTED (dtype, page_size).
 */
typedef struct {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int64_t page_stride;
  int32_t num_pages;
  int32_t page_size;
  int32_t dtype;
} attn_kv_cache;

#define ATTN_CACHE_BF16 0
#define ATTN_CACHE_E4M3 1

/*
 * Pages, slots and positions of the new tokens of B requests, from their lengths.  Request s holds
 * seq_lens[s] tokens and gets new tokens cu_new[s] .. cu_new[s+1]-1 of a packed batch of T; the
 * pages it lacks come from free_pages in order, request by request, starting at entry *free_head:
 *   had_s = ceil(len_s / P), need_s = ceil((len_s + new_s) / P) - had_s,
 *   page j of request s = block_table[s][j] for j < had_s, else
 *                         free_pages[*free_head + sum_{r<s} need_r + j - had_s];
 *   a token at position i of its request has slot page(i / P) * P + i % P.
 *   seq_lens int32[B]; cu_new int32[B+1] (0 to T); block_table int32[B, max_pages], whose new
 *   entries are written; free_pages int32[n_free]; free_head int32[1]
 *   slots int64[T], positions int32[T], seq_lens_out int32[B] (len + new), free_head_out int32[1]
 *   (*free_head + sum of need): outputs.  seq_lens_out and free_head_out must not be seq_lens and
 *   free_head (ATTN_ERR_UNSUPPORTED): every CTA reads the old values.  The call can be repeated
 *   with the same inputs.
 *   max_pages : row length of block_table; page_size : 1 to 65536; B <= 16384 (ATTN_ERR_SHAPE)
 * A token whose page would lie past max_pages, or past the free list, gets slot -1 (and its table
 * entry, if there is one, -1) and the status word reports kind 4; cu_new that is not a
 * non-decreasing prefix sum from 0 to T reports kind 2, is clamped into [0, T], and leaves tokens
 * that belong to no request with slot -1 and position 0.  A negative length counts as 0.
 * (Several new tokens of a request that holds tokens already get pages and slots too: attn_fwd_paged_varlen
 * attends for those.)
 * One launch.  T == 0 copies the lengths and the head; B == 0 does nothing.  Pointers of 4-byte
 * elements must be 4-byte aligned, slots 8-byte.  Returns an attn_status.
 */
ATTN_API int attn_kv_slots(const int32_t* seq_lens, const int32_t* cu_new, int32_t* block_table,
                           const int32_t* free_pages, const int32_t* free_head, int64_t* slots,
                           int32_t* positions, int32_t* seq_lens_out, int32_t* free_head_out,
                           int B, int T, int max_pages, int n_free, int page_size, void* stream);

/*
 * The step before attention: from the rows a projection wrote, token by token, to q, k, v head by
 * head, normed and rotated, and into a paged cache; one pass over the data.  A token's row holds H
 * query heads, H_kv key heads and H_kv value heads of d elements.  For a query or key head x:
 *   n = x * w / sqrt(mean(x^2) + eps)          (n = x where w is NULL)
 *   (y_a, y_b) = rope_scale * (n_a cos t - n_b sin t, n_b cos t + n_a sin t),
 *   t = position * inv_freq[i] for pair i of the first `rot` elements: elements i and i + rot/2, or
 *   2i and 2i + 1 if interleaved; elements from rot on stay n.  Value heads are copied.
 *   qkv       : bf16 [B, N, ld] rows, ld >= (H + 2 H_kv) d elements from one token to the next, a
 *               multiple of 8
 *   wq, wk    : bf16 [d] weights of the norms, each may be NULL (no norm); eps >= 0
 *   inv_freq  : float64 [rot/2], radians a position (any scaling for long contexts is in it);
 *               rot : a multiple of 16 up to d, 0 for no rotation (inv_freq may then be NULL)
 *   positions : int32 [B, N] (NULL only with rot 0).  The angle is reduced modulo a turn in 64-bit
 *               fixed point, so far positions keep fp32 accuracy
 *   q         : bf16 [B, H, N, d];  k, v : bf16 [B, H_kv, N, d], both or neither NULL.  With B = 1
 *               these are the packed layout [H, T, d] of attn_fwd; with N = 1 one new token of
 *               each of B requests, as attn_fwd_paged takes it.  q may be NULL.
 *   cache     : NULL, or the cache that token t's K and V rows go into at slots[t] (int64 [B, N];
 *               negative: not stored).  E4M3 rows: scale = amax / 448 (1 if that is below fp32's
 *               normal range, as for a zero row), code = E4M3 round-to-nearest-even of the fp32
 *               y / scale.  A slot past the cache is not stored and the status word reports kind 5.
 *               What two tokens with one slot leave there is unspecified.
 * Norm and rotation are fp32, rounded once on the way out.  Outputs must not overlap qkv.
 * One launch.  Tensors 16-byte aligned (inv_freq and slots 8, positions 4).  Returns an attn_status
 * (rot, ld, eps, rope_scale out of range: ATTN_ERR_SHAPE for sizes, ATTN_ERR_SCALE for the floats).
 */
ATTN_API int attn_qkv_rope(const void* qkv, int64_t ld, const void* wq, const void* wk, float eps,
                           const double* inv_freq, int rot, int interleaved, float rope_scale,
                           const int32_t* positions, void* q, void* k, void* v,
                           const attn_kv_cache* cache, const int64_t* slots, int B, int N, int H,
                           int H_kv, int d, void* stream);

/*
 * Backward of attn_qkv_rope without a cache.  With g = rope_scale * R(t)^T dy, r = 1/sqrt(mean(x^2)
 * + eps) and u = g w:  dx = r (u - x r^2 mean(u x)),  dw = sum over rows of g x r  (dx = g without a
 * norm);  dv is copied.
 *   dq bf16 [B, H, N, d]; dk, dv bf16 [B, H_kv, N, d]: gradients of q, k, v (as attn_bwd writes them)
 *   dqkv bf16 [B, N, ld_out] : gradient of qkv; columns past (H + 2 H_kv) d are left as they were
 *   dwq, dwk fp32 [d] : written where wq, wk are given (ignored where they are NULL)
 *   workspace : attn_qkv_rope_bwd_workspace_bytes(B, N, H, H_kv, d) bytes, 256-byte aligned, needed
 *               only with a norm (NULL is fine without)
 * Sums over rows are taken in a fixed order (no atomics): equal inputs give equal bits.
 * B * N == 0 writes nothing.  Other arguments and errors as attn_qkv_rope.
 */
ATTN_API int attn_qkv_rope_bwd(const void* dq, const void* dk, const void* dv, const void* qkv,
                               int64_t ld, const void* wq, const void* wk, float eps,
                               const double* inv_freq, int rot, int interleaved, float rope_scale,
                               const int32_t* positions, void* dqkv, int64_t ld_out, float* dwq,
                               float* dwk, int B, int N, int H, int H_kv, int d, void* workspace,
                               size_t workspace_bytes, void* stream);

/* Workspace bytes attn_qkv_rope_bwd needs (0 for invalid sizes). */
ATTN_API size_t attn_qkv_rope_bwd_workspace_bytes(int B, int N, int H, int H_kv, int d);

/*
 * Attention of one new token of each of B requests over a paged cache: for request s and query head
 * h, O = softmax(scale q K^T) V over the first seq_lens[s] rows of the pages block_table[s][0], [1],
 * ... of K/V head h / (H / H_kv), and the log-sum-exp.  (The new token's own K and V are in the
 * cache already, and counted.)
 *   q, o : bf16 [B, H, d] (= [B, H, 1, d]);  lse : fp32 [B, H]
 *   block_table : int32 [B, max_pages]; only the entries that seq_lens needs are read, and a row past
 *     seq_lens is never used, whatever it holds.  seq_lens : int32 [B], clamped to 0 ..
 *     max_pages * page_size.  A request of length 0 gets O = 0 and lse = -inf.
 *   workspace : attn_fwd_paged_workspace_bytes(B, H, H_kv, d) bytes (it does not depend on the
 *     lengths), 256-byte aligned; calls whose work may overlap on the GPU need one each.
 * The rows of all requests are cut into equal shares, one a CTA, whatever the lengths are, and a second
 * launch joins the parts of a request that fell to several CTAs by the block merge of
 * attn_fwd_splitkv.  Everything that depends on lengths is decided on the GPU: a captured call can be
 * replayed with other lengths, tables and contents.  Equal inputs give equal bits.
 * A table entry that is needed and names no page of the cache is read as a page of zeros, and the
 * status word reports kind 5.
 * H_kv must divide H, and B * H_kv * ceil(H / H_kv / 32) * (ceil(max_pages * page_size / 64) + 2), by the
 * tiles that the table's shape allows, must be below 2^31 (ATTN_ERR_SHAPE).  Returns an attn_status.
 */
ATTN_API int attn_fwd_paged(const void* q, const attn_kv_cache* cache, const int32_t* block_table,
                            const int32_t* seq_lens, void* o, float* lse, int B, int H, int H_kv,
                            int d, int max_pages, float scale, void* workspace,
                            size_t workspace_bytes, void* stream);

/* Workspace bytes attn_fwd_paged needs (0 for invalid sizes). */
ATTN_API size_t attn_fwd_paged_workspace_bytes(int B, int H, int H_kv, int d);

/*
 * Attention of several new tokens of each of B requests over a paged cache: a prompt in chunks, a second prompt of
 * a conversation, proposed tokens to verify, or a whole prompt through its pages.  Request s owns tokens
 * cu_new[s] .. cu_new[s+1]-1 of a packed batch of T, the last of the seq_lens[s] rows that its pages
 * block_table[s][0], [1], ... hold (the new tokens' own K and V are in the cache already, and counted).
 * Token i of n sees rows 0 .. seq_lens[s] - n + i of its request (causal), or all seq_lens[s] of them (causal = 0);
 * query head h reads K/V head h / (H / H_kv).  O = softmax(scale q K^T) V, and the log-sum-exp.
 *   q, o : bf16 [H, T, d];  lse : fp32 [H, T]  (the packed layout of attn_fwd and attn_qkv_rope)
 *   block_table : int32 [B, max_pages]; only the entries that seq_lens needs are read, and a row past seq_lens
 *     is never used, whatever it holds.  seq_lens : int32 [B], clamped to 0 .. max_pages * page_size.
 *   cu_new : int32 [B + 1], from 0 up, at most T.  Requests without new tokens are fine; tokens from cu_new[B]
 *     on are padding, and o and lse are left as they were there.  cu_new that does not begin with 0 or passes T is
 *     clamped into [0, T] and the status word reports kind 2 (o and lse are then unspecified); with one that
 *     decreases nothing is computed, with the same report.
 *   A token that sees no row (more new tokens than rows) gets O = 0 and lse = -inf.
 *   E4M3 caches: K scales of at most 2^100 in magnitude, V scales of 2^-100 to 2^100, or 0 (attn_fwd_paged takes any of
 *     either; these are the limits of the kernel for many rows, see below, which takes a query row as two E4M3 pieces:
 *     elements under 2^-9 of its largest are off by up to 2^-17 of that); a query row with an infinity or a NaN gives NaN.
 *   A V row that is not finite may reach, besides the tokens that see it, the other new tokens of its request, in the columns
 *     where it is not finite: keys that a token does not see have the weight 0, and 0 x inf is NaN, as where S is masked
 *     before a plain softmax(S) V.  It reaches no other request.  (A K row reaches only the tokens that see it.)
 *   workspace : attn_fwd_paged_varlen_workspace_bytes(T, H, H_kv, d) bytes (it does not depend on the
 *     lengths), 256-byte aligned; calls whose work may overlap on the GPU need one each.
 * Requests with up to 32 query rows a K/V head (new tokens times H / H_kv; 64 over E4M3 pages) are taken by a kernel that works as
 * attn_fwd_paged does, those with more by one whose products take 256 rows at once.  Each cuts its work into equal
 * shares of key tiles, whatever the lengths are, and a second launch joins what fell to several shares by the block
 * merge of attn_fwd_splitkv: one to four launches, by B, T and the table's shape alone (with so many rows in all, only the
 * first kernel's; with over 64 a request on average, or one request of more, only the second's).  Everything that
 * depends on lengths is decided on the GPU: a captured call can be replayed with other lengths, tables and contents.
 * Equal inputs give equal bits.  A table entry that is needed and names no page of the cache is read as a page of
 * zeros, and the status word reports kind 5.
 * H_kv must divide H; B, max_pages * page_size and T are below 2^31 - 1024, T * H below 2^31, and so is the number of places
 * (128-row key tiles, and two more, of every run of new tokens that shares a product: 256 query rows of a
 * K/V head) that the table's shape allows (ATTN_ERR_SHAPE).  Returns an attn_status.
 */
ATTN_API int attn_fwd_paged_varlen(const void* q, const attn_kv_cache* cache, const int32_t* block_table,
                                   const int32_t* seq_lens, const int32_t* cu_new, void* o, float* lse,
                                   int B, int T, int H, int H_kv, int d, int max_pages, int causal,
                                   float scale, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes attn_fwd_paged_varlen needs (0 for invalid sizes). */
ATTN_API size_t attn_fwd_paged_varlen_workspace_bytes(int T, int H, int H_kv, int d);

/*
 * Attention of one new token of each of B requests whose first rows are shared: requests cu_groups[g] ..
 * cu_groups[g+1]-1 have the prefix_lens[g] rows of the pages prefix_table[g][0], [1], ... before the seq_lens[s] rows
 * of their own, block_table[s][0], [1], ....  O and lse are those of attn_fwd_paged over the rows of both, but the
 * prefix is read once for all requests of a group that a product takes together, 8 to 256 query rows of a K/V head, instead
 * of once a request.  How many those are goes by the mean over all `groups`, also those without requests: a group much
 * larger than that, or few groups with requests among many, have their prefix read more often (64 requests behind 8192
 * rows, 32 query and 8 K/V heads: 52 us as the only group, 97 as one of 32).  The attentions over the prefixes and over the
 * own rows are left in fp32 and joined by the block merge; three or four launches.
 *   q, o : bf16 [B, H, d] (= [B, H, 1, d]);  lse : fp32 [B, H]
 *   prefix_table : int32 [groups, max_prefix_pages];  prefix_lens : int32 [groups], clamped to 0 ..
 *     max_prefix_pages * page_size;  cu_groups : int32 [groups + 1], from 0 up, at most B (as cu_new of
 *     attn_fwd_paged_varlen: o and lse of requests from cu_groups[groups] on are left as they were)
 *   block_table, seq_lens : as attn_fwd_paged, read for all B requests (0 is a fit length for one past cu_groups[groups]).
 *     Either length may be 0; with both, O = 0 and lse = -inf.
 *   workspace : attn_fwd_paged_shared_workspace_bytes(B, H, H_kv, d) bytes, 256-byte aligned; calls whose
 *     work may overlap on the GPU need one each.
 * Pages, table entries, graphs, limits and errors as attn_fwd_paged and attn_fwd_paged_varlen (groups + B as its B).
 */
ATTN_API int attn_fwd_paged_shared(const void* q, const attn_kv_cache* cache, const int32_t* prefix_table,
                                   const int32_t* prefix_lens, const int32_t* cu_groups,
                                   const int32_t* block_table, const int32_t* seq_lens, void* o, float* lse,
                                   int groups, int B, int H, int H_kv, int d, int max_prefix_pages,
                                   int max_pages, float scale, void* workspace, size_t workspace_bytes,
                                   void* stream);

/* Workspace bytes attn_fwd_paged_shared needs (0 for invalid sizes). */
ATTN_API size_t attn_fwd_paged_shared_workspace_bytes(int B, int H, int H_kv, int d);

/*
 * K and V rows into a paged cache, without the step before attention (rows that are rotated already, or need no
 * rotation, or come from attn_kv_read of another cache): token (b, n)'s rows of every K/V head go to slots[b, n]
 * (int64 [B, N]; negative: not stored).  E4M3 caches get codes and scales as from attn_qkv_rope.
 *   k, v : bf16 rows of d contiguous elements, at b * strides[0] + head * strides[1] + n * strides[2]
 *     elements (k_strides, v_strides: host arrays of three; not negative, multiples of 8 where the
 *     dimension has more than one element); 16-byte aligned, not overlapping the cache
 * A slot past the cache is not stored and the status word reports kind 5.  What two tokens with one slot leave
 * there is unspecified.  One launch.  B * N is below 2^31 - 1024.  Returns an attn_status.
 */
ATTN_API int attn_kv_write(const void* k, const int64_t* k_strides, const void* v, const int64_t* v_strides,
                           const attn_kv_cache* cache, const int64_t* slots, int B, int N, int H_kv, int d,
                           void* stream);

/*
 * Rows of B requests back out of a paged cache, packed as attn_fwd and attn_bwd_varlen take them: row
 * cu_rows[s] + i of k and v is row first[s] + i of request s's pages block_table[s][0], [1], ..., for i <
 * cu_rows[s+1] - cu_rows[s].  E4M3 rows become code * scale, rounded once to bf16; bf16 rows are copied.
 *   k, v : bf16 [H_kv, T, d] outputs;  cu_rows : int32 [B + 1], from 0 up, at most T: rows from
 *     cu_rows[B] on are left as they were (cu_rows that decreases, does not begin with 0 or passes T: kind 2);
 *   first : int32 [B], or NULL for zeros;  block_table : int32 [B, max_pages]
 * A row before the first or past the table, or whose entry names no page of the cache, becomes zeros and the
 * status word reports kind 5.  One launch.  B and T are below 2^31 - 1024.  Returns an attn_status.
 */
ATTN_API int attn_kv_read(const attn_kv_cache* cache, const int32_t* block_table, const int32_t* cu_rows,
                          const int32_t* first, void* k, void* v, int B, int T, int H_kv, int d, int max_pages,
                          void* stream);

/*
 * Unfused comparison path (the "standard attention" of the pages: S written to HBM, read back for
 * the softmax, P written to HBM, read back for P V; CS336 GPU/attention notes, "Attention 为什么
 * 容易 memory-bound"; CS336 Lecture 5 notes, section 6.1).  Three kernel launches on `stream`:
 * scores (S = scale * Q K^T in fp32), row softmax (P in bf16 plus lse), and P V.  It computes the
 * same O and lse as attn_fwd and exists only as the memory-wall comparison.
 * Dense layout only (cu_seqlens must be NULL, else ATTN_ERR_UNSUPPORTED).
 *   workspace : caller-owned device buffer of at least attn_fwd_unfused_workspace_bytes(B,H,N,d)
 *               bytes, 256-byte aligned; its contents on return are unspecified.
 */
ATTN_API int attn_fwd_unfused(const void* q, const void* k, const void* v, void* o, float* lse,
                     const int32_t* cu_seqlens, int B, int H, int N, int d, int causal,
                     float scale, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Workspace bytes attn_fwd_unfused needs for a dense [B, H, N, d] problem: the fp32 score matrix
 * and the bf16 (unnormalised) probability matrix of every head, each row padded to a multiple of
 * 128 columns, plus one fp32 normaliser per row: about B * H * N * (6 * Npad + 4) bytes with
 * Npad = N rounded up to 128 (each region rounded up to 256 bytes).  Returns 0 for invalid sizes.
 */
ATTN_API size_t attn_fwd_unfused_workspace_bytes(int B, int H, int N, int d);

/* Size of the built-in scratch array of attn_fwd_unfused_noalloc (64 MiB per GPU). */
#define ATTN_NOALLOC_SCRATCH_BYTES (64u << 20)

/*
 * The unfused comparison path without a workspace argument, for callers that cannot allocate
 * device memory.  (The reference pages have no counterpart: this is a property of this library's
 * interface, not of the method.)  Some callers cannot call cudaMalloc -- code running under a
 * memory manager that owns every device allocation, or a runtime that forbids allocation once it
 * has started -- so this entry point allocates nothing: its scratch is a file-scope device array of
 * ATTN_NOALLOC_SCRATCH_BYTES that every GPU loading this library holds until the process exits.
 *   Arguments as attn_fwd_unfused (dense layout only), without cu_seqlens and the workspace.
 *   Returns ATTN_ERR_SCRATCH_LIMIT when attn_fwd_unfused_workspace_bytes(B, H, N, d) exceeds
 *   ATTN_NOALLOC_SCRATCH_BYTES, before touching the GPU.
 *   Every call looks up the array's device address (cudaGetSymbolAddress, with the calling
 *   device current); nothing is cached, so a device reset between calls leaves no stale address.
 *   The first call in a context loads the module there; make that first call before any stream
 *   capture.
 *   All calls share the array and it keeps the last call's contents (nothing in it needs to start
 *   at zero); calls whose work overlaps on the GPU, e.g. on two streams, race on it.
 */
ATTN_API int attn_fwd_unfused_noalloc(const void* q, const void* k, const void* v, void* o,
                                      float* lse, int B, int H, int N, int d, int causal,
                                      float scale, void* stream);

/*
 * Device-side status of the kernels launched on `stream` since the previous call: 0 if every
 * pipeline wait completed; otherwise a code whose low byte is 1 (a wait exceeded its time limit,
 * after which the kernel drained its in-flight copies, released its tensor memory and returned;
 * bits 8..15 name the waiting role and bits 16..23 the wait site) or 2 (the cu_seqlens given to a
 * packed-batch call was not a non-decreasing prefix sum from 0 to N; the kernel computed on its
 * offsets clamped into [0, N] and read or wrote nothing outside the tensors) or 3 (a kernel's
 * shared-memory layout did not fit the dynamic shared memory it was given at a 1024-byte boundary;
 * that kernel wrote nothing and its outputs are not valid) or 4 (attn_kv_slots had no page for some
 * token) or 5 (a slot or a block-table entry named no page of the cache).  The first problem
 * recorded is kept.  Synchronises `stream`, then clears the status.  Returns ATTN_ERR_LAUNCH (< 0)
 * if the status cannot be read.
 */
ATTN_API int attn_get_last_device_error(void* stream);

/*
 * Diagnostic: one 128-row tensor-core product with the operand layouts and descriptors of the fused
 * kernel, written to d as fp32 row-major.  Not part of the attention path; it isolates the
 * tcgen05 operand encoding (CS336 Lecture 5 notes, section 6.2: the two matmuls of each tile pair).
 *   mode 0: d[128 x 128] = a[128 x dim] * b[128 x dim]^T   (the S = Q K^T shape)
 *   mode 1: d[128 x dim] = a[128 x 128] * b[128 x dim]     (the O += P V shape)
 *   mode 2: as mode 1 with a staged in tensor memory (the P V shape with P kept on chip)
 *   a, b : bf16 row-major device buffers (16-byte aligned); d : fp32 device buffer;
 *   dim  : 64 or 128.  Asynchronous on `stream`; returns an attn_status.
 */
ATTN_API int attn_selftest_mma(const void* a, const void* b, float* d, int mode, int dim, void* stream);

/*
 * Diagnostic: launch one warp that waits on an mbarrier nothing ever arrives on, through the same
 * bounded wait the pipeline kernels use.  After the wait limit (one second) the warp records
 * status 1 | (6 << 8) | (1 << 16) and returns, leaving the context usable; read it with
 * attn_get_last_device_error().  Exercises failure detection without faulting or hanging the GPU.
 * Returns an attn_status (the launch only).
 */
ATTN_API int attn_selftest_wait_timeout(void* stream);

/*
 * Diagnostic of attn_quantize_fp8's division: for every positive finite bf16 number amax and every
 * bf16 x with |x| <= amax (both signs, about 1.07e9 pairs), compares the E4M3 code the quantizer
 * forms for x at the tile scale amax / 448 with the code of the correctly rounded fp32 quotient
 * (the per-tile scaling of CS336 Lecture 5 notes, section 3.1), and writes the number of pairs
 * that differ to *mismatches.  mismatches: device pointer to one 8-byte-aligned 64-bit counter,
 * which the call zeroes first.  Asynchronous on `stream` (about a second of GPU time); returns an
 * attn_status (the launch only).
 */
ATTN_API int attn_selftest_fp8_quotients(unsigned long long* mismatches, void* stream);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
ATTN_API int attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_GB300_H */
