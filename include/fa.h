/*
 * fa.h -- C ABI of libfa.so: exact tiled scaled-dot-product attention on one
 * GB300 GPU (sm_103a), forward and backward.
 *
 * The operation is O = softmax(scale * Q K^T) V for every batch b and head h,
 * as stated in "Pourquoi l'attention est liée à la mémoire" (marketmaker.cc,
 * "Un contexte d'une journée complète bat-il un contexte de dix minutes ?")
 * and in "Problema e motivação" of the FlashAttention reading guide
 * (xyznot.com, arXiv 2205.14135).  The score matrix is never written to
 * device memory: the forward pass streams key/value tiles through on-chip
 * memory with the running-max / running-sum recurrence ("La récurrence
 * softmax en ligne"; "Rastreamento Incremental do Softmax"), and the backward
 * pass recomputes the scores and probabilities tile by tile from Q, K, V and
 * the saved per-row statistic ("Passe arrière : recalculer au lieu de
 * stocker").
 *
 * Conventions shared by every call:
 *   - Tensors Q, K, V, O, dO, dQ, dK, dV are device buffers of shape
 *     [B][H][N][d], contiguous, in the element type `dtype`; their base
 *     addresses must be 16-byte aligned.  LSE is a device fp32 buffer [B][H][N].
 *   - The caller owns every buffer.  The library allocates no device memory of
 *     its own apart from one small status word per device.
 *   - Calls are asynchronous on `stream` (a cudaStream_t, or NULL for the
 *     legacy default stream).  Argument errors are returned before anything is
 *     launched; a failed launch returns FA_ERR_CUDA; a kernel that gives up
 *     waiting on an on-chip barrier records FA_ERR_TIMEOUT in the status word,
 *     which fa_get_status() returns.
 *   - Only the current CUDA device is used; it must be compute capability 10.3.
 *   - A debug build of the library (compiled with FA_DEBUG defined: libfa_debug.so)
 *     checks, in the kernels, every global-memory index it stores to and every
 *     tile coordinate it copies from against the tensor's bounds; a failed check
 *     skips the access and records FA_ERR_BOUNDS in the status word (no trap, so
 *     the context stays usable).  The release build compiles the checks away.
 */
#ifndef FA_H
#define FA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID = -1,     /* null pointer, size out of range, misaligned buffer, bad scale */
  FA_ERR_UNSUPPORTED = -2, /* well-formed request this library does not implement */
  FA_ERR_CUDA = -3,        /* a CUDA runtime or driver call failed */
  FA_ERR_TIMEOUT = -4,     /* a kernel gave up waiting on a barrier (via fa_get_status) */
  FA_ERR_WORKSPACE = -5,   /* workspace missing or smaller than required */
  FA_ERR_DEVICE = -6,      /* the current device is not compute capability 10.3 */
  FA_ERR_BOUNDS = -7,      /* debug build only: a kernel's index check failed (via fa_get_status) */
  FA_ERR_INDEX = -8        /* a page, slot or length outside the cache it was used with (via fa_get_status) */
} fa_status;

typedef enum { FA_F32 = 0, FA_F16 = 1, FA_BF16 = 2 } fa_dtype;

/*
 * Problem description.
 *   B, H, N, d  batch, heads, sequence length (queries = keys), head size.
 *               N >= 1 (any value: tails that are not a multiple of the tile
 *               are masked); d in {64, 128}; B*H*N*d < 2^31.
 *   dtype       element type of Q, K, V, O, dO, dQ, dK, dV (fa_dtype).
 *               FA_F32 runs the fp32 forward only.
 *   scale       positive finite factor applied to Q K^T before the softmax
 *               (1/sqrt(d) for standard attention).
 *   causal      nonzero: query i only sees keys j <= i ("Le masquage causal
 *               est l'endroit où le trading bénéficie d'une remise").
 *   block_mask  device uint8 matrix or NULL ("Extensão: Block-Sparse
 *               FlashAttention"): entry [i / mask_block][j / mask_block]
 *               keeps (nonzero) or hides (0) the pair (query i, key j).  Each
 *               (b, h) uses the T x T row-major matrix at
 *               block_mask + b * mask_stride_b + h * mask_stride_h, with
 *               T = ceil(N / mask_block); strides in elements, 0 broadcasts.
 *               Combined with `causal` by AND.  Hidden tiles are never loaded.
 *   mask_block  tokens per mask entry; a positive multiple of 128 when
 *               block_mask is set (ignored otherwise).
 *   dropout_p   probability in [0, 1) of dropping each attention weight (the
 *               softmax output, after masking); kept weights are scaled by the
 *               inverse of the keep probability.  Dropout is fused into the
 *               kernels ("Fusão de Kernels", reading guide, "Ideias centrais").
 *               0 = none.
 *   dropout_seed, dropout_offset
 *               the keep decision of weight (query i, key j) of head
 *               bh = b * H + h is the 16-bit half (low for even j, high for
 *               odd j) of word (j mod 8) / 2 of Philox4x32-10 (Salmon et al.,
 *               SC 2011) with counter (j / 8, i, bh, dropout_offset) and key
 *               (seed mod 2^32, seed / 2^32): kept when the half is at least
 *               t = floor(p * 2^16), i.e. with probability 1 - t / 2^16 (p to
 *               within 2^-16), and then scaled by 2^16 / (2^16 - t).  The
 *               backward regenerates the same decisions from the same three
 *               values instead of storing them.
 * A query row whose allowed key set is empty gets O = 0 and LSE = -inf, and
 * contributes nothing to the gradients.  With dropout, O is the dropped and
 * rescaled weights times V, while LSE stays the log-sum-exp of the undropped
 * scores (it is what the backward recomputes the weights from).
 */
typedef struct {
  int B, H, N, d;
  int dtype;
  float scale;
  int causal;
  const uint8_t* block_mask;
  int mask_block;
  long long mask_stride_b, mask_stride_h;
  float dropout_p;
  unsigned long long dropout_seed;
  unsigned int dropout_offset;
} fa_params;

/* Host-only validation of `p` (no CUDA call).  for_backward selects the
 * backward's extra limits.  Returns FA_OK, FA_ERR_INVALID or
 * FA_ERR_UNSUPPORTED. */
fa_status fa_check(const fa_params* p, int for_backward);

/*
 * Forward: O = softmax(scale * Q K^T [masked]) V and
 * LSE[b,h,i] = m_i + ln(l_i), the natural-log log-sum-exp of row i of the
 * scaled, masked scores (the running max m and running sum l of "L'algorithme
 * Flash Attention", folded into one number).  O is written in `dtype`; LSE in
 * fp32.  fp16/bf16 run on the tensor cores (tcgen05, fp32 accumulation);
 * fp32 runs a SIMT kernel in fp32 arithmetic.
 */
fa_status fa_fwd(const fa_params* p, const void* Q, const void* K, const void* V, void* O,
                 float* LSE, void* stream);

/* Largest split count fa_fwd_split accepts (the slices of a query tile run as
 * one thread-block cluster, at most 8 CTAs in a portable cluster). */
#define FA_MAX_SPLITS 8

/*
 * Split-KV forward: the same O and LSE as fa_fwd, computed with the key range
 * of every 128-row query tile cut into `num_splits` slices of
 * ceil(ceil(N / 128) / num_splits) key tiles, one CTA per (query tile, slice),
 * so that a problem with few query tiles (one long sequence, few heads) still
 * fills the GPU.  Each slice keeps its own running max m_s and sum l_s; the
 * slices of a query tile run as one thread-block cluster and merge in shared
 * memory with the statistics merge of "Rastreamento Incremental do Softmax"
 * (the reading guide to the FlashAttention paper): m = max_s m_s,
 * l = sum_s exp(m_s - m) l_s, O = sum_s exp(m_s - m) O_s / l and
 * LSE = m + log l, each slice's O_s unnormalised.  Nothing goes through device
 * memory but Q, K, V, O and LSE.  The key-scan parallelism of the decode
 * kernels mentioned in "Что это изменило на практике" ("Почему Flash Attention
 * быстрее") is the same idea.
 *
 * num_splits in [1, min(FA_MAX_SPLITS, ceil(N / 128))], else FA_ERR_INVALID;
 * a count that would leave trailing slices empty runs with the non-empty ones
 * only.  num_splits = 1 is fa_fwd.  fp16/bf16 only for num_splits > 1 (FA_F32
 * -> FA_ERR_UNSUPPORTED).  Results match fa_fwd up to rounding order (the
 * fp32 slices are rounded to `dtype` once, after the merge).
 */
fa_status fa_fwd_split(const fa_params* p, const void* Q, const void* K, const void* V, void* O,
                       float* LSE, int num_splits, void* stream);

/* Split count for fa_fwd_split on a GPU with `num_sms` SMs (<= 0: ask the
 * current device; 1 if that fails).  1 when the unsplit grid of B*H*ceil(N/128)
 * CTAs already fills one wave of 2 * num_sms (two CTAs per SM); otherwise the
 * count with the fewest modelled waves x (key tiles per CTA + 2).  1 for
 * FA_F32, 0 on invalid p.  Host-only when num_sms > 0. */
int fa_fwd_num_splits(const fa_params* p, int num_sms);

/* Bytes of device workspace fa_bwd needs, each part 256-byte aligned.  The
 * backward of "Passe arrière : recalculer au lieu de stocker" (marketmaker.cc)
 * keeps only O and the per-row statistic of the forward and recomputes the rest;
 * what it needs besides is linear in N ("Análise de Complexidade", reading
 * guide: O(N) extra memory): fp32
 * D = rowsum(dO * O) [B*H*N], the fp32 dQ accumulator [B*H*N*d] and, without a
 * block mask, the fp32 partial-sum slots of a sliced main kernel (2 x 128 x d
 * values for each of up to min(160, pairs) slices, where pairs = B*H*T^2 or
 * B*H*T(T+1)/2 causal, T = ceil(N / 128)).  0 on invalid p. */
size_t fa_bwd_workspace_size(const fa_params* p);

/*
 * Backward of the forward above for the loss whose gradient at O is dO, as
 * "Passe arrière : recalculer au lieu de stocker" (marketmaker.cc) and the
 * recomputation bullet of "Ideias centrais" (reading guide) describe it: the
 * score and probability tiles are recomputed block by block from Q, K and the
 * saved LSE instead of being stored.  The formulas (the pages give none) are the
 * derivative of the definition:
 *   P = exp(scale * S - LSE), dV = P^T dO, dP = dO V^T, D = rowsum(dO * O),
 *   dS = P * (dP - D), dQ = scale * dS K, dK = scale * dS^T Q.
 * Q, K, V, O, LSE must be those of the forward call (same params).  dQ, dK, dV
 * are written in `dtype`.  `workspace` is a device buffer of at least
 * fa_bwd_workspace_size(p) bytes, 256-byte aligned, owned by the caller; its
 * contents on entry do not matter.  fp16/bf16 only (FA_F32 -> UNSUPPORTED).
 * Runs fa_bwd_preprocess, fa_bwd_main and fa_bwd_finalize in that order.
 */
fa_status fa_bwd(const fa_params* p, const void* Q, const void* K, const void* V, const void* O,
                 const void* dO, const float* LSE, void* dQ, void* dK, void* dV, void* workspace,
                 size_t workspace_bytes, void* stream);

/* The three stages of fa_bwd, exported so that each can be timed on its own.
 * preprocess: D = rowsum(dO * O) into the workspace, dQ accumulator zeroed.
 * main: recompute P tile by tile, accumulate dK, dV per key tile and add
 *       scale-free dQ contributions into the accumulator.  One CTA per key
 *       tile, whose dK, dV it writes.  Without a block mask, when that would
 *       leave SMs idle, key tiles are cut into slices of their query tiles,
 *       one CTA each, a key tile of several slices getting fp32 partial dK, dV
 *       in the workspace: with fewer key tiles than SMs every key tile (slices
 *       as short as fill one wave), and, non-causal, the key tiles of a last,
 *       partly filled wave (over the SMs that wave leaves idle).
 * finalize: dQ = scale * accumulator, converted to `dtype`, and dK, dV of the
 *       shared key tiles from their partial sums.  Must follow the main stage
 *       of the same call sequence (same p, workspace and fa_set_bwd_ctas). */
fa_status fa_bwd_preprocess(const fa_params* p, const void* O, const void* dO, void* workspace,
                            size_t workspace_bytes, void* stream);
fa_status fa_bwd_main(const fa_params* p, const void* Q, const void* K, const void* V,
                      const void* dO, const float* LSE, void* dK, void* dV, void* workspace,
                      size_t workspace_bytes, void* stream);
fa_status fa_bwd_finalize(const fa_params* p, void* dQ, void* dK, void* dV, void* workspace,
                          size_t workspace_bytes, void* stream);

/* The CTAs per wave that the backward main kernel plans its slices for (0, the
 * default: one per SM, at most 160; n > 0: min(n, that)).  Applies to backward
 * calls made after it; do not change it between the main and finalize stages
 * of one backward pass.  Returns the previous value.  The tests use it to make
 * small problems cut their key tiles into slices. */
int fa_set_bwd_ctas(int n);

/*
 * Maximum workspace, in bytes, that fa_bwd_noalloc can serve (64 MiB); e.g.
 * B=4, H=12, N=2048, d=64 needs about 34 MiB (fa_bwd_workspace_size).
 */
#define FA_NOALLOC_SCRATCH_BYTES (64ull << 20)

/*
 * The backward pass for callers that cannot allocate device memory where they
 * run it -- a plugin handed a fixed memory budget by its host application, an
 * engine that plans every buffer ahead of time and forbids allocation on its
 * execution path, or code that must not enter the CUDA allocator while other
 * work holds it.  The pages have no counterpart of this call; it exists for
 * those callers only.
 *
 * Same arguments and results as fa_bwd without the workspace: the fp32 scratch
 * (D, the dQ accumulator and the partial-sum slots) comes from a FA_NOALLOC_SCRATCH_BYTES array that
 * is part of the library image, so every GPU that loads libfa.so holds that
 * memory until the process exits.  No call here allocates or frees device
 * memory.  A problem whose workspace (fa_bwd_workspace_size) exceeds the array
 * is rejected with FA_ERR_WORKSPACE before anything is launched.
 *
 * The first call on each device looks up the array's device address (with
 * that device current) and caches it; make that first call before any stream
 * capture.  Under the CUDA runtime's default lazy module loading the driver
 * commits the array's device memory at that first lookup (under eager loading,
 * when the context is created), so that first call is where an out-of-memory
 * error can appear: make it during set-up, not on the execution path.  The
 * cached address is that of the runtime's primary context on each device;
 * callers that run the library under another driver context are not served.
 * Every call, on every stream, shares the one array: calls that can overlap on
 * the GPU race on it and must be serialised by the caller.  Each call rewrites
 * all the scratch it reads: D and the dQ accumulator (zeroed first) in the first
 * stage, and the fp32 partial-sum slots of key tiles cut into several slices,
 * each stored in full by the main stage before the finalize stage reads it.  So
 * nothing left by an earlier call affects a call's results.
 */
fa_status fa_bwd_noalloc(const fa_params* p, const void* Q, const void* K, const void* V,
                         const void* O, const void* dO, const float* LSE, void* dQ, void* dK,
                         void* dV, void* stream);

/* Synchronises `stream`, returns the device-side status recorded since the
 * previous call (FA_OK, FA_ERR_TIMEOUT, FA_ERR_INDEX, or FA_ERR_BOUNDS in the
 * debug build; the first one counts) and clears it, so that calls and graphs that
 * run afterwards are not affected; FA_ERR_CUDA if the synchronisation itself
 * fails.  What a launch that recorded FA_ERR_TIMEOUT wrote is void.  The pages
 * have no counterpart: it reports the library's own failure detection (every
 * on-chip barrier wait of every kernel is bounded in time, so a kernel that cannot
 * proceed gives up and records the error instead of hanging), which guards the
 * custom low-level CUDA that "Limitações e questões em aberto" (reading guide)
 * names as the method's cost. */
fa_status fa_get_status(void* stream);

/* Upper bound, in nanoseconds, on any single barrier wait inside the kernels
 * launched after this call (default 2e9).  Returns the previous value. */
unsigned long long fa_set_wait_limit_ns(unsigned long long ns);

/* Launches one CTA that waits on a barrier nothing will complete, so that the
 * wait limit runs out and FA_ERR_TIMEOUT is recorded; used to test the
 * failure path without faulting the GPU.  Returns the launch status. */
fa_status fa_selftest_timeout(void* stream);

/* Static description of a status code. */
const char* fa_status_string(int status);

/* Text of the last CUDA or validation failure seen by this thread. */
const char* fa_last_error(void);

/* Library interface version (major * 100 + minor). */
int fa_version(void);

/* ------------------------------------------------------------------------
 * FP8 forward with incoherent processing ("Trois idées pour FA3",
 * marketmaker.cc, point 3: naive FP8 attention suffers from outlier
 * coordinates; rotating the query and key vectors at random before block
 * quantisation spreads an outlier over all coordinates).  Two calls, so that
 * the quantised operands can be produced once and reused:
 *
 *   fa_fp8_quantize  Q^ = Q D H / d and K^ = K D H, with H the d x d Sylvester
 *                    Hadamard matrix (H_ab = (-1)^popcount(a & b)) and
 *                    D = diag(signs); Q^ K^^T = Q K^T since H H^T = d I.  With
 *                    signs = NULL there is no rotation (Q^ = Q, K^ = K).  V is
 *                    not rotated.  Each block of 128 rows of one head of Q^, K^
 *                    and V gets the smallest power-of-two scale sigma with
 *                    max|x| / sigma <= 448 (1 for an all-zero block; 2^-126 at
 *                    least), and its values become e4m3 codes of x / sigma
 *                    (round to nearest even, saturating to +-448; the rotated
 *                    values are formed in fp32).
 *   fa_fwd_fp8       the forward on those codes: scores
 *                    scale * sigma_q * sigma_k * (q8 . k8) accumulated in fp32
 *                    on the tensor cores, the online softmax against the exact
 *                    running max m, the weights P~ = exp(s - m) <= 1 quantised
 *                    as e4m3(256 P~) for the P~ V product, the row sum l of the
 *                    unquantised P~; O = sum sigma_v P~q V8 / (256 l) in the
 *                    dtype of p, LSE = m + ln l (natural log, fp32).
 *
 * Buffers (device memory, owned by the caller, 16-byte aligned except the
 * scales, which are 4-byte aligned):
 *   q8, k8      uint8 [B*H][N][d]     e4m3 codes of Q^ and K^
 *   vt8         uint8 [B*H][d][ld]    e4m3 codes of V transposed (row c holds
 *                                     column c of V over the keys), ld =
 *                                     fa_fp8_vt_cols(N); entries past N are 0
 *   sq, sk, sv  float [B*H][ceil(N / 128)]  the block scales (powers of two)
 *   signs       float [d]             +-1 (device memory), or NULL
 * p: dtype FA_F16 or FA_BF16 (of Q, K, V and of O), d 64 or 128, causal and
 * block masks as for fa_fwd; dropout and FA_F32 give FA_ERR_UNSUPPORTED.  Both
 * calls are asynchronous on `stream`; validation errors return before any
 * launch.  Codes made elsewhere (any e4m3 values with power-of-two scales in
 * this layout) may be passed to fa_fwd_fp8.
 * ------------------------------------------------------------------------ */
int fa_fp8_vt_cols(int N);
fa_status fa_fp8_quantize(const fa_params* p, const void* Q, const void* K, const void* V,
                          const float* signs, void* q8, void* k8, void* vt8, float* sq, float* sk,
                          float* sv, void* stream);
fa_status fa_fwd_fp8(const fa_params* p, const void* q8, const void* k8, const void* vt8,
                     const float* sq, const float* sk, const float* sv, void* O, float* LSE,
                     void* stream);

/* ------------------------------------------------------------------------
 * Norms of the query and key heads and the rotation by position, in one pass
 * from the projection to the layout the attention reads, and its gradient.
 *
 *   n_c = x_c * r * w_c,  r = 1 / sqrt(mean_c x_c^2 + eps)     for every head row
 *   (y_a, y_b) = (n_a cos t - n_b sin t, n_a sin t + n_b cos t)  for every pair i
 *
 * with t = position * angle per step of pair i.  Pair i is (i, i + rot_dim / 2),
 * or (2 i, 2 i + 1) with `interleaved`, for i < rot_dim / 2; channels from
 * rot_dim on are normed only.  freqs[i] is the pair's angle per step in units of
 * 2^-64 turns: position * freqs[i] mod 2^64 is then the exact phase at any
 * position, and its leading 32 bits give the angle to 2^-32 turns.
 *
 *   B, N, Hq, Hk, d  batch, tokens per batch entry (>= 0), query and key heads,
 *               head size (64 or 128); B*N < 2^30, Hq + Hk < 2^24.
 *   dtype       fa_dtype of q, k, yq, yk and their gradients (fp32 arithmetic
 *               inside); weight_dtype that of wq, wk: `dtype` or FA_F32.
 *   eps         positive and finite.
 *   *_stride    element strides {batch, token, head}; channels are contiguous.
 *               Bases 16-byte aligned, strides multiples of 16 bytes; written
 *               tensors must not overlap themselves.  q and k may be views of one
 *               packed projection.  yq (yk) may be q (k), and dq (dk) may be q or dyq
 *               (k or dyk), with the same strides; other overlaps are not allowed.
 *               Token and head strides below 2^31 bytes.
 *   pos_stride  batch stride of `positions` in elements (0: one row for all).
 * positions: device int32 [B][N], or NULL for positions 0 .. N - 1.
 * ------------------------------------------------------------------------ */
typedef struct {
  int B, N, Hq, Hk, d;
  int dtype, weight_dtype;
  int rot_dim, interleaved;
  float eps;
  long long pos_stride;
  long long q_stride[3], k_stride[3];   /* the projection */
  long long yq_stride[3], yk_stride[3]; /* the result; its gradient in the backward */
  long long dq_stride[3], dk_stride[3]; /* backward: the projection's gradient */
} fa_qk_params;

fa_status fa_qk_norm_rope(const fa_qk_params* p, const void* q, const void* k, const void* wq,
                          const void* wk, const uint64_t* freqs, const int* positions, void* yq,
                          void* yk, void* stream);

/* Bytes of workspace of the backward (fp32 partial sums of the weights'
 * gradients); 0 on invalid p. */
size_t fa_qk_norm_rope_bwd_workspace_size(const fa_qk_params* p);

/* Gradients of fa_qk_norm_rope for the gradients dyq, dyk at its results: with
 * dz the back-rotated dy and h = x r, dx = r (w dz - h mean(w dz h)) and
 * dw = sum over rows of dz h (fp32 [d] each, summed in a fixed order).  q and k
 * are the forward's inputs; r is formed again.  The workspace is 256-byte
 * aligned and owned by the caller; its contents do not matter, and calls that may
 * run at the same time need workspaces of their own. */
fa_status fa_qk_norm_rope_bwd(const fa_qk_params* p, const void* q, const void* k, const void* dyq,
                              const void* dyk, const void* wq, const void* wk,
                              const uint64_t* freqs, const int* positions, void* dq, void* dk,
                              float* dwq, float* dwk, void* workspace, size_t workspace_bytes,
                              void* stream);

/* ------------------------------------------------------------------------
 * A paged key/value cache in 4 bits, and the attention that reads it.
 *
 * The cache is num_pages pages of page_size tokens (a power of two, 16 to 4096) of Hk
 * heads, page_stride bytes apart; a page holds, head by head, page_size / 16 blocks of 16
 * tokens.  A block (fa_kv4_block_bytes(d) bytes) is
 *     uint8  key codes   [16][d / 2]    channel 2 b in the low, 2 b + 1 in the high half of byte b
 *     half2  key pairs   [16][d / 32]   (scale, base) of each 32 channels
 *     the same for the values.
 * Code c of a pair (scale, base) stands for the fp16 number nearest to
 * base + scale * (1 + c / 16): c is the top of the mantissa of an fp16 number in
 * [1, 2), which one fused multiply-add turns into the value.  Token j of page p is
 * slot p * page_size + j.
 * ------------------------------------------------------------------------ */
typedef struct {
  int num_pages, page_size, Hk, d;
  long long page_stride; /* bytes; a multiple of 16, at least one page's blocks */
} fa_kv4_cache;

/* Bytes of a 16-token block of one head: 2560 for d = 128, 1280 for d = 64, else 0. */
int fa_kv4_block_bytes(int d);

/* T tokens' keys and values ([T][Hk][d], element strides {token, head}, of `dtype`);
 * T*Hk < 2^30, strides below 2^31 elements. */
typedef struct {
  int T, dtype;
  long long k_stride[2], v_stride[2];
} fa_kv4_rows;

/* Quantise T tokens' keys and values into their slots (device int32 [T]; a
 * negative slot's token is left out).  For each token, head and 32 channels, of
 * x saturated at +-16384 and widened to fp32 (lo, hi its least and largest):
 *     scale = fp16((hi - lo) * 16 / 15),  base = fp16(lo - scale),
 *     c = min(15, max(0, rint((x - base) * 16 / scale - 16))), 0 where scale = 0.
 * A NaN makes its 32 values NaN.  A slot past the cache is left out and recorded
 * as FA_ERR_INDEX.  The slots >= 0 of one call must be distinct: of two tokens
 * with one slot the result is a mixture. */
fa_status fa_kv4_append(const fa_kv4_cache* c, const fa_kv4_rows* rows, const void* k,
                        const void* v, const int* slots, void* cache, void* stream);

/* The values that T slots hold, rounded to `dtype` (zeros for a negative slot). */
fa_status fa_kv4_gather(const fa_kv4_cache* c, const fa_kv4_rows* rows, const void* cache,
                        const int* slots, void* k, void* v, void* stream);

/*
 * Attention of R requests' newest tokens over their cached keys and values:
 * O = softmax(scale * q K^T) V and LSE (natural log) for query heads Hq, a multiple
 * G of the cache's Hk: query head h reads key head h / G.  Request r has
 * kv_lens[r] cached tokens, token j in page block_table[r][j / page_size]; its
 * queries are rows cu_q[r] .. cu_q[r + 1] of q (row r alone where cu_q is NULL) and
 * stand for its last tokens, so that the i-th of n sees the tokens up to
 * p = kv_lens[r] - n + i, and with window > 0 only those after p - window.  A row
 * that sees no token gets O = 0 and LSE = -inf; rows of q outside every request
 * are not written.  A NaN in a cached key (a pair of NaN) makes O and LSE of the rows that
 * see its token NaN; one in a cached value O's 32 channels of that pair, and nothing else.
 * Tokens that no row sees may hold anything; pairs of seen ones are as fa_kv4_append writes
 * them (finite values, or NaN).
 *   T           rows of q and o ([T][Hq][d], element strides {token, head}, FA_F16 or
 *               FA_BF16); lse: fp32 [T][Hq] or NULL.
 *   max_q_len   the largest number of rows of a request: a hint for the tile height
 *               (a larger one is still computed).
 *   table_width, table_stride  columns of block_table and its row stride.
 * Lengths are device memory: the tokens of all requests are cut into equal shares
 * on the GPU.  A page outside the cache contributes nothing and is recorded as
 * FA_ERR_INDEX, as is a length beyond table_width * page_size, which is cut to that.
 * o and lse must not lie over q or each other, in part neither.  Calls that may run at
 * the same time need workspaces of their own.  Limits: T*Hq < 2^31, table_width * page_size
 * <= 2^30, num_pages * page_size < 2^31, a page below 2^31 bytes.
 */
typedef struct {
  int R, T, Hq, dtype;
  int max_q_len, window;
  int table_width;
  float scale;
  long long table_stride;
  long long q_stride[2], o_stride[2];
} fa_kv4_attn_params;

/* Bytes of workspace (shares that end inside a request's tokens, in fp32), 256-byte
 * aligned, contents on entry do not matter; 0 on invalid arguments. */
size_t fa_kv4_attention_workspace_size(const fa_kv4_cache* c, const fa_kv4_attn_params* p);
fa_status fa_kv4_attention(const fa_kv4_cache* c, const fa_kv4_attn_params* p, const void* q,
                           const void* cache, const int* block_table, const int* kv_lens,
                           const int* cu_q, void* o, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * The same in 8 bits: codes of a signed byte with one scale for each block of 16 tokens
 * of a head (one for its keys, one for its values).  Pages, slots, block tables, rows and
 * requests are as above.  A block (fa_kv8_block_bytes(d) bytes: 32 d + 16) is
 *     int8   keys    [16][d]              at d = 128 the 64-byte halves of odd tokens' rows
 *                                         are in each other's place
 *     int8   values  [d / 4][4][4][4]     channel c of token j at [c/4][j/4][c%4][j%4]
 *     float  scale of the keys, scale of the values
 *     uint16 marks of the keys, of the values: bit j set where token j's hold a NaN
 *     4 bytes of 0
 * and a value is its code times its scale, or NaN where its token is marked.
 *
 * fa_kv8_append: of each side, the scale of a block is the least power of two (at least
 * 2^-64) with max|x| <= 127 * scale over the values x that were put into it since it
 * began, saturated at +-16384, or 0 where they are all 0; a code is rint(x / scale).  A
 * block whose place 0 is among the call's slots begins anew: what it held counts no more.
 * Other blocks keep their tokens: where the new ones need a larger scale, the codes of the
 * others become rint(code * old / new); a token that is written over (a draft that was
 * taken back) leaves the scale it raised, and what was rounded to it.  A token with a NaN is marked and its codes of that side are 0.
 * The tokens of one block must be neighbours in the call (as fa_paged_plan puts them; the
 * 4-bit cache takes any order); slots >= 0 must be distinct.  Where they are not, those
 * blocks' contents are void, and nothing is recorded.
 * fa_kv8_attention: a key's mark makes O and LSE of the rows that see it NaN, a value's
 * mark their O.
 * ------------------------------------------------------------------------ */
typedef fa_kv4_cache fa_kv8_cache;
typedef fa_kv4_rows fa_kv8_rows;
typedef fa_kv4_attn_params fa_kv8_attn_params;

int fa_kv8_block_bytes(int d);
fa_status fa_kv8_append(const fa_kv8_cache* c, const fa_kv8_rows* rows, const void* k,
                        const void* v, const int* slots, void* cache, void* stream);
fa_status fa_kv8_gather(const fa_kv8_cache* c, const fa_kv8_rows* rows, const void* cache,
                        const int* slots, void* k, void* v, void* stream);
size_t fa_kv8_attention_workspace_size(const fa_kv8_cache* c, const fa_kv8_attn_params* p);
fa_status fa_kv8_attention(const fa_kv8_cache* c, const fa_kv8_attn_params* p, const void* q,
                           const void* cache, const int* block_table, const int* kv_lens,
                           const int* cu_q, void* o, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * Block tables and slot maps of one step, from R request lengths, on the GPU.
 * Request r holds seq_lens[r] tokens in the first ceil(seq_lens[r] / page_size)
 * pages of its row of block_table; new_lens[r] tokens are added, or, where it is
 * negative, the request has ended and its pages go back.  free_pages[0 ..
 * free_count) is a stack: the ended requests' pages are put on top of it in order,
 * then each request in turn takes the pages its new tokens need off the top, all
 * or none.  A request is not served (no page, its tokens' slots -1, its length
 * unchanged) when its tokens end past T, its pages past table_width, or, where it
 * needs pages, when the pages wanted up to and including its own exceed the stack.
 * Written:
 *   block_table, free_pages   the entries that changed
 *   kv_lens[R]                tokens held after the step (0 where ended)
 *   cu_q[R + 1]               first of each request's new tokens, cut to T
 *   positions[T], slots[T]    of each new token; 0 and -1 after the last one
 *   counts[3]                 pages left on the stack, new tokens, pages missing
 * kv_lens may be seq_lens and counts may be free_count (three ints): everything is
 * read before anything is written.  Lengths below 0 count as 0 tokens; all arrays
 * are device int32.  R in [1, FA_PLAN_MAX_REQUESTS], T and num_pages at most 2^30.
 */
#define FA_PLAN_MAX_REQUESTS 8192
typedef struct {
  int R, T, page_size, num_pages; /* num_pages: entries of free_pages */
  int table_width;
  long long table_stride;
} fa_plan_params;

fa_status fa_paged_plan(const fa_plan_params* p, const int* seq_lens, const int* new_lens,
                        int* block_table, int* free_pages, const int* free_count, int* kv_lens,
                        int* cu_q, int* positions, int* slots, int* counts, void* stream);

/* ------------------------------------------------------------------------
 * Attention of R sequences of different lengths packed one behind the other, with
 * grouped heads, and its gradient.
 *
 * Sequence r's queries are rows cu_q[r] .. cu_q[r + 1] of q and its keys and values
 * rows cu_k[r] .. cu_k[r + 1] of k and v; query head h reads key head h / (Hq / Hk).
 * With n queries over m keys (any n and m, also 0) and `causal`, query i sees the
 * keys j <= i + m - n: the last query stands at the last key, so that new rows over
 * a longer cached prefix, or a whole prompt (m = n), are the same call.
 *     O = softmax(scale * q K^T) V,  LSE = the log-sum-exp of the scaled scores;
 * a row that sees no key gets O = 0 and LSE = -inf and has no part in the gradients.
 *   R           sequences (1 to 2^24 - 1); cu_q, cu_k: device int32 [R + 1]; cu_k NULL: cu_q
 *               (Tq = Tk).  Offsets outside the tensors or smaller than one before are
 *               taken as the nearest that is neither, and recorded as FA_ERR_INDEX.
 *   Tq, Tk      rows of q and of k and v, at most 2^30; Tq*Hq, Tk*Hk < 2^31.
 *   Hq, Hk, d   query and key heads (Hq / Hk at most 128), head size (64 or 128).
 *   dtype       FA_F16 or FA_BF16 of all tensors; lse: fp32 [Tq][Hq].
 *   *_stride    element strides {token, head} of [T][H][d]; channels are contiguous.
 *               Bases 16-byte aligned, strides multiples of 16 bytes, below 2^38, and not
 *               0; written tensors must not overlap themselves.  q, k and v may be
 *               views of one packed projection, in either order of tokens and heads.
 * Results must not lie over inputs or each other, not in part either, and are refused then
 * (dq may be q, o or do with the same strides).  Views of one buffer whose rows or heads
 * take turns, at the distance of a stride of one of them, lie beside each other.
 * Rows that are in no sequence are neither read into a result nor written.  What is not
 * finite in k, v or q reaches, in the forward pass, the rows that see it (an infinite value
 * makes its channel there infinite or, where its weight is 0 in the type, NaN); in the
 * backward pass it may reach every gradient of its own sequence, and none of another.
 * The workspace is 256-byte aligned and owned by the caller; its contents do not matter;
 * calls that may run at the same time need workspaces of their own.
 * In fp16 the backward pass holds the weights and dS times powers of two (of dS one for each
 * sequence and key head, from its largest |dO|, |V| and |D|), so that small and large incoming
 * gradients, and weights over many keys, keep the type's bits.  lse has to be the forward's: a
 * weight that it makes larger than 4 may be infinite there.
 * The forward pass and dK, dV add in a fixed order; dQ is a sum of parts that arrive in
 * any order (fp32), so that its last bits may differ from call to call, as fa_bwd's.
 * ------------------------------------------------------------------------ */
typedef struct {
  int R, Tq, Tk, Hq, Hk, d;
  int dtype, causal;
  float scale;
  long long q_stride[2], k_stride[2], v_stride[2], o_stride[2];
  long long do_stride[2], dq_stride[2], dk_stride[2], dv_stride[2]; /* backward */
} fa_packed_params;

/* Bytes of workspace (the work list, partial results of long tiles); 0 on invalid p. */
size_t fa_fwd_packed_workspace_size(const fa_packed_params* p);
fa_status fa_fwd_packed(const fa_packed_params* p, const void* q, const void* k, const void* v,
                        const int* cu_q, const int* cu_k, void* o, float* lse, void* workspace,
                        size_t workspace_bytes, void* stream);

/* dQ, dK, dV from the forward's inputs and results (the formulas are fa_bwd's); a key
 * head's dK and dV are the sums over its query heads.  The workspace holds, besides, an
 * fp32 accumulator of dQ. */
size_t fa_bwd_packed_workspace_size(const fa_packed_params* p);
fa_status fa_bwd_packed(const fa_packed_params* p, const void* q, const void* k, const void* v,
                        const void* o, const void* dout, const float* lse, const int* cu_q,
                        const int* cu_k, void* dq, void* dk, void* dv, void* workspace,
                        size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_H */
