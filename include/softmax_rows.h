/*
 * softmax_rows.h -- C ABI of the GB300 (sm_103a) row-wise online softmax library.
 *
 * Library: row_wise_online_gb300/lib/libsoftmax_rows.so.  Every compute call
 * enqueues CUDA kernels on the caller's stream and returns at once; every step
 * of the computation runs in the library's own kernels.
 *
 * The problem (as stated on "5.2 CUDA Online Softmax 实现优化", §1.1 and
 * §2): for each row r of a row-major M x N matrix x,
 *
 *     m_r   = max_j x[r, j]
 *     d_r   = sum_j exp(x[r, j] - m_r)
 *     y[r,j]= exp(x[r, j] - m_r) / d_r
 *     LSE_r = m_r + ln d_r      ("从原始Softmax到在线Softmax", log-sum-exp)
 *
 * computed with the online (m, d) recurrence (§2.1 of the same page): each
 * thread folds its elements into a running max and a rescaled exp-sum, and
 * partial states are merged with m = max(m1, m2),
 * d = d1 e^(m1 - m) + d2 e^(m2 - m)  (§4.1; "Softmax 数值稳定性与 IO-Aware
 * Attention" §4.1).  The empty state (-inf, 0) is the identity of that merge,
 * so a fully masked (-inf) chunk, thread, warp or block contributes nothing
 * and never produces NaN.  A row whose entries are all -inf gives y = 0,
 * m = -inf, d = 0, LSE = -inf.
 *
 * Conventions shared by every call:
 *  - Pointers are DEVICE pointers (except softmax_rows_host), owned by the
 *    caller; the library keeps none of them after the call is enqueued.
 *  - Matrices are row-major and contiguous: row r starts at element r * N.
 *  - dtype is SOFTMAX_F32 (fp32 in / fp32 out), SOFTMAX_BF16 (bf16 bit
 *    patterns in / bf16 out) or SOFTMAX_F16 (IEEE binary16 in / out); 16-bit
 *    outputs are rounded to nearest even (fp16 keeps subnormals).  Arithmetic
 *    is fp32 in every case; exponentials use the hardware ex2 with a log2(e)
 *    prescale.  fp16's range ends at 65504 ("Softmax 数值稳定性与 IO-Aware
 *    Attention" §一, precision and range of the floating-point formats):
 *    inputs cannot exceed it, softmax outputs (in [0, 1]) always fit, and
 *    log-softmax outputs below -65504 round to -inf.
 *  - State outputs m_out, d_out, lse_out are fp32 arrays of M entries; each
 *    may be NULL.  m_out is the raw row maximum (bit-exact max of the inputs,
 *    -0 and +0 equal).  d_out is relative to m_out, natural base.
 *  - stream is a cudaStream_t passed as void* (NULL = the legacy default stream).
 *  - M == 0 is a no-op returning SOFTMAX_OK (the pointers may then be NULL,
 *    as they are for an empty tensor); N, dtype and variant are still checked.
 *  - Return value: a softmax_status.  Argument errors are detected on the
 *    host before anything is enqueued.  A CUDA launch error returns
 *    SOFTMAX_ERR_CUDA (softmax_last_cuda_error() names it).  Errors found by a
 *    kernel while it runs (a bounded wait that ran out) are recorded in a
 *    per-device status word read by softmax_get_status().
 */
#ifndef ROW_WISE_ONLINE_SOFTMAX_ROWS_H
#define ROW_WISE_ONLINE_SOFTMAX_ROWS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
enum softmax_dtype { SOFTMAX_F32 = 0, SOFTMAX_BF16 = 1, SOFTMAX_F16 = 2 };

/* Status codes. */
enum softmax_status {
  SOFTMAX_OK = 0,
  SOFTMAX_ERR_INVALID_ARG = 1, /* NULL pointer, N < 1, M < 0, unknown dtype/variant, size overflow */
  SOFTMAX_ERR_MISALIGNED = 2,  /* a forced vector/bulk-copy variant got a base or row pitch not 16-B aligned */
  SOFTMAX_ERR_UNSUPPORTED = 3, /* a forced variant cannot take this shape (row too large, ...) */
  SOFTMAX_ERR_CUDA = 4,        /* a CUDA runtime call or launch failed */
  SOFTMAX_ERR_TIMEOUT = 5      /* a kernel's bounded wait ran out (reported by softmax_get_status) */
};

/* Kernel variants (softmax_rows_ex).  AUTO picks one from the shape. */
enum softmax_variant {
  SOFTMAX_VARIANT_AUTO = 0,
  /* One read: the row is loaded once into registers with 128-bit loads (rows up to 64 KiB; AUTO
     takes it for fp32 rows up to 64 KiB and 16-bit rows up to 4 KiB). */
  SOFTMAX_VARIANT_ONEREAD_REG = 1,
  /* One read: bulk copies (cp.async.bulk + mbarrier) stage whole rows in shared memory.  Rows
     up to 8 KiB: each warp owns a row at a time and a private ring of row slots that its lane 0
     refills; longer rows (up to 64 KiB; fp32 rows up to 128 KiB, 16-bit rows up to 120 KiB, kept
     packed): a producer warp feeds a CTA-wide consumer group that copies the row to registers
     and frees the slot at once; longer
     rows (16-byte aligned, up to 1 MiB): a thread-block cluster of 2-8 CTAs per row, each CTA's
     segment held in shared and tensor memory until the row's state, merged over distributed
     shared memory, is known.  AUTO takes the last for many rows of 128 - 512 KiB and 768 KiB - 1 MiB. */
  SOFTMAX_VARIANT_ONEREAD_SMEM = 2,
  /* Two passes over global memory: online fold with 128-bit loads, then re-read and normalise
     (any N; the re-read is served from L2 while the row is still resident).  Aligned rows above
     64 KiB run on the cluster-row kernel: rows of ~260 KiB and more are shared by a thread-block
     cluster (2-16 CTAs, states merged over distributed shared memory), so that the rows in
     flight stay within L2. */
  SOFTMAX_VARIANT_TWOPASS = 3,
  /* Split row: one row is spread over every CTA of the grid; CTAs of a thread-block cluster merge
     (m, d) over distributed shared memory, clusters exchange 8-byte states through global memory
     (16-byte aligned rows above about 150 KiB).  Each CTA holds its segment of a row in shared
     memory from the load until the normalisation, so x is read once: rows up to about 17 MB on
     a 152-SM GB300 (at least two segments per SM fit in shared memory; shorter rows keep up to
     eight in flight).  Longer rows run SOFTMAX_VARIANT_SPLITROW_STREAM instead (and
     softmax_last_variant() reports that).  AUTO takes the split row for rows of 8 MiB and more at
     any row count, and for rows of 4 MiB and more when there are at most 16 of them.
     It needs every cluster resident at once, so it must not share the GPU with other kernels
     (softmax_rows_host never uses it): kernels running beside it on other streams can keep
     clusters off the GPU until the exchange wait runs out (SOFTMAX_ERR_TIMEOUT, y undefined). */
  SOFTMAX_VARIANT_SPLITROW = 4,
  /* Split row, streaming: as SOFTMAX_VARIANT_SPLITROW, but nothing of a row is held on chip, so
     rows of any length are taken: every CTA streams its segment twice through a ring of
     shared-memory slots, the fold, then the normalisation, whose re-read is served from L2 while
     the next rows fold. */
  SOFTMAX_VARIANT_SPLITROW_STREAM = 5
};

/*
 * softmax_rows -- y = softmax(x) along each row ("5.2 CUDA Online Softmax
 * 实现优化", §2.2, the whole method).  x and y: device, M x N, dtype.  y may
 * not overlap x unless y == x (in place).
 */
int softmax_rows(const void* x, void* y, int64_t M, int64_t N, int dtype, void* stream);

/*
 * softmax_rows_ex -- softmax_rows with optional per-row state outputs
 * (m_out, d_out, lse_out: fp32[M] or NULL) and a forced variant.  The state
 * is the (m, d) pair each row's online fold ends with ("5.2 CUDA Online
 * Softmax 实现优化", §2.1; "Softmax 数值稳定性与 IO-Aware Attention" §四, the
 * mergeable state) and LSE = m + ln d ("从原始Softmax到在线Softmax",
 * log-sum-exp); the variants are the page's kernel designs re-made for this
 * GPU: the register one-read kernel of §6, the two passes of §2.2 with the
 * vector loads of §5, and the split rows of §7.1.
 * A forced variant that needs 16-byte alignment returns SOFTMAX_ERR_MISALIGNED
 * when x, y or the row pitch N * sizeof(dtype) is not a multiple of 16;
 * AUTO never does (it falls back to scalar-access kernels).
 */
int softmax_rows_ex(const void* x, void* y, float* m_out, float* d_out, float* lse_out, int64_t M,
                    int64_t N, int dtype, int variant, void* stream);

/*
 * softmax_rows_causal -- softmax_rows_ex for rows masked by position, as in causal attention
 * scores: row r keeps its first
 *     L_r = clamp(r % q_period + 1 + key_offset, 0, N)
 * entries (query q = r % q_period sees keys 0 .. q + key_offset; key_offset = 0 when queries and
 * keys have the same length), and entries j >= L_r count as -inf.  Masked entries are never read
 * -- their bytes may hold anything -- and y is 0 there, so each row reads L_r elements instead of
 * N: the block skipping of FlashAttention-2 ("Softmax 数值稳定性与 IO-Aware Attention" §八,
 * skipping the causal mask's invalid blocks) applied to the plain softmax.  A row with L_r = 0
 * gives y = 0, m = -inf, d = 0, LSE = -inf.  q_period >= 1 (else SOFTMAX_ERR_INVALID_ARG); other
 * arguments as softmax_rows_ex.  Rows of at most 16 KiB (16-byte aligned) run one warp per row
 * loading only the live prefix; other rows run the two-pass kernel over the live prefix.
 */
int softmax_rows_causal(const void* x, void* y, float* m_out, float* d_out, float* lse_out, int64_t M,
                        int64_t N, int64_t q_period, int64_t key_offset, int dtype, void* stream);

/* Flags of softmax_rows_strided. */
enum softmax_flags { SOFTMAX_FLAG_LOG = 1 /* y = log softmax instead of softmax */ };

/*
 * softmax_rows_strided -- softmax_rows_ex with a row pitch, a scale and an output choice:
 *     y[r, j] = softmax(scale * x[r, :])_j        (flags = 0)
 *     y[r, j] = log softmax(scale * x[r, :])_j    (flags = SOFTMAX_FLAG_LOG)
 * for r < M, j < N, where row r of x starts at element r * ldx and row r of y at r * ldy (a
 * column block of a wider matrix, or rows with padding).  The scale folds into the exponent slope
 * (scale * log2 e), as attention's 1/sqrt(d) does, at no cost per element; the state outputs
 * describe scale * x: m_out = scale * max_j x[r, j] (rounded once, the maximum of the rounded
 * products), d_out relative to it, LSE = m_out + ln d.
 *   ldx, ldy -- row pitches in ELEMENTS, >= N (0 means N).
 *   scale    -- finite and > 0 (else SOFTMAX_ERR_INVALID_ARG); 1 gives softmax_rows_ex's result.
 *   flags    -- 0 or SOFTMAX_FLAG_LOG.
 *   variant  -- AUTO, ONEREAD_REG, ONEREAD_SMEM (the CTA bulk-copy kernel; for contiguous rows
 *               at scale 1 beyond its reach, the cluster kernel that holds each row on chip) or
 *               TWOPASS; SPLITROW gives SOFTMAX_ERR_UNSUPPORTED.  The vector and bulk-copy paths also need ldx * s and
 *               ldy * s to be multiples of 16 bytes (a forced ONEREAD_SMEM otherwise returns
 *               SOFTMAX_ERR_MISALIGNED; AUTO takes the scalar paths).
 * x and y may be the same matrix (x == y, ldx == ldy); other overlaps are undefined.  Other
 * arguments and errors as softmax_rows_ex.
 */
int softmax_rows_strided(const void* x, int64_t ldx, void* y, int64_t ldy, float* m_out, float* d_out,
                         float* lse_out, int64_t M, int64_t N, int dtype, float scale, int flags, int variant,
                         void* stream);

/*
 * log_softmax_rows -- y = log softmax(x) row by row: y_j = x_j - LSE with LSE = m + ln d
 * ("从原始Softmax到在线Softmax", section "softmax实际代码实现": log_probs = logits - max -
 * log(sum_exp), the step before the cross-entropy loss).  Computed as (x_j - m) - ln d from the
 * online state, so x is read once as for softmax.  An all -inf row gives y = -inf everywhere
 * (log 0).  Arguments, layout, outputs and errors as softmax_rows_ex; `variant` may be AUTO,
 * ONEREAD_REG, ONEREAD_SMEM (the bulk-copy kernels, and for many rows of 128 - 512 KiB and 768 KiB - 1 MiB a
 * thread-block cluster per row held on chip) or TWOPASS.  SPLITROW gives
 * SOFTMAX_ERR_UNSUPPORTED; AUTO never picks it (a single very long row runs TWOPASS).
 */
int log_softmax_rows(const void* x, void* y, float* m_out, float* d_out, float* lse_out, int64_t M,
                     int64_t N, int dtype, int variant, void* stream);

/*
 * cross_entropy_rows -- per-row cross-entropy loss against integer labels:
 *     loss[r] = LSE_r - x[r, labels[r]]  ( = -log softmax(x_r)[labels[r]] )
 * ("从原始Softmax到在线Softmax", section "softmax实际代码实现", cross_entropy_loss, and the
 * worked example "交叉熵损失计算": logits [2.0, 1.0, 0.1], label 0 -> 0.4170), evaluated as
 * (m - x_label) + ln d in the page's order (no cancellation for large |m|).  The page
 * returns the mean over rows; this call returns each row's loss (the mean is the caller's sum
 * over loss / M).  Only x is read (no y is written): one pass over each row for the online
 * state, plus the labelled element.
 *   labels  -- device, int64, M entries.  A negative label marks a row to ignore: loss = 0.
 *              A label >= N gives loss = NaN, x is not read there, and the next
 *              softmax_get_status() returns SOFTMAX_ERR_INVALID_ARG.
 *   loss    -- device, fp32, M entries (required).
 *   lse_out -- device, fp32, M entries, or NULL.
 * Other arguments and errors as softmax_row_state.
 */
int cross_entropy_rows(const void* x, const int64_t* labels, float* loss, float* lse_out, int64_t M, int64_t N,
                       int dtype, void* stream);

/*
 * attention_forward -- O = softmax(scale Q K^T) V row by row, without forming S = Q K^T in memory:
 * the blocked online recurrence of "从原始Softmax到在线Softmax" (m' = max(m, block max),
 * l = e^(m - m') l + sum e^(s - m'), o~ = e^(m - m') o~ + sum e^(s - m') v, o = o~ / l), the
 * FlashAttention forward tile of "5.2 CUDA Online Softmax 实现优化" §8.2, on the tensor cores.
 *   q       -- device, [BH][Sq][d] row-major, dtype elements.
 *   k, v    -- device, [BH][Sk][d].
 *   o       -- device, [BH][Sq][d] (written).
 *   lse_out -- device, fp32 [BH][Sq]: m + ln l of each row (natural log, of scale Q K^T), or NULL.
 *   scale   -- finite, > 0; 0 means 1/sqrt(d), attention's usual scale (rounded to fp32).
 *   causal  -- 1: query row i sees keys j <= i + Sk - Sq (the last query sees every key); 0: all.
 * A row that sees no key gets o = 0, LSE = -inf.  Supported: dtype SOFTMAX_BF16 or SOFTMAX_F16
 * with d = 64 or 128 (fp32 accumulation; P rounded to the element type for the P V product; fp16
 * weights stay below 2^8, O below max |v|); other dtypes or head sizes return
 * SOFTMAX_ERR_UNSUPPORTED, as do BH > 65535 and Sq or Sk > 2^31 - 256.
 * Pointers 16-byte aligned (else SOFTMAX_ERR_MISALIGNED).
 * BH == 0 is a no-op.  A bounded wait that runs out is reported by softmax_get_status.
 */
int attention_forward(const void* q, const void* k, const void* v, void* o, float* lse_out, int64_t BH, int64_t Sq,
                      int64_t Sk, int64_t d, float scale, int causal, int dtype, void* stream);

/*
 * The decoding step: a paged key/value cache held in 4 bits, the attention that reads it, and what is
 * done to the logits before their softmax.  (The pages stop at the attention of a prompt, "Softmax
 * 数值稳定性与 IO-Aware Attention" §八; a step with one token a sequence keeps its keys and values from
 * call to call, and the same online (m, l, o) recurrence runs over them.)
 *
 * The cache is one array of bytes, [num_pages][heads][page_size / 16][20 * head_dim]: a block holds
 * 16 tokens of one key/value head.  Each group of 32 elements of a key or value has a scale s and a
 * zero z (fp16), an element is s * c + z with a code c of 0 .. 15; 5 bits an element in all.  With
 * d = head_dim and G = d / 32, a block is
 *   [0, 8 d)      key codes: 32-bit word r (d / 8) + G t + j (token r < 16, t < 4, j < G) holds
 *                 elements 32 j + 8 t + n of token r in nibble n (bits 4 n .. 4 n + 3), n < 8;
 *   [8 d, 16 d)   value codes: 16-bit word 2 (((8 f + g) 4 + t) G + j) + e (f < 2, g < 8, t < 4, e < 2)
 *                 holds elements 32 j + 4 g + n of token 8 f + 2 t + e in nibble n, n < 4;
 *   16 d          fp16 key scales [16][G], then key zeros [16][G];
 *   16 d + 64 G   fp16 value scales [8][G][2] (token pair, group, token of the pair), then value zeros.
 * Pages belong to the caller, who gives each sequence its pages through the page table; pages may be
 * shared by sequences that only read them.
 *
 * A call handles `tokens` rows: sequence b owns rows cu_tokens[b] .. cu_tokens[b + 1] - 1, its last
 * n_b tokens in the cache, so row i is the token at position seq_lens[b] - (cu_tokens[b + 1] - i).
 * cu_tokens = NULL means one token for each sequence (tokens == batch).  Rows from cu_tokens[batch] on
 * belong to no sequence and are left as they were.
 *
 * Values on the device cannot be checked before the launch.  A page, length, position or offset out
 * of its range is never followed: it is recorded (softmax_get_status returns
 * SOFTMAX_ERR_INVALID_ARG), a row of kv4_append or kv4_gather concerned is skipped, and the sequence's
 * rows of attention_kv4 are undefined.  Where offsets descend, attention_kv4 writes no row at all.
 * A sequence that brings more rows than it has tokens has rows at positions below 0: kv4_append and
 * kv4_gather record and skip them; in attention_kv4 they see no key, and nothing is recorded.
 */
typedef struct kv4_cache {
  void* data;                /* 16-byte aligned */
  const int32_t* page_table; /* [batch][table_width]: page of tokens p * page_size .. of each sequence */
  const int32_t* seq_lens;   /* [batch]: tokens of each sequence, those of this call included */
  const int32_t* cu_tokens;  /* [batch + 1], ascending, or NULL */
  int64_t num_pages;
  int64_t page_size;         /* a multiple of 16 */
  int64_t heads;             /* key/value heads */
  int64_t head_dim;          /* 64 or 128 */
  int64_t batch;
  int64_t table_width;
  int64_t tokens;
} kv4_cache;

/* Rows [tokens][heads][head_dim] of bf16 or fp16 elements: strides in elements, multiples of 8; data
   16-byte aligned; the elements of a head lie side by side. */
typedef struct kv4_rows {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
} kv4_rows;

enum kv4_flags { KV4_FLAG_NEIGHBOURS = 1 /* rotate pairs (2 i, 2 i + 1) instead of (i, i + rotated / 2) */ };

/*
 * kv4_append -- writes this call's keys and values into the cache, keys (and queries) rotated by
 * their positions on the way.
 *   k, v      -- [tokens][heads][head_dim].
 *   q, q_out  -- [tokens][q_heads][head_dim], both or neither: q_out = q rotated (q_out may be q).
 *   cos_sin   -- fp32 [positions][rotated], 16-byte aligned: rotated / 2 cosines, then as many sines of
 *                each position; (a, b) becomes (a cos - b sin, b cos + a sin).  NULL: no rotation.
 *   rotated   -- leading elements of a head that are rotated, a multiple of 8 up to head_dim.
 * Quantisation of a group x of 32 (fp32 arithmetic, every operation rounded by itself, so a host can
 * reproduce the bytes): x limited to +-65504, z = fp16(min x), s = fp16((max x - min x) / 15),
 * c = (x - z) / s rounded to the nearest integer (ties to even) and limited to 0 .. 15, 0 where s = 0.
 * Non-finite inputs give unspecified values in their own group, and in the group of the element that
 * they are rotated with; scales and zeros in the cache are finite whatever comes in.
 * Every token needs a place of its own: two tokens of one call that fall on one place of one page
 * leave it with bytes of either.  head_dim other than 64 and 128, fp32 and sizes beyond 2^31 rows
 * or positions return SOFTMAX_ERR_UNSUPPORTED.
 */
int kv4_append(const kv4_cache* cache, const kv4_rows* k, const kv4_rows* v, const kv4_rows* q, const kv4_rows* q_out, int64_t q_heads,
               const float* cos_sin, int64_t positions, int64_t rotated, int flags, int dtype, void* stream);

/*
 * kv4_gather -- the values s * c + z of this call's tokens (whole sequences where n_b = seq_lens[b]),
 * rounded once to the element type.  k and v: [tokens][heads][head_dim], written.
 * For a prompt whose prefix is in the cache, attention_forward takes such keys and values as [heads][n][head_dim], one
 * length for a call and a key/value head for each query head: read back with head strides of tokens * head_dim, then make
 * a call for each sequence, its heads repeated q_heads / heads times, with causal = 1.
 */
int kv4_gather(const kv4_cache* cache, const kv4_rows* k, const kv4_rows* v, int dtype, void* stream);

/*
 * attention_kv4 -- O = softmax(scale Q K^T) V of this call's tokens over the cache, query head h with
 * key/value head h / (q_heads / heads).  Row i at position p sees the keys at positions 0 .. p, so the
 * call's own tokens must be in the cache (kv4_append) first.  Its bits depend on nothing else that the
 * cache or q holds: not on later tokens, other rows, or bytes where no token lies.  (Scales and zeros of
 * the sequence's tokens are finite, as kv4_append leaves them.)
 *   q         -- [tokens][q_heads][head_dim], bf16 or fp16; finite, with |scale q.k| below 10^6.
 *   o         -- [tokens][q_heads][head_dim], contiguous, written.
 *   lse_out   -- fp32 [tokens][q_heads]: m + ln l of each row (natural log, of scale Q K^T), or NULL.
 *   q_heads   -- a multiple of heads.
 *   scale     -- finite, > 0; 0 means 1/sqrt(head_dim).
 *   workspace -- device memory of at least attention_kv4_workspace(...) bytes, 256-byte aligned, that
 *                no other call uses until this one is done (calls that may run at the same time, captured
 *                graphs among them, need one each).  Nothing in it is kept from call to call.
 * Built for a few tokens a sequence (decoding, drafts): any number is right, but a long prompt runs
 * faster through attention_forward on 16-bit keys and values.  Scores and row states are fp32.  For the
 * product with V a weight is rounded to fp16, and so is its product with a scale of V: 2^-11 of each (in
 * fp16 the second remainder goes on to a later token that the row sees).  The largest weight is held at
 * 2^(9 - e) or more, 2^e the smallest power of two >= 1 not below the scales of V that the row has seen:
 * weights down to 2^-(33 - e) of the largest count.  Scales of V below 2^-14 (values of some 10^-3 at most)
 * lose bits of the products with small weights.  A row that sees no key gets o = 0, LSE = -inf.
 */
int attention_kv4(const kv4_cache* cache, const kv4_rows* q, void* o, float* lse_out, int64_t q_heads, float scale, int dtype,
                  void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace for attention_kv4 on the current device; -1 for sizes that it refuses. */
int64_t attention_kv4_workspace(int64_t batch, int64_t tokens, int64_t q_heads, int64_t heads, int64_t head_dim);

/*
 * logits_process_rows -- penalties for repeated tokens, biases and a mask on M rows of N logits, with
 * the softmax or log softmax that follows in the same pass.  For token j of a row, c its count among
 * the row's generated tokens, "seen" if it is among its prompt or generated tokens:
 *     l = x_j
 *     l = l > 0 ? l / repetition : l * repetition      where j is seen
 *     l = l - (frequency * c + presence)               where c > 0
 *     l = l + (biases of j, added up in list order)
 *     l = l * scale
 *     l = -inf                                         where j's mask bit is 0
 * y = l, softmax(l) or log softmax(l).  A row whose entries are all -inf gives softmax 0, log softmax
 * -inf, LSE -inf.
 *   x, y        -- rows at pitches ldx, ldy in elements (0: N); y may be x (with ldx == ldy).
 *   lse_out     -- fp32 [M]: LSE of l, or NULL.
 *   tokens      -- int32 [M][token_width]: a row's prompt, then its generated tokens; negative entries
 *                  count as absent.  NULL: no penalties.  token_width < 2^20.
 *   prompt_lens -- int32 [M]: how many of them are the prompt (NULL: 0).
 *   token_lens  -- int32 [M]: how many there are, prompt included.
 *   repetition, frequency, presence, scale -- fp32 [M] each, or NULL for 1, 0, 0, 1; repetition and
 *                  scale > 0.
 *   bias_ids, bias_values -- int32 and fp32 [M][bias_count], negative ids count as absent; at most 1024.
 *   mask        -- 32-bit words [M][ld_mask] (0: ceil(N / 32)), bit j % 32 of word j / 32 is set where j is
 *                  allowed; NULL: all.
 * Every pointer is aligned to its elements (else SOFTMAX_ERR_MISALIGNED).
 * A token or bias id >= N is ignored, and softmax_get_status returns SOFTMAX_ERR_INVALID_ARG, as it does
 * for lengths outside 0 <= prompt <= all <= token_width (which are limited to that range).
 * Arithmetic is fp32; the results do not depend on the order in which the GPU counts.
 */
typedef struct logits_rows {
  const void* x;
  int64_t ldx;
  void* y;
  int64_t ldy;
  float* lse_out;
  const int32_t* tokens;
  int64_t token_width;
  const int32_t* prompt_lens;
  const int32_t* token_lens;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const int32_t* bias_ids;
  const float* bias_values;
  int64_t bias_count;
  const uint32_t* mask;
  int64_t ld_mask;
  const float* scale;
} logits_rows;

enum logits_out { LOGITS_OUT_LOGITS = 0, LOGITS_OUT_SOFTMAX = 1, LOGITS_OUT_LOG_SOFTMAX = 2 };

int logits_process_rows(const logits_rows* a, int64_t M, int64_t N, int dtype, int out, void* stream);

/*
 * The training step around the matrix products: the loss of the logits with its gradient, the
 * root-mean-square norm of rows and its backward pass, embedding lookup and its gradient, the norm of all
 * gradients and clipping.  (The pages give the loss, "从原始Softmax到在线Softmax", section "softmax实际代码实现",
 * and stop at the forward pass; the gradients are the derivatives of the formulas stated here.)
 *
 * Rows lie at pitches (ld..., in elements, >= N, 0: N).  Every pointer is aligned to its elements (else
 * SOFTMAX_ERR_MISALIGNED); any length and pitch is taken, and runs faster where rows start on 16-byte
 * boundaries.  Sums are held in fp32, added up in an order that the sizes, pitches, alignments and tokens fix: the same
 * call gives the same bits.  A matrix that a call writes in place of another has that one's pitch (else
 * SOFTMAX_ERR_INVALID_ARG); other overlaps are undefined.  Each workspace is device memory, 256-byte aligned, that no other call uses until this one is done
 * (calls that may run at the same time, captured graphs among them, need one each); nothing in it is kept from
 * call to call.  A count of rows, tokens or tensors of 0 is a no-op unless an output is left to be written.
 */

/*
 * cross_entropy_rows_grad -- the loss of cross_entropy_rows and its gradient, x read once where a row fits on
 * chip.  For each row with label t, p = softmax(x), LSE = m + ln d, and e = label_smoothing, z = z_loss:
 *     loss = (1 - e) (LSE - x_t) + e mean_j (LSE - x_j) + z LSE^2
 *     grad_j = w (p_j (1 + 2 z LSE) - (1 - e) [j = t] - e / N),     w = grad_scale * upstream
 * that is, grad = d(sum_r grad_scale * upstream_r * loss_r) / dx.
 *   x          -- [M][N] at pitch ldx.
 *   labels     -- int64 [M].  A negative label marks a row to ignore: loss = 0 and grad = 0, whatever x holds.  A
 *                 label >= N gives loss = NaN and a grad of NaN, and softmax_get_status returns
 *                 SOFTMAX_ERR_INVALID_ARG.
 *   upstream   -- fp32 [M], the gradient of what is minimised by each row's loss, or NULL for 1.
 *   grad_scale -- finite; 1 / rows for a mean, times a loss scale.
 *   label_smoothing -- in [0, 1).    z_loss -- finite, >= 0.
 *   grad       -- [M][N] at pitch ldg, dtype elements; may be x (with ldg == ldx), other overlaps are undefined.
 *   loss       -- fp32 [M].   lse_out -- fp32 [M] or NULL (every row's, ignored ones too).
 * Masked entries (-inf) have p = 0; a masked label gives loss = +inf, and so does smoothing over masked entries; their
 * gradients stay finite.  A row whose entries are all -inf gives NaN unless it is ignored.
 */
int cross_entropy_rows_grad(const void* x, int64_t ldx, const int64_t* labels, const float* upstream, float grad_scale,
                            float label_smoothing, float z_loss, void* grad, int64_t ldg, float* loss, float* lse_out,
                            int64_t M, int64_t N, int dtype, void* stream);

/*
 * rms_norm_rows -- M rows of N: h = x + residual (rounded to the element type, which is what the norm is taken of),
 *     rstd = 1 / sqrt(mean_j h_j^2 + eps),     y_j = h_j rstd (weight_j + offset)
 *   x, residual -- residual may be NULL (h = x).
 *   sum_out     -- h; required with a residual, NULL without one.  May be x or residual (with its pitch).
 *   weight      -- [N], dtype elements or fp32 (weight_f32 = 1), or NULL for 1 - offset.
 *   eps         -- finite, >= 0.   offset -- finite (1 where weights are kept as their difference from 1).
 *   y           -- out = RMS_NORM_OUT_SAME: dtype elements.  May be x, or residual, where sum_out is not.
 *                  out = RMS_NORM_OUT_E4M3 (y a matrix of its own): 8-bit floats (e4m3, largest 448), with fp32 scales: the value is
 *                  code * scale, scale = max(max |y| / 448, 2^-126) over a group, code = y / scale rounded to the nearest
 *                  (ties to even): of bf16 elements and weights with offset 0, that of the exact quotient, in which rstd
 *                  cancels out (above the least scale).
 *   scales      -- e4m3 only: [M][groups], groups = 1 for group = 0 (a scale for each row), else ceil(N / group).
 *   group       -- 0 or 128 (the last group of a row may be shorter).
 *   rstd_out    -- fp32 [M] or NULL; the backward pass reads it.
 * Squares are added up in fp32: rows of magnitudes up to 1e17, and with eps = 0 down to 1e-18, here and in the backward
 * pass; beyond them rstd is 0 or inf.
 */
typedef struct rms_norm_args {
  const void* x;
  int64_t ldx;
  const void* residual;
  int64_t ld_residual;
  void* sum_out;
  int64_t ld_sum;
  const void* weight;
  int64_t weight_f32;
  void* y;
  int64_t ldy;
  float* scales;
  int64_t group;
  float* rstd_out;
  float eps;
  float offset;
} rms_norm_args;

enum rms_norm_out { RMS_NORM_OUT_SAME = 0, RMS_NORM_OUT_E4M3 = 1 };

int rms_norm_rows(const rms_norm_args* a, int64_t M, int64_t N, int dtype, int out, void* stream);

/*
 * rms_norm_rows_backward -- with xhat = h rstd and g = dy (weight + offset):
 *     dx_j = rstd (g_j - xhat_j mean_i(g_i xhat_i)) + sum_grad_j      (of x and of residual alike)
 *     dweight_j = sum_r dy_rj xhat_rj
 *   dy, h, sum_grad -- [M][N]: the gradient of y; the sum that the norm was taken of; the gradient that reaches
 *                 that sum by its other uses, or NULL.
 *   rstd       -- fp32 [M], from the forward pass.
 *   weight, weight_f32, offset -- as in the forward pass.
 *   dx         -- [M][N]; may be dy, h or sum_grad (with its pitch).
 *   dweight    -- fp32 [N], or NULL.  accumulate = 1 adds to what it holds, 0 overwrites it.
 *   workspace  -- at least rms_norm_backward_workspace(M, N, dtype) bytes (with dweight; else unused).
 */
typedef struct rms_norm_grad_args {
  const void* dy;
  int64_t ld_dy;
  const void* h;
  int64_t ldh;
  const void* sum_grad;
  int64_t ld_sum_grad;
  const float* rstd;
  const void* weight;
  int64_t weight_f32;
  void* dx;
  int64_t ld_dx;
  float* dweight;
  int64_t accumulate;
  float offset;
} rms_norm_grad_args;

int rms_norm_rows_backward(const rms_norm_grad_args* a, int64_t M, int64_t N, int dtype, void* workspace,
                           int64_t workspace_bytes, void* stream);

/* Bytes of workspace on the current device; -1 for sizes that the call refuses. */
int64_t rms_norm_backward_workspace(int64_t M, int64_t N, int dtype);

/*
 * embedding_rows -- y_t = scale * table[tokens_t]: T rows of D elements out of a table of V rows.
 *   tokens -- int32 (token_bytes = 4) or int64 (8), [T].  A negative token is padding: its row is 0.  A token >= V
 *             gives a row of NaN, is not followed, and softmax_get_status returns SOFTMAX_ERR_INVALID_ARG.
 *   scale  -- finite; the product is rounded once.
 * D up to 2^30 (else SOFTMAX_ERR_UNSUPPORTED), here and in the backward pass.
 */
int embedding_rows(const void* table, int64_t ld_table, const void* tokens, int token_bytes, void* y, int64_t ldy,
                   int64_t T, int64_t V, int64_t D, float scale, int dtype, void* stream);

/*
 * embedding_rows_backward -- grad_v = scale * sum over the t with tokens_t = v of dy_t, [V][D] dense: rows that no
 * token names are 0.  accumulate = 1: added to what grad holds (in fp32, then rounded), and rows that no token
 * names are neither read nor written.  The tokens are sorted on the device; a row's sum runs over its tokens in
 * their order, in parts where there are many.
 *   dy         -- [T][D], dtype elements.   grad -- [V][D], grad_dtype elements: fp32 or dtype's.
 *   tokens     -- as in embedding_rows: padding gives no gradient, nor does a token >= V (which is recorded).
 *   workspace  -- at least embedding_backward_workspace(T, V, D) bytes.
 * T up to 2^24, V up to 2^31 - 2 (else SOFTMAX_ERR_UNSUPPORTED).
 */
int embedding_rows_backward(const void* dy, int64_t ld_dy, const void* tokens, int token_bytes, void* grad,
                            int64_t ld_grad, int64_t T, int64_t V, int64_t D, float scale, int accumulate, int dtype,
                            int grad_dtype, void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace; -1 for sizes that the call refuses. */
int64_t embedding_backward_workspace(int64_t T, int64_t V, int64_t D);

/* One tensor of a list: n contiguous elements, and where their scaled values go (out may be grad where the types are
   one; grad_norm does not look at it).  out_dtype: fp32 or dtype. */
typedef struct grad_tensor {
  const void* grad;
  void* out;
  int64_t n;
  int32_t dtype;
  int32_t out_dtype;
} grad_tensor;

/*
 * grad_norm -- norm_out = |scale| sqrt(sum of the squares of all elements of count tensors), fp32.  Squares are taken in
 * fp32, a few dozen at a time, and in fp64 where those run over fp32's range or fall below it: neither large nor small
 * values are lost.  +inf or NaN where an element is not finite (or the norm is above fp32's range).
 * clip_grad_norm -- the same, and
 *     out = grad * scale * min(1, max_norm / norm)
 * for each tensor, the factor in more than fp32's bits and the product rounded once.  Where the norm is inf or NaN nothing is limited: out = grad * scale.  A tensor in
 * place (out == grad) whose factor is 1 is neither read again nor written.
 *   tensors   -- HOST array of count entries (at most 2^20, 2^42 elements in all), read before the call returns.  What
 *                clip_grad_norm writes overlaps no other tensor of the list, read or written, nor its own gradient in part (else
 *                SOFTMAX_ERR_INVALID_ARG).
 *   scale     -- finite: 1 / (loss scale), 1 / (accumulated steps).   max_norm -- finite, > 0.
 *   norm_out  -- fp32 [1], device.
 *   workspace -- at least grad_norm_workspace(count) bytes.
 */
int grad_norm(const grad_tensor* tensors, int64_t count, float scale, float* norm_out, void* workspace,
              int64_t workspace_bytes, void* stream);
int clip_grad_norm(const grad_tensor* tensors, int64_t count, float scale, double max_norm, float* norm_out, void* workspace,
                   int64_t workspace_bytes, void* stream);

/* Bytes of workspace on the current device; -1 for a count that the calls refuse. */
int64_t grad_norm_workspace(int64_t count);

/*
 * softmax_row_state -- only the per-row state (m, d) and LSE: the first pass
 * of the online method ("5.2 CUDA Online Softmax 实现优化", §2.2, pass 1;
 * "Softmax 数值稳定性与 IO-Aware Attention" §四, the mergeable state).  Reads x
 * once; writes 12 bytes per row at most.  At least one of m_out, d_out,
 * lse_out must be non-NULL.  With merge_states this lets a caller fold a row
 * in pieces.
 */
int softmax_row_state(const void* x, float* m_out, float* d_out, float* lse_out, int64_t M,
                      int64_t N, int dtype, void* stream);

/*
 * merge_states -- elementwise merge of two arrays of row states
 * ("5.2 CUDA Online Softmax 实现优化", §4.1; "Softmax 数值稳定性与 IO-Aware
 * Attention" §4.1):  m = max(m_a, m_b),  d = d_a e^(m_a - m) + d_b e^(m_b - m),
 * with (-inf, 0) the identity.  Inputs: fp32[M] device arrays (all required).
 * Outputs: fp32[M] device arrays, m_out and d_out required, lse_out optional.
 * Outputs may alias the inputs of the same index (in place).
 */
int merge_states(const float* m_a, const float* d_a, const float* m_b, const float* d_b,
                 float* m_out, float* d_out, float* lse_out, int64_t M, void* stream);

/*
 * softmax_rows_host -- softmax_rows on HOST buffers (x_host, y_host: M x N of
 * dtype).  When both buffers are page-locked (cudaHostAlloc / cudaHostRegister,
 * e.g. torch pin_memory) and rows are at most 32 KiB, the register one-read
 * kernel reads x and writes y in host memory directly over the host link
 * (zero-copy).  Otherwise row blocks of about 8 MiB are copied host->device,
 * normalised in place on the GPU and copied back, with the copies and kernels
 * of consecutive blocks overlapped on three internal streams; those streams and
 * the device staging buffers (3 x one block) are created on the first call on
 * a device and kept until the process exits, and concurrent calls on one
 * device are serialised.  Returns when y_host holds the result (the call
 * synchronises).  `stream` orders the work after earlier work on that stream.
 */
int softmax_rows_host(const void* x_host, void* y_host, int64_t M, int64_t N, int dtype,
                      void* stream);

/*
 * softmax_rows_splitrow_noalloc -- the split-row softmax (SOFTMAX_VARIANT_SPLITROW, with the same
 * choice between the on-chip and the streaming kernel) for callers that cannot allocate device
 * memory.  The pages describe no such call; it exists for callers
 * such as code held to a device-memory budget fixed in advance, code whose framework allocator
 * owns the device memory, or host threads that must not make a call that may block or
 * synchronise the device.  It allocates nothing (no cudaMalloc, cudaMallocAsync, cudaFree or
 * library allocator): the exchange scratch lives in a fixed 320 KiB device array inside the
 * library (40960 slots of 8 bytes), present on every device that loads the library until the
 * process exits.
 *  - Arguments as softmax_rows_ex (device pointers; x, y 16-byte aligned with N * sizeof(dtype)
 *    a multiple of 16, else SOFTMAX_ERR_MISALIGNED).
 *  - Capacity: M x (number of clusters) <= 40960 slots; with the 19 clusters of 8 CTAs used on a
 *    152-SM GB300 that is M <= 2155 rows (at least 512 rows with up to 80 clusters).  Larger M,
 *    or rows the split kernel cannot take, return SOFTMAX_ERR_UNSUPPORTED without launching.
 *  - The first call on a device looks up the array's device address (cudaGetSymbolAddress, with
 *    that device current) and keeps it; make that first call before any stream capture.
 *  - Like SOFTMAX_VARIANT_SPLITROW it needs every SM of the GPU: kernels running beside it on
 *    other streams can keep its clusters off the GPU until the exchange wait runs out, and the
 *    call then reports SOFTMAX_ERR_TIMEOUT (through softmax_get_status) with y undefined.
 *  - Every call shares the one array and resets the part it uses (a cudaMemsetAsync on `stream`
 *    before the kernel); calls whose executions overlap on the GPU -- on different streams, or
 *    from different threads -- race on it and must be serialised by the caller.
 */
int softmax_rows_splitrow_noalloc(const void* x, void* y, float* m_out, float* d_out, float* lse_out,
                                  int64_t M, int64_t N, int dtype, void* stream);

/*
 * softmax_get_status -- synchronises `stream`, then returns and clears the
 * status word of the current device: SOFTMAX_OK, or the error a kernel
 * recorded since the last call (SOFTMAX_ERR_TIMEOUT for a bounded wait that
 * ran out, which takes precedence; SOFTMAX_ERR_INVALID_ARG for a cross-entropy
 * label >= N, or a page, token, length or position that a call of the decoding
 * or the training step found out of range).  SOFTMAX_ERR_CUDA if the synchronisation itself failed.
 */
int softmax_get_status(void* stream);

/* A static, human-readable name for a status code. */
const char* softmax_status_string(int status);

/* The CUDA error string of the last SOFTMAX_ERR_CUDA on this host thread ("" if none). */
const char* softmax_last_cuda_error(void);

/* The variant (enum softmax_variant) the last successful compute call on this host thread ran. */
int softmax_last_variant(void);

/*
 * softmax_debug_set_fault -- test hook.  fault = 1 makes the next
 * split-row launches skip one cluster's state publication, so every other
 * cluster's bounded wait runs out and the kernel records SOFTMAX_ERR_TIMEOUT
 * instead of hanging; fault = 2 makes the next attention_forward launches with
 * at most 256 keys (Sk <= 256, two key tiles) skip the copy of the first V
 * tile, with the same outcome (the output is then undefined); longer key
 * sequences ignore it.  fault = 0 restores normal behaviour.  Returns the
 * previous value.  Process-wide; not for production use.
 */
int softmax_debug_set_fault(int fault);

/* The wait limit of the split-row exchange and of every wait in attention_forward, in nanoseconds
 * (default 200 ms).  Returns the old value. */
int64_t softmax_debug_set_wait_limit_ns(int64_t ns);

#ifdef __cplusplus
}
#endif

#endif /* ROW_WISE_ONLINE_SOFTMAX_ROWS_H */
