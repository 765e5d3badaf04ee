/*
 * q4g128.h -- C ABI of the int4 group-128 weight-streaming GEMV library for
 * AMD Instinct MI355X (gfx950).
 *
 * Weight format (rumik-oss-1 int4 write-up, rtts.neoandmatrix.me, section
 * "Step 3: an int4 file and a first kernel on the laptop"): a projection
 * matrix W with N output rows and K input columns is quantised in groups of
 * 128 consecutive columns of each row; every group has one fp16 scale and
 * one fp16 minimum, and two 4-bit codes share one byte.  The dequantised
 * weight is
 *
 *     w[n][k] = code[n][k] * scale[n][k / 128] + min[n][k / 128].
 *
 * Canonical layout used by every entry point (readings of the format that
 * the pages leave open are stated here once):
 *   packed  uint8  [N][K/2]  row-major; byte j of row n holds code[n][2j] in
 *                            bits 0..3 and code[n][2j+1] in bits 4..7.
 *   scales  uint16 [N][K/128] row-major fp16 bit patterns.
 *   mins    uint16 [N][K/128] row-major fp16 bit patterns.
 *   x / X   uint16 [B][K]    row-major fp16 bit patterns, one activation
 *                            vector (request or prompt token) per row.
 *   y / Y   float  [B][N]    row-major fp32 results; Y = X * W^T.
 *
 * Ownership and execution model (all entry points):
 *   - Every pointer is DEVICE memory owned by the caller (except the
 *     grouped call's descriptor array, a host array).  The library never
 *     allocates or frees device memory and keeps no pointer after returning;
 *     only the attention calls need a workspace, which the caller gives, and
 *     only the grouped call uses host memory of its own, for checking its
 *     descriptors during the call.
 *   - `stream` is a hipStream_t (NULL = the null stream).  Calls only enqueue
 *     work; they never synchronise the host.  Buffers must stay alive until
 *     the enqueued work completes.
 *   - Outputs are fully overwritten, but for caches and rows that a call is said to
 *     leave alone, and must not overlap any input.
 *   - Arguments are validated on the host before any HIP call; an invalid
 *     call enqueues nothing.
 *   - Results are deterministic: fixed reduction orders; the only atomics
 *     count finished workgroups.
 *
 * Limits: 1 <= N <= 2^31 - 256; K a multiple of 128 with 128 <= K <= 32768;
 * batch / prompt rows at most 2^31 - 256.
 */
#ifndef Q4G128_H
#define Q4G128_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t q4_status;

/* Only the entry points below are exported from libq4g128.so. */
#define Q4_API __attribute__((visibility("default")))

#define Q4_OK 0
/* NULL pointer, N <= 0, B outside [1, 16], M <= 0, or an output that
   overlaps an input; for the cache and attention calls also an option outside
   its range or a workspace that is too small. */
#define Q4_EINVAL (-1)
/* K not a positive multiple of 128, K above 32768, or N / M above
   Q4G128_MAX_N; for the cache and attention calls a size outside the limits
   stated with them. */
#define Q4_ESHAPE (-2)
/* codes / packed / x / X / W not 16-byte aligned; scales / mins not 2-byte
   aligned; y / Y not 4-byte aligned.  For the cache and attention calls: qkv, k,
   v, latent rows, kv, q, q_main, q_rot, out and workspace not 16-byte, norms not
   2-byte, masks not 8-byte, other arrays not 4-byte aligned. */
#define Q4_EALIGN (-3)
/* The HIP runtime reported an error while querying the device or launching;
   q4g128_last_hip_error() returns the hipError_t of the calling thread. */
#define Q4_EDEVICE (-4)

#define Q4G128_GROUP 128
#define Q4G128_MAX_K 32768
#define Q4G128_MAX_BATCH 16
#define Q4G128_MAX_N 0x7FFFFF00LL
#define Q4G128_INT8_MAX_K 8192
/* Limits of the cache and attention calls. */
#define Q4G128_MAX_HEADS 1024
#define Q4G128_MAX_GROUP 64
#define Q4G128_MAX_TOKENS 1048576
#define Q4G128_MAX_SEQUENCES 65536
#define Q4G128_MAX_DRAFT 64
#define Q4G128_ATTN_COUNTER_BYTES 4096
#define Q4G128_LATENT_ROT 64
#define Q4G128_LATENT_MAX_MAIN 1024

/*
 * q4g128_pack -- two codes per byte.
 *   codes  [N][K] uint8, only the low 4 bits of each code are used.
 *   packed [N][K/2] uint8, written.
 * The export step of the rumik write-up ("Step 3": a short CPU job wrote the
 * int4 file) in device form; untimed set-up, not part of the decode step.
 */
Q4_API q4_status q4g128_pack(const uint8_t* codes, uint8_t* packed,
                      int64_t n, int64_t k, void* stream);

/*
 * q4g128_gemm_prefill_epilogue -- the same Y[m][n] = sum_k w[n][k] * X[m][k]
 * in the form of the rumik write-up's prefill ("Step 8: a prefill that
 * stays int4"): each 128-column group is unpacked on chip to exact integer
 * codes and contracted with the activations on the matrix cores (fp32
 * accumulation), and the group's scale and minimum are applied to that
 * result: Y += scale * sum(code*x) + min * sum(x).  No weight is rounded to
 * fp16, so results carry only fp32 summation error (within 512 * 2^-24 *
 * sum_k |w*x| of the exact product).  Same arguments, limits, errors and
 * execution model as q4g128_gemm_prefill; any M >= 1.
 */
Q4_API q4_status q4g128_gemm_prefill_epilogue(const uint8_t* packed, const uint16_t* scales,
                                       const uint16_t* mins, const uint16_t* X, float* Y,
                                       int64_t n, int64_t k, int64_t m, void* stream);

/*
 * q4g128_quantize -- export float32 weights to the format above.
 * The rumik write-up ("Step 3") exports every projection with a short CPU
 * job: groups of 128 columns, one fp16 scale and one fp16 minimum per group.
 * The pages give no formula; the reading implemented is the min/max affine
 * quantiser that the dequantisation w = code*scale + min implies.  For each
 * group, with every step one IEEE fp32 operation rounded to nearest even:
 *     lo = min, hi = max of the group's 128 values
 *     min   = fp16(lo + 0)            (a zero minimum is stored as +0)
 *     scale = fp16((hi - lo) / 15)
 *     code  = clamp(round_half_even((w - min) / scale), 0, 15) against the
 *             stored fp16 min and scale; code 0 everywhere if scale == 0.
 *   W      [N][K] float32, row-major, finite with |w| <= 65504 (other values
 *          give unspecified codes, never a fault).
 *   packed [N][K/2], scales [N][K/128], mins [N][K/128]: written in full.
 * Errors: Q4_EINVAL for a NULL pointer, N <= 0 or outputs that overlap W or
 * each other; Q4_ESHAPE for K outside the limits or more than 2^36 groups;
 * Q4_EALIGN unless W and packed are 16-byte and scales / mins 2-byte
 * aligned.  Untimed set-up work, not part of the decode step.
 */
Q4_API q4_status q4g128_quantize(const float* W, uint8_t* packed, uint16_t* scales,
                          uint16_t* mins, int64_t n, int64_t k, void* stream);

/*
 * q4g128_gemv -- y[n] = sum_k w[n][k] * x[k]   (batch-1 decode product).
 * The operation that dominates batch-1 decoding in the rumik write-up
 * ("Step 3" and "Step 7: why the GEMV was stuck, and a CUDA kernel"): the
 * packed weights are streamed once, dequantised in registers and multiplied
 * by the fp16 activation vector with fp32 accumulation.
 *   packed [N][K/2], scales [N][K/128], mins [N][K/128], x [K] -> y [N] fp32.
 */
Q4_API q4_status q4g128_gemv(const uint8_t* packed, const uint16_t* scales,
                      const uint16_t* mins, const uint16_t* x, float* y,
                      int64_t n, int64_t k, void* stream);

/*
 * q4g128_gemv_grouped -- many independent batch-1 products in few launches:
 *   for every i < count:  descs[i].y = W_i * descs[i].x   (as q4g128_gemv).
 * The rumik write-up ("A detour: the laptop engine on an H100") measures a
 * small projection at about one launch latency on a fast GPU and a decode
 * step as launch-bound, and advises counting launches and issuing far fewer
 * kernels per layer ("What I would tell someone starting this").  Here all
 * projections whose K has the same pass mapping are streamed by one
 * persistent launch of up to 64 projections; the projections are read from
 * `descs` (a HOST array, read during the call and not kept).
 *   descs[i]: packed, scales, mins, x, y, n, k with the layout, alignment and
 *   limits of q4g128_gemv.
 * Every y_i is bit-identical to q4g128_gemv on projection i (same lanes,
 * chunk order and reductions per row).  The projections must be
 * independent: no y_i may overlap any input of any projection or any other
 * output (x and weights may be shared between projections).  The order in
 * which projections execute is unspecified.
 * Errors: Q4_EINVAL for descs == NULL, count < 1 or count above
 * Q4G128_MAX_GROUPED, or any overlap above; every descriptor is checked as
 * q4g128_gemv checks its arguments (first failing status returned), all
 * before any HIP call.  Q4_EDEVICE: a launch failed; projections enqueued
 * before it stay enqueued.
 */
typedef struct q4g128_gemv_desc {
    const uint8_t* packed;   /* [n][k/2] */
    const uint16_t* scales;  /* [n][k/128] fp16 */
    const uint16_t* mins;    /* [n][k/128] fp16 */
    const uint16_t* x;       /* [k] fp16 */
    float* y;                /* [n] fp32, written in full */
    int64_t n;
    int64_t k;
} q4g128_gemv_desc;

#define Q4G128_MAX_GROUPED 65536

Q4_API q4_status q4g128_gemv_grouped(const q4g128_gemv_desc* descs, int64_t count, void* stream);

/*
 * q4g128_gemm_small_batch -- Y[b][n] = sum_k w[n][k] * X[b][k], 1 <= B <= 16.
 * Continuous request batching ("Adding GPU backends to a pure-C TTS engine:
 * Metal, CUDA, and the rented-Mac trick", batching passage): each weight row
 * is read once and used for all B requests.  Row b of Y is bit-identical to
 * q4g128_gemv(X[b]) on the same weights (the same page's lesson on matching
 * the single-stream accumulation order): the arithmetic per output depends
 * on (N, K) only, never on B.
 *   X [B][K] fp16 -> Y [B][N] fp32.
 */
Q4_API q4_status q4g128_gemm_small_batch(const uint8_t* packed, const uint16_t* scales,
                                  const uint16_t* mins, const uint16_t* X, float* Y,
                                  int64_t n, int64_t k, int64_t b, void* stream);

/*
 * q4g128_gemm_prefill -- Y[m][n] = sum_k w[n][k] * X[m][k] for M prompt
 * tokens (rumik write-up, "Step 8: a prefill that stays int4": the weights
 * stay int4 in memory and are unpacked on chip for a matrix-core product).
 * Each weight is dequantised on chip to fp16, fp16(code*scale + min) with
 * one rounding, and contracted with the fp16 activations on the gfx950
 * matrix cores with fp32 accumulation.  M is a runtime argument (any
 * M >= 1, no re-specialisation per M).
 * Accuracy contract: |Y - Y16| <= 256 * 2^-24 * sum_k |fp16(w) * x| where Y16
 * is the exact product of the fp16-rounded weights; against the exact
 * weights the error adds the rounding of each weight, up to 2^-11 * |w|.
 * That term does not shrink with K: at short K (K = 128, one group per row)
 * and millions of outputs a few outputs exceed a 2e-3 relative bound of the
 * exact product (a few per 8 M outputs in tests).  Callers that need the
 * exact-weight accuracy at every output use q4g128_gemm_prefill_epilogue,
 * which keeps exact codes.  Results are not bit-identical to q4g128_gemv.
 *   X [M][K] fp16 -> Y [M][N] fp32.
 */
Q4_API q4_status q4g128_gemm_prefill(const uint8_t* packed, const uint16_t* scales,
                              const uint16_t* mins, const uint16_t* X, float* Y,
                              int64_t n, int64_t k, int64_t m, void* stream);

/*
 * q4g128_gemv_int8 -- y[n] = scale[n] * sum_k q[n][k] * x[k]  (int8 output head).
 * The rumik write-up moved the audio output head to int8 with a kernel of its
 * own: int4 group-128 was measurably too lossy there (the passage on the
 * remaining per-token time after the 36 layers, and "What I would tell
 * someone starting this").  The pages give no int8 layout; the reading
 * implemented is per-row symmetric int8:
 *   q      [N][K] int8, row-major, every value -128..127 accepted;
 *   scales [N] fp16 bit patterns, one per output row;
 *   x      [K] fp16;  y [N] fp32, written in full.
 * Products q*x are exact; sums are fp32 in a fixed order (deterministic).
 * Errors: Q4_EINVAL for a NULL pointer, N <= 0 or y overlapping an input;
 * Q4_ESHAPE unless K is a multiple of 128 with 128 <= K <= 8192 and
 * N <= Q4G128_MAX_N; Q4_EALIGN unless q and x are 16-byte, scales 2-byte
 * and y 4-byte aligned; Q4_EDEVICE as for the other entry points.
 */
Q4_API q4_status q4g128_gemv_int8(const int8_t* q, const uint16_t* scales, const uint16_t* x,
                           float* y, int64_t n, int64_t k, void* stream);

/*
 * Attention between the fused projection and o_proj: calls over one paged
 * key-value cache.
 *
 * The cache is a pool of pages of `page` token positions each; page number
 * table[s][i] holds positions i*page .. i*page + page-1 of sequence s.
 *   k      fp16 [pages][kv_heads][page][dim]   one row per position.
 *   v      fp16 [pages][kv_heads][dim][page]   one row per dimension: eight
 *          positions of one dimension are one 16-byte load in the layout the
 *          matrix cores take, so attention never transposes V.
 * k_stride / v_stride are the elements from one page to the next (at least
 * kv_heads*page*dim, a multiple of 8), so that a pool may hold several layers.
 * A table entry outside [0, pages) is an absent page: nothing is read from or
 * written to it, and its positions are masked.
 *   dim in {64, 96, 128, 192, 256}; page a power of two in 16..256; heads a
 *   multiple of kv_heads with at most 64 heads per kv head (head h reads kv
 *   head h / (heads / kv_heads)); table_cols*page <= 2^31 - 256.
 * Contents are device data and are not checked on the host: lengths below 0
 * count as 0, lengths above max_length as max_length.
 * The struct is host memory, read during the call and not kept.
 */
typedef struct q4g128_kv_cache {
    uint16_t* k;
    uint16_t* v;
    const int32_t* table;  /* [sequences][table_cols] */
    int64_t pages;
    int64_t k_stride;
    int64_t v_stride;
    int64_t sequences;
    int64_t table_cols;
    int32_t kv_heads;
    int32_t dim;
    int32_t page;
} q4g128_kv_cache;

/*
 * q4g128_rope_append -- new tokens into the cache, and their queries.
 * Row t of qkv (fp32, `ld` floats from row to row: the output of any product
 * here, which may go on with other columns) holds `heads` query heads, then
 * kv_heads key heads, then kv_heads value heads of `dim` columns.  For each
 * query and key head:
 *     x = row / sqrt(mean(row^2) + eps) * weight[dim]     (if its norm is given)
 *     pair i < rot/2, angle a = positions[t] * inv_freq[i]:
 *     (x_lo, x_hi) = mscale * (x_lo cos a - x_hi sin a, x_hi cos a + x_lo sin a)
 * with lo, hi = 2i, 2i+1 if interleaved, else i, i + rot/2; dimensions from
 * rot on are not turned.  Angles are formed in 64 bits, everything else in
 * fp32, with one rounding to fp16.  Context scaling is the caller's choice of
 * inv_freq and mscale.
 *   q [tokens][heads][dim] fp16 is written in full; key and value heads go to
 *   position positions[t] of sequence seq[t] (seq NULL: token t is of
 *   sequence t).  A token whose sequence or position is outside the table, or
 *   whose page is absent, writes no cache entry.  Two tokens of one call must
 *   not share a position of a sequence.
 *   rot a multiple of 4 with 0 <= rot <= dim (0: no rotation, inv_freq may be
 *   NULL); ld a multiple of 4; q_norm / k_norm fp16 [dim] or NULL; eps >= 0.
 */
Q4_API q4_status q4g128_rope_append(const float* qkv, int64_t ld, int64_t tokens, int32_t heads,
                             const q4g128_kv_cache* cache, const int32_t* seq,
                             const int32_t* positions, const float* inv_freq, int32_t rot,
                             int32_t interleaved, float mscale, const uint16_t* q_norm,
                             const uint16_t* k_norm, float eps, uint16_t* q, void* stream);

/*
 * q4g128_rope_append_slots -- the same with the cache position apart from the
 * rotary one: a head is turned by positions[t] and written to position slots[t]
 * (a tree's drafted tokens of one depth share the first and not the second).
 */
Q4_API q4_status q4g128_rope_append_slots(const float* qkv, int64_t ld, int64_t tokens, int32_t heads,
                             const q4g128_kv_cache* cache, const int32_t* seq,
                             const int32_t* positions, const int32_t* slots, const float* inv_freq,
                             int32_t rot, int32_t interleaved, float mscale, const uint16_t* q_norm,
                             const uint16_t* k_norm, float eps, uint16_t* q, void* stream);

/*
 * What the attention calls compute for a query at position p of its
 * sequence, over the positions j that it sees:
 *     s_j = scale * (q . k_j);  if softcap > 0: s_j = softcap * tanh(s_j / softcap)
 *     if slopes != NULL:        s_j += slopes[head] * (j - p)
 *     out = sum_j softmax(s)_j v_j
 * It sees j <= p, with window > 0 only j > p - window, and in the prompt call
 * also every j < prefix[s]; the tree call says what drafted tokens see.  Scores,
 * softmax statistics and sums are fp32.  The weights enter the second product
 * rounded to fp16, in units of 2 to a running maximum of the base-2 scores: at most
 * 1 in the decode call, at most 2^8 in the others, whose maximum may lag (2^10 for
 * scores of 2^24 to 2^26; rows with scores beyond that are computed far more slowly); they are
 * summed as rounded.  out is rounded once to fp16.  A query that sees nothing gives zeros.  What a masked
 * position or an absent page holds never reaches a result, NaN included.
 *   scale > 0; softcap >= 0 (0: none); both finite; window >= 0 (0: none).
 */
typedef struct q4g128_attn_options {
    float scale;
    float softcap;
    int64_t window;
    const float* slopes;   /* [heads], or NULL */
    const int32_t* prefix; /* prompt call: [sequences], or NULL; needs window == 0 */
} q4g128_attn_options;

/*
 * q4g128_attn_decode -- one new token per sequence.
 *   q, out [batch][heads][dim] fp16; row b is position lengths[b] - 1 of
 *   sequence b (table row b; cache->sequences >= batch), whose cache holds
 *   lengths[b] positions, this token's among them.
 *   max_length: an upper bound on the lengths, at most table_cols*page; it
 *   sizes the launch.
 *   workspace: q4g128_attn_decode_workspace() bytes, 16-byte aligned.  Its
 *   first Q4G128_ATTN_COUNTER_BYTES must be zero before its first use; every
 *   call leaves them zero.  Calls that may run at the same time (on different
 *   streams) need workspaces of their own; calls of any shape on one stream can
 *   share one, which q4g128_attn_prefill may use too.
 * The cache's length is split over workgroups; the last one of a sequence to
 * finish joins their results, in the order of the positions whichever it is.
 */
Q4_API int64_t q4g128_attn_decode_workspace(int64_t batch, int32_t heads, int32_t dim);
Q4_API q4_status q4g128_attn_decode(const uint16_t* q, const q4g128_kv_cache* cache,
                             const int32_t* lengths, int64_t max_length, int64_t batch,
                             int32_t heads, const q4g128_attn_options* options, uint16_t* out,
                             void* workspace, int64_t workspace_bytes, void* stream);

/*
 * q4g128_attn_prefill -- the prompt tokens of one or more sequences.
 *   q, out [tokens][heads][dim] fp16; rows q_starts[s] .. q_starts[s+1]-1
 *   (q_starts int32 [count + 1], ascending from 0 to tokens) are the last
 *   positions of sequence s, whose cache holds lengths[s] positions, these
 *   tokens among them.  A token before position 0 (more tokens than the length
 *   says) sees nothing.  1 <= count <= 65536 and cache->sequences >= count.
 *   max_length as above.  workspace: q4g128_attn_prefill_workspace() bytes (0:
 *   none is needed, it may be NULL), 16-byte aligned; its first
 *   Q4G128_ATTN_COUNTER_BYTES are left alone, the rest may hold anything.
 */
Q4_API int64_t q4g128_attn_prefill_workspace(int64_t tokens, int64_t count, int32_t heads,
                             int32_t kv_heads, int32_t dim, int64_t max_length);
Q4_API q4_status q4g128_attn_prefill(const uint16_t* q, const q4g128_kv_cache* cache,
                             const int32_t* q_starts, const int32_t* lengths, int64_t max_length,
                             int64_t tokens, int64_t count, int32_t heads,
                             const q4g128_attn_options* options, uint16_t* out,
                             void* workspace, int64_t workspace_bytes, void* stream);

/*
 * q4g128_attn_tree -- drafted tokens of one or more sequences: a decode step of
 * several tokens per sequence, which the cache is read once for.
 *   q, out [tokens][heads][dim] fp16; rows q_starts[s] .. q_starts[s+1]-1 (int32
 *   [count + 1], ascending) are the drafted tokens of sequence s, its last cached
 *   positions: with n of them, drafted token k is position base + k, base =
 *   lengths[s] - n.  Rows of no sequence are left as they were.
 *   masks: uint64 [tokens], or NULL.  A token sees every position below base, and
 *   drafted token k of its sequence where bit k of its mask is set (its own bit
 *   like any other).  Windows and slopes go by a token's place, base + max(bits set
 *   among its sequence's tokens, 1) - 1: for a tree's masks (a token's ancestors and
 *   itself) base + its depth, the position that it is to be turned by; positions below
 *   base are their own places.  NULL: each token sees those before it, as in
 *   q4g128_attn_prefill.  No token sees the 65th or a later drafted token of a mask.
 *   max_new: an upper bound on a sequence's drafted tokens, 1 to Q4G128_MAX_DRAFT;
 *   it sizes the launch, and rows of later tokens are left as they were.
 *   options->prefix must be NULL.  max_length as in q4g128_attn_decode, workspace
 *   (q4g128_attn_tree_workspace() bytes) as in q4g128_attn_prefill.
 */
Q4_API int64_t q4g128_attn_tree_workspace(int64_t tokens, int64_t count, int32_t heads,
                             int32_t kv_heads, int32_t dim, int64_t max_new, int64_t max_length);
Q4_API q4_status q4g128_attn_tree(const uint16_t* q, const q4g128_kv_cache* cache,
                             const int32_t* q_starts, const int32_t* lengths,
                             const uint64_t* masks, int64_t max_new, int64_t max_length,
                             int64_t tokens, int64_t count, int32_t heads,
                             const q4g128_attn_options* options, uint16_t* out, void* workspace,
                             int64_t workspace_bytes, void* stream);

/*
 * q4g128_cache_keep -- the accepted tokens of each draft moved together: for i <
 * n = keep_starts[s+1] - keep_starts[s], position starts[s] + keep[keep_starts[s] +
 * i] of sequence s becomes position starts[s] + i, keys and values of all kv heads.
 *   starts int32 [count]: the committed positions of each sequence; keep_starts
 *   int32 [count + 1], ascending from 0 to total; keep int32 [total], for each
 *   sequence the numbers of its accepted drafted tokens, strictly ascending from 0 on
 *   (what other numbers leave in the sequence's positions is unspecified).  A token whose
 *   old or new position is outside the table or has no page is not moved.  No two
 *   sequences of a call may share a page that a token is moved in.
 *   total 0: nothing is enqueued (keep may be NULL).
 */
Q4_API q4_status q4g128_cache_keep(const q4g128_kv_cache* cache, const int32_t* starts,
                             const int32_t* keep_starts, const int32_t* keep, int64_t total,
                             int64_t count, void* stream);

/*
 * Latent attention: keys and values of all heads come from one row per position,
 * `latent` columns and a rotary key part of Q4G128_LATENT_ROT that all heads share.
 *   rows   fp16 [pages][page][latent + 64], page number and table as in
 *   q4g128_kv_cache; stride: elements from one page to the next (at least
 *   page*(latent+64), a multiple of 8).
 *   latent in {128, 256, 512}; page a power of two in 16..256;
 *   table_cols*page <= 2^31 - 256.
 * The struct is host memory, read during the call and not kept.
 */
typedef struct q4g128_latent_cache {
    uint16_t* rows;
    const int32_t* table;  /* [sequences][table_cols] */
    int64_t pages;
    int64_t stride;
    int64_t sequences;
    int64_t table_cols;
    int32_t latent;
    int32_t page;
} q4g128_latent_cache;

/*
 * q4g128_latent_append -- new tokens' rows into the cache, and their queries.
 * Row t of kv (fp32, `ld` floats from row to row, a multiple of 4; further columns
 * are left alone) holds `latent` columns x and 64 rotary ones r; the position
 * slots[t] of sequence seq[t] (as in q4g128_rope_append) becomes
 *     (x * norm / sqrt(mean(x^2) + eps)  (norm fp16 [latent] given; else x),
 *      r turned by positions[t] as in q4g128_rope_append with rot = 64).
 * The query of token t and head h is (q_main row, q_rot row turned alike): `main`
 * and 64 floats at q_main + t*main_ld + h*main_head and q_rot + t*rot_ld +
 * h*rot_head, strides multiples of 4.  For the absorbed form q_main holds the heads'
 * products with their key weights (main = latent), for the expanded form the heads'
 * own columns.
 *   q [tokens][heads][main + 64] fp16 is written in full; main a multiple of 8, 8 to
 *   Q4G128_LATENT_MAX_MAIN.  heads 0: no queries (their pointers are not used).
 *   inv_freq [32], or NULL: nothing is turned or scaled.
 */
Q4_API q4_status q4g128_latent_append(const float* kv, int64_t ld, int64_t tokens,
                             const q4g128_latent_cache* cache, const int32_t* seq,
                             const int32_t* positions, const int32_t* slots, const float* inv_freq,
                             int32_t interleaved, float mscale, const uint16_t* norm, float eps,
                             const float* q_main, int64_t main_ld, int64_t main_head, int32_t main,
                             const float* q_rot, int64_t rot_ld, int64_t rot_head, int32_t heads,
                             uint16_t* q, void* stream);

/* q4g128_latent_keep -- q4g128_cache_keep for a latent cache. */
Q4_API q4_status q4g128_latent_keep(const q4g128_latent_cache* cache, const int32_t* starts,
                             const int32_t* keep_starts, const int32_t* keep, int64_t total,
                             int64_t count, void* stream);

/*
 * q4g128_latent_attn -- attention over the rows themselves (absorbed form):
 *     out[t][h] = sum_j softmax_j(scale * q[t][h] . c_j) c_j[:latent]
 *   q [tokens][heads][latent + 64], out [tokens][heads][latent] fp16; q_starts,
 *   lengths, masks, max_new and max_length as in q4g128_attn_tree, workspace
 *   (q4g128_latent_attn_workspace() bytes) as in q4g128_attn_prefill; a head's value
 *   weights are applied to out by the caller.  max_new is at most Q4G128_MAX_DRAFT with masks and at most
 *   Q4G128_MAX_TOKENS without; rows of a workgroup and parts of the positions follow it, so it should be
 *   no larger than the longest sequence's rows: 1 for single tokens.  Numerics as stated for the
 *   attention calls.
 *   heads at most Q4G128_MAX_HEADS; scale > 0, finite.
 */
Q4_API int64_t q4g128_latent_attn_workspace(int32_t heads, int32_t latent, int64_t max_new);
Q4_API q4_status q4g128_latent_attn(const uint16_t* q, const q4g128_latent_cache* cache,
                             const int32_t* q_starts, const int32_t* lengths,
                             const uint64_t* masks, int64_t max_new, int64_t max_length,
                             int64_t tokens, int64_t count, int32_t heads, float scale,
                             uint16_t* out, void* workspace, int64_t workspace_bytes,
                             void* stream);

/*
 * q4g128_latent_expand -- keys and values of every head from latent rows, for the
 * prompts of the expanded form: for each position j of sequence s with firsts[s] <=
 * j < lengths[s] (firsts int32 [count], or NULL: 0; lengths above max_length count as
 * max_length) and head h
 *     k[j][h] = (W_k[h] c_j, r_j),  v[j][h] = W_v[h] c_j,
 * c_j the `latent` columns and r_j the 64 rotary ones of its row.  The weights are
 * int4 in the layout above, N = heads * 2 * value rows of K = latent columns, each
 * head's `value` key rows before its value rows; each enters as fp16(code*scale+min)
 * with one rounding, as in q4g128_gemm_prefill; sums are fp32, rounded once to fp16.
 *   expanded: a q4g128_kv_cache with a kv head for every head and dim = value (64 or
 *   128), whose keys are value + 64 wide: k [pages][heads][page][value + 64] (k_stride
 *   at least heads*page*(value+64)), v [pages][heads][value][page].  Its table may be
 *   the latent cache's, if their pages are alike, and with equal strides (in bytes) the
 *   pages of all three pools may interleave in one allocation.  heads at most
 *   Q4G128_MAX_HEADS.  Positions without a page in either cache are not written, and
 *   nothing but the positions named above is.  No two sequences may share a page of
 *   `expanded` that both write.
 */
Q4_API q4_status q4g128_latent_expand(const q4g128_latent_cache* cache, const int32_t* lengths,
                             const int32_t* firsts, int64_t max_length, int64_t count,
                             const uint8_t* packed, const uint16_t* scales, const uint16_t* mins,
                             const q4g128_kv_cache* expanded, void* stream);

/*
 * q4g128_latent_prefill -- q4g128_attn_prefill over expanded keys and values:
 *   q [tokens][heads][value + 64], out [tokens][heads][value] fp16, each head with
 *   keys and values of its own.  Causal, no options but the scale (> 0, finite).
 *   Workspace: q4g128_latent_prefill_workspace() bytes, as in q4g128_attn_prefill.
 */
Q4_API int64_t q4g128_latent_prefill_workspace(int64_t tokens, int64_t count, int32_t heads,
                             int32_t value, int64_t max_length);
Q4_API q4_status q4g128_latent_prefill(const uint16_t* q, const q4g128_kv_cache* expanded,
                             const int32_t* q_starts, const int32_t* lengths, int64_t max_length,
                             int64_t tokens, int64_t count, float scale, uint16_t* out,
                             void* workspace, int64_t workspace_bytes, void* stream);

/* Static, NUL-terminated description of a status code. */
Q4_API const char* q4g128_status_string(q4_status status);

/* hipError_t recorded by the last Q4_EDEVICE return on the calling thread
   (0 if none). */
Q4_API int32_t q4g128_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* Q4G128_H */
