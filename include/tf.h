/*
 * tf.h -- C ABI of the segmented speculative-verify step (LFM2 shared-round
 * decode with drafts) for NVIDIA GB300 (sm_103a).
 *
 * What the step computes comes from the TensorFold pages:
 *   [SRD]   PR #1377 "LFM2: shared-round decode"
 *           - commit "a shared round runs each layer's conv and attention once
 *             over all its streams" (segment table of cache addresses, row
 *             offsets and key counts; one launch per layer over every row;
 *             per-stream attention partials; float64 attention and a host
 *             replay of the conv steps as the checks);
 *           - commit "a verify's greedy rows take the GPU's pick of their
 *             logits" (the largest logit, the lowest id among equal ones,
 *             nonfinite rows flagged);
 *           - commit "the conv, qk, attention and merge kernels' bodies as
 *             inline functions" (qk, attention, merge);
 *           - section "Failures the tests catch" (a scratch too small for
 *             per-stream partials; a table reaching memory it did not declare).
 *   [DSP]   PR #1391 "lfm2: draft with LiquidAI's DSpark drafter (--drafter)":
 *           every draft is verified by the target; the target's attention
 *           stays causal; the drafter's block attention (the same kernels
 *           with a FULL flag, under which every row of a block sees all of
 *           its stream's keys), its Markov head (each draft row adds the
 *           product of W2 with the W1 row of the previous pick to its logits
 *           and takes the argmax, the rows in sequence; the step as the
 *           argmax of bf16(base + bf16(W2 . W1[prev])), lowest token on a
 *           tie, a NaN score flagged) and the held path's kernel that fills
 *           the verify's ids from the drafter's picks (a bad pick raises a
 *           flag for the verify instead of becoming a token).
 *
 * Conventions for every call:
 *   - All tensors are dense, row-major, in DEVICE memory owned by the caller,
 *     and start on a 16-byte boundary. bf16 tensors are passed as `void*`.
 *   - Every call is asynchronous on the caller's CUDA stream `stream` (a
 *     cudaStream_t; NULL is the legacy default stream) and never synchronises.
 *   - Every call returns a tf_status. Invalid arguments are refused on the host
 *     before anything is launched; nothing aborts. A nonfinite logit is data,
 *     reported in the flags, never an error.
 *   - Model widths are fixed (LFM2.5-24B-A2B): TF_H conv channels, conv input
 *     TF_CIN = 3*TF_H as the consecutive slices (B, C, x), kernel width TF_KW,
 *     TF_NQ query heads sharing TF_NKV KV heads of width TF_D.
 */
#ifndef TF_H_INCLUDED
#define TF_H_INCLUDED

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define TF_H        2048
#define TF_CIN      6144
#define TF_KW       3
#define TF_NQ       32
#define TF_NKV      8
#define TF_D        64
#define TF_MAX_ROWS 16          /* window rows per stream (1 + drafts) */
#define TF_MAX_KEYS (1 << 22)   /* cache rows per stream */
#define TF_MAX_PROMPT_ROWS 65536  /* rows of one prompt call (tf_prompt_build) */
#define TF_PROMPT_WINDOW_ROWS 32  /* a prompt call's attention window (tf_prompt_build) */
#define TF_MAX_STREAMS 65536
#define TF_MIN_PAGE_KEYS 16       /* cache rows of a page (paged tables): a power of two */
#define TF_MAX_PAGE_KEYS 256
#define TF_MAX_PAGES (1 << 24)    /* pages of a pool */
#define TF_MAX_PAGE_IDS (1 << 28) /* entries of a paged table's lists together */
#define TF_MK       256         /* width of the drafter's Markov head rows (W1, W2) */
#define TF_SCALE_KEYS 16          /* keys of a head that share a scale in scaled pools */
#define TF_SCALE_COLUMNS 32       /* columns of a row (inputs of a weight) that share a scale */

typedef enum {
    TF_OK = 0,
    TF_EINVAL = 1,   /* null pointer, bad shape, unpacked rows, aliasing, misalignment */
    TF_ERANGE = 2,   /* a size beyond the limits above */
    TF_ENOMEM = 3,   /* the library's own table allocation failed */
    TF_ECUDA = 4,    /* a CUDA call or launch failed (see tf_last_cuda_error) */
    TF_ETIMEOUT = 5  /* a kernel gave up a bounded device wait (tf_segments_status) */
} tf_status;

struct CUstream_st;                       /* cudaStream_t is struct CUstream_st* */
typedef struct CUstream_st* tf_cuda_stream;

/* One stream of a shared round ([SRD]: the table lists each stream's cache
 * addresses, row offset and key count).
 *   rows        window rows r_s = 1 + drafts, 1..TF_MAX_ROWS
 *   row_offset  first row of the stream in every [R][...] tensor; streams are
 *               packed in order: row_offset_0 = 0, row_offset_{s+1} =
 *               row_offset_s + rows_s
 *   keys        k_s, cache entries INCLUDING the window's own rows (their K/V
 *               are already written); window row i sees keys
 *               [0, keys - rows + i + 1) (causal, [DSP]); rows <= keys
 *   kv_capacity cache rows allocated per KV head, keys <= kv_capacity */
typedef struct {
    int32_t rows;
    int32_t row_offset;
    int32_t keys;
    int32_t kv_capacity;
} tf_stream;

/* Host-side sizes of a table, from tf_segments_plan (no GPU needed). */
typedef struct {
    int32_t n_streams;
    int32_t n_rows;           /* R = sum of rows */
    int32_t max_rows;
    int32_t n_conv_tiles;     /* conv tiles of at most 8 rows ([SRD]) */
    int32_t n_attn_items;     /* (stream, key chunk) work items per KV head */
    int32_t attn_kernels;     /* partial-kernel launches per attention layer (1 or 2) */
    int32_t attn_merge_launch;/* 1 if tf_attn also launches the merge kernel */
    int32_t reserved;
    int64_t n_partials;       /* partial records: sum_s rows_s * 32 * chunks_s */
    int64_t partials_bytes;   /* scratch tf_attn_partials needs (see below) */
} tf_plan;

/* The library's own device copy of a segment table. Immutable once built. */
typedef struct tf_segments tf_segments;

/* Split-K chunk of a stream: keys [c*chunk, (c+1)*chunk). The chunk length is
 * 256 * max(rows, 4) keys (partial records stay near 1/64 of the K/V bytes),
 * and 512 * rows for windows of 9 to 16 rows (the tensor-core kernel: fewer,
 * longer units measured faster there); it depends on the stream alone, so a
 * stream's results do not depend on which other streams share the round. */
int32_t tf_chunk_keys(int32_t rows);

/* Validate `streams` and compute the table's sizes. Host only; touches no GPU.
 * Errors: TF_EINVAL (null, rows < 1, unpacked offsets, keys < rows,
 * keys > kv_capacity), TF_ERANGE (beyond TF_MAX_*). n_streams == 0 is an
 * empty round (every call on its table is a no-op). */
int tf_segments_plan(const tf_stream* streams, int n_streams, tf_plan* out);

/* Build the segment table on the device ([SRD] segments.zig).
 *   streams      host array [n_streams]
 *   conv_state   host array [n_conv][n_streams] of device pointers, each to a
 *                bf16 [2][TF_H] rolling conv state (oldest row first), read
 *                and rewritten in place by tf_conv_rows / tf_accept
 *   conv_hist    NULL, or host array [n_conv][n_streams] of device pointers,
 *                each to a bf16 [rows+2][TF_H] history written by
 *                tf_conv_rows (the state before the window, then every row's
 *                gate); entries of one-row streams may be NULL. NULL disables
 *                the conv rewind in tf_accept.
 *   k_cache, v_cache  host arrays [n_attn][n_streams] of device pointers, each
 *                to a bf16 [TF_NKV][kv_capacity][TF_D] cache (head-major)
 * Refuses (TF_EINVAL) null or misaligned pointers and any two buffers of the
 * table that overlap (conv states and histories across every stream and
 * layer; K and V caches likewise) -- the bug class of [SRD]'s planted controls,
 * in which every stream reads or writes stream 0's conv state or KV cache.
 * The table is copied to the device on `stream` before the call returns; the
 * host arrays may be freed at once. *out is owned by the caller and released
 * with tf_segments_free. */
int tf_segments_build(const tf_stream* streams, int n_streams,
                      const void* const* conv_state, const void* const* conv_hist,
                      const void* const* k_cache, const void* const* v_cache,
                      int n_conv, int n_attn, tf_cuda_stream stream,
                      tf_segments** out);

/* Free a table (synchronises the device through cudaFree). NULL is a no-op. */
int tf_segments_free(tf_segments* seg);

/* Sizes of a built table (same as tf_segments_plan's). */
int tf_segments_query(const tf_segments* seg, tf_plan* out);

/* Bytes of partial scratch tf_attn_partials writes and tf_attn_merge reads
 * ([SRD]: each stream keeps its own partials in the scratch).
 * Layout: float o[n_partials][TF_D], then float2 ml[n_partials] (m, l).
 * 0 for a NULL table. */
size_t tf_partials_bytes(const tf_segments* seg);

/* a1. LFM2 gated short conv of one conv layer over every row of every stream
 * ([SRD]: the 30 short-conv layers, each run once over every row).
 *   bcx  bf16 [R][TF_CIN], row = (B, C, x)
 *   w    bf16 [TF_H][TF_KW] depthwise taps; w[c][0] multiplies the oldest row
 *   y    float [R][TF_H] output, y = C * conv
 * Per stream, row by row: bx = bf16_rne(B*x); seq = [state0, state1, bx_0..];
 * conv_i = w0*seq[i] + w1*seq[i+1] + w2*seq[i+2] (fp32). Afterwards the
 * stream's state holds the last two entries of seq and its history (if any)
 * all of them; both are bit-exact. Errors: TF_EINVAL (null/misaligned,
 * conv_layer out of range). */
int tf_conv_rows(const tf_segments* seg, int conv_layer, const void* bcx,
                 const void* w, float* y, tf_cuda_stream stream);

/* a2. Causal GQA attention partials of one attention layer: for every stream,
 * KV head, key chunk, window row and query head, (m, l, o) over the chunk's
 * visible keys ([SRD]: the qk, attention and merge of the 10 attention
 * layers). Streams with windows of 9 rows or more run on the tcgen05
 * tensor-core kernel, the others
 * on the mma.sync kernel; the choice depends on the stream alone (so a
 * stream's bits do not depend on its round), and a round holding both kinds
 * makes one launch of each (tf_plan.attn_kernels). The environment variable
 * TF_ATTN_PATH=mma|tc, read by tf_segments_build, forces one kernel for every
 * window of at most 16 rows (a prompt table's wider windows always run on the
 * tensor cores); the mma.sync kernel takes a window as items of at most 8
 * rows. P.V runs with P and V in fp16 and fp32 accumulation; a piece of work
 * whose fp16 result holds a partial sum that is not finite (a V of 65,536 or
 * more has no fp16 value) or whose partial outputs |o|/l all lie below 2^-10
 * is computed again with V in bf16 and P split into a bf16 high part and a
 * bf16 remainder (the mma.sync kernel per item, the tensor-core kernel per
 * unit of one chunk and KV head, in the launch's last CTA). So every finite
 * V is supported; in an fp16 result only values of V below 2^-14 round, by
 * at most 2^-25 each. Sums of P.V must stay within fp32's range.
 *   q         bf16 [R][TF_NQ][TF_D]
 *   partials  device scratch of tf_partials_bytes(seg) bytes. Record of
 *             stream s, chunk c, KV head g, row i, head 4g+hh:
 *             pbase_s + ((c*8 + g)*rows_s + i)*4 + hh, pbase_s = sum over
 *             earlier streams of rows * 32 * chunks.
 *             m = (largest score) * log2(e), l = sum 2^(s*log2(e) - m),
 *             o[d] = sum 2^(s*log2(e) - m) * v[d]; a chunk without a visible
 *             key has m = -inf, l = 0, o = 0.
 * Score = (q . k) / 8; query head h reads KV head h / 4. Errors: TF_EINVAL. */
int tf_attn_partials(const tf_segments* seg, int attn_layer, const void* q,
                     void* partials, tf_cuda_stream stream);

/* a2+a3 in one call: the attention output of one layer. One launch of the
 * partials kernel(s) in which a stream with a single key chunk writes its
 * output directly and a stream with few partial records (4 * rows * chunks
 * <= 512) is merged by the last CTA to finish each of its KV heads (counted
 * by per-layer counters in the table that reset themselves); streams with
 * more records are merged by one merge launch. ([SRD]: each layer runs once
 * over every row.) A round holding both kinds of window runs the mma.sync
 * launch on a stream of the table's own, forked from `stream` and joined
 * back to it before the call returns, so that the two launches run side by
 * side; work queued on `stream` after the call waits for both. Same
 * arguments as tf_attn_partials plus `out`
 * (float [R][TF_NQ][TF_D]); `partials` is the scratch of tf_partials_bytes.
 * Calls on the same table and layer must not overlap on the GPU.
 * Errors: TF_EINVAL. */
int tf_attn(const tf_segments* seg, int attn_layer, const void* q, void* partials, float* out,
            tf_cuda_stream stream);

/* The drafter's non-causal block attention ([DSP] lfm2_attn_block: the
 * target's attention kernels with a FULL flag, under which every row of a
 * block sees the keys [0, len + 1)). Reading: len + 1 is the stream's key
 * count including
 * the block's own rows, so every window row sees all `keys` keys of its
 * stream (what the last row sees under the causal count). Same arguments,
 * records, kernels, chunking and errors as tf_attn_partials / tf_attn; the
 * merge (tf_attn_merge) is shared. */
int tf_attn_block_partials(const tf_segments* seg, int attn_layer, const void* q,
                           void* partials, tf_cuda_stream stream);
int tf_attn_block(const tf_segments* seg, int attn_layer, const void* q, void* partials,
                  float* out, tf_cuda_stream stream);

/* a3. Log-sum-exp merge of the partials into the attention output
 * ([SRD] lfm2_merge_row): out = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c,
 * M = max_c m_c, empty chunks skipped.
 *   out  float [R][TF_NQ][TF_D]. Errors: TF_EINVAL. */
int tf_attn_merge(const tf_segments* seg, const void* partials, float* out,
                  tf_cuda_stream stream);

/* Attention of one layer (tf_attn_partials then tf_attn_merge) that allocates
 * nothing: the partial scratch is a fixed array of TF_STATIC_SCRATCH_BYTES
 * compiled into the library (no counterpart on the pages; it exists for
 * callers that cannot call cudaMalloc or any allocating routine, such as code
 * under a strict memory budget or an allocator it does not own).
 *   q    bf16 [R][TF_NQ][TF_D], out float [R][TF_NQ][TF_D], as above.
 * Every GPU that loads the library holds the array until the process exits.
 * The first call on a device looks the array's device address up (with that
 * device current); make that first call before any stream capture. The
 * address is kept for the life of the process: a cudaDeviceReset (or
 * anything else that unloads the library's module from a device) leaves it
 * stale, so do not call tf_attn_static after one. Calls
 * share the one array: calls whose launches overlap on the GPU (different
 * streams at once) race and give wrong results. Nothing in the array has to
 * start at zero; each call writes every record it reads.
 * Errors: TF_ERANGE when tf_partials_bytes(seg) > TF_STATIC_SCRATCH_BYTES
 * (nothing is launched), TF_EINVAL as tf_attn_partials. Calls no cudaMalloc,
 * cudaFree or other allocating routine. */
#define TF_STATIC_SCRATCH_BYTES (16u << 20)
int tf_attn_static(const tf_segments* seg, int attn_layer, const void* q, float* out,
                   tf_cuda_stream stream);

/* a4. Greedy pick of each row of bf16 logits ([SRD] lfm2_argmax: the largest
 * logit, the lowest id among equal largest values, and a flag on any row
 * holding a nonfinite value).
 *   logits      bf16, row r at logits + r*row_stride (elements), V per row
 *   pick        int32 [R]: lowest id holding the row's largest value (-0 and
 *               +0 are equal); -1 when the row is flagged
 *   flag        uint8 [R]: 1 if the row holds a NaN, +Inf or -Inf, else 0
 * Needs no table. R == 0 is a no-op. Errors: TF_EINVAL (null, V < 1,
 * row_stride < V), TF_ERANGE (V > 2^30, R > 2^24). Rows are read with 16-byte
 * vector loads when logits and row_stride allow it. One launch takes at most
 * 65,535 rows (the grid's y extent); larger R runs as several launches. */
int tf_argmax_rows(const void* logits, int R, int V, int64_t row_stride,
                   int32_t* pick, uint8_t* flag, tf_cuda_stream stream);

/* Sampled pick of each row of bf16 logits, for rows that a temperature draws
 * instead of tf_argmax_rows' greedy pick; the picks and flags go to tf_accept
 * in the same way (a draft is accepted where the target's draw equals it, so a
 * drafted reply is distributed as an undrafted one). Per row, with its own
 * settings:
 *   - tokens in order of (logit descending, id ascending; -0 equals +0), each
 *     of weight w = exp((x - max) / T);
 *   - top-k keeps the first top_k tokens, of mass Z;
 *   - top-p keeps the shortest prefix of mass at least top_p * Z (one token at
 *     least), min-p the tokens of w >= min_p; the kept tokens are the shortest
 *     prefix of the three;
 *   - the pick is the first token at which the cumulative mass exceeds u times
 *     the mass of the kept tokens.
 * T == 0 picks the first token (the greedy pick). Counts are exact and weights
 * 64-bit fixed point, scaled to the row's mass, so a pick equals the
 * definition's in exact arithmetic except where u lies within 1e-12 of a border
 * (and top_p or min_p likewise).
 *   logits      as in tf_argmax_rows (any 2-byte address and stride); -Inf is a
 *               masked token (never picked)
 *   temperature float [R] or NULL (1); 0 <= T < inf
 *   top_k       int32 [R] or NULL; off where <= 0 or >= V
 *   top_p       float [R] or NULL; off where >= 1; <= 0 keeps one token
 *   min_p       float [R] or NULL; off where <= 0; at most 1
 *   u           float [R] in [0, 1)
 *   pick        int32 [R]; -1 when the row is flagged
 *   prob        float [R] or NULL: w of the pick over the kept mass (1 when
 *               T == 0, 0 when flagged)
 *   flag        uint8 [R]: TF_SAMPLE_NO_LOGITS a NaN or +Inf in the row, or
 *               every token masked; TF_SAMPLE_BAD_SETTING a setting outside
 *               its range or NaN
 * Needs no table. R == 0 is a no-op. Errors: TF_EINVAL (null, an odd address
 * of the logits, one that is no multiple of 4 of a 4-byte array, V < 1,
 * row_stride < V), TF_ERANGE (V > TF_SAMPLE_MAX_VOCAB, R > 2^24). */
#define TF_SAMPLE_MAX_VOCAB (1 << 19)
#define TF_SAMPLE_NO_LOGITS   1
#define TF_SAMPLE_BAD_SETTING 2
int tf_sample_rows(const void* logits, int R, int V, int64_t row_stride,
                   const float* temperature, const int32_t* top_k, const float* top_p,
                   const float* min_p, const float* u, int32_t* pick, float* prob,
                   uint8_t* flag, tf_cuda_stream stream);

/* a5. Greedy verify of every stream: the accepted-draft prefix length
 * ([DSP]: the target verifies every draft; [SRD] verifyFn takes the pick
 * for greedy rows, flagged rows are drawn on the host).
 *   ids         int32 [R]: row 0 of a window is the pending token, rows 1..
 *               the drafts
 *   pick, flag  from tf_argmax_rows
 *   vocab       draft ids outside [0, vocab) never match
 *   accept_len  int32 [S]: a = leading drafts j+1 with pick[j] == ids[j+1]
 *               and row j unflagged (0 <= a <= rows-1)
 *   next_token  int32 [S]: pick of row a, or -1 when row a is flagged
 *   new_keys    int32 [S]: keys - rows + a + 1
 *   sflag       uint8 [S]: bit 0 row a flagged (host draws), bit 1 a draft id
 *               of the window lies outside [0, vocab)
 *   rewind_conv nonzero: rewrite every conv layer's state of every stream with
 *               rows > 1 to history rows a+1, a+2 (the state after row a);
 *               needs the table's conv_hist
 * Errors: TF_EINVAL (null outputs; rewind without histories). */
int tf_accept(const tf_segments* seg, const int32_t* ids, const int32_t* pick,
              const uint8_t* flag, int vocab, int32_t* accept_len,
              int32_t* next_token, int32_t* new_keys, uint8_t* sflag,
              int rewind_conv, tf_cuda_stream stream);

/* The drafter's Markov head over the draft rows of a verify table ([DSP]
 * lfm2_markov_scan / lfm2_markov_pick). Stream s drafts rows_s - 1 tokens;
 * its block rows are packed stream after stream at draft row o_s - s (o_s its
 * window's row offset), R - S rows in all. Block row j of stream s scores
 *   score[v] = bf16(base[v] + bf16(W2[v] . W1[tok]))     (v < vocab)
 * with tok = prev[s] for j = 0 and the pick of row j-1 after that (the rows in
 * sequence); the dot accumulates in fp32 on the tensor cores and is
 * rounded to nearest even, as is the sum. The pick is the lowest token with
 * the largest score.
 *   W1, W2      bf16 [vocab][TF_MK]
 *   base        bf16 logits, draft row k at base + k*base_stride (elements)
 *   prev        int32 [S]: each stream's pending token
 *   pick        int32 [R - S]: the row's pick, -1 when flagged
 *   flag        uint8 [R - S]: bit 0 a nonfinite score in the row, or no
 *               valid previous token (outside [0, vocab), e.g. a flagged row
 *               before it); bit 1 the kernel gave up waiting for its own
 *               copies or MMAs (more than 2 s; the row is not computed)
 * Tables of at most 128 streams run the whole chain in one cooperative launch
 * (one CTA per SM, all resident; the CTAs meet between steps, every wait
 * bounded) after a 16-byte memset of the table's step barrier; larger tables
 * (or TF_MARKOV_PATH=step) take one launch per step (rows_max - 1 launches).
 * Either way W2 is read once a step for up to 128 streams. The table holds the
 * cross-CTA scratch: calls on one table must not overlap on the GPU. Errors: TF_EINVAL (null, misaligned W2 or base,
 * base_stride < vocab or not a multiple of 8, vocab < 1), TF_ERANGE
 * (vocab > 2^24). */
int tf_markov_chain(const tf_segments* seg, const void* W1, const void* W2, int vocab,
                    const void* base, int64_t base_stride, const int32_t* prev,
                    int32_t* pick, uint8_t* flag, tf_cuda_stream stream);

/* The next verify's ids from each stream's pending token and the drafter's
 * picks ([DSP] lfm2_draft_ids, on the GPU so that the host reads no pick
 * between the drafter and the verify). Window row 0 of stream s is prev[s];
 * window row j >= 1 is the draft at packed draft row o_s - s + j - 1 (the
 * layout tf_markov_chain writes). A token outside [0, vocab), or a draft whose
 * draft_flag is nonzero, is written as -1 (the verify never accepts it).
 *   prev        int32 [S] (e.g. tf_accept's next_token)
 *   drafts      int32 [R - S]; may be NULL when every window has one row
 *   draft_flag  uint8 [R - S] or NULL
 *   ids         int32 [R]: the verify's ids
 *   dflag       uint8 [S]: bit 0 (TF_DFLAG_BAD_PENDING) the pending token was
 *               bad, bit 1 (TF_DFLAG_BAD_DRAFT) a draft was bad
 * Errors: TF_EINVAL (null, vocab < 1). */
#define TF_DFLAG_BAD_PENDING 1
#define TF_DFLAG_BAD_DRAFT   2
int tf_draft_ids(const tf_segments* seg, const int32_t* prev, const int32_t* drafts,
                 const uint8_t* draft_flag, int vocab, int32_t* ids, uint8_t* dflag,
                 tf_cuda_stream stream);

/* A prompt (prefill) call of one stream ([SRD]: prompt calls and windows of a
 * single stream still take the per-stream launches; those kernels run them in their own
 * 16-row tiles, here 32-row windows, which fill a 128-lane tensor-core tile
 * with their 4 query heads per KV head):
 * `rows` new rows (row 0 first) whose K/V are already in the cache, so the
 * cache holds `keys` entries in all (keys >= rows). The returned table serves
 * tf_conv_rows (the rows in order with the stream's conv state; no history)
 * and the attention calls (tf_attn, tf_attn_partials + tf_attn_merge,
 * tf_attn_static, tf_partials_bytes): the rows run as windows of
 * W = TF_PROMPT_WINDOW_ROWS rows (the last may be shorter), window t seeing
 * its causal count keys - rows + W*t + i + 1 for its row i, all reading the
 * one cache.
 *   conv_state  [n_conv] -> bf16 [2][TF_H], updated in place
 *   k_cache, v_cache [n_attn] -> bf16 [TF_NKV][kv_capacity][TF_D]
 * The conv input, queries and outputs are [rows][...] as in the verify calls.
 * tf_accept, tf_draft_ids and tf_markov_chain refuse a prompt table.
 * Errors: TF_EINVAL (null/misaligned/overlapping buffers, rows < 1,
 * keys < rows, kv_capacity < keys), TF_ERANGE (rows > TF_MAX_PROMPT_ROWS,
 * kv_capacity > TF_MAX_KEYS), TF_ENOMEM, TF_ECUDA. Free with tf_segments_free. */
int tf_prompt_build(int32_t rows, int32_t keys, int32_t kv_capacity,
                    const void* const* conv_state, const void* const* k_cache,
                    const void* const* v_cache, int n_conv, int n_attn,
                    tf_cuda_stream stream, tf_segments** out);

/* ---- paged caches -----------------------------------------------------------
 * A paged table's streams keep their keys and values in pages of a pool that
 * all streams share, one pool of K and one of V a layer, instead of one
 * contiguous cache each: a stream grows by a page at a time, a forked stream
 * lists its parent's pages, and streams with a common prompt list its pages
 * once written. Key t of a stream is slot t % page_keys of the page that the
 * stream's list names at t / page_keys, the same page in every layer.
 *   pool    bf16 [n_pages][TF_NKV][page_keys][TF_D] (head-major in a page)
 *
 * tf_paged_build is tf_segments_build for pages:
 *   streams     as there; kv_capacity is a multiple of page_keys
 *   pages       host array of page ids, stream after stream, kv_capacity /
 *               page_keys entries each, every entry in [0, n_pages). Entries
 *               past a stream's keys are not read by the calls, but they are the
 *               list's all the same: checked, and uses of their page (below), so
 *               a filler there has to be a page that holds no window rows, one
 *               kept for that purpose or the next pages that the stream grows into
 *   page_keys   a power of two, TF_MIN_PAGE_KEYS..TF_MAX_PAGE_KEYS
 *   k_pool, v_pool  host arrays [n_attn] of device pointers
 * A page may stand in several lists, or several times in one, for reading; a
 * page that holds rows of a stream's window (they are appended there) must
 * stand in the lists exactly once, spare entries included: copy a shared last
 * page first
 * (tf_pages_copy). Refuses what tf_segments_build refuses, pools that overlap,
 * a bad page size, an id out of range and a shared page with window rows
 * (TF_EINVAL); n_pages > TF_MAX_PAGES or more than TF_MAX_PAGE_IDS entries
 * (TF_ERANGE).
 *
 * tf_paged_prompt_build is tf_prompt_build for pages: one list of kv_capacity /
 * page_keys entries.
 *
 * The calls on tables below (tf_attn_paged, tf_qk_rows) refuse a table that was
 * built with another device current (TF_EINVAL); tf_pages_copy and
 * tf_sample_rows refuse pools and logits in another device's memory.
 *
 * Either table serves every call that a dense table of its kind serves, except
 * that its attention is tf_attn_paged: tf_attn, tf_attn_block, their partials
 * forms, tf_attn_merge and tf_attn_static refuse it (TF_EINVAL).
 *
 * tf_paged_scaled_build and tf_paged_scaled_prompt_build are the two for scaled
 * pools (below). */
int tf_paged_build(const tf_stream* streams, int n_streams, const void* const* conv_state,
                   const void* const* conv_hist, const int32_t* pages, int32_t page_keys,
                   int32_t n_pages, const void* const* k_pool, const void* const* v_pool,
                   int n_conv, int n_attn, tf_cuda_stream stream, tf_segments** out);
int tf_paged_prompt_build(int32_t rows, int32_t keys, int32_t kv_capacity,
                          const void* const* conv_state, const int32_t* pages,
                          int32_t page_keys, int32_t n_pages, const void* const* k_pool,
                          const void* const* v_pool, int n_conv, int n_attn,
                          tf_cuda_stream stream, tf_segments** out);

/* The attention of one layer over a paged table in one call: tf_attn (full ==
 * 0) or tf_attn_block (full != 0) with the keys and values in pages. Same
 * masks, kernels, chunks, partial scratch (tf_partials_bytes), failure report
 * and rule on overlapping calls as there; a stream's result does not depend on
 * which pages hold its keys. What a page holds past its stream's keys is never
 * used.
 *   q    bf16 [R][TF_NQ][TF_D]
 *   out  bf16 [R][TF_NQ][TF_D]: the fp32 result rounded once to nearest even
 *        (what the output projection reads; the probabilities are fp16, which
 *        leaves the fp32 result about 2e-4 of its size, a tenth of that
 *        rounding)
 * q, partials and out lie apart (queries may be read again after outputs are
 * written). Errors: TF_EINVAL (a table that is not paged, attn_layer out of
 * range, null, misaligned or overlapping buffers). */
int tf_attn_paged(const tf_segments* seg, int attn_layer, const void* q, void* partials,
                  void* out, int full, tf_cuda_stream stream);

/* The attention inputs of one layer from its projections, over every row of a
 * table (dense or paged, verify or prompt): each query and key head normed and
 * rotated, and the rows' keys and values appended to their streams' caches,
 * where the layer's attention call reads them. It goes between the layer's
 * projections and tf_attn / tf_attn_block / tf_attn_paged, which take q_out.
 * Window row i of a stream has position p = keys - rows + i. For a head's 64
 * values x with norm weight w, in fp32:
 *   n = x * w / sqrt(mean(x^2) + eps)
 *   y[j]    = n[j] cos(p f_j) - n[j+32] sin(p f_j)      f_j = theta^(-2j/64),
 *   y[j+32] = n[j+32] cos(p f_j) + n[j] sin(p f_j)      j < 32 (half-split)
 * rounded once to bf16. Angles are reduced exactly (p times a 64-bit fraction of
 * a turn) before they become fp32, so far positions are as good as near ones.
 * The rest of the caches is left as it is.
 *   q   bf16, row r's TF_NQ heads at q + r*q_stride (elements)
 *   k, v  bf16, row r's TF_NKV heads at k + r*k_stride, v + r*v_stride: the
 *         three may be slices of one projection's rows. v is copied.
 *   q_norm, k_norm  bf16 [TF_D], one weight for all query and all key heads
 *   q_out  bf16 [R][TF_NQ][TF_D]; may be q itself when q_stride is
 *          TF_NQ*TF_D. k and v must not lie in the caches.
 * A NaN or infinity in a head spreads over that head only. Strides are
 * multiples of 8. Calls on different layers may overlap; a call that appends
 * to a layer must not overlap attention on that layer. Errors: TF_EINVAL
 * (null, misaligned, stride below the row or no multiple of 8, q_out
 * overlapping an input, eps not positive and finite, theta below 1 or not
 * finite), TF_ERANGE (a stride beyond 2^32). */
int tf_qk_rows(const tf_segments* seg, int attn_layer, const void* q, int64_t q_stride,
               const void* k, int64_t k_stride, const void* v, int64_t v_stride,
               const void* q_norm, const void* k_norm, float eps, double theta,
               void* q_out, tf_cuda_stream stream);

/* Copies between pages of paged pools, in every given pool alike: keys
 * [0, keys[i]) of page src[i] to page dst[i], i < n_copies. For a fork (the
 * child's own copy of the parent's partly filled last page, before either
 * appends to it) and for moving pages (a compaction).
 *   pools   host array [n_pools] of device pointers, each a bf16 pool
 *           [n_pages][TF_NKV][page_keys][TF_D] (the K and V pools of any layers)
 *   src, dst  host arrays [n_copies] of page ids in [0, n_pages). A page may be
 *           a source several times; a destination is no other copy's source or
 *           destination (the copies run in no order). Chained moves take
 *           several calls.
 *   keys    host array [n_copies], 0..page_keys each, or NULL for whole pages;
 *           the rest of a destination page is left as it is
 * The lists are read before the call returns and travel with the launches, so
 * a captured graph repeats them. Errors: TF_EINVAL (null, misaligned or
 * overlapping pools, a bad page size, an id or a key count out of range, a
 * destination used twice or read), TF_ERANGE (n_pages > TF_MAX_PAGES, more
 * than 8,192 pools), TF_ENOMEM (host memory). */
int tf_pages_copy(void* const* pools, int n_pools, int32_t page_keys, int32_t n_pages,
                  const int32_t* src, const int32_t* dst, const int32_t* keys,
                  int n_copies, tf_cuda_stream stream);

/* ---- scaled pools and rows: 8 bits ------------------------------------------
 * A value of 8 bits is an e4m3 code under a scale 2^(b - 127) that neighbours
 * share, held as the byte b (0..254). The library writes the smallest scale, from
 * 2^-127 on, under which no finite value of its set saturates (the set's largest
 * magnitude is at most 464 times the scale), and codes to nearest even; a NaN or
 * an infinity becomes the code NaN and has no say on the scale. Rounding is off by
 * at most 2^-4 of a value, or 2^-10 of the scale where that is more (then below
 * 2^-17 of the set's largest).
 *
 * Scaled pools hold keys and values that way, half the bytes of a bf16 pool: the
 * scale of K, and of V, is shared by TF_SCALE_KEYS keys (slots 16 j .. 16 j + 15
 * of a page) of one head.
 *   pool    uint8 [n_pages][TF_NKV][page_keys][TF_D], codes
 *   scales  uint8 [n_pages][TF_NKV][page_keys / TF_SCALE_KEYS], at any address
 *
 * tf_paged_scaled_build and tf_paged_scaled_prompt_build are tf_paged_build and
 * tf_paged_prompt_build with a pool of scales beside each pool of codes (host
 * arrays [n_attn] of device pointers); no two pools, scales included, overlap.
 * Their tables serve the calls that a paged table serves:
 *   tf_qk_rows    codes the rows that it appends. A block of 16 keys takes the
 *                 scale of the rows before the window that it holds and of the
 *                 window's rows in it, and rows that it held are coded again where
 *                 the scale moves (the same values, but for those below 2^-14 of
 *                 the block's largest); slots past the window keep their bytes and
 *                 have no say. Pages that are filled in another way keep to the
 *                 format above.
 *   tf_attn_paged reads codes and scales (q and out bf16; the window's own rows
 *                 are read back as coded); a stream's bits depend on that stream
 *                 alone (a row's in tf_norm_rows and tf_linear_rows also on how many
 *                 rows the call has). Windows of 9 rows or more take a quarter of
 *                 the keys a chunk (2,048 at least, tf_chunk_keys at most), prompts
 *                 of few windows less than tf_chunk_keys too (tf_partials_bytes and
 *                 tf_segments_query tell the table's own sizes). P.V runs with fp16
 *                 weights and exact codes, summed in fp32. A weight there is taken
 *                 times its block's V scale, relative to its chunk's largest, and is
 *                 off by at most 2^-11 of itself, or 2^-31 of the row's largest
 *                 product where that is more (keys below do not count in P.V); a
 *                 block of V whose scale is more than 2^64 below its chunk's largest
 *                 counts as if 2^64 below. The tensor-core kernel (windows of 9 rows
 *                 or more, prompts; TF_ATTN_PATH as for tf_attn) takes a query as
 *                 the sum of two e4m3 parts: exact for elements down to 2^-9 of a
 *                 head's largest, smaller ones off by at most 2^-17 of it.
 *                 A NaN reaches the rows that see its key, no other. q, partials
 *                 and out lie apart. */
int tf_paged_scaled_build(const tf_stream* streams, int n_streams, const void* const* conv_state,
                          const void* const* conv_hist, const int32_t* pages, int32_t page_keys,
                          int32_t n_pages, const void* const* k_pool, const void* const* v_pool,
                          const void* const* k_scale, const void* const* v_scale,
                          int n_conv, int n_attn, tf_cuda_stream stream, tf_segments** out);
int tf_paged_scaled_prompt_build(int32_t rows, int32_t keys, int32_t kv_capacity,
                                 const void* const* conv_state, const int32_t* pages, int32_t page_keys,
                                 int32_t n_pages, const void* const* k_pool, const void* const* v_pool,
                                 const void* const* k_scale, const void* const* v_scale,
                                 int n_conv, int n_attn, tf_cuda_stream stream, tf_segments** out);

/* tf_pages_copy for scaled pools: the codes of keys [0, keys[i]) and the scales of
 * the blocks that hold them. Where keys[i] ends inside a block, the destination's
 * codes behind it stay and come under the copied scale.
 *   pools, scales  host arrays [n_pools] of device pointers
 * The other arguments, rules and errors are tf_pages_copy's. */
int tf_pages_copy_scaled(void* const* pools, void* const* scales, int n_pools, int32_t page_keys, int32_t n_pages,
                         const int32_t* src, const int32_t* dst, const int32_t* keys, int n_copies,
                         tf_cuda_stream stream);

/* The residual's addition, the RMS norm and the 8-bit coding of each row, between
 * a projection's output and the next projection's input:
 *   h = bf16(x + res)            (h = x when res is NULL)
 *   n = h * w / sqrt(mean(h^2) + eps)                      in fp32
 * coded with a scale for each TF_SCALE_COLUMNS columns.
 *   x, res  bf16, row r at x + r*x_stride, res + r*res_stride (elements); res may
 *           be NULL, and sum is then NULL too
 *   w       bf16 [width]
 *   sum     bf16, row r at sum + r*sum_stride: h, the residual of the next addition;
 *           may be x or res itself (at the same stride)
 *   codes   uint8 [R][width]
 *   scales  uint8 [R][width / TF_SCALE_COLUMNS], at any address
 * width is a multiple of TF_SCALE_COLUMNS, strides are multiples of 8; other
 * overlaps of an output with anything are refused. A NaN or an infinity in a row
 * makes that row's codes NaN (or, where the root is infinite, 0); finite rows whose
 * mean of squares passes fp32 (h beyond some 2^64) become 0 too. Sums run in an
 * order that R and width fix. Needs no table; R == 0 is a no-op. Errors: TF_EINVAL
 * (null, one of res and sum alone, misaligned,
 * overlaps, a bad width or stride, eps not positive and finite, another device's
 * memory), TF_ERANGE (R > 2^24, width > TF_NORM_MAX_WIDTH, a stride beyond 2^32). */
#define TF_NORM_MAX_WIDTH (1 << 14)
int tf_norm_rows(const void* x, int64_t x_stride, const void* res, int64_t res_stride, const void* w, float eps,
                 int R, int width, void* sum, int64_t sum_stride, void* codes, void* scales,
                 tf_cuda_stream stream);

/* Rows times a matrix of 4-bit weights (a projection, or the logits):
 *   y[r][n] = s[n] * sum_k x[r][k] * g[n][k / 32] * (c[n][k] - 8)
 * summed in fp32 and rounded once to bf16.
 *   x         x_scales NULL: bf16, row r at x + r*x_stride (elements, a multiple
 *             of 8). Otherwise codes, row r at x + r*x_stride (a multiple of 16),
 *             with x_scales uint8 [R][K / TF_SCALE_COLUMNS] (at any address): what
 *             tf_norm_rows writes
 *   w         uint8 [N][K / 2]: codes c in 0..15, the even k in the low four bits
 *   w_scales  uint8 [N][K / TF_SCALE_COLUMNS] (at any address): g, e4m3
 *   s         float [N]
 *   y         bf16, row r at y + r*y_stride (any 2-byte address and stride >= N);
 *             overlaps nothing else
 * K is a multiple of TF_SCALE_COLUMNS. Up to 32 rows take the weights from HBM once;
 * every 32 rows decode them anew, so hundreds of rows run far below the rate of a
 * bf16 matrix product (some 300 of 1,900 TFLOP/s on a GB300).
 * Values of x below bf16's smallest, 2^-133, are rounded to multiples of it; the
 * other products are exact. Sums run in an order that R, K, N and the device's
 * number of SMs fix: a row's bits may differ between calls of different R, not with
 * its place among the rows or with an address. A NaN or an infinity in a row of x
 * reaches that row of y only. Needs no table; R == 0 is a no-op. Errors: TF_EINVAL
 * (null, misaligned, overlaps, a bad K or stride, N < 1, another device's memory),
 * TF_ERANGE (R > TF_LINEAR_MAX_ROWS, K > TF_LINEAR_MAX_INPUTS,
 * N > TF_LINEAR_MAX_OUTPUTS, a stride beyond 2^32). */
#define TF_LINEAR_MAX_ROWS (1 << 20)
#define TF_LINEAR_MAX_INPUTS (1 << 20)
#define TF_LINEAR_MAX_OUTPUTS (1 << 24)
int tf_linear_rows(const void* x, int64_t x_stride, const void* x_scales, int R, int K, const void* w,
                   const void* w_scales, const float* s, int N, void* y, int64_t y_stride,
                   tf_cuda_stream stream);

/* ---- failures on the device ------------------------------------------------
 * The tensor-core attention kernel (tf_attn*, streams of 9 rows or more and
 * prompt windows) and the Markov chain (tf_markov_chain) wait on barriers
 * that other warps or CTAs of the same launch complete. Every such wait is
 * bounded by the wait limit below. A CTA whose wait runs out gives up: it
 * lets its own copies and MMAs in flight land, writes NaN in place of the
 * results it could not compute (attention records; Markov rows get pick -1
 * and flag bit 1), sets a bit in the table's status word and returns. Nothing
 * faults and the context stays usable; the launch itself still reports
 * success, so the failure is read with tf_segments_status (the review of
 * the drafter's held path asks that a failure flag of asynchronous work
 * reach the host: PR #1391, its review of the held path).
 *
 * tf_set_wait_limit_ns sets the limit (process-wide) for every later launch;
 * a launch captured in a CUDA graph keeps the limit it was captured with.
 * Default TF_WAIT_LIMIT_DEFAULT_NS (2 s), at most TF_WAIT_LIMIT_MAX_NS
 * (TF_ERANGE beyond). 0 makes a kernel give up at the first wait that is
 * not already complete when first tested: a way to exercise the failure
 * path, not a setting for real work. tf_wait_limit_ns returns the current
 * limit. */
#define TF_WAIT_LIMIT_DEFAULT_NS 2000000000ull
#define TF_WAIT_LIMIT_MAX_NS 60000000000ull
int tf_set_wait_limit_ns(uint64_t ns);
uint64_t tf_wait_limit_ns(void);

/* Status word bits of a table. */
#define TF_STATUS_ATTN_TIMEOUT   1u   /* the tensor-core attention kernel gave up a wait */
#define TF_STATUS_MARKOV_TIMEOUT 2u   /* the Markov chain gave up a wait */

/* Read and clear a table's status word. Synchronises `stream` (so it must not
 * be called during stream capture), copies the word to *bits (if bits is not
 * NULL) and, when it is nonzero, zeroes the table's cross-CTA scratch
 * (attention merge counters, work counters, Markov step keys and barrier) and
 * the word itself, so the next calls on the table start clean. No call on the
 * table may be in flight on another stream meanwhile.
 * Returns TF_OK (no kernel gave up since the last check), TF_ETIMEOUT (one
 * did: every result the table's calls wrote since the last check is invalid),
 * TF_EINVAL (NULL table) or TF_ECUDA. */
int tf_segments_status(tf_segments* seg, tf_cuda_stream stream, uint32_t* bits);

/* Name of a status code. */
const char* tf_strerror(int status);

/* The CUDA error code behind the last TF_ECUDA of this thread (0 if none). */
int tf_last_cuda_error(void);

#ifdef __cplusplus
}
#endif
#endif /* TF_H_INCLUDED */
