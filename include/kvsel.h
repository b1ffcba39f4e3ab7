/*
 * kvsel.h — C ABI of libkvsel, GB300 (sm_103a) SnapKV observation-window
 * KV-cache selection.
 *
 * Method: page "SnapKV: choosing the KV cache of a long prompt with an
 * observation window" (SnapKV：用观察窗口为长提示词选择 KV Cache,
 * charlestar.github.io, 2026-10-20). For every (layer, sequence, head):
 *   - partition ("要缩小的是提示词缓存" section): prompt length L, window = the
 *     last W tokens, prefix P = L - W, budget C keeps the whole window plus
 *     C - W prefix positions;
 *   - votes ("投票必须来自完整提示词的因果 softmax" section): the W window
 *     queries attend to all L keys with scale 1/sqrt(D) under a causal mask,
 *     the softmax denominator runs over every visible position, and each
 *     prefix position's vote is the sum of its probabilities over the W rows;
 *   - pooling and top-k ("池化把一个峰值扩展成邻域偏好" section): 1-D pooling
 *     of the prefix votes (odd width, stride 1, zero padding; the average
 *     divides by the full width at the edges; or max), then the C - W prefix
 *     positions with the highest pooled score, ties to the smaller position;
 *   - gather ("从 Q 和 K 开始算一次完整选择" section): the kept positions of
 *     K and V with one index list; L < C keeps everything (bypass).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Data layout (row-major, no padding, "layers" outermost):
 *   q_win   [num_layers][num_seqs * W][H][D]  window queries; rows b*W .. b*W+W-1
 *                                             are sequence b's positions P_b .. L_b-1
 *   K, V    [num_layers][T][H][D]             packed prompts (RoPE already applied);
 *                                             sequence b owns tokens
 *                                             seq_offsets[b] .. seq_offsets[b+1]-1
 *   votes, pooled [num_layers][H][T] fp32     entry j of sequence b's token range holds
 *                                             prefix position j's score (j < P_b); window
 *                                             positions hold 0
 *   out_idx [num_layers][T_out][H] int32      positions within the sequence
 *   out_K, out_V [num_layers][T_out][H][D]    same dtype as K and V
 * with T = seq_offsets[num_seqs] and T_out = kvsel_out_tokens(shape, C)
 * = sum_b min(L_b, C); sequence b's output rows start at sum_{b'<b} min(L_b', C).
 * Within a sequence's C output rows: the C - W kept prefix positions in the
 * order (highest pooled score first, equal scores by smaller position), then
 * the window positions P..L-1 ascending. A sequence with L < C (bypass) keeps
 * positions 0..L-1 in order.
 *
 * Memory: every data pointer is device memory allocated by the caller, except
 * shape->seq_offsets, which is HOST memory (it decides launch shapes and which
 * sequences bypass). The library never frees caller memory.
 *
 * Streams and synchronisation: `stream` is a cudaStream_t (NULL = legacy
 * default stream). Calls enqueue work and return without waiting for it.
 * kvsel_score, kvsel_window_logits and kvsel_snapkv use an internal per-device
 * workspace that the library allocates with cudaMalloc and grows on demand
 * (growing synchronises the device); kvsel_release() frees it. Calls that use
 * the workspace on one device must be ordered with one another (one stream,
 * or events between streams): overlapping calls race on it.
 *
 * Errors: arguments are checked on the host before any launch; a rejected
 * call launches nothing. Conditions only the GPU can see (a non-finite window
 * logit, a gather index out of range, a bounded wait that ran out) are
 * recorded in a per-device status word; kvsel_device_status() reads it.
 * Every launch failure returns KVSEL_ERR_CUDA.
 */
#ifndef KVSEL_H_
#define KVSEL_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t kvsel_status;
enum {
  KVSEL_OK = 0,
  KVSEL_ERR_INVALID_ARG = 1,  /* an argument rule failed (see each call) */
  KVSEL_ERR_UNSUPPORTED = 2,  /* valid, but beyond a documented limit */
  KVSEL_ERR_NONFINITE = 3,    /* device: a window logit was NaN or +-Inf */
  KVSEL_ERR_TIMEOUT = 4,      /* device: a bounded wait ran out */
  KVSEL_ERR_CUDA = 5,         /* a CUDA runtime call failed */
  KVSEL_ERR_BAD_INDEX = 6,    /* device: an index, page number or length was out of range */
  KVSEL_ERR_NO_PAGES = 7,     /* device: the pool had too few free pages */
  KVSEL_ERR_SHARED_PAGE = 8   /* device: a page to be rewritten is held by several sequences */
};

enum { KVSEL_POOL_AVG = 0, KVSEL_POOL_MAX = 1 };
enum { KVSEL_BF16 = 0, KVSEL_F32 = 1 };

/* Shape of one call. num_layers >= 1 and num_heads >= 1 and head_dim >= 1;
 * num_seqs >= 0 (0 = nothing to do); dtype is KVSEL_BF16 or KVSEL_F32 (for
 * q_win, K, V and the gathered outputs). seq_offsets: HOST array of
 * num_seqs + 1 entries, seq_offsets[0] == 0, nondecreasing.
 * Grouped-query attention (page section "GQA 下的缓存节省不能只算 C 除以 L"):
 * num_heads counts the query heads H (q_win and every per-head output) and
 * num_kv_heads the heads H_kv of K and V: 0 (= num_heads) or a divisor of
 * num_heads (else INVALID_ARG). Query head h then reads K/V head
 * h / (H / H_kv), the expanded (repeat_kv) reading the page describes; the
 * group-shared selection is kvsel_snapkv_grouped. */
typedef struct kvsel_shape {
  int32_t num_layers;
  int32_t num_seqs;
  int32_t num_heads;
  int32_t head_dim;
  int32_t dtype;
  int32_t num_kv_heads; /* 0 = num_heads */
  const int64_t* seq_offsets;
} kvsel_shape;

/* Library version string (static storage). */
const char* kvsel_version(void);

/* Human-readable name of a status code (static storage). */
const char* kvsel_status_string(kvsel_status status);

/* T_out = sum_b min(L_b, C), the number of output rows per layer and head.
 * Returns -1 if the shape or C (< 1) is invalid. Host only, no GPU work. */
int64_t kvsel_out_tokens(const kvsel_shape* shape, int32_t C);

/* Which window-logit kernel a call with this shape takes: 1 = the tensor-core
 * kernel (TMA + tcgen05, bf16, D in {64,128}, W <= 64), 3 = the tensor-core
 * two-pass kernel (the same shapes, on sequences longer than 64 of the
 * kernel's work items: row statistics first, then the votes from logits
 * recomputed from K, which the second pass reads from L2), 0 = the CUDA-core
 * kernel (any other supported shape), -1 = the call would be rejected.
 * C = 0 means "score every sequence" (kvsel_score); otherwise sequences with
 * L < C are not scored. Host only; queries the current device. */
int32_t kvsel_score_path(const kvsel_shape* shape, int32_t W, int32_t C);

/* Window logits z[r][j] = q_{P_b + r} . k_j / sqrt(D) for every sequence b,
 * window row r < W and token j of b (no mask applied), written to
 * logits[num_layers][H][W][T] (fp32, row r of column j belongs to j's
 * sequence). Rules: W >= 1, W <= L_b for every b, non-null pointers when
 * T > 0. Same kernels as kvsel_score, stopped before the softmax; for tests
 * and diagnostics. */
kvsel_status kvsel_window_logits(const kvsel_shape* shape, const void* q_win, const void* K,
                                 int32_t W, float* logits, void* stream);

/* Votes and pooled scores of every sequence ("votes" and "pooling" sections).
 * votes (may be NULL) and pooled: [num_layers][H][T] fp32, prefix positions
 * filled, window positions 0. Rules: W >= 1, W <= L_b for every b, pool_kind
 * in {AVG, MAX}, pool_k odd and >= 1, non-null q_win/K/pooled when T > 0.
 * Device status: NONFINITE if a window logit (any window row, any token of
 * the sequence) is not finite. */
kvsel_status kvsel_score(const kvsel_shape* shape, const void* q_win, const void* K, int32_t W,
                         int32_t pool_kind, int32_t pool_k, float* votes, float* pooled,
                         void* stream);

/* kvsel_score without any device allocation, for callers that cannot call
 * cudaMalloc (an allocator they must not bypass, or a context where
 * allocating is not permitted). The paper has no counterpart; it is a
 * deployment variant of kvsel_score with the same arguments, rules and
 * results, except that votes must be non-NULL (the caller provides it).
 * Scratch: a fixed 8 MiB array in device memory, part of the library image
 * (every GPU that loads the library holds it until the process exits). The
 * first call on a device looks up that array's device address (once per
 * device, with the device current); make that first call before any stream
 * capture. Calls whose scratch need exceeds 8 MiB return
 * KVSEL_ERR_UNSUPPORTED and launch nothing; kvsel_score_static_bytes gives
 * the exact need of a call. All calls on a device share the array and each
 * call resets what must start out empty, so calls that overlap on the GPU
 * (different streams without ordering) race. */
kvsel_status kvsel_score_static(const kvsel_shape* shape, const void* q_win, const void* K,
                                int32_t W, int32_t pool_kind, int32_t pool_k, float* votes,
                                float* pooled, void* stream);

/* Scratch bytes kvsel_score_static needs for this shape, window and the
 * current device (the sequence tables, the cross-chunk statistics slots and
 * the merged statistics of the scoring kernel it would launch; q_win and K
 * are assumed 16-byte aligned), or -1 if the arguments break a rule of
 * kvsel_score. At most 8 MiB is accepted. Host only. */
int64_t kvsel_score_static_bytes(const kvsel_shape* shape, int32_t W);

/* Top-(C - W) selection from given pooled scores ([num_layers][H][T] fp32,
 * only prefix entries are read) into out_idx ([num_layers][T_out][H] int32);
 * bypass sequences (L < C) get 0..L-1. Ordering of scores: IEEE order with
 * -0 == +0; NaN ranks below every number and sets NONFINITE. Rules: W >= 1,
 * C > W, W <= L_b for every b. Limit: C - W <= 16384 (else UNSUPPORTED). */
kvsel_status kvsel_select(const kvsel_shape* shape, const float* pooled, int32_t W, int32_t C,
                          int32_t* out_idx, void* stream);

/* Gather: out_K[row] = K[idx], out_V[row] = V[idx] for every output row, the
 * same idx for K and V, with out_idx as produced by kvsel_select. Rules: C >= 1,
 * non-null pointers when T_out > 0. Device status: BAD_INDEX if an index is
 * outside [0, L_b) (that row is left unwritten). Bit-exact copy. */
kvsel_status kvsel_compact(const kvsel_shape* shape, const void* K, const void* V,
                           const int32_t* out_idx, int32_t C, void* out_K, void* out_V,
                           void* stream);

/* The whole path: score -> pool -> select -> gather, with no host
 * synchronisation in between. Rules: those of kvsel_score and kvsel_select
 * (W >= 1, C > W, W <= L_b for every b, odd pool_k >= 1, pool_kind valid,
 * C - W <= 16384). Sequences with L < C are copied unscored. */
kvsel_status kvsel_snapkv(const kvsel_shape* shape, const void* q_win, const void* K,
                          const void* V, int32_t W, int32_t C, int32_t pool_kind,
                          int32_t pool_k, int32_t* out_idx, void* out_K, void* out_V,
                          void* stream);

/* Group-shared selection under grouped-query attention: one selection per
 * (layer, sequence, K/V head), shared by the G = H / H_kv query heads of the
 * group, so the kept cache has H_kv heads (the page leaves this design open;
 * our reading): each query head computes its own causal-softmax votes against
 * the group's keys, the group's vote of a prefix position is the sum of its
 * G heads' votes, and pooling, the top-(C - W) selection and the gather then
 * run once per group. On the tensor cores with G a power of two and G * W <=
 * 64 the G heads are scored together (K read once per group; the sum is then
 * taken over all G * W rows at once, equal to the head-ordered sum within
 * fp32 rounding). Layouts: q_win [num_layers][S * W][H][D],
 * K and V [num_layers][T][H_kv][D]; out_idx [num_layers][T_out][H_kv] int32,
 * out_K and out_V [num_layers][T_out][H_kv][D]. Rules and limits those of
 * kvsel_snapkv. With H_kv == H it is kvsel_snapkv. */
kvsel_status kvsel_snapkv_grouped(const kvsel_shape* shape, const void* q_win, const void* K,
                                  const void* V, int32_t W, int32_t C, int32_t pool_kind,
                                  int32_t pool_k, int32_t* out_idx, void* out_K, void* out_V,
                                  void* stream);

/* kvsel_snapkv with the cache in host memory: q_win, K, V, out_idx, out_K and
 * out_V are HOST pointers with kvsel_snapkv's layouts. q_win and K are copied
 * to the device one layer at a time on an internal copy stream (two device
 * slots held by the library, so a layer's copy overlaps the previous layer's
 * kernels); V and the three outputs must be page-locked host memory
 * (cudaHostAlloc or cudaHostRegister): the gather reads the kept V rows and
 * writes the outputs in place, so of V only the kept rows cross the link.
 * Pinned q_win and K copy fastest. Asynchronous and ordered on `stream`: it
 * starts after the work already queued there, and the outputs are complete
 * when `stream` reaches the point after the call; the host buffers must stay
 * valid until then. Rules and limits those of kvsel_snapkv; INVALID_ARG also
 * when V or an output is not page-locked host memory. */
kvsel_status kvsel_snapkv_host(const kvsel_shape* shape, const void* q_win, const void* K,
                               const void* V, int32_t W, int32_t C, int32_t pool_kind,
                               int32_t pool_k, int32_t* out_idx, void* out_K, void* out_V,
                               void* stream);

/* ---------------------------------------------------------------------------
 * Jacap scorer (pages "Jacap reading notes" / "Jacap technical review",
 * section 6 (practical approximation) and section 7 (Algorithm 1): per (layer,
 * sequence, head), over the prefix pool 0 .. P-1 with P = L - W:
 * z_i = k_i . mu_Q / (tau sqrt(D)), alpha = softmax(z) over the pool,
 * kappa_i = k_i^T Lambda_Q k_i, w_i = [alpha_i (1 - alpha_i)]^2 kappa_i / D,
 * A = I + sum_i w_i v_i v_i^T, r_i = w_i v_i^T A^{-1} v_i (the value as the
 * output proxy); mu_Q and the diagonal Lambda_Q from the W window queries by
 * the running mean and second moment of section 11 (Algorithm 2) with rate
 * beta and floor eps, started from the first window query (our reading for a
 * prompt-time selection). Tensor-core path only: bf16, D = 128, num_kv_heads
 * equal to num_heads (UNSUPPORTED otherwise). Argument rules of kvsel_score /
 * kvsel_snapkv plus tau > 0 finite, 0 <= beta < 1, eps >= 0 finite
 * (INVALID_ARG). Device status: NONFINITE if a statistic or the capacity
 * matrix is not finite or not positive definite.
 * ------------------------------------------------------------------------- */

/* Scores r [num_layers][H][T] fp32 (caller owned): r at the prefix positions
 * of every sequence with L > W, 0 elsewhere. Layouts as kvsel_score. */
kvsel_status kvsel_jacap_score(const kvsel_shape* shape, const void* q_win, const void* K,
                               const void* V, int32_t W, float tau, float beta, float eps,
                               float* scores, void* stream);

/* The whole Jacap path: scores, the top C - W prefix positions by (-r, j) (the
 * selection of kvsel_select, no pooling), then the window, and the gather of
 * the kept K and V rows; sequences with L < C are copied unscored. Outputs as
 * kvsel_snapkv. */
kvsel_status kvsel_jacap(const kvsel_shape* shape, const void* q_win, const void* K,
                         const void* V, int32_t W, int32_t C, float tau, float beta, float eps,
                         int32_t* out_idx, void* out_K, void* out_V, void* stream);

/* ---------------------------------------------------------------------------
 * Decode-side consumer of a cache (page section "Why deleting positions
 * changes the output" (删除位置为什么会改变输出): one future query, its softmax
 * over the cache rows, the value sum, and the probability mass the full cache
 * gives the kept rows; section "The current prefill still reads the full K/V"
 * (当前 prefill 仍读完整 K/V，压缩缓存服务后续 decode): after g generated
 * tokens the cache holds min(L, C) + g rows; section "Cache slots cannot
 * stand in for the original RoPE positions" (缓存槽位不能代替 RoPE 的原始位置):
 * the next token's logical position is L + g, its physical slot min(L, C) + g).
 * ------------------------------------------------------------------------- */

/* One query per (layer, sequence, query head) attends, unmasked, to every row
 * of its sequence's cache followed by its g appended rows, with the scale
 * 1/sqrt(D). `shape` describes the cache: seq_offsets are cache row offsets
 * (for a compacted cache from kvsel_snapkv the running sum of min(L_b, C);
 * for the full cache the prompt offsets), num_heads the query heads H,
 * num_kv_heads (0 = H) the cache heads; query head h reads cache head
 * h / (H / H_kv). Layouts (dtype of the shape, rows of D elements, 16-byte
 * aligned): q [num_layers][num_seqs][H][D]; K, V [num_layers][T][H_kv][D];
 * K_new, V_new [num_layers][num_seqs * g][H_kv][D] (sequence b's appended rows
 * at b*g .. b*g + g - 1; may be NULL when g == 0). Outputs (fp32, caller
 * owned, device memory): out [num_layers][num_seqs][H][D] the attention
 * output; lse [num_layers][num_seqs][H] the natural log of the sum of
 * exp(q . k / sqrt(D)) over the attended rows, or NULL. Permuting a
 * sequence's cache rows (K and V together) does not change the result, so
 * kvsel_snapkv's score-ordered rows can be read as they are. Rules:
 * INVALID_ARG for g < 0, a sequence with no rows at all (cache + g == 0),
 * NULL or misaligned pointers; UNSUPPORTED for D not in {64, 128}. Device
 * status: NONFINITE if a sum or an output is not finite. Asynchronous. */
kvsel_status kvsel_decode_attention(const kvsel_shape* shape, const void* q, const void* K,
                                    const void* V, int32_t g, const void* K_new,
                                    const void* V_new, float* out, float* lse, void* stream);

/* ---------------------------------------------------------------------------
 * Reverse-mask attention of the counter-causal scorer (page "来自未来的信号：
 * 用反因果惊奇度做 KV Cache 淘汰" (signals from the future: KV-cache eviction by
 * counter-causal surprise), section 3.2, steps 1, 3 and 5; section 4,
 * Algorithm 3). The part that needs no model weights: every cached row i of
 * a sequence attends, with the scale 1/sqrt(D), to the cached rows j of the
 * same sequence whose original position is larger than its own (a strictly
 * upper-triangular mask in position order), reusing the cached K and V with
 * queries recomputed at the original positions.
 * ------------------------------------------------------------------------- */

/* out_i = sum_{j: pos_j > pos_i} softmax_j(q_i . k_j / sqrt(D)) v_j and lse_i
 * = ln sum_j exp(q_i . k_j / sqrt(D)) over the same j; a row with no such j
 * (the last position) gets out = 0 and lse = -inf (the page gives it the
 * largest surprise). `shape`: seq_offsets are the cache rows of each sequence,
 * num_heads the query heads H, num_kv_heads (0 = H) the cache heads; query head
 * h reads cache head h / (H / H_kv). Layouts (bf16, D = 128, rows 16-byte
 * aligned): Q [num_layers][T][H][D]; K, V [num_layers][T][H_kv][D];
 * positions [T] int32, the sequence-relative original position of each row
 * (NULL: the row order; a refresh that reorders the memory passes them; equal
 * positions do not attend to each other). Outputs (fp32, caller-owned device
 * memory): out [num_layers][T][H][D] (16-byte aligned); lse
 * [num_layers][H][T] natural log, or NULL. Rules: INVALID_ARG for NULL or
 * misaligned pointers; UNSUPPORTED for a dtype other than bf16, D != 128,
 * misaligned Q/K/V, or num_layers * T >= 2^31. Device status: NONFINITE if a
 * row's max or sum is not finite; TIMEOUT if a bounded wait ran out.
 * Asynchronous on `stream`. */
kvsel_status kvsel_reverse_attention(const kvsel_shape* shape, const void* Q, const void* K,
                                     const void* V, const int32_t* positions, float* out,
                                     float* lse, void* stream);

/* Per instance (n of them, e.g. layers * seqs * heads): the retained mass
 * mass[i] = exp(lse_keep[i] - lse_full[i]) (the full-cache probability of the
 * rows that the compacted cache kept, when lse_keep comes from the compacted
 * cache and lse_full from the full one, both with the same appended rows) and
 * err[i] = || out_full[i] - out_keep[i] ||_2 over the D values. All device
 * pointers, fp32. INVALID_ARG for n < 0, D < 1 or NULL pointers (n > 0). */
kvsel_status kvsel_decode_quality(int64_t n, int32_t D, const float* lse_keep,
                                  const float* lse_full, const float* out_keep,
                                  const float* out_full, float* mass, float* err, void* stream);

/* Host bookkeeping for a prompt shape (seq_offsets = prompt offsets), budget
 * C and g appended tokens per sequence: physical_length[b] = min(L_b, C) + g
 * (also the slot the next token is written to) and next_logical[b] = L_b + g
 * (its position for RoPE). Host arrays of num_seqs entries. INVALID_ARG for
 * C < 1, g < 0 or NULL arrays (num_seqs > 0). */
kvsel_status kvsel_cache_lengths(const kvsel_shape* shape, int32_t C, int32_t g,
                                 int64_t* physical_length, int64_t* next_logical);

/* ---------------------------------------------------------------------------
 * Paged caches. A server keeps its sequences' caches in pages of a pool; a
 * cache that kvsel_snapkv or kvsel_select has cut is read, grown, cut again
 * and shared there with the four calls below. They take every length, table
 * and index from device memory, allocate nothing and copy nothing from the
 * host, so one captured graph serves steps whose lengths differ; their scratch
 * is the caller's `workspace` (two calls that may overlap on the GPU, or two
 * graphs that may replay at once, need one each; it needs no initial value).
 * Make the first call on a device before a stream capture (it looks up the
 * status word's address).
 *
 * Pool: K and V [num_layers][num_pages][page_size][H_kv][D], K and V with the
 * same strides. layer_stride and page_stride are in elements, 0 = dense (the
 * layout above); others allow for a pool that interleaves layers or K and V,
 * for instance. Table: [num_seqs][table_width] int32 page numbers, one table for
 * every layer; row j of sequence b (its physical slot, see kvsel_cache_lengths)
 * is row j % page_size of page table[b][j / page_size]. Lengths: int32 rows per
 * sequence, 0 allowed. Only the entries that the lengths reach are read.
 * Rules of every call: INVALID_ARG for a NULL or broken descriptor (counts < 1,
 * num_pages < 0, a stride below a page's elements), NULL pointers where data is
 * needed, K or V or a stride not 32-byte aligned; UNSUPPORTED for D not in
 * {64, 128}, a page_size that is no power of two, a pool of 2^31 or more rows or
 * 128 GiB or more per layer, a table of 2^30 or more rows per sequence. A packed
 * cache [num_layers][T][H_kv][D] is a pool of T pages of one row.
 * ------------------------------------------------------------------------- */
typedef struct kvsel_pages {
  int32_t num_layers;
  int32_t num_pages;
  int32_t page_size;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t dtype;
  int64_t layer_stride; /* elements, 0 = dense */
  int64_t page_stride;  /* elements, 0 = dense */
  void* K;
  void* V;
} kvsel_pages;

/* Rows of new tokens: token n of layer l is `heads` x D contiguous elements at
 * data + l * layer_stride + n * token_stride (elements; each row 16-byte
 * aligned), so q, k and v may be slices of one fused projection. */
typedef struct kvsel_rows {
  const void* data;
  int64_t layer_stride;
  int64_t token_stride;
} kvsel_rows;

/* Position rotation of the first rot_dim elements of a head. Pair i < rot_dim/2
 * turns by the angle position * inv_freq[i] (device, fp32; the angle is off by less
 * than 2^-20 + |position * inv_freq[i]| 2^-43 rad): elements (i, i + rot_dim/2), or
 * (2i, 2i + 1) when interleaved; both results are multiplied by `scale`.
 * rot_dim 0: no rotation. kvsel_rope_frequencies fills inv_freq and scale. */
typedef struct kvsel_rope {
  int32_t rot_dim;
  int32_t interleaved;
  const float* inv_freq;
  float scale;
} kvsel_rope;

enum {
  KVSEL_ROPE_PLAIN = 0,  /* inv_freq[i] = base^(-2i/rot_dim) */
  KVSEL_ROPE_LINEAR = 1, /* all divided by factor */
  KVSEL_ROPE_BASE = 2,   /* base * factor^(rot_dim / (rot_dim - 2)) in place of base */
  KVSEL_ROPE_PARTS = 3   /* pairs of fewer than `low` turns over original_len rows divided by
                            factor, of more than `high` left, in between interpolated linearly
                            in the number of turns; scale = 1 + 0.1 ln(factor) */
};

/* Host only: inv_freq[rot_dim / 2] (HOST array, computed in fp64, rounded once)
 * and *scale (1 but for PARTS) for a context `factor` times as long as the
 * `original_len` rows that a model was made for. INVALID_ARG for rot_dim < 2 or
 * odd, base <= 1, factor < 1, an unknown kind, NULL pointers; for BASE with
 * rot_dim 2; for PARTS with original_len < 1 or not 0 < low < high. */
kvsel_status kvsel_rope_frequencies(int32_t rot_dim, double base, int32_t kind, double factor,
                                    int64_t original_len, double low, double high,
                                    float* inv_freq, float* scale);

/* New tokens into a paged cache, in one pass: the norm of every query and key
 * head, x * rsqrt(mean(x^2) + eps) * weight (q_weight, k_weight
 * [num_layers][D] of the pool's dtype; NULL = no norm), then the rotation to
 * the token's logical position, then q to q_out and k, v to the cache. Sums
 * and rotation in fp32, one rounding at the end; v is copied.
 *   q: num_heads heads a token (NULL: keys and values only); q_out
 *   [num_layers][num_tokens][num_heads][D] dense, may be q's own memory when q
 *   is dense too. k, v: H_kv heads a token (both NULL: queries only).
 *   positions [num_tokens] int32 logical positions (needed when rotating).
 *   cache_pos [num_tokens] int32: the row of the token's sequence that k and v
 *   go to, negative = nowhere (a padding token; its q is written all the same).
 *   seqs [num_tokens] int32: the token's sequence, NULL = token n belongs to
 *   sequence n. table NULL: cache_pos is the row of the pool itself (seqs and
 *   num_seqs are not used), for a packed cache.
 * Two tokens must not name the same row. Rules: INVALID_ARG for negative
 * counts, eps < 0 or not finite, misaligned rows, seqs NULL with num_tokens >
 * num_seqs, k without v; UNSUPPORTED for a rot_dim that is no multiple of 16 or
 * above D, for num_heads + 2 * H_kv > 65535, and for num_layers * num_tokens *
 * (num_heads + 2 * H_kv) >= 2^32. Device status: BAD_INDEX
 * for a sequence, row or page out of range (that token's k and v are not
 * written). Asynchronous; capturable. */
kvsel_status kvsel_paged_append(const kvsel_pages* pages, int32_t num_tokens, int32_t num_heads,
                                const kvsel_rows* q, const kvsel_rows* k, const kvsel_rows* v,
                                const kvsel_rope* rope, const void* q_weight,
                                const void* k_weight, float eps, const int32_t* positions,
                                int32_t num_seqs, const int32_t* table, int32_t table_width,
                                const int32_t* seqs, const int32_t* cache_pos, void* q_out,
                                void* stream);

/* kvsel_decode_attention over a paged cache: one query per (layer, sequence,
 * query head) attends to the first lens[b] rows of its sequence. q
 * [num_layers][num_seqs][num_heads][D] (the pool's dtype, 16-byte aligned),
 * query head h reads cache head h / (num_heads / H_kv). out
 * [num_layers][num_seqs][num_heads][D] fp32 (16-byte aligned), lse
 * [num_layers][num_seqs][num_heads] fp32 natural log, or NULL. A sequence of
 * length 0 gets out = 0, lse = -inf. Rows behind the length are never read.
 * workspace: kvsel_paged_attention_bytes(pages, num_seqs, num_heads) bytes, 16-byte
 * aligned. Calls with the same arguments give the same bits (other lengths in the
 * batch may change a sequence's last bits: the work is split by all of them). Rules:
 * INVALID_ARG for num_heads that H_kv does not divide, a workspace that is too
 * small or misaligned; UNSUPPORTED for num_seqs > 8192, num_layers * num_seqs *
 * num_heads >= 2^31 or num_seqs * table_width * page_size > 2^34. Device status:
 * BAD_INDEX for a length outside [0, table_width * page_size] (taken as the
 * nearer end) or a page out of range (its rows are left out), NONFINITE if a sum
 * or an output is not finite (fp32: also for values of 2^127 or more).
 * Asynchronous; capturable. */
kvsel_status kvsel_paged_attention(const kvsel_pages* pages, int32_t num_seqs, int32_t num_heads,
                                   const void* q, const int32_t* table, int32_t table_width,
                                   const int32_t* lens, float* out, float* lse, void* workspace,
                                   int64_t workspace_bytes, void* stream);

/* Workspace bytes of kvsel_paged_attention on the current device, or -1 if a rule is
 * broken. Does not depend on the lengths. Host only. */
int64_t kvsel_paged_attention_bytes(const kvsel_pages* pages, int32_t num_seqs,
                                    int32_t num_heads);

/* Cuts paged caches to their kept rows, in place. keep_idx
 * [num_layers][keep_rows][H_kv] int32 (kvsel_select's or kvsel_snapkv_grouped's
 * out_idx, any order): entries keep_offsets[b] .. keep_offsets[b+1]-1 are sequence
 * b's kept rows, n of them, distinct, in [0, lens[b]). Afterwards slots 0 .. n-1
 * of the sequence hold the kept rows: a kept row j < n stays at slot j, and the
 * slots left over, ascending, take the kept rows j >= n in the list's order (a
 * future query's result does not depend on the order of the rows). Only rows
 * that change their slot are read and written; what lies in slots >= n is
 * left as it is, and kvsel_pages_update then frees their pages. slot_pos
 * [num_layers][keep_rows][H_kv] int32 (or NULL; not keep_idx's own memory): the row that each
 * slot now holds.
 * keep_offsets [num_seqs + 1] int32 on the device, nondecreasing from 0.
 * max_keep: an upper bound on n (0: nothing is done). ref [num_pages] int32 (or NULL: not checked): the
 * references from kvsel_pages_update; a sequence whose slots 0 .. n-1 touch a page with
 * ref > 1 while n < lens[b] is left whole and SHARED_PAGE recorded.
 * Rules: INVALID_ARG for num_seqs < 0, max_keep < 0, keep_rows < 0; UNSUPPORTED for
 * max_keep > 32768 or num_layers * num_seqs * H_kv >= 2^31. Device status: BAD_INDEX for
 * offsets, lengths or pages out of range, n > max_keep, n > lens[b], a kept row outside
 * [0, lens[b]) or named twice below n (that layer's and head's rows of the
 * sequence are left as they were, its slot_pos too).
 * Asynchronous; capturable. */
kvsel_status kvsel_paged_compact(const kvsel_pages* pages, int32_t num_seqs, const int32_t* table,
                                 int32_t table_width, const int32_t* lens,
                                 const int32_t* keep_idx, int64_t keep_rows,
                                 const int32_t* keep_offsets, int32_t max_keep,
                                 const int32_t* ref, int32_t* slot_pos, void* stream);

/* One step of a pool's bookkeeping: from the num_in sequences (table, lens) to
 * num_out sequences (table_out, new_lens). New sequence b goes on from old
 * sequence parents[b] (-1: from nothing; parents NULL: from sequence b, num_in ==
 * num_out) with its first m = min(lens[parent], new_lens[b]) rows, and gets
 * pages for new_lens[b] rows: rows m and later are the caller's to write. So one
 * call forks, reorders beams, grows for the next token, cuts and frees (a page
 * that no new sequence holds is free). Pages that are whole within the m rows
 * are shared; the page of a started row group (m % page_size > 0) stays with the
 * lowest b that continues it, if no sequence holds it whole, and the others get a
 * copy of its m % page_size rows (every layer, K and V). Pages are handed out
 * lowest number first, in the order of (b, column). The result depends only on
 * the arguments; table_out must not overlap table.
 *   table_out [num_out][table_width] int32, -1 past the pages held; ref
 *   [num_pages] int32: how many new sequences hold each page; free_pages [1] int32
 *   (or NULL): pages left free, negative = pages that were missing (their entries
 *   are -1, NO_PAGES is recorded).
 * workspace: kvsel_pages_update_bytes(pages, num_out) bytes, 16-byte aligned. Rules:
 * INVALID_ARG for negative counts, a workspace that is too small or misaligned,
 * parents NULL with num_in != num_out > 0; UNSUPPORTED for num_out * table_width >=
 * 2^31. Device status: BAD_INDEX for a parent, length or page out of range (such a
 * sequence becomes empty; such a page's entry becomes -1).
 * Asynchronous; capturable. */
kvsel_status kvsel_pages_update(const kvsel_pages* pages, int32_t num_in, const int32_t* table,
                                int32_t table_width, const int32_t* lens, int32_t num_out,
                                const int32_t* parents, const int32_t* new_lens,
                                int32_t* table_out, int32_t* ref, int32_t* free_pages,
                                void* workspace, int64_t workspace_bytes, void* stream);

/* Workspace bytes of kvsel_pages_update, or -1 if a rule is broken. Host only. */
int64_t kvsel_pages_update_bytes(const kvsel_pages* pages, int32_t num_out);

/* Synchronises `stream`, then returns and clears the current device's status
 * word: the first device-side error recorded since the last call, or
 * KVSEL_OK. Returns KVSEL_ERR_CUDA if the synchronisation itself failed. */
kvsel_status kvsel_device_status(void* stream);

/* Upper bound, in nanoseconds, on every spin-wait inside the kernels (default
 * 2e9). A wait that runs out records KVSEL_ERR_TIMEOUT and the kernel skips
 * the dependent work and exits normally. Must be >= 1000. */
kvsel_status kvsel_set_wait_limit_ns(uint64_t ns);

/* Test hook for the bounded waits. what = 1: the next tensor-core scoring
 * launch withholds the row statistics of its first work item, so the other
 * work items of that (layer, sequence, head) wait until the limit and report
 * KVSEL_ERR_TIMEOUT. what = 0 clears it. */
kvsel_status kvsel_debug_inject(int32_t what);

/* Stage timing of kvsel_snapkv with CUDA events recorded on the caller's
 * stream around each stage: [0] scoring kernel(s), [1] selection with the
 * fused K/V gather, [2] unused (0; the gather runs inside stage [1]). kvsel_profile_begin(n) arms it for the next n calls on
 * the current device (n in 1..100000; creates the events); each call records
 * its events without synchronising. kvsel_profile_end() synchronises, writes
 * the summed milliseconds per stage to stage_ms[0..2] and the number of
 * recorded calls to *calls, and disarms. */
kvsel_status kvsel_profile_begin(int32_t max_calls);
kvsel_status kvsel_profile_end(double* stage_ms, int32_t* calls);

/* Frees the internal workspace of every device this process used. Calls
 * still running on the GPU must have finished (the call synchronises each
 * device first). */
void kvsel_release(void);

/* Bytes of the internal workspace (the cudaMalloc'd scratch of every entry
 * point but kvsel_score_static) currently held on the current device; 0
 * before the first call that needs one and after kvsel_release. Host only. */
int64_t kvsel_workspace_bytes(void);

#ifdef __cplusplus
}
#endif

#endif /* KVSEL_H_ */
