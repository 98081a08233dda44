/*
 * moekv.h — the operators a decoder layer needs beside the routed FFN of
 * moecache.h: a paged key-value cache with its page bookkeeping, in values or in
 * 4-bit codes, attention over it (of the newest tokens of many sequences, and of
 * prompt chunks), rotary positions, a linear layer with 4-bit weights and group
 * scales for the projections, and the draw of the next token from its logits.
 *
 * Conventions are those of moecache.h: every call returns moe_status_t and
 * nothing throws across the ABI; moe_last_error(NULL) describes the last
 * failing call of this thread; device pointers are borrowed; calls are
 * stream-ordered and do not synchronise unless stated, so a decode step can
 * be captured in a CUDA graph.
 *
 * The cache is bounded, like the expert slots: n_pages pages of page_tokens
 * tokens each, shared by every sequence and laid out
 *   k, v: [n_layers][n_pages][n_kv_heads][page_tokens][head_dim],
 * so that the tokens of one head in one page are one contiguous block. A
 * sequence s holds ceil(lens[s] / page_tokens) pages, named in order by the
 * leading entries of table[s]; its other entries are -1. ref[p] counts the
 * table entries that name page p; 0 means free. One table serves all layers.
 * Only these calls change table, lens and ref of a cache in use: a length that
 * the caller lowers leaves pages behind that the next reserve does not return.
 *
 * With MOE_KV_I4 in dtype the pages hold 4-bit codes, 0.5625 bytes a value, for
 * queries, results and new tokens of the other part of dtype: each head of a page
 * is an affine INT4 matrix [page_tokens][head_dim] in groups of 64 along the head,
 * in the split-plane layout of one expert matrix (MOE_I4_G64 of moecache.h): the
 * codes, then the bf16 pairs (s, b). k and v are then bytes,
 * [n_layers][n_pages][n_kv_heads][page_tokens * head_dim * 9 / 16], and a value is
 * s*q + b. Storing a group takes b = its least value and s = (its largest - b) times
 * fp32's 1/15, both rounded to bf16, and q = (x - b) / s rounded to the nearest integer,
 * ties to even, within 0..15 (0 where s is 0), in fp32. A group with an infinity, a NaN
 * or a magnitude above 2^126 becomes NaN as a whole.
 *
 * The cache's arrays and a call's tensors are on the current device.
 */
#ifndef MOEKV_H
#define MOEKV_H

#include "moecache.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Added to a cache's dtype: pages of 4-bit codes. */
enum { MOE_KV_I4 = 16 };

/* Device arrays of a cache, owned by the caller. */
typedef struct {
  void* k;             /* [n_layers][n_pages][n_kv_heads][page_tokens][head_dim] */
  void* v;             /* the same */
  int32_t* table;      /* [max_seqs][max_pages] page of the sequence's i-th page, or -1 */
  int32_t* lens;       /* [max_seqs] tokens held */
  int32_t* ref;        /* [n_pages] table entries naming the page (0: free) */
  void* work;          /* scratch of moe_kv_work_bytes bytes, zeroed once by the caller */
  int64_t work_bytes;
  int32_t n_layers;
  int32_t n_pages;
  int32_t n_kv_heads;
  int32_t page_tokens; /* 16, 32, 64, 128 or 256 */
  int32_t head_dim;    /* multiple of 8, 8..256; with MOE_KV_I4 of 64 */
  int32_t dtype;       /* moe_dtype_t of k and v, and of q, out and new tokens; or that | MOE_KV_I4 */
  int32_t max_seqs;    /* 1..65536 */
  int32_t max_pages;   /* most pages of one sequence; max_pages * page_tokens <= 2^30 */
} moe_kv_t;

/* Scratch bytes of a cache of this geometry on the current device (the
 * pointers of *kv are not read). The scratch holds the cache's error word,
 * page lists and the partial results of split attention; it must be zero
 * before the first call. Calls on one cache must not overlap on the GPU. */
moe_status_t moe_kv_work_bytes(const moe_kv_t* kv, int64_t* bytes);

/* Synchronise stream, report failures that kernels recorded on this cache
 * since the last check, and clear them. MOE_ERR_CAPACITY: a reserve found too
 * few free pages or too narrow a table. MOE_ERR_ARG: a sequence or page id
 * out of range or listed twice, or a fork into a sequence that holds tokens.
 * MOE_ERR_STATE: a write to a page that other sequences share, or past the
 * sequence's length. MOE_ERR_TIMEOUT: a bounded device wait ran out.
 * While a failure is pending, the calls that change the cache (fork,
 * reserve, write, free, compact, copy_pages) do nothing. (A captured write that
 * failed and is replayed with no other call on the cache between does again
 * what it did.) */
moe_status_t moe_kv_check_errors(const moe_kv_t* kv, moe_stream_t stream);

/* dst[i] becomes a sequence with src[i]'s tokens, sharing its pages (their
 * ref grows by one). src, dst: device int32 [n]. Every dst must be empty and
 * listed once; one src may be listed often. Sources are read as they were
 * before the call. All or nothing. */
moe_status_t moe_kv_fork(const moe_kv_t* kv, const int32_t* src, const int32_t* dst, int32_t n,
                         moe_stream_t stream);

/* Make room for n_new[i] more tokens at the end of sequence seqs[i] (device
 * int32 [n], each sequence once, n_new >= 0) and add them to its length;
 * moe_kv_write then fills them in, layer by layer. The pages needed are the
 * lowest free ones, handed out in list order. If the sequence's last page is
 * partly filled and other sequences share it, the sequence first gets a page
 * of its own with a copy of the filled tokens of every layer (of sharers
 * listed together, the last one that no unlisted sequence shares with keeps
 * the old page). All or nothing. */
moe_status_t moe_kv_reserve(const moe_kv_t* kv, const int32_t* seqs, const int32_t* n_new, int32_t n,
                            moe_stream_t stream);

/* Store the newest tokens of n sequences in one layer: sequence seqs[i] gets
 * rows cu[i] .. cu[i+1]-1 of k_new and v_new as its last cu[i+1]-cu[i] tokens.
 * k_new, v_new: device [n_rows][n_kv_heads][head_dim] of the cache's dtype,
 * rows ldk and ldv elements apart (a slice of a fused projection), rows
 * 16-byte aligned; cu: device int32 [n+1]; rows outside cu[0] .. cu[n]-1 belong
 * to no sequence and are ignored. A chunk longer than its sequence or not wholly
 * within the n_rows rows and a token whose page is shared are not written (an
 * error is recorded); the others of the call are. Without rows cu is not read. */
moe_status_t moe_kv_write(const moe_kv_t* kv, int32_t layer, const void* k_new, int64_t ldk, const void* v_new,
                          int64_t ldv, const int32_t* seqs, const int32_t* cu, int32_t n, int32_t n_rows,
                          moe_stream_t stream);

/* Rotary positions. The leading dim columns of a head are pairs, (x[i], x[i + dim/2])
 * or with interleaved = 1 (x[2i], x[2i+1]), and a pair (a, b) of a token at position
 * p becomes magnitude * (a cos t - b sin t, b cos t + a sin t), t = p * angles[i]. The
 * columns from dim on stay. turns: device, [dim / 2], the angles in turns a position
 * modulo 1, times 2^64 (moe_rotary_turns), so that far positions lose nothing. */
typedef struct {
  const uint64_t* turns;
  int32_t dim;         /* even, 2..head size */
  int32_t interleaved; /* 0: halves, 1: neighbours */
  double magnitude;    /* 1 for a plain rotation */
} moe_rotary_t;

/* Angles a position, in radians: angles[i] = base^(-2i/dim) (host, [dim / 2]), for
 * long contexts divided by factor: all of them with context = 0; else those that
 * make at most turns_low turns within `context` tokens, while those of at least
 * turns_high turns stay and the ones between are interpolated linearly in their
 * turns. (A rule that interpolates in the frequency's index gives other angles between
 * the two: hand those to moe_rotary_turns.)
 * moe_rotary_turns: angles (host, any finite ones) as fractions of a turn times
 * 2^64 (host, [n]). Host only, no CUDA call. */
moe_status_t moe_rotary_angles(int32_t dim, double base, double factor, int32_t context, double turns_low,
                               double turns_high, double* angles);
moe_status_t moe_rotary_turns(const double* angles, int32_t n, uint64_t* turns);

/* y = x turned to pos (device int32 [n_rows], any value): x and y device
 * [n_rows][n_heads][head_dim] (xt MOE_F32 or MOE_BF16), rows ldx and ldy elements
 * apart and 16-byte aligned; head_dim a multiple of 8, 8..256. Arithmetic is fp32,
 * rounded once. y may be x (with ldy = ldx), and must not overlap it otherwise. */
moe_status_t moe_rotary(const moe_rotary_t* rot, const int32_t* pos, const void* x, int32_t xt, int64_t ldx,
                        int32_t n_rows, int32_t n_heads, int32_t head_dim, void* y, int64_t ldy, moe_stream_t stream);

/* moe_kv_write with the rotation on the way: row r of a chunk is turned to its
 * position in its sequence, k_new into the pages (from fp32 if they hold codes) and
 * q [n_rows][n_heads][head_dim] into q_out, which may be q (with ldqo = ldq) and
 * must not overlap q, k_new or v_new otherwise. v_new is stored as it is. Rows that
 * moe_kv_write would ignore or leave out are left as they are in q_out. Each sequence
 * is listed once (else a token may hold codes of one row and a scale of another). */
moe_status_t moe_kv_write_rotary(const moe_kv_t* kv, int32_t layer, const moe_rotary_t* rot, const void* q, int64_t ldq,
                                 int32_t n_heads, void* q_out, int64_t ldqo, const void* k_new, int64_t ldk,
                                 const void* v_new, int64_t ldv, const int32_t* seqs, const int32_t* cu, int32_t n,
                                 int32_t n_rows, moe_stream_t stream);

/* The newest tokens of n sequences out of their pages, shared ones too: rows cu[i] ..
 * cu[i+1]-1 of k and v (as k_new and v_new of moe_kv_write) become the last
 * cu[i+1]-cu[i] tokens of seqs[i]. Rows outside of cu[0] .. cu[n]-1 are left as they
 * are, and so, with an error recorded, are those of a chunk that moe_kv_write would
 * not store. */
moe_status_t moe_kv_read(const moe_kv_t* kv, int32_t layer, void* k, int64_t ldk, void* v, int64_t ldv,
                         const int32_t* seqs, const int32_t* cu, int32_t n, int32_t n_rows, moe_stream_t stream);

/* Drop n sequences (device int32 [n], each once): their pages lose one
 * reference, their table rows become -1 and their lengths 0. The bytes of
 * freed pages are left as they are. All or nothing. */
moe_status_t moe_kv_free(const moe_kv_t* kv, const int32_t* seqs, int32_t n, moe_stream_t stream);

/* Bring the pages in use together: of the N pages in use, those with ids
 * >= N move, in ascending order, to the free pages with ids < N, also
 * ascending, in every layer; table and ref follow. */
moe_status_t moe_kv_compact(const moe_kv_t* kv, moe_stream_t stream);

/* Copy whole pages src[i] -> dst[i] in every layer (device int32 [n]; no dst
 * may be listed twice or be a src). Table and ref are the caller's business.
 * With a page id out of range nothing is copied. */
moe_status_t moe_kv_copy_pages(const moe_kv_t* kv, const int32_t* src, const int32_t* dst, int32_t n,
                               moe_stream_t stream);

/* Attention over the cache. Query row (i, h), head h of n_heads, is the query
 * of a token at position p of its sequence. It sees the sequence's tokens
 * j <= p; with window > 0 only those with p - j < window or j < sinks:
 *   out[i, h] = sum_j softmax_j(scale * q[i, h] . k_j) v_j,
 * with the keys and values of cache head h / (n_heads / n_kv_heads). A row
 * whose position is negative sees nothing and is 0. What a row does not see
 * does not reach it, infinities and NaN included. q and out: device
 * [rows][n_heads][head_dim] of the cache's dtype (without MOE_KV_I4), rows ldq and
 * ldo elements apart and 16-byte aligned. Scores, softmax statistics and sums are
 * fp32; for bf16 the softmax's numerators enter the value product as bf16. Over pages
 * of codes bf16 calls multiply f16 over powers of two. Of two that go by one power the
 * smaller loses bits when the other is 2^24 times as large, and counts as 0 when it is
 * 2^34 times as large. One power have
 *   a query's values;
 *   prompt chunks of heads of 64 and 128: the keys of 128 tokens and a cache head, the
 *     values that the rows of a chunk see, and a row's weights (of the softmax);
 *   decode, and chunks of larger heads: a row's weights times the groups' scales that
 *     the sequence's rows see (the groups' offsets are summed in fp32). Scores are held
 *     up to 2^14 times as large as they are: keys from 2^100 on may overflow.
 * (f32 calls have fp32's range.)
 *
 * moe_attn_decode: the newest n_q (1..8) tokens of each of n sequences; rows
 * i*n_q .. i*n_q+n_q-1 belong to seqs[i] (device int32 [n], n <= 65536), at
 * positions lens-n_q .. lens-1. The work is split over the cache's length and
 * joined, so a few long sequences use the whole GPU.
 *
 * moe_attn_prefill: chunks of any length; rows cu[i] .. cu[i+1]-1 (device
 * int32 [n+1], cu[0] = 0, cu[n] = n_rows; anything else is recorded as an
 * error, or refused where n is 0) are the newest tokens of seqs[i]. Rows that have
 * no sequence can be given to an empty one, and are 0. Without rows cu is not read.
 *
 * scale must be positive. seqs may be NULL: sequences 0 .. n-1. n_heads must
 * be a multiple of n_kv_heads, at most 64 times as many. */
moe_status_t moe_attn_decode(const moe_kv_t* kv, int32_t layer, const void* q, int64_t ldq, const int32_t* seqs,
                             int32_t n, int32_t n_q, int32_t n_heads, float scale, int32_t window, int32_t sinks,
                             void* out, int64_t ldo, moe_stream_t stream);
moe_status_t moe_attn_prefill(const moe_kv_t* kv, int32_t layer, const void* q, int64_t ldq, const int32_t* seqs,
                              const int32_t* cu, int32_t n, int32_t n_rows, int32_t n_heads, float scale,
                              int32_t window, int32_t sinks, void* out, int64_t ldo, moe_stream_t stream);

/* Test hook of the attention kernels' bounded waits: the next moe_attn_decode
 * or moe_attn_prefill of this thread (one launch; the hook then clears itself)
 * limits its waits to wait_cycles SM clock cycles (0: the default, about 2 s),
 * and every CTA stops copying after `copies` tiles of K and V (-1: off), so that
 * the wait for a next one runs out. The kernel then drains what it did issue and
 * ends, moe_kv_check_errors reports MOE_ERR_TIMEOUT, and the cache stays usable.
 * No wait is removed and nothing faults. */
moe_status_t moe_debug_attn_wait_timeout(int64_t wait_cycles, int32_t copies);

/* y[t, n] = sum_k W[n, k] x[t, k] (+ bias[n]) for a 4-bit matrix W [N, K] in
 * the split-plane layout of one expert matrix: quant MOE_Q4_0 (K a multiple of
 * 32) or MOE_I4_G64 (K a multiple of 64), K below 2^25 and N below 2^31 - 512.
 * w: device, N*K/2 quant bytes followed by N*K/16 scale bytes; x: device [T, K],
 * rows ldx elements apart (xt MOE_F32 or MOE_BF16); y: device [T, N], rows ldy
 * apart (yt likewise); bias: device fp32 [N] or NULL. w and x rows 16-byte
 * aligned. Products are exact and sums those of the matrix units in fp32 for both
 * types of x, codes times x over a group and then its scale; where an affine
 * group's codes and offset nearly cancel, the error is that of the parts. An
 * output that is not finite is formed again weight by weight, so infinities and
 * NaN in x give what weight times x gives, and only the outputs' own sums overflow.
 * Meant for few tokens; T is not bounded, T = 0 does nothing. */
moe_status_t moe_quant_linear(const void* w, int32_t quant, int32_t N, int32_t K, const void* x, int32_t xt,
                              int64_t ldx, int32_t T, const float* bias, void* y, int32_t yt, int64_t ldy,
                              moe_stream_t stream);

/* How moe_sample draws: one value for all rows, or device arrays [rows] (NULL: the
 * value). Of a row's tokens in the order of falling logits, ties by index, a prefix
 * is kept:
 *   temperature T: token i weighs exp((z_i - max z) / T). 0, less or NaN: the first
 *     token of the order is the row's.
 *   top_k: the first k tokens; off if 0 or less, or the number of tokens or more.
 *   top_p: of those the shortest prefix with at least top_p of their weight; at least
 *     one token; off if 1 or more (or NaN).
 *   min_p: of those the ones that weigh at least min_p times the first; off if 0 or
 *     less, 1 if more. */
typedef struct {
  float temperature, top_p, min_p;
  int32_t top_k;
  const float* temperatures;
  const float* top_ps;
  const float* min_ps;
  const int32_t* top_ks;
} moe_sampling_t;

/* Draw one token of each row: the first, by index, up to which the kept weights
 * exceed u[row] times their sum. logits: device [rows][V] (zt MOE_F32 or MOE_BF16),
 * rows ld elements apart (0: one row for all), aligned to their type; 1 <= V <= 2^20.
 * u: device [rows], in [0, 1). token: device int32 [rows]; prob: device [rows], the token's share of the
 * kept weight, or NULL. A NaN counts as -inf. Infinite logits share all the weight. A
 * row without a logit above -inf gets token -1 and probability 0. Weights are formed
 * to about 2^-31 of themselves, down to 2^-43 of the first, and added without
 * rounding, so a result does not depend on how the work is split. */
moe_status_t moe_sample(const void* logits, int32_t zt, int64_t ld, int32_t rows, int32_t V, const float* u,
                        const moe_sampling_t* by, int32_t* token, float* prob, moe_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOEKV_H */
