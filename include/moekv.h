/*
 * moekv.h — the operators a decoder layer needs beside the routed FFN of
 * moecache.h: a paged key-value cache with its page bookkeeping, attention
 * over it (of the newest tokens of many sequences, and of prompt chunks), and
 * a linear layer with 4-bit weights and group scales for the projections.
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
 * The cache's arrays and a call's tensors are on the current device.
 */
#ifndef MOEKV_H
#define MOEKV_H

#include "moecache.h"

#ifdef __cplusplus
extern "C" {
#endif

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
  int32_t head_dim;    /* multiple of 8, 8..256 */
  int32_t dtype;       /* moe_dtype_t of k and v, and of q, out and new tokens */
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
 * [rows][n_heads][head_dim] of the cache's dtype, rows ldq and ldo elements
 * apart and 16-byte aligned. Scores, softmax statistics and sums are fp32;
 * for bf16 the softmax's numerators enter the value product as bf16.
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

#ifdef __cplusplus
}
#endif
#endif /* MOEKV_H */
