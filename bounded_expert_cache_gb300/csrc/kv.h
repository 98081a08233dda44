// Declarations shared by the KV-cache, attention and 4-bit linear units.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/moekv.h"
#include "internal.h"

namespace moe {

// Additional error bits of a cache's error word (beside MOE_DEVERR_*).
enum : uint32_t {
  KV_DEVERR_SHARED = 32u,  // write to a shared page or past the length
};

// Head of a cache's scratch, before its page lists and partial results.
struct KvWork {
  uint32_t err;       // error word
  int32_t n_copies;   // page copies planned by reserve or compact
  uint64_t late;      // errors of a write (low half) and that write's number
  int32_t n_live;     // pages in use, of the last compact
  int32_t pad[59];
};
constexpr int kPartRows = 64;        // most rows of one partial result (decode)
constexpr int kPrefillTickets = 8;   // tickets a CTA (prefill)
constexpr int kPrefillPartRows = 256;
constexpr int kTcHeadDim = 128;      // largest head size of the tensor-core prefill

struct KvLayout {
  // byte offsets into the scratch: page lists (src, dst, map, shr, last: one
  // int per page; filled: one per listed sequence), tickets, records of cut units, partial results
  int64_t src, dst, filled, map, shr, last, tickets, cuts, part, bytes;
};
constexpr int kMaxList = 8192;  // most sequences of one page call
KvLayout kv_layout(const moe_kv_t& kv, int num_sms);

// A unit that several CTAs of an attention launch hold parts of, recorded by
// the first of them: the parts are in CTAs c .. c + count - 1.
struct Cut {
  int32_t count, rt, h, row0, m, len;
};

struct AttnArgs {
  const void* q;
  void* out;
  const void* k;  // layer base
  const void* v;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* seqs;  // or nullptr: 0 .. n-1
  const int32_t* cu;    // or nullptr: n_q rows a sequence
  int64_t ldq, ldo;     // elements
  int32_t n, n_q, n_rows, Hq, Hkv, g, D;
  int32_t page_shift, max_pages, max_seqs, n_pages;
  float scale_log2;     // scale * log2(e)
  int32_t window, sinks;
  float* part;          // partial results
  unsigned int* tickets;  // prefill: arrivals at a cut unit, zero between launches
  Cut* cuts;              // [CTAs]
  uint32_t* err;
  int32_t row_tiles;    // row tiles a sequence and cache head (decode)
  bool wide_out;        // rows of out are multiples of 32 bytes, 32-byte aligned
  int64_t wait_cycles;  // limit of a wait on a barrier
  uint32_t copies;      // test hook: K and V tiles that a CTA copies before it stops; ~0: all
};
cudaError_t launch_attn_decode(const AttnArgs& a, int32_t dtype, int num_sms, cudaStream_t st);
cudaError_t launch_attn_prefill(const AttnArgs& a, int32_t dtype, int32_t n_rows, int num_sms, cudaStream_t st);

cudaError_t launch_attn_prefill_tc(const AttnArgs& a, int num_sms, cudaStream_t st);

cudaError_t launch_kv_fork(const moe_kv_t& kv, const KvLayout& l, const int32_t* src, const int32_t* dst, int32_t n,
                           cudaStream_t st);
cudaError_t launch_kv_reserve(const moe_kv_t& kv, const KvLayout& l, const int32_t* seqs, const int32_t* n_new,
                              int32_t n, int num_sms, cudaStream_t st);
cudaError_t launch_kv_write(const moe_kv_t& kv, const KvLayout& l, int32_t layer, const void* k_new, int64_t ldk,
                            const void* v_new, int64_t ldv, const int32_t* seqs, const int32_t* cu, int32_t n,
                            int32_t n_rows, cudaStream_t st);
cudaError_t launch_kv_free(const moe_kv_t& kv, const KvLayout& l, const int32_t* seqs, int32_t n, cudaStream_t st);
cudaError_t launch_kv_compact(const moe_kv_t& kv, const KvLayout& l, int num_sms, cudaStream_t st);
cudaError_t launch_kv_copy_pages(const moe_kv_t& kv, const KvLayout& l, const int32_t* src, const int32_t* dst,
                                 int32_t n, int num_sms, cudaStream_t st);

struct LinearArgs {
  const uint8_t* w;
  const uint8_t* meta;  // scale plane
  const void* x;
  const float* bias;
  void* y;
  int64_t ldx, ldy;
  int32_t N, K, T, xt, yt;
};
cudaError_t launch_quant_linear(const LinearArgs& a, int32_t quant, int num_sms, cudaStream_t st);

}  // namespace moe
