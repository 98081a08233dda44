// What the kernels of the cache's pages share: the arrays of a cache as they see
// them, pending errors, and the way from a row of new tokens to its page.
#pragma once

#include <cstddef>

#include "kv.h"

namespace moe {
namespace {

struct Kv {
  int32_t* table;
  int32_t* lens;
  int32_t* ref;
  KvWork* work;
  int32_t *src, *dst, *filled, *map, *shr, *last;
  int32_t S, W, P, page, page_shift;
};

__device__ __forceinline__ int pages_of(const Kv& kv, int64_t tokens) {
  return static_cast<int>((tokens + kv.page - 1) >> kv.page_shift);
}
// Is a failure of an earlier call pending? A write records its own errors under
// its number beside the error word, because its other blocks may still have to
// read that: so a write stops for earlier calls' errors and never for its own, and
// what it writes does not depend on timing. The next call moves them to the word.
__device__ __forceinline__ bool pending(const Kv& kv, bool a_write = false, uint32_t number = 0) {
  static_assert(offsetof(KvWork, err) == 0 && offsetof(KvWork, late) == 8, "one load of both");
  uint64_t head, late;  // (32,768 rows: 14 us with one load a warp, 23 with two, all of one line)
  asm volatile("ld.volatile.global.v2.u64 {%0, %1}, [%2];" : "=l"(head), "=l"(late) : "l"(kv.work) : "memory");
  if (late == 0 || (a_write && static_cast<uint32_t>(late >> 32) == number)) return static_cast<uint32_t>(head) != 0u;
  if (threadIdx.x == 0) atomicOr(&kv.work->err, static_cast<uint32_t>(late));
  return true;
}

__device__ __forceinline__ bool held_ok(const Kv& kv, int len) {
  return len >= 0 && pages_of(kv, len) <= kv.W;
}

// A write's own error, beside its number, by one lane.
__device__ __forceinline__ void record_late(const Kv& kv, uint32_t number, uint32_t why, int lane) {
  if (lane == 0)
    atomicOr(reinterpret_cast<unsigned long long*>(&kv.work->late), static_cast<unsigned long long>(number) << 32 | why);
}
// The last i with cu[i] <= row, by a warp: 32 probes a step.
__device__ __forceinline__ int chunk_of(const int32_t* __restrict__ cu, int n, int row, int lane) {
  int lo = 0, span = n;  // it is in [lo, lo + span)
  while (span > 1) {
    const int step = (span + 31) / 32, at = lo + lane * step;
    const unsigned int b = __ballot_sync(~0u, at < lo + span && __ldg(cu + at) <= row);
    const int hit = b ? 31 - __clz(b) : 0;
    const int next = lo + hit * step;
    span = min(step, lo + span - next);
    lo = next;
  }
  return lo;
}
// Where a row of chunks that end with their sequences' newest tokens is held: its
// position, its page (-1: nowhere) and the error that leaves it out, if any.
struct Place {
  int pos, page;
  uint32_t why;
};
// lo: the row's chunk. OWN: its page must be this sequence's alone.
template <bool OWN>
__device__ __forceinline__ Place place_of(const Kv& kv, const int32_t* __restrict__ seqs, const int32_t* __restrict__ cu, int lo,
                                          int n_rows, int row) {
  Place p{0, -1, 0u};
  const int r0 = __ldg(cu + lo), r1 = __ldg(cu + lo + 1);
  if (row < r0 || row >= r1) return p;
  if (r0 < 0 || r1 > n_rows) {  // nothing of such a chunk
    p.why = MOE_DEVERR_BADIDX;
    return p;
  }
  const int s = seqs ? __ldg(seqs + lo) : lo;
  if (s < 0 || s >= kv.S) {
    p.why = MOE_DEVERR_BADIDX;
    return p;
  }
  const int len = kv.lens[s], at = len - (r1 - row);
  if (len - (r1 - r0) < 0 || !held_ok(kv, len)) {  // the chunk does not fit: nothing of it
    p.why = KV_DEVERR_SHARED;
    return p;
  }
  const int page = kv.table[static_cast<int64_t>(s) * kv.W + (at >> kv.page_shift)];
  if (page < 0 || page >= kv.P || (OWN && kv.ref[page] != 1)) {
    p.why = page < 0 || page >= kv.P ? MOE_DEVERR_BADIDX : KV_DEVERR_SHARED;
    return p;
  }
  p.pos = at;
  p.page = page;
  return p;
}

Kv kv_of(const moe_kv_t& a, const KvLayout& l) {
  Kv kv;
  char* w = static_cast<char*>(a.work);
  kv.table = a.table;
  kv.lens = a.lens;
  kv.ref = a.ref;
  kv.work = reinterpret_cast<KvWork*>(w);
  kv.src = reinterpret_cast<int32_t*>(w + l.src);
  kv.dst = reinterpret_cast<int32_t*>(w + l.dst);
  kv.filled = reinterpret_cast<int32_t*>(w + l.filled);
  kv.map = reinterpret_cast<int32_t*>(w + l.map);
  kv.shr = reinterpret_cast<int32_t*>(w + l.shr);
  kv.last = reinterpret_cast<int32_t*>(w + l.last);
  kv.S = a.max_seqs;
  kv.W = a.max_pages;
  kv.P = a.n_pages;
  kv.page = a.page_tokens;
  kv.page_shift = __builtin_ctz(a.page_tokens);
  return kv;
}

}  // namespace
}  // namespace moe
