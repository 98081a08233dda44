// Device pieces shared by the attention kernels: a call's sequences, the token
// tiles that a range of query tokens sees, small arithmetic helpers.
#pragma once

#include <cuda_bf16.h>

#include "kv.h"

namespace moe {

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&p);
}
// Either half of a bf16 pair is an infinity or a NaN.
__device__ __forceinline__ bool nonfinite2(uint32_t v) {
  return (v & 0x7F80u) == 0x7F80u || (v & 0x7F800000u) == 0x7F800000u;
}

// One sequence's share of the call.
struct Seq {
  int id;    // table row
  int len;   // tokens held
  int m;     // query tokens
  int row0;  // first query row
};

// Query rows of chunk b; 0 (with an error recorded) if cu leaves the rows given.
__device__ __forceinline__ int chunk_rows(const AttnArgs& a, int b) {
  const int r0 = __ldg(a.cu + b), r1 = __ldg(a.cu + b + 1);
  if (r0 < 0 || r1 < r0 || r1 > a.n_rows) {
    atomicOr(a.err, MOE_DEVERR_BADIDX);
    return 0;
  }
  return r1 - r0;
}
// Chunks that do not cover all rows are an error: the host counts on every
// row's work when it decides how partial results meet. One thread of the grid.
__device__ __forceinline__ void check_chunks(const AttnArgs& a) {
  if (__ldg(a.cu) != 0 || __ldg(a.cu + a.n) != a.n_rows) atomicOr(a.err, MOE_DEVERR_BADIDX);
}

__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int b) {
  Seq s;
  s.id = a.seqs ? __ldg(a.seqs + b) : b;
  if (a.cu) {
    s.row0 = __ldg(a.cu + b);
    s.m = chunk_rows(a, b);
  } else {
    s.row0 = b * a.n_q;
    s.m = a.n_q;
  }
  s.len = 0;
  if (s.id < 0 || s.id >= a.max_seqs) {
    atomicOr(a.err, MOE_DEVERR_BADIDX);
    s.id = 0;
  } else {
    s.len = max(0, __ldg(a.lens + s.id));
    if (s.len > static_cast<int64_t>(a.max_pages) << a.page_shift) {
      atomicOr(a.err, MOE_DEVERR_BADIDX);
      s.len = 0;
    }
  }
  return s;
}

// a / b in 32 bits where both fit (a 64-bit division takes several hundred cycles)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// A line of `total` positions cut into n runs that differ by one at most.
struct Runs {
  int64_t n, per, rem;
  __device__ __forceinline__ Runs(int64_t total, int64_t most) : n(min(total, most)), per(quotient(total, n)), rem(total - per * n) {}
  __device__ __forceinline__ int64_t start(int64_t x) const { return x * per + min(x, rem); }
  // the run that holds a position
  __device__ __forceinline__ int64_t of(int64_t at) const {
    const int64_t big = rem * (per + 1);
    return at < big ? quotient(at, per + 1) : rem + quotient(at - big, per);
  }
};

// Token tiles that rows of query tokens [i0, i1) see: the n0 tiles that hold
// the first tokens, then tiles lo .. lo + n - n0 - 1. At least one tile, so
// that every unit is visited and writes its rows.
struct Span {
  int n, n0, lo;
  int low;  // tokens in [sinks, low) are seen by no row
  int end;  // tokens >= end are seen by no row
  __device__ __forceinline__ int tile(int t) const { return t < n0 ? t : lo + t - n0; }
};
template <int KT>
__device__ __forceinline__ Span span_of(const AttnArgs& a, const Seq& s, int i0, int i1) {
  Span r;
  r.end = max(0, s.len - s.m + i1);
  r.low = 0;
  if (a.window > 0) r.low = max(0, s.len - s.m + i0 - a.window + 1);
  r.lo = r.low / KT;
  r.n0 = min(r.lo, (min(a.sinks, r.low) + KT - 1) / KT);
  r.n = max(1, (r.end + KT - 1) / KT - r.lo + r.n0);
  return r;
}

}  // namespace moe
