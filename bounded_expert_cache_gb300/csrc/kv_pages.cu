// Bookkeeping of the paged key-value cache on the device: fork, reserve with
// copy-on-write, write, free, compact, copy.
//
// The integer work (page counts, lowest free pages, moves) runs in one cluster
// of 8 CTAs (one CTA is slower even for a pool of 260 pages and 36 sequences:
// fork 6.1 against 5.5 us, reserve 11.6 against 10.7, cold): every phase reads a
// consistent state, a cluster barrier separates it from the phase that changes
// that state, and nothing returns to the host, so a decode step that grows its
// sequences stays capturable in a CUDA graph.
// A call first checks its whole list in every CTA of the cluster (the same
// reads, so the same verdict) and then changes either everything or nothing; a
// page copy likewise, in every block. A write judges every token by itself.
//
// Page ids come from prefix sums over ref, never from the order of atomics:
// the lowest free page first, in list order.
//
// What bounds it: the small calls are latency (a few dependent reads and two
// or three cluster barriers); the copies are HBM: a fragmented pool of 3,000
// pages (64 tokens, 2 heads of 128, 10 layers, 48 sequences) is brought together
// in 157 us of a captured graph (a call among others: 178), 973 MB read and
// written at 6.2 TB/s.
#include <cooperative_groups.h>

#include <atomic>
#include <cstddef>

#include "kv.h"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int kCtas = 8, kThreads = 1024;
constexpr int kWarps = kThreads / 32, kAll = kCtas * kThreads, kAllWarps = kCtas * kWarps;
constexpr int kBitmapWords = 65536 / 32;

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

// Threads that share one listed sequence: a power of two, at least a warp.
__device__ __forceinline__ int lanes_per(int n) {
  int t = 32;
  while (t * 2 * n <= kAll) t *= 2;
  return t;
}

// Mark id in the bitmap; false if it is out of range or was marked.
__device__ __forceinline__ bool mark(uint32_t* bits, int id, int S) {
  if (id < 0 || id >= S) return false;
  return !(atomicOr(bits + (id >> 5), 1u << (id & 31)) & (1u << (id & 31)));
}
__device__ __forceinline__ bool held_ok(const Kv& kv, int len) {
  return len >= 0 && pages_of(kv, len) <= kv.W;
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
    fork_kernel(Kv kv, const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n) {
  __shared__ uint32_t bits[kBitmapWords];
  auto cluster = cg::this_cluster();
  const int tid = threadIdx.x, rank = cluster.block_rank();
  for (int i = tid; i < kBitmapWords; i += kThreads) bits[i] = 0u;
  const bool stop = pending(kv);
  __syncthreads();
  bool ok = true;
  for (int i = tid; i < n; i += kThreads) {
    const int s = src[i], d = dst[i];
    ok &= mark(bits, d, kv.S) && kv.lens[d] == 0;
    ok &= s >= 0 && s < kv.S && held_ok(kv, kv.lens[s]);
  }
  ok = __syncthreads_and(ok);
  cluster.sync();  // every CTA has its verdict before anything changes
  if (stop) return;
  if (!ok) {
    if (rank == 0 && tid == 0) atomicOr(&kv.work->err, MOE_DEVERR_BADIDX);
    return;
  }
  const int per = lanes_per(n), g = (rank * kThreads + tid) / per, lane = (rank * kThreads + tid) % per;
  for (int i = g; i < n; i += kAll / per) {
    const int s = src[i], d = dst[i];
    // a source that is also a destination was empty before the call
    const int len = (bits[s >> 5] >> (s & 31)) & 1u ? 0 : kv.lens[s];
    const int np = pages_of(kv, len);
    for (int j = lane; j < np; j += per) {
      const int p = kv.table[static_cast<int64_t>(s) * kv.W + j];
      kv.table[static_cast<int64_t>(d) * kv.W + j] = p;
      if (p >= 0 && p < kv.P)
        atomicAdd(kv.ref + p, 1);
      else
        atomicOr(&kv.work->err, MOE_DEVERR_BADIDX);
    }
    if (lane == 0 && len > 0) kv.lens[d] = len;
  }
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
    free_kernel(Kv kv, const int32_t* __restrict__ seqs, int n) {
  __shared__ uint32_t bits[kBitmapWords];
  auto cluster = cg::this_cluster();
  const int tid = threadIdx.x, rank = cluster.block_rank();
  for (int i = tid; i < kBitmapWords; i += kThreads) bits[i] = 0u;
  const bool stop = pending(kv);
  __syncthreads();
  bool ok = true;
  for (int i = tid; i < n; i += kThreads) {
    const int s = seqs[i];
    ok &= mark(bits, s, kv.S) && held_ok(kv, kv.lens[s]);
  }
  ok = __syncthreads_and(ok);
  cluster.sync();
  if (stop) return;
  if (!ok) {
    if (rank == 0 && tid == 0) atomicOr(&kv.work->err, MOE_DEVERR_BADIDX);
    return;
  }
  const int per = lanes_per(n), g = (rank * kThreads + tid) / per, lane = (rank * kThreads + tid) % per;
  for (int i = g; i < n; i += kAll / per) {
    const int s = seqs[i], np = pages_of(kv, kv.lens[s]);
    for (int j = lane; j < np; j += per) {
      int32_t* e = kv.table + static_cast<int64_t>(s) * kv.W + j;
      const int p = *e;
      if (p >= 0 && p < kv.P)
        atomicSub(kv.ref + p, 1);
      else
        atomicOr(&kv.work->err, MOE_DEVERR_BADIDX);
      *e = -1;
    }
  }
  cluster.sync();  // lengths were read by every thread of their group
  for (int i = rank * kThreads + tid; i < n; i += kAll) kv.lens[seqs[i]] = 0;
}

// Pages of one warp of the cluster: [first, last), whole strips of 32.
struct Strip {
  int first, last;
};
__device__ __forceinline__ Strip strip_of(int P, int w) {
  const int per = ((P + 31) / 32 + kAllWarps - 1) / kAllWarps;  // strips of 32 a warp
  Strip s;
  s.first = min(P, w * per * 32);
  s.last = min(P, (w + 1) * per * 32);
  return s;
}
// Free pages in a warp's strips (every lane gets the count).
__device__ __forceinline__ int count_free(const Kv& kv, Strip s, int lane) {
  int c = 0;
#pragma unroll 8
  for (int p0 = s.first; p0 < s.last; p0 += 32) c += p0 + lane < s.last && kv.ref[p0 + lane] == 0;
  return __reduce_add_sync(~0u, c);
}
// Give every CTA of the cluster every warp's count.
__device__ __forceinline__ void share_counts(cg::cluster_group& cluster, int* counts, int w, int lane, int c) {
  if (lane < kCtas) *cluster.map_shared_rank(counts + w, lane) = c;
  cluster.sync();
}
// Sum of the counts of warps before w, and of all.
__device__ __forceinline__ int2 prefix_of(const int* counts, int w, int lane) {
  int before = 0, all = 0;
  #pragma unroll
  for (int i = lane; i < kAllWarps; i += 32) {
    const int c = counts[i];
    all += c;
    before += i < w ? c : 0;
  }
  return make_int2(__reduce_add_sync(~0u, before), __reduce_add_sync(~0u, all));
}

// Block-wide inclusive scan; the total in 64 bits: 1,024 values of up to 2^26
// pages do not fit in 32 (a warp's 32 do). The scan itself wraps where the total does.
__device__ __forceinline__ uint32_t block_incl(uint32_t v, uint32_t* tmp, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(~0u, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  const uint32_t t = tmp[lane];
  const uint32_t below = __reduce_add_sync(~0u, lane < warp ? t : 0u);
  const uint32_t low = __reduce_add_sync(~0u, t & 0xFFFFu), high = __reduce_add_sync(~0u, t >> 16);
  *total = (static_cast<int64_t>(high) << 16) + low;
  __syncthreads();
  return x + below;
}

// first[i]: requests of the sequences before the i-th; info[i]: its pages
// before the call, times two, plus one if it copies its last page first;
// copies[i]: such sequences before it.
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
    reserve_kernel(Kv kv, const int32_t* __restrict__ seqs, const int32_t* __restrict__ n_new, int n) {
  extern __shared__ int dyn[];
  int* first = dyn;
  int* info = dyn + n + 1;
  int* copies = info + n;
  __shared__ uint32_t bits[kBitmapWords];
  __shared__ int counts[kAllWarps];
  __shared__ uint32_t scan[kWarps];
  auto cluster = cg::this_cluster();
  const int tid = threadIdx.x, rank = cluster.block_rank(), lane = tid & 31;
  const int w = rank * kWarps + (tid >> 5);
  for (int i = tid; i < kBitmapWords; i += kThreads) bits[i] = 0u;
  const bool stop = pending(kv);
  __syncthreads();
  // the list, and the sharers of every partly filled shared last page
  bool ok = true, room = true;
  for (int i = tid; i < n; i += kThreads) {
    const int s = seqs[i], add = n_new[i];
    if (!mark(bits, s, kv.S) || add < 0 || !held_ok(kv, kv.lens[s])) {
      ok = false;
      continue;
    }
    const int len = kv.lens[s];
    if (static_cast<int64_t>(len) + add > static_cast<int64_t>(kv.W) << kv.page_shift) room = false;
    if (add > 0 && (len & (kv.page - 1))) {
      const int p = kv.table[static_cast<int64_t>(s) * kv.W + (len >> kv.page_shift)];
      if (p < 0 || p >= kv.P)
        ok = false;
      else if (i / kThreads % kCtas == rank && kv.ref[p] > 1) {
        atomicAdd(kv.shr + p, 1);
        atomicMax(kv.last + p, i + 1);
      }
    }
  }
  ok = __syncthreads_and(ok);
  room = __syncthreads_and(room);
  const Strip st = strip_of(kv.P, w);
  const int mine = count_free(kv, st, lane);
  share_counts(cluster, counts, w, lane, mine);  // also publishes shr and last
  // requests of every listed sequence
  int64_t wanted = 0;  // pages
  int n_copies = 0;
  if (ok && room && !stop) {
    for (int i0 = 0; i0 < n; i0 += kThreads) {
      const int i = i0 + tid;
      int need = 0, cow = 0;
      if (i < n) {
        const int s = seqs[i], len = kv.lens[s], add = n_new[i];
        const int have = pages_of(kv, len);
        if (add > 0 && (len & (kv.page - 1))) {
          const int p = kv.table[static_cast<int64_t>(s) * kv.W + have - 1];
          const int k = __ldcg(kv.shr + p);
          // every sharer copies; if all of them are listed, the last one stays
          cow = kv.ref[p] > 1 && !(k == kv.ref[p] && __ldcg(kv.last + p) == i + 1);
        }
        need = cow + pages_of(kv, static_cast<int64_t>(len) + add) - have;
        info[i] = have * 2 + cow;
      }
      int64_t t, c;
      const uint32_t incl = block_incl(need, scan, &t);
      // (used only if all is granted: then it is below the pages there are)
      if (i < n) first[i] = static_cast<int>(static_cast<uint32_t>(wanted) + incl - need);
      const uint32_t before = block_incl(cow, scan, &c) - cow;
      if (i < n) copies[i] = n_copies + before;
      n_copies += static_cast<int>(c);
      wanted += t;
    }
    if (tid == 0) first[n] = static_cast<int>(wanted);
  }
  const int2 pre = prefix_of(counts, w, lane);
  if (wanted > pre.y) room = false;
  const int total = room ? static_cast<int>(wanted) : 0;
  __syncthreads();
  const bool go = ok && room && !stop;
  // the lowest free pages, in order
  if (go) {
    int r = pre.x;
    for (int p0 = st.first; p0 < st.last && r < total; p0 += 32) {
      const bool f = p0 + lane < st.last && kv.ref[p0 + lane] == 0;
      const unsigned int b = __ballot_sync(~0u, f);
      const int q = r + __popc(b & ((1u << lane) - 1u));
      if (f && q < total) kv.src[q] = p0 + lane;
      r += __popc(b);
    }
  }
  cluster.sync();
  // the sharer counts go back to zero whatever the verdict
  for (int i = rank * kThreads + tid; i < n; i += kAll) {
    const int s = seqs[i];
    if (s < 0 || s >= kv.S) continue;
    const int len = kv.lens[s];
    if (!held_ok(kv, len) || !(len & (kv.page - 1))) continue;
    const int p = kv.table[static_cast<int64_t>(s) * kv.W + (len >> kv.page_shift)];
    if (p < 0 || p >= kv.P) continue;
    kv.shr[p] = 0;
    kv.last[p] = 0;
  }
  if (!go) {
    if (rank == 0 && tid == 0) {
      kv.work->n_copies = 0;
      if (!stop) atomicOr(&kv.work->err, !ok ? MOE_DEVERR_BADIDX : MOE_DEVERR_CAPACITY);
    }
    return;
  }
  cluster.sync();  // lengths and table rows were read above
  for (int q = rank * kThreads + tid; q < total; q += kAll) {
    int lo = 0, hi = n;  // the sequence i with first[i] <= q < first[i + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= q)
        lo = mid;
      else
        hi = mid;
    }
    const int j = q - first[lo], cow = info[lo] & 1, e = (info[lo] >> 1) + j - cow;
    const int p = kv.src[q];
    int32_t* at = kv.table + static_cast<int64_t>(seqs[lo]) * kv.W + e;
    if (cow && j == 0) {
      atomicSub(kv.ref + *at, 1);
      kv.map[copies[lo]] = *at;
      kv.dst[copies[lo]] = p;
    }
    *at = p;
    kv.ref[p] = 1;
  }
  for (int i = rank * kThreads + tid; i < n; i += kAll) {
    const int s = seqs[i], len = kv.lens[s];
    kv.lens[s] = len + n_new[i];
    if (info[i] & 1) kv.filled[copies[i]] = len & (kv.page - 1);
  }
  if (rank == 0 && tid == 0) kv.work->n_copies = n_copies;
}

// x / d and x % d, in 32 bits where x fits (a 64-bit division takes several hundred cycles)
__device__ __forceinline__ uint32_t take_mod(uint64_t& x, uint32_t d) {
  if (x >> 32) {
    const uint64_t q = x / d;
    const uint32_t r = static_cast<uint32_t>(x - q * d);
    x = q;
    return r;
  }
  const uint32_t y = static_cast<uint32_t>(x), q = y / d;
  x = q;
  return y - q * d;
}

// The copies of reserve: copy i takes the first filled[i] tokens of page map[i]
// to page dst[i], in every layer and head of k and v. A warp copies 128 vectors
// (2 KB) at a time, four loads a lane in flight.
constexpr int kCowPiece = 128;
__global__ void __launch_bounds__(256)
    cow_copy_kernel(Kv kv, uint4* k, uint4* v, int L, int H, int tok_vecs, int64_t page_vecs) {
  const int n = kv.work->n_copies, lane = threadIdx.x & 31;
  const int pieces = (kv.page * tok_vecs + kCowPiece - 1) / kCowPiece;
  const uint64_t items = static_cast<uint64_t>(n) * L * 2 * H * pieces;
  for (uint64_t it = blockIdx.x * 8ull + (threadIdx.x >> 5); it < items; it += gridDim.x * 8ull) {
    uint64_t r = it;
    const int p = take_mod(r, pieces), h = take_mod(r, H);
    uint4* pool = take_mod(r, 2) ? v : k;
    const int l = take_mod(r, L), i = static_cast<int>(r);
    const int vecs = kv.filled[i] * tok_vecs - p * kCowPiece;  // of this piece on
    if (vecs <= 0) continue;
    const int64_t head = static_cast<int64_t>(h) * kv.page * tok_vecs + p * kCowPiece;
    const uint4* from = pool + (static_cast<int64_t>(l) * kv.P + kv.map[i]) * page_vecs + head;
    uint4* to = pool + (static_cast<int64_t>(l) * kv.P + kv.dst[i]) * page_vecs + head;
    uint4 t[kCowPiece / 32];
#pragma unroll
    for (int x = 0; x < kCowPiece / 32; ++x)
      if (lane + 32 * x < vecs) t[x] = from[lane + 32 * x];
#pragma unroll
    for (int x = 0; x < kCowPiece / 32; ++x)
      if (lane + 32 * x < vecs) to[lane + 32 * x] = t[x];
  }
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads) compact_kernel(Kv kv) {
  __shared__ int counts[kAllWarps], below[kAllWarps];
  auto cluster = cg::this_cluster();
  const int tid = threadIdx.x, rank = cluster.block_rank(), lane = tid & 31;
  const int w = rank * kWarps + (tid >> 5);
  const bool stop = pending(kv);
  const Strip st = strip_of(kv.P, w);
  const int free_mine = count_free(kv, st, lane);
  share_counts(cluster, counts, w, lane, free_mine);
  const int2 pre = prefix_of(counts, w, lane);
  const int live = kv.P - pre.y;
  // holes below the new end = pages in use above it
  int c = 0;
#pragma unroll 8
  for (int p0 = st.first; p0 < st.last; p0 += 32) c += p0 + lane < min(st.last, live) && kv.ref[p0 + lane] == 0;
  share_counts(cluster, below, w, lane, __reduce_add_sync(~0u, c));
  const int holes = prefix_of(below, w, lane).y;
  if (stop) {
    if (rank == 0 && tid == 0) {
      kv.work->n_copies = 0;
      kv.work->n_live = kv.P;
    }
    return;
  }
  int f = pre.x;  // free pages before the strip
  for (int p0 = st.first; p0 < st.last; p0 += 32) {
    const int p = p0 + lane;
    const bool in = p < st.last, fr = in && kv.ref[p] == 0;
    const unsigned int b = __ballot_sync(~0u, fr);
    const int before = f + __popc(b & ((1u << lane) - 1u));
    if (fr && p < live) kv.dst[before] = p;
    // pages in use before p, less those below the new end
    if (in && !fr && p >= live) kv.src[p - before - (live - holes)] = p;
    f += __popc(b);
  }
  cluster.sync();
  for (int r = rank * kThreads + tid; r < holes; r += kAll) {
    const int s = kv.src[r], d = kv.dst[r];
    kv.map[s] = d;
    kv.ref[d] = kv.ref[s];
    kv.ref[s] = 0;
  }
  if (rank == 0 && tid == 0) {
    kv.work->n_copies = holes;
    kv.work->n_live = live;
  }
}

// The list of a page copy: all of it is checked before anything is copied, so
// that no block copies while another finds an error. Every block checks a short
// list itself, which saves a launch (one page: 4 us instead of 5.3); a longer one
// is checked once, before the copies' launch.
constexpr int kShortList = 2048;
__device__ __forceinline__ bool copy_ok(const Kv& kv, int s, int d) { return s >= 0 && s < kv.P && d >= 0 && d < kv.P; }
__global__ void __launch_bounds__(kThreads)
    check_pages_kernel(Kv kv, const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n) {
  if (pending(kv)) return;  // (by now perhaps this launch's own error, of which one record is enough)
  bool ok = true;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * kThreads)
    ok &= copy_ok(kv, src[i], dst[i]);
  if (!ok) atomicOr(&kv.work->err, MOE_DEVERR_BADIDX);
}

// Whole pages src[i] -> dst[i] in every layer, pieces of kPiece vectors, and
// (REMAP) the table entries of moved pages.
constexpr int kPiece = 1024;  // 16 KB
template <bool REMAP>
__global__ void __launch_bounds__(256)
    page_copy_kernel(Kv kv, uint4* k, uint4* v, const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n,
                     int L, int64_t page_vecs) {
  if (REMAP) {
    n = kv.work->n_copies;
  } else {
    const bool stop = pending(kv);
    bool ok = true;
    if (n <= kShortList)
      for (int i = threadIdx.x; i < n; i += 256) ok &= copy_ok(kv, src[i], dst[i]);
    ok = __syncthreads_and(ok);
    if (!ok && !stop && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&kv.work->err, MOE_DEVERR_BADIDX);
    if (__syncthreads_or(stop) || !ok) return;  // (of a good list's launch no block sets the word)
  }
  const int pieces = static_cast<int>((page_vecs + kPiece - 1) / kPiece);
  const uint64_t items = static_cast<uint64_t>(n) * L * 2 * pieces;
  for (uint64_t it = blockIdx.x; it < items; it += gridDim.x) {
    uint64_t r = it;
    const int piece = take_mod(r, pieces);
    uint4* pool = take_mod(r, 2) ? v : k;
    const int l = take_mod(r, L), i = static_cast<int>(r);
    const int s = src[i], d = dst[i];
    const uint4* from = pool + (static_cast<int64_t>(l) * kv.P + s) * page_vecs + static_cast<int64_t>(piece) * kPiece;
    uint4* to = pool + (static_cast<int64_t>(l) * kv.P + d) * page_vecs + static_cast<int64_t>(piece) * kPiece;
    const int vecs = static_cast<int>(min(static_cast<int64_t>(kPiece), page_vecs - static_cast<int64_t>(piece) * kPiece));
    uint4 t[kPiece / 256];
#pragma unroll
    for (int x = 0; x < kPiece / 256; ++x)
      if (static_cast<int>(threadIdx.x) + x * 256 < vecs) t[x] = __ldcs(from + threadIdx.x + x * 256);
#pragma unroll
    for (int x = 0; x < kPiece / 256; ++x)
      if (static_cast<int>(threadIdx.x) + x * 256 < vecs) __stcs(to + threadIdx.x + x * 256, t[x]);
  }
  if (REMAP) {
    const int live = kv.work->n_live, lane = threadIdx.x & 31;
    const int warps = gridDim.x * 8;
    for (int s = blockIdx.x * 8 + (threadIdx.x >> 5); s < kv.S; s += warps) {
      const int len = kv.lens[s];
      const int np = held_ok(kv, len) ? pages_of(kv, len) : 0;
      for (int j = lane; j < np; j += 32) {
        int32_t* e = kv.table + static_cast<int64_t>(s) * kv.W + j;
        if (*e >= live && *e < kv.P) *e = kv.map[*e];
      }
    }
  }
}

// One warp per new token: K and V of every head to its place in its page.
__global__ void __launch_bounds__(256)
    write_kernel(Kv kv, uint4* k, uint4* v, const uint4* __restrict__ nk, int64_t ldk, const uint4* __restrict__ nv,
                 int64_t ldv, const int32_t* __restrict__ seqs, const int32_t* __restrict__ cu, int n, int n_rows,
                 int H, int tok_vecs, uint32_t number) {
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= n_rows) return;
  const uint4* fk = nk + row * ldk;
  const uint4* fv = nv + row * ldv;
  const int vecs = H * tok_vecs;
  uint4 k0, v0;  // the row's first pieces, while its place is looked up
  if (lane < vecs) {
    k0 = __ldg(fk + lane);
    v0 = __ldg(fv + lane);
  }
  const bool stop = pending(kv, true, number);
  auto record = [&](uint32_t why) {
    if (lane == 0) atomicOr(reinterpret_cast<unsigned long long*>(&kv.work->late), static_cast<unsigned long long>(number) << 32 | why);
  };
  // the last i with cu[i] <= row: 32 probes a step
  int lo = 0, span = n;  // it is in [lo, lo + span)
  while (span > 1) {
    const int step = (span + 31) / 32, at = lo + lane * step;
    const unsigned int b = __ballot_sync(~0u, at < lo + span && __ldg(cu + at) <= row);
    const int hit = b ? 31 - __clz(b) : 0;
    const int next = lo + hit * step;
    span = min(step, lo + span - next);
    lo = next;
  }
  if (stop) return;
  // tokens that the rows do not reach (of a chunk that no row is in, too)
  if (row == 0 && __ldg(cu + n) > n_rows) record(MOE_DEVERR_BADIDX);
  const int r0 = __ldg(cu + lo), r1 = __ldg(cu + lo + 1);
  if (row < r0 || row >= r1) return;
  if (r0 < 0 || r1 > n_rows) {  // none of such a chunk is written
    record(MOE_DEVERR_BADIDX);
    return;
  }
  const int s = seqs ? __ldg(seqs + lo) : lo;
  if (s < 0 || s >= kv.S) {
    record(MOE_DEVERR_BADIDX);
    return;
  }
  const int len = kv.lens[s], at = len - (r1 - row);
  if (len - (r1 - r0) < 0 || !held_ok(kv, len)) {  // the chunk does not fit: none of it is written
    record(KV_DEVERR_SHARED);
    return;
  }
  const int p = kv.table[static_cast<int64_t>(s) * kv.W + (at >> kv.page_shift)];
  if (p < 0 || p >= kv.P || kv.ref[p] != 1) {
    record(p < 0 || p >= kv.P ? MOE_DEVERR_BADIDX : KV_DEVERR_SHARED);
    return;
  }
  const int64_t base = ((static_cast<int64_t>(p) * H) << kv.page_shift) + (at & (kv.page - 1));
  for (int x = lane; x < vecs; x += 32) {
    const int h = x / tok_vecs, c = x - h * tok_vecs;
    const int64_t to = (base + (static_cast<int64_t>(h) << kv.page_shift)) * tok_vecs + c;
    k[to] = x < 32 ? k0 : __ldg(fk + x);
    v[to] = x < 32 ? v0 : __ldg(fv + x);
  }
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
// 16-byte vectors of one token of one head, and of a page of one layer
int tok_vecs(const moe_kv_t& a) { return a.head_dim * (a.dtype == MOE_F32 ? 4 : 2) / 16; }
int64_t page_vecs(const moe_kv_t& a) { return static_cast<int64_t>(a.n_kv_heads) * a.page_tokens * tok_vecs(a); }

}  // namespace

cudaError_t launch_kv_fork(const moe_kv_t& a, const KvLayout& l, const int32_t* src, const int32_t* dst, int32_t n,
                           cudaStream_t st) {
  fork_kernel<<<kCtas, kThreads, 0, st>>>(kv_of(a, l), src, dst, n);
  return cudaGetLastError();
}

cudaError_t launch_kv_reserve(const moe_kv_t& a, const KvLayout& l, const int32_t* seqs, const int32_t* n_new,
                              int32_t n, int num_sms, cudaStream_t st) {
  const int smem = (3 * n + 1) * 4;
  cudaError_t e = cudaFuncSetAttribute(reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (3 * kMaxList + 1) * 4);
  if (e != cudaSuccess) return e;
  const Kv kv = kv_of(a, l);
  reserve_kernel<<<kCtas, kThreads, smem, st>>>(kv, seqs, n_new, n);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int pieces = (a.page_tokens * tok_vecs(a) + kCowPiece - 1) / kCowPiece;
  const int64_t items = static_cast<int64_t>(n) * a.n_layers * 2 * a.n_kv_heads * pieces;
  const int grid = static_cast<int>(std::min<int64_t>((items + 7) / 8, 8ll * num_sms));
  cow_copy_kernel<<<grid, 256, 0, st>>>(kv, static_cast<uint4*>(a.k), static_cast<uint4*>(a.v), a.n_layers,
                                        a.n_kv_heads, tok_vecs(a), page_vecs(a));
  return cudaGetLastError();
}

cudaError_t launch_kv_write(const moe_kv_t& a, const KvLayout& l, int32_t layer, const void* k_new, int64_t ldk,
                            const void* v_new, int64_t ldv, const int32_t* seqs, const int32_t* cu, int32_t n,
                            int32_t n_rows, cudaStream_t st) {
  const int per = a.dtype == MOE_F32 ? 4 : 8;
  const int64_t off = layer * (static_cast<int64_t>(a.n_pages) * page_vecs(a));
  static std::atomic<uint32_t> number{0};
  write_kernel<<<(n_rows + 7) / 8, 256, 0, st>>>(kv_of(a, l), static_cast<uint4*>(a.k) + off,
                                                  static_cast<uint4*>(a.v) + off, static_cast<const uint4*>(k_new),
                                                  ldk / per, static_cast<const uint4*>(v_new), ldv / per, seqs, cu, n,
                                                  n_rows, a.n_kv_heads, tok_vecs(a), ++number);
  return cudaGetLastError();
}

cudaError_t launch_kv_free(const moe_kv_t& a, const KvLayout& l, const int32_t* seqs, int32_t n, cudaStream_t st) {
  free_kernel<<<kCtas, kThreads, 0, st>>>(kv_of(a, l), seqs, n);
  return cudaGetLastError();
}

cudaError_t launch_kv_compact(const moe_kv_t& a, const KvLayout& l, int num_sms, cudaStream_t st) {
  const Kv kv = kv_of(a, l);
  compact_kernel<<<kCtas, kThreads, 0, st>>>(kv);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  page_copy_kernel<true><<<8 * num_sms, 256, 0, st>>>(kv, static_cast<uint4*>(a.k), static_cast<uint4*>(a.v), kv.src,
                                                      kv.dst, 0, a.n_layers, page_vecs(a));
  return cudaGetLastError();
}

cudaError_t launch_kv_copy_pages(const moe_kv_t& a, const KvLayout& l, const int32_t* src, const int32_t* dst,
                                 int32_t n, int num_sms, cudaStream_t st) {
  const Kv kv = kv_of(a, l);
  if (n > kShortList) {
    check_pages_kernel<<<std::min((n - 1) / kThreads + 1, num_sms), kThreads, 0, st>>>(kv, src, dst, n);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  page_copy_kernel<false><<<8 * num_sms, 256, 0, st>>>(kv, static_cast<uint4*>(a.k), static_cast<uint4*>(a.v), src, dst,
                                                       n, a.n_layers, page_vecs(a));
  return cudaGetLastError();
}

}  // namespace moe
