// The next token of each row of logits: temperature, top-k, top-p and min-p, drawn
// with a given random number.
//
// With M the row's largest logit, token i weighs w_i = 2^-d_i, d_i = (M - z_i) log2(e) / T.
// In the order of falling logits, ties by index, what is kept is a prefix: the first
// k; of these the shortest with top_p of their weight; of these those with w >= min_p.
// The token is the first, by index, up to which the kept weights exceed u times
// their sum.
//
// Which token u falls on is decided by sums over the whole vocabulary, so they must
// not depend on the order of adding, nor be off by what fp32 sums are. Weights are
// whole numbers of 2^-43: sums of them in 64 bits are exact in any order. A weight's
// own error is about 2^-31 of it: d is formed as a pair of fp32 (2^-34), cut into a
// whole n, a multiple a of 2^-8 and a rest r, and 2^-d = 2^-n 2^-a (1 + (2^-r - 1))
// takes 2^-a from a table and the rest from its power series.
//
// One cluster of CTAs a row. Each holds a slice of the row in shared memory, so the
// logits are read once. With neither top-k nor top-p two passes follow: the weights'
// sums of every warp's tokens, and the one warp's in which the token is. Else the end of
// the prefix is looked for first:
// - With top-k, bins of d, 1,024 of them, bound it by the threads' own largest logits:
//   the k-th largest of them is no larger than the k-th of all. If that leaves few
//   tokens, as it mostly does, they go to the first CTA, and the others are done. Of a
//   few hundred that CTA counts each one's place among them, and needs no search.
// - Histograms (tokens, weight) follow, over the bins and then, within the bin that
//   holds the end, over the place in the order, (logit, index) as one number, ten bits a
//   round, until the end is decided: mostly one round. The first CTA does that by
//   itself, if the bin's tokens, or all before its end, fit into its list. (Top-p's
//   share is of the first histogram's total. A pass for the total alone, after which
//   most tokens can be left out of the histogram, cost more: 64 rows 95 us, not 75.)
//
// What bounds it: few rows the latency of the passes and cluster barriers; many that a CTA
// loads, finds the maximum, forms weights and looks for the token in turn, with cluster
// barriers between, and two CTAs on an SM hardly hide that for each other (64 rows with
// neither cut: half the issue slots used, HBM a tenth; the weights' arithmetic alone, some 40
// instructions a token, would take 8 to 9 us), in 1.7 waves of clusters, so two. Top-p adds
// three atomics in shared memory for every token with weight. 131,072 fp32 logits: a row with
// top-k 50 and top-p 12.6 us in a captured graph, with top-p alone 28; 64 such rows 37 us
// with neither, 35 with top-k 50, 62 with settings of all kinds, with top-p alone 72 to 100,
// by how many tokens share a bin. Their reading takes 5.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <cmath>

#include "kv.h"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int kSampleThreads = 512, kSampleWarps = kSampleThreads / 32;
constexpr int kBins = 1024, kMostCtas = 16, kList = 2048, kFew = 256;
constexpr int kFraction = 43;  // weights are whole numbers of 2^-43
constexpr float kReach = 44.f;  // weights from here on are none
constexpr float kBinsPer = kBins / kReach;
constexpr int kIndexBits = 20;

// 2^-(i - 128) / 256 times 2^31
struct PowerTable {
  uint32_t p[257];
};
struct Power {  // the same, and as fp32
  uint32_t whole;
  float rounded;
};

struct alignas(16) Hist {
  uint32_t count[kBins];
  unsigned long long weight[kBins];
};
// What a search round starts from, or its result.
struct Search {
  int bin;               // the end's bin of d
  int shift;             // of the round's digits
  unsigned long long lo, hi;  // the end's place is in [lo, hi]
  unsigned long long before, bin_before;  // weight of the tokens before lo, and before the bin
  unsigned int n_before, bin_n;           // and their number
  int done;              // 1: the end is decided: bin and hi; 2: there is none, all are kept
  unsigned long long sum;     // then: the weight kept
  unsigned int kept;          // and the number; before: of tokens up to and with the bin
};
struct SampleShared {
  Hist first, next;
  alignas(16) uint32_t maxima[kBins];
  alignas(16) unsigned long long list[kList];
  unsigned long long chunk[kMostCtas * kSampleWarps];
  unsigned long long sum[kMostCtas];
  unsigned long long warp64[kSampleWarps];
  unsigned int warp32[kSampleWarps];
  unsigned long long found64;
  uint32_t top[kMostCtas];
  int found;
  unsigned int listed[4], index;  // tokens listed by each gathering: this CTA's, then the first one's all
  unsigned int lists_of[4][kMostCtas];
  Search search;
  float c_hi, c_lo;
  Power power[257];
};

__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t u = __float_as_uint(z);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }
// place in the order: falling logits, ties by index
__device__ __forceinline__ unsigned long long place(float z, int i) {
  return static_cast<unsigned long long>(~order_key(z + 0.f)) << kIndexBits | static_cast<unsigned int>(i);  // (-0 is 0)
}
__device__ __forceinline__ float logit_of(unsigned long long place) { return of_key(~static_cast<uint32_t>(place >> kIndexBits)); }

// Differences of logits are halved, which loses nothing and does not overflow; c is 2 log2(e) / T.
struct Row {
  float top, half, c_hi, c_lo;
  const Power* power;
  // bin of d; kBins: no weight. Does not fall as z falls.
  __device__ __forceinline__ int bin(float z) const {
    if (z == top) return 0;
    const float d = fmaf(z, -0.5f, half) * c_hi;
    return d < kReach ? min(static_cast<int>(d * kBinsPer), kBins - 1) : kBins;
  }
  // weight of a token
  __device__ __forceinline__ unsigned long long weight(float z) const {
    if (z == top) return 1ull << kFraction;
    // (top - z) / 2, and the rest of its rounding
    const float y = 0.5f * z, d0 = half - y, yy = half - d0, rest = (half - (d0 + yy)) + (yy - y);
    const float p = d0 * c_hi;
    if (!(p < kReach)) return 0ull;
    const float e = fmaf(d0, c_hi, -p) + (d0 * c_lo + rest * c_hi);
    constexpr float kWhole = 12582912.f;        // 1.5 * 2^23: adding it rounds to a whole number
    constexpr float kPart = 49152.f;            // 1.5 * 2^15: to a multiple of 2^-8
    const float n = p + kWhole, f = p - (n - kWhole);
    const float a = f + kPart, r = (f - (a - kPart)) + e;
    const Power t = power[__float_as_int(a) - 0x47400000 + 128];  // (0x47400000: kPart)
    constexpr float kLn2 = 0.693147181f;
    const float x = r * -kLn2;  // 2^-r = e^x, |x| < 2^-9
    const float q = x * fmaf(x, fmaf(x, 1.f / 6.f, 0.5f), 1.f);
    const float add = t.rounded * q + kWhole;  // below 2^22
    const uint32_t w = t.whole + (__float_as_uint(add) - 0x4B400000u);
    const int by = __float_as_int(n) - 0x4B400000;
    return (static_cast<unsigned long long>(w) << (kFraction - 31)) >> by;
  }
};

// Adds to 64 bits in shared memory by 32-bit atomics, which are native there; the sum
// of several is whole when all are done.
__device__ __forceinline__ void add_shared(unsigned long long* at, unsigned long long w) {
  uint32_t* half = reinterpret_cast<uint32_t*>(at);
  const uint32_t low = static_cast<uint32_t>(w), old = atomicAdd(half, low);
  const uint32_t high = static_cast<uint32_t>(w >> 32) + (old + low < old);
  if (high) atomicAdd(half + 1, high);
}
__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int x = 16; x; x >>= 1) v += __shfl_xor_sync(~0u, v, x);
  return v;
}
// inclusive over the block's threads, in order
template <class T>
__device__ __forceinline__ T block_scan_incl(T v, T* tmp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T y = __shfl_up_sync(~0u, v, d);
    if (lane >= d) v += y;
  }
  if (lane == 31) tmp[warp] = v;
  __syncthreads();
  T below = lane < warp ? tmp[lane & (kSampleWarps - 1)] : static_cast<T>(0);
#pragma unroll
  for (int d = kSampleWarps / 2; d; d >>= 1) below += __shfl_xor_sync(~0u, below, d);
  __syncthreads();
  return v + __shfl_sync(~0u, below, 0);
}

struct SampleArgs {
  const void* z;
  int64_t ld;
  int V;
  const float* u;
  moe_sampling_t by;
  int32_t* token;
  float* prob;
  int slice;   // tokens a CTA, a multiple of 512
  int staged;  // of them in shared memory
};

// (NaN stays, and is none of the largest, of the bins or of the weights)
template <class T>
__device__ __forceinline__ T raw_logit(const SampleArgs& a, int row, int i) {
  return __ldg(static_cast<const T*>(a.z) + row * a.ld + i);
}

// u times s, rounded down; u in [0, 1)
__device__ __forceinline__ unsigned long long share_of(float u, unsigned long long s, bool up) {
  const unsigned long long f = u <= 0.f ? 0ull : static_cast<unsigned long long>(static_cast<double>(u) * 18446744073709551616.0);
  return __umul64hi(f, s) + (up && f * s != 0ull);
}

template <class T>
__global__ void __launch_bounds__(kSampleThreads, 2)
    sample_kernel(const __grid_constant__ SampleArgs a, const __grid_constant__ PowerTable table) {
  extern __shared__ __align__(16) unsigned char sm_raw[];
  SampleShared& sh = *reinterpret_cast<SampleShared*>(sm_raw);
  T* const held = reinterpret_cast<T*>(sm_raw + sizeof(SampleShared));
  auto cluster = cg::this_cluster();
  cluster.barrier_arrive();  // that it runs, for the first access of another CTA to its shared memory
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int row = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // this warp's tokens: [w0, w0 + per) of the slice
  const int slice0 = rank * a.slice, per = a.slice / kSampleWarps, w0 = warp * per;
  const int n_mine = max(0, min(per, a.V - slice0 - w0));
  const float temperature = a.by.temperatures ? a.by.temperatures[row] : a.by.temperature;
  const int top_k = a.by.top_ks ? a.by.top_ks[row] : a.by.top_k;
  const float top_p = a.by.top_ps ? a.by.top_ps[row] : a.by.top_p;
  const float min_p = a.by.min_ps ? a.by.min_ps[row] : a.by.min_p;
  const float u = a.u[row];
  const bool k_on = top_k > 0 && top_k < a.V, p_on = top_p < 1.f;
  const bool first_wins = !(temperature > 0.f) || top_k == 1;

  if (k_on || p_on)
    for (int i = tid; i < kBins; i += kSampleThreads) {
      sh.first.count[i] = sh.next.count[i] = sh.maxima[i] = 0u;
      sh.first.weight[i] = sh.next.weight[i] = 0ull;
    }
  for (int i = tid; i < 257; i += kSampleThreads) sh.power[i] = Power{table.p[i], static_cast<float>(table.p[i])};
  if (tid == 0) {
    const double c = 2.8853900817779268148 / static_cast<double>(temperature);
    sh.c_hi = static_cast<float>(c);
    sh.c_lo = isfinite(sh.c_hi) ? static_cast<float>(c - static_cast<double>(sh.c_hi)) : 0.f;
    for (int i = 0; i < 4; ++i) sh.listed[i] = 0u;
    sh.index = ~0u;
  }

  // ---- the slice, and the largest logit
  float mine = -INFINITY;
  {
    int j = lane;
    for (; j + 7 * 32 < n_mine; j += 8 * 32) {  // eight loads in flight
      T z[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) z[x] = raw_logit<T>(a, row, slice0 + w0 + j + 32 * x);
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        if (w0 + j + 32 * x < a.staged) held[w0 + j + 32 * x] = z[x];
        mine = fmaxf(mine, static_cast<float>(z[x]));
      }
    }
    for (; j < n_mine; j += 32) {
      const T z = raw_logit<T>(a, row, slice0 + w0 + j);
      if (w0 + j < a.staged) held[w0 + j] = z;
      mine = fmaxf(mine, static_cast<float>(z));
    }
    uint32_t k = __reduce_max_sync(~0u, order_key(mine));
    if (lane == 0) sh.warp32[warp] = k;
    cluster.barrier_wait();  // every CTA of the cluster has started (one with an empty slice is here before others are)
    __syncthreads();
    if (warp == 0) {
      k = __reduce_max_sync(~0u, lane < kSampleWarps ? sh.warp32[lane] : 0u);
      if (lane < C) *cluster.map_shared_rank(&sh.top[rank], lane) = k;
    }
  }
  cluster.sync();
  uint32_t top_key = sh.top[0];
  for (int i = 1; i < C; ++i) top_key = max(top_key, sh.top[i]);
  Row r;
  r.top = of_key(top_key) + 0.f;
  r.half = 0.5f * r.top;
  r.c_hi = sh.c_hi;
  r.c_lo = sh.c_lo;
  r.power = sh.power;
  if (r.top == -INFINITY) {  // nothing to choose from
    if (rank == 0 && tid == 0) {
      a.token[row] = -1;
      if (a.prob) a.prob[row] = 0.f;
    }
    return;  // (every CTA's stores to the others were before the barrier)
  }
  bool solo = false;  // the first CTA alone, with the tokens of its list
  int lists = 0;      // gatherings so far
  // f(logit, index) of this warp's tokens, a lane every 32nd
  auto each = [&](auto&& f) {
    if (solo) {
      for (unsigned int j = tid; j < sh.listed[lists - 1]; j += kSampleThreads) f(logit_of(sh.list[j]), static_cast<int>(sh.list[j] & ((1u << kIndexBits) - 1)));
      return;
    }
#pragma unroll 4
    for (int j = lane; j < n_mine; j += 32) {
      const int i = slice0 + w0 + j;
      f(static_cast<float>(w0 + j < a.staged ? held[w0 + j] : raw_logit<T>(a, row, i)), i);
    }
  };
  SampleShared& lead = *cluster.map_shared_rank(&sh, 0);
  auto sync = [&]() {
    if (solo)
      __syncthreads();
    else
      cluster.sync();
  };
  if (first_wins) {  // nothing to choose: the first of the largest
    unsigned int at = ~0u;
    each([&](float z, int i) {
      if (z == r.top) at = min(at, static_cast<unsigned int>(i));
    });
    at = __reduce_min_sync(~0u, at);
    if (lane == 0 && at != ~0u) atomicMin(&lead.index, at);
    cluster.sync();
    if (rank == 0 && tid == 0) {
      a.token[row] = static_cast<int32_t>(sh.index);
      if (a.prob) a.prob[row] = 1.f;
    }
    return;
  }
  auto tell = [&](auto* field, auto v) {  // every CTA, by the first one's first threads
    if (tid < C) *cluster.map_shared_rank(field, tid) = v;
  };
  // The tokens of bins low .. most into the first CTA's list, by way of each CTA's own.
  // Whether they all fitted.
  auto gather = [&](int low, int most) -> bool {
    auto value = [&](int j) {
      return j < n_mine ? static_cast<float>(w0 + j < a.staged ? held[w0 + j] : raw_logit<T>(a, row, slice0 + w0 + j)) : -INFINITY;
    };
    unsigned int* const mine_n = &sh.listed[lists];
#pragma unroll 4
    for (int j0 = 0; j0 < n_mine; j0 += 32) {
      const float z = value(j0 + lane);
      const int b = r.bin(z);
      const bool in = b >= low && b <= most;
      const unsigned int all = __ballot_sync(~0u, in);
      if (all) {
        unsigned int at = 0;
        if (lane == 0) at = atomicAdd(mine_n, __popc(all));
        at = __shfl_sync(~0u, at, 0) + __popc(all & ((1u << lane) - 1u));
        if (in && at < kList) sh.list[at] = place(z, slice0 + w0 + j0 + lane);
      }
    }
    __syncthreads();
    const unsigned int n = *mine_n;
    if (tid < C) cluster.map_shared_rank(&sh, tid)->lists_of[lists][rank] = n;
    cluster.sync();
    unsigned int total = 0, before = 0;
    for (int i = 0; i < C; ++i) {
      const unsigned int m = sh.lists_of[lists][i];
      if (i < rank) before += m;
      total += m;
    }
    const bool fit = total <= kList;
    if (fit && rank > 0)
      for (unsigned int i = tid; i < n; i += kSampleThreads) lead.list[before + i] = sh.list[i];
    if (fit && rank == 0 && tid == 0) *mine_n = total;
    ++lists;
    if (fit) cluster.sync();
    return fit;
  };

  auto least_weight = [&]() {  // by min-p
    return min_p > 0.f ? static_cast<unsigned long long>(ceil(fmin(static_cast<double>(min_p), 1.0) * static_cast<double>(1ull << kFraction))) : 0ull;
  };
  auto drawn = [&](int i, unsigned long long w, unsigned long long total) {
    a.token[row] = i;
    if (a.prob) a.prob[row] = static_cast<float>(static_cast<double>(w) / static_cast<double>(total));
  };
  auto goal_of = [&](unsigned long long total) {  // the first sum above it
    return min(u < 1.f ? share_of(u, total, false) : ~0ull, total - 1);
  };
  // The rest, by the first CTA, of a short list of all tokens up to the end or more, one
  // a thread: each counts the tokens before its own, in the order and by index. sum: all
  // weight, where there is no top-k. (64 rows of 131,072 with top-k 50: 35 us, with the
  // searches below 43; top-k 200, 42 and 45; 300, in lists of up to 512, 50 and 46.)
  auto few = [&](unsigned long long sum) {
    const int n = static_cast<int>(sh.listed[lists - 1]);
    const unsigned long long mine = tid < n ? sh.list[tid] : ~0ull;
    const uint32_t index = static_cast<uint32_t>(mine) & ((1u << kIndexBits) - 1);
    if (tid < 8) sh.list[n + tid] = ~0ull;  // (before no token, in either way)
    __syncthreads();
    int at = 0, by_index = 0;
    if (tid < n)
      for (int j = 0; j < n; j += 8)
#pragma unroll
        for (int x = 0; x < 8; x += 2) {
          const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&sh.list[j + x]);
          at += (o.x < mine) + (o.y < mine);
          by_index += ((static_cast<uint32_t>(o.x) & ((1u << kIndexBits) - 1)) < index) +
                      ((static_cast<uint32_t>(o.y) & ((1u << kIndexBits) - 1)) < index);
        }
    const unsigned long long w = tid < n && !(k_on && at >= top_k) ? r.weight(logit_of(mine)) : 0ull;
    if (tid < n) sh.first.weight[at] = w;
    __syncthreads();
    const unsigned long long v = tid < n ? sh.first.weight[tid] : 0ull, upto = block_scan_incl(v, sh.warp64);
    if (tid < n) sh.first.weight[tid] = upto - v;
    if (tid == kSampleThreads - 1) sh.found64 = upto;
    __syncthreads();
    if (k_on) sum = sh.found64;
    const unsigned long long end = p_on ? max(share_of(top_p, sum, true), 1ull) : ~0ull;
    const bool in = tid < n && w >= least_weight() && sh.first.weight[at] < end;
    if (tid < n) {
      sh.next.weight[by_index] = in ? w : 0ull;
      sh.next.count[by_index] = index;
    }
    __syncthreads();
    const unsigned long long x = tid < n ? sh.next.weight[tid] : 0ull, sums = block_scan_incl(x, sh.warp64);
    if (tid == kSampleThreads - 1) sh.found64 = sums;
    __syncthreads();
    const unsigned long long total = sh.found64, goal = goal_of(total);
    if (goal < sums && goal >= sums - x) drawn(static_cast<int>(sh.next.count[tid]), x, total);
  };

  int end_bin = kBins - 1;                   // kept: bin <= end_bin and place <= end
  unsigned long long end = ~0ull;
  if (k_on || p_on) {
    // ---- bins that can hold the end
    int most = kBins - 1;
    unsigned long long sum = 0;  // all weight, where top-p needs it
    if (k_on) {
      const int b = mine == -INFINITY ? kBins : r.bin(mine);
      if (b < kBins) atomicAdd(&sh.maxima[b], 1u);
      cluster.sync();
      if (rank == 0) {
        uint32_t n0 = 0, n1 = 0;
        for (int x = 0; x < C; ++x) {
          const uint2 n = *reinterpret_cast<const uint2*>(&cluster.map_shared_rank(&sh, x)->maxima[2 * tid]);
          n0 += n.x;
          n1 += n.y;
        }
        const uint32_t upto = block_scan_incl(n0 + n1, sh.warp32);
        if (tid == 0) sh.found = kBins - 1;
        __syncthreads();
        const uint32_t k = static_cast<uint32_t>(top_k);
        if (upto >= k && upto - n0 - n1 < k) sh.found = upto - n1 >= k ? 2 * tid : 2 * tid + 1;
        __syncthreads();
        const int f = sh.found;
        __syncthreads();
        tell(&sh.found, f);
      }
      cluster.sync();
      most = sh.found;
      if (gather(0, most)) {
        if (rank > 0) return;
        if (sh.listed[lists - 1] <= kFew) return few(0);
        solo = true;
      }
    }
    // ---- tokens and weight by bins of d
    each([&](float z, int) {
      const int b = r.bin(z);
      if (b <= most) {
        atomicAdd(&sh.first.count[b], 1u);
        add_shared(&sh.first.weight[b], r.weight(z));
      }
    });
    // The first CTA reads the others' histograms (adding theirs to its own by atomics
    // took longer than all the rest: 46 us of one row's top-p); they leave them until
    // after the next barrier.
    auto merge = [&](Hist& h) {
      sync();
      if (rank == 0 && !solo) {
        uint2 n = *reinterpret_cast<const uint2*>(&h.count[2 * tid]);
        ulonglong2 w = *reinterpret_cast<const ulonglong2*>(&h.weight[2 * tid]);
        for (int x = 1; x < C; ++x) {
          const Hist& o = *cluster.map_shared_rank(&h, x);
          const uint2 on = *reinterpret_cast<const uint2*>(&o.count[2 * tid]);
          const ulonglong2 ow = *reinterpret_cast<const ulonglong2*>(&o.weight[2 * tid]);
          n.x += on.x, n.y += on.y, w.x += ow.x, w.y += ow.y;
        }
        *reinterpret_cast<uint2*>(&h.count[2 * tid]) = n;
        *reinterpret_cast<ulonglong2*>(&h.weight[2 * tid]) = w;
      }
    };
    merge(sh.first);
    // ---- one search after the other: by number, then by weight
    bool cut_k = false;
#pragma unroll 1
    for (int by_weight = 0; by_weight < 2; ++by_weight) {
      if (by_weight ? !p_on : !k_on) continue;
      // round 0 is over bins of d, later ones over places
      unsigned long long goal = 0;  // the end is where the number or weight reaches it
      bool alone = false;           // the first CTA looks for the end, with the tokens of its bin
#pragma unroll 1
      for (int round = 0;; ++round) {
        if (rank == 0) {
          Hist& h = round == 0 ? sh.first : sh.next;
          if (round == 0 && by_weight) {
            if (cut_k) {  // what top-k has left of its last bin
              __syncthreads();
              if (tid == 0) {
                sh.first.weight[end_bin] = sh.search.sum - sh.search.bin_before;
                sh.first.count[end_bin] = sh.search.kept - sh.search.bin_n;
              }
            }
          }
          if (round == 0) goal = by_weight ? max(share_of(top_p, sum, true), 1ull) : static_cast<unsigned long long>(top_k);
          __syncthreads();
          uint32_t n0 = h.count[2 * tid], n1 = h.count[2 * tid + 1];
          unsigned long long s0 = h.weight[2 * tid], s1 = h.weight[2 * tid + 1];
          if (round == 0 && cut_k) {
            if (2 * tid > end_bin) n0 = 0, s0 = 0;
            if (2 * tid + 1 > end_bin) n1 = 0, s1 = 0;
          }
          const uint32_t nb = round == 0 ? 0u : sh.search.n_before;
          const unsigned long long sb = round == 0 ? 0ull : sh.search.before;
          const uint32_t n = nb + block_scan_incl(n0 + n1, sh.warp32);
          const unsigned long long s = sb + block_scan_incl(s0 + s1, sh.warp64);
          if (round == 0 && by_weight && !k_on) {
            if (tid == kSampleThreads - 1) sh.found64 = s;
            __syncthreads();
            sum = sh.found64;
            goal = max(share_of(top_p, sum, true), 1ull);
          }
          if (tid == 0) sh.found = 0;
          __syncthreads();
          // the bin in which the goal is reached
          const unsigned long long after = by_weight ? s : n, m0 = by_weight ? s0 : n0, m1 = by_weight ? s1 : n1;
          const bool here = after >= goal && after - m0 - m1 < goal && m0 + m1 > 0;
          if (here) {
            const bool second = after - m1 < goal;
            const int b = 2 * tid + second;
            Search q = sh.search;
            q.n_before = second ? n - n1 : n - n0 - n1;
            q.before = second ? s - s1 : s - s0 - s1;
            const uint32_t in = second ? n1 : n0;
            const unsigned long long weight_in = second ? s1 : s0;
            if (round == 0) {
              q.bin_n = q.n_before;
              q.bin_before = q.before;
              // the bin's logits, with room for rounding
              q.bin = b;
              const float per_bin = 2.f / (kBinsPer * r.c_hi), room = fabsf(r.top) * 0x1p-20f + per_bin * 0.01f;
              q.lo = b == 0 ? 0ull : place(r.top - per_bin * b + room, 0);
              q.hi = place(fmaxf(r.top - per_bin * (b + 1) - room, -3.402823466e38f), (1 << kIndexBits) - 1);
            } else {
              const unsigned long long lo = q.lo + (static_cast<unsigned long long>(b) << q.shift);
              q.hi = min(q.hi, lo + (1ull << q.shift) - 1);
              q.lo = lo;
            }
            // one token, or all of the bin's: no need to look closer
            q.done = in == 1 || (!by_weight && q.n_before + in == goal) || (round > 0 && q.shift == 0);
            q.sum = q.before + weight_in;
            q.kept = q.n_before + in;
            if (q.lo >> kIndexBits == q.hi >> kIndexBits)
              q.hi = min(q.hi, (q.hi >> kIndexBits << kIndexBits) + static_cast<unsigned int>(a.V - 1));
            q.shift = max(0, 54 - __clzll(static_cast<long long>(q.hi - q.lo) | 1));
            sh.search = q;
            sh.found = 1;
          }
          __syncthreads();
          if (tid == 0 && !sh.found) {  // fewer tokens than k have weight
            Search q = sh.search;
            q.bin = kBins - 1;
            q.lo = 0;
            q.hi = ~0ull;
            q.done = 2;
            q.kept = ~0u;
            sh.search = q;
          }
          if (tid == kSampleThreads - 1) sh.found64 = s;  // all weight (round 0)
          __syncthreads();
          if (sh.search.done == 2 && tid == 0) sh.search.sum = sh.found64;
          __syncthreads();
          if (!solo) {
            const Search q = sh.search;
            if (tid > 0 && tid < C) *cluster.map_shared_rank(&sh.search, tid) = q;
          }
        }
        sync();
        const Search q = sh.search;
        for (int i = tid; i < kBins; i += kSampleThreads) {
          sh.next.count[i] = 0u;
          sh.next.weight[i] = 0ull;
        }
        __syncthreads();
        if (!solo && !k_on && round == 0 && q.kept <= kList) {  // few tokens up to the end's bin
          if (gather(0, q.bin)) {
            if (rank > 0) return;
            if (sh.listed[lists - 1] <= kFew) return few(sum);
            solo = true;
          }
        }
        if (q.done) break;
        if (!solo && round == 0 && q.kept - q.n_before <= kList && gather(q.bin, q.bin)) {
          alone = true;
          if (rank > 0) break;
          solo = true;
        }
        each([&](float z, int i) {
          if (r.bin(z) != q.bin) return;
          const unsigned long long at = place(z, i);
          if (at < q.lo || at > q.hi || (q.bin == end_bin && at > end)) return;
          const int d = static_cast<int>((at - q.lo) >> q.shift);
          atomicAdd(&sh.next.count[d], 1u);
          add_shared(&sh.next.weight[d], r.weight(z));
        });
        merge(sh.next);
      }
      if (alone) {
        solo = false;
        if (rank == 0) {
          __syncthreads();
          const Search q = sh.search;
          if (tid > 0 && tid < C) *cluster.map_shared_rank(&sh.search, tid) = q;
        }
        cluster.sync();
      }
      const Search q = sh.search;
      if (q.done == 1) {
        end = q.bin == end_bin ? min(end, q.hi) : q.hi;
        end_bin = q.bin;
      }
      cut_k = q.done == 1;
      if (!by_weight) sum = q.sum;
      sync();  // the search is read before the next one's is written
    }
  }

  // ---- weights kept, in the order of the vocabulary
  const unsigned long long least = least_weight();
  const bool cut = end != ~0ull;
  auto kept = [&](float z, int i) -> unsigned long long {
    if (cut) {
      const int b = r.bin(z);
      if (b > end_bin || (b == end_bin && place(z, i) > end)) return 0ull;
    }
    const unsigned long long w = r.weight(z);
    return w >= least ? w : 0ull;
  };
  if (solo) {
    // by index: 1,024 stretches of the vocabulary, then the tokens of one of them
    const int shift = max(0, 32 - __clz(a.V - 1) - 10);
    for (int i = tid; i < kBins; i += kSampleThreads) sh.next.weight[i] = 0ull;
    __syncthreads();
    each([&](float z, int i) {
      const unsigned long long w = kept(z, i);
      if (w) add_shared(&sh.next.weight[i >> shift], w);
    });
    __syncthreads();
    const unsigned long long s0 = sh.next.weight[2 * tid], s1 = sh.next.weight[2 * tid + 1];
    const unsigned long long upto = block_scan_incl(s0 + s1, sh.warp64);
    if (tid == kSampleThreads - 1) sh.found64 = upto;
    __syncthreads();
    const unsigned long long total = sh.found64, goal = goal_of(total);
    __syncthreads();
    if (goal < upto && goal >= upto - s0 - s1) {
      const bool second = goal >= upto - s1;
      sh.found = 2 * tid + second;
      sh.found64 = goal - (second ? upto - s1 : upto - s0 - s1);
    }
    __syncthreads();
    const int stretch = sh.found;
    const unsigned long long rest = sh.found64;
    // of the stretch's tokens, at most 1,024, the one up to which the weights exceed what is left
    if (tid == 0) sh.index = 0u;
    __syncthreads();
    each([&](float z, int i) {
      if (i >> shift != stretch) return;
      const unsigned long long w = kept(z, i);
      if (!w) return;
      const unsigned int at = atomicAdd(&sh.index, 1u);
      sh.first.count[at] = static_cast<uint32_t>(i);
      sh.first.weight[at] = w;
    });
    __syncthreads();
    const unsigned int n = sh.index;
    for (unsigned int j = tid; j < n; j += kSampleThreads) {
      const uint32_t i = sh.first.count[j];
      const unsigned long long w = sh.first.weight[j];
      unsigned long long before = 0;
      for (unsigned int o = 0; o < n; ++o)
        if (sh.first.count[o] < i) before += sh.first.weight[o];
      if (before <= rest && rest < before + w) drawn(static_cast<int>(i), w, total);
    }
    return;
  }
  unsigned long long v = 0;
  if (cut)
    each([&](float z, int i) { v += kept(z, i); });
  else if (least)
    each([&](float z, int) {
      const unsigned long long w = r.weight(z);
      v += w >= least ? w : 0ull;
    });
  else
    each([&](float z, int) { v += r.weight(z); });
  v = warp_sum(v);
  if (lane < C) *cluster.map_shared_rank(&sh.chunk[rank * kSampleWarps + warp], lane) = v;
  cluster.sync();
  // (no CTA stores to another's shared memory from here on)
  unsigned long long total = 0, to_cta = 0;
  for (int i = lane; i < C * kSampleWarps; i += 32) {
    total += sh.chunk[i];
    if (i < rank * kSampleWarps) to_cta += sh.chunk[i];
  }
  total = warp_sum(total);
  to_cta = warp_sum(to_cta);
  const unsigned long long goal = goal_of(total);
  unsigned long long at = to_cta;  // before chunk c of this CTA
  int c = 0;
  for (; c < kSampleWarps; ++c) {
    const unsigned long long x = sh.chunk[rank * kSampleWarps + c];
    if (goal < at + x) break;
    at += x;
  }
  if (goal < to_cta || c == kSampleWarps) return;
  // ---- the token's warp chunk, cut between the CTA's warps
  const int part = ((per + kSampleWarps - 1) / kSampleWarps + 31) / 32 * 32, p0 = c * per + warp * part;
  const int p1 = min(c * per + per, p0 + part);
  auto weight_at = [&](int j) -> unsigned long long {
    const int i = slice0 + j;
    if (j >= p1 || i >= a.V) return 0ull;
    return kept(static_cast<float>(j < a.staged ? held[j] : raw_logit<T>(a, row, i)), i);
  };
  v = 0;
  for (int j = p0 + lane; j < p1; j += 32) v += weight_at(j);
  v = warp_sum(v);
  __syncthreads();
  if (lane == 0) sh.warp64[warp] = v;
  __syncthreads();
  for (int w = 0; w < warp; ++w) at += sh.warp64[w];
  if (goal < at || goal >= at + v) return;
  for (int j0 = p0; j0 < p1; j0 += 32) {
    const unsigned long long w = weight_at(j0 + lane);
    unsigned long long x = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned long long y = __shfl_up_sync(~0u, x, d);
      if (lane >= d) x += y;
    }
    const unsigned int above = __ballot_sync(~0u, at + x > goal);
    if (above) {
      if (lane == __ffs(above) - 1) drawn(slice0 + j0 + lane, w, total);
      return;
    }
    at += __shfl_sync(~0u, x, 31);
  }
}

const PowerTable& powers() {
  static const PowerTable t = [] {
    PowerTable p;
    for (int i = 0; i < 257; ++i) p.p[i] = static_cast<uint32_t>(std::llround(std::ldexp(std::exp2(-(i - 128) / 256.0), 31)));
    return p;
  }();
  return t;
}

template <class T>
cudaError_t sample(SampleArgs a, int rows, int num_sms, cudaStream_t st) {
  // CTAs a row: slices of 18,432 tokens at most, and smaller ones, down to 2,048,
  // while there are SMs without a CTA; 16, above the portable size, for a few long rows
  // alone (a row of 131,072 with top-k and top-p: 20.8 us against 24.9 with 8).
  int ctas = 1;
  while (ctas < 8 && (a.V > 18432 * ctas || (static_cast<int64_t>(rows) * ctas < num_sms && a.V >= 4096 * ctas))) ctas *= 2;
  if (ctas == 8 && rows * 32 <= num_sms && a.V >= 32768) ctas = kMostCtas;
  const int each = (a.V + ctas - 1) / ctas;
  a.slice = (each + kSampleThreads - 1) / kSampleThreads * kSampleThreads;
  constexpr int kMostSmem = 227 * 1024;
  constexpr int kBytes = static_cast<int>(sizeof(T));
  a.staged = std::min(a.slice, (kMostSmem - static_cast<int>(sizeof(SampleShared))) / kBytes);
  const int smem = static_cast<int>(sizeof(SampleShared)) + a.staged * kBytes;
  cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
  if (e != cudaSuccess) return e;
  if (ctas > 8 && (e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * ctas);
  cfg.blockDim = dim3(kSampleThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a, powers());
}

}  // namespace

cudaError_t launch_sample(const void* z, int32_t zt, int64_t ld, int32_t rows, int32_t V, const float* u, const moe_sampling_t& by,
                          int32_t* token, float* prob, int num_sms, cudaStream_t st) {
  SampleArgs a{};
  a.z = z;
  a.ld = ld;
  a.V = V;
  a.u = u;
  a.by = by;
  a.token = token;
  a.prob = prob;
  return zt == MOE_F32 ? sample<float>(a, rows, num_sms, st) : sample<__nv_bfloat16>(a, rows, num_sms, st);
}

}  // namespace moe
