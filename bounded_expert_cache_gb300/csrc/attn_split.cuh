// The launch that the attention kernels of warp-level instructions share: a
// unit's walk along the line of token tiles, the ring of tiles in shared memory,
// the join of partial results. An engine (of bf16, f32 or 4-bit pages) forms a
// tile's scores and adds its values. What is general about them stands in attn.cu.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "attn.cuh"
#include "pdl.cuh"
#include "prefill.h"
#include "tc.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr int kWarps = 8;  // computing warps; the first warp of a third warpgroup copies
constexpr int kCompute = 32 * kWarps;
constexpr int kThreads = kCompute + 128;

// barrier of the computing warps
__device__ __forceinline__ void sync_compute() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z) {
  tma4d(dst, m, bar, x, y, 0, z);
}
// A CTA's walk along the line: units in order, of each the tiles [t0, t1) that
// fall into the run. On the line a unit is `cost` positions, for its Q and its
// results, and then one per tile.
struct Cursor {
  int b, rt, h;   // sequence, row tile, cache head
  int rows;       // rows of the unit
  int tok0, hq0;  // the first one's token and its head in the group
  int t, t0, t1;  // tile of the unit, and this run's
  int per;        // tiles of the unit
  int cost;
  int64_t tiles0; // line position of the unit's first tile
  int64_t end;    // end of the run
  Seq s;
  Span sp;
  __device__ __forceinline__ void open(int64_t at) {
    t0 = static_cast<int>(max(at - tiles0, static_cast<int64_t>(0)));
    t1 = static_cast<int>(min(end - tiles0, static_cast<int64_t>(per)));
    t = t0;
  }
  __device__ __forceinline__ bool more() const { return tiles0 + per + cost < end; }
  // Row tile x of R rows. The (token, head) rows of a chunk may pass 32 bits
  // (WIDE), those of the newest few tokens do not; their first tile, mostly the
  // only one, needs no division (one context of 777 tokens: 11.5 us with it, 10.3).
  template <bool WIDE>
  __device__ __forceinline__ void row_tile(const AttnArgs& a, int x, int R) {
    rt = x;
    if (WIDE) {
      const int64_t r0 = static_cast<int64_t>(x) * R;
      tok0 = static_cast<int>(quotient(r0, a.g));
      hq0 = static_cast<int>(r0 - static_cast<int64_t>(tok0) * a.g);
      rows = static_cast<int>(min(static_cast<int64_t>(R), static_cast<int64_t>(s.m) * a.g - r0));
    } else {
      tok0 = x == 0 ? 0 : x * R / a.g;
      hq0 = x * R - tok0 * a.g;
      rows = min(R, s.m * a.g - x * R);
    }
  }
  // token of row r of the unit within the chunk, and its head
  __device__ __forceinline__ int token(const AttnArgs& a, int r) const { return tok0 + (hq0 + r) / a.g; }
  __device__ __forceinline__ int head(const AttnArgs& a, int r) const { return h * a.g + (hq0 + r) % a.g; }
};

// Tiles from the cursor's on that go together: neighbours, of this run.
template <int GROUP>
__device__ __forceinline__ int group_of(const Cursor& c) {
  if (GROUP == 1) return 1;
  const int n = min(GROUP, c.t1 - c.t);
  return c.t < c.sp.n0 ? min(n, c.sp.n0 - c.t) : n;
}

template <int KT>
__device__ __forceinline__ void open_seq(const AttnArgs& a, Cursor& c) {
  c.s = load_seq(a, c.b);
  c.sp = span_of<KT>(a, c.s, 0, c.s.m);
  c.per = c.sp.n;
}
// The next unit (decode); only called while c.more(), so there is one with a tile.
template <int KT, int R>
__device__ __forceinline__ void next_unit(const AttnArgs& a, Cursor& c) {
  c.tiles0 += c.per + c.cost;
  if (++c.h == a.Hkv) {
    c.h = 0;
    int rt = c.rt + 1;
    if (rt == a.row_tiles) {
      rt = 0;
      ++c.b;
      open_seq<KT>(a, c);
    }
    c.template row_tile<false>(a, rt, R);
  }
  c.open(c.tiles0);
}

// A tile in shared memory: per page (box of `rows` = min(page, KT) tokens),
// per column block of 128 bytes, `rows` rows of 128 bytes whose 16-byte pieces
// the copy has swizzled: piece c of row r lies at c ^ (r & 7).
struct Tile {
  uint32_t base;
  int shift;  // log2 of rows
  // start of the 128-byte row of token r in column block 0
  template <int NB>
  __device__ __forceinline__ uint32_t row(int r) const {
    return base + (((r >> shift) * NB) << (shift + 7)) + ((r & ((1 << shift) - 1)) << 7);
  }
  __device__ __forceinline__ uint32_t block() const { return 128u << shift; }
};

template <class T>
__device__ __forceinline__ void store4(T* dst, float4 v);
template <>
__device__ __forceinline__ void store4<float>(float* dst, float4 v) {
  *reinterpret_cast<float4*>(dst) = v;
}
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* dst, float4 v) {
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

// The result of a row: o / l, 0 for a row that sees nothing.
template <class T>
__device__ __forceinline__ void write_out(const AttnArgs& a, const Cursor& c, int r, int col, float4 v, float L) {
  const int i = c.token(a, r);
  const float inv = c.s.len - c.s.m + i < 0 ? 0.f : 1.f / L;
  T* dst = static_cast<T*>(a.out) + (c.s.row0 + i) * a.ldo + c.head(a, r) * a.D + col;
  if (inv == 0.f && c.s.len - c.s.m + i < 0)
    v = make_float4(0.f, 0.f, 0.f, 0.f);
  else
    v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
  store4<T>(dst, v);
}

// Block-wide inclusive scan of one int64 per thread; returns the thread's
// exclusive prefix and the total.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* tmp, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(~0u, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  int64_t base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) base += tmp[w];
    all += tmp[w];
  }
  __syncthreads();
  *total = all;
  return base + x - v;
}

// The ring takes what the merge buffer leaves of 220 KB (224 of codes), at most E::kMostSlots slots.
template <class E>
struct Ring {
  // a slot is a tile of K or of V; of codes, which are few bytes, up to E::kGroup of both
  static constexpr int kSlot = static_cast<int>(E::kTileBytes) * (E::kCodes ? 2 * E::kGroup : 1);
  static constexpr int kFit = ((E::kCodes ? 224 : 220) * 1024 - E::kMergeBytes) / kSlot;
  static constexpr int kSlots = kFit > E::kMostSlots ? E::kMostSlots : kFit;
  static constexpr int kSmem = kSlots * kSlot + E::kMergeBytes;
};

// SPLIT: runs of the line of tiles (decode). Otherwise one unit a CTA (chunks).
template <class E, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, AttnArgs a,
                int boxes) {
  constexpr int NS = Ring<E>::kSlots;
  static_assert(NS >= (E::kCodes ? 2 : 3), "ring");
  constexpr int KT = E::KT, R = E::kRows;
  extern __shared__ __align__(1024) unsigned char sm[];
  __shared__ uint64_t b_full[NS], b_empty[NS];
  __shared__ int64_t s_scan[kThreads / 32];
  __shared__ int64_t s_found[2];
  __shared__ float2 s_ml[E::kMl];
  __shared__ int s_abort;
  const uint32_t ring = su32(sm);
  if (ring & 1023u) {  // the swizzle's pattern starts at such a boundary
    if (threadIdx.x == 0) atomicOr(a.err, MOE_DEVERR_TIMEOUT);
    return;
  }
  if (SPLIT) {
    pdl_trigger();  // the joining launch may be scheduled; it waits for this one's end
    if (threadIdx.x == 0) a.cuts[blockIdx.x].count = 0;
  } else if (blockIdx.x == 0 && threadIdx.x == kThreads - 1) {
    check_chunks(a);
  }
  constexpr uint32_t kSlotBytes = Ring<E>::kSlot;
  float* merge = reinterpret_cast<float*>(sm + NS * kSlotBytes);
  const int rt_n = a.row_tiles;
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    s_abort = 0;
    s_found[0] = -1;
    for (int i = 0; i < NS; ++i) {
      mbar_init(su32(&b_full[i]), 1);
      mbar_init(su32(&b_empty[i]), kWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();

  // ---- this CTA's run of the line
  Cursor cp;
  cp.cost = SPLIT ? E::kUnitCost : 0;
  int64_t run0 = 0, total = 1;
  if (SPLIT) {
    auto line_of = [&](int b) -> int64_t {  // positions of a sequence
      if (b >= a.n) return 0;
      Seq s = load_seq(a, b);
      return static_cast<int64_t>(span_of<KT>(a, s, 0, s.m).n + E::kUnitCost) * rt_n * a.Hkv;
    };
    int64_t mine = 0, ex = 0, all = 0;
    for (int b0 = 0; b0 < a.n; b0 += kThreads) {
      mine = line_of(b0 + threadIdx.x);
      int64_t t;
      ex = block_scan(mine, s_scan, &t);
      all += t;
    }
    total = all;
    const Runs runs(total, gridDim.x);
    if (blockIdx.x >= runs.n) return;
    run0 = runs.start(blockIdx.x);
    int64_t base = 0;
    for (int b0 = 0; b0 < a.n; b0 += kThreads) {
      int64_t t = total;
      if (a.n > kThreads) {
        mine = line_of(b0 + threadIdx.x);
        ex = base + block_scan(mine, s_scan, &t);
      }
      if (run0 >= ex && run0 < ex + mine) {
        s_found[0] = b0 + threadIdx.x;
        s_found[1] = ex;
      }
      base += t;
      __syncthreads();
      if (run0 < base) break;
    }
    cp.b = static_cast<int>(s_found[0]);
    open_seq<KT>(a, cp);
    const int u = static_cast<int>(quotient(run0 - s_found[1], cp.per + E::kUnitCost));
    cp.template row_tile<false>(a, u / a.Hkv, R);
    cp.h = u % a.Hkv;
    cp.tiles0 = s_found[1] + static_cast<int64_t>(u) * (cp.per + E::kUnitCost) + E::kUnitCost;
    cp.end = runs.start(blockIdx.x + 1);
    cp.open(run0);
    if (cp.t1 <= cp.t0) return;  // a run within a unit's fixed cost
  } else {
    // row tiles of every sequence in order, cache heads innermost
    const int want = blockIdx.x / a.Hkv;
    cp.h = blockIdx.x % a.Hkv;
    int64_t base = 0;
    for (int b0 = 0; b0 < a.n && base <= want; b0 += kThreads) {
      int64_t mine = 0, t;
      if (b0 + static_cast<int>(threadIdx.x) < a.n)
        mine = (static_cast<int64_t>(chunk_rows(a, b0 + threadIdx.x)) * a.g + R - 1) / R;
      const int64_t ex = base + block_scan(mine, s_scan, &t);
      if (want >= ex && want < ex + mine) {
        s_found[0] = b0 + threadIdx.x;
        s_found[1] = want - ex;
      }
      base += t;
    }
    __syncthreads();
    if (s_found[0] < 0) return;
    cp.b = static_cast<int>(s_found[0]);
    cp.s = load_seq(a, cp.b);
    cp.template row_tile<true>(a, static_cast<int>(s_found[1]), R);
    cp.sp = span_of<KT>(a, cp.s, cp.tok0, cp.token(a, cp.rows - 1) + 1);
    cp.per = cp.sp.n;
    cp.tiles0 = 0;
    cp.end = cp.per;
    cp.open(0);
  }
  const int shift = min(a.page_shift, 31 - __clz(KT));  // log2 of a box's tokens

  // Registers: the block is launched with 384 x 168; the computing warpgroups
  // take 216 a thread, the third keeps 72 (256 x 216 + 128 x 72 = 384 x 168).
  if (warp >= kWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp > kWarps) return;
    // ---------------- copies: lane i brings page i of the tile; pages that no
    // row sees are left out
    RingPos rp;
    uint32_t n = 0, done = 0;  // slots filled, tiles of K and V in them
    const uint32_t most = a.copies;
    bool ok = true;
    while (ok && done < most) {
      // a lane's pages: every 32nd of the tiles'
      constexpr int kEach = (E::kGroup * KT / 16 + 31) / 32;
      const int tiles = group_of<E::kGroup>(cp);
      const uint32_t box_bytes = (E::kTileBytes / KT) << shift;
      int page[kEach], y[kEach];  // -1: none
      uint32_t bytes = 0;
#pragma unroll
      for (int x = 0; x < kEach; ++x) {
        const int box = lane + 32 * x, tok = cp.sp.tile(cp.t) * KT + (box << shift);
        y[x] = tok & ((1 << a.page_shift) - 1);
        page[x] = -1;
        if (box < (tiles * KT) >> shift && tok < cp.sp.end && (tok < a.sinks || tok + (1 << shift) > cp.sp.low)) {
          page[x] = __ldg(a.table + static_cast<int64_t>(cp.s.id) * a.max_pages + (tok >> a.page_shift));
          if (page[x] < 0 || page[x] >= a.n_pages) {
            atomicOr(a.err, MOE_DEVERR_BADIDX);
            page[x] = -1;
          }
        }
        bytes += __popc(__ballot_sync(~0u, page[x] >= 0)) * box_bytes;
      }
#pragma unroll
      for (int kv = 0; kv < (E::kCodes ? 1 : 2); ++kv) {
        const uint32_t full = su32(&b_full[rp.s]);
        if (n >= NS && !mbar_wait(su32(&b_empty[rp.s]), rp.ph ^ 1u, &s_abort, a.err, a.wait_cycles)) ok = false;
        // (computing warps whose wait has failed hand slots on whose copies may still be on their way)
        if (*static_cast<volatile int*>(&s_abort)) ok = false;
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(full, E::kCodes ? 2 * bytes : bytes);  // without pages the barrier completes by this arrival
        __syncwarp();
#pragma unroll
        for (int b = 0; b < kEach; ++b) {
          if (page[b] < 0) continue;
          const int box = lane + 32 * b, z = page[b] * a.Hkv + cp.h;
          if constexpr (E::kCodes) {
            // a head's codes of a page, and behind them its scales and offsets
            constexpr uint32_t kCode = E::kRowBytes, kMeta = E::kTileBytes / KT - kCode;
            const int64_t block = (static_cast<int64_t>(z) * (kCode + kMeta)) << a.page_shift;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const char* src = static_cast<const char*>(x ? a.v : a.k) + block;
              const uint32_t dst = ring + rp.s * kSlotBytes + x * (kSlotBytes / 2);
              bulk_copy(dst + ((box * kCode) << shift), src + y[b] * kCode, kCode << shift, full);
              bulk_copy(dst + E::kGroup * KT * kCode + ((box * kMeta) << shift),
                        src + (static_cast<int64_t>(kCode) << a.page_shift) + y[b] * kMeta, kMeta << shift, full);
            }
          } else {
            const uint32_t dst = ring + rp.s * kSlotBytes + box * box_bytes;
            for (int x = 0; x < boxes; ++x)
              tma_page(dst + x * (128u << shift), kv ? &map_v : &map_k, full, x * (128 / static_cast<int>(sizeof(typename E::T))),
                       y[b], z);
          }
        }
        __syncwarp();
        ++n;
        rp.next(NS);
      }
      done += E::kCodes ? tiles : 2;
      cp.t += tiles;
      if (cp.t < cp.t1) continue;
      if (!cp.more()) break;
      next_unit<KT, R>(a, cp);
    }
    // drain: copies in flight land before the CTA ends
    if (lane == 0)
      for (uint32_t j = 0; j < n && j < NS; ++j)
        mbar_drain(su32(&b_full[(n - 1 - j) % NS]), ((n - 1 - j) / NS) & 1u, a.err, kPrefillWaitCycles);
    return;
  }

  // ---------------- computing warps
  asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
  E eng;
  eng.place(merge);
  RingPos rp;
  Tile tile;
  tile.shift = shift;
  auto wait_tile = [&]() {
    mbar_wait(su32(&b_full[rp.s]), rp.ph, &s_abort, a.err, a.wait_cycles);
    tile.base = ring + rp.s * kSlotBytes;
  };
  auto free_tile = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(su32(&b_empty[rp.s]));
    rp.next(NS);
  };
  while (true) {
    // ---- one unit's share of the run
    eng.begin(a, cp);
    if constexpr (E::kCodes) {
      for (int tiles; cp.t < cp.t1; cp.t += tiles) {
        tiles = group_of<E::kGroup>(cp);
        wait_tile();
        eng.tiles(a, cp, tile.base, tiles);
        free_tile();
      }
    } else {
      for (; cp.t < cp.t1; ++cp.t) {
        wait_tile();
        eng.scores(a, cp, tile);
        free_tile();
        wait_tile();
        eng.values(a, cp, tile);
        free_tile();
      }
    }
    if (cp.t1 - cp.t0 == cp.per) {
      eng.end(a, cp, merge, s_ml, [&](int r, int col, float4 v, float, float L) {
        write_out<typename E::T>(a, cp, r, col, v, L);
      });
    } else {
      // partial rows of this CTA, (m, l, -, -) and the row: slot 0 if its run
      // starts inside the unit's tiles, else 1
      constexpr int kPS = E::DP + 4;
      constexpr int64_t kSlot = static_cast<int64_t>(kPartRows) * kPS;
      float* mine = a.part + (2 * static_cast<int64_t>(blockIdx.x) + (run0 > cp.tiles0 ? 0 : 1)) * kSlot;
      eng.end(a, cp, merge, s_ml, [&](int r, int col, float4 v, float M, float L) {
        *reinterpret_cast<float4*>(mine + r * kPS + 4 + col) = v;
        if (col == 0) *reinterpret_cast<float2*>(mine + r * kPS) = make_float2(M, L);
      });
      if (threadIdx.x == 0 && run0 <= cp.tiles0) {  // the unit's first part: the record for the join
        const Runs runs(total, gridDim.x);
        Cut cut;
        cut.count = static_cast<int>(runs.of(cp.tiles0 + cp.per - 1)) - static_cast<int>(blockIdx.x) + 1;
        cut.rt = cp.rt;
        cut.h = cp.h;
        cut.row0 = cp.s.row0;
        cut.m = cp.s.m;
        cut.len = cp.s.len;
        a.cuts[blockIdx.x] = cut;
      }
    }
    if (!cp.more()) break;
    next_unit<KT, R>(a, cp);
  }
}

// Join of one row of the unit whose first part is CTA c0's (blockIdx.x): the
// threads are DP / 4 column quads by part groups; the groups are added in order.
// Only c0's run starts no later than the unit's tiles, so its part is in its
// slot 1 and the others' in slot 0.
constexpr int kJoinThreads = 256;
constexpr int kMostParts = 256;  // CTAs of a launch
template <class T, int DP>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttnArgs a, int rows_per_tile) {
  constexpr int kC4 = DP / 4, kPG = kJoinThreads / kC4, kPS = DP + 4;
  constexpr int64_t kSlot = static_cast<int64_t>(kPartRows) * kPS;
  __shared__ float s_w[kMostParts];
  __shared__ float s_red[kJoinThreads / 32];
  __shared__ float4 s_sum[kJoinThreads];
  pdl_wait();
  const Cut cut = a.cuts[blockIdx.x];
  const int r = blockIdx.y;
  if (cut.count == 0 || r >= min(rows_per_tile, cut.m * a.g - cut.rt * rows_per_tile)) return;
  const int c0 = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  auto part = [&](int i) { return a.part + (2 * (c0 + i) + (i == 0 ? 1 : 0)) * kSlot + r * kPS; };
  const int c4 = tid % kC4, pg = tid / kC4;
  // a part's weight is 2^(m_i - M); parts are at most as many as threads
  float2 ml = make_float2(-INFINITY, 0.f);
  if (tid < cut.count) ml = __ldcg(reinterpret_cast<const float2*>(part(tid)));
  float M = ml.x;
#pragma unroll
  for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, x));
  if (lane == 0) s_red[tid >> 5] = M;
  __syncthreads();
  M = s_red[lane & 7];
#pragma unroll
  for (int x = 4; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, x));
  const float w = ex2(ml.x - (M == -INFINITY ? 0.f : M));
  s_w[tid] = tid < cut.count ? w : 0.f;
  float L = tid < cut.count ? w * ml.y : 0.f;
#pragma unroll
  for (int x = 16; x; x >>= 1) L += __shfl_xor_sync(~0u, L, x);
  __syncthreads();
  if (lane == 0) s_red[tid >> 5] = L;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c4 * 4 < a.D) {
#pragma unroll 8
    for (int i = pg; i < cut.count; i += kPG) {
      const float4 u = __ldcg(reinterpret_cast<const float4*>(part(i) + 4 + c4 * 4));
      const float f = s_w[i];
      v.x += f * u.x;
      v.y += f * u.y;
      v.z += f * u.z;
      v.w += f * u.w;
    }
  }
  s_sum[tid] = v;
  __syncthreads();
  if (pg > 0 || c4 * 4 >= a.D) return;
  L = 0.f;
#pragma unroll
  for (int i = 0; i < kJoinThreads / 32; ++i) L += s_red[i];
#pragma unroll
  for (int i = 1; i < kPG; ++i) {
    const float4 u = s_sum[i * kC4 + c4];
    v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
  }
  Cursor c;
  c.h = cut.h;
  c.s.row0 = cut.row0;
  c.s.m = cut.m;
  c.s.len = cut.len;
  c.row_tile<false>(a, cut.rt, rows_per_tile);
  write_out<T>(a, c, r, c4 * 4, v, L);
}

template <class E, bool SPLIT>
cudaError_t launch(const AttnArgs& a, int grid, cudaStream_t st) {
  constexpr int es = static_cast<int>(sizeof(typename E::T));
  cudaError_t e = E::kCodes ? cudaSuccess : encoder();
  if (e != cudaSuccess) return e;
  CUtensorMap mk{}, mv{};  // (pages of codes are copied without)
  const int page = 1 << a.page_shift;
  const int64_t blocks = static_cast<int64_t>(a.n_pages) * a.Hkv;
  int boxes = 0;
  if (!E::kCodes &&
      ((e = map_page_cols(&mk, a.k, es, a.D, page, blocks, std::min(page, E::KT), E::NB, &boxes)) != cudaSuccess ||
       (e = map_page_cols(&mv, a.v, es, a.D, page, blocks, std::min(page, E::KT), E::NB, &boxes)) != cudaSuccess))
    return e;
  constexpr int smem = Ring<E>::kSmem;
  e = cudaFuncSetAttribute(attn_kernel<E, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  attn_kernel<E, SPLIT><<<grid, kThreads, smem, st>>>(mk, mv, a, boxes);
  return cudaGetLastError();
}

template <class E>
cudaError_t decode_rows(AttnArgs a, int num_sms, cudaStream_t st) {
  a.row_tiles = (a.n_q * a.g + E::kRows - 1) / E::kRows;
  const int ctas = std::min(num_sms, kMostParts);
  cudaError_t e = launch<E, true>(a, ctas, st);
  if (e != cudaSuccess) return e;
  return pdl_launch(join_kernel<typename E::T, E::DP>, dim3(ctas, std::min(E::kRows, a.n_q * a.g)), dim3(kJoinThreads), 0,
                    st, a, E::kRows);
}

}  // namespace
}  // namespace moe
