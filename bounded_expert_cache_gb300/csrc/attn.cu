// Attention over the paged cache on warp-level matrix instructions (bf16) and
// on the CUDA cores (f32): the newest tokens of many sequences, split over the
// cache's length and joined; and whole row tiles of prompt chunks.
//
// For a row at position p with visible tokens J:
//   s_j = c q.k_j (c = scale log2 e),  m = max s_j,  o = sum 2^(s_j-m) v_j / sum 2^(s_j-m),
// computed in one pass over the tokens with a running (m, l, o): a tile with a
// larger maximum m' scales l and o by 2^(m-m') first. Two partial results of
// disjoint token sets join by the same rule, which is what lets several warps,
// and several CTAs, share one row's tokens.
//
// Rows: the group's query heads share a cache head, so a unit of work is one
// (sequence, row tile, cache head) whose rows are (token, head of the group)
// pairs, and K and V are read once for all of them.
//
// Decode work split: the token tiles of all units (and a unit's fixed cost)
// form one line, cut into one equal run per CTA (one CTA per SM). A run covers
// whole units or ends inside one; a unit cut by run ends leaves partial
// (m, l, o) rows in the scratch, and
// a second small launch (a block per row, scheduled while the first drains)
// joins them in run order, so results do not depend on timing. One CTA joining
// a unit's parts after the last had arrived took up to 20 us of the 96 that
// 4 x 32,768 tokens at D 256 took, against 3 for the launch. Every CTA derives
// the cut from the lengths itself: no planning launch, no host copy of lengths.
//
// What bounds it: HBM. One warp walks the run and brings K and V tiles in by
// TMA, a box per page, into a ring in shared memory; eight warps compute. The
// copies run ahead across tiles and units, so the memory pipe stays full while
// a unit ends. Waits are bounded; after a time-out (recorded as an error) the
// loops run to their end on whatever is there, so no barrier is left waiting.
// Measured, bf16: three contexts of 131,072 to 262,143 tokens, 8 heads of 128:
// 354 us, 6.9 TB/s; 40 contexts of 0 to 32,768 tokens, 4 new tokens, 2 heads of
// 256: 65 us, 4.4 TB/s (the fixed costs of 78 units; 63 in a captured graph); one
// of 777: 10 us (9 in a graph), the latency of the dependent loads and of the
// second launch. Prompts here are not split, and run at the rate of warp-level
// instructions or of the CUDA cores: 4,096 tokens at 32K, 16 heads of 256: 7.6 ms;
// f32, 2,048 rows of 8,192 tokens, 8 heads of 80: 2.35 ms.
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
// Reads of shared memory: volatile keeps them behind the waits for the data;
// without a memory clobber other work may move across them.
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// ------------------------------------------------------------ bf16 engine
// RG row groups of 16 rows by KG = 8 / RG token groups, one warp each. Per
// tile a warp forms S = Q K^T for its 16 rows and KT / KG tokens (m16n8k16,
// K rows as the columns of B), updates its own (m, l), and adds P V with P
// straight from its accumulators. DP: head size padded to 64, 128 or 256.
template <int DP_, int RG_, int KT_>
struct MmaEngine {
  using T = __nv_bfloat16;
  static constexpr int DP = DP_, RG = RG_, KT = KT_;
  static constexpr int KG = kWarps / RG, kRows = RG * 16, KC = KT / KG / 16;
  static constexpr int NB = DP / 64;  // column blocks
  // Tiles' worth of time of a unit's Q, edge tile, merge of the warps and results
  // (40 contexts of 0 to 32,768 tokens, 4 new ones, heads of 256: 75 us with 4,
  // 68 with 5, 62.6 with 6, 63.4 with 8; of 128: 47.7 with 2, 42 with 3 and 4).
  static constexpr int kUnitCost = DP > 128 ? 6 : 3;
  static constexpr uint32_t kTileBytes = KT * DP * 2;
  // Q of large heads stays in shared memory: its fragments would not fit
  // beside the results' in registers
  static constexpr bool kQInSmem = DP > 128;
  static constexpr int kQPitch = DP * 2 + 16;
  static constexpr int kMergeBytes = kWarps * 16 * 64 * 4 + (kQInSmem ? kRows * kQPitch : 0);
  static_assert(KC >= 1 && KC * KG * 16 == KT, "token groups");

  uint32_t qf[kQInSmem ? 1 : DP / 16][4];
  uint32_t qs;        // shared copy of Q
  float o[DP / 8][4];
  float s[KC][2][4];
  uint32_t p[KC][4];
  float m[2], l[2];
  int pos[2];     // positions of this thread's rows lane / 4 and + 8; -1: no row
  bool active;    // the warp has a row
  bool edge;      // the tile holds a token seen by some but not all of the warp's rows
  uint32_t seen[KC];  // of an edge tile, per chunk: bit 4r+i of s[r][i] visible
  int rg, kg;

  __device__ __forceinline__ void begin(const AttnArgs& a, const Cursor& c) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    rg = warp / KG;
    kg = warp % KG;
    const int first = rg * 16, total = c.rows;
    active = first < total;
    const T* q[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = first + lane / 4 + 8 * h;
      pos[h] = -1;
      q[h] = nullptr;
      if (r < total) {
        const int i = c.token(a, r);
        pos[h] = c.s.len - c.s.m + i;
        q[h] = static_cast<const T*>(a.q) + (c.s.row0 + i) * a.ldq + c.head(a, r) * a.D;
      }
      m[h] = -INFINITY;
      l[h] = 0.f;
    }
    if constexpr (kQInSmem) {
      // this warp's rows, a lane a 16-byte piece; the KG warps of a row group
      // write the same
      static_assert(DP / 8 == 32, "a lane a piece");
      int i = c.token(a, first), hq = c.head(a, first) - c.h * a.g;
      const T* src = static_cast<const T*>(a.q) + c.h * a.g * a.D + lane * 8;
#pragma unroll 1
      for (int r0 = 0; r0 < 16; r0 += 8) {
        uint4 v[8];  // eight loads in flight
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          v[x] = make_uint4(0u, 0u, 0u, 0u);
          if (first + r0 + x < total && lane * 8 < a.D)
            v[x] = __ldg(reinterpret_cast<const uint4*>(src + (c.s.row0 + i) * a.ldq + hq * a.D));
          if (++hq == a.g) {
            hq = 0;
            ++i;
          }
        }
#pragma unroll
        for (int x = 0; x < 8; ++x)
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(qs + (rg * 16 + r0 + x) * kQPitch + lane * 16),
                       "r"(v[x].x), "r"(v[x].y), "r"(v[x].z), "r"(v[x].w)
                       : "memory");
      }
      __syncwarp();
    } else {
#pragma unroll
      for (int k = 0; k < DP / 16; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int d = k * 16 + (i >> 1) * 8 + (lane & 3) * 2;
          qf[k][i] = (q[i & 1] && d < a.D) ? __ldg(reinterpret_cast<const unsigned int*>(q[i & 1] + d)) : 0u;
        }
    }
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
  }

  __device__ __forceinline__ void scores(const AttnArgs& a, const Cursor& c, const Tile& kt) {
    if (!active) return;
    const int lane = threadIdx.x & 31;
    const int tile0 = c.sp.tile(c.t) * KT;
    // every row of the warp sees every token of the tile, or some do not
    const int lo_pos = c.s.len - c.s.m + c.token(a, rg * 16);
    const int hi_pos = c.s.len - c.s.m + c.token(a, min(rg * 16 + 15, c.rows - 1));
    edge = tile0 + KT - 1 > lo_pos;
    if (a.window > 0) edge |= hi_pos - tile0 >= a.window;
#pragma unroll
    for (int ch = 0; ch < KC; ++ch) {
      const int key0 = (ch * KG + kg) * 16;
#pragma unroll
      for (int i = 0; i < 8; ++i) s[ch][i >> 2][i & 3] = 0.f;
      // matrices: tokens 0-7 (d, d+8), tokens 8-15 (d, d+8)
      const int r = key0 + (lane & 7) + ((lane >> 4) << 3);
      const uint32_t at = kt.row<NB>(r);
#pragma unroll
      for (int k = 0; k < DP / 16; ++k) {
        uint32_t b[4];
        const int piece = 2 * k + ((lane >> 3) & 1);
        ldsm4(b, at + (piece >> 3) * kt.block() + (((piece & 7) ^ (r & 7)) << 4));
        if constexpr (kQInSmem) {
          uint32_t qa[4];
          ldsm4(qa, qs + (rg * 16 + (lane & 15)) * kQPitch + (2 * k + (lane >> 4)) * 16);
          mma16816(s[ch][0], qa, b[0], b[1]);
          mma16816(s[ch][1], qa, b[2], b[3]);
        } else {
          mma16816(s[ch][0], qf[k], b[0], b[1]);
          mma16816(s[ch][1], qf[k], b[2], b[3]);
        }
      }
    }
    float mx[2] = {m[0], m[1]};
#pragma unroll
    for (int ch = 0; ch < KC; ++ch) {
      seen[ch] = 0xFFu;
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v = s[ch][r][i] * a.scale_log2;
          if (edge) {
            const int j = tile0 + (ch * KG + kg) * 16 + r * 8 + (lane & 3) * 2 + (i & 1);
            const int back = pos[i >> 1] - j;
            const bool see = back >= 0 && (a.window == 0 || back < a.window || j < a.sinks);
            if (!see) {
              v = -INFINITY;
              seen[ch] &= ~(1u << (4 * r + i));
            }
          }
          s[ch][r][i] = v;
          mx[i >> 1] = fmaxf(mx[i >> 1], v);
        }
    }
    float f[2], mu[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(~0u, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(~0u, mx[h], 2));
      mu[h] = mx[h] == -INFINITY ? 0.f : mx[h];  // nothing seen yet: every numerator is 2^-inf = 0
      f[h] = ex2(m[h] - mu[h]);
      m[h] = mx[h];
      l[h] *= f[h];
    }
#pragma unroll
    for (int ch = 0; ch < KC; ++ch) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[ch][r][i] = ex2(s[ch][r][i] - mu[i >> 1]);
          l[i >> 1] += s[ch][r][i];
        }
      // numerators round to bf16 for the matrix product (the sum l keeps fp32):
      // relative 2^-8 each at most, as the rounding of a bf16 result
      p[ch][0] = pack_bf16(s[ch][0][0], s[ch][0][1]);
      p[ch][1] = pack_bf16(s[ch][0][2], s[ch][0][3]);
      p[ch][2] = pack_bf16(s[ch][1][0], s[ch][1][1]);
      p[ch][3] = pack_bf16(s[ch][1][2], s[ch][1][3]);
    }
    if (__any_sync(~0u, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
      for (int n = 0; n < DP / 8; ++n) {
        o[n][0] *= f[0];
        o[n][1] *= f[0];
        o[n][2] *= f[1];
        o[n][3] *= f[1];
      }
    }
  }

  __device__ __forceinline__ void values(const AttnArgs& a, const Cursor& c, const Tile& vt) {
    if (!active) return;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int ch = 0; ch < KC; ++ch) {
      const int key0 = (ch * KG + kg) * 16;
      if (edge) {
        // a product with a zero numerator would carry the infinity or NaN of a
        // token into rows that do not see it
        const bool bad = clean(a, c, vt, key0);
        if (bad) {
          values_by_row(vt, key0, ch);
          continue;
        }
      }
      const int r = key0 + (lane & 7) + (((lane >> 3) & 1) << 3);
      const uint32_t at = vt.row<NB>(r);
#pragma unroll
      for (int n = 0; n < DP / 16; ++n) {
        uint32_t b[4];
        const int piece = 2 * n + (lane >> 4);
        ldsm4t(b, at + (piece >> 3) * vt.block() + (((piece & 7) ^ (r & 7)) << 4));
        mma16816(o[2 * n], p[ch], b[0], b[1]);
        mma16816(o[2 * n + 1], p[ch], b[2], b[3]);
      }
    }
    if (edge) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the zeros, before the slot's next copy
  }

  // Zero the chunk's tokens that no row of the unit sees (the slot may hold
  // anything there); is there an infinity or NaN among the others?
  __device__ __forceinline__ bool clean(const AttnArgs& a, const Cursor& c, const Tile& vt, int key0) const {
    const int lane = threadIdx.x & 31;
    const int j0 = c.sp.tile(c.t) * KT + key0;
    bool bad = false;
#pragma unroll
    for (int x = 0; x < NB; ++x) {  // a column block: four pieces a lane
      uint32_t at[4], w[4][4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int r = y * 4 + (lane >> 3);
        at[y] = vt.row<NB>(key0 + r) + x * vt.block() + ((lane & 7) << 4);
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[y][0]), "=r"(w[y][1]), "=r"(w[y][2]), "=r"(w[y][3])
                     : "r"(at[y]));
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int j = j0 + y * 4 + (lane >> 3);
        if (j >= c.sp.end || (j >= a.sinks && j < c.sp.low))
          asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(at[y]), "r"(0) : "memory");
        else
          bad |= nonfinite2(w[y][0]) || nonfinite2(w[y][1]) || nonfinite2(w[y][2]) || nonfinite2(w[y][3]);
      }
    }
    bad = __any_sync(~0u, bad);
    __syncwarp();  // (a vote orders no memory) other lanes read these zeros
    return bad;
  }

  __device__ __forceinline__ void values_by_row(const Tile& vt, int key0, int ch) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int key = 0; key < 16; ++key) {
      // the quad's thread (key % 8) / 2 holds this token's numerators
      const int from = (lane & ~3) | ((key & 7) >> 1);
      float pr[2];
      uint32_t mask = 0;
#pragma unroll
      for (int cc = 0; cc < KC; ++cc) {
        if (cc != ch) continue;
        mask = __shfl_sync(~0u, seen[cc], from);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t w = __shfl_sync(~0u, key < 8 ? p[cc][h] : p[cc][2 + h], from);
          pr[h] = __uint_as_float((key & 1) ? (w & 0xFFFF0000u) : (w << 16));
        }
      }
      const int r = key0 + key;
      const uint32_t at = vt.row<NB>(r) + (lane & 3) * 4;
#pragma unroll
      for (int n = 0; n < DP / 8; ++n) {
        uint32_t w;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(at + (n >> 3) * vt.block() + (((n & 7) ^ (r & 7)) << 4)));
        const float v[2] = {__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((mask >> (4 * (key >> 3) + (i >> 1) * 2 + (key & 1))) & 1) o[n][i] += pr[i >> 1] * v[i & 1];
      }
    }
  }

  // Join the token groups' results in shared memory, 64 columns at a time, and
  // hand (row, column, 4 values, m, l) to store. Called by every thread.
  template <class F>
  __device__ __forceinline__ void end(const AttnArgs& a, const Cursor& c, float* buf, float2* ml, F&& store) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(~0u, l[h], 1);
      l[h] += __shfl_xor_sync(~0u, l[h], 2);
      if ((lane & 3) == 0) ml[warp * 16 + lane / 4 + 8 * h] = make_float2(m[h], l[h]);
    }
    const int rows = c.rows;
#pragma unroll
    for (int n0 = 0; n0 < DP; n0 += 64) {
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(buf + (warp * 16 + lane / 4 + 8 * h) * 64 + ((n * 8 + (lane & 3) * 2) ^ ((lane & 12) << 1))) =
              make_float2(o[n0 / 8 + n][2 * h], o[n0 / 8 + n][2 * h + 1]);
      sync_compute();
      for (int e = threadIdx.x; e < rows * 16; e += kCompute) {
        const int r = e >> 4, col = (e & 15) * 4;
        if (n0 + col < a.D) {
          const int w0 = (r >> 4) * KG, rr = r & 15;
          float M = -INFINITY;
#pragma unroll
          for (int k = 0; k < KG; ++k) M = fmaxf(M, ml[(w0 + k) * 16 + rr].x);
          const float Mu = M == -INFINITY ? 0.f : M;
          float L = 0.f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < KG; ++k) {
            const float2 t = ml[(w0 + k) * 16 + rr];
            const float f = ex2(t.x - Mu);
            L += f * t.y;
            const float4 u =
                *reinterpret_cast<const float4*>(buf + ((w0 + k) * 16 + rr) * 64 + (col ^ ((rr & 3) << 3)));
            v.x += f * u.x;
            v.y += f * u.y;
            v.z += f * u.z;
            v.w += f * u.w;
          }
          store(r, n0 + col, v, M, L);
        }
      }
      sync_compute();
    }
  }
};

// ------------------------------------------------------------- f32 engine
// R rows (4 or 16) in fp32 on the CUDA cores; K and V are read from shared
// memory once for all of them. Scores: the lanes of a warp are TPW tokens by
// 32 / TPW parts of the head, each for every row. Softmax: a warp a row, or two.
// Values: a thread owns four columns of every row and each TG-th token; the
// token groups are added when the unit ends.
template <int DP_, int R_>
struct FmaEngine {
  using T = float;
  static constexpr int DP = DP_, kRows = R_, KT = DP == 256 ? 32 : 64;
  static constexpr int NB = DP / 32;                // column blocks
  // as the bf16 engine's (9 contexts in a window of 1,024, heads of 96: 13.2 us
  // with 1, 12.9 with 2, 14.4 with 3; 16 to 29,004 tokens, 4 new ones, heads of
  // 256: 261 with 2, 238 with 3 and 4)
  static constexpr int kUnitCost = DP > 128 ? 3 : 2;
  static constexpr uint32_t kTileBytes = KT * DP * 4;
  static constexpr int kC4 = DP / 4;                // column quads
  static constexpr int kTok4 = KT / 4;              // threads along the tokens (scores)
  static constexpr int P = kCompute / (kTok4 * (kRows / 4));  // parts of the head
  static constexpr int TG = kCompute / kC4;         // token groups (values)
  static constexpr int kSum = TG * 4 * DP;          // floats of the groups' results of 4 rows
  static constexpr int kSP = kRows + 4;             // pitch of a token's numerators
  static constexpr int kMergeBytes = (kSum + kRows * DP + kRows * KT + KT * kSP + kRows) * 4;
  static_assert(P >= 4 && P <= 32 && KT % TG == 0, "work of a thread");

  float4 o[kRows];
  float m[2], l[2];  // of this warp's rows: warp, and warp + 8
  float *sum, *qs, *ss, *ps, *fs;
  bool edge;

  __device__ __forceinline__ void place(float* buf) {
    sum = buf;
    qs = sum + kSum;
    ss = qs + kRows * DP;
    ps = ss + kRows * KT;
    fs = ps + KT * kSP;
  }
  __device__ __forceinline__ void begin(const AttnArgs& a, const Cursor& c) {
    for (int e = threadIdx.x; e < kRows * DP; e += kCompute) {
      const int r = e / DP, d = e % DP;
      float v = 0.f;
      if (r < c.rows && d < a.D)
        v = __ldg(static_cast<const float*>(a.q) + (c.s.row0 + c.token(a, r)) * a.ldq + c.head(a, r) * a.D + d);
      qs[e] = v;
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.f;
    }
    sync_compute();
  }

  __device__ __forceinline__ static float4 lds4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
  }
  // position of row r of the tile, -1 past the last row
  __device__ __forceinline__ static int pos_of(const AttnArgs& a, const Cursor& c, int r) {
    return r < c.rows ? c.s.len - c.s.m + c.token(a, r) : -1;
  }
  __device__ __forceinline__ static bool sees(const AttnArgs& a, int pos, int j) {
    const int back = pos - j;
    return back >= 0 && (a.window == 0 || back < a.window || j < a.sinks);
  }

  __device__ __forceinline__ void scores(const AttnArgs& a, const Cursor& c, const Tile& kt) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile0 = c.sp.tile(c.t) * KT;
    {
      const int part = threadIdx.x % P, rest = threadIdx.x / P, rg = rest / kTok4, tg = rest % kTok4;
      // neighbouring token threads four rows apart: eight lanes of a read then
      // meet eight different banks (P = 4), whatever the swizzle
      const int t0 = kTok4 >= 8 ? (tg & ~7) | ((tg & 1) << 2) | ((tg & 7) >> 1) : tg;
      uint32_t at[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) at[i] = kt.row<NB>(t0 + kTok4 * i);
      const float* q0 = qs + rg * 4 * DP;
      float acc[16] = {};
      for (int d4 = part; d4 * 4 < a.D; d4 += P) {  // columns past the head are zeros
        float4 k[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          k[i] = lds4(at[i] + (d4 >> 3) * kt.block() + (((d4 & 7) ^ ((t0 + kTok4 * i) & 7)) << 4));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float4 q = *reinterpret_cast<const float4*>(q0 + r * DP + d4 * 4);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[r * 4 + i] += q.x * k[i].x + q.y * k[i].y + q.z * k[i].z + q.w * k[i].w;
        }
      }
      int first = 0, n = 16;  // of the 16 sums, this lane keeps [first, first + n)
#pragma unroll
      for (int x = 1; x < P; x <<= 1) {
        const bool up = part & x;
        if (n > 1) {
          n /= 2;
          if (up) first += n;
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            if (v >= n) break;
            const float keep = up ? acc[v + n] : acc[v], give = up ? acc[v] : acc[v + n];
            acc[v] = keep + __shfl_xor_sync(~0u, give, x);
          }
        } else {
          acc[0] += __shfl_xor_sync(~0u, acc[0], x);
        }
      }
#pragma unroll
      for (int v = 0; v < 16 / (P < 16 ? P : 16); ++v) {
        const int e = first + v;
        ss[(rg * 4 + (e >> 2)) * KT + t0 + kTok4 * (e & 3)] = acc[v];
      }
    }
    const int lo_pos = pos_of(a, c, 0);
    const int hi_pos = c.s.len - c.s.m + c.token(a, c.rows - 1);
    edge = tile0 + KT - 1 > lo_pos || (a.window > 0 && hi_pos - tile0 >= a.window);
    sync_compute();
#pragma unroll
    for (int h = 0; h < (kRows + kWarps - 1) / kWarps; ++h) {
      const int rr = warp + kWarps * h;
      if (rr >= kRows) break;
      const int pos = pos_of(a, c, rr);
      float v[KT / 32], mx = m[h];
#pragma unroll
      for (int x = 0; x < KT / 32; ++x) {
        const int t = lane + 32 * x;
        v[x] = sees(a, pos, tile0 + t) ? ss[rr * KT + t] * a.scale_log2 : -INFINITY;
        mx = fmaxf(mx, v[x]);
      }
#pragma unroll
      for (int x = 16; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, x));
      const float mu = mx == -INFINITY ? 0.f : mx, f = ex2(m[h] - mu);
      m[h] = mx;
      l[h] *= f;  // this lane's tokens only, until the end
#pragma unroll
      for (int x = 0; x < KT / 32; ++x) {
        const float p = ex2(v[x] - mu);
        l[h] += p;
        ps[(lane + 32 * x) * kSP + rr] = p;
      }
      if (lane == 0) fs[rr] = f;
    }
    sync_compute();
  }

  __device__ __forceinline__ void values(const AttnArgs& a, const Cursor& c, const Tile& vt) {
    const int c4 = threadIdx.x % kC4, tg = threadIdx.x / kC4;
    const int tile0 = c.sp.tile(c.t) * KT;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float f = fs[r];
      o[r].x *= f, o[r].y *= f, o[r].z *= f, o[r].w *= f;
    }
#pragma unroll 2
    for (int key = tg; key < KT; key += TG) {
      const float4 v = lds4(vt.row<NB>(key) + (c4 >> 3) * vt.block() + (((c4 & 7) ^ (key & 7)) << 4));
      const float4* p4 = reinterpret_cast<const float4*>(ps + key * kSP);
      if (edge && !(isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w))) {
        // a hidden token's infinity or NaN times its zero numerator is not added
        for (int r = 0; r < kRows; ++r) {
          const bool see = sees(a, pos_of(a, c, r), tile0 + key);
          const float p = ps[key * kSP + r];
          add_row(r, see, p, v);
        }
        continue;
      }
#pragma unroll
      for (int q = 0; q < kRows / 4; ++q) {
        const float4 p = p4[q];
        const float pr[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[4 * q + i].x += pr[i] * v.x;
          o[4 * q + i].y += pr[i] * v.y;
          o[4 * q + i].z += pr[i] * v.z;
          o[4 * q + i].w += pr[i] * v.w;
        }
      }
    }
  }
  __device__ __forceinline__ void add_row(int row, bool see, float p, const float4& v) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (r != row || !see) continue;
      o[r].x += p * v.x;
      o[r].y += p * v.y;
      o[r].z += p * v.z;
      o[r].w += p * v.w;
    }
  }

  template <class F>
  __device__ __forceinline__ void end(const AttnArgs& a, const Cursor& c, float*, float2* ml, F&& store) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < (kRows + kWarps - 1) / kWarps; ++h) {
      float t = l[h];
#pragma unroll
      for (int x = 16; x; x >>= 1) t += __shfl_xor_sync(~0u, t, x);
      if (lane == 0 && warp + kWarps * h < kRows) ml[warp + kWarps * h] = make_float2(m[h], t);
    }
    const int c4 = threadIdx.x % kC4, tg = threadIdx.x / kC4;
    const int rows = c.rows;
#pragma unroll
    for (int r0 = 0; r0 < kRows; r0 += 4) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<float4*>(sum + (tg * 4 + r) * DP + c4 * 4) = o[r0 + r];
      sync_compute();
      for (int e = threadIdx.x; e < 4 * kC4; e += kCompute) {
        const int r = e / kC4, col = e % kC4 * 4;
        if (r0 + r < rows && col < a.D) {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int g = 0; g < TG; ++g) {
            const float4 u = *reinterpret_cast<const float4*>(sum + (g * 4 + r) * DP + col);
            v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
          }
          store(r0 + r, col, v, ml[r0 + r].x, ml[r0 + r].y);
        }
      }
      sync_compute();
    }
  }
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

// The ring takes what the merge buffer leaves of 220 KB, at most 8 tiles.
template <class E>
struct Ring {
  static constexpr int kFit = (220 * 1024 - E::kMergeBytes) / static_cast<int>(E::kTileBytes);
  static constexpr int kSlots = kFit > 8 ? 8 : kFit;
  static constexpr int kSmem = kSlots * static_cast<int>(E::kTileBytes) + E::kMergeBytes;
};

// SPLIT: runs of the line of tiles (decode). Otherwise one unit a CTA (chunks).
template <class E, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, AttnArgs a,
                int boxes) {
  constexpr int NS = Ring<E>::kSlots;
  static_assert(NS >= 3, "ring");
  constexpr int KT = E::KT, R = E::kRows;
  extern __shared__ __align__(1024) unsigned char sm[];
  __shared__ uint64_t b_full[NS], b_empty[NS];
  __shared__ int64_t s_scan[kThreads / 32];
  __shared__ int64_t s_found[2];
  __shared__ float2 s_ml[kWarps * 16];
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
  float* merge = reinterpret_cast<float*>(sm + NS * E::kTileBytes);
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
    const int per = KT >> shift;
    RingPos rp;
    uint32_t n = 0;  // tiles issued
    const uint32_t most = a.copies;
    bool ok = true;
    while (ok && n < most) {
      const int tok = cp.sp.tile(cp.t) * KT + (lane << shift);
      bool need = lane < per && tok < cp.sp.end && (tok < a.sinks || tok + (1 << shift) > cp.sp.low);
      int page = 0;
      if (need) {
        page = __ldg(a.table + static_cast<int64_t>(cp.s.id) * a.max_pages + (tok >> a.page_shift));
        if (page < 0 || page >= a.n_pages) {
          atomicOr(a.err, MOE_DEVERR_BADIDX);
          need = false;
        }
      }
      const uint32_t box_bytes = (128u * E::NB) << shift;
      const uint32_t bytes = __popc(__ballot_sync(~0u, need)) * box_bytes;
      const int y = tok & ((1 << a.page_shift) - 1), z = page * a.Hkv + cp.h;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t full = su32(&b_full[rp.s]);
        if (n >= NS && !mbar_wait(su32(&b_empty[rp.s]), rp.ph ^ 1u, &s_abort, a.err, a.wait_cycles)) ok = false;
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(full, bytes);  // without pages the barrier completes by this arrival
        __syncwarp();
        if (need) {
          const uint32_t dst = ring + rp.s * E::kTileBytes + lane * box_bytes;
          for (int x = 0; x < boxes; ++x)
            tma_page(dst + x * (128u << shift), kv ? &map_v : &map_k, full, x * (128 / static_cast<int>(sizeof(typename E::T))),
                     y, z);
        }
        __syncwarp();
        ++n;
        rp.next(NS);
      }
      if (++cp.t < cp.t1) continue;
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
  if constexpr (sizeof(typename E::T) == 4)
    eng.place(merge);
  else
    eng.qs = su32(merge) + kWarps * 16 * 64 * 4;
  RingPos rp;
  Tile tile;
  tile.shift = shift;
  auto wait_tile = [&]() {
    mbar_wait(su32(&b_full[rp.s]), rp.ph, &s_abort, a.err, a.wait_cycles);
    tile.base = ring + rp.s * E::kTileBytes;
  };
  auto free_tile = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(su32(&b_empty[rp.s]));
    rp.next(NS);
  };
  while (true) {
    // ---- one unit's share of the run
    eng.begin(a, cp);
    for (; cp.t < cp.t1; ++cp.t) {
      wait_tile();
      eng.scores(a, cp, tile);
      free_tile();
      wait_tile();
      eng.values(a, cp, tile);
      free_tile();
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
  cudaError_t e = encoder();
  if (e != cudaSuccess) return e;
  CUtensorMap mk, mv;
  const int page = 1 << a.page_shift;
  const int64_t blocks = static_cast<int64_t>(a.n_pages) * a.Hkv;
  int boxes = 0;
  if ((e = map_page_cols(&mk, a.k, es, a.D, page, blocks, std::min(page, E::KT), E::NB, &boxes)) != cudaSuccess ||
      (e = map_page_cols(&mv, a.v, es, a.D, page, blocks, std::min(page, E::KT), E::NB, &boxes)) != cudaSuccess)
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

// f32: four rows a unit if that holds them all, else sixteen
template <int DP>
cudaError_t decode_f32(const AttnArgs& a, int num_sms, cudaStream_t st) {
  return a.n_q * a.g <= 4 ? decode_rows<FmaEngine<DP, 4>>(a, num_sms, st)
                          : decode_rows<FmaEngine<DP, 16>>(a, num_sms, st);
}

}  // namespace

cudaError_t launch_attn_decode(const AttnArgs& a, int32_t dtype, int num_sms, cudaStream_t st) {
  if (dtype == MOE_F32) {
    if (a.D <= 64) return decode_f32<64>(a, num_sms, st);
    if (a.D <= 128) return decode_f32<128>(a, num_sms, st);
    return decode_f32<256>(a, num_sms, st);
  }
  // the fewest row groups that hold the rows: more token groups per tile
  const int rows = a.n_q * a.g;
  if (a.D <= 64) {
    if (rows <= 16) return decode_rows<MmaEngine<64, 1, 128>>(a, num_sms, st);
    if (rows <= 32) return decode_rows<MmaEngine<64, 2, 128>>(a, num_sms, st);
    return decode_rows<MmaEngine<64, 4, 128>>(a, num_sms, st);
  }
  if (a.D <= 128) {
    if (rows <= 16) return decode_rows<MmaEngine<128, 1, 128>>(a, num_sms, st);
    if (rows <= 32) return decode_rows<MmaEngine<128, 2, 128>>(a, num_sms, st);
    return decode_rows<MmaEngine<128, 4, 128>>(a, num_sms, st);
  }
  if (rows <= 32) return decode_rows<MmaEngine<256, 2, 64>>(a, num_sms, st);
  return decode_rows<MmaEngine<256, 4, 64>>(a, num_sms, st);
}

cudaError_t launch_attn_prefill(const AttnArgs& a, int32_t dtype, int32_t n_rows, int num_sms, cudaStream_t st) {
  if (dtype == MOE_BF16 && a.D <= kTcHeadDim) return launch_attn_prefill_tc(a, num_sms, st);
  // every sequence has at most one partly filled row tile
  auto grid = [&](int rows) {
    return static_cast<int>(((static_cast<int64_t>(n_rows) * a.g + rows - 1) / rows + a.n) * a.Hkv);
  };
  if (dtype == MOE_F32) {
    if (a.D <= 64) return launch<FmaEngine<64, 16>, false>(a, grid(16), st);
    if (a.D <= 128) return launch<FmaEngine<128, 16>, false>(a, grid(16), st);
    return launch<FmaEngine<256, 16>, false>(a, grid(16), st);
  }
  return launch<MmaEngine<256, 4, 64>, false>(a, grid(64), st);
}

}  // namespace moe
