// Attention of prompt chunks over the paged cache on the 5th-generation tensor
// cores (bf16, head sizes up to 128; pages of bf16, or of 4-bit codes and heads of 64 or 128).
//
// A unit of work is 256 rows of one sequence and cache head, a row being a
// (token, head of the group) pair, so that K and V are read once for all the
// heads that share them. The rows are two tiles of 128; per tile of 128 tokens
//   S = Q K^T           128 x 128, fp32 in tensor memory
//   P = 2^(c S - c m)   row by row, one thread a row, rounded to bf16 and
//                       written back over S in tensor memory
//   O = O + P V         128 x D, fp32 in tensor memory, P from tensor memory
// with c = scale log2 e and m the row's running maximum. m is only raised (and
// O and the row's sum scaled) when the maximum has grown by more than 2^8
// since: numerators then stay below 2^8, which bf16 and fp32 hold as precisely
// as those below 1, and O is hardly ever read back.
//
// The two row tiles take turns on the tensor cores: while one's scores are
// exponentiated the other's products run. Order of the issuing thread:
//   QK0(0) QK1(0) | PV0(0) QK0(1) PV1(0) QK1(1) | PV0(1) QK0(2) ...
// These execute in order, so the barrier of a QK also says that the PV before
// it is done, and P may share S's columns. The time from S to the next S of a
// row tile is its softmax and its two products; the products of the other row
// tile fit into it. PV starts on the first 64 tokens while the numerators of
// the others are formed.
// Heads of at most 64 leave tensor memory for P beside S: the scores of the next
// tile are formed as soon as those of this one are in registers, in the order
//   QK0(j+1) PV0(j) QK1(j+1) PV1(j),
// and a row tile's time is that of its softmax alone.
//
// Warps: 0-3 and 4-7 softmax of row tiles 0 and 1, one thread a row (they also
// write the results), 8 TMA of K and V pages, 9 MMA issue, 10 and 11 load Q
// (each a row tile, one unit ahead: Q is free once the unit's last scores are
// formed) and check V.
// The V check: a token that only some rows see must not reach the others, but
// 0 * NaN is NaN in a matrix product. In tiles with such tokens the warps zero
// the tokens that no row sees, and infinities and NaN among the rest; if there
// was one, the rows that see it add numerator times value when the unit ends.
//
// Work split: the token tiles of all units form one line, cut into one equal
// run per CTA (one CTA per SM), as in the decode kernel: causal units differ in
// length, and whole units would leave SMs idle in the last wave. A unit counts
// unit_cost tiles more than it has, for its Q and its results. A unit cut by
// run ends leaves partial rows (m, l, O), joined in run order: up to four parts
// by the warp that arrives last, which hides behind the other CTAs' tiles (a
// launch for it costs 7 us of 88 on the windowed ragged prompts), more by a
// second small launch (a short chunk over a long cache has dozens: 64 tokens at
// 20,000, 4 cache heads, take 31 us so, 52 with the last warp).
//
// Pages of codes: a warp copies them into a ring by bulk copies and four warps make f16
// tiles of them, in the place of the TMA's. 2,048 tokens at 32,768, 16 heads / 2, of 128:
// 438 us, 1.22 PFLOP/s (bf16 pages: 330 to 350). Tensor cores 42% of the time: the conversion
// of a tile, which every CTA does for itself, and the softmax share the issue slots, and
// the roles' code together passes the instruction cache. Prompts of many short units pay
// for that at every unit, where Q and the results are waited for: 24 ragged prompts of up to
// 4,000 tokens, 16 heads / 4, of 128: 765 us, in a window of 1,024 621.
//
// Every wait is bounded, as in the prefill GEMMs: on a time-out all roles leave
// their loops, copies and MMAs in flight are drained, an error is recorded.
#include <cuda.h>
#include <cuda_fp16.h>

#include "attn.cuh"
#include "packed.cuh"
#include "pdl.cuh"
#include "prefill.h"
#include "tc.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr int kSoftWarps = 8;
constexpr int kKT = 128;      // tokens a tile
constexpr int kQT = 128;      // rows a row tile
constexpr int kUnitRows = 2 * kQT;
constexpr int kInlineParts = 4;  // parts of a unit joined without a launch
constexpr float kRaise = 8.f;  // log2 of the growth that raises m
// With f16 numerators, over pages of codes: they stay below 2^5 and are kept 2^10 times as large,
// so that f16 holds those from 2^-24 of the row's largest on as it does that one, and drops none
// above 2^-35. (With 8 and 7 the time is the same to 0.3%.)
constexpr float kRaiseCodes = 5.f;
constexpr int kLiftCodes = 10;

template <int DP, bool APART, bool CODES>
struct Cfg {
  // warps: after the softmax's, TMA, MMA and two of Q; or four of codes, MMA, two of Q and one that copies codes
  static constexpr int kThreads = CODES ? 512 : 384;
  static constexpr int kMmaWarp = CODES ? 12 : 9, kQWarp = CODES ? 13 : 10;
  static constexpr int kFillers = CODES ? 4 : 1;  // arrivals that fill a slot
  static constexpr uint32_t kHalf = kKT * 128;              // 64 columns of a tile: 128-byte rows
  static constexpr uint32_t kTile = kHalf * (DP / 64);      // a Q, K or V tile
  static constexpr int kKS = DP == 64 ? 4 : 2, kVS = DP == 64 ? 4 : (CODES ? 2 : 3);  // ring slots of K and V
  // codes: a tile's rows of codes, then its scales and offsets, and the ring of them
  static constexpr int kCodeRow = DP / 2, kMetaRow = DP / 16, kRaw = kKT * (kCodeRow + kMetaRow);
  static constexpr int kRS = !CODES ? 0 : (DP == 64 ? 6 : 3);
  static constexpr int kTiles = (2 + kKS + kVS) * static_cast<int>(kTile) + kRS * kRaw;
  // tensor memory columns: S0 S1 O0 O1, and where O leaves room for them, P0 P1
  static constexpr bool kApart = APART;
  static_assert(!APART || DP == 64, "columns");
  static constexpr uint32_t kTmemS = 0, kTmemO = 256;
  static constexpr uint32_t kTmemP = kApart ? 384 : kTmemS, kStrideP = kApart ? 64 : 128;
  // partial rows of one row tile: (m, l, -, -), then O by column quads
  static constexpr int64_t kPart = static_cast<int64_t>(kQT) * (DP + 4);
};

// Tiles' worth of time of a unit's Q and results. Without a window units run long
// and are cut more often, which counts as theirs (ragged prompts of up to 4,000
// tokens, heads of 64 and 128: 167 and 230 us with 3, 154 and 214 with 5, 157 and
// 220 with 7; in a window of 1,024 86 and 115 with 3, 90 and 119 with 5).
__host__ __device__ __forceinline__ int unit_cost(const AttnArgs& a) { return a.window > 0 ? 3 : 5; }

__device__ __forceinline__ void umma_ss(uint32_t dt, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(dt),
      "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
// Descriptor of an operand whose contiguous direction is its M or N direction
// (V: tokens x columns): 128-byte swizzle, blocks of 64 columns `lbo` bytes
// apart, groups of 8 tokens 1024 bytes apart.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr, uint32_t lbo) {
  uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFF) >> 4);
  d |= static_cast<uint64_t>(lbo >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
__device__ __forceinline__ void tma3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          dst),
      "l"(m), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// 32 columns of this warp's 32 lanes, without waiting
__device__ __forceinline__ void tmem_ld32_async(uint32_t ta, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
        "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
        "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]),
        "=f"(r[23]), "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]),
        "=f"(r[30]), "=f"(r[31])
      : "r"(ta));
}
__device__ __forceinline__ void tmem_ld16_async(uint32_t ta, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
        "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(ta));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// the n lowest bits; none for n <= 0, all for n >= 32
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : ~0u >> (32 - min(n, 32));
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred q; elect.sync _|q, 0xFFFFFFFF; selp.u32 %0, 1, 0, q; }" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// A CTA's walk along the line: units (sequence, row tile, cache head) in order,
// of each the tiles [t0, t0 + nt) that fall into the run. On the line a unit is
// `cost` positions and then one per tile.
struct Walk {
  int b, rt, h;
  int t0, nt;         // this segment
  int cost;
  int64_t unit0;      // line position of the unit
  int64_t end;        // end of the run
  Seq s;
  Span sp;
  int rows;           // rows of the unit
  __device__ __forceinline__ bool whole() const { return nt == sp.n; }
  __device__ __forceinline__ int64_t tiles0() const { return unit0 + cost; }
  __device__ __forceinline__ bool more() const { return tiles0() + sp.n + cost < end; }
};
// Shared memory behind the tiles.
template <int DP, bool APART, bool CODES>
struct Shared {
  using C = Cfg<DP, APART, CODES>;
  // kf/ke, vf/ve: full and empty slots of the rings; vr: V checked; qr, qe: Q
  // tile ready, free; sr: scores ready; sc: scores read (kApart); pa, pb:
  // numerators of the first and the last 64 tokens ready; pv: P read, O current
  // (kApart); of: O final
  uint64_t kf[C::kKS], ke[C::kKS], vf[C::kVS], ve[C::kVS], vr[C::kVS];
  uint64_t rf[6], re[6];  // codes: full and empty slots of their ring
  uint64_t qr[2], qe[2], sr[2], sc[2], pa[2], pb[2], pv[2], of[2], drain;
  int64_t scan[C::kThreads / 32];
  Walk walk;
  uint32_t poison[8];  // ring over units: number + 1 of the last one with infinities or NaN taken out of V
  uint32_t tmem;
  int abort;
  // codes: exponents of the powers of two taken out of the last tiles of K and V, by the
  // tile's number, and out of Q's rows, by the number of units in which the row tile had rows.
  // (By the number of all units its warp could pass by many that have rows in the other row
  // tile alone and take the place of powers that are still to be read.)
  struct Powers {
    int k, v;
  } powers[8];
  int8_t q_power[2][2][kQT];
  alignas(16) uint32_t fill_top[2][2][4];  // of a tile's K and V, by its number: the converting warps' largest values
};
template <int DP, bool APART, bool CODES>
constexpr int kSmem = Cfg<DP, APART, CODES>::kTiles + static_cast<int>(sizeof(Shared<DP, APART, CODES>));
static_assert(kSmem<128, false, true> <= 227 * 1024, "shared memory");

__device__ __forceinline__ int unit_count(const AttnArgs& a, int m) {
  return static_cast<int>((static_cast<int64_t>(m) * a.g + kUnitRows - 1) / kUnitRows);
}
__device__ __forceinline__ Span unit_span(const AttnArgs& a, const Seq& s, int rt) {
  const int64_t r0 = static_cast<int64_t>(rt) * kUnitRows, total = static_cast<int64_t>(s.m) * a.g;
  const int64_t r1 = min(r0 + kUnitRows, total) - 1;
  return span_of<kKT>(a, s, static_cast<int>(quotient(r0, a.g)), static_cast<int>(quotient(r1, a.g)) + 1);
}
// The segment from line position `at` (inside the unit) on.
__device__ __forceinline__ void open_unit(const AttnArgs& a, Walk& w, int64_t at) {
  w.sp = unit_span(a, w.s, w.rt);
  w.rows = static_cast<int>(min(static_cast<int64_t>(kUnitRows),
                                static_cast<int64_t>(w.s.m) * a.g - static_cast<int64_t>(w.rt) * kUnitRows));
  w.t0 = static_cast<int>(max(at - w.tiles0(), static_cast<int64_t>(0)));
  w.nt = static_cast<int>(min(w.end - w.tiles0(), static_cast<int64_t>(w.sp.n))) - w.t0;
}
// The next unit; only called while w.more(), so there is one with a tile.
__device__ __forceinline__ void next_segment(const AttnArgs& a, Walk& w) {
  w.unit0 = w.tiles0() + w.sp.n;
  if (++w.h == a.Hkv) {
    w.h = 0;
    if (++w.rt >= unit_count(a, w.s.m)) {
      w.rt = 0;
      do {
        ++w.b;
        if (w.b < a.n) w.s = load_seq(a, w.b);
      } while (w.b < a.n && w.s.m == 0);
    }
  }
  open_unit(a, w, w.unit0);
}

// Some rows of the unit see all or part of this tile's tokens and others do not.
// (Tiles of first tokens only are seen by every row after them.)
__device__ __forceinline__ bool mixed_tile(const AttnArgs& a, int tile0, int lo_pos, int hi_pos) {
  return tile0 + kKT - 1 > lo_pos || (a.window > 0 && hi_pos - tile0 >= a.window && tile0 + kKT > a.sinks);
}
// Position of the unit's first row; the last one's is sp.end - 1.
__device__ __forceinline__ int first_pos(const AttnArgs& a, const Walk& w) {
  return w.s.len - w.s.m + static_cast<int>(quotient(static_cast<int64_t>(w.rt) * kUnitRows, a.g));
}

// The infinities and NaN among the values of mixed tiles, which the matrix
// product has taken as zeros: numerator times value, added for the 32 columns
// from d0 of a row that sees them. m: the maximum that the row's numerators were
// formed with. A unit has about ten mixed tiles at most, whatever the context
// (1,024 tokens of 200,000, 16 heads of 128: 1.03 ms, with one NaN among the last
// 500 values 1.65, with NaN in all of the chunk's 7.6).
__device__ __noinline__ void add_nonfinite(const AttnArgs& a, const Walk& w, const __nv_bfloat16* q, int pos, float m,
                                           int d0, float* acc) {
  const float mc = m == -INFINITY ? 0.f : m * a.scale_log2;
  const int lo_pos = first_pos(a, w);
  const int32_t* row = a.table + static_cast<int64_t>(w.s.id) * a.max_pages;
  for (int t = w.t0; t < w.t0 + w.nt; ++t) {
    const int tile0 = w.sp.tile(t) * kKT;
    if (!mixed_tile(a, tile0, lo_pos, w.sp.end - 1)) continue;
    for (int j = tile0; j < tile0 + kKT; ++j) {
      const int back = pos - j;
      if (back < 0 || (a.window > 0 && back >= a.window && j >= a.sinks)) continue;
      const int p = __ldg(row + (j >> a.page_shift));
      if (p < 0 || p >= a.n_pages) continue;
      const int64_t tok =
          ((((static_cast<int64_t>(p) * a.Hkv + w.h) << a.page_shift) + (j & ((1 << a.page_shift) - 1)))) * a.D;
      const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + tok;
      bool bad = false;
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        if (d0 + i >= a.D) break;
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(v + d0 + i));
        bad |= nonfinite2(u.x) || nonfinite2(u.y) || nonfinite2(u.z) || nonfinite2(u.w);
      }
      if (!bad) continue;
      const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k) + tok;
      float s = 0.f;
      for (int d = 0; d < a.D; d += 8) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(q + d)), y = __ldg(reinterpret_cast<const uint4*>(k + d));
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s += __uint_as_float(xs[i] << 16) * __uint_as_float(ys[i] << 16) +
               __uint_as_float(xs[i] & 0xFFFF0000u) * __uint_as_float(ys[i] & 0xFFFF0000u);
      }
      const float e = ex2(s * a.scale_log2 - mc);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (d0 + i >= a.D) break;
        const float x = __bfloat162float(v[d0 + i]);
        if (!isfinite(x)) acc[i] += e * x;
      }
    }
  }
}

// A warp's 64 rows of 128 bytes: zeros in place of infinities and NaN.
__device__ __noinline__ void zero_nonfinite(uint32_t rows) {
#pragma unroll 1
  for (uint32_t at = rows + (threadIdx.x & 31) * 16u; at < rows + 8192u; at += 512u) {
    uint32_t v[4];
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(at)
                 : "memory");
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      if ((v[y] & 0x7F80u) == 0x7F80u) v[y] &= 0xFFFF0000u;
      if ((v[y] & 0x7F800000u) == 0x7F800000u) v[y] &= 0xFFFFu;
    }
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
  }
}

// ---- pages of 4-bit codes. A tile's values s q + b become f16, whose 11 bits keep
// what 8 of bf16 would not (keys rounded to bf16 put 0.25% of noise on every
// numerator: 3.4e-3 of the results' norm instead of 2.0e-3); Q and the numerators are
// f16 with them. f16's range is made up for by powers of two: a row of Q and a tile of K are
// divided by one that makes their largest value about 2^13, and the scores are multiplied by
// both. A unit's V is divided by one that makes its first tile's largest value about 2^11, and
// by a larger one from a tile on whose values would pass 2^15; O is kept in that unit. So a
// value (and the scale that it is formed with, a fifteenth of it or so) keeps its bits down to
// 2^-24 of the largest one beside it and is more than nothing down to 2^-34. Of the eight values of a
// word, nibbles i and i + 4 come out as a pair, so that columns lie in the order 0 4
// 1 5 2 6 3 7: Q is laid out the same, and results are put back as they are read.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void in_order(float* o, float f) {
#pragma unroll
  for (int x = 0; x < 32; x += 8) {
    float t[8];
#pragma unroll
    for (int y = 0; y < 8; ++y) t[y] = o[x + (y < 4 ? 2 * y : 2 * y - 7)] * f;
#pragma unroll
    for (int y = 0; y < 8; ++y) o[x + y] = t[y];
  }
}
// The exponent of what values are divided by: their largest one's, a float's upper nine bits, less
// what is left to it. (From -112 on all that fp32 holds as it is, 2^-126 and up, f16 does too.)
__device__ __forceinline__ int exponent_of(uint32_t top, int left) { return max(-112, static_cast<int>(top) - 127 - left); }
constexpr int kLeftQk = 13, kLeftV = 11, kRoomV = 3;
__device__ __forceinline__ bool finite_words(uint32_t m) { return !nonfinite2(m); }
__device__ __forceinline__ bool any_of_fillers(bool x) {
  uint32_t r;
  asm volatile("{ .reg .pred p, q; setp.ne.u32 p, %1, 0; bar.red.or.pred q, 2, 128, p; selp.u32 %0, 1, 0, q; }"
               : "=r"(r)
               : "r"(static_cast<uint32_t>(x))
               : "memory");
  return r != 0;
}

// One warp copies the codes of every tile of K and V, with their scales and offsets, into
// a ring: lane i those of page i of the tile.
template <int DP, class Sh>
__device__ __forceinline__ void copy_codes(const AttnArgs& a, Walk w, Sh& sh, uint32_t raw) {
  using C = typename Sh::C;
  const int lane = threadIdx.x & 31;
  const int boxr = min(1 << a.page_shift, kKT), per = kKT / boxr;
  volatile int* abort_flag = &sh.abort;
  RingPos rp;
  uint32_t n = 0;  // tiles of K and V copied
  bool ok = true;
  while (ok) {
    const int32_t* row = a.table + static_cast<int64_t>(w.s.id) * a.max_pages;
    for (int i = 0; i < w.nt && ok && n / 2 < a.copies; ++i) {
      const int tok = w.sp.tile(w.t0 + i) * kKT + lane * boxr;
      bool need = lane < per && tok < w.sp.end && (tok < a.sinks || tok + boxr > w.sp.low);
      int page = 0;
      if (need) {
        page = __ldg(row + (tok >> a.page_shift));
        if (page < 0 || page >= a.n_pages) {
          atomicOr(a.err, MOE_DEVERR_BADIDX);
          need = false;
        }
      }
      const uint32_t bytes = __popc(__ballot_sync(~0u, need)) * static_cast<uint32_t>(boxr * (C::kCodeRow + C::kMetaRow));
      const int y = tok & ((1 << a.page_shift) - 1);
      const int64_t block = ((static_cast<int64_t>(page) * a.Hkv + w.h) * (C::kCodeRow + C::kMetaRow)) << a.page_shift;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t full = su32(&sh.rf[rp.s]);
        if (n >= C::kRS && !mbar_wait(su32(&sh.re[rp.s]), rp.ph ^ 1u, abort_flag, a.err, a.wait_cycles)) ok = false;
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(full, bytes);  // without pages the barrier completes by this arrival
        __syncwarp();
        if (need) {
          const char* src = static_cast<const char*>(kv ? a.v : a.k) + block;
          const uint32_t dst = raw + rp.s * C::kRaw;
          bulk_copy(dst + lane * boxr * C::kCodeRow, src + y * C::kCodeRow, boxr * C::kCodeRow, full);
          bulk_copy(dst + kKT * C::kCodeRow + lane * boxr * C::kMetaRow,
                    src + (static_cast<int64_t>(C::kCodeRow) << a.page_shift) + y * C::kMetaRow, boxr * C::kMetaRow, full);
        }
        __syncwarp();
        ++n;
        rp.next(C::kRS);
      }
    }
    if (*abort_flag || n / 2 >= a.copies) ok = false;
    ok = __all_sync(~0u, ok) && w.more();
    if (ok) next_segment(a, w);
  }
  // drain: copies in flight land before the CTA ends
  if (lane == 0)
    for (uint32_t j = 0; j < n && j < C::kRS; ++j)
      mbar_drain(su32(&sh.rf[(n - 1 - j) % C::kRS]), ((n - 1 - j) / C::kRS) & 1u, a.err, kPrefillWaitCycles);
}

// Four warps turn the codes of every tile into K and V. The loops are kept short: all
// roles' code runs at once, and unrolled (loads to registers a tile ahead, 16 kB of
// instructions) the warps waited for instructions most of the time (2,048 tokens at 32K, 16
// heads of 128: 810 us; one piece of 16 bytes a turn 468, two 449; of 64: 370 and 418; a
// word of 4 bytes a turn 570; eight warps, which take issue slots of the softmax's: 539).
template <int DP, class Sh>
__device__ __forceinline__ void fill_tiles(const AttnArgs& a, Walk w, Sh& sh, uint32_t sk, uint32_t sv, uint32_t raw) {
  using C = typename Sh::C;
  constexpr int kPieces = DP / 32, kStep = 128 / kPieces, G = DP / 64;
  const int t = threadIdx.x - 256, lane = t & 31, piece = t % kPieces, row0 = t / kPieces;
  volatile int* abort_flag = &sh.abort;
  // Values of the raw tile at `src`, times f, into the slot at `dst`: a thread takes 16
  // bytes, 32 values, of every kStep-th token. Their four pieces of eight go out in an
  // order that differs between the halves of a head of 128, for the banks' sake.
  auto convert = [&](uint32_t src, uint32_t dst, float f) {
    uint32_t from = src + row0 * C::kCodeRow + piece * 16, meta = src + kKT * C::kCodeRow + row0 * C::kMetaRow + (piece >> 1) * 4;
    dst += (piece >> 1) * C::kHalf + row0 * 128u;
    const uint32_t turn = piece & 2, magic = in_register(0x64006400u);
    uint32_t c[4], m;
    auto read = [&]() {
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3]) : "r"(from));
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(m) : "r"(meta));
    };
    read();
#pragma unroll kPieces / 2
    for (int i = 0; i < kPieces; ++i) {
      const uint32_t word[4] = {turn ? c[2] : c[0], turn ? c[3] : c[1], turn ? c[0] : c[2], turn ? c[1] : c[3]};
      const __half2 s = __float2half2_rn(__uint_as_float(m << 16) * f);
      const __half2 b = __float2half2_rn(__uint_as_float(m & 0xFFFF0000u) * f);
      from += kStep * C::kCodeRow;
      meta += kStep * C::kMetaRow;
      if (i + 1 < kPieces) read();
      const uint32_t swz = (row0 + i * kStep) & 7;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        uint32_t o[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          // 1024 + q has q as its last bits, 1024 + 16 q as the four before: one shift a word
          const uint32_t at = z < 2 ? word[y] : word[y] >> 8;
          const uint32_t n = z & 1 ? and_or<0x00F000F0u>(at, magic) : and_or<0x000F000Fu>(at, magic);
          const __half2 h = *reinterpret_cast<const __half2*>(&n);
          const __half2 q = z & 1 ? __hfma2(h, __float2half2_rn(0.0625f), __float2half2_rn(-64.f)) : __hsub2(h, __float2half2_rn(1024.f));
          const __half2 val = __hfma2(q, s, b);
          o[z] = *reinterpret_cast<const uint32_t*>(&val);
        }
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst + ((((piece & 1) * 4 + (y ^ turn)) ^ swz) << 4)), "r"(o[0]),
                     "r"(o[1]), "r"(o[2]), "r"(o[3])
                     : "memory");
      }
      dst += kStep * 128;
    }
  };
  RingPos kp, vp, rp;
  uint32_t n = 0;  // tiles filled
  // The warps meet at barriers without a limit, so they leave together: one whose wait has
  // failed does no more work, but comes to the next tile's meeting, where all learn of it.
  bool ok = true;
  auto wait = [&](uint64_t* b, uint32_t ph) {
    ok = ok && mbar_wait(su32(b), ph, abort_flag, a.err, a.wait_cycles);
    ok = __all_sync(~0u, ok);
  };
  auto tell = [&](uint64_t* b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(su32(b));
  };
  for (uint32_t unit = 0;; ++unit) {
    const int lo_pos = first_pos(a, w), hi_pos = w.sp.end - 1;
    int ve = -1000;  // V's power of two so far
    for (int j = 0; j < w.nt; ++j) {
      RingPos next = rp;
      next.next(C::kRS);
      wait(&sh.rf[rp.s], rp.ph);
      wait(&sh.rf[next.s], next.ph);
      const uint32_t rk = raw + rp.s * C::kRaw, rv = raw + next.s * C::kRaw;
      if (ok) {
        // One thread a token looks at its scales and offsets.
        const int tile0 = w.sp.tile(w.t0 + j) * kKT, tok = tile0 + t;
        const bool seen = tok < w.sp.end && (tok < a.sinks || tok >= w.sp.low), mixed = mixed_tile(a, tile0, lo_pos, hi_pos);
        bool changed = false;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          float top = 0.f;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const uint32_t at = (kv ? rv : rk) + kKT * C::kCodeRow + t * C::kMetaRow + 4 * g;
            uint32_t m;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(m) : "r"(at));
            const float s = __uint_as_float(m << 16), b = __uint_as_float(m & 0xFFFF0000u);
            const bool fine = finite_words(m);
            // Tokens that no row sees become zeros. So do values that are infinite or NaN
            // in a tile with tokens that only some rows see; the rows that see them learn
            // of it at the unit's end.
            if (!seen || (kv && mixed && !fine)) {
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(0) : "memory");
              changed = true;
              if (seen) *const_cast<volatile uint32_t*>(&sh.poison[unit & 7]) = unit + 1;
            } else if (fine) {
              top = fmaxf(top, fminf(fmaxf(fabsf(b), fabsf(fmaf(15.f, s, b))), 3.3e38f));
            }
          }
          const uint32_t most = __reduce_max_sync(~0u, __float_as_uint(top));
          if (lane == 0) sh.fill_top[n & 1][kv][t >> 5] = most;
        }
        if (changed) fence_async_smem();  // these writes, before the slot's next copy
      }
      if (any_of_fillers(!ok)) return;
      // the tile's powers of two, the same in every thread. (The next tile's maxima have places of
      // their own, and the next but one's are written after the next meeting.)
      auto exponent = [&](int kv, int left) {
        const uint4 m = *reinterpret_cast<const uint4*>(sh.fill_top[n & 1][kv]);
        return exponent_of(max(max(m.x, m.y), max(m.z, m.w)) >> 23, left);
      };
      const int ke = exponent(0, kLeftQk), v_now = exponent(1, kLeftV);
      if (v_now > ve + kRoomV) ve = v_now;
      if (t == 0) {
        sh.powers[n & 7].k = ke;
        sh.powers[n & 7].v = ve;
      }
      if (n >= C::kKS) wait(&sh.ke[kp.s], kp.ph ^ 1u);
      if (ok) {
        convert(rk, sk + kp.s * C::kTile, two_to(-ke));
        fence_async_smem();
        tell(&sh.kf[kp.s]);
        tell(&sh.re[rp.s]);
      }
      kp.next(C::kKS);
      if (n >= C::kVS) wait(&sh.ve[vp.s], vp.ph ^ 1u);
      if (ok) {
        convert(rv, sv + vp.s * C::kTile, two_to(-ve));
        fence_async_smem();
        tell(&sh.vf[vp.s]);
        tell(&sh.re[next.s]);
      }
      vp.next(C::kVS);
      rp = next;
      rp.next(C::kRS);
      ++n;
    }
    if (!w.more()) return;
    next_segment(a, w);
  }
}

// A warp brings in Q of row tile t of every unit, as f16 in the columns' order, each row over
// its own power of two. Short loops here, too (24 ragged prompts of up to 4,000 tokens, heads of
// 128: 769 us; unrolled four times, four rows a turn 822; rows by way of registers 893).
template <int DP, class Sh>
__device__ __forceinline__ void convert_q(const AttnArgs& a, Walk w, Sh& sh, uint32_t sq, int t) {
  using C = typename Sh::C;
  constexpr int kPieces = DP / 8, kRowsPer = 32 / kPieces, kBatch = 2;
  const int lane = threadIdx.x & 31, p = lane % kPieces;
  volatile int* abort_flag = &sh.abort;
  uint32_t mine = 0;  // units in which this row tile had rows
  while (true) {
    if (t * kQT < w.rows) {
      if (mine > 0) {
        bool ok = mbar_wait(su32(&sh.qe[t]), (mine - 1) & 1u, abort_flag, a.err, a.wait_cycles);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
      }
      const int rows = w.rows - t * kQT;
      const int64_t rg = static_cast<int64_t>(w.rt) * kUnitRows + t * kQT + lane / kPieces;
      const int i = static_cast<int>(quotient(rg, a.g));
      int hq = static_cast<int>(rg - static_cast<int64_t>(i) * a.g);
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + (static_cast<int64_t>(w.s.row0) + i) * a.ldq +
                                 static_cast<int64_t>(w.h * a.g + hq) * a.D + p * 8;
      const int64_t step = kRowsPer * a.D, wrap = a.ldq - static_cast<int64_t>(a.g) * a.D;
      const uint32_t dst = sq + (p >> 3) * C::kHalf;
      auto at = [&](int r) { return dst + r * 128u + (((p & 7) ^ (r & 7)) << 4); };
#pragma unroll 1
      for (int r = lane / kPieces; r < kQT; r += kRowsPer) {  // rows past the end are zero
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at(r)), "l"(r < rows ? src : a.q), "r"(r < rows ? 16 : 0)
                     : "memory");
        src += step;  // the next row's head, or the next token's first ones
        hq += kRowsPer;
        while (hq >= a.g) {
          hq -= a.g;
          src += wrap;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      // in place: a lane's pieces are those that it has copied. (The scores of the unit before
      // are formed, so those of the one before that have been read, and their powers with them.)
      int8_t* power = sh.q_power[t][mine & 1];
#pragma unroll 1
      for (int r0 = lane / kPieces; r0 < kQT; r0 += kRowsPer * kBatch) {
        uint4 u[kBatch];
#pragma unroll
        for (int x = 0; x < kBatch; ++x)
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(u[x].x), "=r"(u[x].y), "=r"(u[x].z), "=r"(u[x].w)
                       : "r"(at(r0 + x * kRowsPer))
                       : "memory");
        // the rows' largest magnitudes, as bf16 bits, of two rows in a word. (With an infinity or
        // NaN in a row no score of it is finite, whatever the power.)
        uint32_t top[kBatch / 2];
#pragma unroll
        for (int x = 0; x < kBatch; x += 2) {
          auto most = [](uint4 q) {
            constexpr uint32_t kMagnitude = 0x7FFF7FFFu;
            return __vmaxu2(__vmaxu2(q.x & kMagnitude, q.y & kMagnitude), __vmaxu2(q.z & kMagnitude, q.w & kMagnitude));
          };
          const uint32_t m0 = most(u[x]), m1 = most(u[x + 1]);
          top[x / 2] = __vmaxu2(__byte_perm(m0, m1, 0x5410), __byte_perm(m0, m1, 0x7632));
        }
#pragma unroll
        for (int d = 1; d < kPieces; d <<= 1)
#pragma unroll
          for (int x = 0; x < kBatch / 2; ++x) top[x] = __vmaxu2(top[x], __shfl_xor_sync(~0u, top[x], d));
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          const int r = r0 + x * kRowsPer, e = exponent_of(x & 1 ? top[x / 2] >> 23 : (top[x / 2] & 0xFFFFu) >> 7, kLeftQk);
          const float f = two_to(-e);
          const uint32_t ws[4] = {u[x].x, u[x].y, u[x].z, u[x].w};
          float v[8];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            v[2 * y] = __uint_as_float(ws[y] << 16) * f;
            v[2 * y + 1] = __uint_as_float(ws[y] & 0xFFFF0000u) * f;
          }
          if (p == 0) power[r] = static_cast<int8_t>(e);
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at(r)), "r"(pack_f16(v[0], v[4])), "r"(pack_f16(v[1], v[5])),
                       "r"(pack_f16(v[2], v[6])), "r"(pack_f16(v[3], v[7]))
                       : "memory");
        }
      }
      ++mine;
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(su32(&sh.qr[t]));
    }
    if (!w.more()) break;
    next_segment(a, w);
  }
}

// The column groups of a row that the tokens it sees, in tiles with tokens that only
// some rows see, make NaN.
template <int DP>
__device__ __noinline__ uint32_t lost_groups(const AttnArgs& a, const Walk& w, int pos) {
  uint32_t lost = 0;
  const int lo_pos = first_pos(a, w);
  const int32_t* row = a.table + static_cast<int64_t>(w.s.id) * a.max_pages;
  for (int t = w.t0; t < w.t0 + w.nt; ++t) {
    const int tile0 = w.sp.tile(t) * kKT;
    if (!mixed_tile(a, tile0, lo_pos, w.sp.end - 1)) continue;
    for (int j = tile0; j < tile0 + kKT; ++j) {
      const int back = pos - j;
      if (back < 0 || (a.window > 0 && back >= a.window && j >= a.sinks)) continue;
      const int p = __ldg(row + (j >> a.page_shift));
      if (p < 0 || p >= a.n_pages) continue;
      const char* block = static_cast<const char*>(a.v) + (((static_cast<int64_t>(p) * a.Hkv + w.h) * (DP / 2 + DP / 16)) << a.page_shift);
      const char* meta = block + (static_cast<int64_t>(DP / 2) << a.page_shift) + (j & ((1 << a.page_shift) - 1)) * (DP / 16);
#pragma unroll
      for (int g = 0; g < DP / 64; ++g)
        if (!finite_words(__ldg(reinterpret_cast<const uint32_t*>(meta + 4 * g)))) lost |= 1u << g;
    }
  }
  return lost;
}

template <int DP, bool APART, bool CODES>
__global__ void __launch_bounds__(Cfg<DP, APART, CODES>::kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, AttnArgs a) {
  const long long wait_cycles = a.wait_cycles;
  using C = Cfg<DP, APART, CODES>;
  constexpr int kThreads = C::kThreads;
  extern __shared__ __align__(1024) unsigned char smraw[];
  const uint32_t sbase = su32(smraw);
  if (sbase & 1023u) {  // the swizzle's pattern starts at such a boundary
    if (threadIdx.x == 0) atomicOr(a.err, MOE_DEVERR_TIMEOUT);
    return;
  }
  const uint32_t sq = sbase, sk = sbase + 2 * C::kTile, sv = sk + C::kKS * C::kTile;
  using Sh = Shared<DP, APART, CODES>;
  Sh& sh = *reinterpret_cast<Sh*>(smraw + C::kTiles);
  int* const s_first = reinterpret_cast<int*>(smraw);  // before the tiles are in use
  volatile int* abort_flag = &sh.abort;
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;

  pdl_trigger();  // the joining launch may be scheduled; it waits for this one's end
  if (tid == 0) a.cuts[blockIdx.x].count = 0;
  if (blockIdx.x == 0 && tid == kThreads - 1) check_chunks(a);

  // ---- this CTA's run. Units are counted sequence block by sequence block;
  // a unit's length follows from its last token's position.
  auto scan = [&](int64_t v, int64_t* total) -> int64_t {  // exclusive prefix over the block
    int64_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(~0u, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) sh.scan[warp] = x;
    __syncthreads();
    int64_t base = 0, all = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) base += sh.scan[i];
      all += sh.scan[i];
    }
    __syncthreads();
    *total = all;
    return base + x - v;
  };
  // visit(b, rt, span length, line position) for every unit row, in parallel;
  // strips: rounds it took
  int strips = 0;
  const int cost = unit_cost(a);
  auto visit_units = [&](auto&& f) -> int64_t {
    int64_t line = 0;
    strips = 0;
    for (int b0 = 0; b0 < a.n; b0 += kThreads) {
      const int b = b0 + tid;
      int64_t units;
      const int64_t mine = b < a.n ? unit_count(a, chunk_rows(a, b)) : 0;
      const int64_t first = scan(mine, &units);
      s_first[tid] = static_cast<int>(first);
      __syncthreads();
      for (int64_t u0 = 0; u0 < units; u0 += kThreads) {
        const int64_t u = u0 + tid;
        int n = 0, sb = 0, rt = 0;
        if (u < units) {
          int lo = 0, hi = min(kThreads, a.n - b0);
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_first[mid] <= u)
              lo = mid;
            else
              hi = mid;
          }
          sb = b0 + lo;
          rt = static_cast<int>(u - s_first[lo]);
          n = unit_span(a, load_seq(a, sb), rt).n;
        }
        int64_t all;
        const int64_t at = line + scan(u < units ? static_cast<int64_t>(n + cost) * a.Hkv : 0, &all);
        if (n > 0) f(sb, rt, n, at);
        line += all;
        ++strips;
      }
      __syncthreads();
    }
    return line;
  };
  int my_b = 0, my_rt = 0, my_n = 0;  // this thread's unit row of the last round
  int64_t my_at = 0;
  const int64_t total = visit_units([&](int b, int rt, int n, int64_t at) {
    my_b = b;
    my_rt = rt;
    my_n = n;
    my_at = at;
  });
  if (total == 0) return;
  const Runs runs(total, gridDim.x);
  if (blockIdx.x >= runs.n) return;
  const int64_t run0 = runs.start(blockIdx.x), run1 = runs.start(blockIdx.x + 1);
  if (tid == 0) sh.walk.nt = 0;
  __syncthreads();
  auto start_in = [&](int b, int rt, int n, int64_t at) {  // if the run starts in this unit row
    const int64_t per = n + cost;
    if (run0 >= at && run0 < at + per * a.Hkv) {
      Walk w;
      w.cost = cost;
      w.b = b;
      w.rt = rt;
      w.h = static_cast<int>(quotient(run0 - at, per));
      w.unit0 = at + w.h * per;
      w.end = run1;
      w.s = load_seq(a, b);
      open_unit(a, w, run0);
      sh.walk = w;
    }
  };
  if (strips > 1) {
    visit_units(start_in);
  } else {  // every unit row is still some thread's
    if (my_n > 0) start_in(my_b, my_rt, my_n, my_at);
    __syncthreads();
  }
  if (sh.walk.nt <= 0) return;  // a run within a unit's fixed cost

  if (tid == 0) {
    sh.abort = 0;
    for (int i = 0; i < C::kKS; ++i) {
      mbar_init(su32(&sh.kf[i]), C::kFillers);
      mbar_init(su32(&sh.ke[i]), 1);
    }
    for (int i = 0; i < C::kVS; ++i) {
      mbar_init(su32(&sh.vf[i]), C::kFillers);
      mbar_init(su32(&sh.ve[i]), 1);
      mbar_init(su32(&sh.vr[i]), 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(su32(&sh.qr[t]), 1);
      mbar_init(su32(&sh.qe[t]), 1);
      mbar_init(su32(&sh.sr[t]), 1);
      mbar_init(su32(&sh.sc[t]), kSoftWarps / 2);
      mbar_init(su32(&sh.pv[t]), 1);
      mbar_init(su32(&sh.pa[t]), kSoftWarps / 2);
      mbar_init(su32(&sh.pb[t]), kSoftWarps / 2);
      mbar_init(su32(&sh.of[t]), 1);
    }
    mbar_init(su32(&sh.drain), 1);
    for (int i = 0; i < C::kRS; ++i) {
      mbar_init(su32(&sh.rf[i]), 1);
      mbar_init(su32(&sh.re[i]), C::kFillers);
    }
    for (int i = 0; i < 8; ++i) sh.poison[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == C::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&sh.tmem)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sh.tmem;
  Walk w = sh.walk;

  // Codes: the block is launched with 512 x 128 registers; the softmax's warpgroups
  // take 168 a thread, the others keep 88 (256 x 168 + 256 x 88 = 512 x 128).
  if (CODES && warp >= 8 && warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    fill_tiles<DP>(a, w, sh, sk, sv, sv + C::kVS * C::kTile);
  } else if (!CODES && warp == 8) {
    // ---------------- TMA: lane i copies page i of the tile (its 64-column
    // halves); pages that no row sees are left out
    const int boxr = min(1 << a.page_shift, kKT), per = kKT / boxr;
    RingPos kp, vp;
    uint32_t nk = 0, nv = 0;  // tiles issued
    const uint32_t most = a.copies;
    bool ok = true;
    while (ok) {
      const int32_t* row = a.table + static_cast<int64_t>(w.s.id) * a.max_pages;
      for (int i = 0; i < w.nt && ok && nk < most; ++i) {
        const int tok = w.sp.tile(w.t0 + i) * kKT + lane * boxr;
        bool need = lane < per && tok < w.sp.end && (tok < a.sinks || tok + boxr > w.sp.low);
        int page = 0;
        if (need) {
          page = __ldg(row + (tok >> a.page_shift));
          if (page < 0 || page >= a.n_pages) {
            atomicOr(a.err, MOE_DEVERR_BADIDX);
            need = false;
          }
        }
        const uint32_t bytes = __popc(__ballot_sync(~0u, need)) * static_cast<uint32_t>(boxr) * 128u * (DP / 64);
        const int y = tok & ((1 << a.page_shift) - 1), z = page * a.Hkv + w.h;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          RingPos& rp = kv ? vp : kp;
          uint32_t& n = kv ? nv : nk;
          const uint32_t slots = kv ? C::kVS : C::kKS;
          const uint32_t full = su32(kv ? &sh.vf[rp.s] : &sh.kf[rp.s]);
          if (n >= slots && !mbar_wait(su32(kv ? &sh.ve[rp.s] : &sh.ke[rp.s]), rp.ph ^ 1u, abort_flag, a.err, wait_cycles))
            ok = false;
          ok = __all_sync(~0u, ok);
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(full, bytes);  // without pages the barrier completes by this arrival
          __syncwarp();
          if (need) {
            const uint32_t dst = (kv ? sv : sk) + rp.s * C::kTile + lane * boxr * 128u;
#pragma unroll
            for (int hf = 0; hf < DP / 64; ++hf) tma3d(dst + hf * C::kHalf, kv ? &map_v : &map_k, full, hf * 64, y, z);
          }
          __syncwarp();
          ++n;
          rp.next(slots);
        }
      }
      if (*abort_flag || nk >= most) ok = false;
      ok = __all_sync(~0u, ok) && w.more();
      if (ok) next_segment(a, w);
    }
    // drain: copies in flight land before the CTA ends
    if (lane == 0) {
      for (uint32_t j = 0; j < nk && j < C::kKS; ++j)
        mbar_drain(su32(&sh.kf[(nk - 1 - j) % C::kKS]), ((nk - 1 - j) / C::kKS) & 1u, a.err, kPrefillWaitCycles);
      for (uint32_t j = 0; j < nv && j < C::kVS; ++j)
        mbar_drain(su32(&sh.vf[(nv - 1 - j) % C::kVS]), ((nv - 1 - j) / C::kVS) & 1u, a.err, kPrefillWaitCycles);
    }
  } else if (CODES ? warp >= C::kMmaWarp : warp == C::kMmaWarp) {
    // ---------------- MMA issue, by one elected thread: elect.sync under a
    // branch that is uniform in the warp lets the compiler keep descriptors in
    // uniform registers. (A lane comparison does not: 100 cycles an MMA. The
    // tensor cores take 73 cycles for 128 x 128 x 16 with A in tensor memory and
    // 105 with A in shared memory.)
    // (With codes the warpgroup's other warps are here too, as it lowers its registers in one instruction.)
    if (CODES) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (CODES && warp >= C::kQWarp) {
      if (warp < C::kQWarp + 2)
        convert_q<DP>(a, w, sh, sq + (warp - C::kQWarp) * C::kTile, warp - C::kQWarp);
      else
        copy_codes<DP>(a, w, sh, sv + C::kVS * C::kTile);
    } else if (elect_one()) {
      constexpr uint32_t kOperands = CODES ? 0u : (1u << 7) | (1u << 10);  // f16 or bf16
      const uint32_t id_qk = (1u << 4) | kOperands | ((kKT >> 3) << 17) | ((kQT >> 4) << 24);
      const uint32_t id_pv = (1u << 4) | kOperands | (1u << 16) | ((DP >> 3) << 17) | ((kQT >> 4) << 24);
      RingPos kp, vp;
      uint32_t q_ph = 0;            // units seen by row tile 0; tile 1 counts its own
      uint32_t q_ph1 = 0;
      uint32_t p_ph[2] = {0, 0};
      bool ok = true;
      auto wait = [&](uint64_t* b, uint32_t ph) { return mbar_wait(su32(b), ph, abort_flag, a.err, wait_cycles); };
      auto qk = [&](int t) {
        const uint64_t qa = sdesc(sq + t * C::kTile), kb = sdesc(sk + kp.s * C::kTile);
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const uint32_t off = (k >> 2) * (C::kHalf >> 4) + (k & 3) * 2;
          umma_ss(tmem + C::kTmemS + t * 128u, qa + off, kb + off, id_qk, k > 0);
        }
        umma_commit(su32(&sh.sr[t]));
      };
      // O += P V of tile j of the unit
      auto pv = [&](int t, int j) -> bool {
        const uint64_t vb = sdesc_mn(sv + vp.s * C::kTile, C::kHalf);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          if (!wait(hf ? &sh.pb[t] : &sh.pa[t], p_ph[t])) return false;
          fence_after();
#pragma unroll
          for (int k = 4 * hf; k < 4 * hf + 4; ++k)
            umma_ts(tmem + C::kTmemO + t * static_cast<uint32_t>(DP), tmem + C::kTmemP + t * C::kStrideP + 8u * k,
                    vb + k * (2048u >> 4), id_pv, k > 0 || j > 0);
        }
        p_ph[t] ^= 1u;
        if (C::kApart) umma_commit(su32(&sh.pv[t]));
        return true;
      };
      uint32_t s_n[2] = {0, 0};  // scores formed (kApart)
      auto scores_read = [&](int t) -> bool {
        if (!C::kApart) return true;
        const uint32_t n = s_n[t]++;
        return n == 0 || wait(&sh.sc[t], (n - 1) & 1u);
      };
      while (ok) {
        const int nq = w.rows > kQT ? 2 : 1;
        if (!(ok = wait(&sh.kf[kp.s], kp.ph))) break;
        for (int t = 0; t < nq && ok; ++t) {
          uint32_t& ph = t ? q_ph1 : q_ph;
          if (!(ok = wait(&sh.qr[t], ph) && scores_read(t))) break;
          ph ^= 1u;
          fence_after();
          qk(t);
          if (w.nt == 1) umma_commit(su32(&sh.qe[t]));
        }
        if (!ok) break;
        umma_commit(su32(&sh.ke[kp.s]));
        kp.next(C::kKS);
        for (int j = 0; j < w.nt && ok; ++j) {
          const bool more = j + 1 < w.nt;
          for (int t = 0; t < nq; ++t) {
            // (kApart: first the scores of the next tile, which need only this one's to be in registers)
            if (C::kApart && more) {
              if (t == 0 && !(ok = wait(&sh.kf[kp.s], kp.ph))) break;
              if (!(ok = scores_read(t))) break;
              fence_after();
              qk(t);
              if (j + 2 == w.nt) umma_commit(su32(&sh.qe[t]));
            }
            if (t == 0 && !(ok = wait(CODES ? &sh.vf[vp.s] : &sh.vr[vp.s], vp.ph))) break;
            if (CODES) fence_after();
            if (!(ok = pv(t, j))) break;
            if (!more) {
              umma_commit(su32(&sh.of[t]));
            } else if (!C::kApart) {
              if (t == 0 && !(ok = wait(&sh.kf[kp.s], kp.ph))) break;
              qk(t);
              if (j + 2 == w.nt) umma_commit(su32(&sh.qe[t]));
            }
          }
          if (!ok) break;
          umma_commit(su32(&sh.ve[vp.s]));
          vp.next(C::kVS);
          if (more) {
            umma_commit(su32(&sh.ke[kp.s]));
            kp.next(C::kKS);
          }
        }
        if (!ok || !w.more() || *abort_flag) break;
        next_segment(a, w);
      }
      // drain: every MMA issued here is done before tensor memory is released
      umma_commit(su32(&sh.drain));
      mbar_drain(su32(&sh.drain), 0, a.err, kPrefillWaitCycles);
    }
  } else if (!CODES && warp >= C::kQWarp) {
    // ---------------- Q of row tile t, and the check of half of every V tile
    const int t = warp - C::kQWarp;
    RingPos vp;
    uint32_t qe_ph = 0;
    bool ok = true, q_used = false;
    for (uint32_t unit = 0; ok; ++unit) {
      if (t * kQT < w.rows) {
        if (q_used) {
          ok = mbar_wait(su32(&sh.qe[t]), qe_ph, abort_flag, a.err, wait_cycles);
          ok = __all_sync(~0u, ok);
          if (!ok) break;
          qe_ph ^= 1u;
        }
        q_used = true;
        // 16-byte pieces, swizzled as TMA would; rows and columns past the end are zero
        constexpr int kPieces = DP / 8, kRowsPer = 32 / kPieces;
        const int p = lane % kPieces, rows = w.rows - t * kQT;
        const int64_t rg = static_cast<int64_t>(w.rt) * kUnitRows + t * kQT + lane / kPieces;
        const int i = static_cast<int>(quotient(rg, a.g));
        int hq = static_cast<int>(rg - static_cast<int64_t>(i) * a.g);
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + (static_cast<int64_t>(w.s.row0) + i) * a.ldq +
                                   static_cast<int64_t>(w.h * a.g + hq) * a.D + p * 8;
        const int64_t step = kRowsPer * a.D, wrap = a.ldq - static_cast<int64_t>(a.g) * a.D;
        const bool col_in = p * 8 < a.D;
        uint32_t dst = sq + t * C::kTile + (p >> 3) * C::kHalf;
#pragma unroll 4
        for (int r = lane / kPieces; r < kQT; r += kRowsPer) {
          const bool in = col_in && r < rows;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + r * 128u + (((p & 7) ^ (r & 7)) << 4)),
                       "l"(in ? src : a.q), "r"(in ? 16 : 0)
                       : "memory");
          src += step;  // the next row's head, or the next token's first ones
          hq += kRowsPer;
          while (hq >= a.g) {
            hq -= a.g;
            src += wrap;
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(su32(&sh.qr[t]));
      }
      const int lo_pos = first_pos(a, w), hi_pos = w.sp.end - 1;
      for (int i = 0; i < w.nt; ++i) {
        ok = mbar_wait(su32(&sh.vf[vp.s]), vp.ph, abort_flag, a.err, wait_cycles);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        const int tile0 = w.sp.tile(w.t0 + i) * kKT;
        if (mixed_tile(a, tile0, lo_pos, hi_pos)) {
          const uint32_t st = sv + vp.s * C::kTile;
          bool bad = false;
          // this warp's 64 tokens: 8 pieces a row of 128 bytes, column halves one after the other
#pragma unroll 1
          for (int hf = 0; hf < DP / 64; ++hf) {
#pragma unroll 8
            for (int e = lane; e < 64 * 8; e += 32) {
              const int j = tile0 + t * 64 + (e >> 3);
              const uint32_t at = st + hf * C::kHalf + t * 8192u + e * 16u;
              if (j >= w.sp.end || (j >= a.sinks && j < w.sp.low)) {
                asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(at), "r"(0) : "memory");
              } else {
                uint32_t v[4];
                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                             : "r"(at));
                bad |= nonfinite2(v[0]) || nonfinite2(v[1]) || nonfinite2(v[2]) || nonfinite2(v[3]);
              }
            }
          }
          if (__any_sync(~0u, bad)) {
            // zeros in their place; the rows that see them add them at the end of the unit
            for (int hf = 0; hf < DP / 64; ++hf) zero_nonfinite(st + hf * C::kHalf + t * 8192u);
            if (lane == 0) *const_cast<volatile uint32_t*>(&sh.poison[unit & 7]) = unit + 1;
          }
          fence_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(su32(&sh.vr[vp.s]));
        vp.next(C::kVS);
      }
      if (!ok || !w.more()) break;
      next_segment(a, w);
    }
  } else {
    // ---------------- softmax: one thread a row
    if (CODES) asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    const int t = warp >> 2, r = (warp & 3) * 32 + lane;  // row tile, row
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + C::kTmemS + t * 128u + lanes, tp = tmem + C::kTmemP + t * C::kStrideP + lanes;
    const uint32_t to = tmem + C::kTmemO + t * static_cast<uint32_t>(DP) + lanes;
    // (codes: maxima are in units of log2, as a score's unit differs from tile to tile)
    const float c = CODES ? 1.f : a.scale_log2, raise = (CODES ? kRaiseCodes : kRaise) / c;
    uint32_t s_ph = 0, o_ph = 0, p_n = 0;  // p_n: numerators written (kApart)
    uint32_t tile_n = 0, mine = 0;         // tiles before this unit's, and units in which this row tile had rows
    bool ok = true;
    for (uint32_t unit = 0; ok; ++unit) {
      if (t * kQT < w.rows) {
        const bool row_ok = t * kQT + r < w.rows;
        const int64_t rg = static_cast<int64_t>(w.rt) * kUnitRows + t * kQT + r;
        const int qi = static_cast<int>(quotient(rg, a.g));
        const int pos = row_ok ? w.s.len - w.s.m + qi : -1;
        // positions of the warp's rows, for the tiles that need no mask
        const int lo_pos = w.s.len - w.s.m + static_cast<int>(quotient(rg - lane, a.g));
        const int64_t r_last = min(rg - lane + 31, static_cast<int64_t>(w.s.m) * a.g - 1);
        const int hi_pos = w.s.len - w.s.m + static_cast<int>(quotient(r_last, a.g));
        float m = -INFINITY, thr = -INFINITY, l = 0.f;  // thr: a maximum above it raises m
        int o_exp = 0;                                  // codes: O is kept divided by 2^o_exp
        for (int j = 0; j < w.nt; ++j) {
          ok = mbar_wait(su32(&sh.sr[t]), s_ph, abort_flag, a.err, wait_cycles);
          ok = __all_sync(~0u, ok);
          if (!ok) break;
          s_ph ^= 1u;
          fence_after();
          const int tile0 = w.sp.tile(w.t0 + j) * kKT;
          const bool edge = tile0 + kKT - 1 > lo_pos || (a.window > 0 && hi_pos - tile0 >= a.window);
          const int last = pos - tile0;                              // columns after it are hidden
          const int from = a.window > 0 ? last - a.window + 1 : -1;  // columns before it are hidden, but for
          const int keep = a.sinks - tile0;                          // the first `keep`
          float s[128];
          auto hide = [&](int x) {  // bit y of see: column x + y is visible
            const uint32_t see = low_bits(last + 1 - x) & (~low_bits(from - x) | low_bits(keep - x));
            if (__all_sync(~0u, see == ~0u)) return;
#pragma unroll
            for (int y = 0; y < 32; ++y) s[x + y] = (see >> y) & 1u ? s[x + y] : -INFINITY;
          };
          float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
          auto top = [&](int x) {
#pragma unroll
            for (int y = x; y < x + 64; y += 8) {
              mx0 = max3(mx0, s[y], s[y + 1]);
              mx1 = max3(mx1, s[y + 2], s[y + 3]);
              mx2 = max3(mx2, s[y + 4], s[y + 5]);
              mx3 = max3(mx3, s[y + 6], s[y + 7]);
            }
          };
#pragma unroll
          for (int x = 0; x < 128; x += 32) tmem_ld32_async(ts + x, s + x);
          float cj = c;  // codes: a score's factor, from the powers of two of its tile of K and of Q
          int v_exp = 0;
          if constexpr (CODES) {
            const volatile Sh& vs = sh;
            cj = score_factor(a.scale_log2, vs.q_power[t][mine & 1][r] + vs.powers[(tile_n + j) & 7].k);
            v_exp = vs.powers[(tile_n + j) & 7].v;
          }
          tmem_wait_ld();
          if (C::kApart) {
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(su32(&sh.sc[t]));
          }
          if (edge) {
            hide(0);
            hide(32);
            hide(64);
            hide(96);
          }
          top(0);
          top(64);
          float mx = max3(fmaxf(mx0, mx1), mx2, mx3);
          if constexpr (CODES) mx *= cj;
          if (C::kApart && p_n++ > 0) {  // the product of the tile before has read P and brought O up to date
            ok = mbar_wait(su32(&sh.pv[t]), p_n & 1u, abort_flag, a.err, wait_cycles);
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            fence_after();
          }
          const bool up = mx > thr;
          if (__any_sync(~0u, up) || (CODES && v_exp != o_exp)) {
            const float mn = up ? mx : m;
            float f = up ? ex2((m - mn) * c) : 1.f;  // 0 for the first maximum
            m = mn;
            thr = up ? m + raise : thr;
            l *= f;
            if (CODES && v_exp != o_exp) {  // O's unit grows with its values'
              f *= exp2f(static_cast<float>(o_exp - v_exp));
              o_exp = v_exp;
            }
            if (j > 0) {
#pragma unroll 1
              for (int x = 0; x < DP; x += 16) {
                float o[16];
                tmem_ld16_async(to + x, o);
                tmem_wait_ld();
                uint32_t u[16];
#pragma unroll
                for (int y = 0; y < 16; ++y) u[y] = __float_as_uint(o[y] * f);
                tmem_st16(to + x, u);
              }
            }
          }
          const float mc = (m == -INFINITY ? 0.f : m * c) - (CODES ? kLiftCodes : 0.f);
          const F2 c2 = f2(cj, cj), m2 = f2(-mc, -mc);
          F2 l0 = 0ull, l1 = 0ull;
#pragma unroll
          for (int x = 0; x < 128; x += 32) {
            uint32_t p[16];
#pragma unroll
            for (int y = 0; y < 32; y += 4) {
              const float2 u = both(fma2(f2(s[x + y], s[x + y + 1]), c2, m2));
              const float2 v = both(fma2(f2(s[x + y + 2], s[x + y + 3]), c2, m2));
              const float e0 = ex2(u.x), e1 = ex2(u.y), e2 = ex2(v.x), e3 = ex2(v.y);
              // the sum takes the numerators before their rounding to bf16
              l0 = add2(l0, f2(e0, e1));
              l1 = add2(l1, f2(e2, e3));
              p[y / 2] = CODES ? pack_f16(e0, e1) : pack_bf16(e0, e1);
              p[y / 2 + 1] = CODES ? pack_f16(e2, e3) : pack_bf16(e2, e3);
            }
            if (x == 64) {  // the first half is in place by now
              tmem_wait_st();
              fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(su32(&sh.pa[t]));
            }
            tmem_st16(tp + x / 2, p);  // (over scores that have been read, where P has no columns of its own)
          }
          tmem_wait_st();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(su32(&sh.pb[t]));
          const float2 la = both(add2(l0, l1));
          l += la.x + la.y;
        }
        if (!ok) break;
        ok = mbar_wait(su32(&sh.of[t]), o_ph, abort_flag, a.err, wait_cycles);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        o_ph ^= 1u;
        fence_after();
        const int hq = w.h * a.g + static_cast<int>(rg - static_cast<int64_t>(qi) * a.g);
        const int64_t row = static_cast<int64_t>(w.s.row0) + qi;
        // (A later number has taken the place of this unit's, if it had one: then there is
        // nothing to find at worst.)
        const bool poisoned =
            __any_sync(~0u, static_cast<int>(*const_cast<volatile uint32_t*>(&sh.poison[unit & 7]) - (unit + 1)) >= 0);
        // codes: the groups of 64 columns that a visible token's scale or offset makes NaN
        const uint32_t lost = CODES && poisoned ? lost_groups<DP>(a, w, pos) : 0u;
        if (!CODES && poisoned) {
          const Walk seg = w;
          const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + row * a.ldq + static_cast<int64_t>(hq) * a.D;
#pragma unroll 1
          for (int x = 0; x < DP; x += 32) {
            float o[32];
            tmem_ld32_async(to + x, o);
            tmem_wait_ld();
            if (pos >= 0) add_nonfinite(a, seg, q, pos, m, x, o);
            __syncwarp();
            uint32_t u[32];
#pragma unroll
            for (int y = 0; y < 32; ++y) u[y] = __float_as_uint(o[y]);
            tmem_st16(to + x, u);
            tmem_st16(to + x + 16, u + 16);
          }
          tmem_wait_st();
        }
        // ---- results of the segment
        const bool seen = pos >= 0;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row * a.ldo + static_cast<int64_t>(hq) * a.D;
        auto store32 = [&](const float* o, float f, int x) {
          if (!row_ok) return;
          uint32_t v[16];
#pragma unroll
          for (int y = 0; y < 16; ++y) v[y] = pack_bf16(seen ? o[2 * y] * f : 0.f, seen ? o[2 * y + 1] * f : 0.f);
#pragma unroll
          for (int y = 0; y < 16; y += 8) {
            if (x + 2 * y >= a.D) break;
            if (a.wide_out) {  // a sector a thread
              asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(out + x + 2 * y), "r"(v[y]),
                           "r"(v[y + 1]), "r"(v[y + 2]), "r"(v[y + 3]), "r"(v[y + 4]), "r"(v[y + 5]), "r"(v[y + 6]),
                           "r"(v[y + 7])
                           : "memory");
            } else {
              *reinterpret_cast<uint4*>(out + x + 2 * y) = make_uint4(v[y], v[y + 1], v[y + 2], v[y + 3]);
              if (x + 2 * y + 8 < a.D)
                *reinterpret_cast<uint4*>(out + x + 2 * y + 8) = make_uint4(v[y + 4], v[y + 5], v[y + 6], v[y + 7]);
            }
          }
        };
        const bool whole = w.whole();
        // a partial result: slot 0 if the run starts inside the unit's tiles, else
        // 1; (m, l, -, -) of every row, then O by column quads
        if (CODES) l *= two_to(-kLiftCodes);
        float* part = a.part + ((2 * static_cast<int64_t>(blockIdx.x) + (run0 > w.tiles0() ? 0 : 1)) * 2 + t) * C::kPart;
        if (!whole) *reinterpret_cast<float2*>(part + r * 4) = make_float2(m, l);
        const float inv = 1.f / l;  // no weight at all on what is seen: 0/0
        const float unit_of_o = CODES ? two_to(o_exp - kLiftCodes) : 1.f;
#pragma unroll 1
        for (int x = 0; x < DP; x += 32) {
          float o[32];
          tmem_ld32_async(to + x, o);
          tmem_wait_ld();
          if constexpr (CODES) in_order(o, (lost >> (x / 64)) & 1u ? NAN : unit_of_o);
          if (whole) {
            store32(o, inv, x);
          } else {
#pragma unroll
            for (int y = 0; y < 32; y += 4)
              *reinterpret_cast<float4*>(part + kQT * 4 + ((x + y) / 4 * kQT + r) * 4) =
                  make_float4(o[y], o[y + 1], o[y + 2], o[y + 3]);
          }
        }
        const int64_t c0 = whole ? 0 : runs.of(w.tiles0()), c1 = whole ? 0 : runs.of(w.tiles0() + w.sp.n - 1);
        if (!whole && c1 - c0 >= kInlineParts) {
          if (tid == 0 && run0 <= w.tiles0()) {  // the unit's first part: the record for the joining launch
            Cut cut;
            cut.count = static_cast<int>(c1 - c0) + 1;
            cut.rt = w.rt;
            cut.h = w.h;
            cut.row0 = w.s.row0;
            cut.m = w.s.m;
            cut.len = w.s.len;
            a.cuts[blockIdx.x] = cut;
          }
        } else if (!whole) {
          // one ticket a warp: its rows of the unit whose first tile is in c0's run
          unsigned int* ticket = a.tickets + c0 * kSoftWarps + warp;
          __threadfence();
          __syncwarp();
          unsigned int done = 0;
          if (lane == 0) done = atomicAdd(ticket, 1u);
          done = __shfl_sync(~0u, done, 0);
          if (done == static_cast<unsigned int>(c1 - c0)) {
            if (lane == 0) *ticket = 0u;  // zero between launches
            __threadfence();
            auto part_of = [&](int64_t x) {  // only c0's run starts before the unit's tiles
              return a.part + ((2 * x + (x == c0 ? 1 : 0)) * 2 + t) * C::kPart;
            };
            float2 ml[kInlineParts];
#pragma unroll
            for (int x = 0; x < kInlineParts; ++x)
              ml[x] = c0 + x <= c1 ? __ldcg(reinterpret_cast<const float2*>(part_of(c0 + x) + r * 4)) : make_float2(-INFINITY, 0.f);
            float M = ml[0].x, L = 0.f, wt[kInlineParts];
#pragma unroll
            for (int x = 1; x < kInlineParts; ++x) M = fmaxf(M, ml[x].x);
#pragma unroll
            for (int x = 0; x < kInlineParts; ++x) {
              wt[x] = ex2((ml[x].x - (M == -INFINITY ? 0.f : M)) * c);
              L += wt[x] * ml[x].y;
            }
            const float inv_l = 1.f / L;
#pragma unroll 1
            for (int y = 0; y < DP; y += 32) {
              float o[32] = {};
#pragma unroll
              for (int x0 = 0; x0 < kInlineParts; x0 += 2) {  // two parts' loads in flight
                if (c0 + x0 > c1) break;
                float4 u[2][8];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const float* p = part_of(min(c0 + x0 + i, c1));  // (a part past the last weighs nothing)
#pragma unroll
                  for (int z = 0; z < 8; ++z)
                    u[i][z] = __ldcg(reinterpret_cast<const float4*>(p + kQT * 4 + ((y / 4 + z) * kQT + r) * 4));
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  if (c0 + x0 + i > c1) break;
#pragma unroll
                  for (int z = 0; z < 8; ++z) {
                    o[4 * z] += wt[x0 + i] * u[i][z].x;
                    o[4 * z + 1] += wt[x0 + i] * u[i][z].y;
                    o[4 * z + 2] += wt[x0 + i] * u[i][z].z;
                    o[4 * z + 3] += wt[x0 + i] * u[i][z].w;
                  }
                }
              }
              store32(o, inv_l, y);
            }
          }
        }
        // the next unit's products overwrite O only after this read
        fence_before();
        ++mine;
      }
      tile_n += w.nt;
      if (!w.more()) break;
      next_segment(a, w);
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == C::kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

// Join of 16 columns of one row tile of the unit whose first part is CTA
// blockIdx.x's: the threads are 128 rows by two groups of parts (even, odd),
// added in order. Only the first part's run starts no later than the unit's
// tiles, so that part is in its CTA's slot 1 and the others in slot 0. Most
// blocks find no unit to join: they are small (with four groups an empty launch
// takes 6 us, with two 3).
constexpr int kJoinCols = 16, kJoinGroups = 2;
template <int DP>
__global__ void __launch_bounds__(kQT * kJoinGroups) prefill_join_kernel(AttnArgs a) {
  constexpr int64_t kPart = static_cast<int64_t>(kQT) * (DP + 4);
  __shared__ float s_m[kJoinGroups][kQT];
  __shared__ float s_o[kJoinCols + 1][kQT];  // the odd parts' columns, and their sum of weights
  pdl_wait();
  const Cut cut = a.cuts[blockIdx.x];
  const int t = blockIdx.y & 1, col0 = (blockIdx.y >> 1) * kJoinCols;
  const int r = threadIdx.x % kQT, grp = threadIdx.x / kQT;
  const int64_t total = static_cast<int64_t>(cut.m) * a.g, rg = static_cast<int64_t>(cut.rt) * kUnitRows + t * kQT + r;
  if (cut.count == 0 || rg - r >= total || col0 >= a.D) return;
  const float c = a.scale_log2;
  auto part = [&](int i) {
    return a.part + ((2 * static_cast<int64_t>(blockIdx.x + i) + (i == 0 ? 1 : 0)) * 2 + t) * kPart;
  };
  float M = -INFINITY;
#pragma unroll 8
  for (int i = grp; i < cut.count; i += kJoinGroups) M = fmaxf(M, __ldcg(part(i) + r * 4));
  s_m[grp][r] = M;
  __syncthreads();
  M = fmaxf(s_m[0][r], s_m[1][r]);
  const float Mu = M == -INFINITY ? 0.f : M;
  float o[kJoinCols] = {}, L = 0.f;
#pragma unroll 6
  for (int i = grp; i < cut.count; i += kJoinGroups) {
    const float* p = part(i);
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(p + r * 4));
    const float f = ex2((ml.x - Mu) * c);
    L += f * ml.y;
#pragma unroll
    for (int z = 0; z < kJoinCols / 4; ++z) {
      const float4 u = __ldcg(reinterpret_cast<const float4*>(p + kQT * 4 + ((col0 / 4 + z) * kQT + r) * 4));
      o[4 * z] += f * u.x;
      o[4 * z + 1] += f * u.y;
      o[4 * z + 2] += f * u.z;
      o[4 * z + 3] += f * u.w;
    }
  }
  if (grp == 1) {
#pragma unroll
    for (int x = 0; x < kJoinCols; ++x) s_o[x][r] = o[x];
    s_o[kJoinCols][r] = L;
  }
  __syncthreads();
  if (grp == 1 || rg >= total) return;
#pragma unroll
  for (int x = 0; x < kJoinCols; ++x) o[x] += s_o[x][r];
  L += s_o[kJoinCols][r];
  const int i = static_cast<int>(quotient(rg, a.g)), hq = cut.h * a.g + static_cast<int>(rg - static_cast<int64_t>(i) * a.g);
  const bool seen = cut.len - cut.m + i >= 0;
  const float inv = 1.f / L;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (static_cast<int64_t>(cut.row0) + i) * a.ldo +
                       static_cast<int64_t>(hq) * a.D + col0;
#pragma unroll
  for (int x = 0; x < kJoinCols; x += 8) {
    if (col0 + x >= a.D) continue;
    uint32_t v[4];
#pragma unroll
    for (int y = 0; y < 4; ++y)
      v[y] = pack_bf16(seen ? o[x + 2 * y] * inv : 0.f, seen ? o[x + 2 * y + 1] * inv : 0.f);
    *reinterpret_cast<uint4*>(out + x) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// Whether a unit could have more than kInlineParts parts, from what the host
// knows: a unit's most tiles, against the least length of a run (every unit is
// a tile and its fixed cost at least).
bool may_need_join(const AttnArgs& a, int num_sms) {
  int64_t tokens = static_cast<int64_t>(a.max_pages) << a.page_shift;
  if (a.window > 0) tokens = std::min<int64_t>(tokens, static_cast<int64_t>(a.window) + kUnitRows / a.g + 1 + kKT + a.sinks + kKT);
  const int64_t tiles = tokens / kKT + 1;
  const int64_t units = (static_cast<int64_t>(a.n_rows) * a.g + kUnitRows - 1) / kUnitRows * a.Hkv;
  const int64_t run = std::max<int64_t>(1, units * (1 + unit_cost(a)) / num_sms);
  return std::min(tiles, (tiles + run - 1) / run + 1) > kInlineParts;
}

template <int DP, bool APART, bool CODES>
cudaError_t launch(const AttnArgs& a, int num_sms, cudaStream_t st) {
  CUtensorMap mk{}, mv{};  // (codes are loaded without)
  const int page = 1 << a.page_shift;
  cudaError_t e;
  if (CODES) {
  } else if ((e = map_pages(&mk, a.k, a.D, page, static_cast<int64_t>(a.n_pages) * a.Hkv, std::min(page, kKT))) != cudaSuccess ||
      (e = map_pages(&mv, a.v, a.D, page, static_cast<int64_t>(a.n_pages) * a.Hkv, std::min(page, kKT))) != cudaSuccess)
    return e;
  constexpr int smem = kSmem<DP, APART, CODES>;
  e = cudaFuncSetAttribute(prefill_kernel<DP, APART, CODES>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  prefill_kernel<DP, APART, CODES><<<num_sms, Cfg<DP, APART, CODES>::kThreads, smem, st>>>(mk, mv, a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (!may_need_join(a, num_sms)) return cudaSuccess;
  AttnArgs j = a;
  if (CODES) j.scale_log2 = 1.f;  // the parts' maxima are in units of log2
  return pdl_launch(prefill_join_kernel<DP>, dim3(num_sms, 2 * DP / kJoinCols), dim3(kQT * kJoinGroups), 0, st, j);
}

}  // namespace

cudaError_t launch_attn_prefill_tc(const AttnArgs& a, int num_sms, cudaStream_t st) {
  cudaError_t e = encoder();
  if (e != cudaSuccess) return e;
  if (a.D > 64) return launch<128, false, false>(a, num_sms, st);
  // P beside S pays where most tiles need no mask (4,096 tokens at 32K, 16 heads
  // of 64: 554 -> 500 us), not in a window's few tiles (ragged prompts, window
  // 1,024: 92 -> 100 us)
  return a.window > 0 ? launch<64, false, false>(a, num_sms, st) : launch<64, true, false>(a, num_sms, st);
}
cudaError_t launch_attn_prefill_codes_tc(const AttnArgs& a, int num_sms, cudaStream_t st) {
  if (a.D > 64) return launch<128, false, true>(a, num_sms, st);
  return a.window > 0 ? launch<64, false, true>(a, num_sms, st) : launch<64, true, true>(a, num_sms, st);
}

}  // namespace moe
