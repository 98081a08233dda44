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
#include "attn_split.cuh"

namespace moe {
namespace {

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
  static constexpr int kMl = kWarps * 16;
  static constexpr bool kCodes = false;
  static constexpr int kRowBytes = 0, kMostSlots = 8, kGroup = 1;
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

  __device__ __forceinline__ void place(float* buf) { qs = su32(buf) + kWarps * 16 * 64 * 4; }
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
  static constexpr int kMl = kWarps * 16;
  static constexpr bool kCodes = false;
  static constexpr int kRowBytes = 0, kMostSlots = 8, kGroup = 1;
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
