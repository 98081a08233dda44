// The engine of attention over pages of 4-bit codes, on warp-level matrix
// instructions.
//
// A head of a page is an affine matrix of groups of 64 along the head: the value
// of code q (0 to 15) of token t and group g is s_tg q + b_tg = s_tg (q - 8) +
// b'_tg with b' = b + 8 s, so that for a query x and numerators p
//   x.k_t   = sum_g s_tg (sum_d x_d (q_td - 8)) + b'_tg sum_d x_d
//   sum_t p_t v_td = sum_t (p_t s_tg) (q_td - 8) + sum_t p_t b'_tg.
// The matrix instructions multiply codes, q - 8, which are exact in f16 and in bf16.
// Scales and offsets are applied in fp32 to the scores of a group, and to the numerators
// before they become an operand; the offsets' sums stay in fp32. bf16 calls multiply f16:
// x as it is, p s rounded to f16 once (error against 64 bits 1.7e-3 of the norm, nearly all
// of it the result's own rounding to bf16; with p s in bf16 2.4e-3). f16's range is made
// up for by powers of two. A row's x is divided by one that makes its largest about 2^14:
// with the factor of 16 below, x loses no bits down to 2^-24 of that. p s is divided by that
// of a unit's first scale, or of a later one 4 times as large, and kept 2^10 times as large
// (p is below 2^3): it loses no bits down to 2^-24 of a token that has both the row's largest
// weight and the largest scale, and is more than nothing down to 2^-34. (Scores are in x's
// unit, up to 2^14 times as large as they are: scales from 2^100 on may take them beyond
// fp32.) f32 calls multiply x and p s as three bf16 that add up to them.
// V's codes are centred because the rounding of p s is multiplied by them: of q itself
// it would carry 2.5 times the noise. K's are not, for f16: their operand keeps the
// magnitude of 1024 that unpacking gives them (and the factor of 16 of every other
// pair, which x is divided by), and the sum starts at what that adds up to, negative.
// Sums of some thousand times x then keep 2^-24 of that, a score's 2^-15 or so.
//
// The scores are formed transposed, S^T = K Q^T, so that a warp's 16 tokens are
// the rows of the instruction and eight query rows its columns: eight heads that
// share a cache head leave no row of the instruction empty. The values follow as
// O^T = V^T P^T with P^T turned from one fragment layout to the other by
// movmatrix. Which of a group's dimensions takes which place of a fragment is
// free as long as both operands agree: a thread takes whole words of eight codes,
// and nibbles i and i + 4 (K), or nibble i of two tokens (V), become a pair of
// f16 by one and-or into the mantissa of 1024 and one subtraction. The integer pipe,
// at half the rate of the others, is what bounds few rows: f16's ten bits take a
// nibble at either end of a byte, so a word needs one shift, bf16's seven three.
//
// What a row does not see cannot reach it: hidden scores are -inf by selection,
// and a hidden token's scale and offset, which may be anything, are left out of
// its numerator's products by selection.
#pragma once

#include <cuda_fp16.h>

#include "attn_split.cuh"

namespace moe {
namespace {

// d = a b + c; HALF: f16 operands, else bf16
template <bool HALF>
__device__ __forceinline__ void mma_codes(float* d, const uint32_t* a, const uint32_t* b, const float* c) {
#define MOE_MMA(T, C0, C1, C2, C3)                                                                                          \
  asm("mma.sync.aligned.m16n8k16.row.col.f32." T "." T ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"      \
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])                                                                       \
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(C0), "f"(C1), "f"(C2), "f"(C3))
  if constexpr (HALF)
    MOE_MMA("f16", c[0], c[1], c[2], c[3]);
  else
    MOE_MMA("bf16", c[0], c[1], c[2], c[3]);
#undef MOE_MMA
}
// q - 8 of nibbles i and i + 4 of a word as a pair: the magnitude that a nibble is the last bits of goes off again
template <bool HALF>
constexpr uint32_t kMagic = HALF ? 0x64006400u : 0x43004300u;
// 1024 + q of nibbles 0 and 4 or 2 and 6, 1024 + 16 q of the others
__device__ __forceinline__ uint32_t raised(uint32_t w, int i, uint32_t magic) {
  const uint32_t at = i < 2 ? w : w >> 8;
  return i & 1 ? and_or<0x00F000F0u>(at, magic) : and_or<0x000F000Fu>(at, magic);
}
template <bool HALF>
__device__ __forceinline__ uint32_t centred(uint32_t w, int i, uint32_t magic) {
  if constexpr (HALF) {
    const uint32_t m = raised(w, i, magic);
    const __half2 h = *reinterpret_cast<const __half2*>(&m);
    const __half2 v = i & 1 ? __hfma2(h, __float2half2_rn(0.0625f), __float2half2_rn(-72.f)) : __hsub2(h, __float2half2_rn(1032.f));
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const uint32_t m = and_or<0x000F000Fu>(w >> (4 * i), magic);  // 128 + q
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&m), __floats2bfloat162_rn(136.f, 136.f));
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}
__device__ __forceinline__ uint32_t transposed(uint32_t m) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(m));
  return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
  return r;
}
// scale and offset (for centred codes) of a metadata word
__device__ __forceinline__ float scale_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float offset_of(uint32_t w) { return fmaf(8.f, scale_of(w), __uint_as_float(w & 0xFFFF0000u)); }
// a token's metadata words
template <int G>
__device__ __forceinline__ void load_meta(uint32_t at, uint32_t* m) {
  if constexpr (G == 4) {
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(m[0]), "=r"(m[1]), "=r"(m[2]), "=r"(m[3]) : "r"(at));
  } else if constexpr (G == 2) {
    const uint2 v = lds64(at);
    m[0] = v.x;
    m[1] = v.y;
  } else {
#pragma unroll
    for (int g = 0; g < G; ++g) m[g] = lds32(at + 4 * g);
  }
}
// a pair as f16 (N = 1), or its bf16 parts: what is left after each is the next one's
template <int N>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t* part) {
  if constexpr (N == 1) {
    const __half2 h = __floats2half2_rn(x, y);
    part[0] = *reinterpret_cast<const uint32_t*>(&h);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      part[i] = pack_bf16(x, y);
      if (i + 1 < N) {
        x -= __uint_as_float(part[i] << 16);
        y -= __uint_as_float(part[i] & 0xFFFF0000u);
      }
    }
  }
}

// G groups of 64 a head, 8 NR query rows, tiles of 128 tokens of which each warp takes
// 16. Up to GROUP tiles are worked on together: a warp's steps are chains of dependent
// instructions, and several chains hide each other (three contexts of 131K to 262K
// tokens: 212 us with 1, 171 with 2, 154 with 4, which leaves three slots, and with 6,
// which leaves two; heads of 64: 93 with 4, 83 with 8); one by one at a unit's end (in
// twos, too: 161, for the code's size).
template <class T_, int G_, int NR_, int GROUP>
struct CodesEngine {
  using T = T_;
  static constexpr int G = G_, NR = NR_, KT = 16 * kWarps, kGroup = GROUP;
  static constexpr int DP = G == 1 ? 64 : (G == 2 ? 128 : 256);
  static constexpr int kRows = 8 * NR, NB = 1;
  static constexpr bool kHalf = sizeof(T) == 2;
  static constexpr int kParts = kHalf ? 1 : 3;  // parts of an operand
  // f16: numerators stay below 2^3 and scales below 4 of their unit, so that their products may be
  // kept 2^10 times as large
  static constexpr float kRaise = kHalf ? 3.f : 8.f;
  static constexpr int kRoom = 2, kLift = 10;
  static constexpr bool kCodes = true;
  static constexpr int kRowBytes = 32 * G, kMetaBytes = 4 * G, kMostSlots = 12;
  static constexpr uint32_t kTileBytes = KT * (kRowBytes + kMetaBytes);
  // tiles' worth of time of a unit's Q, join of the warps and results (10 contexts to
  // 32,768 tokens, heads of 256: 41 us with 2, 35 with 6; 40 contexts, of 128: 31 with 3, 34 with 8)
  static constexpr int kUnitCost = G > 2 ? 6 : 3;
  static constexpr int kSteps = 4 * G;  // products of 16 dimensions
  // Q as fragments in registers, or in shared memory where there are too many
  static constexpr bool kQInSmem = kSteps * NR * kParts > 32;
  static constexpr int kQBytes = kQInSmem ? kSteps * NR * kParts * 256 : 0;
  static constexpr int kMl = kWarps * kRows;
  static constexpr int kMergeCols = NR == 1 ? 32 : 64;  // columns joined at a time
  static constexpr int kMergeBytes = kWarps * kRows * kMergeCols * 4 + kQBytes;

  uint32_t qf[kQInSmem ? 1 : kParts * NR * kSteps][2];
  uint32_t qs;           // shared copy of the fragments
  // of this thread's columns (query rows 8 nt + 2 c and + 1): sums of a group's x, and
  // what its products with the magnitudes of K's operand add up to, negative
  float qsum[G][NR][2], lift[G][NR][2];
  float o[4 * G][NR][4];
  float bias[G][NR][2];  // this thread's share of the offsets' sums
  float x[GROUP][NR][4]; // scores, then numerators: tokens r and r + 8, two columns each
  uint32_t seen[GROUP];  // of an edge tile: bit 4 nt + i of x visible
  float m[NR][2], thr[NR][2], l[NR][2];
  float cs[NR][2];       // scale log2(e), times the power of two that the row's x was divided by
  // f16: the numerators' products are kept divided by a power of two: 1 / it, and the
  // bits of the scale from which on it has to grow (0: any)
  float v_inv;
  uint32_t v_limit;
  uint32_t magic;        // kMagic
  int pos[NR][2];        // -1: no row
  int lo_pos, hi_pos;    // of the unit's rows
  bool edge;             // the tile holds a token seen by some but not all of the rows

  __device__ __forceinline__ void place(float* buf) {
    qs = su32(buf) + kWarps * kRows * kMergeCols * 4;
    magic = in_register(kMagic<kHalf>);
  }
  __device__ __forceinline__ const uint32_t* fragment(int part, int nt, int step, uint32_t* tmp) const {
    const int at = (part * NR + nt) * kSteps + step;
    if constexpr (kQInSmem) {
      const uint2 v = lds64(qs + at * 256 + (threadIdx.x & 31) * 8);
      tmp[0] = v.x;
      tmp[1] = v.y;
      return tmp;
    } else {
      return qf[at];
    }
  }

  // eight values in fp32; zeros without an address
  __device__ __forceinline__ static void load8(const T* at, float* v) {
    if constexpr (sizeof(T) == 4) {
      const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 u0 = at ? __ldg(reinterpret_cast<const float4*>(at)) : z, u1 = at ? __ldg(reinterpret_cast<const float4*>(at) + 1) : z;
      v[0] = u0.x, v[1] = u0.y, v[2] = u0.z, v[3] = u0.w, v[4] = u1.x, v[5] = u1.y, v[6] = u1.z, v[7] = u1.w;
    } else {
      const uint4 u = at ? __ldg(reinterpret_cast<const uint4*>(at)) : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t us[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(us[i] << 16);
        v[2 * i + 1] = __uint_as_float(us[i] & 0xFFFF0000u);
      }
    }
  }
  __device__ __forceinline__ void begin(const AttnArgs& a, const Cursor& c) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, cc = lane & 3;
    lo_pos = c.s.len - c.s.m + c.token(a, 0);
    hi_pos = c.s.len - c.s.m + c.token(a, c.rows - 1);
#pragma unroll
    for (int nt = 0; nt < NR; ++nt) {
      const int row = 8 * nt + r;
      const T* q = nullptr;
      if (row < c.rows)
        q = static_cast<const T*>(a.q) + static_cast<int64_t>(c.s.row0 + c.token(a, row)) * a.ldq + c.head(a, row) * a.D;
      float v[G][2][8];
      float top = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          load8(q ? q + 64 * g + 16 * cc + 8 * w : nullptr, v[g][w]);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (fabsf(v[g][w][i]) < INFINITY) top = fmaxf(top, fabsf(v[g][w][i]));
        }
      float f = 1.f, c_row = a.scale_log2;
      if constexpr (kHalf) {
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127 - 14, -116);  // about 2^14 is left
        f = two_to(-e);
        c_row = score_factor(a.scale_log2, e);
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float sum = 0.f, up = 0.f;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          // a product takes pairs (i, i + 4) of eight dimensions
          float (&u)[8] = v[g][w];
#pragma unroll
          for (int i = 0; i < 8; ++i) u[i] *= f;
          sum += ((u[0] + u[1]) + (u[2] + u[3])) + ((u[4] + u[5]) + (u[6] + u[7]));
          uint32_t pair[4][kParts];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float d = kHalf && (i & 1) ? 0.0625f : 1.f;  // (K's codes are 16-fold there)
            split_pair<kParts>(u[i] * d, u[i + 4] * d, pair[i]);
            if constexpr (kHalf) {
              const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&pair[i][0]));
              up -= 1024.f * z.x + 1024.f * z.y;
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
              const int at = (part * NR + nt) * kSteps + (g * 2 + w) * 2 + h;
              if constexpr (kQInSmem) {
                if (at % kWarps == warp)
                  asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(qs + at * 256 + lane * 8), "r"(pair[2 * h][part]),
                               "r"(pair[2 * h + 1][part])
                               : "memory");
              } else {
                qf[at][0] = pair[2 * h][part];
                qf[at][1] = pair[2 * h + 1][part];
              }
            }
        }
        sum += __shfl_xor_sync(~0u, sum, 1);
        sum += __shfl_xor_sync(~0u, sum, 2);
        up += __shfl_xor_sync(~0u, up, 1);
        up += __shfl_xor_sync(~0u, up, 2);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          qsum[g][nt][e] = __shfl_sync(~0u, sum, 8 * cc + 4 * e);
          lift[g][nt][e] = __shfl_sync(~0u, up, 8 * cc + 4 * e);
          bias[g][nt][e] = 0.f;
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = 8 * nt + 2 * cc + e;
        pos[nt][e] = col < c.rows ? c.s.len - c.s.m + c.token(a, col) : -1;
        m[nt][e] = thr[nt][e] = -INFINITY;
        cs[nt][e] = __shfl_sync(~0u, c_row, 8 * cc + 4 * e);
        l[nt][e] = 0.f;
      }
#pragma unroll
      for (int t = 0; t < 4 * G; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[t][nt][i] = 0.f;
    }
    v_inv = 1.f;
    v_limit = 0u;
    if constexpr (kQInSmem) sync_compute();
  }

  // n tiles of K and V, from the cursor's on
  __device__ __forceinline__ void tiles(const AttnArgs& a, const Cursor& c, uint32_t base, int n) {
    const int tile0 = c.sp.tile(c.t) * KT;
    if (GROUP > 1 && n == GROUP) {
      scores<GROUP>(a, tile0, base, 0);
      values<GROUP>(base, 0);
    } else {
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        scores<1>(a, tile0 + i * KT, base, i);
        values<1>(base, i);
      }
    }
  }

  // CH tiles, the first of them the slot's i0-th
  template <int CH>
  __device__ __forceinline__ void scores(const AttnArgs& a, int tile0, uint32_t base, int i0) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, cc = lane & 3;
    edge = tile0 + CH * KT - 1 > lo_pos || (a.window > 0 && hi_pos - tile0 >= a.window);
    const uint32_t key0 = (i0 * kWarps + warp) * 16 + r;
    const uint32_t at0 = base + key0 * kRowBytes + 8 * cc, meta0 = base + GROUP * KT * kRowBytes + key0 * kMetaBytes;
#pragma unroll
    for (int ch = 0; ch < CH; ++ch) {
      const uint32_t at = at0 + ch * KT * kRowBytes, meta = meta0 + ch * KT * kMetaBytes;
#pragma unroll
      for (int nt = 0; nt < NR; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[ch][nt][i] = 0.f;
      uint32_t m0[G], m1[G];
      load_meta<G>(meta, m0);
      load_meta<G>(meta + 8 * kMetaBytes, m1);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const uint2 w0 = lds64(at + 32 * g), w1 = lds64(at + 8 * kRowBytes + 32 * g);
        // f16: codes of q, lifted; f32: of q - 8
        float acc[NR][4];
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[nt][i] = lift[g][nt][i & 1];
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t c0 = w ? w0.y : w0.x, c1 = w ? w1.y : w1.x;
            uint32_t k[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t c = i & 1 ? c1 : c0;
              k[i] = kHalf ? raised(c, 2 * h + (i >> 1), magic) : centred<kHalf>(c, 2 * h + (i >> 1), magic);
            }
#pragma unroll
            for (int nt = 0; nt < NR; ++nt)
#pragma unroll
              for (int part = 0; part < kParts; ++part) {
                uint32_t tmp[2];
                mma_codes<kHalf>(acc[nt], k, fragment(part, nt, (g * 2 + w) * 2 + h, tmp), acc[nt]);
              }
          }
        const float s0 = scale_of(m0[g]), s1 = scale_of(m1[g]);
        const float b0 = kHalf ? __uint_as_float(m0[g] & 0xFFFF0000u) : offset_of(m0[g]);
        const float b1 = kHalf ? __uint_as_float(m1[g] & 0xFFFF0000u) : offset_of(m1[g]);
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            x[ch][nt][e] += s0 * acc[nt][e] + b0 * qsum[g][nt][e];
            x[ch][nt][2 + e] += s1 * acc[nt][2 + e] + b1 * qsum[g][nt][e];
          }
      }
    }
    if (edge) {
#pragma unroll
      for (int ch = 0; ch < CH; ++ch) {
        seen[ch] = 0u;
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = tile0 + (ch * kWarps + warp) * 16 + r + 8 * (i >> 1);
            const int back = pos[nt][i & 1] - j;
            const bool see = back >= 0 && (a.window == 0 || back < a.window || j < a.sinks);
            if (see)
              seen[ch] |= 1u << (4 * nt + i);
            else
              x[ch][nt][i] = -INFINITY;
          }
      }
    }
    // m is raised only when a score passes it by kRaise: numerators up to there lose nothing
    float mx[NR][2];
    bool up = false;
#pragma unroll
    for (int nt = 0; nt < NR; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = fmaxf(x[0][nt][e], x[0][nt][2 + e]);
#pragma unroll
        for (int ch = 1; ch < CH; ++ch) v = fmaxf(v, fmaxf(x[ch][nt][e], x[ch][nt][2 + e]));
        mx[nt][e] = v;
        up |= v > thr[nt][e];
      }
    if (__any_sync(~0u, up)) {
#pragma unroll
      for (int nt = 0; nt < NR; ++nt) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = mx[nt][e];
          v = fmaxf(v, __shfl_xor_sync(~0u, v, 4));
          v = fmaxf(v, __shfl_xor_sync(~0u, v, 8));
          v = fmaxf(v, __shfl_xor_sync(~0u, v, 16));
          f[e] = 1.f;
          if (v > thr[nt][e]) {
            f[e] = ex2((m[nt][e] - v) * cs[nt][e]);  // 0 for the first maximum
            m[nt][e] = v;
            thr[nt][e] = v + kRaise / cs[nt][e];
          }
          l[nt][e] *= f[e];
#pragma unroll
          for (int g = 0; g < G; ++g) bias[g][nt][e] *= f[e];
        }
#pragma unroll
        for (int t = 0; t < 4 * G; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[t][nt][i] *= f[i & 1];
      }
    }
#pragma unroll
    for (int nt = 0; nt < NR; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mc = m[nt][e] == -INFINITY ? 0.f : m[nt][e] * cs[nt][e];
#pragma unroll
        for (int ch = 0; ch < CH; ++ch)
#pragma unroll
          for (int i = e; i < 4; i += 2) {
            x[ch][nt][i] = ex2(fmaf(x[ch][nt][i], cs[nt][e], -mc));
            l[nt][e] += x[ch][nt][i];
          }
      }
  }

  template <int CH>
  __device__ __forceinline__ void values(uint32_t base, int i0) {
    if (edge)
      add_values<CH, true>(base, i0);
    else
      add_values<CH, false>(base, i0);
  }
  template <int CH, bool EDGE>
  __device__ __forceinline__ void add_values(uint32_t base, int i0) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, cc = lane & 3;
    const uint32_t v0 = base + GROUP * kTileBytes, key0 = (i0 * kWarps + warp) * 16;
    const uint32_t at0 = v0 + (key0 + 2 * cc) * kRowBytes + 4 * r, meta0 = v0 + GROUP * KT * kRowBytes + (key0 + r) * kMetaBytes;
#pragma unroll
    for (int ch = 0; ch < CH; ++ch) {
      const uint32_t at = at0 + ch * KT * kRowBytes, meta = meta0 + ch * KT * kMetaBytes;
      uint32_t m0[G], m1[G];
      load_meta<G>(meta, m0);
      load_meta<G>(meta + 8 * kMetaBytes, m1);
      if constexpr (kHalf) {  // the largest scale, of what a row sees: the low halves as they are
        const bool see0 = !EDGE || (seen[ch] & 0x33333333u), see1 = !EDGE || (seen[ch] & 0xCCCCCCCCu);
        uint32_t most = 0;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          most = __vmaxu2(most, see0 ? m0[g] : 0u);
          most = __vmaxu2(most, see1 ? m1[g] : 0u);
        }
        if (__any_sync(~0u, (most << 16) >= v_limit)) widen(m0, m1, see0, see1);
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const uint32_t w0 = lds32(at + 32 * g), w1 = lds32(at + kRowBytes + 32 * g);
        const uint32_t w2 = lds32(at + 8 * kRowBytes + 32 * g), w3 = lds32(at + 9 * kRowBytes + 32 * g);
        const float s[2] = {kHalf ? scale_of(m0[g]) * v_inv : scale_of(m0[g]), kHalf ? scale_of(m1[g]) * v_inv : scale_of(m1[g])};
        const float b[2] = {offset_of(m0[g]), offset_of(m1[g])};
        uint32_t p[NR][kParts][2];
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float n = x[ch][nt][2 * h + e];
              const bool see = !EDGE || ((seen[ch] >> (4 * nt + 2 * h + e)) & 1u);
              v[e] = see ? n * s[h] : 0.f;
              if (see) bias[g][nt][e] += n * b[h];
            }
            uint32_t part[kParts];
            split_pair<kParts>(v[0], v[1], part);
#pragma unroll
            for (int i = 0; i < kParts; ++i) p[nt][i][h] = transposed(part[i]);
          }
        // a pair's halves are nibble i of two tokens
        const uint32_t lo[2] = {__byte_perm(w0, w1, 0x5410), __byte_perm(w2, w3, 0x5410)};
        const uint32_t hi[2] = {__byte_perm(w0, w1, 0x7632), __byte_perm(w2, w3, 0x7632)};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t v[4] = {centred<kHalf>(lo[0], j, magic), centred<kHalf>(hi[0], j, magic), centred<kHalf>(lo[1], j, magic),
                                 centred<kHalf>(hi[1], j, magic)};
#pragma unroll
          for (int nt = 0; nt < NR; ++nt) {
            if constexpr (kParts == 1) {
              mma_codes<kHalf>(o[4 * g + j][nt], v, p[nt][0], o[4 * g + j][nt]);
            } else {
              // f32: a chunk's products are added up on their own and then to the sum in one rounding
              float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int i = 0; i < kParts; ++i) mma_codes<kHalf>(t, v, p[nt][kParts - 1 - i], t);
#pragma unroll
              for (int i = 0; i < 4; ++i) o[4 * g + j][nt][i] += t[i];
            }
          }
        }
      }
    }
  }

  // Products are kept divided by the power of two of the first scale, until one is 4 times as large. (A negative
  // scale, or one that is infinite or NaN, comes here too, and changes nothing by itself.)
  __device__ __forceinline__ void widen(const uint32_t* m0, const uint32_t* m1, bool see0, bool see1) {
    float top = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float s0 = fabsf(scale_of(m0[g])), s1 = fabsf(scale_of(m1[g]));
      if (see0 && s0 < INFINITY) top = fmaxf(top, s0);
      if (see1 && s1 < INFINITY) top = fmaxf(top, s1);
    }
    const uint32_t most = __reduce_max_sync(~0u, __float_as_uint(top));
    if (most < v_limit || !__any_sync(~0u, see0 || see1)) return;
    const int e = max(static_cast<int>(most >> 23) - 127, -116);
    const float inv = two_to(kLift - e), f = inv / v_inv;
    v_inv = inv;
    v_limit = __float_as_uint(two_to(min(e + kRoom, 127)));
#pragma unroll
    for (int t = 0; t < 4 * G; ++t)
#pragma unroll
      for (int nt = 0; nt < NR; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[t][nt][i] *= f;
  }

  // Join the warps' results in shared memory, a group's 64 columns at a time, and
  // hand (row, column, 4 values, m, l) to store. Called by every thread.
  template <class F>
  __device__ __forceinline__ void end(const AttnArgs& a, const Cursor& c, float* buf, float2* ml, F&& store) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, cc = lane & 3;
    auto over_tokens = [](float v) {
      v += __shfl_xor_sync(~0u, v, 4);
      v += __shfl_xor_sync(~0u, v, 8);
      return v + __shfl_xor_sync(~0u, v, 16);
    };
#pragma unroll
    for (int nt = 0; nt < NR; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float sum = over_tokens(l[nt][e]);
        if (r == 0) ml[warp * kRows + 8 * nt + 2 * cc + e] = make_float2(m[nt][e] * cs[nt][e], sum);
      }
    const int rows = c.rows;
    const float unit = kHalf ? 1.f / v_inv : 1.f;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int nt = 0; nt < NR; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) bias[g][nt][e] = over_tokens(bias[g][nt][e]);
    // a thread's columns of a group: 8 r .. 8 r + 7, in two quads
#pragma unroll
    for (int col0 = 0; col0 < 64 * G; col0 += kMergeCols) {
      const int g = col0 / 64;
#pragma unroll
      for (int nt = 0; nt < NR; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float b = bias[g][nt][e];
          float* at = buf + (warp * kRows + 8 * nt + 2 * cc + e) * kMergeCols;
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (kMergeCols == 64 || (r >> 2) == (col0 & 32) / 32)
              *reinterpret_cast<float4*>(at + (((8 * r + 4 * h) & (kMergeCols - 1)) ^ (cc << 3))) =
                  make_float4(fmaf(o[4 * g][nt][2 * h + e], unit, b), fmaf(o[4 * g + 1][nt][2 * h + e], unit, b),
                              fmaf(o[4 * g + 2][nt][2 * h + e], unit, b), fmaf(o[4 * g + 3][nt][2 * h + e], unit, b));
        }
      sync_compute();
      for (int e = threadIdx.x; e < rows * (kMergeCols / 4); e += kCompute) {
        const int row = e / (kMergeCols / 4), col = e % (kMergeCols / 4) * 4;
        float M = -INFINITY;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) M = fmaxf(M, ml[k * kRows + row].x);
        const float Mu = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          const float2 t = ml[k * kRows + row];
          const float f = ex2(t.x - Mu);
          L += f * t.y;
          const float4 u = *reinterpret_cast<const float4*>(buf + (k * kRows + row) * kMergeCols + (col ^ (((row >> 1) & 3) << 3)));
          v.x += f * u.x;
          v.y += f * u.y;
          v.z += f * u.z;
          v.w += f * u.w;
        }
        store(row, col0 + col, v, M, L);
      }
      sync_compute();
    }
  }
};

}  // namespace
}  // namespace moe
