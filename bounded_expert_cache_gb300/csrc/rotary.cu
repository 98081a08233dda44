// Rotary positions, and a step's keys and values written into the paged cache with
// the rotation on the way; values read back from pages.
//
// The pair (a, b) = (x_i, x_i+dim/2) or (x_2i, x_2i+1) of a head at position p
// becomes (a c - b s, b c + a s) with c, s = magnitude times cos, sin of p f_i.
// p f_i reaches 10^6 radians, of which fp32 would keep a sixteenth: the frequencies
// are given in turns as 64-bit fractions, so that p times one wraps whole turns
// away exactly. What is left is the nearest 256th of a turn, whose cosine and sine
// are in a table, and an angle b of at most 2 pi / 512: cos(a + b) = cos a + (cos a
// (cos b - 1) - sin a sin b), where b's series need two terms and what is added is so
// small that c and s are the fp32 next to the exact values but for one in thirty.
// Products and sums are fp32, each rounded, and then the result is to its type (not
// before 4-bit codes): with that and such c and s, codes are those of the same steps
// done one by one, where a last bit's difference puts a few in a million on the other
// side of a border between two codes. (sincospif and fused products: the same times.)
//
// Pages of 4-bit codes: four threads hold a group of 64 values; with lo and hi its
// least and largest, b = bf16(lo), s = bf16((hi - b) (1 / 15)), q = round((x - b) / s)
// within 0..15 (0 where s is 0), in fp32 as in IEEE. A group with an
// infinity, a NaN or a magnitude above 2^126 becomes NaN as a whole.
//
// What bounds them: one row the latency of its lookups (chunk, sequence, length,
// table, page count: five dependent reads) and of one sine (rotary 2.3 us in a graph,
// a write of one token 4.5); prompts HBM. A row's sines and cosines are formed once and
// shared by its heads; a thread owns both halves of a pair, so that a result may
// overwrite its input. 16,384 rows of 40 bf16 heads of 128: 56 us, 5.9 TB/s, halves or
// neighbours, in fp32 110 us, 6.1 TB/s. Halves that do not fill 16 bytes go value by value, a
// third of that: heads of 96 with 24 columns turned 148 us, of 80 with 20 129 (HBM: 37 and 31),
// and writes into pages with such a rotation, 7,592 rows, 32 + 2 x 8 heads of 128: 103 us, not
// the 42 of whole heads (4.4 TB/s). Blocks of 256 threads with 32 registers, eight on an SM: with 40 registers
// and the next item read ahead 68. 7,591 rows of ragged prompts, 32 + 2 x 8 heads of 128
// into 4-bit pages, and these values read back: 60 us, of which q's heads (124 MB) take
// 18, near HBM's rate; the codes, the values read back and the lookups are bound by
// instructions.
#include <cuda_bf16.h>

#include "kv_device.cuh"
#include "packed.cuh"

namespace moe {
namespace {

constexpr int kRotThreads = 256, kMostRows = 4;

// u c - v s and v c + u s (one by one: packed products and sums become fused instructions, .rn or not)
__device__ __forceinline__ float2 turn(float u, float v, float c, float s) {
  return make_float2(__fsub_rn(__fmul_rn(u, c), __fmul_rn(v, s)), __fadd_rn(__fmul_rn(v, c), __fmul_rn(u, s)));
}
template <class T>
struct Vec {
  static constexpr int N = 16 / static_cast<int>(sizeof(T));
};
// 16 bytes of values, as they are in memory, and in fp32
__device__ __forceinline__ uint4 load16(const void* p) { return *static_cast<const uint4*>(p); }
template <class T>
__device__ __forceinline__ void widen(uint4 u, float* v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (sizeof(T) == 4) {
      v[j] = __uint_as_float(w[j]);
    } else {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}
template <class T>
__device__ __forceinline__ uint4 narrow(const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (sizeof(T) == 4) {
      w[j] = __float_as_uint(v[j]);
    } else {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// eight values
template <class T>
__device__ __forceinline__ void load8(const T* p, float* v) {
#pragma unroll
  for (int i = 0; i < 8; i += Vec<T>::N) widen<T>(load16(p + i), v + i);
}
template <class T>
__device__ __forceinline__ void store8(T* p, const float* v) {
#pragma unroll
  for (int i = 0; i < 8; i += Vec<T>::N) *reinterpret_cast<uint4*>(p + i) = narrow<T>(v + i);
}
template <class T>
__device__ __forceinline__ float value(const T* p) {
  return static_cast<float>(*p);
}

// t / n for t <= kRotThreads: (t + 1/2) / n is at least 1 / 2n off a whole number
__device__ __forceinline__ int quotient(int t, int n) { return static_cast<int>((t + 0.5f) * __frcp_rn(static_cast<float>(n))); }

// Items (row, head, item of a head) dealt out to a block's threads in order.
struct Walk {
  int r, h, i;
  int heads, per, dr, dh, di;
  __device__ __forceinline__ Walk(int heads, int per) : heads(heads), per(per) {
    const int u = quotient(threadIdx.x, per), d = quotient(kRotThreads, per);
    r = quotient(u, heads);
    h = u - r * heads;
    i = threadIdx.x - u * per;
    dr = quotient(d, heads);
    dh = d - dr * heads;
    di = kRotThreads - d * per;
  }
  __device__ __forceinline__ void next() {
    i += di;
    h += dh;
    r += dr;
    if (i >= per) {
      i -= per;
      ++h;
    }
    if (h >= heads) {
      h -= heads;
      ++r;
    }
  }
};

// Cosines and sines of the 256ths of a turn, each as a sum of two fp32.
struct TurnTable {
  float cs[256][4];
};
constexpr TurnTable turn_table() {
  TurnTable t{};
  for (int j = 0; j < 256; ++j) {
    const double x = (j < 128 ? j : j - 256) * (3.14159265358979323846 / 128);
    double c = 0, s = 0, term = 1;  // the series of both
    for (int k = 0; k < 40; k += 2) {
      c += term;
      term *= x / (k + 1);
      s += term;
      term *= -x / (k + 2);
    }
    t.cs[j][0] = static_cast<float>(c);
    t.cs[j][1] = static_cast<float>(c - static_cast<float>(c));
    t.cs[j][2] = static_cast<float>(s);
    t.cs[j][3] = static_cast<float>(s - static_cast<float>(s));
  }
  return t;
}
alignas(16) __device__ const TurnTable kTurnTable = turn_table();

// magnitude times (cos, sin) of a position's angle
__device__ __forceinline__ float2 turned(const Rotary& rot, int i, int pos, const float4* table) {
  const uint64_t t = __ldg(rot.turns + i) * static_cast<uint64_t>(static_cast<int64_t>(pos));
  const uint64_t at = t + (1ull << 55);
  const float4 a = table[at >> 56];
  const float b = __ll2float_rn(static_cast<int64_t>(at & ((1ull << 56) - 1)) - (1ll << 55)) * 3.40612158e-19f;  // 2 pi / 2^64
  const float bb = b * b, c1 = bb * fmaf(bb, 1.f / 24, -0.5f), sb = fmaf(b * bb, -1.f / 6, b);
  const float dc = fmaf(a.x, c1, fmaf(-a.z, sb, a.y)), ds = fmaf(a.z, c1, fmaf(a.x, sb, a.w));
  const float m = rot.magnitude, c = m * a.x, s = m * a.z;
  return make_float2(c + fmaf(m, dc, fmaf(rot.magnitude_rest, a.x, fmaf(m, a.x, -c))),
                     s + fmaf(m, ds, fmaf(rot.magnitude_rest, a.z, fmaf(m, a.z, -s))));
}

// How a head's values are dealt out: halves whose vectors match, neighbours, or
// halves of other sizes, value by value.
enum { kHalves = 0, kPairs = 1, kSingle = 2 };
template <class T>
__host__ __device__ __forceinline__ int layout_of(int dim, int interleaved) {
  return interleaved ? kPairs : ((dim / 2) % Vec<T>::N ? kSingle : kHalves);
}

// Heads from h0 on of the block's rows from x to y.
template <class T>
struct Heads {
  static constexpr int N = Vec<T>::N;
  const T* x;
  T* y;
  int64_t ldx, ldy;
  int h0, D, half, layout, turned_items, heads;  // items of a head from turned_items on are copied
  int items;

  static __device__ __forceinline__ int turned_of(const Rotary& rot, int layout) {
    return layout == kHalves ? rot.dim / 2 / N : (layout == kPairs ? (rot.dim + N - 1) / N : rot.dim / 2);
  }
  static __device__ __forceinline__ int items_of(const Rotary& rot, int layout, int D, bool in_place) {
    const int t = turned_of(rot, layout);
    if (in_place) return t;  // what is not turned is there
    return t + (layout == kSingle ? D - rot.dim : (layout == kPairs ? D / N - t : (D - rot.dim) / N));
  }
  // the block's rows from x and y on
  __device__ __forceinline__ Heads(const T* x, int64_t ldx, T* y, int64_t ldy, int h0, int heads, int D, const Rotary& rot)
      : x(x), y(y), ldx(ldx), ldy(ldy), h0(h0), D(D), half(rot.dim / 2), layout(layout_of<T>(rot.dim, rot.interleaved)),
        turned_items(turned_of(rot, layout)), heads(heads), items(items_of(rot, layout, D, x == y && ldx == ldy)) {}
  __device__ __forceinline__ int64_t offset(const Walk& w, int64_t ld) const { return w.r * ld + (h0 + w.h) * D + w.i * N; }
  // neighbours: 16 bytes
  __device__ __forceinline__ void turn_pairs(uint4 u, const Walk& w, const float* cs) const {
    float v[N];
    widen<T>(u, v);
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      const int p = w.i * (N / 2) + j;
      if (p < half) {
        const float2 t = moe::turn(v[2 * j], v[2 * j + 1], cs[p], cs[half + p]);
        v[2 * j] = t.x;
        v[2 * j + 1] = t.y;
      }
    }
    *reinterpret_cast<uint4*>(y + offset(w, ldy)) = narrow<T>(v);
  }
  template <int LAYOUT>
  __device__ __forceinline__ void turn(const Walk& w, const float* cs) const {
    const int column = (h0 + w.h) * D;
    const T* from = x + w.r * ldx + column;
    T* to = y + w.r * ldy + column;
    if constexpr (LAYOUT == kHalves) {
      if (w.i < turned_items) {
        float u[N], v[N], c[N], s[N];
        widen<T>(load16(from + w.i * N), u);
        widen<T>(load16(from + half + w.i * N), v);
#pragma unroll
        for (int j = 0; j < N; j += 4) {
          *reinterpret_cast<float4*>(c + j) = *reinterpret_cast<const float4*>(cs + w.i * N + j);
          *reinterpret_cast<float4*>(s + j) = *reinterpret_cast<const float4*>(cs + half + w.i * N + j);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float2 t = moe::turn(u[j], v[j], c[j], s[j]);
          u[j] = t.x;
          v[j] = t.y;
        }
        *reinterpret_cast<uint4*>(to + w.i * N) = narrow<T>(u);
        *reinterpret_cast<uint4*>(to + half + w.i * N) = narrow<T>(v);
      } else {
        *reinterpret_cast<uint4*>(to + (w.i + turned_items) * N) = load16(from + (w.i + turned_items) * N);
      }
    } else {
      if (w.i < half) {
        const float2 t = moe::turn(value(from + w.i), value(from + half + w.i), cs[w.i], cs[half + w.i]);
        to[w.i] = static_cast<T>(t.x);
        to[half + w.i] = static_cast<T>(t.y);
      } else {
        to[half + w.i] = from[half + w.i];  // items past the pairs are the columns from dim on
      }
    }
  }
  // Rows that are not ok are left as they are.
  template <int LAYOUT>
  __device__ __forceinline__ void turn(int rows, const int* ok, const float* cs) const {
    if constexpr (LAYOUT == kPairs) {
      // (two items' loads at once: 16 bytes a thread are too few in flight, 59.7 us of the above)
      for (Walk w(heads, items); w.r < rows; w.next()) {
        const Walk first = w;
        const bool one = ok[w.r];
        uint4 u, v;
        if (one) u = load16(x + offset(w, ldx));
        w.next();
        const bool two = w.r < rows && ok[w.r];
        if (two) v = load16(x + offset(w, ldx));
        if (one) turn_pairs(u, first, cs + first.r * 2 * half);
        if (two) turn_pairs(v, w, cs + w.r * 2 * half);
      }
    } else {
      for (Walk w(heads, items); w.r < rows; w.next())
        if (ok[w.r]) turn<LAYOUT>(w, cs + w.r * 2 * half);
    }
  }
  __device__ __forceinline__ void turn(int rows, const int* ok, const float* cs) const {
    if (heads == 0) return;
    switch (layout) {
      case kHalves: return turn<kHalves>(rows, ok, cs);
      case kPairs: return turn<kPairs>(rows, ok, cs);
      default: return turn<kSingle>(rows, ok, cs);
    }
  }
};

// this block's share of `heads` heads
__device__ __forceinline__ int2 share(int heads) {
  return make_int2(static_cast<int>(static_cast<int64_t>(heads) * blockIdx.y / gridDim.y),
                   static_cast<int>(static_cast<int64_t>(heads) * (blockIdx.y + 1) / gridDim.y));
}
// The table into shared memory, while a row's place is looked for.
__device__ __forceinline__ void load_table(float4* table) {
  static_assert(kRotThreads == 256, "one entry a thread");
  table[threadIdx.x] = __ldg(reinterpret_cast<const float4*>(kTurnTable.cs[threadIdx.x]));
}
// the rows' cosines, half of them a row, and sines
__device__ __forceinline__ void angles(const Rotary& rot, const int* pos, int rows, const float4* table, float* cs) {
  const int half = rot.dim / 2;
  if (half == 0) return;
  int r = quotient(threadIdx.x, half), i = threadIdx.x - r * half;
  const int dr = quotient(kRotThreads, half), di = kRotThreads - dr * half;
  while (r < rows) {
    const float2 w = turned(rot, i, pos[r], table);
    cs[r * 2 * half + i] = w.x;
    cs[r * 2 * half + half + i] = w.y;
    i += di;
    r += dr;
    if (i >= half) {
      i -= half;
      ++r;
    }
  }
}

template <class T>
__global__ void __launch_bounds__(kRotThreads, 8)
    rotary_kernel(Rotary rot, const int32_t* __restrict__ pos, const T* x, int64_t ldx, T* y, int64_t ldy, int n_rows, int heads,
                  int D, int per_block) {
  extern __shared__ __align__(16) float cs[];
  __shared__ int ok[kMostRows], s_pos[kMostRows];
  __shared__ float4 table[256];
  load_table(table);
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * per_block;
  const int rows = static_cast<int>(min(static_cast<int64_t>(per_block), n_rows - row0));
  if (threadIdx.x < rows) {
    s_pos[threadIdx.x] = __ldg(pos + row0 + threadIdx.x);
    ok[threadIdx.x] = 1;
  }
  __syncthreads();
  angles(rot, s_pos, rows, table, cs);
  __syncthreads();
  const int2 hs = share(heads);
  Heads<T>(x + row0 * ldx, ldx, y + row0 * ldy, ldy, hs.x, hs.y - hs.x, D, rot).turn(rows, ok, cs);
}

// Values 8 o .. 8 o + 7 of a head, turned.
template <class T>
__device__ __forceinline__ void turn8(const T* from, int o, const Rotary& rot, const float* cs, float* v) {
  const int half = rot.dim / 2;
  if (8 * o >= rot.dim) return;
  if (half % 8 == 0 && !rot.interleaved) {
    const bool first = 8 * o < half;
    float u[8], c[8], s[8];
    load8<T>(from + 8 * o + (first ? half : -half), u);
    const float* at = cs + 8 * o - (first ? 0 : half);
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      *reinterpret_cast<float4*>(c + j) = *reinterpret_cast<const float4*>(at + j);
      *reinterpret_cast<float4*>(s + j) = *reinterpret_cast<const float4*>(at + half + j);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = first ? turn(v[j], u[j], c[j], s[j]).x : turn(u[j], v[j], c[j], s[j]).y;
  } else if (rot.interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (4 * o + j >= half) break;
      const float2 t = turn(v[2 * j], v[2 * j + 1], cs[4 * o + j], cs[half + 4 * o + j]);
      v[2 * j] = t.x;
      v[2 * j + 1] = t.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = 8 * o + j;
      if (e < half)
        v[j] = turn(v[j], value(from + e + half), cs[e], cs[half + e]).x;
      else if (e < rot.dim)
        v[j] = turn(value(from + e - half), v[j], cs[e - half], cs[e]).y;
    }
  }
}

// the lesser and the larger; NaN if either is
__device__ __forceinline__ float least(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float most(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The codes of sixteen values of a group that four neighbouring lanes hold, and the
// group's scale and offset as one word.
// A code is d / s rounded to the nearest whole number, to the even one of two as near,
// with d = v - b. A division for each takes more time (77 us against 68 in all for the
// prompts above): n is rounded from d / s less 2^-20 of it, so it is the code or the whole number below, and the code
// is above if d - n s is more than s / 2, or as much and n is odd. That remainder is
// exact: it is a multiple of d's or s's last place, and s has eight bits.
__device__ __forceinline__ uint2 quantised(const float* v, uint32_t* meta) {
  const unsigned int lanes = 0xFu << (threadIdx.x & 28);
  constexpr float kMost = 0x1p126f, kWhole = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number
  float lo = v[0], hi = v[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) {
    lo = least(lo, v[i]);
    hi = most(hi, v[i]);
  }
#pragma unroll
  for (int x = 1; x < 4; x <<= 1) {
    lo = least(lo, __shfl_xor_sync(lanes, lo, x));
    hi = most(hi, __shfl_xor_sync(lanes, hi, x));
  }
  if (!(lo >= -kMost && hi <= kMost)) {
    *meta = 0x7FC07FC0u;
    return make_uint2(0u, 0u);
  }
  const __nv_bfloat16 b16 = __float2bfloat16_rn(lo);
  const float b = __bfloat162float(b16);
  const __nv_bfloat16 s16 = __float2bfloat16_rn((hi - b) * (1.f / 15.f));
  const float s = __bfloat162float(s16);
  const uint32_t offset = static_cast<uint32_t>(__bfloat16_as_ushort(b16)) << 16;
  *meta = offset;
  if (!(s > 0.f)) return make_uint2(0u, 0u);
  *meta = offset | __bfloat16_as_ushort(s16);
  uint32_t w[2] = {0u, 0u};
  if (s < 0x1p-100f) {  // (1 / s may be infinite, and s be short of bits)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[0] |= static_cast<uint32_t>(fminf(fmaxf(rintf(__fdiv_rn(v[i] - b, s)), 0.f), 15.f)) << (4 * i);
      w[1] |= static_cast<uint32_t>(fminf(fmaxf(rintf(__fdiv_rn(v[8 + i] - b, s)), 0.f), 15.f)) << (4 * i);
    }
    return make_uint2(w[0], w[1]);
  }
  const float inv = __frcp_rn(s) * (1.f - 0x1p-20f);
  const int half = __float_as_int(0.5f * s);
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const float2 d = both(add2(f2(v[i], v[i + 1]), f2(-b, -b)));
    const F2 dd = f2(fmaxf(d.x, 0.f), fmaxf(d.y, 0.f)), mm = fma2(dd, f2(inv, inv), f2(kWhole, kWhole));
    const float2 m = both(mm), rest = both(fma2(add2(mm, f2(-kWhole, -kWhole)), f2(-s, -s), dd));
    int n0 = __float_as_int(m.x), n1 = __float_as_int(m.y);
    if (__float_as_int(rest.x) + (n0 & 1) > half) ++n0;  // (a negative rest is a negative integer)
    if (__float_as_int(rest.y) + (n1 & 1) > half) ++n1;
    w[i / 8] += static_cast<uint32_t>(n0) << (4 * (i & 7));  // n is 0x4B400000 and the code, at most 15
    w[i / 8] += static_cast<uint32_t>(n1) << (4 * (i & 7) + 4);
  }
  constexpr uint32_t kRaised = 0x4B400000u * 0x11111111u;
  return make_uint2(w[0] - kRaised, w[1] - kRaised);
}

struct WriteArgs {
  Kv kv;
  Rotary rot;  // dim 0: there is no q, and k is stored as it is
  const void *q, *k, *v;
  void *q_out, *pk, *pv;  // pages of the layer
  int64_t ldq, ldqo, ldk, ldv;
  const int32_t *seqs, *cu;
  int n, n_rows, Hq, H, D, per_block;
  uint32_t number;
};

// A warp a row finds its place, then q's heads are turned and k and v are stored,
// eight values a thread at a time, or for codes sixteen: items of k's heads, then of
// v's. (Sixteen need 48 registers, five blocks on an SM: 60 us for the prompts above;
// with six blocks 61, with eight 63, as with eight values.)
template <class T, bool CODES>
__global__ void __launch_bounds__(kRotThreads, CODES ? 5 : 8) write_rotary_kernel(const WriteArgs a) {
  extern __shared__ __align__(16) float cs[];
  __shared__ int ok[kMostRows], s_pos[kMostRows], s_page[kMostRows];
  __shared__ float4 table[256];
  if (a.q) load_table(table);
  const Kv& kv = a.kv;
  const int row0 = blockIdx.x * a.per_block, rows = min(a.per_block, a.n_rows - row0), half = a.rot.dim / 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool stop = pending(kv, true, a.number);
  if (warp < rows) {
    const int row = row0 + warp, lo = chunk_of(a.cu, a.n, row, lane);
    Place p = place_of<true>(kv, a.seqs, a.cu, lo, a.n_rows, row);
    if (!stop && blockIdx.y == 0) {
      // tokens that the rows do not reach (of a chunk that no row is in, too)
      if (row == 0 && __ldg(a.cu + a.n) > a.n_rows) record_late(kv, a.number, MOE_DEVERR_BADIDX, lane);
      if (p.why) record_late(kv, a.number, p.why, lane);
    }
    if (lane == 0) {
      ok[warp] = p.page >= 0;
      s_pos[warp] = p.pos;
      s_page[warp] = p.page;
    }
  }
  // (warps read the word of errors at different times, and a block goes one way)
  if (__syncthreads_or(stop)) return;
  angles(a.rot, s_pos, rows, table, cs);
  __syncthreads();
  if (a.q) {
    const int2 hs = share(a.Hq);
    Heads<T>(static_cast<const T*>(a.q) + row0 * a.ldq, a.ldq, static_cast<T*>(a.q_out) + row0 * a.ldqo, a.ldqo, hs.x, hs.y - hs.x,
             a.D, a.rot)
        .turn(rows, ok, cs);
  }
  const int2 hs = share(a.H);
  const int heads = hs.y - hs.x;
  if (heads == 0) return;
  constexpr int kItem = CODES ? 16 : 8;  // values
  for (Walk w(2 * heads, a.D / kItem); w.r < rows; w.next()) {
    if (!ok[w.r]) continue;  // (a group's lanes are of one row)
    const bool is_v = w.h >= heads;
    const T* from = static_cast<const T*>(is_v ? a.v : a.k) + (row0 + w.r) * (is_v ? a.ldv : a.ldk) +
                    (hs.x + w.h - (is_v ? heads : 0)) * a.D;
    float v[kItem];
#pragma unroll
    for (int j = 0; j < kItem / 8; ++j) {
      const int octet = w.i * (kItem / 8) + j;
      load8<T>(from + 8 * octet, v + 8 * j);
      if (!is_v) turn8<T>(from, octet, a.rot, cs + w.r * 2 * half, v + 8 * j);
    }
    char* pages = static_cast<char*>(is_v ? a.pv : a.pk);
    const int64_t block = static_cast<int64_t>(s_page[w.r]) * a.H + hs.x + w.h - (is_v ? heads : 0);
    const int place = s_pos[w.r] & (kv.page - 1);
    if constexpr (CODES) {
      uint32_t meta;
      const uint2 codes = quantised(v, &meta);
      const int row_bytes = a.D / 2, meta_bytes = a.D / 16;
      char* to = pages + ((block * (row_bytes + meta_bytes)) << kv.page_shift);
      *reinterpret_cast<uint2*>(to + place * row_bytes + 8 * w.i) = codes;
      if ((w.i & 3) == 0)
        *reinterpret_cast<uint32_t*>(to + (row_bytes << kv.page_shift) + place * meta_bytes + w.i) = meta;
    } else {
      store8<T>(reinterpret_cast<T*>(pages) + ((block << kv.page_shift) + place) * a.D + 8 * w.i, v);
    }
  }
}

// 2^(23 - 4 j), and that and code j < 5 of w
__device__ __forceinline__ float one_of(int j) { return __uint_as_float(0x4B000000u - (j << 25)); }
__device__ __forceinline__ float code_in(uint32_t w, int j) {
  return __uint_as_float((w & (15u << (4 * j))) | (0x4B000000u - (j << 25)));
}
// the values of a word of codes
template <class T>
__device__ __forceinline__ void store_values(T* to, uint32_t c, float s, float b) {
  float v[8];
  // a code in its place in the fraction of 2^(23 - 4 j) adds the code to it
  const uint32_t c5 = c >> 20;
  const F2 ss = f2(s, s), bb = f2(b, b);
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const int j0 = j < 5 ? j : j - 5, j1 = j < 4 ? j + 1 : j - 4;
    const F2 u = f2(code_in(j < 5 ? c : c5, j0), code_in(j < 4 ? c : c5, j1));
    const float2 x = both(fma2(add2(u, f2(-one_of(j0), -one_of(j1))), ss, bb));
    v[j] = x.x;
    v[j + 1] = x.y;
  }
  store8<T>(to, v);
}
// The newest tokens of sequences out of their pages, eight values a thread, or
// sixteen codes (of the 60 us above two less than with eight).
template <class T, bool CODES>
__global__ void __launch_bounds__(kRotThreads) read_kernel(const WriteArgs a) {
  __shared__ int s_pos[kMostRows], s_page[kMostRows];
  const Kv& kv = a.kv;
  const int row0 = blockIdx.x * a.per_block, rows = min(a.per_block, a.n_rows - row0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < rows) {
    const int row = row0 + warp, lo = chunk_of(a.cu, a.n, row, lane);
    const Place p = place_of<false>(kv, a.seqs, a.cu, lo, a.n_rows, row);
    if (lane == 0 && blockIdx.y == 0) {
      const uint32_t why = p.why | (row == 0 && __ldg(a.cu + a.n) > a.n_rows ? MOE_DEVERR_BADIDX : 0u);
      if (why) atomicOr(&kv.work->err, why);
    }
    if (lane == 0) {
      s_pos[warp] = p.pos;
      s_page[warp] = p.page;
    }
  }
  __syncthreads();
  const int2 hs = share(a.H);
  const int heads = hs.y - hs.x;
  if (heads == 0) return;
  constexpr int kItem = CODES ? 16 : 8;  // values
  for (Walk w(2 * heads, a.D / kItem); w.r < rows; w.next()) {
    if (s_page[w.r] < 0) continue;
    const bool is_v = w.h >= heads;
    const int h = hs.x + w.h - (is_v ? heads : 0);
    const char* pages = static_cast<const char*>(is_v ? a.pv : a.pk);
    const int64_t block = static_cast<int64_t>(s_page[w.r]) * a.H + h;
    const int place = s_pos[w.r] & (kv.page - 1);
    T* to = static_cast<T*>(const_cast<void*>(is_v ? a.v : a.k)) + (row0 + w.r) * (is_v ? a.ldv : a.ldk) + h * a.D + kItem * w.i;
    if constexpr (CODES) {
      const int row_bytes = a.D / 2, meta_bytes = a.D / 16;
      const char* from = pages + ((block * (row_bytes + meta_bytes)) << kv.page_shift);
      const uint2 c = *reinterpret_cast<const uint2*>(from + place * row_bytes + 8 * w.i);
      const uint32_t m = *reinterpret_cast<const uint32_t*>(from + (row_bytes << kv.page_shift) + place * meta_bytes + w.i / 4 * 4);
      const float s = __uint_as_float(m << 16), b = __uint_as_float(m & 0xFFFF0000u);
      store_values<T>(to, c.x, s, b);
      store_values<T>(to + 8, c.y, s, b);
    } else {
      const T* from = reinterpret_cast<const T*>(pages) + ((block << kv.page_shift) + place) * a.D + 8 * w.i;
#pragma unroll
      for (int j = 0; j < 8; j += Vec<T>::N) *reinterpret_cast<uint4*>(to + j) = load16(from + j);
    }
  }
}

// Rows a block and blocks a row: four rows share a block's latencies once there are
// blocks enough (the prompts above: 76 us with two, 68 with eight, of which an SM gets
// six or seven at once and no more), and a row is cut by its heads while blocks are short
// of the SMs and have work for their threads.
struct Shape {
  int per_block;
  dim3 grid;
};
Shape shape_of(int64_t rows, int heads, int64_t row_items, int num_sms) {
  Shape s;
  s.per_block = rows >= 8ll * num_sms ? kMostRows : 1;
  const int64_t cut = std::min<int64_t>(std::min<int64_t>(heads, row_items / kRotThreads), 2ll * num_sms / std::max<int64_t>(1, rows));
  s.grid = dim3(static_cast<unsigned>((rows + s.per_block - 1) / s.per_block), static_cast<unsigned>(std::max<int64_t>(1, cut)));
  return s;
}

template <class T>
cudaError_t rotary(const Rotary& rot, const int32_t* pos, const void* x, int64_t ldx, void* y, int64_t ldy, int32_t rows,
                   int32_t heads, int32_t D, int num_sms, cudaStream_t st) {
  const Shape s = shape_of(rows, heads, static_cast<int64_t>(heads) * D / Vec<T>::N, num_sms);
  rotary_kernel<T><<<s.grid, kRotThreads, s.per_block * rot.dim * sizeof(float), st>>>(
      rot, pos, static_cast<const T*>(x), ldx, static_cast<T*>(y), ldy, rows, heads, D, s.per_block);
  return cudaGetLastError();
}

WriteArgs args_of(const moe_kv_t& a, const KvLayout& l, int32_t layer, const int32_t* seqs, const int32_t* cu, int32_t n,
                  int32_t n_rows) {
  WriteArgs w{};
  const int64_t off = layer * layer_bytes(a);
  w.kv = kv_of(a, l);
  w.pk = static_cast<char*>(a.k) + off;
  w.pv = static_cast<char*>(a.v) + off;
  w.seqs = seqs;
  w.cu = cu;
  w.n = n;
  w.n_rows = n_rows;
  w.H = a.n_kv_heads;
  w.D = a.head_dim;
  return w;
}

}  // namespace

cudaError_t launch_rotary(const Rotary& rot, const int32_t* pos, const void* x, int32_t xt, int64_t ldx, void* y, int64_t ldy,
                          int32_t rows, int32_t heads, int32_t D, int num_sms, cudaStream_t st) {
  return xt == MOE_F32 ? rotary<float>(rot, pos, x, ldx, y, ldy, rows, heads, D, num_sms, st)
                       : rotary<__nv_bfloat16>(rot, pos, x, ldx, y, ldy, rows, heads, D, num_sms, st);
}

cudaError_t launch_kv_write_rotary(const moe_kv_t& a, const KvLayout& l, int32_t layer, const Rotary& rot, const void* q,
                                   int64_t ldq, int32_t n_heads, void* q_out, int64_t ldqo, const void* k, int64_t ldk,
                                   const void* v, int64_t ldv, const int32_t* seqs, const int32_t* cu, int32_t n, int32_t n_rows,
                                   int num_sms, cudaStream_t st) {
  WriteArgs w = args_of(a, l, layer, seqs, cu, n, n_rows);
  w.rot = rot;
  w.q = q;
  w.ldq = ldq;
  w.Hq = n_heads;
  w.q_out = q_out;
  w.ldqo = ldqo;
  w.k = k;
  w.ldk = ldk;
  w.v = v;
  w.ldv = ldv;
  w.number = next_write();
  const Shape s = shape_of(n_rows, std::max(n_heads, a.n_kv_heads), (n_heads + 2ll * a.n_kv_heads) * a.head_dim / 8, num_sms);
  w.per_block = s.per_block;
  const size_t smem = s.per_block * rot.dim * sizeof(float);
  const bool codes = a.dtype & MOE_KV_I4, f32 = token_type(a) == MOE_F32;
  if (codes && f32)
    write_rotary_kernel<float, true><<<s.grid, kRotThreads, smem, st>>>(w);
  else if (codes)
    write_rotary_kernel<__nv_bfloat16, true><<<s.grid, kRotThreads, smem, st>>>(w);
  else if (f32)
    write_rotary_kernel<float, false><<<s.grid, kRotThreads, smem, st>>>(w);
  else
    write_rotary_kernel<__nv_bfloat16, false><<<s.grid, kRotThreads, smem, st>>>(w);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const moe_kv_t& a, const KvLayout& l, int32_t layer, void* k, int64_t ldk, void* v, int64_t ldv,
                           const int32_t* seqs, const int32_t* cu, int32_t n, int32_t n_rows, int num_sms, cudaStream_t st) {
  WriteArgs w = args_of(a, l, layer, seqs, cu, n, n_rows);
  w.k = k;
  w.ldk = ldk;
  w.v = v;
  w.ldv = ldv;
  const Shape s = shape_of(n_rows, a.n_kv_heads, 2ll * a.n_kv_heads * a.head_dim / 8, num_sms);
  w.per_block = s.per_block;
  const bool codes = a.dtype & MOE_KV_I4, f32 = token_type(a) == MOE_F32;
  if (codes && f32)
    read_kernel<float, true><<<s.grid, kRotThreads, 0, st>>>(w);
  else if (codes)
    read_kernel<__nv_bfloat16, true><<<s.grid, kRotThreads, 0, st>>>(w);
  else if (f32)
    read_kernel<float, false><<<s.grid, kRotThreads, 0, st>>>(w);
  else
    read_kernel<__nv_bfloat16, false><<<s.grid, kRotThreads, 0, st>>>(w);
  return cudaGetLastError();
}

}  // namespace moe
