// Rotary positions, and a step's keys and values written into the paged cache with
// the rotation on the way; values read back from pages.
//
// The pair (a, b) = (x_i, x_i+dim/2) or (x_2i, x_2i+1) of a head at position p
// becomes (a c - b s, b c + a s) with c, s = magnitude times cos, sin of p f_i.
// p f_i reaches 10^6 radians, of which fp32 would keep a sixteenth: the frequencies
// are given in turns as 64-bit fractions, so that p times one wraps whole turns
// away exactly, and what is left is rounded to fp32 once. Rotation is in fp32, one
// rounding to the type of the result (none before 4-bit codes).
//
// Pages of 4-bit codes: eight threads hold a group of 64 values; with lo and hi its
// least and largest, b = bf16(lo), s = bf16((hi - b) / 15), q = round((x - b) / s)
// within 0..15 (0 where s is 0), divisions and rounding as in IEEE. A group with an
// infinity, a NaN or a magnitude above 2^126 becomes NaN as a whole.
//
// What bounds them: one row the latency of its lookups (chunk, sequence, length,
// table, page count: five dependent reads) and of one sine; prompts HBM. A row's
// sines and cosines are formed once and shared by its heads; a thread owns both
// halves of a pair, so that a result may overwrite its input.
#include <cuda_bf16.h>

#include "kv_device.cuh"

namespace moe {
namespace {

constexpr int kRotThreads = 256, kMostRows = 4;

template <class T>
struct Vec {
  static constexpr int N = 16 / static_cast<int>(sizeof(T));
};
template <class T, int N>
__device__ __forceinline__ void load(const T* p, float* v) {
#pragma unroll
  for (int i = 0; i < N; i += Vec<T>::N) {
    const uint4 u = *reinterpret_cast<const uint4*>(p + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 4) {
        v[i + j] = __uint_as_float(w[j]);
      } else {
        v[i + 2 * j] = __uint_as_float(w[j] << 16);
        v[i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  }
}
template <class T, int N>
__device__ __forceinline__ void store(T* p, const float* v) {
#pragma unroll
  for (int i = 0; i < N; i += Vec<T>::N) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 4) {
        w[j] = __float_as_uint(v[i + j]);
      } else {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[i + 2 * j], v[i + 2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    *reinterpret_cast<uint4*>(p + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
template <class T>
__device__ __forceinline__ float value(const T* p) {
  return static_cast<float>(*p);
}

// magnitude times (cos, sin) of a position's angle
__device__ __forceinline__ float2 turned(const Rotary& rot, int i, int pos) {
  const int64_t t = static_cast<int64_t>(__ldg(rot.turns + i) * static_cast<uint64_t>(static_cast<int64_t>(pos)));
  float s, c;  // t / 2^63 half turns in [-1, 1)
  sincospif(__ll2float_rn(t) * 0x1p-63f, &s, &c);
  return make_float2(c * rot.magnitude, s * rot.magnitude);
}

// How a head's values are dealt out: halves whose vectors match, neighbours, or
// halves of other sizes, value by value.
enum { kHalves = 0, kPairs = 1, kSingle = 2 };
template <class T>
__host__ __device__ __forceinline__ int layout_of(int dim, int interleaved) {
  return interleaved ? kPairs : ((dim / 2) % Vec<T>::N ? kSingle : kHalves);
}

// Heads [h0, h1) of the block's rows from x to y, turned by cs. Rows that are not
// ok are left as they are.
template <class T, int LAYOUT>
__device__ __forceinline__ void turn_heads(const T* x, int64_t ldx, T* y, int64_t ldy, int64_t row0, int rows, const int* ok,
                                           int h0, int h1, int D, int dim, const float2* cs) {
  constexpr int N = Vec<T>::N;
  const int half = dim / 2, heads = h1 - h0;
  const bool in_place = x == y && ldx == ldy;  // what is not turned is there
  const int turned_items = LAYOUT == kHalves ? half / N : (LAYOUT == kPairs ? (dim + N - 1) / N : half);
  const int rest = LAYOUT == kSingle ? D - dim : (LAYOUT == kPairs ? D / N - turned_items : (D - dim) / N);
  const int per = turned_items + (in_place ? 0 : rest);
  if (heads <= 0 || per == 0) return;
  // (row, head, item) of this thread, and the way to its next one
  int r = threadIdx.x / (heads * per), h = threadIdx.x / per % heads, i = threadIdx.x % per;
  const int dr = kRotThreads / (heads * per), dh = kRotThreads / per % heads, di = kRotThreads % per;
  while (r < rows) {
    if (ok[r]) {
      const int64_t at = static_cast<int64_t>(h0 + h) * D;
      const T* from = x + (row0 + r) * ldx + at;
      T* to = y + (row0 + r) * ldy + at;
      const float2* t = cs + r * half;
      if constexpr (LAYOUT == kHalves) {
        if (i < turned_items) {
          float a[N], b[N];
          load<T, N>(from + i * N, a);
          load<T, N>(from + half + i * N, b);
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const float2 w = t[i * N + j];
            const float u = a[j] * w.x - b[j] * w.y;
            b[j] = b[j] * w.x + a[j] * w.y;
            a[j] = u;
          }
          store<T, N>(to + i * N, a);
          store<T, N>(to + half + i * N, b);
        } else {
          const int e = dim + (i - turned_items) * N;
          *reinterpret_cast<uint4*>(to + e) = *reinterpret_cast<const uint4*>(from + e);
        }
      } else if constexpr (LAYOUT == kPairs) {
        float a[N];
        load<T, N>(from + i * N, a);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          const int p = i * (N / 2) + j;
          if (p < half) {
            const float2 w = t[p];
            const float u = a[2 * j] * w.x - a[2 * j + 1] * w.y;
            a[2 * j + 1] = a[2 * j + 1] * w.x + a[2 * j] * w.y;
            a[2 * j] = u;
          }
        }
        store<T, N>(to + i * N, a);
      } else {
        if (i < half) {
          const float a = value(from + i), b = value(from + half + i);
          const float2 w = t[i];
          to[i] = static_cast<T>(a * w.x - b * w.y);
          to[half + i] = static_cast<T>(b * w.x + a * w.y);
        } else {
          to[half + i] = from[half + i];  // items past the pairs are the columns from dim on
        }
      }
    }
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
}
template <class T>
__device__ __forceinline__ void turn_heads(const T* x, int64_t ldx, T* y, int64_t ldy, int64_t row0, int rows, const int* ok,
                                           int h0, int h1, int D, const Rotary& rot, const float2* cs) {
  switch (layout_of<T>(rot.dim, rot.interleaved)) {
    case kHalves: return turn_heads<T, kHalves>(x, ldx, y, ldy, row0, rows, ok, h0, h1, D, rot.dim, cs);
    case kPairs: return turn_heads<T, kPairs>(x, ldx, y, ldy, row0, rows, ok, h0, h1, D, rot.dim, cs);
    default: return turn_heads<T, kSingle>(x, ldx, y, ldy, row0, rows, ok, h0, h1, D, rot.dim, cs);
  }
}

// this block's share of `heads` heads
__device__ __forceinline__ int2 share(int heads) {
  return make_int2(static_cast<int>(static_cast<int64_t>(heads) * blockIdx.y / gridDim.y),
                   static_cast<int>(static_cast<int64_t>(heads) * (blockIdx.y + 1) / gridDim.y));
}

template <class T>
__global__ void __launch_bounds__(kRotThreads)
    rotary_kernel(Rotary rot, const int32_t* __restrict__ pos, const T* x, int64_t ldx, T* y, int64_t ldy, int n_rows, int heads,
                  int D, int per_block) {
  extern __shared__ float2 cs[];
  __shared__ int ok[kMostRows];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * per_block;
  const int rows = static_cast<int>(min(static_cast<int64_t>(per_block), n_rows - row0)), half = rot.dim / 2;
  if (threadIdx.x < kMostRows) ok[threadIdx.x] = 1;
  for (int e = threadIdx.x; e < rows * half; e += kRotThreads) cs[e] = turned(rot, e % half, __ldg(pos + row0 + e / half));
  __syncthreads();
  const int2 hs = share(heads);
  turn_heads<T>(x, ldx, y, ldy, row0, rows, ok, hs.x, hs.y, D, rot, cs);
}

// Values 8 o .. 8 o + 7 of a head, turned.
template <class T>
__device__ __forceinline__ void turned8(const T* from, int o, const Rotary& rot, const float2* t, float* v) {
  load<T, 8>(from + 8 * o, v);
  const int half = rot.dim / 2;
  if (8 * o >= rot.dim) return;
  if (rot.interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (4 * o + j >= half) break;
      const float2 w = t[4 * o + j];
      const float u = v[2 * j] * w.x - v[2 * j + 1] * w.y;
      v[2 * j + 1] = v[2 * j + 1] * w.x + v[2 * j] * w.y;
      v[2 * j] = u;
    }
  } else if (half % 8 == 0) {
    const bool first = 8 * o < half;
    float b[8];
    load<T, 8>(from + 8 * o + (first ? half : -half), b);
    const float2* w = t + 8 * o - (first ? 0 : half);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = first ? v[j] * w[j].x - b[j] * w[j].y : v[j] * w[j].x + b[j] * w[j].y;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = 8 * o + j;
      if (e < half)
        v[j] = v[j] * t[e].x - value(from + e + half) * t[e].y;
      else if (e < rot.dim)
        v[j] = v[j] * t[e - half].x + value(from + e - half) * t[e - half].y;
    }
  }
}

// The codes of eight values of a group that eight neighbouring lanes hold, and the
// group's scale and offset as one word.
__device__ __forceinline__ uint32_t quantised(const float* v, uint32_t* meta) {
  const unsigned int lanes = 0xFFu << (threadIdx.x & 24);
  constexpr float kMost = 0x1p126f;
  float lo = v[0], hi = v[0];
  bool fine = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, v[i]);
    hi = fmaxf(hi, v[i]);
    fine &= fabsf(v[i]) <= kMost;
  }
#pragma unroll
  for (int x = 1; x < 8; x <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(lanes, lo, x));
    hi = fmaxf(hi, __shfl_xor_sync(lanes, hi, x));
  }
  fine = __all_sync(lanes, fine);
  const __nv_bfloat16 b16 = __float2bfloat16_rn(lo);
  const float b = __bfloat162float(b16);
  const __nv_bfloat16 s16 = __float2bfloat16_rn(__fdiv_rn(hi - b, 15.f));
  const float s = __bfloat162float(s16);
  uint32_t w = 0;
  if (fine && s > 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w |= static_cast<uint32_t>(fminf(fmaxf(rintf(__fdiv_rn(v[i] - b, s)), 0.f), 15.f)) << (4 * i);
  }
  *meta = fine ? static_cast<uint32_t>(__bfloat16_as_ushort(s > 0.f ? s16 : __float2bfloat16_rn(0.f))) |
                     static_cast<uint32_t>(__bfloat16_as_ushort(b16)) << 16
               : 0x7FC07FC0u;
  return w;
}

struct WriteArgs {
  Kv kv;
  Rotary rot;  // dim 0: k is stored as it is
  const void *q, *k, *v;
  void *q_out, *pk, *pv;  // pages of the layer
  int64_t ldq, ldqo, ldk, ldv;
  const int32_t *seqs, *cu;
  int n, n_rows, Hq, H, D, per_block;
  uint32_t number;
};

// One to four rows a block: a warp a row finds its place, then q's heads are
// turned and k and v are stored, eight values a thread at a time.
template <class T, bool CODES>
__global__ void __launch_bounds__(kRotThreads) write_rotary_kernel(const WriteArgs a) {
  extern __shared__ float2 cs[];
  __shared__ int ok[kMostRows], s_pos[kMostRows], s_page[kMostRows];
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
  for (int e = threadIdx.x; e < rows * half; e += kRotThreads) {
    const int r = e / half;
    cs[e] = turned(a.rot, e - r * half, s_pos[r]);
  }
  __syncthreads();
  if (a.q) {
    const int2 hs = share(a.Hq);
    turn_heads<T>(static_cast<const T*>(a.q), a.ldq, static_cast<T*>(a.q_out), a.ldqo, row0, rows, ok, hs.x, hs.y, a.D, a.rot, cs);
  }
  // k and v: items (row, k or v, head, octet); the octets of a group are neighbouring lanes'
  const int2 hs = share(a.H);
  const int heads = hs.y - hs.x, octets = a.D / 8, per_row = 2 * heads * octets;
  for (int e = threadIdx.x; e < rows * per_row; e += kRotThreads) {
    int i = e;
    const int r = i / per_row;
    i -= r * per_row;
    const int is_v = i >= heads * octets;
    i -= is_v * heads * octets;
    const int h = i / octets, o = i - h * octets;
    if (!ok[r]) continue;  // (a group's lanes are of one row)
    const T* from = static_cast<const T*>(is_v ? a.v : a.k) + static_cast<int64_t>(row0 + r) * (is_v ? a.ldv : a.ldk) +
                    static_cast<int64_t>(hs.x + h) * a.D;
    float v[8];
    if (is_v)
      load<T, 8>(from + 8 * o, v);
    else
      turned8<T>(from, o, a.rot, cs + r * half, v);
    char* pages = static_cast<char*>(is_v ? a.pv : a.pk);
    const int64_t block = static_cast<int64_t>(s_page[r]) * a.H + hs.x + h;
    const int place = s_pos[r] & (kv.page - 1);
    if constexpr (CODES) {
      uint32_t meta;
      const uint32_t w = quantised(v, &meta);
      const int row_bytes = a.D / 2, meta_bytes = a.D / 16;
      char* at = pages + ((block * (row_bytes + meta_bytes)) << kv.page_shift);
      *reinterpret_cast<uint32_t*>(at + place * row_bytes + 4 * o) = w;
      if ((o & 7) == 0)
        *reinterpret_cast<uint32_t*>(at + (row_bytes << kv.page_shift) + place * meta_bytes + o / 2) = meta;
    } else {
      store<T, 8>(reinterpret_cast<T*>(pages) + ((block << kv.page_shift) + place) * a.D + 8 * o, v);
    }
  }
}

// The newest tokens of sequences out of their pages, eight values a thread.
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
  const int heads = hs.y - hs.x, octets = a.D / 8, per_row = 2 * heads * octets;
  for (int e = threadIdx.x; e < rows * per_row; e += kRotThreads) {
    int i = e;
    const int r = i / per_row;
    i -= r * per_row;
    const int is_v = i >= heads * octets;
    i -= is_v * heads * octets;
    const int h = i / octets, o = i - h * octets;
    if (s_page[r] < 0) continue;
    const char* pages = static_cast<const char*>(is_v ? a.pv : a.pk);
    const int64_t block = static_cast<int64_t>(s_page[r]) * a.H + hs.x + h;
    const int place = s_pos[r] & (kv.page - 1);
    T* to = static_cast<T*>(const_cast<void*>(is_v ? a.v : a.k)) + static_cast<int64_t>(row0 + r) * (is_v ? a.ldv : a.ldk) +
            static_cast<int64_t>(hs.x + h) * a.D + 8 * o;
    float v[8];
    if constexpr (CODES) {
      const int row_bytes = a.D / 2, meta_bytes = a.D / 16;
      const char* at = pages + ((block * (row_bytes + meta_bytes)) << kv.page_shift);
      const uint32_t w = *reinterpret_cast<const uint32_t*>(at + place * row_bytes + 4 * o);
      const uint32_t m = *reinterpret_cast<const uint32_t*>(at + (row_bytes << kv.page_shift) + place * meta_bytes + o / 8 * 4);
      const float s = __uint_as_float(m << 16), b = __uint_as_float(m & 0xFFFF0000u);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = static_cast<float>((w >> (4 * j)) & 15u) * s + b;
    } else {
      load<T, 8>(reinterpret_cast<const T*>(pages) + ((block << kv.page_shift) + place) * a.D + 8 * o, v);
    }
    store<T, 8>(to, v);
  }
}

// Rows a block and blocks a row: a row is cut by its heads while blocks are short
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
  rotary_kernel<T><<<s.grid, kRotThreads, s.per_block * rot.dim / 2 * sizeof(float2), st>>>(
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
  const size_t smem = s.per_block * rot.dim / 2 * sizeof(float2);
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
