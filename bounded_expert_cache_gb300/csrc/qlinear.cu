// Linear layer with 4-bit weights and group scales for few tokens.
//
//   Q4_0 (groups of 32):    y[t,n] = sum_g d_g sum_{k in g} (q_k - 8) x_k
//   I4_G64 (groups of 64):  y[t,n] = sum_g (s_g sum_{k in g} q_k x_k + b_g sum_{k in g} x_k)
//
// What bounds it: HBM, the 4.5 bits a weight, as long as a weight costs less
// than about three instructions of a thread. The inner sums therefore run on
// warp-level matrix instructions (m16n8k16, weights as A, tokens as B): codes
// become bf16 integers by a mask and a subtraction for two of them, products of
// a 4-bit integer and a bf16 are exact, sums are fp32, and the group's factor is
// applied in fp32 to the 16 x 8 sums. An fp32 x is the exact sum of three bf16
// (8 + 8 + 8 significand bits), one instruction each. Measured, 131,072 x 2,048
// Q4_0 (151 MB, 22 us of HBM): 39 us for one token, 59 for 24 (57 in a captured
// graph), where the warps issue in 55% of cycles, the tensor pipe works in 40% and
// shared memory in 53%; 2,560 x 2,048 for one token: 3.6 us in a graph, the latency
// of a launch and of a few dependent loads. Tokens past 24 go in blocks of 24 that
// each unpack the matrix again: 4,096 tokens of the same take 370 us.
//
// The order of k within an instruction is free as long as A and B agree, so x
// is stored in the order in which a lane's 4-byte word yields its eight codes:
// a lane's eight x of a group are 16 contiguous bytes.
//
// A CTA (one per SM) holds the tokens' x in shared memory, in slices of K if
// they do not fit, and walks row tiles. Its sixteen warps are 16 / WK groups of
// 16 rows by WK slices of K, so that a matrix of few rows still fills the GPU;
// the slices are added in shared memory. Each warp copies its own stages (16
// rows x 256 k: 2 KB of codes, 256 B of scales) into a ring of its own by
// asynchronous copies and meets no other warp within a tile: with one ring for
// the block and a barrier a stage, all warps unpacked and multiplied in step,
// and issued in half of the cycles.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv.h"

namespace moe {
namespace {

constexpr int kThreads = 512, kWarps = 16;
constexpr int kWK = 256;                      // k of a warp's stage
constexpr int kCodeBytes = 16 * 128;          // codes of a warp's stage
constexpr int kMetaBytes = 16 * 16;           // scales
constexpr int kWarpStage = kCodeBytes + kMetaBytes;
constexpr int kStageBytes = kWarps * kWarpStage;
constexpr int kMaxTok = 24;                   // tokens of a launch's y block

constexpr int kPieces = kCodeBytes / 16 / 32;  // 16-byte pieces a lane and stage

struct Plan {
  int tok;         // tokens of a block
  int kx;          // k of a slice of x, a multiple of 256 * WK
  int x_pitch;     // bytes of a token's slice: 64 modulo 128
  int x_bytes;     // all tokens and parts
  int slots;       // ring
  int tiles;       // row tiles
  uint32_t one;    // 128 in both halves, as bf16
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
// Four blocks of 8 rows x 16 bytes, one row address a lane: a lane gets word
// lane % 4 of row lane / 4 of each.
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma0(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {  // onto zero
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// d[0..1] += s * v[0..1]; as one instruction where the pair (s, s) serves several
template <bool PACKED>
__device__ __forceinline__ void fma2(float* d, float s, const float* v) {
  if (!PACKED) {
    d[0] += s * v[0];
    d[1] += s * v[1];
    return;
  }
  unsigned long long dd, vv, ss;
  asm("mov.b64 %0, {%1, %2};" : "=l"(dd) : "f"(d[0]), "f"(d[1]));
  asm("mov.b64 %0, {%1, %2};" : "=l"(vv) : "f"(v[0]), "f"(v[1]));
  asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "f"(s));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(dd) : "l"(ss), "l"(vv));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d[0]), "=f"(d[1]) : "l"(dd));
}
// The eight codes of a 4-byte word as bf16 integers less `bias` - 128: the
// nibble becomes the low mantissa bits of 128 (exact), bias is subtracted
// (exact). o[0], o[1]: low nibbles of bytes 0,2 and 1,3; o[2], o[3]: high ones.
// (w & mask) | one is one instruction only if `one` (128 in both halves) sits in
// a register, which the compiler grants a value it does not know: it comes with
// the launch's parameters.
__device__ __forceinline__ uint32_t code2(uint32_t w, uint32_t one) {
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(r) : "r"(w), "r"(one));
  return r;
}
__device__ __forceinline__ void codes(uint32_t w, uint32_t one, uint32_t bias2, uint32_t* o) {
  o[0] = code2(w, one);
  o[1] = code2(w >> 8, one);
  o[2] = code2(w >> 4, one);
  o[3] = code2(w >> 12, one);
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(o[i]) : "r"(bias2));
}

// The three bf16 of an fp32: each the leading 8 significand bits of what is
// left, so their sum is exact. Infinities and NaN stay in the first.
__device__ __forceinline__ void split3(float x, uint32_t* p) {
  const uint32_t u = __float_as_uint(x);
  const bool odd = (u & 0x7F800000u) == 0x7F800000u;
  p[0] = odd && (u & 0x007FFFFFu) ? 0x7FC0u : u >> 16;
  const float r1 = odd ? 0.f : x - __uint_as_float(u & 0xFFFF0000u);
  const uint32_t u1 = __float_as_uint(r1);
  p[1] = u1 >> 16;
  p[2] = __float_as_uint(r1 - __uint_as_float(u1 & 0xFFFF0000u)) >> 16;
}

// x of tokens [t0, t0 + tok) and k [k0, k0 + kx) to shared memory, zeros past K;
// for I4_G64 also each token's sum over every group of 64.
template <int QUANT, bool XF32>
__device__ __forceinline__ void load_x(const LinearArgs& a, const Plan& p, int t0, int tok, int k0, uint32_t xs,
                                       float* sums) {
  constexpr int kParts = XF32 ? 3 : 1;
  const int chunks = p.kx / 8;  // of 8 x: (group of 32, lane of a quad)
  const int part_bytes = p.tok * p.x_pitch;
  const int total = tok * chunks;  // kx is a multiple of 256: a warp has 32 chunks of one token
#pragma unroll 2
  for (int e = threadIdx.x; e < total; e += kThreads) {
    const int t = e / chunks, c = e - t * chunks;
    // element offsets of the two runs of four
    const int ka = QUANT == MOE_Q4_0 ? k0 + (c >> 2) * 32 + (c & 3) * 4 : k0 + c * 8;
    const int kb = QUANT == MOE_Q4_0 ? ka + 16 : ka + 4;
    const bool in = ka < a.K;  // K is a multiple of 32: both runs are in or out
    const uint32_t at = xs + t * p.x_pitch + c * 16;
    float sum = 0.f;
    if constexpr (XF32) {
      const float* x = static_cast<const float*>(a.x) + (t0 + t) * a.ldx;
      float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
      if (in) {
        u = __ldg(reinterpret_cast<const float4*>(x + ka));
        v = __ldg(reinterpret_cast<const float4*>(x + kb));
      }
      float f[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
      if (QUANT != MOE_Q4_0) sum = ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
      // the order of a word's codes
      constexpr int kQ4[8] = {0, 2, 1, 3, 4, 6, 5, 7}, kI4[8] = {0, 4, 2, 6, 1, 5, 3, 7};
      uint32_t s[8][3];
#pragma unroll
      for (int i = 0; i < 8; ++i) split3(f[QUANT == MOE_Q4_0 ? kQ4[i] : kI4[i]], s[i]);
#pragma unroll
      for (int q = 0; q < kParts; ++q)
        sts128(at + q * part_bytes, make_uint4(s[0][q] | s[1][q] << 16, s[2][q] | s[3][q] << 16,
                                               s[4][q] | s[5][q] << 16, s[6][q] | s[7][q] << 16));
    } else {
      const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x) + (t0 + t) * a.ldx;
      uint2 u = make_uint2(0u, 0u), v = u;
      if (in) {
        u = __ldg(reinterpret_cast<const uint2*>(x + ka));
        v = __ldg(reinterpret_cast<const uint2*>(x + kb));
      }
      if (QUANT == MOE_Q4_0) {
        sts128(at, make_uint4(__byte_perm(u.x, u.y, 0x5410), __byte_perm(u.x, u.y, 0x7632),
                              __byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632)));
      } else {
        const uint32_t w[4] = {u.x, u.y, v.x, v.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += __uint_as_float(w[i] << 16) + __uint_as_float(w[i] & 0xFFFF0000u);
        sts128(at, make_uint4(__byte_perm(u.x, v.x, 0x5410), __byte_perm(u.y, v.y, 0x5410),
                              __byte_perm(u.x, v.x, 0x7632), __byte_perm(u.y, v.y, 0x7632)));
      }
    }
    if (QUANT != MOE_Q4_0) {
      // eight lanes hold a group of 64
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(~0u, sum, d);
      if ((c & 7) == 0) sums[(c >> 3) * kMaxTok + t] = sum;
    }
  }
}

// Outputs that came out infinite or NaN, formed again weight by weight. A group's
// sum of codes times x can overflow where the sum of weights times x does not
// (|x| above 1e35), and an infinite x makes s sum(q x) + b sum(x) a NaN where
// (s q + b) x is an infinity. Once not finite a sum stays so, hence this finds
// every such output. A warp a row of the CTA's tiles, lanes along K.
template <int QUANT, bool XF32>
__device__ __noinline__ void form_again(const LinearArgs& a, int t0, int tok, int tiles, int R) {
  const int lane = threadIdx.x & 31;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    for (int r = threadIdx.x >> 5; r < R && tile * R + r < a.N; r += kWarps) {
      const int n = tile * R + r;
      bool bad = false;
      if (lane < tok) {
        const int64_t at = (t0 + lane) * a.ldy + n;
        bad = !isfinite(a.yt == MOE_F32 ? static_cast<const float*>(a.y)[at]
                                        : __bfloat162float(static_cast<const __nv_bfloat16*>(a.y)[at]));
      }
      const uint8_t* row = a.w + static_cast<int64_t>(n) * (a.K / 2);
      const uint16_t* meta = reinterpret_cast<const uint16_t*>(a.meta + static_cast<int64_t>(n) * (a.K / 16));
      for (uint32_t left = __ballot_sync(~0u, bad); left; left &= left - 1) {
        const int t = __ffs(left) - 1;
        float v = 0.f;
        for (int k = lane; k < a.K; k += 32) {
          float w;
          if (QUANT == MOE_Q4_0) {
            const int c = __ldg(row + (k >> 5) * 16 + (lane & 15)) >> (lane & 16 ? 4 : 0) & 15;
            w = __half2float(__ushort_as_half(__ldg(meta + (k >> 5)))) * static_cast<float>(c - 8);  // exact
          } else {
            const int c = __ldg(row + (k >> 1)) >> (k & 1 ? 4 : 0) & 15;
            const uint32_t sb = __ldg(reinterpret_cast<const uint32_t*>(meta) + (k >> 6));
            w = fmaf(__uint_as_float(sb << 16), static_cast<float>(c), __uint_as_float(sb & 0xFFFF0000u));
          }
          const int64_t at = (t0 + t) * a.ldx + k;
          v += w * (XF32 ? __ldg(static_cast<const float*>(a.x) + at)
                         : __bfloat162float(static_cast<const __nv_bfloat16*>(a.x)[at]));
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
        if (lane == 0) {
          if (a.bias) v += __ldg(a.bias + n);
          const int64_t at = (t0 + t) * a.ldy + n;
          if (a.yt == MOE_F32)
            static_cast<float*>(a.y)[at] = v;
          else
            static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
        }
      }
    }
  }
}

template <int QUANT, bool XF32, int NT, int WK>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const __grid_constant__ LinearArgs a, Plan p) {
  constexpr int kParts = XF32 ? 3 : 1, R = 16 * kWarps / WK;  // rows of a tile
  extern __shared__ __align__(128) unsigned char sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t xs = smem_u32(sm) + p.slots * kStageBytes;
  const uint32_t ring = smem_u32(sm) + warp * (p.slots * kWarpStage);
  float* const sums = reinterpret_cast<float*>(sm + p.slots * kStageBytes + p.x_bytes);
  // [2][16 warps][16 rows][8], WK > 1
  float* const red = sums + (QUANT == MOE_Q4_0 ? 0 : p.kx / 64 * kMaxTok);
  const int wr = warp / WK, wk = warp % WK;  // row group, slice of K
  const int t0 = blockIdx.y * p.tok, tok = min(p.tok, a.T - t0);
  constexpr int stage_k = kWK * WK;
  const int n_slices = (a.K + p.kx - 1) / p.kx;
  const int stages_tile = (a.K + stage_k - 1) / stage_k;  // slices hold whole stages

  // One stage of the warp: codes [16 rows][128 bytes], 16-byte pieces (32 codes)
  // swizzled by the row; scales [16 rows][16 bytes]. Zeros past N and K. A lane
  // copies piece lane % 8 of rows lane / 8 + 4 i, and the scales of row lane.
  int ld_tile = blockIdx.x, ld_stage = 0, ld_slot = 0;
  const int piece = lane & 7;
  uint32_t dst[kPieces];  // within a slot
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int row = (lane >> 3) + 4 * i;
    dst[i] = row * 128 + ((piece ^ (row & 7)) << 4);
  }
  // Of the tile being copied: its codes and scales, this lane's offsets into
  // them (the same in every tile), and whether the warp's rows are all rows.
  const uint8_t *code0, *meta0;
  bool full_rows;
  uint32_t off[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
    off[i] = static_cast<uint32_t>(wr * 16 + (lane >> 3) + 4 * i) * (a.K / 2) + wk * (kWK / 2) + piece * 16;
  const uint32_t moff = static_cast<uint32_t>(wr * 16 + (lane & 15)) * (a.K / 16) + wk * (kWK / 16);
  auto open_tile = [&]() {
    code0 = a.w + static_cast<int64_t>(ld_tile) * R * (a.K / 2);
    meta0 = a.meta + static_cast<int64_t>(ld_tile) * R * (a.K / 16);
    full_rows = ld_tile * R + wr * 16 + 16 <= a.N;
  };
  open_tile();
  auto issue = [&]() {
    if (ld_tile < p.tiles) {
      const uint32_t st = ring + ld_slot * kWarpStage;
      const int k0 = ld_stage * stage_k, left = a.K - k0 - wk * kWK;  // k of this warp's stage
      const uint32_t md = st + kCodeBytes + (lane & 15) * 16;
      if (full_rows && left >= kWK) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) cp16(st + dst[i], code0 + (off[i] + k0 / 2));
      } else {
        const int n0 = ld_tile * R + wr * 16 + (lane >> 3);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const bool in = n0 + 4 * i < a.N && piece * 32 < left;
          cp16(st + dst[i], in ? code0 + (off[i] + k0 / 2) : a.w, in);
        }
      }
      if (lane < 16) {
        const bool in = full_rows || ld_tile * R + wr * 16 + lane < a.N;
        const uint8_t* src = meta0 + (moff + k0 / 16);
        if ((a.K & 255) == 0) {
          cp16(md, in && left > 0 ? src : a.w, in && left > 0);
        } else if ((a.K & 63) == 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) cp4(md + i * 4, in && i * 64 < left ? src + i * 4 : a.w, in && i * 64 < left);
        } else {  // an odd number of groups a row: scales are 2-byte aligned
          uint32_t v[4] = {};
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (in && i * 32 < left)
              v[i >> 1] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(src) + i)) << (16 * (i & 1));
          sts128(md, make_uint4(v[0], v[1], v[2], v[3]));
        }
      }
      if (++ld_slot == p.slots) ld_slot = 0;
      if (++ld_stage == stages_tile) {
        ld_stage = 0;
        ld_tile += gridDim.x;
        if (ld_tile < p.tiles) open_tile();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");  // empty groups keep the count
  };
  for (int i = 0; i < p.slots - 1; ++i) issue();
  load_x<QUANT, XF32>(a, p, t0, tok, 0, xs, sums);
  __syncthreads();
  int have = 0;  // slice of x in shared memory

  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
  const int r = lane >> 2, c = lane & 3;  // rows r and r + 8, quad lane
  const uint32_t part_bytes = p.tok * p.x_pitch;
  // this lane's x: token r of each block of eight (a token past the last reads
  // the last one's: its sums are not stored)
  uint32_t xt[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) xt[n] = xs + min(n * 8 + r, tok - 1) * p.x_pitch + c * 16;
  constexpr uint32_t kBias = QUANT == MOE_Q4_0 ? 0x43084308u : 0x43004300u;  // 136, 128
  // ldmatrix: lanes 0-7 and 8-15 address rows 0-7 and 8-15 of a group's piece, lanes 16-31 the next group's
  const uint32_t q_off = (lane & 15) * 128, q_phase = ((lane & 7) ^ (lane >> 4)) << 4, m_off = kCodeBytes + r * 16;

  float probe = 0.f;  // NaN once a sum is not finite (a bias of -inf is no reason to form one again)
  auto store = [&](int n, int t, float v) {
    probe = fmaf(v, 0.f, probe);
    if (a.bias) v += __ldg(a.bias + n);
    const int64_t at = (t0 + t) * a.ldy + n;
    if (a.yt == MOE_F32)
      static_cast<float*>(a.y)[at] = v;
    else
      static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
  };

  int slot = 0, stage = 0, round = 0;
  for (int tile = blockIdx.x; tile < p.tiles;) {
    switch (p.slots) {
      case 3: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
      case 4: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
      default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;  // five
    }
    __syncwarp();  // the warp's stage is there, and the one before it used up
    issue();
    if (n_slices > 1) {
      const int slice = stage * stage_k / p.kx;
      if (slice != have) {  // x does not fit: the next slice
        __syncthreads();
        load_x<QUANT, XF32>(a, p, t0, tok, slice * p.kx, xs, sums);
        have = slice;
        __syncthreads();
      }
    }
    const int k0 = stage * stage_k - have * p.kx + wk * kWK;  // within the slice
    const uint32_t st = ring + slot * kWarpStage, xk = k0 * 2;
    static_assert(kWarpStage % 128 == 0, "a slot's rows start at multiples of 128, so a piece's offset can be XORed in");
    const uint32_t q0 = (st + q_off) ^ q_phase;
    const uint4 m0 = lds128(st + m_off), m1 = lds128(st + m_off + 128);
    const uint32_t ma[4] = {m0.x, m0.y, m0.z, m0.w}, mb[4] = {m1.x, m1.y, m1.z, m1.w};
    const int left = a.K - (stage * stage_k + wk * kWK);  // k of this warp's stage; may be negative
#pragma unroll
    for (int g2 = 0; g2 < 4; ++g2) {  // 64 k: two groups of Q4_0, one of I4_G64
      if (g2 * 64 >= left) break;
      uint32_t w[4];  // rows r and r + 8 of group 2 g2, then of the next
      ldsm4(w, q0 ^ (static_cast<uint32_t>(g2) << 5));
      float s[2][NT][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int g = 2 * g2 + h;
        uint32_t wa[4], wb[4];
        codes(w[2 * h], p.one, kBias, wa);
        codes(w[2 * h + 1], p.one, kBias, wb);
        const uint32_t f0[4] = {wa[0], wb[0], wa[1], wb[1]}, f1[4] = {wa[2], wb[2], wa[3], wb[3]};
        float(*d)[4] = s[QUANT == MOE_Q4_0 ? h : 0];
#pragma unroll
        for (int q = 0; q < kParts; ++q)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint4 x = lds128(xt[n] + xk + q * part_bytes + g * 64);
            if (q == 0 && (QUANT == MOE_Q4_0 || h == 0))
              mma0(d[n], f0, x.x, x.y);
            else
              mma(d[n], f0, x.x, x.y);
            mma(d[n], f1, x.z, x.w);
          }
      }
      if (QUANT == MOE_Q4_0) {
        const float2 da = __half22float2(*reinterpret_cast<const __half2*>(&ma[g2]));
        const float2 db = __half22float2(*reinterpret_cast<const __half2*>(&mb[g2]));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          fma2<(NT > 1)>(acc[n], da.x, s[0][n]);
          fma2<(NT > 1)>(acc[n] + 2, db.x, s[0][n] + 2);
          fma2<(NT > 1)>(acc[n], da.y, s[1][n]);
          fma2<(NT > 1)>(acc[n] + 2, db.y, s[1][n] + 2);
        }
      } else {
        const float sa = __uint_as_float(ma[g2] << 16), ba = __uint_as_float(ma[g2] & 0xFFFF0000u);
        const float sb = __uint_as_float(mb[g2] << 16), bb = __uint_as_float(mb[g2] & 0xFFFF0000u);
        const float* su = sums + (k0 / 64 + g2) * kMaxTok + c * 2;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float2 u = *reinterpret_cast<const float2*>(su + n * 8);
          const float xsum[2] = {u.x, u.y};
          fma2<(NT > 1)>(acc[n], sa, s[0][n]);
          fma2<(NT > 1)>(acc[n] + 2, sb, s[0][n] + 2);
          fma2<(NT > 1)>(acc[n], ba, xsum);
          fma2<(NT > 1)>(acc[n] + 2, bb, xsum);
        }
      }
    }
    if (++slot == p.slots) slot = 0;
    if (++stage < stages_tile) continue;
    // ---- the tile's rows: slices of K added in order, bias, one rounding
    stage = 0;
    if constexpr (WK == 1) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = tile * R + wr * 16 + r + 8 * (i >> 1), t = n * 8 + c * 2 + (i & 1);
          if (row < a.N && t < tok) store(row, t, acc[n][i]);
          acc[n][i] = 0.f;
        }
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        // the WK warps of the rows meet; two buffers, so that one barrier a
        // round also keeps a write behind the reads of the round before last
        float* const buf = red + (round & 1) * (kWarps * 16 * 8);
        ++round;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          *reinterpret_cast<float2*>(buf + (warp * 16 + r + 8 * h) * 8 + c * 2) =
              make_float2(acc[n][2 * h], acc[n][2 * h + 1]);
          acc[n][2 * h] = acc[n][2 * h + 1] = 0.f;
        }
        asm volatile("bar.sync %0, %1;" ::"r"(1 + wr), "r"(32 * WK) : "memory");
#pragma unroll
        for (int e = wk * 32 + lane; e < 16 * 8; e += 32 * WK) {
          const int row = e & 15, t = e >> 4, nn = tile * R + wr * 16 + row;
          if (nn >= a.N || n * 8 + t >= tok) continue;
          float v = 0.f;
#pragma unroll
          for (int k = 0; k < WK; ++k) v += buf[((wr * WK + k) * 16 + row) * 8 + t];
          store(nn, n * 8 + t, v);
        }
      }
    }
    tile += gridDim.x;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (__syncthreads_or(probe != 0.f)) form_again<QUANT, XF32>(a, t0, tok, p.tiles, R);
}

constexpr int kFull = 226 * 1024;              // dynamic shared memory of a CTA
constexpr int kRedBytes = 2 * kWarps * 16 * 8 * 4;

// Shared bytes of x of a slice and its sums.
inline int64_t x_bytes(int quant, int parts, int tok, int64_t kx) {
  return static_cast<int64_t>(tok) * parts * (kx * 2 + 64) + (quant == MOE_Q4_0 ? 0 : kx / 64 * kMaxTok * 4);
}

template <int QUANT, bool XF32, int NT, int WK>
cudaError_t launch(const LinearArgs& a, int blocks_t, int num_sms, cudaStream_t st) {
  constexpr int R = 16 * kWarps / WK, kParts = XF32 ? 3 : 1, stage_k = kWK * WK;
  Plan p;
  p.tok = (a.T + blocks_t - 1) / blocks_t;
  p.tiles = (a.N + R - 1) / R;
  p.one = 0x43004300u;
  // a ring of five to three slots beside all of x, else x in slices of whole stages
  const int stages = (a.K + stage_k - 1) / stage_k;
  int n = 1;
  auto slice = [&] { return (stages + n - 1) / n * stage_k; };
  auto need = [&](int slots) { return x_bytes(QUANT, kParts, p.tok, slice()) + kRedBytes + slots * kStageBytes; };
  p.slots = 5;
  while (p.slots > 3 && need(p.slots) > kFull) --p.slots;
  while (need(p.slots) > kFull) {
    if (slice() == stage_k) return cudaErrorInvalidValue;
    ++n;
  }
  p.kx = slice();
  p.x_pitch = p.kx * 2 + 64;
  p.x_bytes = p.tok * kParts * p.x_pitch;
  cudaError_t e = cudaFuncSetAttribute(linear_kernel<QUANT, XF32, NT, WK>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFull);
  if (e != cudaSuccess) return e;
  const dim3 grid(std::min(p.tiles, std::max(1, num_sms / blocks_t)), blocks_t);
  linear_kernel<QUANT, XF32, NT, WK><<<grid, kThreads, static_cast<int>(need(p.slots)), st>>>(a, p);
  return cudaGetLastError();
}

// Rows of a tile: the largest of 256, 128, 64 and 32 that leaves each SM six
// tiles (they end unevenly), 32 where none does. A stage of small tiles is long
// in K: not longer than K, and one stage of x has to fit. Where x goes in slices
// every tile loads all of it again, so tiles are large: one for two SMs is
// enough (32,768 x 8,192 at 24 tokens: 64 rows 154 us).
template <int QUANT, bool XF32, int NT>
cudaError_t by_rows(const LinearArgs& a, int blocks_t, int num_sms, cudaStream_t st) {
  constexpr int kParts = XF32 ? 3 : 1;
  const int tok = (a.T + blocks_t - 1) / blocks_t;
  auto fits = [&](int64_t k) { return x_bytes(QUANT, kParts, tok, k) + kRedBytes + 3 * kStageBytes <= kFull; };
  const int64_t want = fits((a.K + kWK - 1) / kWK * kWK) ? 6 * num_sms : num_sms / 2;
  int wk = 1;
  while (wk < 8 && a.N < 256 / wk * want && a.K > wk * kWK && fits(2 * wk * kWK)) wk *= 2;
  switch (wk) {
    case 1: return launch<QUANT, XF32, NT, 1>(a, blocks_t, num_sms, st);
    case 2: return launch<QUANT, XF32, NT, 2>(a, blocks_t, num_sms, st);
    case 4: return launch<QUANT, XF32, NT, 4>(a, blocks_t, num_sms, st);
    default: return launch<QUANT, XF32, NT, 8>(a, blocks_t, num_sms, st);
  }
}

template <int QUANT, bool XF32>
cudaError_t by_tokens(const LinearArgs& a, int num_sms, cudaStream_t st) {
  const int blocks_t = (a.T + kMaxTok - 1) / kMaxTok, tok = (a.T + blocks_t - 1) / blocks_t;
  if (tok <= 8) return by_rows<QUANT, XF32, 1>(a, blocks_t, num_sms, st);
  if (tok <= 16) return by_rows<QUANT, XF32, 2>(a, blocks_t, num_sms, st);
  return by_rows<QUANT, XF32, 3>(a, blocks_t, num_sms, st);
}

}  // namespace

cudaError_t launch_quant_linear(const LinearArgs& args, int32_t quant, int num_sms, cudaStream_t st) {
  // a grid has at most 65,535 blocks of tokens
  constexpr int kMost = 65535 * kMaxTok;
  LinearArgs a = args;
  for (int64_t t0 = 0; t0 < args.T; t0 += kMost) {
    a.T = static_cast<int32_t>(std::min<int64_t>(kMost, args.T - t0));
    a.x = static_cast<const char*>(args.x) + t0 * args.ldx * (args.xt == MOE_F32 ? 4 : 2);
    a.y = static_cast<char*>(args.y) + t0 * args.ldy * (args.yt == MOE_F32 ? 4 : 2);
    cudaError_t e;
    if (quant == MOE_Q4_0)
      e = a.xt == MOE_F32 ? by_tokens<MOE_Q4_0, true>(a, num_sms, st) : by_tokens<MOE_Q4_0, false>(a, num_sms, st);
    else
      e = a.xt == MOE_F32 ? by_tokens<MOE_I4_G64, true>(a, num_sms, st) : by_tokens<MOE_I4_G64, false>(a, num_sms, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe
