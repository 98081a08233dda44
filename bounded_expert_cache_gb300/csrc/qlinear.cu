// Linear layer with 4-bit weights and group scales for few tokens.
//
//   Q4_0 (groups of 32):    y[t,n] = sum_g d_g sum_{k in g} (q_k - 8) x_k
//   I4_G64 (groups of 64):  y[t,n] = sum_g (s_g sum_{k in g} q_k x_k + b_g sum_{k in g} x_k)
//
// What bounds it: HBM, the 4.5 bits a weight. A warp takes one row; its lanes
// take 16 weight bytes (32 weights) each, four tokens at a time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv.h"

namespace moe {
namespace {

constexpr int kTok = 4;

template <class X>
__device__ __forceinline__ void load8(const X* p, float* v);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float* v) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float* v) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

template <class X, class Y, int QUANT>
__global__ void __launch_bounds__(256) linear_kernel(LinearArgs a) {
  const int lane = threadIdx.x & 31;
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (n >= a.N) return;
  const int t0 = blockIdx.y * kTok, nt = min(kTok, a.T - t0);
  const uint8_t* row = a.w + static_cast<int64_t>(n) * (a.K / 2);
  const uint8_t* meta = a.meta + static_cast<int64_t>(n) * (a.K / 16);
  float acc[kTok] = {};
  for (int b = lane; b < a.K / 32; b += 32) {
    const uint4 w4 = __ldg(reinterpret_cast<const uint4*>(row) + b);
    const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
    float s, bias = 0.f;
    if (QUANT == MOE_Q4_0) {
      s = __half2float(__ldg(reinterpret_cast<const __half*>(meta) + b));
    } else {
      const uint32_t sb = __ldg(reinterpret_cast<const uint32_t*>(meta) + b / 2);
      s = __uint_as_float(sb << 16);
      bias = __uint_as_float(sb & 0xFFFF0000u);
    }
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
      if (t >= nt) break;
      const X* x = static_cast<const X*>(a.x) + (t0 + t) * a.ldx + b * 32;
      float dot = 0.f, sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v[8];
        load8<X>(x + 8 * i, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // Q4_0: elements 0-15 are the low nibbles of bytes 0-15, 16-31 the high ones
          const int e = 8 * i + j;
          const int byte = QUANT == MOE_Q4_0 ? e & 15 : e / 2, high = QUANT == MOE_Q4_0 ? e >> 4 : e & 1;
          const int q = (w[byte >> 2] >> ((byte & 3) * 8 + high * 4)) & 15;
          dot += static_cast<float>(QUANT == MOE_Q4_0 ? q - 8 : q) * v[j];
          sum += v[j];
        }
      }
      acc[t] += s * dot;
      if (QUANT != MOE_Q4_0) acc[t] += bias * sum;
    }
  }
#pragma unroll
  for (int t = 0; t < kTok; ++t) {
    float v = acc[t];
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    if (t < nt && lane == 0) {
      if (a.bias) v += __ldg(a.bias + n);
      Y* y = static_cast<Y*>(a.y) + (t0 + t) * a.ldy + n;
      if constexpr (sizeof(Y) == 4)
        *y = v;
      else
        *y = __float2bfloat16_rn(v);
    }
  }
}

template <class X, class Y>
cudaError_t by_quant(const LinearArgs& a, int32_t quant, cudaStream_t st) {
  const dim3 grid((a.N + 7) / 8, (a.T + kTok - 1) / kTok);
  if (quant == MOE_Q4_0)
    linear_kernel<X, Y, MOE_Q4_0><<<grid, 256, 0, st>>>(a);
  else
    linear_kernel<X, Y, MOE_I4_G64><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quant_linear(const LinearArgs& a, int32_t quant, int num_sms, cudaStream_t st) {
  (void)num_sms;
  if (a.xt == MOE_F32)
    return a.yt == MOE_F32 ? by_quant<float, float>(a, quant, st) : by_quant<float, __nv_bfloat16>(a, quant, st);
  return a.yt == MOE_F32 ? by_quant<__nv_bfloat16, float>(a, quant, st)
                         : by_quant<__nv_bfloat16, __nv_bfloat16>(a, quant, st);
}

}  // namespace moe
