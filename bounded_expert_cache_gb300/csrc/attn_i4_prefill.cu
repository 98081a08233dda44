// Attention of prompt chunks over pages of 4-bit codes in f32 and of heads above 128:
// row tiles of the engine of attn_i4.cuh, one a CTA. (bf16 heads of 64 and 128 run on
// the 5th-generation tensor cores, attn_prefill.cu.) Every CTA converts all tokens its 16
// rows see, and that bounds it: 1,024 tokens at 32,768, 16 heads / 2, of 256, bf16:
// 4.6 ms; 2,048 at 8,192, f32, 8 / 8, of 64: 0.36 ms.
#include "attn_i4.cuh"

namespace moe {
namespace {

template <class E>
cudaError_t chunks(const AttnArgs& a, cudaStream_t st) {
  // every sequence has at most one partly filled row tile
  const int64_t grid = ((static_cast<int64_t>(a.n_rows) * a.g + E::kRows - 1) / E::kRows + a.n) * a.Hkv;
  return launch<E, false>(a, static_cast<int>(grid), st);
}
template <class T>
cudaError_t prefill_of(const AttnArgs& a, cudaStream_t st) {
  if constexpr (sizeof(T) == 4) {
    if (a.D == 64) return chunks<CodesEngine<T, 1, 2, 2>>(a, st);
    if (a.D == 128) return chunks<CodesEngine<T, 2, 2, 2>>(a, st);
  }
  switch (a.D / 64) {
    case 3: return chunks<CodesEngine<T, 3, 2, 1>>(a, st);
    default: return chunks<CodesEngine<T, 4, 2, 1>>(a, st);
  }
}

}  // namespace

cudaError_t launch_attn_prefill_codes(const AttnArgs& a, int32_t dtype, int num_sms, cudaStream_t st) {
  if (dtype == MOE_BF16 && a.D <= kTcHeadDim) return launch_attn_prefill_codes_tc(a, num_sms, st);
  return dtype == MOE_F32 ? prefill_of<float>(a, st) : prefill_of<__nv_bfloat16>(a, st);
}

}  // namespace moe
