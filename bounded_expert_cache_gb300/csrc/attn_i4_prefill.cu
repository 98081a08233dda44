// Attention of prompt chunks over pages of 4-bit codes: row tiles of the engine of
// attn_i4.cuh, one a CTA.
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
  constexpr int kNR = sizeof(T) == 4 ? 2 : 4;
  switch (a.D / 64) {
    case 1: return chunks<CodesEngine<T, 1, kNR, 256>>(a, st);
    case 2: return chunks<CodesEngine<T, 2, kNR, 256>>(a, st);
    case 3: return chunks<CodesEngine<T, 3, 2, 128>>(a, st);
    default: return chunks<CodesEngine<T, 4, 2, 128>>(a, st);
  }
}

}  // namespace

cudaError_t launch_attn_prefill_codes(const AttnArgs& a, int32_t dtype, cudaStream_t st) {
  return dtype == MOE_F32 ? prefill_of<float>(a, st) : prefill_of<__nv_bfloat16>(a, st);
}

}  // namespace moe
