// Attention of the newest tokens over pages of 4-bit codes: the split and join of
// attn_split.cuh with the engine of attn_i4.cuh.
//
// What bounds it: with few rows HBM, 0.5625 bytes a value.
#include "attn_i4.cuh"

namespace moe {
namespace {

// the fewest rows a unit that hold them all
template <class T, int G, int KT>
cudaError_t decode_codes(const AttnArgs& a, int num_sms, cudaStream_t st) {
  const int rows = a.n_q * a.g;
  if (rows <= 8) return decode_rows<CodesEngine<T, G, 1, (G <= 2 && sizeof(T) == 2) ? 512 : KT, (G <= 2 && sizeof(T) == 2) ? 16 : 8>>(a, num_sms, st);
  if (rows <= 16 || G > 2 || sizeof(T) == 4) return decode_rows<CodesEngine<T, G, 2, KT, 8>>(a, num_sms, st);
  if constexpr (G <= 2 && sizeof(T) == 2) return decode_rows<CodesEngine<T, G, 4, KT, 8>>(a, num_sms, st);
  return cudaErrorInvalidValue;
}
template <class T>
cudaError_t decode_of(const AttnArgs& a, int num_sms, cudaStream_t st) {
  switch (a.D / 64) {
    case 1: return decode_codes<T, 1, 256>(a, num_sms, st);
    case 2: return decode_codes<T, 2, 256>(a, num_sms, st);
    case 3: return decode_codes<T, 3, 128>(a, num_sms, st);
    default: return decode_codes<T, 4, 128>(a, num_sms, st);
  }
}

}  // namespace

cudaError_t launch_attn_decode_codes(const AttnArgs& a, int32_t dtype, int num_sms, cudaStream_t st) {
  return dtype == MOE_F32 ? decode_of<float>(a, num_sms, st) : decode_of<__nv_bfloat16>(a, num_sms, st);
}

}  // namespace moe
