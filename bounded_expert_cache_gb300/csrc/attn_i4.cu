// Attention of the newest tokens over pages of 4-bit codes: the split and join of
// attn_split.cuh with the engine of attn_i4.cuh.
//
// Measured: three contexts of 131,072 to 262,143 tokens, 8 heads of 128, 4 rows each:
// 156 us, 4.4 TB/s of 0.5625 bytes a value (bf16 pages: 354); copies alone take 112, and
// with all pages in L2 the call still 152. What bounds it are the chains of dependent
// instructions with two computing warps a scheduler (issue slots 46% used) and the masks on
// the integer pipe (41% of its cycles). 40 contexts of 1 to 32,768 tokens, 2 heads of 128,
// one new token: 27 us (bf16 pages: 35; bytes take 6), four: 56: a unit's Q and join, and
// the second launch. One of 777: 12 us (9.7 in a captured graph).
#include "attn_i4.cuh"

namespace moe {
namespace {

// Eight rows a unit if that holds them all, else sixteen. (Units of 32 rows, which read
// K and V once for them, run out of registers: 4 new tokens of 8 heads a cache head,
// contexts of 30,000 to 100,000 tokens: 123 us, two units of sixteen 86.)
template <class T, int G>
cudaError_t decode_codes(const AttnArgs& a, int num_sms, cudaStream_t st) {
  constexpr bool kLean = G <= 2 && sizeof(T) == 2;  // registers for more tiles at once
  if (a.n_q * a.g <= 8) return decode_rows<CodesEngine<T, G, 1, kLean ? 8 / G : (G <= 2 ? 2 : 1)>>(a, num_sms, st);
  return decode_rows<CodesEngine<T, G, 2, G <= 2 ? 2 : 1>>(a, num_sms, st);
}
template <class T>
cudaError_t decode_of(const AttnArgs& a, int num_sms, cudaStream_t st) {
  switch (a.D / 64) {
    case 1: return decode_codes<T, 1>(a, num_sms, st);
    case 2: return decode_codes<T, 2>(a, num_sms, st);
    case 3: return decode_codes<T, 3>(a, num_sms, st);
    default: return decode_codes<T, 4>(a, num_sms, st);
  }
}

}  // namespace

cudaError_t launch_attn_decode_codes(const AttnArgs& a, int32_t dtype, int num_sms, cudaStream_t st) {
  return dtype == MOE_F32 ? decode_of<float>(a, num_sms, st) : decode_of<__nv_bfloat16>(a, num_sms, st);
}

}  // namespace moe
