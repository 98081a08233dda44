// C ABI entry points of the KV cache, attention and the 4-bit linear layer:
// argument checks, scratch layout, launches.
#include <atomic>
#include <cmath>
#include <cstddef>
#include <string>

#include "kv.h"
#include "prefill.h"

namespace {

// Test hook of the attention kernels' bounded waits, for this thread's next call.
struct WaitHook {
  int64_t wait_cycles = 0;
  int32_t copies = -1;
};
thread_local WaitHook t_hook;

moe_status_t fail(moe_status_t st, const char* call, const std::string& why) {
  moe::set_thread_error(std::string(call) + ": " + why);
  return st;
}
moe_status_t cuda_fail(const char* call, cudaError_t e) { return fail(MOE_ERR_CUDA, call, cudaGetErrorString(e)); }

// Nothing is thrown across the ABI: the only C++ exceptions here come from
// building an error message.
template <class F>
moe_status_t guarded(F&& f) noexcept {
  try {
    return f();
  } catch (...) {
    return MOE_ERR_STATE;
  }
}

// SM count of the current device; 0 if there is none.
cudaError_t sm_count(int* n) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  return cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int elem_bytes(int32_t dtype) { return dtype == MOE_F32 ? 4 : 2; }
int token_elem_bytes(const moe_kv_t& a) { return elem_bytes(moe::token_type(a)); }

// Geometry of a cache; nullptr if it is fine.
const char* bad_geometry(const moe_kv_t& a) {
  const int32_t type = moe::token_type(a);
  if (type != MOE_F32 && type != MOE_BF16) return "dtype is neither MOE_F32 nor MOE_BF16, with or without MOE_KV_I4";
  if (a.n_layers < 1 || a.n_pages < 1 || a.n_kv_heads < 1) return "n_layers, n_pages or n_kv_heads < 1";
  if (a.page_tokens < 16 || a.page_tokens > 256 || (a.page_tokens & (a.page_tokens - 1)))
    return "page_tokens is not 16, 32, 64, 128 or 256";
  if (a.head_dim < 8 || a.head_dim > 256 || a.head_dim % 8) return "head_dim is not a multiple of 8 in 8..256";
  if ((a.dtype & MOE_KV_I4) && a.head_dim % 64) return "head_dim is not a multiple of 64 in a cache of 4-bit codes";
  if (a.n_kv_heads > 1024) return "n_kv_heads above 1024";
  if (a.max_seqs < 1 || a.max_seqs > 65536) return "max_seqs outside 1..65536";
  if (a.max_pages < 1 || static_cast<int64_t>(a.max_pages) * a.page_tokens > 1ll << 30)
    return "max_pages < 1 or max_pages * page_tokens above 2^30";
  if (static_cast<int64_t>(a.n_pages) * a.n_kv_heads > 0x7FFFFFFFll) return "n_pages * n_kv_heads above 2^31 - 1";
  return nullptr;
}

// Checks shared by every call on a cache, and its scratch layout.
moe_status_t open_kv(const char* call, const moe_kv_t* kv, moe::KvLayout* l, int* sms) {
  if (!kv) return fail(MOE_ERR_ARG, call, "kv is NULL");
  if (const char* why = bad_geometry(*kv)) return fail(MOE_ERR_ARG, call, why);
  if (!kv->k || !kv->v || !kv->table || !kv->lens || !kv->ref || !kv->work)
    return fail(MOE_ERR_ARG, call, "a cache pointer is NULL");
  if (!aligned16(kv->k) || !aligned16(kv->v) || !aligned16(kv->work))
    return fail(MOE_ERR_ARG, call, "k, v or work is not 16-byte aligned");
  cudaError_t e = sm_count(sms);
  if (e != cudaSuccess) return cuda_fail(call, e);
  *l = moe::kv_layout(*kv, *sms);
  if (kv->work_bytes < l->bytes) return fail(MOE_ERR_ARG, call, "work_bytes is smaller than moe_kv_work_bytes");
  return MOE_OK;
}

moe_status_t launched(const char* call, cudaError_t e) { return e == cudaSuccess ? MOE_OK : cuda_fail(call, e); }

moe_status_t check_list(const char* call, const void* p, int32_t n) {
  if (n < 0 || n > moe::kMaxList) return fail(MOE_ERR_ARG, call, "n outside 0..8192");
  if (n > 0 && !p) return fail(MOE_ERR_ARG, call, "a list is NULL");
  return MOE_OK;
}

// Checks shared by the calls that take rows of keys and values; *none: there are none.
moe_status_t open_rows(const char* call, const moe_kv_t* kv, int32_t layer, const void* k, int64_t ldk, const void* v,
                       int64_t ldv, const int32_t* seqs, const int32_t* cu, int32_t n, int32_t n_rows, moe::KvLayout* l,
                       int* sms, bool* none) {
  moe_status_t st = open_kv(call, kv, l, sms);
  if (st != MOE_OK) return st;
  if (layer < 0 || layer >= kv->n_layers) return fail(MOE_ERR_ARG, call, "layer out of range");
  if (n < 0 || n > 65536 || n_rows < 0) return fail(MOE_ERR_ARG, call, "n outside 0..65536 or n_rows < 0");
  if (!seqs && n > kv->max_seqs) return fail(MOE_ERR_ARG, call, "n above max_seqs without seqs");
  *none = n == 0 || n_rows == 0;
  if (*none) return MOE_OK;
  if (!k || !v || !cu) return fail(MOE_ERR_ARG, call, "k, v or cu is NULL");
  const int64_t width = static_cast<int64_t>(kv->n_kv_heads) * kv->head_dim;
  const int per = 16 / token_elem_bytes(*kv);
  if (!aligned16(k) || !aligned16(v) || ldk % per || ldv % per)
    return fail(MOE_ERR_ARG, call, "rows of k or v are not 16-byte aligned");
  if (ldk < width || ldv < width) return fail(MOE_ERR_ARG, call, "ldk or ldv is smaller than a row");
  return MOE_OK;
}

// A rotation of heads of D values as the kernels see it.
moe_status_t open_rotary(const char* call, const moe_rotary_t* rot, int32_t D, moe::Rotary* r) {
  if (!rot || !rot->turns) return fail(MOE_ERR_ARG, call, "the rotation or its turns are NULL");
  if (reinterpret_cast<uintptr_t>(rot->turns) % 8) return fail(MOE_ERR_ARG, call, "turns is not 8-byte aligned");
  if (rot->dim < 2 || rot->dim % 2 || rot->dim > D) return fail(MOE_ERR_ARG, call, "the rotation's dim is not an even number in 2..head_dim");
  if (rot->interleaved != 0 && rot->interleaved != 1) return fail(MOE_ERR_ARG, call, "interleaved is neither 0 nor 1");
  const float magnitude = static_cast<float>(rot->magnitude);
  if (!std::isfinite(magnitude)) return fail(MOE_ERR_ARG, call, "magnitude is not finite in fp32");
  *r = moe::Rotary{rot->turns, rot->dim, rot->interleaved, magnitude, static_cast<float>(rot->magnitude - magnitude)};
  return MOE_OK;
}
// Rows of heads that go from x to y.
moe_status_t check_heads(const char* call, const void* x, int64_t ldx, const void* y, int64_t ldy, int32_t heads, int32_t D,
                         int32_t type) {
  const int per = 16 / elem_bytes(type);
  if (!aligned16(x) || !aligned16(y) || ldx % per || ldy % per) return fail(MOE_ERR_ARG, call, "rows of heads are not 16-byte aligned");
  const int64_t width = static_cast<int64_t>(heads) * D;
  if (ldx < width || ldy < width) return fail(MOE_ERR_ARG, call, "a row stride is smaller than a row");
  return MOE_OK;
}

moe_status_t attention(const char* call, bool decode, const moe_kv_t* kv, int32_t layer, const void* q, int64_t ldq,
                       const int32_t* seqs, const int32_t* cu, int32_t n, int32_t n_q, int32_t n_rows,
                       int32_t n_heads, float scale, int32_t window, int32_t sinks, void* out, int64_t ldo,
                       moe_stream_t stream) {
  moe::KvLayout l;
  int sms = 0;
  moe_status_t st = open_kv(call, kv, &l, &sms);
  if (st != MOE_OK) return st;
  if (layer < 0 || layer >= kv->n_layers) return fail(MOE_ERR_ARG, call, "layer out of range");
  if (n < 0 || n > 65536) return fail(MOE_ERR_ARG, call, "n outside 0..65536");
  if (decode && (n_q < 1 || n_q > 8)) return fail(MOE_ERR_ARG, call, "n_q outside 1..8");
  if (!decode && n_rows < 0) return fail(MOE_ERR_ARG, call, "n_rows < 0");
  if (!seqs && n > kv->max_seqs) return fail(MOE_ERR_ARG, call, "n above max_seqs without seqs");
  if (n_heads < 1 || n_heads % kv->n_kv_heads || n_heads / kv->n_kv_heads > 64)
    return fail(MOE_ERR_ARG, call, "n_heads is not a multiple of n_kv_heads, or above 64 times as many");
  if (!std::isfinite(scale) || !(scale > 0.f)) return fail(MOE_ERR_ARG, call, "scale is not finite and positive");
  if (window < 0 || sinks < 0) return fail(MOE_ERR_ARG, call, "window or sinks < 0");
  const int32_t rows = decode ? n * n_q : n_rows;
  if (!decode && n == 0 && n_rows > 0) return fail(MOE_ERR_ARG, call, "rows without a sequence (n is 0)");
  if (rows == 0) return MOE_OK;
  if (!q || !out || (!decode && !cu)) return fail(MOE_ERR_ARG, call, "q, out or cu is NULL");
  const int64_t width = static_cast<int64_t>(n_heads) * kv->head_dim;
  const int per = 16 / token_elem_bytes(*kv);
  if (!aligned16(q) || !aligned16(out) || ldq % per || ldo % per)
    return fail(MOE_ERR_ARG, call, "rows of q or out are not 16-byte aligned");
  if (ldq < width || ldo < width) return fail(MOE_ERR_ARG, call, "ldq or ldo is smaller than a row");
  if (!decode && rows > 1 << 30) return fail(MOE_ERR_ARG, call, "n_rows above 2^30");
  // one CTA's index space of the prefill grid
  if (!decode && (static_cast<int64_t>(rows) * (n_heads / kv->n_kv_heads) / 16 + n + 1) * kv->n_kv_heads > 0x7FFFFFFFll)
    return fail(MOE_ERR_ARG, call, "too many rows for one call");
  moe::AttnArgs a{};
  a.q = q;
  a.out = out;
  a.k = static_cast<const char*>(kv->k) + layer * moe::layer_bytes(*kv);
  a.v = static_cast<const char*>(kv->v) + layer * moe::layer_bytes(*kv);
  a.table = kv->table;
  a.lens = kv->lens;
  a.seqs = seqs;
  a.cu = decode ? nullptr : cu;
  a.ldq = ldq;
  a.ldo = ldo;
  a.wide_out = reinterpret_cast<uintptr_t>(out) % 32 == 0 && (ldo * token_elem_bytes(*kv)) % 32 == 0 &&
               (kv->head_dim * token_elem_bytes(*kv)) % 32 == 0;
  a.n = n;
  a.n_q = n_q;
  a.n_rows = rows;
  a.Hq = n_heads;
  a.Hkv = kv->n_kv_heads;
  a.g = n_heads / kv->n_kv_heads;
  a.D = kv->head_dim;
  a.page_shift = __builtin_ctz(kv->page_tokens);
  a.max_pages = kv->max_pages;
  a.max_seqs = kv->max_seqs;
  a.n_pages = kv->n_pages;
  a.scale_log2 = scale * 1.4426950408889634f;
  // a window that no row's past exceeds hides nothing
  const int32_t most = kv->max_pages * kv->page_tokens;
  a.window = window >= most ? 0 : window;
  a.sinks = std::min(sinks, most);
  char* w = static_cast<char*>(kv->work);
  a.part = reinterpret_cast<float*>(w + l.part);
  a.tickets = reinterpret_cast<unsigned int*>(w + l.tickets);
  a.cuts = reinterpret_cast<moe::Cut*>(w + l.cuts);
  a.err = &reinterpret_cast<moe::KvWork*>(w)->err;
  a.copies = static_cast<uint32_t>(t_hook.copies);
  a.wait_cycles = t_hook.wait_cycles > 0 ? t_hook.wait_cycles : moe::kPrefillWaitCycles;
  t_hook = WaitHook{};
  if (kv->dtype & MOE_KV_I4)
    return launched(call, decode ? moe::launch_attn_decode_codes(a, moe::token_type(*kv), sms, stream)
                                 : moe::launch_attn_prefill_codes(a, moe::token_type(*kv), sms, stream));
  return launched(call, decode ? moe::launch_attn_decode(a, kv->dtype, sms, stream)
                               : moe::launch_attn_prefill(a, kv->dtype, rows, sms, stream));
}

}  // namespace

namespace moe {

uint32_t next_write() {
  static std::atomic<uint32_t> number{0};
  return ++number;
}

KvLayout kv_layout(const moe_kv_t& kv, int num_sms) {
  KvLayout l;
  int64_t at = sizeof(KvWork);
  auto take = [&](int64_t bytes) {
    const int64_t p = at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  const int64_t list = static_cast<int64_t>(std::max(kv.n_pages, kMaxList)) * 4;
  l.src = take(list);
  l.dst = take(list);
  l.map = take(list);
  l.filled = take(kMaxList * 4ll);
  l.shr = take(kv.n_pages * 4ll);
  l.last = take(kv.n_pages * 4ll);
  l.tickets = take(num_sms * kPrefillTickets * 4ll);
  l.cuts = take(num_sms * static_cast<int64_t>(sizeof(Cut)));
  // two partial results a CTA: rows of (m, l, -, -, head size padded)
  const int64_t dp = kv.head_dim <= 64 ? 64 : (kv.head_dim <= 128 ? 128 : 256);
  const bool tc = token_type(kv) == MOE_BF16 && kv.head_dim <= kTcHeadDim;
  l.part = take(2ll * num_sms * (tc ? kPrefillPartRows : kPartRows) * (dp + 4) * 4);
  l.bytes = at;
  return l;
}

}  // namespace moe

extern "C" moe_status_t moe_kv_work_bytes(const moe_kv_t* kv, int64_t* bytes) {
  return guarded([&] {
    const char* call = "moe_kv_work_bytes";
    if (!kv || !bytes) return fail(MOE_ERR_ARG, call, "kv or bytes is NULL");
    if (const char* why = bad_geometry(*kv)) return fail(MOE_ERR_ARG, call, why);
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return cuda_fail(call, e);
    *bytes = moe::kv_layout(*kv, sms).bytes;
    return MOE_OK;
  });
}

extern "C" moe_status_t moe_kv_check_errors(const moe_kv_t* kv, moe_stream_t stream) {
  return guarded([&] {
    const char* call = "moe_kv_check_errors";
    moe::KvLayout l;
    int sms = 0;
    moe_status_t st = open_kv(call, kv, &l, &sms);
    if (st != MOE_OK) return st;
    // both error words, with the count of planned copies between them
    constexpr size_t kHead = offsetof(moe::KvWork, late) + sizeof(uint64_t);
    moe::KvWork head{};
    cudaError_t e = cudaMemcpyAsync(&head, kv->work, kHead, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaMemsetAsync(kv->work, 0, kHead, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return cuda_fail(call, e);
    const uint32_t err = head.err | static_cast<uint32_t>(head.late);
    if (err & MOE_DEVERR_TIMEOUT) {
      // units left unjoined have left their tickets behind; gone before the return, for whichever stream is next
      e = cudaMemsetAsync(static_cast<char*>(kv->work) + l.tickets, 0, sms * moe::kPrefillTickets * 4, stream);
      if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
      if (e != cudaSuccess) return cuda_fail(call, e);
      return fail(MOE_ERR_TIMEOUT, call, "a bounded device wait ran out");
    }
    if (err & MOE_DEVERR_BADIDX)
      return fail(MOE_ERR_ARG, call, "a sequence or page id out of range or listed twice, or a fork into a sequence "
                                     "that holds tokens");
    if (err & MOE_DEVERR_CAPACITY) return fail(MOE_ERR_CAPACITY, call, "too few free pages, or a table row too short");
    if (err & moe::KV_DEVERR_SHARED)
      return fail(MOE_ERR_STATE, call, "a write to a shared page or past a sequence's length");
    return MOE_OK;
  });
}

extern "C" moe_status_t moe_debug_attn_wait_timeout(int64_t wait_cycles, int32_t copies) {
  return guarded([&] {
    if (wait_cycles < 0 || copies < -1)
      return fail(MOE_ERR_ARG, "moe_debug_attn_wait_timeout", "wait_cycles < 0 or copies < -1");
    t_hook = WaitHook{copies >= 0 ? wait_cycles : 0, copies};
    return MOE_OK;
  });
}

extern "C" moe_status_t moe_kv_fork(const moe_kv_t* kv, const int32_t* src, const int32_t* dst, int32_t n,
                                    moe_stream_t stream) {
  return guarded([&] {
    const char* call = "moe_kv_fork";
    moe::KvLayout l;
    int sms = 0;
    moe_status_t st = open_kv(call, kv, &l, &sms);
    if (st != MOE_OK) return st;
    if ((st = check_list(call, src, n)) != MOE_OK || (st = check_list(call, dst, n)) != MOE_OK) return st;
    if (n == 0) return MOE_OK;
    return launched(call, moe::launch_kv_fork(*kv, l, src, dst, n, stream));
  });
}

extern "C" moe_status_t moe_kv_reserve(const moe_kv_t* kv, const int32_t* seqs, const int32_t* n_new, int32_t n,
                                       moe_stream_t stream) {
  return guarded([&] {
    const char* call = "moe_kv_reserve";
    moe::KvLayout l;
    int sms = 0;
    moe_status_t st = open_kv(call, kv, &l, &sms);
    if (st != MOE_OK) return st;
    if ((st = check_list(call, seqs, n)) != MOE_OK || (st = check_list(call, n_new, n)) != MOE_OK) return st;
    if (n == 0) return MOE_OK;
    return launched(call, moe::launch_kv_reserve(*kv, l, seqs, n_new, n, sms, stream));
  });
}

extern "C" moe_status_t moe_kv_write(const moe_kv_t* kv, int32_t layer, const void* k_new, int64_t ldk,
                                     const void* v_new, int64_t ldv, const int32_t* seqs, const int32_t* cu,
                                     int32_t n, int32_t n_rows, moe_stream_t stream) {
  return guarded([&] {
    const char* call = "moe_kv_write";
    moe::KvLayout l;
    int sms = 0;
    bool none = false;
    moe_status_t st = open_rows(call, kv, layer, k_new, ldk, v_new, ldv, seqs, cu, n, n_rows, &l, &sms, &none);
    if (st != MOE_OK || none) return st;
    if (kv->dtype & MOE_KV_I4)
      return launched(call, moe::launch_kv_write_rotary(*kv, l, layer, moe::Rotary{}, nullptr, 0, 0, nullptr, 0, k_new, ldk, v_new,
                                                        ldv, seqs, cu, n, n_rows, sms, stream));
    return launched(call, moe::launch_kv_write(*kv, l, layer, k_new, ldk, v_new, ldv, seqs, cu, n, n_rows, stream));
  });
}

extern "C" moe_status_t moe_kv_write_rotary(const moe_kv_t* kv, int32_t layer, const moe_rotary_t* rot, const void* q,
                                            int64_t ldq, int32_t n_heads, void* q_out, int64_t ldqo, const void* k_new,
                                            int64_t ldk, const void* v_new, int64_t ldv, const int32_t* seqs,
                                            const int32_t* cu, int32_t n, int32_t n_rows, moe_stream_t stream) {
  return guarded([&] {
    const char* call = "moe_kv_write_rotary";
    moe::KvLayout l;
    int sms = 0;
    bool none = false;
    moe_status_t st = open_rows(call, kv, layer, k_new, ldk, v_new, ldv, seqs, cu, n, n_rows, &l, &sms, &none);
    if (st != MOE_OK) return st;
    moe::Rotary r{};
    if ((st = open_rotary(call, rot, kv->head_dim, &r)) != MOE_OK) return st;
    if (n_heads < 1 || n_heads > 65536) return fail(MOE_ERR_ARG, call, "n_heads outside 1..65536");
    if (none) return MOE_OK;
    if (!q || !q_out) return fail(MOE_ERR_ARG, call, "q or q_out is NULL");
    if ((st = check_heads(call, q, ldq, q_out, ldqo, n_heads, kv->head_dim, moe::token_type(*kv))) != MOE_OK) return st;
    return launched(call, moe::launch_kv_write_rotary(*kv, l, layer, r, q, ldq, n_heads, q_out, ldqo, k_new, ldk, v_new, ldv,
                                                      seqs, cu, n, n_rows, sms, stream));
  });
}

extern "C" moe_status_t moe_kv_read(const moe_kv_t* kv, int32_t layer, void* k, int64_t ldk, void* v, int64_t ldv,
                                    const int32_t* seqs, const int32_t* cu, int32_t n, int32_t n_rows,
                                    moe_stream_t stream) {
  return guarded([&] {
    const char* call = "moe_kv_read";
    moe::KvLayout l;
    int sms = 0;
    bool none = false;
    moe_status_t st = open_rows(call, kv, layer, k, ldk, v, ldv, seqs, cu, n, n_rows, &l, &sms, &none);
    if (st != MOE_OK || none) return st;
    return launched(call, moe::launch_kv_read(*kv, l, layer, k, ldk, v, ldv, seqs, cu, n, n_rows, sms, stream));
  });
}

extern "C" moe_status_t moe_rotary_angles(int32_t dim, double base, double factor, int32_t context, double turns_low,
                                          double turns_high, double* angles) {
  return guarded([&] {
    const char* call = "moe_rotary_angles";
    if (dim < 2 || dim % 2 || dim > 65536) return fail(MOE_ERR_ARG, call, "dim is not an even number in 2..65536");
    if (!(base > 0.0) || !std::isfinite(base)) return fail(MOE_ERR_ARG, call, "base is not finite and positive");
    if (!(factor > 0.0) || !std::isfinite(factor)) return fail(MOE_ERR_ARG, call, "factor is not finite and positive");
    if (context < 0) return fail(MOE_ERR_ARG, call, "context < 0");
    if (context > 0 && !(turns_high > turns_low && std::isfinite(turns_low) && std::isfinite(turns_high)))
      return fail(MOE_ERR_ARG, call, "turns_high is not above turns_low, or not finite");
    if (!angles) return fail(MOE_ERR_ARG, call, "angles is NULL");
    constexpr double kTurn = 6.283185307179586476925;
    for (int32_t i = 0; i < dim / 2; ++i) {
      const double f = std::pow(base, -2.0 * i / dim);
      double keep = 0.0;  // the share of the frequency that is not stretched
      if (context > 0) keep = std::min(1.0, std::max(0.0, (f * context / kTurn - turns_low) / (turns_high - turns_low)));
      angles[i] = f * (keep + (1.0 - keep) / factor);
    }
    return MOE_OK;
  });
}

extern "C" moe_status_t moe_rotary_turns(const double* angles, int32_t n, uint64_t* turns) {
  return guarded([&] {
    const char* call = "moe_rotary_turns";
    if (n < 0 || (n > 0 && (!angles || !turns))) return fail(MOE_ERR_ARG, call, "n < 0, or angles or turns is NULL");
    constexpr double kTurn = 6.283185307179586476925;
    for (int32_t i = 0; i < n; ++i)
      if (!std::isfinite(angles[i])) return fail(MOE_ERR_ARG, call, "an angle is not finite");
    for (int32_t i = 0; i < n; ++i) {
      double t = angles[i] / kTurn;
      t -= std::floor(t);  // whole turns are none
      turns[i] = t >= 1.0 ? 0 : static_cast<uint64_t>(t * 18446744073709551616.0);
    }
    return MOE_OK;
  });
}

extern "C" moe_status_t moe_rotary(const moe_rotary_t* rot, const int32_t* pos, const void* x, int32_t xt, int64_t ldx,
                                   int32_t n_rows, int32_t n_heads, int32_t head_dim, void* y, int64_t ldy,
                                   moe_stream_t stream) {
  return guarded([&] {
    const char* call = "moe_rotary";
    if (xt != MOE_F32 && xt != MOE_BF16) return fail(MOE_ERR_ARG, call, "x is neither MOE_F32 nor MOE_BF16");
    if (head_dim < 8 || head_dim > 256 || head_dim % 8) return fail(MOE_ERR_ARG, call, "head_dim is not a multiple of 8 in 8..256");
    moe::Rotary r{};
    moe_status_t st = open_rotary(call, rot, head_dim, &r);
    if (st != MOE_OK) return st;
    if (n_rows < 0 || n_rows > 1 << 30) return fail(MOE_ERR_ARG, call, "n_rows outside 0..2^30");
    if (n_heads < 1 || n_heads > 65536) return fail(MOE_ERR_ARG, call, "n_heads outside 1..65536");
    if (n_rows == 0) return MOE_OK;
    if (!pos || !x || !y) return fail(MOE_ERR_ARG, call, "pos, x or y is NULL");
    if ((st = check_heads(call, x, ldx, y, ldy, n_heads, head_dim, xt)) != MOE_OK) return st;
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return cuda_fail(call, e);
    return launched(call, moe::launch_rotary(r, pos, x, xt, ldx, y, ldy, n_rows, n_heads, head_dim, sms, stream));
  });
}

extern "C" moe_status_t moe_kv_free(const moe_kv_t* kv, const int32_t* seqs, int32_t n, moe_stream_t stream) {
  return guarded([&] {
    const char* call = "moe_kv_free";
    moe::KvLayout l;
    int sms = 0;
    moe_status_t st = open_kv(call, kv, &l, &sms);
    if (st != MOE_OK) return st;
    if ((st = check_list(call, seqs, n)) != MOE_OK) return st;
    if (n == 0) return MOE_OK;
    return launched(call, moe::launch_kv_free(*kv, l, seqs, n, stream));
  });
}

extern "C" moe_status_t moe_kv_compact(const moe_kv_t* kv, moe_stream_t stream) {
  return guarded([&] {
    const char* call = "moe_kv_compact";
    moe::KvLayout l;
    int sms = 0;
    moe_status_t st = open_kv(call, kv, &l, &sms);
    if (st != MOE_OK) return st;
    return launched(call, moe::launch_kv_compact(*kv, l, sms, stream));
  });
}

extern "C" moe_status_t moe_kv_copy_pages(const moe_kv_t* kv, const int32_t* src, const int32_t* dst, int32_t n,
                                          moe_stream_t stream) {
  return guarded([&] {
    const char* call = "moe_kv_copy_pages";
    moe::KvLayout l;
    int sms = 0;
    moe_status_t st = open_kv(call, kv, &l, &sms);
    if (st != MOE_OK) return st;
    if (n < 0) return fail(MOE_ERR_ARG, call, "n < 0");
    if (n == 0) return MOE_OK;
    if (!src || !dst) return fail(MOE_ERR_ARG, call, "a list is NULL");
    return launched(call, moe::launch_kv_copy_pages(*kv, l, src, dst, n, sms, stream));
  });
}

extern "C" moe_status_t moe_attn_decode(const moe_kv_t* kv, int32_t layer, const void* q, int64_t ldq,
                                        const int32_t* seqs, int32_t n, int32_t n_q, int32_t n_heads, float scale,
                                        int32_t window, int32_t sinks, void* out, int64_t ldo, moe_stream_t stream) {
  return guarded([&] {
    return attention("moe_attn_decode", true, kv, layer, q, ldq, seqs, nullptr, n, n_q, 0, n_heads, scale, window,
                     sinks, out, ldo, stream);
  });
}

extern "C" moe_status_t moe_attn_prefill(const moe_kv_t* kv, int32_t layer, const void* q, int64_t ldq,
                                         const int32_t* seqs, const int32_t* cu, int32_t n, int32_t n_rows,
                                         int32_t n_heads, float scale, int32_t window, int32_t sinks, void* out,
                                         int64_t ldo, moe_stream_t stream) {
  return guarded([&] {
    return attention("moe_attn_prefill", false, kv, layer, q, ldq, seqs, cu, n, 0, n_rows, n_heads, scale, window,
                     sinks, out, ldo, stream);
  });
}

extern "C" moe_status_t moe_quant_linear(const void* w, int32_t quant, int32_t N, int32_t K, const void* x, int32_t xt,
                                         int64_t ldx, int32_t T, const float* bias, void* y, int32_t yt, int64_t ldy,
                                         moe_stream_t stream) {
  return guarded([&] {
    const char* call = "moe_quant_linear";
    if (quant != MOE_Q4_0 && quant != MOE_I4_G64) return fail(MOE_ERR_ARG, call, "quant is neither MOE_Q4_0 nor MOE_I4_G64");
    const int group = quant == MOE_Q4_0 ? 32 : 64;
    if (N < 1 || K < group || K % group) return fail(MOE_ERR_ARG, call, "N < 1, or K not a positive multiple of the group");
    // offsets within a tile of rows are 32 bits, row numbers 31
    if (K >= 1 << 25 || N > 0x7FFFFFFF - 512) return fail(MOE_ERR_ARG, call, "K above 2^25 - 1 or N above 2^31 - 513");
    if ((xt != MOE_F32 && xt != MOE_BF16) || (yt != MOE_F32 && yt != MOE_BF16))
      return fail(MOE_ERR_ARG, call, "x or y is neither MOE_F32 nor MOE_BF16");
    if (T < 0) return fail(MOE_ERR_ARG, call, "T < 0");
    if (T == 0) return MOE_OK;
    if (!w || !x || !y) return fail(MOE_ERR_ARG, call, "w, x or y is NULL");
    if (!aligned16(w) || !aligned16(x) || ldx % (16 / elem_bytes(xt)))
      return fail(MOE_ERR_ARG, call, "w or the rows of x are not 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(y) % elem_bytes(yt)) || (reinterpret_cast<uintptr_t>(bias) % 4))
      return fail(MOE_ERR_ARG, call, "y or bias is not aligned to its type");
    if (ldx < K || ldy < N) return fail(MOE_ERR_ARG, call, "ldx or ldy is smaller than a row");
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return cuda_fail(call, e);
    moe::LinearArgs a{};
    a.w = static_cast<const uint8_t*>(w);
    a.meta = a.w + static_cast<int64_t>(N) * (K / 2);
    a.x = x;
    a.bias = bias;
    a.y = y;
    a.ldx = ldx;
    a.ldy = ldy;
    a.N = N;
    a.K = K;
    a.T = T;
    a.xt = xt;
    a.yt = yt;
    return launched(call, moe::launch_quant_linear(a, quant, sms, stream));
  });
}

extern "C" moe_status_t moe_sample(const void* logits, int32_t zt, int64_t ld, int32_t rows, int32_t V, const float* u,
                                   const moe_sampling_t* by, int32_t* token, float* prob, moe_stream_t stream) {
  return guarded([&] {
    const char* call = "moe_sample";
    if (zt != MOE_F32 && zt != MOE_BF16) return fail(MOE_ERR_ARG, call, "logits are neither MOE_F32 nor MOE_BF16");
    if (V < 1 || V > 1 << 20) return fail(MOE_ERR_ARG, call, "V outside 1..2^20");
    if (rows < 0 || rows > 1 << 24) return fail(MOE_ERR_ARG, call, "rows outside 0..2^24");
    if (!by) return fail(MOE_ERR_ARG, call, "by is NULL");
    if (rows == 0) return MOE_OK;
    if (!logits || !u || !token) return fail(MOE_ERR_ARG, call, "logits, u or token is NULL");
    if (ld < V && ld != 0) return fail(MOE_ERR_ARG, call, "ld is smaller than a row, and not 0");
    auto unaligned = [](const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) % bytes) != 0; };
    if (unaligned(logits, elem_bytes(zt)) || unaligned(u, 4) || unaligned(token, 4) || unaligned(prob, 4) ||
        unaligned(by->temperatures, 4) || unaligned(by->top_ks, 4) || unaligned(by->top_ps, 4) || unaligned(by->min_ps, 4))
      return fail(MOE_ERR_ARG, call, "a pointer is not aligned to its type");
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return cuda_fail(call, e);
    return launched(call, moe::launch_sample(logits, zt, ld, rows, V, u, *by, token, prob, sms, stream));
  });
}
