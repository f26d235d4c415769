// kv_attend_bf16.cu -- il_kv_attend over a bf16 cache (see kv_attend.cuh), and the plan of a
// call for either format.
#include "kv_attend.cuh"

namespace il {

cudaError_t prepare_kv_attend_bf16(const KvAttendPlan& p, int dim, bool wide, int ctas, Launch* out) {
  return attend::prepare_format<false>(p, dim, wide, ctas, out);
}

namespace {

int padded_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

bool wide_block(const KvAttendArgs& a) { return a.n_q_heads / a.kv.n_heads > 8; }

}  // namespace

// The counters, and two parts for each CTA of the grid, one CTA per SM: the largest part is 16 rows of 256 columns
// in two halves, each with the rows' maxima and sums.
size_t kv_workspace_bytes(int num_sms) { return kKvCounterBytes + (size_t)num_sms * 2 * 16 * (256 + 4) * sizeof(float); }

cudaError_t prepare_kv_attend(const KvAttendArgs& a, int num_sms, void* ws, Launch* out) {
  static_assert(attend::kMaxCtas * sizeof(unsigned) <= kKvCounterBytes, "a counter for each CTA");
  num_sms = std::min(num_sms, attend::kMaxCtas);
  const bool wide = wide_block(a);
  KvAttendPlan p{};
  p.a = a;
  p.cap = (int)std::min<int64_t>(a.table_width * a.kv.page_size, INT32_MAX);
  p.window = (int)std::min<int64_t>(a.window, INT32_MAX);
  p.by_page = FastDiv((uint32_t)a.kv.page_size);
  p.group = a.n_q_heads / a.kv.n_heads;
  p.blocks = (p.group + (wide ? 15 : 7)) / (wide ? 16 : 8);
  p.by_blocks = FastDiv((uint32_t)p.blocks);
  p.q_scale = a.scale * 1.4426950408889634f;
  // Simple copies: pages of whole groups of 16 tokens; strides of 32 bits; a token's scales copied as 16 bytes (8 for heads of
  // 64) where they are aligned and all of a padded row exists
  const KvView& kv = a.kv;
  const bool q8 = kv.format == IL_Q8;
  const int dim = padded_dim(kv.head_dim), unit = dim == 64 ? 2 : 4;
  const int64_t es = q8 ? 1 : 2;
  const auto fits = [&](int64_t page, int64_t token, int64_t head) {
    return page <= UINT32_MAX && token * kv.page_size + head * kv.n_heads <= INT32_MAX;
  };
  const auto even = [&](int64_t stride) { return stride % unit == 0; };
  const uintptr_t bases = reinterpret_cast<uintptr_t>(kv.k_scale) | reinterpret_cast<uintptr_t>(kv.v_scale);
  p.simple = kv.page_size % attend::kGroup == 0 && fits(kv.page * es, kv.token * es, kv.head * es);
  if (q8 && p.simple)
    p.simple = kv.head_dim == dim && fits(kv.spage * 4, kv.stoken * 4, kv.shead * 4) && bases % (4 * unit) == 0 &&
               even(kv.spage) && even(kv.stoken) && even(kv.shead);
  p.page_bytes = (uint32_t)(kv.page * es), p.token_bytes = (uint32_t)(kv.token * es), p.head_bytes = (uint32_t)(kv.head * es);
  p.spage_bytes = (uint32_t)(kv.spage * 4), p.stoken_bytes = (uint32_t)(kv.stoken * 4);
  p.shead_bytes = (uint32_t)(kv.shead * 4);
  p.arrived = static_cast<unsigned*>(ws);
  p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kKvCounterBytes);
  return a.kv.format == IL_Q8 ? prepare_kv_attend_q8(p, dim, wide, num_sms, out)
                              : prepare_kv_attend_bf16(p, dim, wide, num_sms, out);
}

}  // namespace il
