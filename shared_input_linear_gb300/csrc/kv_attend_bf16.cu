// kv_attend_bf16.cu -- il_kv_attend over a bf16 cache (see kv_attend.cuh), and the plan of a
// call for any format.
#include "kv_attend.cuh"

namespace il {

cudaError_t prepare_kv_attend_bf16(const KvAttendPlan& p, int dim, int blocks, int ctas, Launch* out) {
  return attend::prepare_format<IL_BF16, false>(p, dim, blocks, ctas, out);
}

namespace {

int padded_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

// Whether query heads are in the MMAs' columns: A4, and Q8 with scores (one query head a K/V head, biased, 32 sequences
// of up to 4096 tokens: with 8 rows for it 85.4 us, in columns 78.6).  Plain Q8 keeps the order that its bits came from.
bool in_columns(const KvAttendArgs& a) { return a.kv.format == IL_A4 || (a.kv.format == IL_Q8 && a.scored); }

// Blocks of 8 (in columns: 4) query heads that a warp takes at once.  In columns 8 heads at most: larger groups read K and V
// again, from L2, where 16 heads' sums would not fit the registers (128 heads on 8 of 128, 32 sequences of 4096: 143 us;
// two blocks of 8 117 us then, 123 after the steps that followed).
int head_blocks(const KvAttendArgs& a) {
  const int group = a.n_q_heads / a.kv.n_heads;
  return group > (in_columns(a) ? 4 : 8) ? 2 : 1;
}

}  // namespace

// The counters, and two parts for each CTA of the grid, one CTA per SM: the largest part is 16 rows of 256 columns
// in two halves, each with the rows' maxima and sums.
size_t kv_workspace_bytes(int num_sms) { return kKvCounterBytes + (size_t)num_sms * 2 * 16 * (256 + 4) * sizeof(float); }

cudaError_t prepare_kv_attend(const KvAttendArgs& a, int num_sms, void* ws, Launch* out) {
  static_assert(attend::kMaxCtas * sizeof(unsigned) <= kKvCounterBytes, "a counter for each CTA");
  num_sms = std::min(num_sms, attend::kMaxCtas);
  const int per_warp = head_blocks(a), rows = per_warp * (in_columns(a) ? 4 : 8);
  KvAttendPlan p{};
  p.a = a;
  p.cap = (int)std::min<int64_t>(a.table_width * a.kv.page_size, INT32_MAX);
  p.window = (int)std::min<int64_t>(a.window, INT32_MAX);
  p.by_page = FastDiv((uint32_t)a.kv.page_size);
  p.group = a.n_q_heads / a.kv.n_heads;
  p.blocks = (p.group + rows - 1) / rows;
  p.by_blocks = FastDiv((uint32_t)p.blocks);
  p.q_scale = a.cap > 0.f ? a.scale / a.cap : a.scale * 1.4426950408889634f;
  p.cap_log2 = a.cap * 1.4426950408889634f;
  if (a.positions != nullptr) p.cap = (int)std::min<int64_t>(p.cap, a.positions_width);
  // Simple copies: pages of whole groups of 16 tokens; strides of 32 bits; a token's scales copied as 16 bytes (8 for heads of
  // 64) where they are aligned and all of a padded row exists
  const KvView& kv = a.kv;
  const bool scaled = kv.format != IL_BF16;
  const int dim = padded_dim(kv.head_dim), unit = dim == 64 ? 2 : 4;
  const int64_t es = scaled ? 1 : 2;  // bytes of what the strides count
  const auto fits = [&](int64_t page, int64_t token, int64_t head) {
    return page <= UINT32_MAX && token * kv.page_size + head * kv.n_heads <= INT32_MAX;
  };
  const auto even = [&](int64_t stride) { return stride % unit == 0; };
  const uintptr_t bases = reinterpret_cast<uintptr_t>(kv.k_scale) | reinterpret_cast<uintptr_t>(kv.v_scale);
  p.simple = kv.page_size % attend::kGroup == 0 && fits(kv.page * es, kv.token * es, kv.head * es);
  if (scaled && p.simple)
    p.simple = kv.head_dim == dim && fits(kv.spage * 4, kv.stoken * 4, kv.shead * 4) && bases % (4 * unit) == 0 &&
               even(kv.spage) && even(kv.stoken) && even(kv.shead);
  if (in_columns(a)) {
    // offsets in 16 bytes and in pairs of steps fit 32 bits
    const auto ends = [&](int64_t page, int64_t token, int64_t head) {
      return (kv.n_pages - 1) * page + (kv.page_size - 1) * token + (kv.n_heads - 1) * head <= UINT32_MAX;
    };
    p.simple = kv.head_dim == dim && bases % (4 * unit) == 0 && even(kv.spage) && even(kv.stoken) && even(kv.shead) &&
               ends(kv.page / 16, kv.token / 16, kv.head / 16) && ends(kv.spage, kv.stoken, kv.shead);
  }
  p.page_bytes = (uint32_t)(kv.page * es), p.token_bytes = (uint32_t)(kv.token * es), p.head_bytes = (uint32_t)(kv.head * es);
  p.spage_bytes = (uint32_t)(kv.spage * 4), p.stoken_bytes = (uint32_t)(kv.stoken * 4);
  p.shead_bytes = (uint32_t)(kv.shead * 4);
  if (in_columns(a)) {
    p.page_bytes = (uint32_t)(kv.page / 16), p.token_bytes = (uint32_t)(kv.token / 16), p.head_bytes = (uint32_t)(kv.head / 16);
    p.spage_bytes = (uint32_t)kv.spage, p.stoken_bytes = (uint32_t)kv.stoken, p.shead_bytes = (uint32_t)kv.shead;
  }
  p.arrived = static_cast<unsigned*>(ws);
  p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kKvCounterBytes);
  if (a.scored) {
    const auto prepare = kv.format == IL_BF16 ? prepare_kv_attend_bf16_scored
                         : kv.format == IL_Q8 ? prepare_kv_attend_q8_scored
                                              : prepare_kv_attend_a4_scored;
    return prepare(p, dim, per_warp, num_sms, out);
  }
  const auto prepare = kv.format == IL_BF16 ? prepare_kv_attend_bf16
                       : kv.format == IL_Q8 ? prepare_kv_attend_q8
                                            : prepare_kv_attend_a4;
  return prepare(p, dim, per_warp, num_sms, out);
}

}  // namespace il
