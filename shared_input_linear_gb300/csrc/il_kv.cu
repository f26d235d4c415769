// il_kv.cu -- entry points of the paged K/V cache (include/il.h: il_kv_extend, il_kv_append, il_kv_read,
// il_kv_attend, il_kv_attend_scored, il_kv_weigh, il_kv_evict): every argument that the host can see is checked and
// the launch prepared before it is enqueued, as in the matmul entry points.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "il_internal.cuh"

using namespace il;

namespace {

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

int bad(int code, const char* fn, const char* what) {
  char buf[256];
  snprintf(buf, sizeof buf, "%s: %s", fn, what);
  return api_fail(code, buf);
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

struct Range {
  const void* p;
  int64_t bytes;
  bool written;
};

// Whether two ranges overlap of which at least one is written.
bool clash(const Range& a, const Range& b) {
  if (a.p == nullptr || b.p == nullptr || a.bytes <= 0 || b.bytes <= 0 || !(a.written || b.written)) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + (uintptr_t)b.bytes && b0 < a0 + (uintptr_t)a.bytes;
}

// Whether n rows of `row` floats at a and at b lie side by side, as columns of one buffer.
bool side_by_side(const float* a, int64_t a_stride, const float* b, int64_t b_stride, int64_t n, int64_t row) {
  if (n <= 1 || a_stride != b_stride || a_stride <= 0) return false;
  const int64_t apart = std::abs((int64_t)(reinterpret_cast<intptr_t>(a) - reinterpret_cast<intptr_t>(b))) / 4 % a_stride;
  return apart >= row && a_stride - apart >= row;
}

// Strides of one pool: positive multiples of `unit`, at least a row where the dimension has
// more than one entry, and an extent that 64-bit offsets hold.
bool stride_ok(int64_t s, int64_t extent, int64_t row, int64_t unit) {
  return extent <= 1 || (s >= row && s % unit == 0 && s <= (INT64_MAX >> 4) / extent);
}

int check_cache(const char* fn, const il_kv* kv, KvView* out) {
  if (kv == nullptr) return bad(IL_ERR_ARG, fn, "kv is NULL");
  if (kv->format != IL_BF16 && kv->format != IL_Q8 && kv->format != IL_A4)
    return bad(IL_ERR_FORMAT, fn, "the cache must be IL_BF16, IL_Q8 or IL_A4");
  const bool blocks_of_32 = kv->format != IL_BF16;
  if (kv->page_size < 1 || kv->page_size > (1 << 20) || kv->n_pages < 1 || kv->n_pages > INT32_MAX / kv->page_size)
    return bad(IL_ERR_SHAPE, fn, "page_size or n_pages out of range");
  if (kv->n_heads < 1 || kv->n_heads > 1024) return bad(IL_ERR_SHAPE, fn, "n_heads out of range");
  if (kv->head_dim < 8 || kv->head_dim > kMaxKvDim || kv->head_dim % (blocks_of_32 ? 32 : 8) != 0)
    return bad(IL_ERR_SHAPE, fn, "head_dim must be at most 256 and a multiple of 8 (bf16) or of 32 (Q8, A4)");
  if (kv->k == nullptr || kv->v == nullptr) return bad(IL_ERR_ARG, fn, "the cache's k or v is NULL");
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16)) return bad(IL_ERR_ARG, fn, "the cache's k or v is not 16-byte aligned");
  const int64_t unit = blocks_of_32 ? 16 : 8, blocks = kv->head_dim / 32;
  const int64_t row = kv->format == IL_A4 ? kv->head_dim / 2 : kv->head_dim;  // in what the strides count
  if (!stride_ok(kv->page_stride, kv->n_pages, row, unit) || !stride_ok(kv->token_stride, kv->page_size, row, unit) ||
      !stride_ok(kv->head_stride, kv->n_heads, row, unit))
    return bad(IL_ERR_SHAPE, fn, "a stride of the cache is smaller than a row or not a multiple of 16 bytes");
  if (blocks_of_32) {
    if (kv->k_scale == nullptr || kv->v_scale == nullptr)
      return bad(IL_ERR_ARG, fn, "a Q8 or A4 cache needs k_scale and v_scale");
    if (!aligned(kv->k_scale, 4) || !aligned(kv->v_scale, 4))
      return bad(IL_ERR_ARG, fn, "the cache's scales are not 4-byte aligned");
    if (!stride_ok(kv->scale_page_stride, kv->n_pages, blocks, 1) ||
        !stride_ok(kv->scale_token_stride, kv->page_size, blocks, 1) ||
        !stride_ok(kv->scale_head_stride, kv->n_heads, blocks, 1))
      return bad(IL_ERR_SHAPE, fn, "a stride of the cache's scales is smaller than a row");
  } else if (kv->k_scale != nullptr || kv->v_scale != nullptr) {
    return bad(IL_ERR_ARG, fn, "a bf16 cache has no scales");
  }
  KvView& w = *out;
  w.format = kv->format;
  w.page_size = kv->page_size;
  w.n_heads = kv->n_heads;
  w.head_dim = kv->head_dim;
  w.n_pages = kv->n_pages;
  w.n_slots = kv->n_pages * kv->page_size;
  w.k = static_cast<uint8_t*>(kv->k);
  w.v = static_cast<uint8_t*>(kv->v);
  w.k_scale = kv->k_scale;
  w.v_scale = kv->v_scale;
  w.page = kv->n_pages > 1 ? kv->page_stride : 0;
  w.token = kv->page_size > 1 ? kv->token_stride : 0;
  w.head = kv->n_heads > 1 ? kv->head_stride : 0;
  w.spage = kv->n_pages > 1 ? kv->scale_page_stride : 0;
  w.stoken = kv->page_size > 1 ? kv->scale_token_stride : 0;
  w.shead = kv->n_heads > 1 ? kv->scale_head_stride : 0;
  return IL_OK;
}

// Byte extent of a pool.
int64_t extent_bytes(const KvView& w, bool scales) {
  const int64_t last = (w.n_pages - 1) * (scales ? w.spage : w.page) + (w.page_size - 1) * (scales ? w.stoken : w.token) +
                       (w.n_heads - 1) * (scales ? w.shead : w.head);
  if (scales) return 4 * (last + w.head_dim / 32);
  return w.format == IL_BF16 ? 2 * (last + w.head_dim) : last + (w.format == IL_A4 ? w.head_dim / 2 : w.head_dim);
}

int enqueue(const char* fn, const Launch& L, void* stream) {
  int n = 0;
  const cudaError_t e = run_launches({L}, static_cast<cudaStream_t>(stream), &n);
  return e == cudaSuccess ? IL_OK : api_cuda_fail(e, fn);
}

int rows_call(const char* fn, bool write, const il_kv* kv, float* k, int64_t k_stride, float* v, int64_t v_stride,
              const int32_t* slots, int64_t n, void* stream) {
  NvtxRange range(fn);
  api_clear_error();
  KvView w;
  int rc = check_cache(fn, kv, &w);
  if (rc != IL_OK) return rc;
  if (n < 0 || n > INT32_MAX) return bad(IL_ERR_ARG, fn, "n out of range");
  if (n == 0) return IL_OK;
  if (k == nullptr || v == nullptr || slots == nullptr) return bad(IL_ERR_ARG, fn, "k, v and slots must not be NULL");
  if (!aligned(k, 16) || !aligned(v, 16)) return bad(IL_ERR_ARG, fn, "k or v is not 16-byte aligned");
  if (!aligned(slots, 4)) return bad(IL_ERR_ARG, fn, "slots is not 4-byte aligned");
  const int64_t row = (int64_t)w.n_heads * w.head_dim;
  if (n > 1 && (k_stride < row || v_stride < row || k_stride % 4 != 0 || v_stride % 4 != 0 ||
                k_stride > INT64_MAX / 8 / n || v_stride > INT64_MAX / 8 / n))
    return bad(IL_ERR_SHAPE, fn, "k_stride or v_stride is smaller than a row or not a multiple of 4");
  // k and v may be columns of one buffer: only what the kernel writes must lie apart from the rest,
  // and interleaved rows of k and v are told apart by their place in a row
  const int64_t kb = 4 * ((n - 1) * (n > 1 ? k_stride : 0) + row), vb = 4 * ((n - 1) * (n > 1 ? v_stride : 0) + row);
  const Range kr{k, kb, !write}, vr{v, vb, !write}, sr{slots, 4 * n, false};
  const Range ck{w.k, extent_bytes(w, false), write}, cv{w.v, extent_bytes(w, false), write};
  const Range ds{w.k_scale, extent_bytes(w, true), write}, dv{w.v_scale, extent_bytes(w, true), write};
  for (const Range& c : {ck, cv, ds, dv})
    for (const Range& r : {kr, vr, sr})
      if (clash(c, r)) return bad(IL_ERR_ARG, fn, "k, v and slots must not overlap the cache");
  if (clash(kr, sr) || clash(vr, sr)) return bad(IL_ERR_ARG, fn, "k and v must not overlap slots");
  if (!write && clash(kr, vr) && !side_by_side(k, k_stride, v, v_stride, n, row))
    return bad(IL_ERR_ARG, fn, "k and v must not overlap");
  int num_sms = 0;
  unsigned* status = nullptr;
  const int dev = api_device(&num_sms, &status);
  if (dev < 0) return dev;
  Launch L;
  const cudaError_t e = prepare_kv_rows(write, w, k, k_stride, v, v_stride, slots, n, status, num_sms, &L);
  if (e != cudaSuccess) return api_cuda_fail(e, fn);
  return enqueue(fn, L, stream);
}

// The parts of a score into `a` (nothing where score is nullptr).
int check_score(const char* fn, const il_kv_score* score, float scale, int64_t n_seq, KvAttendArgs* a) {
  if (score == nullptr) return IL_OK;
  const il_kv_score& c = *score;
  // (beyond these, cap log2(e) or q scale / cap leaves fp32 where the logit itself does not)
  if (!(c.cap == 0.0f || (c.cap >= 0x1p-100f && c.cap <= 0x1p100f))) return bad(IL_ERR_ARG, fn, "cap must be 0, or 2^-100 to 2^100");
  if (c.cap > 0.0f && !(scale / c.cap - scale / c.cap == 0.0f)) return bad(IL_ERR_ARG, fn, "scale / cap is not finite");
  if (!aligned(c.slopes, 4) || !aligned(c.starts, 4) || !aligned(c.positions, 4))
    return bad(IL_ERR_ARG, fn, "slopes, starts or positions is not 4-byte aligned");
  if (c.positions != nullptr &&
      (c.positions_width < 1 || c.positions_width > INT32_MAX ||
       (n_seq > 1 && (c.positions_stride < c.positions_width || c.positions_stride > INT32_MAX))))
    return bad(IL_ERR_SHAPE, fn, "positions_width or positions_stride out of range");
  a->scored = c.cap > 0.0f || c.slopes != nullptr || c.starts != nullptr;
  a->cap = c.cap;
  a->slopes = c.slopes;
  a->starts = c.starts;
  if (c.positions != nullptr) {
    a->positions = c.positions;
    a->positions_width = c.positions_width;
    a->positions_stride = n_seq > 1 ? c.positions_stride : 0;
  }
  return IL_OK;
}

// The arguments that il_kv_attend, il_kv_attend_scored and il_kv_weigh share, into `a`; score: nullptr or what it adds.  For n_seq = 0
// (a no-op) the arrays are not looked at.
int check_attended(const char* fn, const il_kv* kv, const float* q, int64_t q_stride, const int32_t* table, int64_t table_stride,
                   int64_t table_width, const int32_t* lens, int64_t n_seq, int64_t n_q_heads, float scale, int64_t window,
                   const il_kv_score* score, KvAttendArgs* a) {
  memset(a, 0, sizeof *a);
  int rc = check_cache(fn, kv, &a->kv);
  if (rc != IL_OK) return rc;
  if (n_seq < 0 || n_seq > kMaxKvSeqs) return bad(IL_ERR_ARG, fn, "n_seq out of range");
  if (n_q_heads < 1 || n_q_heads > 32768 || n_q_heads % a->kv.n_heads != 0)
    return bad(IL_ERR_SHAPE, fn, "n_q_heads must be a multiple of the cache's n_heads, at most 32768");
  if (window < 0) return bad(IL_ERR_ARG, fn, "window is negative");
  if (!(scale - scale == 0.0f)) return bad(IL_ERR_ARG, fn, "scale is not finite");
  rc = check_score(fn, score, scale, n_seq, a);
  if (rc != IL_OK || n_seq == 0) return rc;
  if (q == nullptr || table == nullptr || lens == nullptr) return bad(IL_ERR_ARG, fn, "q, table and lens must not be NULL");
  if (!aligned(q, 16)) return bad(IL_ERR_ARG, fn, "q is not 16-byte aligned");
  if (!aligned(table, 4) || !aligned(lens, 4)) return bad(IL_ERR_ARG, fn, "table or lens is not 4-byte aligned");
  if (n_seq > 1 && (q_stride < n_q_heads * a->kv.head_dim || q_stride % 4 != 0 || q_stride > INT64_MAX / 8 / n_seq))
    return bad(IL_ERR_SHAPE, fn, "q_stride is smaller than a row or not a multiple of 4");
  if (table_width < 1 || table_width > INT32_MAX || (n_seq > 1 && (table_stride < table_width || table_stride > INT32_MAX)))
    return bad(IL_ERR_SHAPE, fn, "table_width or table_stride out of range");
  a->q = q;
  a->q_stride = n_seq > 1 ? q_stride : 0;
  a->table = table;
  a->table_stride = n_seq > 1 ? table_stride : 0;
  a->table_width = table_width;
  a->lens = lens;
  a->n_seq = (int)n_seq;
  a->n_q_heads = (int)n_q_heads;
  a->scale = scale;
  a->window = window;
  return IL_OK;
}

// What a call of those arguments reads: q first.
struct Ranges {
  Range r[10];
};
Ranges ranges_of(const KvAttendArgs& a) {
  const int64_t n = a.n_seq, row = (int64_t)a.n_q_heads * a.kv.head_dim;
  return {{{a.q, 4 * ((n - 1) * a.q_stride + row), false},
           {a.table, 4 * ((n - 1) * a.table_stride + a.table_width), false},
           {a.lens, 4 * n, false},
           {a.kv.k, extent_bytes(a.kv, false), false},
           {a.kv.v, extent_bytes(a.kv, false), false},
           {a.kv.k_scale, extent_bytes(a.kv, true), false},
           {a.kv.v_scale, extent_bytes(a.kv, true), false},
           {a.slopes, 4 * (int64_t)a.n_q_heads, false},
           {a.starts, 4 * n, false},
           {a.positions, 4 * ((n - 1) * a.positions_stride + a.positions_width), false}}};
}

int attend_call(const char* fn, const il_kv* kv, const float* q, int64_t q_stride, const int32_t* table, int64_t table_stride,
                int64_t table_width, const int32_t* lens, int64_t n_seq, int64_t n_q_heads, float scale, int64_t window,
                const il_kv_score* score, float* out, int64_t out_stride, float* lse, void* stream) {
  NvtxRange range(fn);
  api_clear_error();
  KvAttendArgs a;
  int rc = check_attended(fn, kv, q, q_stride, table, table_stride, table_width, lens, n_seq, n_q_heads, scale, window, score, &a);
  if (rc != IL_OK || n_seq == 0) return rc;
  if (out == nullptr) return bad(IL_ERR_ARG, fn, "out must not be NULL");
  if (!aligned(out, 16)) return bad(IL_ERR_ARG, fn, "out is not 16-byte aligned");
  if (!aligned(lse, 4)) return bad(IL_ERR_ARG, fn, "lse is not 4-byte aligned");
  const int64_t row = n_q_heads * a.kv.head_dim;
  if (n_seq > 1 && (out_stride < row || out_stride % 4 != 0 || out_stride > INT64_MAX / 8 / n_seq))
    return bad(IL_ERR_SHAPE, fn, "out_stride is smaller than a row or not a multiple of 4");
  const int64_t os = n_seq > 1 ? out_stride : 0;
  const Range outs[] = {{out, 4 * ((n_seq - 1) * os + row), true}, {lse, 4 * n_seq * n_q_heads, true}};
  const Ranges ins = ranges_of(a);
  for (const Range& o : outs)
    for (const Range& i : ins.r)
      if (clash(o, i) && !(&o == outs && &i == ins.r && side_by_side(out, os, q, a.q_stride, n_seq, row)))
        return bad(IL_ERR_ARG, fn, "out and lse must not overlap q, table, lens, the score's arrays or the cache");
  if (clash(outs[0], outs[1])) return bad(IL_ERR_ARG, fn, "out and lse must not overlap");
  int num_sms = 0;
  const int dev = api_device(&num_sms, &a.status);
  if (dev < 0) return dev;
  a.out = out;
  a.out_stride = os;
  a.lse = lse;
  void* ws = nullptr;
  rc = api_kv_workspace(dev, static_cast<cudaStream_t>(stream), num_sms, &ws);
  if (rc != IL_OK) return rc;
  Launch L;
  const cudaError_t e = prepare_kv_attend(a, num_sms, ws, &L);
  if (e != cudaSuccess) return api_cuda_fail(e, fn);
  return enqueue(fn, L, stream);
}

constexpr int64_t kMaxWeightsRow = 1 << 30;

// Rows of one number a token, [n_seq][width].
int check_side(const char* fn, const void* in, const void* out, int64_t stride, int64_t width, int64_t n_seq, const char* what) {
  char buf[96];
  snprintf(buf, sizeof buf, "%s: NULL, not 4-byte aligned, or a width or stride out of range", what);
  if (in == nullptr || out == nullptr || !aligned(in, 4) || !aligned(out, 4)) return bad(IL_ERR_ARG, fn, buf);
  if (width < 1 || width > kMaxWeightsRow || (n_seq > 1 && (stride < width || stride > INT32_MAX))) return bad(IL_ERR_SHAPE, fn, buf);
  return IL_OK;
}

}  // namespace

extern "C" {

int il_kv_extend(int64_t n_seq, int64_t page_size, const int32_t* lens, const int32_t* add, int32_t* table,
                 int64_t table_stride, int64_t table_width, int32_t* ring, int64_t ring_size, const int64_t* cursor,
                 int32_t* lens_out, int64_t* cursor_out, int32_t* slots, int64_t max_slots, int32_t* positions,
                 int32_t* first, int64_t* info, void* stream) try {
  const char* fn = "il_kv_extend";
  NvtxRange range(fn);
  api_clear_error();
  if (n_seq < 0 || n_seq > kMaxKvSeqs) return bad(IL_ERR_ARG, fn, "n_seq out of range");
  if (page_size < 1 || page_size > (1 << 20)) return bad(IL_ERR_SHAPE, fn, "page_size out of range");
  if (n_seq == 0) return IL_OK;
  if (lens == nullptr || add == nullptr || table == nullptr || ring == nullptr || cursor == nullptr ||
      lens_out == nullptr || cursor_out == nullptr || (slots == nullptr && max_slots != 0))
    return bad(IL_ERR_ARG, fn, "lens, add, table, ring, cursor, lens_out, cursor_out and slots must not be NULL");
  if (max_slots < 0 || max_slots > INT32_MAX) return bad(IL_ERR_ARG, fn, "max_slots out of range");
  if (table_width < 1 || table_width > INT32_MAX || (n_seq > 1 && (table_stride < table_width || table_stride > INT32_MAX)))
    return bad(IL_ERR_SHAPE, fn, "table_width or table_stride out of range");
  if (ring_size < 1 || ring_size > INT32_MAX) return bad(IL_ERR_SHAPE, fn, "ring_size out of range");
  for (const void* p : {(const void*)lens, (const void*)add, (const void*)table, (const void*)ring, (const void*)lens_out,
                        (const void*)slots, (const void*)positions, (const void*)first})
    if (!aligned(p, 4)) return bad(IL_ERR_ARG, fn, "an int32 array is not 4-byte aligned");
  if (!aligned(cursor, 8) || !aligned(cursor_out, 8) || !aligned(info, 8))
    return bad(IL_ERR_ARG, fn, "an int64 array is not 8-byte aligned");
  const Range rs[] = {{lens, 4 * n_seq, false},
                      {add, 4 * n_seq, false},
                      {cursor, 16, false},
                      {table, 4 * ((n_seq - 1) * (n_seq > 1 ? table_stride : 0) + table_width), true},
                      {ring, 4 * ring_size, true},
                      {lens_out == lens ? nullptr : lens_out, 4 * n_seq, true},
                      {cursor_out == cursor ? nullptr : cursor_out, 16, true},
                      {slots, 4 * max_slots, true},
                      {positions, 4 * max_slots, true},
                      {first, 4 * (n_seq + 1), true},
                      {info, 32, true}};
  const Range in_place[] = {{lens_out, 4 * n_seq, true}, {cursor_out, 16, true}};
  const int n = (int)(sizeof rs / sizeof rs[0]);
  for (int i = 0; i < n; ++i) {
    for (int j = i + 1; j < n; ++j)
      if (clash(rs[i], rs[j])) return bad(IL_ERR_ARG, fn, "the outputs must not overlap each other or an input");
    // a state updated in place is an output too
    if (i != 0 && i != 5 && clash(in_place[0], rs[i])) return bad(IL_ERR_ARG, fn, "lens_out overlaps another array");
    if (i != 2 && i != 6 && clash(in_place[1], rs[i])) return bad(IL_ERR_ARG, fn, "cursor_out overlaps another array");
  }
  int num_sms = 0;
  unsigned* status = nullptr;
  const int dev = api_device(&num_sms, &status);
  if (dev < 0) return dev;
  void* ws = nullptr;
  const int rc = api_kv_workspace(dev, static_cast<cudaStream_t>(stream), num_sms, &ws);
  if (rc != IL_OK) return rc;
  KvExtendArgs a;
  memset(&a, 0, sizeof a);
  a.n_seq = (int)n_seq;
  a.page_size = (int)page_size;
  a.lens = lens;
  a.add = add;
  a.table = table;
  a.table_stride = n_seq > 1 ? table_stride : 0;
  a.table_width = table_width;
  a.ring = ring;
  a.ring_size = ring_size;
  a.cursor = cursor;
  a.lens_out = lens_out;
  a.cursor_out = cursor_out;
  a.slots = slots;
  a.max_slots = max_slots;
  a.positions = positions;
  a.first = first;
  a.info = info;
  a.arrived = static_cast<unsigned*>(ws);
  Launch L;
  const cudaError_t e = prepare_kv_extend(a, num_sms, &L);
  if (e != cudaSuccess) return api_cuda_fail(e, fn);
  return enqueue(fn, L, stream);
} catch (const std::bad_alloc&) {  // of the launch lists
  return api_cuda_fail(cudaErrorMemoryAllocation, "il_kv_extend");
}

int il_kv_append(const il_kv* kv, const float* k, int64_t k_stride, const float* v, int64_t v_stride,
                 const int32_t* slots, int64_t n, void* stream) try {
  return rows_call("il_kv_append", true, kv, const_cast<float*>(k), k_stride, const_cast<float*>(v), v_stride, slots, n,
                   stream);
} catch (const std::bad_alloc&) {  // of the launch lists
  return api_cuda_fail(cudaErrorMemoryAllocation, "il_kv_append");
}

int il_kv_read(const il_kv* kv, const int32_t* slots, int64_t n, float* k, int64_t k_stride, float* v, int64_t v_stride,
               void* stream) try {
  return rows_call("il_kv_read", false, kv, k, k_stride, v, v_stride, slots, n, stream);
} catch (const std::bad_alloc&) {  // of the launch lists
  return api_cuda_fail(cudaErrorMemoryAllocation, "il_kv_read");
}

int il_kv_attend(const il_kv* kv, const float* q, int64_t q_stride, const int32_t* table, int64_t table_stride,
                 int64_t table_width, const int32_t* lens, int64_t n_seq, int64_t n_q_heads, float scale, int64_t window,
                 float* out, int64_t out_stride, float* lse, void* stream) try {
  return attend_call("il_kv_attend", kv, q, q_stride, table, table_stride, table_width, lens, n_seq, n_q_heads, scale, window,
                     nullptr, out, out_stride, lse, stream);
} catch (const std::bad_alloc&) {  // of the launch lists
  return api_cuda_fail(cudaErrorMemoryAllocation, "il_kv_attend");
}

int il_kv_attend_scored(const il_kv* kv, const float* q, int64_t q_stride, const int32_t* table, int64_t table_stride,
                        int64_t table_width, const int32_t* lens, int64_t n_seq, int64_t n_q_heads, float scale,
                        int64_t window, const il_kv_score* score, float* out, int64_t out_stride, float* lse, void* stream) try {
  return attend_call("il_kv_attend_scored", kv, q, q_stride, table, table_stride, table_width, lens, n_seq, n_q_heads, scale,
                     window, score, out, out_stride, lse, stream);
} catch (const std::bad_alloc&) {  // of the launch lists
  return api_cuda_fail(cudaErrorMemoryAllocation, "il_kv_attend_scored");
}

int il_kv_weigh(const il_kv* kv, const float* q, int64_t q_stride, const int32_t* table, int64_t table_stride,
                int64_t table_width, const int32_t* lens, int64_t n_seq, int64_t n_q_heads, float scale, int64_t window,
                const il_kv_score* score, const float* lse, const int32_t* add, const float* weights, float* weights_out,
                int64_t weights_stride, int64_t weights_width, void* stream) try {
  const char* fn = "il_kv_weigh";
  NvtxRange range(fn);
  api_clear_error();
  KvWeighArgs w;
  KvAttendArgs& a = w.attend;
  int rc = check_attended(fn, kv, q, q_stride, table, table_stride, table_width, lens, n_seq, n_q_heads, scale, window, score, &a);
  if (rc != IL_OK || n_seq == 0) return rc;
  if (lse == nullptr) return bad(IL_ERR_ARG, fn, "lse must not be NULL");
  if (!aligned(lse, 4) || !aligned(add, 4)) return bad(IL_ERR_ARG, fn, "lse or add is not 4-byte aligned");
  rc = check_side(fn, weights, weights_out, weights_stride, weights_width, n_seq, "weights, weights_out");
  if (rc != IL_OK) return rc;
  w.add = add;
  w.weights = weights;
  w.weights_out = weights_out;
  w.weights_stride = n_seq > 1 ? weights_stride : 0;
  w.weights_width = weights_width;
  const int64_t bytes = 4 * ((n_seq - 1) * w.weights_stride + weights_width);
  const Range o{weights_out, bytes, true};
  const Range more[] = {{lse, 4 * n_seq * n_q_heads, false},
                        {add, 4 * n_seq, false},
                        {weights == weights_out ? nullptr : weights, bytes, false}};
  bool apart = true;
  for (const Range& i : ranges_of(a).r) apart &= !clash(o, i);
  for (const Range& i : more) apart &= !clash(o, i);
  if (!apart) return bad(IL_ERR_ARG, fn, "weights_out must not overlap an input, but for weights itself");
  int num_sms = 0;
  const int dev = api_device(&num_sms, &a.status);
  if (dev < 0) return dev;
  a.lse = const_cast<float*>(lse);
  Launch L;
  const cudaError_t e = prepare_kv_weigh(w, num_sms, &L);
  if (e != cudaSuccess) return api_cuda_fail(e, fn);
  return enqueue(fn, L, stream);
} catch (const std::bad_alloc&) {  // of the launch lists
  return api_cuda_fail(cudaErrorMemoryAllocation, "il_kv_weigh");
}

int il_kv_evict(const il_kv* kv, const int32_t* table, int64_t table_stride, int64_t table_width, const int32_t* lens,
                int64_t n_seq, int64_t keep, int64_t first, int64_t recent, const float* weights, float* weights_out,
                int64_t weights_stride, int64_t weights_width, const int32_t* positions, int32_t* positions_out,
                int64_t positions_stride, int64_t positions_width, int32_t* kept, int64_t kept_stride, int32_t* drop,
                void* stream) try {
  const char* fn = "il_kv_evict";
  NvtxRange range(fn);
  api_clear_error();
  KvEvictArgs a;
  memset(&a, 0, sizeof a);
  int rc = check_cache(fn, kv, &a.kv);
  if (rc != IL_OK) return rc;
  if (n_seq < 0 || n_seq > kMaxKvSeqs) return bad(IL_ERR_ARG, fn, "n_seq out of range");
  if (keep < 1 || keep > kMaxWeightsRow || first < 0 || recent < 0 || first > keep || recent > keep - first)
    return bad(IL_ERR_ARG, fn, "keep must be 1 to 2^30, first and recent not negative and together at most keep");
  if (n_seq == 0) return IL_OK;
  if (table == nullptr || lens == nullptr || kept == nullptr || drop == nullptr)
    return bad(IL_ERR_ARG, fn, "table, lens, kept and drop must not be NULL");
  if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(kept, 4) || !aligned(drop, 4))
    return bad(IL_ERR_ARG, fn, "table, lens, kept or drop is not 4-byte aligned");
  if (table_width < 1 || table_width > INT32_MAX || (n_seq > 1 && (table_stride < table_width || table_stride > INT32_MAX)))
    return bad(IL_ERR_SHAPE, fn, "table_width or table_stride out of range");
  if (n_seq > 1 && (kept_stride < keep || kept_stride > INT32_MAX)) return bad(IL_ERR_SHAPE, fn, "kept_stride out of range");
  rc = check_side(fn, weights, weights_out, weights_stride, weights_width, n_seq, "weights, weights_out");
  if (rc != IL_OK) return rc;
  if (positions != nullptr || positions_out != nullptr) {
    rc = check_side(fn, positions, positions_out, positions_stride, positions_width, n_seq, "positions, positions_out");
    if (rc != IL_OK) return rc;
    a.positions = positions;
    a.positions_out = positions_out;
    a.positions_stride = n_seq > 1 ? positions_stride : 0;
  }
  a.table = table;
  a.table_stride = n_seq > 1 ? table_stride : 0;
  a.lens = lens;
  a.n_seq = (int)n_seq;
  a.cap = (int)std::min({std::min<int64_t>(table_width * a.kv.page_size, INT32_MAX), weights_width,
                         positions != nullptr ? positions_width : INT32_MAX});
  a.keep = (int)keep;
  a.first = (int)first;
  a.recent = (int)recent;
  a.weights = weights;
  a.weights_out = weights_out;
  a.weights_stride = n_seq > 1 ? weights_stride : 0;
  a.kept = kept;
  a.kept_stride = n_seq > 1 ? kept_stride : 0;
  a.drop = drop;
  const int64_t wb = 4 * ((n_seq - 1) * a.weights_stride + weights_width);
  const int64_t pb = positions == nullptr ? 0 : 4 * ((n_seq - 1) * a.positions_stride + positions_width);
  // the cache is read and written; weights and positions may be their own outputs
  const Range rs[] = {{kept, 4 * ((n_seq - 1) * a.kept_stride + keep), true},
                      {drop, 4 * n_seq, true},
                      {weights_out, wb, true},
                      {positions_out, pb, true},
                      {a.kv.k, extent_bytes(a.kv, false), true},
                      {a.kv.v, extent_bytes(a.kv, false), true},
                      {a.kv.k_scale, extent_bytes(a.kv, true), true},
                      {a.kv.v_scale, extent_bytes(a.kv, true), true},
                      {weights == weights_out ? nullptr : weights, wb, false},
                      {positions == positions_out ? nullptr : positions, pb, false},
                      {table, 4 * ((n_seq - 1) * a.table_stride + table_width), false},
                      {lens, 4 * n_seq, false}};
  const int n_ranges = (int)(sizeof rs / sizeof rs[0]);
  for (int i = 0; i < n_ranges; ++i)
    for (int j = i + 1; j < n_ranges; ++j) {
      // K and V (and their scales) may be interleaved in one buffer
      const bool pools = i >= 4 && j <= 7;
      if (!pools && clash(rs[i], rs[j])) return bad(IL_ERR_ARG, fn, "the outputs and the cache must not overlap each other or an input");
    }
  int num_sms = 0;
  const int dev = api_device(&num_sms, &a.status);
  if (dev < 0) return dev;
  std::vector<Launch> launches;
  cudaError_t e = prepare_kv_evict(a, num_sms, &launches);
  if (e == cudaSuccess) {
    int n = 0;
    e = run_launches(launches, static_cast<cudaStream_t>(stream), &n);
  }
  return e == cudaSuccess ? IL_OK : api_cuda_fail(e, fn);
} catch (const std::bad_alloc&) {  // of the launch lists
  return api_cuda_fail(cudaErrorMemoryAllocation, "il_kv_evict");
}

}  // extern "C"
