// il_kv.cu -- entry points of the paged K/V cache (include/il.h: il_kv_extend, il_kv_append,
// il_kv_read, il_kv_attend): every argument that the host can see is checked and the launch
// prepared before it is enqueued, as in the matmul entry points.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <cstring>
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
  if (kv->format != IL_BF16 && kv->format != IL_Q8) return bad(IL_ERR_FORMAT, fn, "the cache must be IL_BF16 or IL_Q8");
  const bool q8 = kv->format == IL_Q8;
  if (kv->page_size < 1 || kv->page_size > (1 << 20) || kv->n_pages < 1 || kv->n_pages > INT32_MAX / kv->page_size)
    return bad(IL_ERR_SHAPE, fn, "page_size or n_pages out of range");
  if (kv->n_heads < 1 || kv->n_heads > 1024) return bad(IL_ERR_SHAPE, fn, "n_heads out of range");
  if (kv->head_dim < 8 || kv->head_dim > kMaxKvDim || kv->head_dim % (q8 ? 32 : 8) != 0)
    return bad(IL_ERR_SHAPE, fn, "head_dim must be at most 256 and a multiple of 8 (bf16) or of 32 (Q8)");
  if (kv->k == nullptr || kv->v == nullptr) return bad(IL_ERR_ARG, fn, "the cache's k or v is NULL");
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16)) return bad(IL_ERR_ARG, fn, "the cache's k or v is not 16-byte aligned");
  const int64_t unit = q8 ? 16 : 8, dim = kv->head_dim, blocks = dim / 32;
  if (!stride_ok(kv->page_stride, kv->n_pages, dim, unit) || !stride_ok(kv->token_stride, kv->page_size, dim, unit) ||
      !stride_ok(kv->head_stride, kv->n_heads, dim, unit))
    return bad(IL_ERR_SHAPE, fn, "a stride of the cache is smaller than a row or not a multiple of 16 bytes");
  if (q8) {
    if (kv->k_scale == nullptr || kv->v_scale == nullptr) return bad(IL_ERR_ARG, fn, "a Q8 cache needs k_scale and v_scale");
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

// Byte extent of a pool (elements of `size` bytes, rows of `row` elements).
int64_t extent_bytes(const KvView& w, bool scales) {
  const int64_t last = (w.n_pages - 1) * (scales ? w.spage : w.page) + (w.page_size - 1) * (scales ? w.stoken : w.token) +
                       (w.n_heads - 1) * (scales ? w.shead : w.head);
  return scales ? 4 * (last + w.head_dim / 32) : (w.format == IL_BF16 ? 2 : 1) * (last + w.head_dim);
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

}  // namespace

extern "C" {

int il_kv_extend(int64_t n_seq, int64_t page_size, const int32_t* lens, const int32_t* add, int32_t* table,
                 int64_t table_stride, int64_t table_width, int32_t* ring, int64_t ring_size, const int64_t* cursor,
                 int32_t* lens_out, int64_t* cursor_out, int32_t* slots, int64_t max_slots, int32_t* positions,
                 int32_t* first, int64_t* info, void* stream) {
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
}

int il_kv_append(const il_kv* kv, const float* k, int64_t k_stride, const float* v, int64_t v_stride,
                 const int32_t* slots, int64_t n, void* stream) {
  return rows_call("il_kv_append", true, kv, const_cast<float*>(k), k_stride, const_cast<float*>(v), v_stride, slots, n,
                   stream);
}

int il_kv_read(const il_kv* kv, const int32_t* slots, int64_t n, float* k, int64_t k_stride, float* v, int64_t v_stride,
               void* stream) {
  return rows_call("il_kv_read", false, kv, k, k_stride, v, v_stride, slots, n, stream);
}

int il_kv_attend(const il_kv* kv, const float* q, int64_t q_stride, const int32_t* table, int64_t table_stride,
                 int64_t table_width, const int32_t* lens, int64_t n_seq, int64_t n_q_heads, float scale, int64_t window,
                 float* out, int64_t out_stride, float* lse, void* stream) {
  const char* fn = "il_kv_attend";
  NvtxRange range(fn);
  api_clear_error();
  KvAttendArgs a;
  memset(&a, 0, sizeof a);
  int rc = check_cache(fn, kv, &a.kv);
  if (rc != IL_OK) return rc;
  if (n_seq < 0 || n_seq > kMaxKvSeqs) return bad(IL_ERR_ARG, fn, "n_seq out of range");
  if (n_q_heads < 1 || n_q_heads > 32768 || n_q_heads % a.kv.n_heads != 0)
    return bad(IL_ERR_SHAPE, fn, "n_q_heads must be a multiple of the cache's n_heads, at most 32768");
  if (window < 0) return bad(IL_ERR_ARG, fn, "window is negative");
  if (!(scale - scale == 0.0f)) return bad(IL_ERR_ARG, fn, "scale is not finite");
  if (n_seq == 0) return IL_OK;
  if (q == nullptr || table == nullptr || lens == nullptr || out == nullptr)
    return bad(IL_ERR_ARG, fn, "q, table, lens and out must not be NULL");
  if (!aligned(q, 16) || !aligned(out, 16)) return bad(IL_ERR_ARG, fn, "q or out is not 16-byte aligned");
  if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(lse, 4))
    return bad(IL_ERR_ARG, fn, "table, lens or lse is not 4-byte aligned");
  const int64_t row = n_q_heads * a.kv.head_dim;
  if (n_seq > 1 && (q_stride < row || out_stride < row || q_stride % 4 != 0 || out_stride % 4 != 0 ||
                    q_stride > INT64_MAX / 8 / n_seq || out_stride > INT64_MAX / 8 / n_seq))
    return bad(IL_ERR_SHAPE, fn, "q_stride or out_stride is smaller than a row or not a multiple of 4");
  if (table_width < 1 || table_width > INT32_MAX || (n_seq > 1 && (table_stride < table_width || table_stride > INT32_MAX)))
    return bad(IL_ERR_SHAPE, fn, "table_width or table_stride out of range");
  const int64_t qs = n_seq > 1 ? q_stride : 0, os = n_seq > 1 ? out_stride : 0, ts = n_seq > 1 ? table_stride : 0;
  const Range outs[] = {{out, 4 * ((n_seq - 1) * os + row), true}, {lse, 4 * n_seq * n_q_heads, true}};
  const Range ins[] = {{q, 4 * ((n_seq - 1) * qs + row), false},
                       {table, 4 * ((n_seq - 1) * ts + table_width), false},
                       {lens, 4 * n_seq, false},
                       {a.kv.k, extent_bytes(a.kv, false), false},
                       {a.kv.v, extent_bytes(a.kv, false), false},
                       {a.kv.k_scale, extent_bytes(a.kv, true), false},
                       {a.kv.v_scale, extent_bytes(a.kv, true), false}};
  for (const Range& o : outs)
    for (const Range& i : ins)
      if (clash(o, i) && !(&o == outs && &i == ins && side_by_side(out, os, q, qs, n_seq, row))) return bad(IL_ERR_ARG, fn, "out and lse must not overlap q, table, lens or the cache");
  if (clash(outs[0], outs[1])) return bad(IL_ERR_ARG, fn, "out and lse must not overlap");
  int num_sms = 0;
  const int dev = api_device(&num_sms, &a.status);
  if (dev < 0) return dev;
  a.q = q;
  a.q_stride = qs;
  a.table = table;
  a.table_stride = ts;
  a.table_width = table_width;
  a.lens = lens;
  a.n_seq = (int)n_seq;
  a.n_q_heads = (int)n_q_heads;
  a.scale = scale;
  a.window = window;
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

}  // extern "C"
