// kv_cache.cu -- bookkeeping of the paged K/V cache: block tables and slot maps from the
// sequences' lengths (il_kv_extend), rows into the cache's slots and back (il_kv_append,
// il_kv_read).
#include <algorithm>
#include <type_traits>

#include "il_internal.cuh"

namespace il {

namespace {

// ---------------------------------------------------------------------------
// il_kv_extend
// ---------------------------------------------------------------------------
// With L the length, N = max(0, L + add), pages had = ceil(L / P), has = ceil(N / P):
//   take = max(0, has - had), give = max(0, had - has), grow = max(0, add),
// and everything else follows from the exclusive sums of the three over the sequences: token i
// of sequence r has position L + i; its page is in the table below `had` and otherwise the
// ring entry head + (sum of take before r) + (page - had); the first token of a page taken
// writes the table entry.
//
// Bound by latency: 16 bytes a sequence, 8 a token.  So it is one launch without a second pass: every
// CTA computes all sums itself (512 threads, each a run of ceil(n_seq / 512) sequences; the
// lengths come from L2) and then does its share of the tokens, which finds its sequence by a
// binary search over the runs' sums in shared memory and a walk inside the run.  The state is
// written where no CTA reads it any more: table entries taken, the ring's tail and separate
// outputs at once, lens and cursor in place by the last CTA to finish.  Measured, device time: 32 sequences by one token
// 3.1 us, 1024 sequences of a mixed batch (0.55 MB in all) 5.5 us.
constexpr int kExtendThreads = 512;
constexpr int kExtendWarps = kExtendThreads / 32;

struct Change {
  uint32_t len, now, had, has;  // lengths and pages before and after (now is below 2^32)
  bool wide;                    // does not fit the table or 31 bits
  __device__ uint32_t take() const { return has > had ? has - had : 0; }
  __device__ uint32_t give() const { return had > has ? had - has : 0; }
  __device__ uint32_t grow() const { return now > len ? now - len : 0; }
};

__device__ __forceinline__ Change change_of(const KvExtendArgs& a, int r) {
  Change c;
  c.len = (uint32_t)max(a.lens[r], 0);
  c.now = (uint32_t)max((long long)c.len + a.add[r], 0ll);
  const uint32_t P = (uint32_t)a.page_size;
  c.had = c.len / P + (c.len % P != 0);
  c.has = c.now / P + (c.now % P != 0);
  c.wide = c.now > 0x7fffffffu || c.had > a.table_width || c.has > a.table_width;
  return c;
}

struct Sums {
  long long take, give, grow;
};

__device__ __forceinline__ Sums shift_add(const Sums& s, int by, bool use) {
  Sums o;
  o.take = __shfl_up_sync(~0u, s.take, by);
  o.give = __shfl_up_sync(~0u, s.give, by);
  o.grow = __shfl_up_sync(~0u, s.grow, by);
  return use ? Sums{s.take + o.take, s.give + o.give, s.grow + o.grow} : s;
}

// Last run whose sum before it is at most i (of 512 runs; the next run's is above i).
__device__ __forceinline__ int find_run(const uint32_t* before, uint32_t i) {
  int lo = 0;
#pragma unroll
  for (int step = kExtendThreads / 2; step > 0; step /= 2)
    if (before[lo + step] <= i) lo += step;
  return lo;
}

__global__ void __launch_bounds__(kExtendThreads) kv_extend_kernel(const KvExtendArgs a) {
  __shared__ uint32_t s_take[kExtendThreads], s_give[kExtendThreads], s_grow[kExtendThreads];
  __shared__ Sums s_warp[kExtendWarps];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (a.n_seq + kExtendThreads - 1) / kExtendThreads;
  const int r0 = min(tid * run, a.n_seq), r1 = min(r0 + run, a.n_seq);
  grid_dep_launch();
  grid_dep_wait();

  const long long head = a.cursor[0], tail = a.cursor[1], size = a.ring_size;
  Sums mine = {0, 0, 0};
  bool wide = false;
  for (int r = r0; r < r1; ++r) {
    const Change c = change_of(a, r);
    mine.take += c.take();
    mine.give += c.give();
    mine.grow += c.grow();
    wide |= c.wide;
  }
  Sums incl = mine;
#pragma unroll
  for (int by = 1; by < 32; by *= 2) incl = shift_add(incl, by, lane >= by);
  if (lane == 31) s_warp[warp] = incl;
  wide = __syncthreads_or(wide);
  Sums all = lane < kExtendWarps ? s_warp[lane] : Sums{0, 0, 0};
#pragma unroll
  for (int by = 1; by < kExtendWarps; by *= 2) all = shift_add(all, by, lane >= by);
  auto at = [&](long long v, int src) { return __shfl_sync(~0u, v, src); };
  const Sums total = {at(all.take, kExtendWarps - 1), at(all.give, kExtendWarps - 1), at(all.grow, kExtendWarps - 1)};
  Sums before = {at(all.take, max(warp - 1, 0)), at(all.give, max(warp - 1, 0)), at(all.grow, max(warp - 1, 0))};
  if (warp == 0) before = Sums{0, 0, 0};
  before.take += incl.take - mine.take;
  before.give += incl.give - mine.give;
  before.grow += incl.grow - mine.grow;

  const bool odd_ring = head < 0 || tail < head || tail - head > size;
  const int code = (total.take > tail - head ? 1 : 0) | (wide ? 2 : 0) | (total.grow > a.max_slots ? 4 : 0) |
                   (odd_ring || tail - head + total.give > size ? 8 : 0);
  const bool first_cta = blockIdx.x == 0;
  if (first_cta && tid == 0 && a.info != nullptr) {
    a.info[0] = code;
    a.info[1] = total.grow;
    a.info[2] = total.take;
    a.info[3] = total.give;
  }
  const uint32_t stride = gridDim.x * kExtendThreads;
  const uint32_t i0 = blockIdx.x * kExtendThreads + tid;
  if (code != 0) {  // nothing changes
    for (int64_t i = i0; i < a.max_slots; i += stride) {
      a.slots[i] = -1;
      if (a.positions != nullptr) a.positions[i] = -1;
    }
    if (first_cta) {
      for (int r = r0; r < r1; ++r) {
        if (a.lens_out != a.lens) a.lens_out[r] = a.lens[r];
        if (a.first != nullptr) a.first[r] = 0;
      }
      if (tid == 0) {
        if (a.first != nullptr) a.first[a.n_seq] = 0;
        if (a.cursor_out != a.cursor) {
          a.cursor_out[0] = head;
          a.cursor_out[1] = tail;
        }
      }
    }
    return;
  }

  // every total fits 31 bits here: the new tokens fit max_slots, the pages the ring
  s_take[tid] = (uint32_t)before.take;
  s_give[tid] = (uint32_t)before.give;
  s_grow[tid] = (uint32_t)before.grow;
  __syncthreads();
  const uint32_t ring_size = (uint32_t)size;
  const uint32_t head_at = (uint32_t)(head % size), tail_at = (uint32_t)(tail % size);
  auto ring_at = [&](uint32_t from, uint32_t i) {  // from, i < ring_size < 2^31
    const uint32_t p = from + i;
    return p >= ring_size ? p - ring_size : p;
  };
  const uint32_t P = (uint32_t)a.page_size;
  for (int64_t i = i0; i < a.max_slots; i += stride) {
    int32_t slot = -1, pos = -1;
    if (i < total.grow) {
      const int j = find_run(s_grow, (uint32_t)i);
      int r = j * run;
      uint32_t k = (uint32_t)i - s_grow[j], taken = s_take[j];
      Change c = change_of(a, r);
      while (k >= c.grow()) {
        k -= c.grow();
        taken += c.take();
        c = change_of(a, ++r);
      }
      const uint32_t p = c.len + k, col = p / P, in_page = p - col * P;
      int32_t* entry = a.table + r * a.table_stride + col;
      int32_t page;
      if (col < c.had) {
        page = *entry;
      } else {
        page = a.ring[ring_at(head_at, taken + (col - c.had))];
        if (in_page == 0) *entry = page;
      }
      // a page that no cache has (negative, or with slots past 31 bits) gives a slot that none has
      slot = (int32_t)min((unsigned long long)(uint32_t)page * P + in_page, 0x7fffffffull);
      pos = (int32_t)p;
    }
    a.slots[i] = slot;
    if (a.positions != nullptr) a.positions[i] = pos;
  }
  for (uint32_t i = i0; i < (uint32_t)total.give; i += stride) {
    const int j = find_run(s_give, i);
    int r = j * run;
    uint32_t k = i - s_give[j];
    Change c = change_of(a, r);
    while (k >= c.give()) {
      k -= c.give();
      c = change_of(a, ++r);
    }
    a.ring[ring_at(tail_at, i)] = a.table[r * a.table_stride + c.has + k];
  }
  if (first_cta && a.first != nullptr) {
    uint32_t f = (uint32_t)before.grow;
    for (int r = r0; r < r1; ++r) {
      a.first[r] = (int32_t)f;
      f += change_of(a, r).grow();
    }
    if (tid == 0) a.first[a.n_seq] = (int32_t)total.grow;
  }
  // the new state: by the first CTA where nobody reads what it overwrites, else by the last
  bool writer = first_cta;
  __syncthreads();
  if (gridDim.x > 1 && (a.lens_out == a.lens || a.cursor_out == a.cursor)) {
    if (tid == 0) {
      __threadfence();
      const unsigned n = atomicAdd(a.arrived, 1u);
      s_last = n == gridDim.x - 1;
      if (s_last) *a.arrived = 0;
    }
    __syncthreads();
    writer = s_last != 0;
  }
  if (writer) {
    for (int r = r0; r < r1; ++r) a.lens_out[r] = (int32_t)change_of(a, r).now;
    if (tid == 0) {
      a.cursor_out[0] = head + total.take;
      a.cursor_out[1] = tail + total.give;
    }
  }
}

// ---------------------------------------------------------------------------
// il_kv_append / il_kv_read
// ---------------------------------------------------------------------------
// One thread moves units of 8 elements of K and the same 8 of V (32 bytes of fp32 and 16 or 8 of the cache each).
// Bound by HBM where there are many tokens; at Q8 the arithmetic comes near it, so that:
// - q = round(w / d) is taken from w times an approximate 1 / d, which is off by at most 127 * (2^-23 + 2^-23) =
//   3.1e-5, and by the definition's division only where the product lies within 5e-5 of half way between integers;
// - a float's integer is read from its low byte after adding 1.5 * 2^23, and made from a byte by the reverse;
// - the four lanes of a 32-element block share its largest |w| with two shuffles; d = amax / 127 is the IEEE
//   division, so that d and q are the definition's bit for bit.
// Measured (8 heads of 128, device time): append of 16384 tokens bf16 30.4 us, 6.6 TB/s, Q8 31.3 us, 5.5 TB/s; of 4097 Q8
// 10.0 us; read of 16384 bf16 32.9 us, 6.1 TB/s, Q8 28.8 us, 6.0 TB/s, of 4097 Q8 9.2 us; append of one token 1.3 us.
constexpr int kRowThreads = 256;
// Units of a thread at a time: two, all loads first, but for Q8's quantiser, where more warps hide its chains
// better (when it was chosen, 4097 tokens of 8 x 128: 13.0 us with two, 11.0 us with one; bf16 append 9.6 and 9.2,
// Q8 read of 16384 28.8 and 31.1).
constexpr int row_units(bool write, bool q8) { return write && q8 ? 1 : 2; }

struct RowArgs {
  KvView kv;
  float *k, *v;
  int64_t k_stride, v_stride;
  const int32_t* slots;
  int64_t n, run;                        // tokens, tokens whose units 31 bits count
  FastDiv per_token, per_head, by_page;  // units of a token and of a head
  int whole;                             // a unit's 32 bytes of fp32 are aligned: one access
  unsigned* status;
};

struct Eight {
  float4 lo, hi;
};

// 32 bytes of fp32: one access where they are aligned (two 16-byte stores each cover half of every sector).
__device__ __forceinline__ Eight load8(const float* p, bool whole) {
  Eight e;
  if (whole) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(e.lo.x), "=f"(e.lo.y), "=f"(e.lo.z), "=f"(e.lo.w), "=f"(e.hi.x), "=f"(e.hi.y), "=f"(e.hi.z), "=f"(e.hi.w)
                 : "l"(p)
                 : "memory");
  } else {
    e.lo = reinterpret_cast<const float4*>(p)[0];
    e.hi = reinterpret_cast<const float4*>(p)[1];
  }
  return e;
}
__device__ __forceinline__ void store8(float* p, const Eight& e, bool whole) {
  if (whole) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(e.lo.x), "f"(e.lo.y), "f"(e.lo.z),
                 "f"(e.lo.w), "f"(e.hi.x), "f"(e.hi.y), "f"(e.hi.z), "f"(e.hi.w)
                 : "memory");
  } else {
    reinterpret_cast<float4*>(p)[0] = e.lo;
    reinterpret_cast<float4*>(p)[1] = e.hi;
  }
}

// max that gives NaN where an operand is NaN
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ void write8(const Eight& e, __nv_bfloat16* to) {
  const float4 &x = e.lo, &y = e.hi;
  *reinterpret_cast<uint4*>(to) =
      make_uint4(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w), pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
}

constexpr float kToInt = 12582912.f;  // 1.5 * 2^23

__device__ __forceinline__ void write8(const Eight& e, int8_t* to, float* scale, unsigned quad, bool first_of_block) {
  const float4 &x = e.lo, &y = e.hi;
  const float w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(w[i]));
  m = max_nan(m, __shfl_xor_sync(quad, m, 1));
  m = max_nan(m, __shfl_xor_sync(quad, m, 2));
  const float d = __fdiv_rn(m, 127.0f);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(d));
  uint32_t f[8];
  uint32_t unsure = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = w[i] * inv, r = t + kToInt;
    f[i] = __float_as_uint(r);
    if (!(fabsf(t - (r - kToInt)) < 0.49995f)) unsure |= 1u << i;  // NaN too
  }
  const bool normal = d > 0.f && d < __int_as_float(0x7f800000);  // otherwise q = 0 (and d = 0, NaN or infinity)
#pragma unroll 1
  while (unsure != 0) {
    const int i = __ffs(unsure) - 1;
    unsure &= unsure - 1;
    float v = w[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) v = j == i ? w[j] : v;
    const uint32_t q = normal ? (uint32_t)(int)fminf(fmaxf(rintf(__fdiv_rn(v, d)), -127.f), 127.f) : 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = j == i ? q : f[j];
  }
  auto word = [&](int i) {
    return __byte_perm(__byte_perm(f[i], f[i + 1], 0x0040), __byte_perm(f[i + 2], f[i + 3], 0x0040), 0x5410);
  };
  *reinterpret_cast<uint2*>(to) = make_uint2(word(0), word(4));
  if (first_of_block) *scale = d;
}

__device__ __forceinline__ Eight read8(const uint4& u, float) {
  return {make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y)),
          make_float4(bf16_lo(u.z), bf16_hi(u.z), bf16_lo(u.w), bf16_hi(u.w))};
}

__device__ __forceinline__ Eight read8(const uint2& u, float d) {
  auto four = [&](uint32_t word) {
    const uint32_t b = word ^ 0x80808080u;  // q + 128
    auto one = [&](uint32_t sel) { return d * (__uint_as_float(__byte_perm(b, 0x4b000000u, sel)) - 8388736.f); };
    return make_float4(one(0x7440), one(0x7441), one(0x7442), one(0x7443));
  };
  return {four(u.x), four(u.y)};
}

template <bool WRITE, bool Q8>
__global__ void __launch_bounds__(kRowThreads, WRITE && Q8 ? 5 : 4) kv_rows_kernel(const RowArgs a) {
  using T = typename std::conditional<Q8, int8_t, __nv_bfloat16>::type;
  constexpr int kRowUnits = row_units(WRITE, Q8);
  using Cached = typename std::conditional<Q8, uint2, uint4>::type;  // 8 elements
  grid_dep_launch();
  grid_dep_wait();
  const KvView& kv = a.kv;
  const unsigned quad = 0xfu << (threadIdx.x & 28);
  const uint32_t step = gridDim.x * kRowThreads;
  for (int64_t t0 = 0; t0 < a.n; t0 += a.run) {
    const uint32_t units = (uint32_t)min(a.run, a.n - t0) * a.per_token.d;
    for (uint32_t first = blockIdx.x * kRowThreads + threadIdx.x; first < units; first += kRowUnits * step) {
      float *k[kRowUnits], *v[kRowUnits];
      int64_t off[kRowUnits], soff[kRowUnits];
      bool live[kRowUnits], block_start[kRowUnits];
      Eight x[WRITE ? kRowUnits : 1][2];
      Cached c[WRITE ? 1 : kRowUnits][2];
      float d[kRowUnits][2];
#pragma unroll
      for (int j = 0; j < kRowUnits; ++j) {
        const bool in = first + j * step < units;
        const uint32_t u = in ? first + j * step : first;
        const uint32_t t = a.per_token.of(u), in_token = u - t * a.per_token.d;
        const uint32_t head = a.per_head.of(in_token), i = 8 * (in_token - head * a.per_head.d);
        const int32_t slot = in ? a.slots[t0 + t] : -1;
        live[j] = slot >= 0 && slot < kv.n_slots;
        if (slot >= kv.n_slots) atomicOr(a.status, kStatusBadSlot);
        k[j] = in ? a.k + (t0 + t) * a.k_stride + (int64_t)head * kv.head_dim + i : nullptr;
        v[j] = a.v + (t0 + t) * a.v_stride + (int64_t)head * kv.head_dim + i;
        const uint32_t page = a.by_page.of((uint32_t)max(slot, 0)), at = (uint32_t)slot - page * a.by_page.d;
        off[j] = page * kv.page + at * kv.token + (int64_t)head * kv.head + i;
        soff[j] = Q8 ? page * kv.spage + at * kv.stoken + (int64_t)head * kv.shead + i / 32 : 0;
        block_start[j] = i % 32 == 0;
        if (live[j]) {
          if constexpr (WRITE) {
            x[j][0] = load8(k[j], a.whole);
            x[j][1] = load8(v[j], a.whole);
          } else {
            c[j][0] = *reinterpret_cast<const Cached*>(reinterpret_cast<const T*>(kv.k) + off[j]);
            c[j][1] = *reinterpret_cast<const Cached*>(reinterpret_cast<const T*>(kv.v) + off[j]);
            if constexpr (Q8) d[j][0] = kv.k_scale[soff[j]], d[j][1] = kv.v_scale[soff[j]];
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kRowUnits; ++j) {
        if (!live[j]) {
          if (!WRITE && k[j] != nullptr) {
            const Eight z = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
            store8(k[j], z, a.whole);
            store8(v[j], z, a.whole);
          }
          continue;
        }
        if constexpr (WRITE) {
          T* const ck = reinterpret_cast<T*>(kv.k) + off[j];
          T* const cv = reinterpret_cast<T*>(kv.v) + off[j];
          if constexpr (Q8) {
            write8(x[j][0], ck, kv.k_scale + soff[j], quad, block_start[j]);
            write8(x[j][1], cv, kv.v_scale + soff[j], quad, block_start[j]);
          } else {
            write8(x[j][0], ck);
            write8(x[j][1], cv);
          }
        } else {
          store8(k[j], read8(c[j][0], d[j][0]), a.whole);
          store8(v[j], read8(c[j][1], d[j][1]), a.whole);
        }
      }
    }
  }
}

}  // namespace

cudaError_t prepare_kv_extend(const KvExtendArgs& a, int num_sms, Launch* out) {
  // a CTA for each 512 slots from 2048 on (below that, one CTA and no arrival counter)
  const int64_t ctas = a.max_slots <= 2048 ? 1 : std::min<int64_t>(num_sms, (a.max_slots + kExtendThreads - 1) / kExtendThreads);
  out->fn = reinterpret_cast<const void*>(kv_extend_kernel);
  out->grid = dim3((unsigned)ctas);
  out->block = dim3(kExtendThreads);
  if (!out->set_args(a)) return cudaErrorMemoryAllocation;
  if (kUsePdl) out->allow_early_start();
  return cudaSuccess;
}

cudaError_t prepare_kv_rows(bool write, const KvView& kv, float* k, int64_t k_stride, float* v, int64_t v_stride,
                            const int32_t* slots, int64_t n, unsigned* status, int num_sms, Launch* out) {
  const bool q8 = kv.format == IL_Q8;
  const uint32_t per_head = (uint32_t)kv.head_dim / 8, per_token = per_head * kv.n_heads;
  // runs of tokens whose units (and a grid's step beyond them) 31 bits count
  const int64_t run = std::max<int64_t>(1, (int64_t)((0x7fffffffu - (1u << 24)) / per_token));
  const RowArgs a = {kv, k, v, k_stride, v_stride, slots, n, run, FastDiv(per_token), FastDiv(per_head),
                     FastDiv((uint32_t)kv.page_size),
                     (reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % 32 == 0 &&
                         (n == 1 || (k_stride % 8 == 0 && v_stride % 8 == 0)),
                     status};
  out->fn = write ? (q8 ? reinterpret_cast<const void*>(kv_rows_kernel<true, true>)
                        : reinterpret_cast<const void*>(kv_rows_kernel<true, false>))
                  : (q8 ? reinterpret_cast<const void*>(kv_rows_kernel<false, true>)
                        : reinterpret_cast<const void*>(kv_rows_kernel<false, false>));
  const int64_t units = n * per_token;  // one a thread while that fills the GPU's threads less than once
  out->grid = dim3((unsigned)std::min<int64_t>((units + kRowThreads - 1) / kRowThreads, (int64_t)num_sms * 8));
  out->block = dim3(kRowThreads);
  if (!out->set_args(a)) return cudaErrorMemoryAllocation;
  if (kUsePdl) out->allow_early_start();
  return cudaSuccess;
}

}  // namespace il
