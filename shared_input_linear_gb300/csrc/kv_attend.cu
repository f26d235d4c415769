// kv_attend.cu -- attention of one new token per sequence over the paged cache (il_kv_attend).
#include <algorithm>

#include "il_internal.cuh"

namespace il {

namespace {

// One CTA per (query head, sequence): its warps take the tokens in turn, each lane holds the
// elements d = lane, lane + 32, ... of q and of the running sum, with the running maximum and
// sum of the softmax; the warps' parts are joined at the end.
constexpr int kAttendWarps = 4;

template <bool Q8>
__global__ void __launch_bounds__(32 * kAttendWarps) kv_attend_kernel(const KvAttendArgs a) {
  __shared__ float s_m[kAttendWarps], s_l[kAttendWarps], s_o[kAttendWarps][kMaxKvDim];
  const KvView& kv = a.kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.y, s = blockIdx.x, D = kv.head_dim;
  const int64_t hk = h / (a.n_q_heads / kv.n_heads);
  grid_dep_launch();
  grid_dep_wait();
  const int64_t len = min((int64_t)max(a.lens[s], 0), a.table_width * kv.page_size);
  const int64_t begin = a.window > 0 ? max(len - a.window, (int64_t)0) : 0;
  float q[8], o[8], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int d = lane + 32 * i;
    q[i] = d < D ? a.q[s * a.q_stride + (int64_t)h * D + d] * (a.scale * 1.4426950408889634f) : 0.f;
    o[i] = 0.f;
  }
  for (int64_t t = begin + warp; t < len; t += kAttendWarps) {
    const int64_t col = t / kv.page_size;
    const int64_t page = a.table[s * a.table_stride + col];
    if (page < 0 || page >= kv.n_pages) {
      if (lane == 0) atomicOr(a.status, kStatusBadSlot);
      continue;
    }
    const int64_t at = t - col * kv.page_size;
    const int64_t off = page * kv.page + at * kv.token + hk * kv.head;
    const int64_t soff = page * kv.spage + at * kv.stoken + hk * kv.shead;
    auto value = [&](const uint8_t* pool, const float* scale, int i) {
      const int d = lane + 32 * i;
      if (d >= D) return 0.f;
      if constexpr (Q8) return scale[soff + i] * (float)reinterpret_cast<const int8_t*>(pool)[off + d];
      return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(pool)[off + d]);
    };
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) x = fmaf(q[i], value(kv.k, kv.k_scale, i), x);
#pragma unroll
    for (int by = 16; by > 0; by /= 2) x += __shfl_xor_sync(~0u, x, by);
    const float m1 = fmaxf(m, x), f = exp2f(m - m1), p = exp2f(x - m1);
    l = fmaf(l, f, p);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = fmaf(o[i], f, p * value(kv.v, kv.v_scale, i));
    m = m1;
  }
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
  for (int i = 0; i < 8; ++i) s_o[warp][lane + 32 * i] = o[i];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < kAttendWarps; ++w) M = fmaxf(M, s_m[w]);
  const float base = M == -INFINITY ? 0.f : M;
  for (int w = 0; w < kAttendWarps; ++w) L += s_l[w] * exp2f(s_m[w] - base);
  for (int d = threadIdx.x; d < D; d += 32 * kAttendWarps) {
    float x = 0.f;
    for (int w = 0; w < kAttendWarps; ++w) x += s_o[w][d] * exp2f(s_m[w] - base);
    a.out[s * a.out_stride + (int64_t)h * D + d] = L == 0.f ? 0.f : x / L;
  }
  if (threadIdx.x == 0 && a.lse != nullptr)
    a.lse[(int64_t)s * a.n_q_heads + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

}  // namespace

size_t kv_attend_workspace_bytes(const KvAttendArgs&, int) { return 0; }

cudaError_t prepare_kv_attend(const KvAttendArgs& a, int, void*, size_t, Launch* out) {
  out->fn = a.kv.format == IL_Q8 ? reinterpret_cast<const void*>(kv_attend_kernel<true>)
                                 : reinterpret_cast<const void*>(kv_attend_kernel<false>);
  out->grid = dim3((unsigned)a.n_seq, (unsigned)a.n_q_heads);
  out->block = dim3(32 * kAttendWarps);
  if (!out->set_args(a)) return cudaErrorMemoryAllocation;
  if (kUsePdl) out->allow_early_start();
  return cudaSuccess;
}

}  // namespace il
