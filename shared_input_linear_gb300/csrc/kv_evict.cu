// kv_evict.cu -- il_kv_evict: which tokens of a sequence stay, and the rows that move for it.
//
// Of n > keep tokens the first, the recent and the heaviest stay.  Those of them at `keep` and behind (movers) go to the places
// of those before it that do not (holes), the i-th mover to the i-th hole: there are as many of either, no row is both read
// and written, and what need not move stays.  A compaction in order would move nearly every row.
#include <algorithm>

#include "il_internal.cuh"
#include "il_ptx.cuh"

namespace il {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

// Order of a token: larger stays.  Weights as unsigned numbers of the same order (-0 as 0), NaN below all, the
// tokens that stay whatever their weight above all.
__device__ __forceinline__ uint32_t key_of(float weight, bool always) {
  const uint32_t b = __float_as_uint(weight + 0.f);
  if (always) return 0xffffffffu;
  if (weight != weight) return 0u;
  return b >> 31 ? ~b : b | 0x80000000u;
}

// The choice, a CTA a sequence: the keep-th largest key by its bytes, from the highest (four passes, each a histogram of the keys
// that match so far); among equal keys those of the lowest index, up to the last one taken; then the list of movers, which
// is put at the end of the sequence's row of `kept` -- the j-th hole lies before the j-th of the list's M places there, so that
// filling the holes in order never overwrites an entry that is still needed -- and the entries from it.
__global__ void __launch_bounds__(kThreads) kv_choose_kernel(const KvEvictArgs a) {
  __shared__ uint32_t s_count[256], s_warp[kWarps], s_pick[2], s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_launch();
  grid_dep_wait();
#pragma unroll 1
  for (int s = blockIdx.x; s < a.n_seq; s += gridDim.x) {
    const int n = min(max(a.lens[s], 0), a.cap), left = min(n, a.keep);
    const float* const weights = a.weights + s * a.weights_stride;
    float* const weights_out = a.weights_out + s * a.weights_stride;
    const int32_t* const positions = a.positions == nullptr ? nullptr : a.positions + s * a.positions_stride;
    int32_t* const positions_out = a.positions == nullptr ? nullptr : a.positions_out + s * a.positions_stride;
    int32_t* const kept = a.kept + s * a.kept_stride;
    if (tid == 0) a.drop[s] = left - n;
    for (int i = left + tid; i < a.keep; i += kThreads) kept[i] = -1;
    if (n == left) {
      for (int i = tid; i < n; i += kThreads) {
        kept[i] = i;
        if (weights_out != weights) weights_out[i] = weights[i];
        if (positions_out != positions) positions_out[i] = positions[i];
      }
      continue;
    }
    const long long newest = positions == nullptr ? n - 1 : positions[n - 1];
    auto key_at = [&](int i) {
      const long long p = positions == nullptr ? i : positions[i];
      return key_of(weights[i], p < a.first || p > newest - a.recent);
    };

    // ---- the smallest key that stays, and how many of that key do
    uint32_t bar = 0, wanted = (uint32_t)a.keep;
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) s_count[tid] = 0;
      __syncthreads();
      for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + tid;
        const uint32_t key = i < n ? key_at(i) : 0u;
        const bool in = i < n && (shift == 24 || key >> (shift + 8) == bar >> (shift + 8));
        const uint32_t digit = key >> shift & 255u, peers = __match_any_sync(~0u, in ? digit : 256u + lane);
        if (in && lane == __ffs(peers) - 1) atomicAdd(&s_count[digit], (uint32_t)__popc(peers));
      }
      __syncthreads();
      if (warp == 0) {  // from the largest digit down: lane l has digits 255 - 8 l and the next seven below
        uint32_t mine = 0;
        for (int k = 0; k < 8; ++k) mine += s_count[255 - 8 * lane - k];
        uint32_t incl = mine;
        for (int by = 1; by < 32; by *= 2) {
          const uint32_t o = __shfl_up_sync(~0u, incl, by);
          if (lane >= by) incl += o;
        }
        uint32_t before = incl - mine;
        if (before < wanted && wanted <= incl) {
          int digit = 255 - 8 * lane;
          while (before + s_count[digit] < wanted) before += s_count[digit--];
          s_pick[0] = digit;
          s_pick[1] = wanted - before;
        }
      }
      __syncthreads();
      bar |= s_pick[0] << shift;
      wanted = s_pick[1];
    }

    // ---- the index of the last token of that key that stays.  A warp has a run of the tokens, whole groups of 32.
    auto run_of = [&](int from, int to, int& r0, int& r1) {
      const int groups = (to - from + 31) / 32, per = (groups + kWarps - 1) / kWarps;
      r0 = min(from + warp * per * 32, to);
      r1 = min(from + (warp + 1) * per * 32, to);
    };
    auto sum_before = [&](uint32_t mine, uint32_t& all) {  // of the warps before this one
      if (lane == 0) s_warp[warp] = mine;
      __syncthreads();
      const uint32_t v = s_warp[lane];
      uint32_t incl = v;
      for (int by = 1; by < 32; by *= 2) {
        const uint32_t o = __shfl_up_sync(~0u, incl, by);
        if (lane >= by) incl += o;
      }
      all = __shfl_sync(~0u, incl, 31);
      const uint32_t before = __shfl_sync(~0u, incl - v, warp);
      __syncthreads();
      return before;
    };
    int r0, r1;
    run_of(0, n, r0, r1);
    uint32_t same = 0, all = 0;
    for (int i = r0; i < r1; i += 32) same += __popc(__ballot_sync(~0u, i + lane < r1 && key_at(i + lane) == bar));
    uint32_t before = sum_before(same, all);
    if (before < wanted && wanted <= before + same) {
      for (int i = r0; i < r1; i += 32) {
        uint32_t hits = __ballot_sync(~0u, i + lane < r1 && key_at(i + lane) == bar);
        if (before + __popc(hits) >= wanted) {
          for (uint32_t skip = wanted - before - 1; skip > 0; --skip) hits &= hits - 1;
          if (lane == 0) s_last = i + __ffs(hits) - 1;
          break;
        }
        before += __popc(hits);
      }
    }
    __syncthreads();
    const int last = (int)s_last;
    auto stays = [&](int i) {
      const uint32_t key = key_at(i);
      return key > bar || (key == bar && i <= last);
    };

    // ---- movers, in order, to the end of the row
    run_of(a.keep, n, r0, r1);
    uint32_t mine = 0, movers = 0;
    for (int i = r0; i < r1; i += 32) mine += __popc(__ballot_sync(~0u, i + lane < r1 && stays(i + lane)));
    uint32_t rank = sum_before(mine, movers);
    for (int i = r0; i < r1; i += 32) {
      const bool hit = i + lane < r1 && stays(i + lane);
      const uint32_t hits = __ballot_sync(~0u, hit);
      if (hit) kept[a.keep - movers + rank + __popc(hits & ((1u << lane) - 1))] = i + lane;
      rank += __popc(hits);
    }
    __syncthreads();

    // ---- the entries, in order: every thread reads before any writes
    uint32_t holes = 0;
    for (int i0 = 0; i0 < a.keep; i0 += kThreads) {
      const int i = i0 + tid;
      const bool hole = i < a.keep && !stays(i);
      const uint32_t hits = __ballot_sync(~0u, hole);
      uint32_t here;
      const uint32_t at = holes + sum_before(__popc(hits), here) + __popc(hits & ((1u << lane) - 1));
      const int from = hole ? kept[a.keep - movers + at] : i;
      holes += here;
      __syncthreads();
      if (i < a.keep) {
        kept[i] = from;
        if (hole || weights_out != weights) weights_out[i] = weights[from];
        if (positions != nullptr && (hole || positions_out != positions)) positions_out[i] = positions[from];
      }
    }
    __syncthreads();
  }
}

constexpr int kMoveThreads = 256;

// The rows, a warp an entry: K and V of all heads, 16 bytes a lane, four loads of each in flight; then the scales, 4 bytes a lane.  A lane looks
// up one of the warp's next 32 entries.
__global__ void __launch_bounds__(kMoveThreads) kv_move_kernel(const KvEvictArgs a, const FastDiv by_page,
                                                               const FastDiv by_chunks, const FastDiv by_blocks) {
  const KvView& kv = a.kv;
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (kMoveThreads / 32), total = (long long)a.n_seq * a.keep;
  const int es = kv.format == IL_BF16 ? 2 : 1;
  const uint32_t chunks = by_chunks.d * kv.n_heads, scales = kv.format == IL_BF16 ? 0 : by_blocks.d * kv.n_heads;
  grid_dep_launch();
  grid_dep_wait();
  for (long long e0 = blockIdx.x * (kMoveThreads / 32) + threadIdx.x / 32; e0 < total; e0 += 32 * warps) {
    const long long e = e0 + lane * warps;
    long long to = 0, from = 0, sto = 0, sfrom = 0;  // byte offsets of the token's K (and V), and in words of its scales
    bool moves = false;
    if (e < total) {
      const int s = (int)(e / a.keep), i = (int)(e - (long long)s * a.keep);
      const int j = a.kept[s * a.kept_stride + i];
      if (j >= 0 && j != i) {
        const uint32_t col[2] = {by_page.of(i), by_page.of(j)};
        const uint32_t page[2] = {(uint32_t)a.table[s * a.table_stride + col[0]], (uint32_t)a.table[s * a.table_stride + col[1]]};
        moves = page[0] < (uint32_t)kv.n_pages && page[1] < (uint32_t)kv.n_pages;
        if (!moves) atomicOr(a.status, kStatusBadSlot);
        const uint32_t in_page[2] = {i - col[0] * by_page.d, j - col[1] * by_page.d};
        to = (page[0] * kv.page + in_page[0] * kv.token) * es;
        from = (page[1] * kv.page + in_page[1] * kv.token) * es;
        sto = page[0] * kv.spage + in_page[0] * kv.stoken;
        sfrom = page[1] * kv.spage + in_page[1] * kv.stoken;
      }
    }
    uint32_t todo = __ballot_sync(~0u, moves);
    while (todo != 0) {
      const int src = __ffs(todo) - 1;
      todo &= todo - 1;
      const long long t = __shfl_sync(~0u, to, src), f = __shfl_sync(~0u, from, src);
      const long long st = __shfl_sync(~0u, sto, src), sf = __shfl_sync(~0u, sfrom, src);
      for (uint32_t c0 = lane; c0 < chunks; c0 += 128) {
        uint4 k[4], v[4];
        long long off[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t c = c0 + 32 * x, head = by_chunks.of(c);
          off[x] = (long long)head * kv.head * es + (c - head * by_chunks.d) * 16;
          if (c < chunks) {
            k[x] = *reinterpret_cast<const uint4*>(kv.k + f + off[x]);
            v[x] = *reinterpret_cast<const uint4*>(kv.v + f + off[x]);
          }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (c0 + 32 * x < chunks) {
            *reinterpret_cast<uint4*>(kv.k + t + off[x]) = k[x];
            *reinterpret_cast<uint4*>(kv.v + t + off[x]) = v[x];
          }
      }
      for (uint32_t c = lane; c < scales; c += 32) {
        const uint32_t head = by_blocks.of(c);
        const long long off = (long long)head * kv.shead + (c - head * by_blocks.d);
        kv.k_scale[st + off] = kv.k_scale[sf + off];
        kv.v_scale[st + off] = kv.v_scale[sf + off];
      }
    }
  }
}

}  // namespace

cudaError_t prepare_kv_evict(const KvEvictArgs& a, int num_sms, std::vector<Launch>* out) {
  out->resize(2);
  Launch &choose = (*out)[0], &move = (*out)[1];
  choose.fn = reinterpret_cast<const void*>(kv_choose_kernel);
  choose.grid = dim3((unsigned)std::min(a.n_seq, 2 * num_sms));
  choose.block = dim3(kThreads);
  if (!choose.set_args(a)) return cudaErrorMemoryAllocation;
  move.fn = reinterpret_cast<const void*>(kv_move_kernel);
  const int64_t entries = (int64_t)a.n_seq * a.keep, per_cta = kMoveThreads / 32;
  move.grid = dim3((unsigned)std::min<int64_t>((entries + per_cta - 1) / per_cta, (int64_t)num_sms * 8));
  move.block = dim3(kMoveThreads);
  const uint32_t row = (uint32_t)(a.kv.format == IL_BF16 ? 2 * a.kv.head_dim : a.kv.format == IL_Q8 ? a.kv.head_dim : a.kv.head_dim / 2);
  if (!move.set_args(a, FastDiv((uint32_t)a.kv.page_size), FastDiv(row / 16), FastDiv((uint32_t)std::max(1, a.kv.head_dim / 32))))
    return cudaErrorMemoryAllocation;
  if (kUsePdl) {
    choose.allow_early_start();
    move.allow_early_start();
  }
  return cudaSuccess;
}

}  // namespace il
