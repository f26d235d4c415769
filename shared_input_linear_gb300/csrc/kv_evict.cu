// kv_evict.cu -- il_kv_evict: which tokens of a sequence stay, and the rows that move for it.
//
// Of n > keep tokens the first, the recent and the heaviest stay.  Those of them at `keep` and behind (movers) go to the places
// of those before it that do not (holes), the i-th mover to the i-th hole: there are as many of either, no row is both read
// and written, and what need not move stays.  A compaction in order would move nearly every row.
//
// Measured (GB300, 8 heads of 128, device time): 64 sequences of 1025 bf16 tokens cut to 1024 8.4 us; one of 32768 cut to 4096
// 18.2 us, of which about 12 choose (8 CTAs: barriers of the cluster, exchanges, L2 latencies) and 6 move 3584 rows (29 MB
// read and written); 32 of 500 to 8192 Q8 tokens cut to 2048 about 45 us.  Rows wider than 8 CTAs hold take one CTA a sequence: one of
// 393,216 4-bit tokens of one head of 64 cut to 4096 53 us, of 393,217 819 us, of 1,000,000 2050 (with positions 2810).
#include <algorithm>
#include <atomic>
#include <cstddef>

#include <cooperative_groups.h>

#include "il_internal.cuh"
#include "il_ptx.cuh"

namespace il {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMostKeys = 49152;  // that a CTA holds in shared memory (192 KB)
constexpr int kMostCtas = 8;      // of a cluster
constexpr int kFewRows = 64;      // rows of a sequence that its own CTAs move

// Order of a token: larger stays.  Weights as unsigned numbers of the same order (-0 as 0), NaN below all, the
// tokens that stay whatever their weight above all.
__device__ __forceinline__ uint32_t key_of(float weight, bool always) {
  const uint32_t b = __float_as_uint(weight + 0.f);
  if (always) return 0xffffffffu;
  if (weight != weight) return 0u;
  return b >> 31 ? ~b : b | 0x80000000u;
}

// What the rows' copies need of the cache beside its view.
struct Rows {
  FastDiv by_page, by_chunks, by_blocks;  // tokens of a page; 16-byte chunks, and scales, of a head's row
  int es;                                 // bytes of what the strides count
  uint32_t chunks, scales;                // of a token's K (or V): of all heads
};

// A token's place: bytes into k (and v), and words into their scales.
struct Place {
  long long at, scale;
  bool there;
};

__device__ __forceinline__ Place place_of(const KvEvictArgs& a, const Rows& R, int s, int i) {
  const uint32_t col = R.by_page.of(i), in_page = i - col * R.by_page.d;
  const uint32_t page = (uint32_t)a.table[s * a.table_stride + col];
  return {(page * a.kv.page + in_page * a.kv.token) * R.es, page * a.kv.spage + in_page * a.kv.stoken,
          page < (uint32_t)a.kv.n_pages};
}

// K and V of all heads, 16 bytes a lane of the warp, and the scales, 4 bytes a lane, from f, sf to t, st: all loads before the
// stores where a token has up to 64 chunks.
__device__ __forceinline__ void copy_token(const KvView& kv, const Rows& R, long long t, long long f, long long st, long long sf,
                                           int lane) {
  long long soff = 0;  // of the lane's first scale
  float ks = 0.f, vs = 0.f;
  if (lane < R.scales) {
    const uint32_t head = R.by_blocks.of(lane);
    soff = (long long)head * kv.shead + (lane - head * R.by_blocks.d);
    ks = kv.k_scale[sf + soff];
    vs = kv.v_scale[sf + soff];
  }
  for (uint32_t c0 = lane; c0 < R.chunks; c0 += 64) {
    uint4 k[2], v[2];
    long long off[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint32_t c = c0 + 32 * x, head = R.by_chunks.of(c);
      off[x] = (long long)head * kv.head * R.es + (c - head * R.by_chunks.d) * 16;
      if (c < R.chunks) {
        k[x] = *reinterpret_cast<const uint4*>(kv.k + f + off[x]);
        v[x] = *reinterpret_cast<const uint4*>(kv.v + f + off[x]);
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
      if (c0 + 32 * x < R.chunks) {
        *reinterpret_cast<uint4*>(kv.k + t + off[x]) = k[x];
        *reinterpret_cast<uint4*>(kv.v + t + off[x]) = v[x];
      }
  }
  if (lane < R.scales) {
    kv.k_scale[st + soff] = ks;
    kv.v_scale[st + soff] = vs;
  }
  for (uint32_t c = lane + 32; c < R.scales; c += 32) {
    const uint32_t head = R.by_blocks.of(c);
    const long long off = (long long)head * kv.shead + (c - head * R.by_blocks.d);
    kv.k_scale[st + off] = kv.k_scale[sf + off];
    kv.v_scale[st + off] = kv.v_scale[sf + off];
  }
}

// The choice, in both kernels below: the keep-th largest key digit by digit, from the highest (a histogram of the keys that
// match so far); among equal keys those of the lowest index, up to the last one taken; then the list of movers, which is put
// at the end of the sequence's row of `kept`; then the entries from it.  Of the list's M places the j-th lies at the j-th hole
// or behind it, and an entry that is no hole lies before every place that a later hole needs: filling the entries in order,
// each read before it is written, loses nothing.

// Any length: a CTA a sequence, keys computed again in each pass.
__global__ void __launch_bounds__(kThreads) kv_choose_long_kernel(const KvEvictArgs a) {
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
    if (tid == 0) a.drop[s] = left - max(a.lens[s], 0);
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
        if (in) atomicAdd(&s_count[key >> shift & 255u], 1u);
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

// The histogram of a digit.
struct alignas(16) Digits {
  uint32_t bins[2048], sums[64];  // sums: of 32 bins each
};
static_assert(alignof(Digits) % sizeof(uint2) == 0 && offsetof(Digits, sums) % sizeof(uint2) == 0 && sizeof(Digits) % sizeof(uint2) == 0,
              "bins and sums are read in pairs");

// Up to kMostKeys tokens a CTA: a cluster of 1 to 8 CTAs a sequence, the CTA of rank c with the c-th run of its tokens and
// their keys in shared memory, read once.  Bound by latency (barriers, and 12 bytes a token from a few SMs): up to three passes
// of 11, 11 and 10 bits (the last ones are left where all of a bin stay), whose histograms a warp of every CTA adds up
// through distributed shared memory, first sums of 32 bins, then the 32 bins that the digit is among (all 2048 in each CTA took
// 1 to 1.5 us more a pass), and one exchange of the numbers of movers and holes.  Where no more than kFewRows rows of a
// sequence can move it moves them too, and there is no second launch.
template <int CTAS, bool MOVE>
__global__ void __launch_bounds__(kThreads) kv_choose_kernel(const KvEvictArgs a, const Rows R) {
  extern __shared__ uint32_t s_keys[];
  __shared__ Digits s_digits[2];
  __shared__ uint32_t s_pick[4];
  __shared__ unsigned long long s_warp[kWarps], s_total;
  __shared__ int s_whole, s_last, s_moves, s_to[MOVE ? kFewRows : 1];
  constexpr int ctas = CTAS;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = CTAS == 1 ? 0 : (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto sync_all = [&]() {
    if constexpr (CTAS == 1)
      __syncthreads();
    else
      cluster.sync();
  };
  auto of_rank = [&](auto* p, int c) { return CTAS == 1 ? p : cluster.map_shared_rank(p, c); };
  // Sum of `mine` over the warps before this one (a warp's lanes have the same), and over all.
  auto sum_before = [&](unsigned long long mine, unsigned long long& all) {
    if (lane == 0) s_warp[warp] = mine;
    __syncthreads();
    const unsigned long long v = s_warp[lane];
    unsigned long long incl = v;
#pragma unroll
    for (int by = 1; by < 32; by *= 2) {
      const unsigned long long o = __shfl_up_sync(~0u, incl, by);
      if (lane >= by) incl += o;
    }
    all = __shfl_sync(~0u, incl, 31);
    const unsigned long long before = __shfl_sync(~0u, incl - v, warp);
    __syncthreads();
    return before;
  };
  grid_dep_launch();
  grid_dep_wait();
#pragma unroll 1
  for (int s = blockIdx.x / ctas; s < a.n_seq; s += gridDim.x / ctas) {
    const int n = min(max(a.lens[s], 0), a.cap), left = min(n, a.keep);
    const float* const weights = a.weights + s * a.weights_stride;
    float* const weights_out = a.weights_out + s * a.weights_stride;
    const int32_t* const positions = a.positions == nullptr ? nullptr : a.positions + s * a.positions_stride;
    int32_t* const positions_out = a.positions == nullptr ? nullptr : a.positions_out + s * a.positions_stride;
    int32_t* const kept = a.kept + s * a.kept_stride;
    if (tid == 0 && rank == 0) a.drop[s] = left - max(a.lens[s], 0);
    for (int i = left + rank * kThreads + tid; i < a.keep; i += ctas * kThreads) kept[i] = -1;
    if (n == left) {
      for (int i = rank * kThreads + tid; i < n; i += ctas * kThreads) {
        kept[i] = i;
        if (weights_out != weights) weights_out[i] = weights[i];
        if (positions_out != positions) positions_out[i] = positions[i];
      }
      continue;
    }
    // this CTA's run of tokens, its warps' runs of it (whole groups of 32), and its part before `keep`
    const int per = ((n + ctas - 1) / ctas + 31) & ~31, i0 = min(rank * per, n), i1 = min(i0 + per, n);
    const int per_warp = (((i1 - i0 + kWarps - 1) / kWarps) + 31) & ~31;
    const int w0 = min(i0 + warp * per_warp, i1), w1 = min(w0 + per_warp, i1);
    const int mid = max(i0, min(i1, a.keep));
    {
      const long long newest = positions == nullptr ? n - 1 : positions[n - 1];
#pragma unroll 1
      for (int at = i0 + tid; at < i1; at += 4 * kThreads) {
        float w[4];
        int p[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = at + k * kThreads;
          w[k] = i < i1 ? weights[i] : 0.f;
          p[k] = i < i1 && positions != nullptr ? positions[i] : i;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = at + k * kThreads;
          if (i < i1) s_keys[i - i0] = key_of(w[k], p[k] < a.first || p[k] > newest - a.recent);
        }
      }
    }

    // ---- the smallest key that stays, and how many of that key do
    uint32_t bar = 0, wanted = (uint32_t)a.keep;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, above = pass == 1 ? 21 : 10;
      const uint32_t mask = pass == 2 ? 1023u : 2047u;
      uint32_t *const count = s_digits[pass & 1].bins, *const coarse = s_digits[pass & 1].sums;  // the others are still read by other CTAs
      count[tid] = 0;
      count[tid + kThreads] = 0;
      __syncthreads();
      for (int at = w0 + lane; at < w1; at += 32) {
        const uint32_t key = s_keys[at - i0];
        if (pass == 0 || key >> above == bar >> above) atomicAdd(&count[key >> shift & mask], 1u);
      }
      __syncthreads();
      {
        const uint2 two = *reinterpret_cast<const uint2*>(count + 2 * tid);
        uint32_t sum = two.x + two.y;
#pragma unroll
        for (int by = 1; by < 16; by *= 2) sum += __shfl_xor_sync(~0u, sum, by);
        if (lane % 16 == 0) coarse[tid / 16] = sum;
      }
      sync_all();
      if (warp == 0) {
        // from the largest digit down: the 32 bins that it is in, two sums a lane, then the bin
        auto before_of = [&](uint32_t mine) {
          uint32_t incl = mine;
#pragma unroll
          for (int by = 1; by < 32; by *= 2) {
            const uint32_t o = __shfl_up_sync(~0u, incl, by);
            if (lane >= by) incl += o;
          }
          return incl - mine;
        };
        uint2 two[CTAS];
        uint32_t low = 0, high = 0, v[CTAS], sum = 0;
#pragma unroll
        for (int c = 0; c < CTAS; ++c) two[c] = *reinterpret_cast<const uint2*>(of_rank(coarse, c) + 62 - 2 * lane);
#pragma unroll
        for (int c = 0; c < CTAS; ++c) low += two[c].x, high += two[c].y;
        uint32_t before = before_of(low + high);
        const int in = __ffs(__ballot_sync(~0u, before < wanted && wanted <= before + low + high)) - 1;
        const bool upper = wanted <= before + high;
        const int group = __shfl_sync(~0u, 62 - 2 * lane + upper, in);
        const uint32_t rest = wanted - __shfl_sync(~0u, before + (upper ? 0u : high), in);
        const int digit = 32 * group + 31 - lane;
#pragma unroll
        for (int c = 0; c < CTAS; ++c) v[c] = of_rank(count, c)[digit];
#pragma unroll
        for (int c = 0; c < CTAS; ++c) sum += v[c];
        before = before_of(sum);
        if (before < rest && rest <= before + sum) {
          s_pick[0] = digit;
          s_pick[1] = rest - before;
          uint32_t lower = 0, here = 0;
#pragma unroll
          for (int c = 0; c < CTAS; ++c) {
            if (c < rank) lower += v[c];
            if (c == rank) here = v[c];
          }
          // where all of the bin stay, every key from its least on does, and the lower bits need not be looked at
          const bool whole = rest - before == sum;
          s_pick[2] = whole ? 0u : lower;
          s_pick[3] = whole ? 0u : here;
          s_whole = whole;
        }
      }
      __syncthreads();
      bar |= s_pick[0] << shift;
      wanted = s_pick[1];
      if (s_whole) break;
    }
    const uint32_t same_before = s_pick[2], same_here = s_pick[3];  // tokens of that key in lower ranks, and here

    // ---- the index of the last token of that key that stays
    const uint32_t quota = wanted > same_before ? min(wanted - same_before, same_here) : 0u;
    int last = quota == same_here ? i1 : -1;
    if (quota != 0 && quota != same_here) {
      uint32_t same = 0;
      for (int at = w0; at < w1; at += 32) same += __popc(__ballot_sync(~0u, at + lane < w1 && s_keys[at + lane - i0] == bar));
      unsigned long long all;
      uint32_t before = (uint32_t)sum_before(same, all);
      if (before < quota && quota <= before + same) {
        for (int at = w0; at < w1; at += 32) {
          uint32_t hits = __ballot_sync(~0u, at + lane < w1 && s_keys[at + lane - i0] == bar);
          if (before + __popc(hits) >= quota) {
            for (uint32_t skip = quota - before - 1; skip > 0; --skip) hits &= hits - 1;
            if (lane == 0) s_last = at + __ffs(hits) - 1;
            break;
          }
          before += __popc(hits);
        }
      }
      __syncthreads();
      last = s_last;
    }
    auto stays = [&](int i) {
      const uint32_t key = s_keys[i - i0];
      return key > bar || (key == bar && i <= last);
    };

    // ---- movers (in the lower halves of the sums) and holes (in the upper ones)
    unsigned long long mine = 0, here, before_me = 0, in_all = 0;
    for (int at = w0; at < w1; at += 32) {
      const int i = at + lane;
      const bool stay = i < w1 && stays(i);
      mine += __popc(__ballot_sync(~0u, stay && i >= a.keep));
      mine += (unsigned long long)__popc(__ballot_sync(~0u, i < w1 && i < a.keep && !stay)) << 32;
    }
    const unsigned long long in_cta = sum_before(mine, here);
    if (tid == 0) s_total = here;
    sync_all();
    {
      unsigned long long v[CTAS];
#pragma unroll
      for (int c = 0; c < CTAS; ++c) v[c] = *of_rank(&s_total, c);
#pragma unroll
      for (int c = 0; c < CTAS; ++c) {
        if (c < rank) before_me += v[c];
        in_all += v[c];
      }
    }
    if (MOVE && tid == 0) s_moves = 0;
    uint32_t mover = (uint32_t)(before_me + in_cta), hole = (uint32_t)((before_me + in_cta) >> 32);
    int32_t* const list = kept + (a.keep - (uint32_t)in_all);
    for (int at = max(w0, a.keep & ~31); at < w1; at += 32) {
      const int i = at + lane;
      const bool hit = i < w1 && i >= a.keep && i >= w0 && stays(i);
      const uint32_t hits = __ballot_sync(~0u, hit);
      if (hit) list[mover + __popc(hits & ((1u << lane) - 1))] = i;
      mover += __popc(hits);
    }
    sync_all();

    // ---- the entries: all of them read, then written
    const int end = min(w1, mid);
    for (int at = w0; at < end; at += 128) {
      uint32_t from[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = at + 32 * k + lane;
        const bool hit = i < end && !stays(i);
        const uint32_t hits = __ballot_sync(~0u, hit);
        from[k] = hit ? (uint32_t)list[hole + __popc(hits & ((1u << lane) - 1))] : (uint32_t)i;
        hole += __popc(hits);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (at + 32 * k + lane < end) s_keys[at + 32 * k + lane - i0] = from[k];
    }
    sync_all();
#pragma unroll 1
    for (int at = i0 + tid; at < mid; at += 4 * kThreads) {
      float w[4];
      int from[4], p[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = at + k * kThreads;
        from[k] = i < mid ? (int)s_keys[i - i0] : i;
        const bool moves = from[k] != i;
        w[k] = i < mid && (moves || weights_out != weights) ? weights[from[k]] : 0.f;
        p[k] = i < mid && positions != nullptr && (moves || positions_out != positions) ? positions[from[k]] : 0;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = at + k * kThreads;
        if (i >= mid) continue;
        const bool moves = from[k] != i;
        kept[i] = from[k];
        if (moves || weights_out != weights) weights_out[i] = w[k];
        if (positions != nullptr && (moves || positions_out != positions)) positions_out[i] = p[k];
        if (MOVE && moves) s_to[atomicAdd(&s_moves, 1)] = i;  // in any order: the rows lie apart
      }
    }
    __syncthreads();
    if constexpr (MOVE) {
      for (int m = warp; m < s_moves; m += kWarps) {
        const int i = s_to[m];
        const Place to = place_of(a, R, s, i), from = place_of(a, R, s, (int)s_keys[i - i0]);
        if (to.there && from.there)
          copy_token(a.kv, R, to.at, from.at, to.scale, from.scale, lane);
        else if (lane == 0)
          atomicOr(a.status, kStatusBadSlot);
      }
      __syncthreads();
    }
  }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveCtas = 4;  // an SM

// The rows, a warp an entry; a lane looks up one of the warp's next 32 entries.  Bound by HBM where many rows move.  Four CTAs an
// SM, all at once: with six (40 registers, which spill) 3584 of 4096 rows took 2.2 us more, with five 0.5, with three 1.6.
__global__ void __launch_bounds__(kMoveThreads, kMoveCtas) kv_move_kernel(const KvEvictArgs a, const Rows R) {
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (kMoveThreads / 32), total = (long long)a.n_seq * a.keep;
  grid_dep_launch();
  grid_dep_wait();
  for (long long e0 = blockIdx.x * (kMoveThreads / 32) + threadIdx.x / 32; e0 < total; e0 += 32 * warps) {
    const long long e = e0 + lane * warps;
    Place to = {0, 0, false}, from = {0, 0, false};
    if (e < total) {
      const int s = (int)(e / a.keep), i = (int)(e - (long long)s * a.keep);
      const int j = a.kept[s * a.kept_stride + i];
      if (j >= 0 && j != i) {
        to = place_of(a, R, s, i);
        from = place_of(a, R, s, j);
        if (!to.there || !from.there) atomicOr(a.status, kStatusBadSlot);
      }
    }
    uint32_t todo = __ballot_sync(~0u, to.there && from.there);
    while (todo != 0) {
      const int src = __ffs(todo) - 1;
      todo &= todo - 1;
      copy_token(a.kv, R, __shfl_sync(~0u, to.at, src), __shfl_sync(~0u, from.at, src), __shfl_sync(~0u, to.scale, src),
                 __shfl_sync(~0u, from.scale, src), lane);
    }
  }
}

}  // namespace

namespace {

template <int CTAS>
const void* choose_fn(bool move) {
  return move ? reinterpret_cast<const void*>(kv_choose_kernel<CTAS, true>)
              : reinterpret_cast<const void*>(kv_choose_kernel<CTAS, false>);
}

}  // namespace

cudaError_t prepare_kv_evict(const KvEvictArgs& a, int num_sms, std::vector<Launch>* out) {
  const KvView& kv = a.kv;
  const uint32_t row = (uint32_t)(kv.format == IL_BF16 ? 2 * kv.head_dim : kv.format == IL_Q8 ? kv.head_dim : kv.head_dim / 2);
  Rows R;
  R.by_page = FastDiv((uint32_t)kv.page_size);
  R.by_chunks = FastDiv(row / 16);
  R.by_blocks = FastDiv((uint32_t)std::max(1, kv.head_dim / 32));
  R.es = kv.format == IL_BF16 ? 2 : 1;
  R.chunks = row / 16 * kv.n_heads;
  R.scales = kv.format == IL_BF16 ? 0 : kv.head_dim / 32 * kv.n_heads;
  out->resize(1);
  Launch& choose = (*out)[0];
  choose.block = dim3(kThreads);
  const bool any_length = a.cap > kMostCtas * kMostKeys;
  // A sequence's own CTAs move its rows where few can move: one launch less (64 sequences of 1025 tokens cut to 1024: 12.5 ->
  // 7.9 us)
  const bool move = !any_length && a.cap - a.keep <= kFewRows;
  if (any_length) {
    choose.fn = reinterpret_cast<const void*>(kv_choose_long_kernel);
    choose.grid = dim3((unsigned)std::min(a.n_seq, 2 * num_sms));
    if (!choose.set_args(a)) return cudaErrorMemoryAllocation;
  } else {
    // CTAs of a sequence: as many as hold its keys, and more while that leaves each 4096 or more and all run at once
    int n = 0;
    while (n < 3 && (((int64_t)kMostKeys << n) < a.cap || (((int64_t)2 << n) * a.n_seq <= num_sms && (4096 << n) < a.cap))) ++n;
    const int ctas = 1 << n, per = ((a.cap + ctas - 1) / ctas + 31) & ~31;
    choose.fn = n == 0 ? choose_fn<1>(move) : n == 1 ? choose_fn<2>(move) : n == 2 ? choose_fn<4>(move) : choose_fn<8>(move);
    choose.smem = (size_t)per * 4;
    choose.grid = dim3((unsigned)(ctas * std::min(a.n_seq, std::max(1, 2 * num_sms / ctas))));
    static std::atomic<unsigned long long> attr_set[8];  // one bit per device, for each kernel (setting it twice is harmless)
    std::atomic<unsigned long long>& set = attr_set[2 * n + move];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !(set.load() & (1ull << dev))) {
      const cudaError_t e = cudaFuncSetAttribute(choose.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostKeys * 4);
      if (e != cudaSuccess) return e;
      if (dev < 64) set.fetch_or(1ull << dev);
    }
    if (ctas > 1) choose.set_cluster(ctas);
    if (!choose.set_args(a, R)) return cudaErrorMemoryAllocation;
  }
  if (kUsePdl) choose.allow_early_start();
  if (move) return cudaSuccess;
  out->resize(2);
  Launch& rows = (*out)[1];
  rows.fn = reinterpret_cast<const void*>(kv_move_kernel);
  const int64_t entries = (int64_t)a.n_seq * a.keep, per_cta = kMoveThreads / 32;
  rows.grid = dim3((unsigned)std::min<int64_t>((entries + per_cta - 1) / per_cta, (int64_t)num_sms * kMoveCtas));
  rows.block = dim3(kMoveThreads);
  if (!rows.set_args(a, R)) return cudaErrorMemoryAllocation;
  if (kUsePdl) rows.allow_early_start();
  return cudaSuccess;
}

}  // namespace il
