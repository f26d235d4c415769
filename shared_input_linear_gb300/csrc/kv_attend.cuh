// kv_attend.cuh -- attention of one new token per sequence over the paged cache (il_kv_attend):
// the kernel, instantiated per cache format in kv_attend_bf16.cu and kv_attend_q8.cu.
//
// For every sequence and K/V head, with G query heads reading that head:
//   s = scale q K^T, p = exp(s - max), out = p V / sum p        ([G][len] by [len][D])
// Each K and V byte is used G times, so the kernel is bound by HBM: it has to keep copies in
// flight on every SM for the whole launch, whatever the lengths, and do the arithmetic beside them.
//
// Work.  The tokens of a (sequence, K/V head) pair -- a row -- are cut into tiles of 16.  All tiles of all
// rows form one list, and every warp of the launch (one CTA per SM) takes an equal contiguous
// run of it, found from the prefix sums of the lengths that each CTA computes itself: ragged batches, long
// sequences and idle slots balance to one tile a warp without any host knowledge of the lengths.
// A row inside a warp's run is finished by the warp alone.  The ends of runs are parts of rows;
// they are joined in shared memory by the CTA (one barrier, after its stream), and rows that cross CTAs
// through the split workspace by the last CTA of the row to arrive, in CTA order: the result does
// not depend on the order of arrival.
//
// Stream.  Every warp owns a ring of stages, one tile of K and V each, filled with 16-byte
// cp.async (any strides, any page size: a lane looks up its token's page one tile ahead) and zeros for
// tokens outside the attended range.  No barrier other than the warp's own sits in the stream.
//
// Arithmetic.  Query heads are the rows of m16n8k16 MMAs and tokens (then elements of V) the
// columns; a softmax row lives in the four lanes of a quad.  q and p are fp32 and are split
// exactly enough to keep fp32's accuracy: against bf16 K and V into three bf16 parts (hi + mid + lo,
// 24 bits); against int8 into two fp16 parts (22 bits), with K's and V's integers decoded to exact
// fp16, K's block scales applied to each block's fp32 sum and V's to p, under a running power of two.
// With up to 8 heads (R = 1) hi fills rows 0-7 of an MMA and mid (int8: lo) rows 8-15, so the
// split costs one more MMA at bf16 and none at int8; with 9 to 16 heads (R = 2) every part is an MMA
// of its own.  Each tile's product starts from zero accumulators and joins the running sum in fp32
// FMAs (with the factor of the running maximum), which round to nearest.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "il_internal.cuh"
#include "il_ptx.cuh"

namespace il {

// What the host adds to KvAttendArgs for the kernel.
struct KvAttendPlan {
  KvAttendArgs a;
  int cap;                // longest length: table_width * page_size, at most 2^31 - 1
  int window;             // 0: all
  uint32_t div_m, div_s;  // t / page_size = (mulhi(div_m, t) + t) >> div_s
  int group;              // query heads of a K/V head
  int blocks;             // blocks of 8 R query heads of a K/V head
  float q_scale;          // scale * log2(e)
  unsigned* arrived;      // one counter a CTA, zero before and after
  float* parts;           // two parts a CTA
};

namespace attend {

constexpr int kTile = 16;
constexpr int kSmemLimit = 232448;  // 227 KB

template <bool Q8, int DP, int R>
struct Config {
  static constexpr int kRows = 8 * R;         // query heads of a block
  static constexpr int kBlocks = DP / 32;     // 32-element blocks of a row
  static constexpr int kPart = kRows * (DP + 2);  // floats of a part: sums, maxima, sums of p
  static constexpr int kRowBytes = Q8 ? DP : 2 * DP;
  static constexpr int kPool = kTile * kRowBytes;               // K or V of a tile
  static constexpr int kScales = Q8 ? kTile * kBlocks * 4 : 0;  // its scales
  static constexpr int kStage = 2 * (kPool + kScales);
  static constexpr int kWarps = !Q8 && DP == 256 ? 4 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kFixed = (kThreads + 2) * 8 + kWarps * 64 + 64;
  static constexpr int kRoom = (kSmemLimit - kFixed - kWarps * kPart * 4) / (kWarps * kStage);
  static constexpr int kStages = kRoom > 6 ? 6 : kRoom;
  static constexpr size_t kSmem = (size_t)kFixed + kWarps * kPart * 4 + (size_t)kWarps * kStages * kStage;
  static_assert(kStages >= 2 && kSmem <= kSmemLimit, "the ring does not fit");
  static_assert(kStages * kStage >= kPart * 4, "a part must fit the warp's ring");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool use) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(use ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool use) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(use ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void lds128(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
__device__ __forceinline__ void lds64(uint32_t& x, uint32_t& y, uint32_t at) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(at));
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(at));
  return r;
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}

template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float pow2_biased(int e) { return __int_as_float(e << 23); }  // 2^(e - 127), 0 < e < 255

// x, y as packed pairs of parts whose sum is them: three bf16 or two fp16.
__device__ __forceinline__ void split3(float x, float y, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  auto pack = [](float u, float v) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(u, v);
    return *reinterpret_cast<const uint32_t*>(&p);
  };
  hi = pack(x, y);
  x -= bf16_lo(hi);
  y -= bf16_hi(hi);
  mid = pack(x, y);
  lo = pack(x - bf16_lo(mid), y - bf16_hi(mid));
}
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// A sequence's attended range in tiles, and a place in the list of tiles.
struct Seq {
  uint32_t len, begin, first, tiles;
};
struct Walk {
  int s;          // sequence
  int vh;         // K/V head * blocks + block of query heads
  uint32_t tile;  // of the row
  Seq q;
};

__device__ __forceinline__ Seq seq_of(const KvAttendPlan& P, int s) {
  Seq q;
  const int len = min(max(P.a.lens[s], 0), P.cap);
  q.len = (uint32_t)len;
  q.begin = P.window > 0 ? (uint32_t)max(len - P.window, 0) : 0u;
  q.first = q.begin / kTile;
  q.tiles = len == 0 ? 0u : (q.len + kTile - 1) / kTile - q.first;
  return q;
}

__device__ __forceinline__ void advance(Walk& w, const KvAttendPlan& P, int rows_per_seq) {
  if (++w.tile < w.q.tiles) return;
  w.tile = 0;
  if (++w.vh < rows_per_seq) return;
  w.vh = 0;
  do w.q = seq_of(P, ++w.s);
  while (w.q.tiles == 0 && w.s + 1 < P.a.n_seq);
}

// What a warp leaves for the CTA: part 0, the end (or all) of a row begun before its run, and
// part 1, the beginning of a row that goes on behind it.
struct Left {
  int has0, end0, s0, vh0;
  int has1, s1, vh1;
  uint32_t tiles0, tiles1;
  long long row0, row1;  // first tiles of the rows in the list
};
static_assert(sizeof(Left) <= 64, "see Config::kFixed");

template <bool Q8, int DP, int R>
__global__ void __launch_bounds__(Config<Q8, DP, R>::kThreads, 1) kv_attend_kernel(const KvAttendPlan P) {
  using C = Config<Q8, DP, R>;
  constexpr int NB = C::kBlocks, NT = C::kThreads, NW = C::kWarps, S = C::kStages, ROWS = C::kRows;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* const ring_mem = smem;
  float* const part_mem = reinterpret_cast<float*>(smem + (size_t)NW * S * C::kStage);
  long long* const s_before = reinterpret_cast<long long*>(reinterpret_cast<uint8_t*>(part_mem) + NW * C::kPart * 4);
  Left* const s_left = reinterpret_cast<Left*>(s_before + NT + 2);
  long long* const s_warp = reinterpret_cast<long long*>(part_mem);  // of the scan: done before a part is written
  int* const s_flag = reinterpret_cast<int*>(s_left + NW);

  const KvAttendArgs& a = P.a;
  const KvView& kv = a.kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q4 = lane & 3;
  const int rows_per_seq = kv.n_heads * P.blocks, D = kv.head_dim;
  grid_dep_launch();
  grid_dep_wait();

  // ---- tiles before each run of sequences; sequences without tokens get their zeros
  const int run = (a.n_seq + NT - 1) / NT;
  long long mine = 0;
  for (int k = 0; k < run; ++k) {
    const int s = tid * run + k;
    const bool in = s < a.n_seq;
    const Seq q = in ? seq_of(P, s) : Seq{0, 0, 0, 0};
    mine += q.tiles;
    unsigned none = __ballot_sync(~0u, in && q.tiles == 0 && s % gridDim.x == blockIdx.x);
    while (none != 0) {
      const int src = __ffs(none) - 1;
      none &= none - 1;
      const int64_t z = __shfl_sync(~0u, s, src);
      for (int i = lane; i < a.n_q_heads * D / 4; i += 32)
        reinterpret_cast<float4*>(a.out + z * a.out_stride)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (a.lse != nullptr)
        for (int i = lane; i < a.n_q_heads; i += 32) a.lse[z * a.n_q_heads + i] = -INFINITY;
    }
  }
  long long incl = mine;
#pragma unroll
  for (int by = 1; by < 32; by *= 2) {
    const long long o = __shfl_up_sync(~0u, incl, by);
    if (lane >= by) incl += o;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  long long total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const long long t = s_warp[w];
    if (w < warp) before += t;
    total += t;
  }
  s_before[tid] = before + incl - mine;
  if (tid == 0) s_before[NT] = total;
  __syncthreads();

  // ---- this warp's run of the list: equal shares, the first `more` one tile longer
  const long long units = total * rows_per_seq;
  const int ctas = (int)min((long long)gridDim.x, (units + NW - 1) / NW);
  if ((int)blockIdx.x >= ctas) return;
  const int warps = ctas * NW;
  const long long share = units < (1ll << 32) ? (long long)((uint32_t)units / (uint32_t)warps) : units / warps;
  const int more = (int)(units - share * warps);
  auto begin_of = [&](int w) { return w * share + min(w, more); };
  const int my = blockIdx.x * NW + warp;
  const long long u0 = begin_of(my);
  const int n = (int)(begin_of(my + 1) - u0);  // a share of 2^31 tiles would be 10^5 GB of cache

  Left left;
  left.has0 = left.has1 = 0;
  if (n > 0) {
    Walk in;  // next tile to be fetched
    {
      int lo = 0;
#pragma unroll
      for (int step = NT / 2; step > 0; step /= 2)
        if (s_before[lo + step] * rows_per_seq <= u0) lo += step;
      long long at = u0 - s_before[lo] * rows_per_seq;
      in.s = lo * run;
      in.q = seq_of(P, in.s);
      while (at >= (long long)in.q.tiles * rows_per_seq && in.s + 1 < a.n_seq) {
        at -= (long long)in.q.tiles * rows_per_seq;
        in.q = seq_of(P, ++in.s);
      }
      in.vh = (int)(at < (1ll << 32) ? (uint32_t)at / in.q.tiles : at / in.q.tiles);
      in.tile = (uint32_t)(at - (long long)in.vh * in.q.tiles);
    }
    Walk at = in;  // tile being used
    const uint32_t ring = smem_u32(ring_mem) + warp * S * C::kStage;

    auto token_of = [&](const Walk& w) { return (w.q.first + w.tile) * kTile + (lane & 15); };
    auto column_of = [&](uint32_t t) { return (__umulhi(P.div_m, t) + t) >> P.div_s; };
    auto page_of = [&](const Walk& w) {  // page of this lane's token of the tile (lanes 16-31 repeat 0-15)
      const uint32_t t = token_of(w);
      int page = -1;
      if (t >= w.q.begin && t < w.q.len) {
        page = a.table[w.s * a.table_stride + column_of(t)];
      }
      return page;
    };
    // Copies the tile at `w`; gives the mask of its tokens that exist.
    auto fetch = [&](const Walk& w, int page, int stage) {
      const uint32_t t = token_of(w);
      const bool want = t >= w.q.begin && t < w.q.len;
      const bool ok = want && page >= 0 && page < kv.n_pages;
      if (want && !ok) atomicOr(a.status, kStatusBadSlot);
      const uint32_t in_page = t - column_of(t) * (uint32_t)kv.page_size;
      const int hk = w.vh / P.blocks;
      long long off = -1, soff = 0;
      if (ok) off = page * kv.page + in_page * kv.token + hk * kv.head;
      if (Q8 && ok) soff = page * kv.spage + in_page * kv.stoken + hk * kv.shead;
      constexpr int CPR = C::kRowBytes / 16, PER = 32 / CPR;  // 16-byte chunks of a row, rows of a copy
      const int chunk = lane % CPR;
      const bool in_row = chunk * (Q8 ? 16 : 8) < D;
      const uint32_t to = ring + stage * C::kStage;
#pragma unroll
      for (int i = 0; i < kTile / PER; ++i) {
        const int row = i * PER + lane / CPR;
        const long long o = __shfl_sync(~0u, off, row);
        const bool use = o >= 0 && in_row;
        const long long src = use ? (Q8 ? o + chunk * 16 : 2 * o + chunk * 16) : 0;
        int kc, vc, vrow = row;  // chunk positions: see the reads below
        if constexpr (Q8) {
          kc = chunk ^ ((DP == 64 ? (row >> 1) & 1 : row & 3) << 1);
          if (DP == 64) vrow = (row >> 1) | ((row & 1) << 3);
          vc = chunk ^ ((DP == 64 ? (vrow >> 1) & 1 : (row >> 1) & 3) << 1);
        } else {
          kc = chunk ^ ((row & 1) << 2);
          vc = chunk ^ (row & 7);
        }
        cp16(to + row * C::kRowBytes + kc * 16, kv.k + src, use);
        cp16(to + C::kPool + vrow * C::kRowBytes + vc * 16, kv.v + src, use);
      }
      if constexpr (Q8) {
        const uint32_t st = to + 2 * C::kPool;
#pragma unroll
        for (int i = 0; i < kTile * NB / 32; ++i) {
          const int row = (i * 32 + lane) / NB, b = (i * 32 + lane) % NB;
          const long long so = __shfl_sync(~0u, soff, row);
          const bool use = __shfl_sync(~0u, ok, row) && b * 32 < D;
          const long long src = use ? so + b : 0;
          cp4(st + (i * 32 + lane) * 4, kv.k_scale + src, use);
          cp4(st + C::kScales + (i * 32 + lane) * 4, kv.v_scale + src, use);
        }
      }
      return __ballot_sync(~0u, ok) & 0xffffu;
    };

    uint32_t mask[S];  // of the tiles in the ring
    int page = page_of(in);
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      if (i < n) {
        mask[i] = fetch(in, page, i);
        if (i + 1 < n) {
          advance(in, P, rows_per_seq);
          page = page_of(in);
        }
      }
      cp_commit();
    }

    // ---- the row being worked on
    constexpr int QR = Q8 ? 4 * R : 6 * R;  // registers of q for 16 elements
    uint32_t qf[2 * NB][QR];
    float q_back[R];  // Q8: the power of two that q was divided by
    constexpr int OC = 2 * R;
    float o[DP / 8][OC], m[R], l[R];
    int v_exp = 14;  // Q8: biased exponent of the largest V scale so far (of the sums' unit)

    auto load_q = [&]() {
      const int hk = at.vh / P.blocks, block = at.vh - hk * P.blocks;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int in_group = block * ROWS + r * 8 + g;
        const bool use = in_group < P.group;
        const float* src = a.q + at.s * a.q_stride + (int64_t)(hk * P.group + in_group) * D + 8 * q4;
        float x[NB][8];
        float top = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const bool in_row = use && 32 * b + 8 * q4 < D;
          const float4 u = in_row ? *reinterpret_cast<const float4*>(src + 32 * b) : make_float4(0.f, 0.f, 0.f, 0.f);
          const float4 v = in_row ? *reinterpret_cast<const float4*>(src + 32 * b + 4) : make_float4(0.f, 0.f, 0.f, 0.f);
          x[b][0] = u.x, x[b][1] = u.y, x[b][2] = u.z, x[b][3] = u.w;
          x[b][4] = v.x, x[b][5] = v.y, x[b][6] = v.z, x[b][7] = v.w;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[b][i] *= P.q_scale;
            if (Q8) top = fmaxf(top, fabsf(x[b][i]));
          }
        }
        if constexpr (Q8) {
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
          const int e = max((int)(__float_as_uint(top) >> 23), 14);
          const float up = pow2_biased(267 - e);  // the row's largest |q| becomes 2^13 .. 2^14
          q_back[r] = pow2_biased(e - 13);
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t hi, lo;
              split2(x[b][2 * i] * up, x[b][2 * i + 1] * up, hi, lo);
              qf[2 * b + i / 2][(i & 1) * 2 * R + r] = hi;
              qf[2 * b + i / 2][(i & 1) * 2 * R + R + r] = lo;
            }
        } else {
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t hi, mid, lo;
              split3(x[b][2 * i], x[b][2 * i + 1], hi, mid, lo);
              qf[2 * b + i / 2][(i & 1) * 3 * R + r] = hi;
              qf[2 * b + i / 2][(i & 1) * 3 * R + R + r] = mid;
              qf[2 * b + i / 2][(i & 1) * 3 * R + 2 * R + r] = lo;
            }
        }
        m[r] = -INFINITY;
        l[r] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < DP / 8; ++j)
#pragma unroll
        for (int c = 0; c < OC; ++c) o[j][c] = 0.f;
      v_exp = 14;
    };

    bool begun_here = at.tile == 0;
    load_q();
    for (int i0 = 0; i0 < n; i0 += S) {
#pragma unroll
      for (int st = 0; st < S; ++st) {
        const int i = i0 + st;
        if (i < n) {
          cp_wait<S - 2>();
          __syncwarp();
          // the stage used by the tile before this one takes the tile S - 1 ahead
          if (i + S - 1 < n) {
            mask[(st + S - 1) % S] = fetch(in, page, (st + S - 1) % S);
            if (i + S < n) {
              advance(in, P, rows_per_seq);
              page = page_of(in);
            }
          }
          cp_commit();
          const uint32_t from = ring + st * C::kStage;

          // ---- s = q K^T: s[r][2 nt + c] of head row g + 8 r, token 8 nt + 2 q4 + c
          float s[R][4];
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const int row = 8 * nt + g;
            if constexpr (Q8) {
              const uint32_t sc = from + 2 * C::kPool + (8 * nt + 2 * q4) * NB * 4;
#pragma unroll
              for (int r = 0; r < R; ++r) s[r][2 * nt] = s[r][2 * nt + 1] = 0.f;
#pragma unroll
              for (int b = 0; b < NB; ++b) {
                // element order inside a block: lane q4 holds 8 q4 .. 8 q4 + 7, as q does
                const int seg = b ^ (DP == 64 ? (row >> 1) & 1 : row & 3);
                uint32_t w0, w1, b0, b1, b2, b3;
                lds64(w0, w1, from + row * C::kRowBytes + seg * 32 + q4 * 8);
                q8_word_to_f16x2(w0 ^ 0x80808080u, b0, b1);
                q8_word_to_f16x2(w1 ^ 0x80808080u, b2, b3);
                float c[4] = {0.f, 0.f, 0.f, 0.f};
                const uint32_t(&x)[QR] = qf[2 * b];
                const uint32_t(&y)[QR] = qf[2 * b + 1];
                const float d0 = __uint_as_float(lds32(sc + b * 4)), d1 = __uint_as_float(lds32(sc + (NB + b) * 4));
                if constexpr (R == 1) {
                  mma<true>(c, x[0], x[1], x[2], x[3], b0, b1);
                  mma<true>(c, y[0], y[1], y[2], y[3], b2, b3);
                  s[0][2 * nt] = fmaf(c[0] + c[2], d0, s[0][2 * nt]);
                  s[0][2 * nt + 1] = fmaf(c[1] + c[3], d1, s[0][2 * nt + 1]);
                } else {
                  mma<true>(c, x[0], x[1], x[4], x[5], b0, b1);
                  mma<true>(c, y[0], y[1], y[4], y[5], b2, b3);
                  mma<true>(c, x[2], x[3], x[6], x[7], b0, b1);
                  mma<true>(c, y[2], y[3], y[6], y[7], b2, b3);
                  s[0][2 * nt] = fmaf(c[0], d0, s[0][2 * nt]);
                  s[0][2 * nt + 1] = fmaf(c[1], d1, s[0][2 * nt + 1]);
                  s[R - 1][2 * nt] = fmaf(c[2], d0, s[R - 1][2 * nt]);
                  s[R - 1][2 * nt + 1] = fmaf(c[3], d1, s[R - 1][2 * nt + 1]);
                }
              }
#pragma unroll
              for (int r = 0; r < R; ++r) s[r][2 * nt] *= q_back[r], s[r][2 * nt + 1] *= q_back[r];
            } else {
              float c[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int b = 0; b < NB; ++b) {
                uint32_t w[4];
                lds128(w, from + row * C::kRowBytes + (((4 * b + q4) ^ ((row & 1) << 2)) << 4));
                const uint32_t(&x)[QR] = qf[2 * b];
                const uint32_t(&y)[QR] = qf[2 * b + 1];
                if constexpr (R == 1) {
                  mma<false>(c, x[0], x[1], x[3], x[4], w[0], w[1]);
                  mma<false>(e, x[2], 0u, x[5], 0u, w[0], w[1]);
                  mma<false>(c, y[0], y[1], y[3], y[4], w[2], w[3]);
                  mma<false>(e, y[2], 0u, y[5], 0u, w[2], w[3]);
                } else {
                  mma<false>(c, x[0], x[1], x[6], x[7], w[0], w[1]);
                  mma<false>(e, x[2], x[3], x[8], x[9], w[0], w[1]);
                  mma<false>(e, x[4], x[5], x[10], x[11], w[0], w[1]);
                  mma<false>(c, y[0], y[1], y[6], y[7], w[2], w[3]);
                  mma<false>(e, y[2], y[3], y[8], y[9], w[2], w[3]);
                  mma<false>(e, y[4], y[5], y[10], y[11], w[2], w[3]);
                }
              }
              if constexpr (R == 1) {
                s[0][2 * nt] = c[0] + (c[2] + e[0]);
                s[0][2 * nt + 1] = c[1] + (c[3] + e[1]);
              } else {
                s[0][2 * nt] = c[0] + e[0];
                s[0][2 * nt + 1] = c[1] + e[1];
                s[R - 1][2 * nt] = c[2] + e[2];
                s[R - 1][2 * nt + 1] = c[3] + e[3];
              }
            }
          }

          // ---- softmax: the tile's maximum, p, and the factor of what came before
          const uint32_t mk = mask[st];
          if (mk != 0xffffu) {
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c)
                if (!((mk >> (8 * nt + 2 * q4 + c)) & 1))
#pragma unroll
                  for (int r = 0; r < R; ++r) s[r][2 * nt + c] = -INFINITY;
          }
          float keep[R];
#pragma unroll
          for (int r = 0; r < R; ++r) {
            float top = fmaxf(fmaxf(s[r][0], s[r][1]), fmaxf(s[r][2], s[r][3]));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
            const float now = fmaxf(m[r], top), base = now == -INFINITY ? 0.f : now;
            keep[r] = exp2_fast(m[r] - base);
            m[r] = now;
#pragma unroll
            for (int c = 0; c < 4; ++c) s[r][c] = exp2_fast(s[r][c] - base);
            l[r] = fmaf(l[r], keep[r], (s[r][0] + s[r][1]) + (s[r][2] + s[r][3]));
          }

          // ---- o = o * keep + p V
          const uint32_t fv = from + C::kPool;
          if constexpr (Q8) {
            const uint32_t sv = from + 2 * C::kPool + C::kScales;
            float d[4][NB];  // scales of tokens 2 q4, 2 q4 + 1, and 8 more
            uint32_t top = 0;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
              for (int b = 0; b < NB; ++b) {
                const uint32_t u = lds32(sv + ((2 * q4 + (t & 1) + 8 * (t >> 1)) * NB + b) * 4);
                d[t][b] = __uint_as_float(u);
                top = max(top, u & 0x7fffffffu);
              }
            top = max(top, __shfl_xor_sync(~0u, top, 1));
            top = max(top, __shfl_xor_sync(~0u, top, 2));
            const int e = max(v_exp, (int)(top >> 23));
            const float up = pow2_biased(267 - e);  // the largest scale becomes 2^13 .. 2^14
            const float shift = e - v_exp > 126 ? 0.f : pow2_biased(127 + v_exp - e);
            v_exp = e;
#pragma unroll
            for (int r = 0; r < R; ++r) keep[r] *= shift;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              uint32_t p[4 * R];  // hi of tokens 2 q4 .. (of every row), lo, then of the tokens 8 further
#pragma unroll
              for (int r = 0; r < R; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  split2(s[r][2 * h] * (d[2 * h][b] * up), s[r][2 * h + 1] * (d[2 * h + 1][b] * up), p[2 * R * h + r],
                         p[2 * R * h + R + r]);
              uint32_t f[2][4];  // V of tokens (2 q4, 2 q4 + 1) and 8 further, elements 32 b + 4 g + 0..3
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                auto word = [&](int t) {
                  const int vrow = DP == 64 ? (t >> 1) | ((t & 1) << 3) : t;
                  const int seg = b ^ (DP == 64 ? (vrow >> 1) & 1 : (t >> 1) & 3);
                  return lds32(fv + vrow * C::kRowBytes + seg * 32 + g * 4) ^ 0x80808080u;
                };
                const uint32_t x = word(8 * h + 2 * q4), y = word(8 * h + 2 * q4 + 1);
                q8_word_to_f16x2(__byte_perm(x, y, 0x5140), f[h][0], f[h][1]);
                q8_word_to_f16x2(__byte_perm(x, y, 0x7362), f[h][2], f[h][3]);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                float c[4] = {0.f, 0.f, 0.f, 0.f};
                float(&acc)[OC] = o[4 * b + j];
                if constexpr (R == 1) {
                  mma<true>(c, p[0], p[1], p[2], p[3], f[0][j], f[1][j]);
                  acc[0] = fmaf(acc[0], keep[0], c[0] + c[2]);
                  acc[1] = fmaf(acc[1], keep[0], c[1] + c[3]);
                } else {
                  mma<true>(c, p[0], p[1], p[4], p[5], f[0][j], f[1][j]);
                  mma<true>(c, p[2], p[3], p[6], p[7], f[0][j], f[1][j]);
#pragma unroll
                  for (int x = 0; x < 4; ++x) acc[x % OC] = fmaf(acc[x % OC], keep[(x / 2) % R], c[x]);
                }
              }
            }
          } else {
            uint32_t hi[2 * R], mid[2 * R], lo[2 * R];  // of tokens 2 q4 .. and 8 further, by row
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                split3(s[r][2 * h], s[r][2 * h + 1], hi[R * h + r], mid[R * h + r], lo[R * h + r]);
#pragma unroll
            for (int j = 0; j < DP / 8; j += 2) {
              uint32_t w[4];
              const int t = lane & 15;
              ldmatrix4_trans(w, fv + t * C::kRowBytes + (((j + (lane >> 4)) ^ (t & 7)) << 4));
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float c[4] = {0.f, 0.f, 0.f, 0.f};
                float(&acc)[OC] = o[j + h];
                if constexpr (R == 1) {
                  mma<false>(c, hi[0], mid[0], hi[1], mid[1], w[2 * h], w[2 * h + 1]);
                  mma<false>(c, lo[0], 0u, lo[1], 0u, w[2 * h], w[2 * h + 1]);
                  acc[0] = fmaf(acc[0], keep[0], c[0] + c[2]);
                  acc[1] = fmaf(acc[1], keep[0], c[1] + c[3]);
                } else {
                  mma<false>(c, hi[0], hi[1], hi[2 % (2 * R)], hi[3 % (2 * R)], w[2 * h], w[2 * h + 1]);
                  mma<false>(c, mid[0], mid[1], mid[2 % (2 * R)], mid[3 % (2 * R)], w[2 * h], w[2 * h + 1]);
                  mma<false>(c, lo[0], lo[1], lo[2 % (2 * R)], lo[3 % (2 * R)], w[2 * h], w[2 * h + 1]);
#pragma unroll
                  for (int x = 0; x < 4; ++x) acc[x % OC] = fmaf(acc[x % OC], keep[(x / 2) % R], c[x]);
                }
              }
            }
          }

          // ---- the row's or the run's end
          const bool row_ends = at.tile + 1 == at.q.tiles;
          if (row_ends || i + 1 == n) {
            const float unit = Q8 ? pow2_biased(v_exp - 13) : 1.f;
            const bool alone = begun_here && row_ends;
            float* part = nullptr;
            if (!alone) {
              const long long row = u0 + i - at.tile;
              if (!begun_here) {
                left.has0 = 1, left.end0 = row_ends, left.s0 = at.s, left.vh0 = at.vh;
                left.tiles0 = at.q.tiles, left.row0 = row;
                part = part_mem + warp * C::kPart;
              } else {  // the run's last tile: nothing is in flight into the ring any more
                left.has1 = 1, left.s1 = at.s, left.vh1 = at.vh;
                left.tiles1 = at.q.tiles, left.row1 = row;
                part = reinterpret_cast<float*>(ring_mem + (size_t)warp * S * C::kStage);
                cp_wait<0>();
                __syncwarp();
              }
            }
            const int hk = at.vh / P.blocks, block = at.vh - hk * P.blocks;
#pragma unroll
            for (int r = 0; r < R; ++r) {
              float sum = l[r];
              sum += __shfl_xor_sync(~0u, sum, 1);
              sum += __shfl_xor_sync(~0u, sum, 2);
              const int in_group = block * ROWS + 8 * r + g;
              const int64_t head = (int64_t)hk * P.group + in_group;
              const float f = alone ? (sum == 0.f ? 0.f : unit / sum) : unit;
              float* to = alone ? a.out + at.s * a.out_stride + head * D : part + (8 * r + g) * DP;
              if (in_group < P.group) {
                if constexpr (Q8) {
#pragma unroll
                  for (int b = 0; b < NB; ++b)
                    if (32 * b < D) {
#pragma unroll
                      for (int c = 0; c < 2; ++c)
                        *reinterpret_cast<float4*>(to + 32 * b + 8 * q4 + 4 * c) =
                            make_float4(o[4 * b][2 * r + c] * f, o[4 * b + 1][2 * r + c] * f, o[4 * b + 2][2 * r + c] * f,
                                        o[4 * b + 3][2 * r + c] * f);
                    }
                } else {
#pragma unroll
                  for (int j = 0; j < DP / 8; ++j)
                    if (8 * j < D)
                      *reinterpret_cast<float2*>(to + 8 * j + 2 * q4) = make_float2(o[j][2 * r] * f, o[j][2 * r + 1] * f);
                }
                if (q4 == 0) {
                  if (alone) {
                    if (a.lse != nullptr)
                      a.lse[(int64_t)at.s * a.n_q_heads + head] =
                          sum == 0.f ? -INFINITY : (m[r] + log2f(sum)) * 0.6931471805599453f;
                  } else {
                    part[ROWS * DP + 8 * r + g] = m[r];
                    part[ROWS * DP + ROWS + 8 * r + g] = sum;
                  }
                }
              }
            }
          }
          if (i + 1 < n) {
            advance(at, P, rows_per_seq);
            if (at.tile == 0) {
              begun_here = true;
              load_q();
            }
          }
        }
      }
    }
    cp_wait<0>();
  }
  if (lane == 0) s_left[warp] = left;
  __syncthreads();

  // ---- parts of rows: sums of the CTA's, to the output or to the workspace
  // Adds up parts in order; `of(i)` is the i-th, in shared memory or (past this SM's L1) in the workspace.
  // Thread e takes four elements of a row.
  auto join = [&](auto in_workspace, int count, int s, int vh, auto of, float* to_part) {
    constexpr bool kL2 = decltype(in_workspace)::value;
    auto load = [](const auto* x) {
      if constexpr (kL2)
        return __ldcg(x);
      else
        return *x;
    };
    const int hk = vh / P.blocks, block = vh - hk * P.blocks;
    const int rows = min(ROWS, P.group - block * ROWS);
    for (int e = tid; e < rows * (DP / 4); e += NT) {
      const int row = e / (DP / 4), c = 4 * (e % (DP / 4));
      if (c >= D) continue;
      float M = -INFINITY, L = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int i = 0; i < count; ++i) {
        const float* p = of(i);
        const float pm = load(p + ROWS * DP + row), pl = load(p + ROWS * DP + ROWS + row);
        const float4 y = load(reinterpret_cast<const float4*>(p + row * DP + c));
        const float now = fmaxf(M, pm), base = now == -INFINITY ? 0.f : now;
        const float f = exp2_fast(M - base), h = exp2_fast(pm - base);
        M = now;
        L = fmaf(L, f, pl * h);
        x.x = fmaf(x.x, f, y.x * h);
        x.y = fmaf(x.y, f, y.y * h);
        x.z = fmaf(x.z, f, y.z * h);
        x.w = fmaf(x.w, f, y.w * h);
      }
      if (to_part != nullptr) {
        *reinterpret_cast<float4*>(to_part + row * DP + c) = x;
        if (c == 0) {
          to_part[ROWS * DP + row] = M;
          to_part[ROWS * DP + ROWS + row] = L;
        }
      } else {
        const int64_t head = (int64_t)hk * P.group + block * ROWS + row;
        const float f = L == 0.f ? 0.f : 1.f / L;
        *reinterpret_cast<float4*>(a.out + s * a.out_stride + head * D + c) = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
        if (c == 0 && a.lse != nullptr)
          a.lse[(int64_t)s * a.n_q_heads + head] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
      }
    }
  };
  auto global_part = [&](int cta, int which) { return P.parts + ((int64_t)cta * 2 + which) * C::kPart; };

  bool crosses[2] = {false, false};
  for (int w = -1; w < NW; ++w) {  // the row that came into the CTA, then those that warp w left open
    if (w < 0 ? !s_left[0].has0 : !s_left[w].has1) continue;
    int end = w + 1;
    bool ends = false;
    while (end < NW && s_left[end].has0 && !ends) ends = s_left[end++].end0 != 0;
    const int s = w < 0 ? s_left[0].s0 : s_left[w].s1, vh = w < 0 ? s_left[0].vh0 : s_left[w].vh1;
    const bool whole = w >= 0 && ends;
    if (!whole) crosses[w < 0 ? 0 : 1] = true;
    const int count = end - max(w, 0);
    auto of = [&](int i) -> const float* {
      const int at = max(w, 0) + i;
      return at == w ? reinterpret_cast<const float*>(ring_mem + (size_t)at * S * C::kStage) : part_mem + at * C::kPart;
    };
    join(std::false_type(), count, s, vh, of, whole ? nullptr : global_part(blockIdx.x, w < 0 ? 0 : 1));
  }
  if (!crosses[0] && !crosses[1]) return;

  // ---- rows that cross CTAs: the last to arrive sums them in CTA order
  auto owner = [&](long long u) {  // CTA of tile u of the list
    const long long split = more * (share + 1);
    const long long w = u < split ? u / (share + 1) : more + (u - split) / share;
    return (int)(w / NW);
  };
  __threadfence();
  __syncthreads();
  for (int which = 0; which < 2; ++which) {
    if (!crosses[which]) continue;
    int w = 0;  // the warp that knows the row
    if (which == 1) {
      w = NW - 1;
      while (!s_left[w].has1) --w;
    }
    const Left& r = s_left[w];
    const long long row = which == 0 ? r.row0 : r.row1;
    const int c0 = owner(row), c1 = owner(row + (which == 0 ? r.tiles0 : r.tiles1) - 1);
    const int count = c1 - c0 + 1;
    if (tid == 0) {
      const unsigned seen = atomicAdd(P.arrived + c0, 1u);
      *s_flag = seen == (unsigned)count - 1;
      if (*s_flag) P.arrived[c0] = 0;
    }
    __syncthreads();
    if (*s_flag) {
      __threadfence();
      join(std::true_type(), count, which == 0 ? r.s0 : r.s1, which == 0 ? r.vh0 : r.vh1,
           [&](int i) -> const float* { return global_part(c0 + i, i == 0 ? 1 : 0); }, nullptr);
    }
    __syncthreads();
  }
}

template <bool Q8, int DP, int R>
cudaError_t prepare_variant(const KvAttendPlan& p, int ctas, Launch* out) {
  using C = Config<Q8, DP, R>;
  static std::atomic<unsigned long long> attr_set{0};  // one bit per device (setting it twice is harmless)
  const void* fn = reinterpret_cast<const void*>(kv_attend_kernel<Q8, DP, R>);
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !(attr_set.load() & (1ull << dev))) {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set.fetch_or(1ull << dev);
  }
  out->fn = fn;
  out->grid = dim3((unsigned)ctas);
  out->block = dim3(C::kThreads);
  out->smem = C::kSmem;
  if (!out->set_args(p)) return cudaErrorMemoryAllocation;
  if (kUsePdl) out->allow_early_start();
  return cudaSuccess;
}

// The variant of a cache: head_dim rounded up to 64, 128 or 256, and blocks of 8 query heads, or of
// 16 where the group has more than 8 and the registers hold them (head_dim <= 128).
template <bool Q8>
cudaError_t prepare_format(const KvAttendPlan& p, int dim, bool wide, int ctas, Launch* out) {
  if (dim == 256) return prepare_variant<Q8, 256, 1>(p, ctas, out);
  if (dim == 128) return wide ? prepare_variant<Q8, 128, 2>(p, ctas, out) : prepare_variant<Q8, 128, 1>(p, ctas, out);
  return wide ? prepare_variant<Q8, 64, 2>(p, ctas, out) : prepare_variant<Q8, 64, 1>(p, ctas, out);
}

}  // namespace attend

cudaError_t prepare_kv_attend_bf16(const KvAttendPlan& p, int dim, bool wide, int ctas, Launch* out);
cudaError_t prepare_kv_attend_q8(const KvAttendPlan& p, int dim, bool wide, int ctas, Launch* out);

}  // namespace il
