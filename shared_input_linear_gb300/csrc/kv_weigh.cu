// kv_weigh.cu -- il_kv_weigh: the attention weight that one new token per sequence gives each cached token, summed over the
// query heads and added to what the token has collected.
//
//   out[t] = (new ? 0 : w[t]) + sum_h exp(s_ht - lse_h)
// K is read once and V not at all; the sum over the heads of a token is made where its K is, so that nothing but 8 bytes a
// token goes beside K.
//
// Measured (GB300, 32 query heads on 8 K/V heads of 128, device time): 64 sequences of 1 to 8192 tokens bf16 104 us, 6.3 TB/s,
// Q8 66 us, 5.6 TB/s, A4 51 us, 4.1 TB/s; one of 131071 A4 24 us; one of 2048 bf16 6.3 us.  A4 in other layouts, 64 sequences: 64
// heads on 8 of 128, 4096 tokens, 62 us, 2.8 TB/s; 8192 tokens of 32 on 8 of 64 52 us, 3.3 TB/s, of 8 on one of 256 46 us, 1.9 TB/s.
// What bounds it: HBM at bf16; at A4 issue (343 instructions for 32 tokens of a K/V head, about as many as there are slots at HBM's rate, of
// which 62 % are used; ALU 52 %) and what the CTAs lose at the ends of pieces; of a short call the latencies before the first tile.
//
// Work.  Tiles of 32 tokens (16 of bf16 heads above 128) of all sequences form one list, of which every CTA takes an equal
// run.  A run's piece of one sequence is worked off by the CTA's warps, a tile each at a time, over all K/V heads; of the last
// tiles of a piece, fewer than the warps, each is shared by several warps that take every second, fourth or eighth head, and
// whose sums are added in order.  Which warp does what depends on the lengths alone: equal calls give equal bits.
//
// q is split into the MMAs' parts once per sequence and CTA (by its warps, a K/V head each) and read from shared memory as
// fragments; heads beyond what fits there are taken in batches.  Each warp has a ring of K tiles of its own, filled with
// cp.async ahead of use across heads, tiles and sequences.
//
// Arithmetic.  Tokens are the rows of m16n8k16 MMAs and query heads the columns, two for each of four heads, as in
// kv_a4.cuh: the hi and lo parts of q in fp16 against 4-bit and 8-bit integers (K's bytes u = q + 128 as subnormals, the
// products with the 128 taken off by where the sums start), or three bf16 parts in two MMAs against bf16.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "il_internal.cuh"
#include "il_ptx.cuh"
#include "kv_a4.cuh"

namespace il {

namespace weigh {

struct Plan {
  KvWeighArgs w;
  int cap, window;
  FastDiv by_page;
  int group, blocks;  // query heads of a K/V head, blocks of 4 of them
  float q_scale, cap_log2;
  int hks, cols;      // K/V heads, and blocks of each, whose q is in shared memory at a time
  int whole;          // a token's scales can be copied as 16 bytes (8 for heads of 64), and offsets below fit 32 bits
  uint32_t page, token;    // strides in 16 bytes
  uint32_t spage, stoken;  // of the scales in words
};

// The largest of x over the four lanes of a quad.
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(~0u, x, 1));
  return fmaxf(x, __shfl_xor_sync(~0u, x, 2));
}

// Four query heads against 16 tokens of a cache, per format.  load(e, x) gives elements e .. of head g / 2 of the four, times
// the scale of the logits, four or two of them; dot gives s[h] of head q4 with token 8 h + g.  kWords: registers of a lane,
// kept in shared memory between uses.
template <int F, int NB>
struct Heads;

template <int NB>
struct Heads<IL_A4, NB> {
  static constexpr int kWords = 5 * NB + 2;
  a4::Query<NB, 1, true> q;
  template <class Load>
  __device__ __forceinline__ void take(const Load& load, int lane) {
    float x[NB][8], top = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        float y[4];
        load(32 * b + 8 * (lane & 3) + j, y);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[b][j + k] = y[k], top = fmaxf(top, fabsf(y[k]));
      }
    q.take(0, x, quad_max(top), lane);
  }
  __device__ __forceinline__ uint32_t& word(int i) {
    return i < 4 * NB ? q.f[0][i] : i < 5 * NB ? q.sum[0][i - 4 * NB] : reinterpret_cast<uint32_t&>(q.back[0][i - 5 * NB]);
  }
  __device__ __forceinline__ void dot(float (&s)[2], uint32_t tile, uint32_t steps, int first, int lane) const {
    uint32_t chunks[NB / 2];
#pragma unroll
    for (int i = 0; i < NB / 2; ++i) chunks[i] = a4::chunk_at<NB>(lane & 15, 2 * i + (lane >> 4));
    float t[1][2];
    q.dot(t, tile + first * 16 * NB, steps + first * 4 * NB, chunks, lane);
    s[0] = t[0][0], s[1] = t[0][1];
  }
};

template <int NB>
struct Heads<IL_Q8, NB> {
  static constexpr int kWords = 5 * NB + 2;
  a4::Query8<NB, 1> q;
  template <class Load>
  __device__ __forceinline__ void take(const Load& load, int lane) {
    float x[NB][8], top = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        float y[4];
        load(32 * b + 4 * j + 4 * (lane & 3), y);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[b][j + k] = y[k], top = fmaxf(top, fabsf(y[k]));
      }
    q.take(0, x, quad_max(top), lane);
  }
  __device__ __forceinline__ uint32_t& word(int i) {
    return i < 4 * NB ? q.f[0][i] : reinterpret_cast<uint32_t&>(i < 5 * NB ? q.start[0][i - 4 * NB] : q.back[0][i - 5 * NB]);
  }
  __device__ __forceinline__ void dot(float (&s)[2], uint32_t tile, uint32_t steps, int first, int lane) const {
    uint32_t chunks[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) chunks[i] = a4::chunk_at<2 * NB>(lane & 15, 2 * i + (lane >> 4));
    float t[1][2];
    q.dot(t, tile + first * 32 * NB, steps + first * 4 * NB, chunks, lane);
    s[0] = t[0][0], s[1] = t[0][1];
  }
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int NB>
struct Heads<IL_BF16, NB> {
  static constexpr int kWords = 8 * NB;
  uint32_t f[8 * NB];  // of 16-element chunk i: elements 16 i + 2 q4, + 1 and + 8, + 9 as (hi, mid), then as (lo, 0)
  template <class Load>
  __device__ __forceinline__ void take(const Load& load, int lane) {
    const int q4 = lane & 3;
    const bool second = (lane >> 2) & 1;
    auto pack = [](float u, float v) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(u, v);
      return *reinterpret_cast<const uint32_t*>(&p);
    };
    float all[2 * NB][2][2];
#pragma unroll
    for (int i = 0; i < 4 * NB; ++i) load(16 * (i / 2) + 2 * q4 + 8 * (i % 2), all[i / 2][i % 2]);
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x = all[i][j][0], y = all[i][j][1];
        const uint32_t hi = pack(x, y);
        x -= bf16_lo(hi), y -= bf16_hi(hi);
        const uint32_t mid = pack(x, y);
        f[4 * i + j] = second ? mid : hi;
        f[4 * i + 2 + j] = second ? 0u : pack(x - bf16_lo(mid), y - bf16_hi(mid));
      }
  }
  __device__ __forceinline__ uint32_t& word(int i) { return f[i]; }
  __device__ __forceinline__ void dot(float (&s)[2], uint32_t tile, uint32_t, int first, int lane) const {
    float c[4] = {0.f, 0.f, 0.f, 0.f}, l[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i) {
      uint32_t k[4];
      a4::ldmatrix4(k, tile + a4::chunk_at<4 * NB>(first + (lane & 15), 2 * i + (lane >> 4)));
      mma_bf16(c, k, f[4 * i], f[4 * i + 1]);
      mma_bf16(l, k, f[4 * i + 2], f[4 * i + 3]);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) s[t] = c[2 * t] + (c[2 * t + 1] + l[2 * t]);
  }
};

constexpr int kSmemLimit = 232448;

template <int F, int W>
struct Config {
  static constexpr int kBlocks = W / 32;
  static constexpr int kRowBytes = F == IL_BF16 ? 2 * W : F == IL_Q8 ? W : W / 2;
  static constexpr int kTile = F == IL_BF16 && W == 256 ? 16 : 32;
  static constexpr int kChunk = 16 * W / kRowBytes;  // elements of 16 bytes
  static constexpr int kPool = kTile * kRowBytes;
  static constexpr int kScales = F == IL_BF16 ? 0 : kTile * kBlocks * 4;
  static constexpr int kStage = kPool + kScales;
  // As many as the registers and the rings leave.  A4, 64 ragged sequences of heads of 128: 8 warps 63 us, 12 and 16 56 us;
  // 8192 tokens of heads of 64: 68, 56, 53 us.  Q8 72 to 76 us with 8 or 12.
  static constexpr int kWarps = F == IL_BF16 || W == 256 ? 8 : F == IL_A4 ? 16 : 12;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kStages = kStage > 5000 ? 2 : 3;
  static constexpr int kRowsOf = kTile * kRowBytes / 512;  // copies of a lane, a row each
  static constexpr int kRing = kStages * kStage;
  // Of a lane, in fours: the fragments, and of head q4 the lse, times log2(e), and the slope
  static constexpr int kFours = (Heads<F, kBlocks>::kWords + 2 + 3) / 4;
  static constexpr int kHeads = 512 * kFours;  // bytes of four query heads
  static constexpr int kFixed = kThreads * 8 + kWarps * 8 + 2 * kWarps * kTile * 4 + kWarps * 32;
  static constexpr int kBatch = (kSmemLimit - kFixed - kWarps * kRing) / kHeads;  // fours of heads that fit
  static_assert(kBatch >= 1, "the ring leaves no room for q");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool use) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(use ? 16 : 0) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void cp_small(uint32_t dst, const void* src, bool use) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(use ? BYTES : 0) : "memory");
}

struct Seq {
  uint32_t len, begin, first, tiles;  // tiles from `first` on hold the seen tokens
};

// What a CTA has of one sequence: `count` tiles from tile0 (of the seen ones) on, the first of them tile `at` of the list.
struct Piece {
  int s;
  Seq q;
  uint32_t tile0, count;
  long long at;
};

template <int T, bool SCORED>
__device__ __forceinline__ Seq seq_of(const Plan& P, int s) {
  Seq q;
  const int len = min(max(P.w.attend.lens[s], 0), P.cap);
  q.len = (uint32_t)len;
  q.begin = P.window > 0 ? (uint32_t)max(len - P.window, 0) : 0u;
  if (SCORED && P.w.attend.starts != nullptr) q.begin = max(q.begin, (uint32_t)min(max(P.w.attend.starts[s], 0), len));
  q.first = q.begin / T;
  q.tiles = q.begin == q.len ? 0u : (q.len + T - 1) / T - q.first;
  return q;
}

template <int F, bool SCORED, int W>
__global__ void __launch_bounds__(Config<F, W>::kThreads, 1) kv_weigh_kernel(const Plan P) {
  using C = Config<F, W>;
  using Q = Heads<F, C::kBlocks>;
  constexpr int T = C::kTile, NB = C::kBlocks, NW = C::kWarps, NT = C::kThreads, S = C::kStages, NV = T / 8;
  extern __shared__ __align__(128) uint8_t smem[];
  uint4* const heads_mem = reinterpret_cast<uint4*>(smem + NW * C::kRing);  // [four][kFours][lane]
  long long* const s_before = reinterpret_cast<long long*>(smem + NW * C::kRing + (size_t)P.hks * P.cols * C::kHeads);
  long long* const s_warp = s_before + NT;
  float* const s_sums = reinterpret_cast<float*>(s_warp + NW);             // [2][NW][T]
  uint32_t* const s_seen = reinterpret_cast<uint32_t*>(s_sums + 2 * NW * T);  // [NW][8]: tokens seen, of a warp's latest tiles

  const KvAttendArgs& a = P.w.attend;
  const KvView& kv = a.kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q4 = lane & 3, D = kv.head_dim;
  const int64_t ws = P.w.weights_stride;
  grid_dep_launch();
  grid_dep_wait();

  // ---- tiles before each run of sequences
  const int run = (a.n_seq + NT - 1) / NT;
  long long mine = 0;
#pragma unroll 1
  for (int k = 0; k < run && tid * run + k < a.n_seq; ++k) mine += seq_of<T, SCORED>(P, tid * run + k).tiles;
  long long incl = mine;
#pragma unroll
  for (int by = 1; by < 32; by *= 2) {
    const long long o = __shfl_up_sync(~0u, incl, by);
    if (lane >= by) incl += o;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  long long total = 0, before = incl - mine;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  s_before[tid] = before;

  // ---- tokens before the tiles (or of sequences without): nothing is added to what they have
  if (P.w.weights_out != P.w.weights || P.w.add != nullptr) {
    const int per_seq = max(1, (int)gridDim.x / a.n_seq), part = blockIdx.x % per_seq;
#pragma unroll 1
    for (int s = blockIdx.x / per_seq; s < a.n_seq; s += gridDim.x / per_seq) {
      const Seq q = seq_of<T, SCORED>(P, s);
      const uint32_t end = q.tiles == 0 ? q.len : q.first * T;
      const uint32_t fresh = P.w.add == nullptr ? 0u : (uint32_t)min(max(P.w.add[s], 0), (int)q.len);
      for (uint32_t t = part * NT + tid; t < end; t += per_seq * NT)
        P.w.weights_out[s * ws + t] = t >= q.len - fresh ? 0.f : P.w.weights[s * ws + t];
    }
  }
  __syncthreads();
  if (total == 0) return;

  // ---- this CTA's run of the list, and how many warps share a tile
  const long long from = total * blockIdx.x / gridDim.x, to = total * (blockIdx.x + 1) / gridDim.x;
  if (from == to) return;
  // Of a piece's tiles whole rounds go a tile a warp; warps that the rest would leave idle share its tiles, each share-th
  // head a warp
  auto share_of = [&](uint32_t rest) {
    int share = 1;
    while (NW % (2 * share) == 0 && 2 * share <= kv.n_heads && rest * 2 * share <= NW) share *= 2;
    return share;
  };

  auto first_piece = [&]() {
    int lo = 0;
#pragma unroll
    for (int step = NT / 2; step > 0; step /= 2)
      if (s_before[lo + step] <= from) lo += step;
    Piece p;
    p.s = lo * run;
    p.q = seq_of<T, SCORED>(P, p.s);
    long long off = from - s_before[lo];
    while (off >= (long long)p.q.tiles) {
      off -= p.q.tiles;
      p.q = seq_of<T, SCORED>(P, ++p.s);
    }
    p.tile0 = (uint32_t)off;
    p.at = from;
    p.count = (uint32_t)min(to - from, (long long)p.q.tiles - off);
    return p;
  };
  auto next_piece = [&](Piece& p) {  // false behind the last
    p.at += p.count;
    if (p.at >= to) return false;
    do p.q = seq_of<T, SCORED>(P, ++p.s);
    while (p.q.tiles == 0);
    p.tile0 = 0;
    p.count = (uint32_t)min(to - p.at, (long long)p.q.tiles);
    return true;
  };

  // ---- copies ahead: the next (tile, K/V head) of this warp
  constexpr int CPR = C::kRowBytes / 16, PER = 32 / CPR;
  constexpr int ES = F == IL_BF16 ? 2 : 1;
  const uint32_t ring = smem_u32(smem) + warp * C::kRing;
  Piece ahead = first_piece();
  uint32_t ahead_round = 0;  // first tile of the round
  int ahead_head = 0, ahead_share = 1;
  bool more = true;
  long long off = 0, soff = 0;  // of this lane's token of that tile
  uint32_t rows[C::kRowsOf];    // and, where all tokens are there, of the rows that this lane copies, in 16 bytes
  bool ok = false, all = false;
  uint32_t located = 0;  // tiles so far
  const int chunk = lane % CPR, sub = lane / CPR;
  const bool in_row = chunk * C::kChunk < D;
  auto locate = [&]() {  // this warp's tile of the round, or of the next that has one for it
    uint32_t tile;
    for (;; ahead_round += NW) {
      while (ahead_round >= ahead.count) {
        more = next_piece(ahead);
        if (!more) return;
        ahead_round = 0;
      }
      const uint32_t rest = ahead.count - ahead_round;
      ahead_share = rest >= NW ? 1 : share_of(rest);
      tile = ahead_round + warp / ahead_share;
      ahead_head = warp % ahead_share;
      if (tile < ahead.count) break;
    }
    const uint32_t t = (ahead.q.first + ahead.tile0 + tile) * T + (lane & (T - 1));
    const bool want = t >= ahead.q.begin && t < ahead.q.len;
    const uint32_t col = P.by_page.of(t);
    const uint32_t page = want ? (uint32_t)a.table[ahead.s * a.table_stride + col] : 0u;
    ok = want && page < (uint32_t)kv.n_pages;
    if (want && !ok) atomicOr(a.status, kStatusBadSlot);
    const uint32_t seen = __ballot_sync(~0u, ok), in_page = t - col * P.by_page.d;
    if (lane == 0) s_seen[warp * 8 + (located & 7)] = seen;
    ++located;
    all = P.whole && seen == ~0u;
    if (all) {
      const uint32_t o = page * P.page + in_page * P.token;
#pragma unroll
      for (int i = 0; i < C::kRowsOf; ++i) rows[i] = __shfl_sync(~0u, o, i * PER + sub);
      soff = page * P.spage + in_page * P.stoken;
    } else {
      off = ok ? (page * kv.page + in_page * kv.token) * ES : 0;
      soff = ok ? page * kv.spage + in_page * kv.stoken : 0;
    }
  };
  int stage_in = 0;
  auto fetch = [&]() {
    if (more) {
      const uint32_t to_smem = ring + stage_in * C::kStage, st = to_smem + C::kPool + lane * NB * 4;
      const uint8_t* const kb = kv.k + ((long long)ahead_head * kv.head * ES + chunk * 16);
      const float* const sc = kv.k_scale + (soff + (long long)ahead_head * kv.shead);
      if (all) {
#pragma unroll
        for (int i = 0; i < C::kRowsOf; ++i)
          cp16(to_smem + a4::chunk_at<CPR>(i * PER + sub, chunk), kb + (uint64_t)rows[i] * 16, in_row);
        if constexpr (F != IL_BF16) {
          constexpr int SB = NB == 2 ? 8 : 16;
#pragma unroll
          for (int i = 0; i < NB * 4 / SB; ++i) cp_small<SB>(st + i * SB, sc + i * (SB / 4), true);
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < C::kRowsOf; ++i) {
          const int row = i * PER + sub;
          const long long o = __shfl_sync(~0u, off, row);
          const bool use = __shfl_sync(~0u, (int)ok, row) && in_row;
          cp16(to_smem + a4::chunk_at<CPR>(row, chunk), use ? kb + o : kv.k, use);
        }
        if constexpr (F != IL_BF16) {
#pragma unroll 1
          for (int b = 0; b < NB; ++b) {
            const bool use = ok && 32 * b < D;
            cp_small<4>(st + 4 * b, use ? sc + b : kv.k_scale, use);
          }
        }
      }
      ahead_head += ahead_share;
      if (ahead_head >= kv.n_heads) {
        ahead_round += NW;
        locate();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    stage_in = stage_in + 1 == S ? 0 : stage_in + 1;
  };
  locate();
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch();

  // ---- the pieces
  int stage = 0, staged_s = -1, staged_h = -1, staged_c = -1, parity = 0;
  uint32_t used = 0;  // tiles of this warp so far
  Piece piece = first_piece();
  do {
    const int s = piece.s;
    const Seq q = piece.q;
    const int newest = !SCORED ? 0 : a.positions != nullptr ? a.positions[s * a.positions_stride + q.len - 1] : (int)q.len - 1;
    const uint32_t fresh = P.w.add == nullptr ? 0u : (uint32_t)min(max(P.w.add[s], 0), (int)q.len);
#pragma unroll 1
    for (uint32_t k0 = 0; k0 < piece.count; k0 += NW) {
      const int share = piece.count - k0 >= NW ? 1 : share_of(piece.count - k0), part = warp % share;
      const uint32_t tile_at = k0 + warp / share;
      const bool active = tile_at < piece.count;
      const uint32_t t0 = (q.first + piece.tile0 + tile_at) * T;
      float sums[NV], far[SCORED ? NV : 1], had = 0.f;
      bool use[NV];
      if (active) {
        __syncwarp();
        const uint32_t seen = s_seen[warp * 8 + (used++ & 7)], t = t0 + (lane & (T - 1));
        const bool there = (seen >> lane) & 1;
        if (part == 0 && t < q.len - fresh) had = P.w.weights[s * ws + t];
        int place = (int)t;
        if (SCORED && a.positions != nullptr && there) place = a.positions[s * a.positions_stride + t];
#pragma unroll
        for (int c = 0; c < NV; ++c) {
          sums[c] = 0.f;
          use[c] = (seen >> (8 * c + g)) & 1;
          if (SCORED) far[c] = (float)(__shfl_sync(~0u, place, 8 * c + g) - newest);
        }
      }
#pragma unroll 1
      for (int h0 = 0; h0 < kv.n_heads; h0 += P.hks) {
#pragma unroll 1
        for (int c0 = 0; c0 < P.blocks; c0 += P.cols) {
          const int h1 = min(h0 + P.hks, kv.n_heads), c1 = min(c0 + P.cols, P.blocks), cols = c1 - c0;
          if (staged_s != s || staged_h != h0 || staged_c != c0) {
            __syncthreads();
            // q as fragments, a warp four heads at a time
#pragma unroll 1
            for (int four = warp; four < (h1 - h0) * cols; four += NW) {
              const int hk = h0 + four / cols, block = c0 + four % cols, in_group = 4 * block + g / 2;
              const float* const src = a.q + s * a.q_stride + ((int64_t)hk * P.group + in_group) * D;
              const int mine = 4 * block + q4;  // the head of this lane's logits; p = 0 beyond the last
              const int64_t at = (int64_t)hk * P.group + mine;
              const bool exists = mine < P.group;
              const float lse = exists ? a.lse[(int64_t)s * a.n_q_heads + at] * 1.4426950408889634f : INFINITY;
              const float slope = SCORED && a.slopes != nullptr && exists ? a.slopes[at] * 1.4426950408889634f : 0.f;
              Q h;
              // (rows of q are 16-byte aligned, and D a multiple of 8)
              h.take(
                  [&](int e, auto& x) {
                    constexpr int N = sizeof(x) / 4;
                    using Vec = typename std::conditional<N == 4, float4, float2>::type;
                    Vec v = {};
                    if (in_group < P.group && e < D) v = *reinterpret_cast<const Vec*>(src + e);
                    const float* const f = reinterpret_cast<const float*>(&v);
#pragma unroll
                    for (int k = 0; k < N; ++k) x[k] = f[k] * P.q_scale;
                  },
                  lane);
              uint4* const to_mem = heads_mem + four * (C::kFours * 32) + lane;
              auto word = [&](int i) {
                return i < Q::kWords        ? h.word(i)
                       : i == Q::kWords     ? __float_as_uint(lse)
                       : i == Q::kWords + 1 ? __float_as_uint(slope)
                                            : 0u;
              };
#pragma unroll
              for (int i = 0; i < C::kFours; ++i)
                to_mem[i * 32] = make_uint4(word(4 * i), word(4 * i + 1), word(4 * i + 2), word(4 * i + 3));
            }
            __syncthreads();
            staged_s = s, staged_h = h0, staged_c = c0;
          }
          if (!active) continue;
#pragma unroll 1
          for (int hk = h0 + ((part - h0) & (share - 1)); hk < h1; hk += share) {
            if (c0 == 0) {
              asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
              __syncwarp();
              fetch();
            }
            const uint32_t tile = ring + stage * C::kStage;
            const uint4* from_mem = heads_mem + (hk - h0) * cols * (C::kFours * 32) + lane;
#pragma unroll 1
            for (int block = c0; block < c1; ++block, from_mem += C::kFours * 32) {
              Q h;
              float lse = 0.f, slope = 0.f;
#pragma unroll
              for (int i = 0; i < C::kFours; ++i) {
                const uint4 v = from_mem[i * 32];
                const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  if (4 * i + j < Q::kWords) h.word(4 * i + j) = word[j];
                  if (4 * i + j == Q::kWords) lse = __uint_as_float(word[j]);
                  if (4 * i + j == Q::kWords + 1) slope = __uint_as_float(word[j]);
                }
              }
#pragma unroll
              for (int k = 0; k < T / 16; ++k) {
                float v[2];
                h.dot(v, tile, tile + C::kPool, 16 * k, lane);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  float x = v[c];
                  if constexpr (SCORED) {
                    if (P.cap_log2 > 0.f) x = P.cap_log2 * tanhf(x);
                    x = fmaf(slope, far[2 * k + c], x);
                  }
                  float p;
                  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(x - lse));
                  sums[2 * k + c] += use[2 * k + c] ? p : 0.f;
                }
              }
            }
            if (c1 == P.blocks) stage = stage + 1 == S ? 0 : stage + 1;
          }
        }
      }
      // ---- over the four lanes of a token, then over the warps of a tile
      float* const shared = s_sums + (parity * NW + warp) * T;
      if (active) {
#pragma unroll
        for (int c = 0; c < NV; ++c) {
          sums[c] += __shfl_xor_sync(~0u, sums[c], 1);
          sums[c] += __shfl_xor_sync(~0u, sums[c], 2);
          if (q4 == 0) shared[8 * c + g] = sums[c];
        }
      }
      if (share > 1)
        __syncthreads();
      else
        __syncwarp();
      if (active && part == 0 && lane < T) {
        float sum = 0.f;
        for (int w = 0; w < share; ++w) sum += shared[w * T + lane];
        const uint32_t t = t0 + lane;
        if (t < q.len) P.w.weights_out[s * ws + t] = had + (t >= q.begin ? sum : 0.f);
      }
      parity ^= 1;
    }
  } while (next_piece(piece));
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int F, bool SCORED, int W>
cudaError_t prepare(const Plan& p, int num_sms, Launch* out) {
  using C = Config<F, W>;
  const void* const fn = reinterpret_cast<const void*>(kv_weigh_kernel<F, SCORED, W>);
  // whole K/V heads where their blocks fit
  Plan plan = p;
  plan.cols = std::min(p.blocks, C::kBatch);
  plan.hks = plan.cols < p.blocks ? 1 : std::min(p.w.attend.kv.n_heads, C::kBatch / p.blocks);
  const size_t smem = (size_t)C::kFixed + C::kWarps * C::kRing + (size_t)plan.hks * plan.cols * C::kHeads;
  static std::atomic<unsigned long long> attr_set{0};  // one bit per device (setting it twice is harmless)
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !(attr_set.load() & (1ull << dev))) {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set.fetch_or(1ull << dev);
  }
  out->fn = fn;
  out->grid = dim3((unsigned)num_sms);
  out->block = dim3(C::kThreads);
  out->smem = smem;
  if (!out->set_args(plan)) return cudaErrorMemoryAllocation;
  if (kUsePdl) out->allow_early_start();
  return cudaSuccess;
}

template <int F>
cudaError_t prepare_format(const Plan& p, int num_sms, Launch* out) {
  const int dim = p.w.attend.kv.head_dim;
  const auto of = [&](auto scored) {
    constexpr bool SCORED = decltype(scored)::value;
    return dim <= 64    ? prepare<F, SCORED, 64>(p, num_sms, out)
           : dim <= 128 ? prepare<F, SCORED, 128>(p, num_sms, out)
                        : prepare<F, SCORED, 256>(p, num_sms, out);
  };
  return p.w.attend.scored ? of(std::true_type{}) : of(std::false_type{});
}

}  // namespace weigh

cudaError_t prepare_kv_weigh(const KvWeighArgs& w, int num_sms, Launch* out) {
  const KvAttendArgs& a = w.attend;
  const KvView& kv = a.kv;
  weigh::Plan p{};
  p.w = w;
  p.cap = (int)std::min<int64_t>({a.table_width * kv.page_size, w.weights_width,
                                  a.positions != nullptr ? a.positions_width : INT32_MAX});
  p.window = (int)std::min<int64_t>(a.window, INT32_MAX);
  p.by_page = FastDiv((uint32_t)kv.page_size);
  p.group = a.n_q_heads / kv.n_heads;
  p.blocks = (p.group + 3) / 4;
  p.q_scale = a.cap > 0.f ? a.scale / a.cap : a.scale * 1.4426950408889634f;
  p.cap_log2 = a.cap * 1.4426950408889634f;
  const int dim = kv.head_dim <= 64 ? 64 : kv.head_dim <= 128 ? 128 : 256, unit = dim == 64 ? 2 : 4;
  const int64_t es = kv.format == IL_BF16 ? 2 : 1;
  const auto ends = [&](int64_t page, int64_t token) { return (kv.n_pages - 1) * page + (kv.page_size - 1) * token <= UINT32_MAX; };
  p.whole = ends(kv.page * es / 16, kv.token * es / 16);
  if (kv.format != IL_BF16 && p.whole)
    p.whole = kv.head_dim == dim && reinterpret_cast<uintptr_t>(kv.k_scale) % (4 * unit) == 0 && kv.spage % unit == 0 &&
              kv.stoken % unit == 0 && kv.shead % unit == 0 && ends(kv.spage, kv.stoken);
  p.page = (uint32_t)(kv.page * es / 16), p.token = (uint32_t)(kv.token * es / 16);
  p.spage = (uint32_t)kv.spage, p.stoken = (uint32_t)kv.stoken;
  return kv.format == IL_BF16 ? weigh::prepare_format<IL_BF16>(p, num_sms, out)
         : kv.format == IL_Q8 ? weigh::prepare_format<IL_Q8>(p, num_sms, out)
                              : weigh::prepare_format<IL_A4>(p, num_sms, out);
}

}  // namespace il
