// kv_attend.cuh -- attention of one new token per sequence over the paged cache (il_kv_attend, il_kv_attend_scored):
// the kernel, instantiated per cache format, plain and scored, in the six kv_attend_*.cu.
//
// For every sequence and K/V head, with G query heads reading that head:
//   s = scale q K^T, p = exp(s - max), out = p V / sum p        ([G][len] by [len][D])
// Each K and V byte is used G times, so the kernel is bound by HBM: it has to keep copies in
// flight on every SM for the whole launch, whatever the lengths, and do the arithmetic beside them.
//
// Work.  The tokens of a (sequence, K/V head) pair -- a row -- are cut into tiles of 16 or 32.  All tiles of all
// rows form one list, and every warp of the launch (one CTA per SM) takes an equal contiguous
// run of it, found from the prefix sums of the lengths that each CTA computes itself: ragged batches, long
// sequences and idle slots balance to one tile a warp without any host knowledge of the lengths.
// A row inside a warp's run is finished by the warp alone.  The ends of runs are parts of rows;
// they are joined in shared memory by the CTA (one barrier, after its stream), and rows that cross CTAs
// through the workspace by the last CTA of the row to arrive, in CTA order: the result does
// not depend on the order of arrival.
//
// Stream.  Every warp owns a ring of stages, one tile of K and V each, filled with 16-byte
// cp.async (any strides, any page size: a lane looks up its token's page one tile ahead) and zeros for
// tokens outside the attended range.  Where pages hold whole groups of 16 tokens their addresses are one base and
// constants of the lane (heads in columns: any pages, offsets of 32 bits that the lanes hand to one another).  No barrier
// other than the warp's own sits in the stream.  A head of more than 128 elements takes a pair of warps, half of its columns
// each: they trade their halves of s through shared memory, with a barrier of the two.
//
// Arithmetic.  Query heads are the rows of m16n8k16 MMAs and tokens (then elements of V) the
// columns; a softmax row lives in the four lanes of a quad.  q and p are fp32 and are split
// exactly enough to keep fp32's accuracy: against bf16 K and V into three bf16 parts (hi + mid + lo,
// 24 bits); against int8 into two fp16 parts (22 bits), with K's and V's integers decoded to exact
// fp16, K's block scales applied to each block's fp32 sum and V's to p, under a running power of two.
// With up to 8 heads (R = 1) q's hi fills rows 0-7 of an MMA and mid (int8: lo) rows 8-15, so the
// split costs one more MMA at bf16 and none at int8; with 9 to 16 heads (R = 2) every part is an MMA
// of its own.  p V is computed transposed: the quad layout of s is that of a B operand, so p goes in as it is.
// Each tile's product starts from zero accumulators and joins the running sum in fp32
// FMAs (with the factor of the running maximum), which round to nearest.  A4, and Q8 where it is scored, have the operands
// the other way round, query heads in the columns (kv_a4.cuh), which takes fewer instructions: 875 of A4 for 32 tokens of 128
// columns, the loop and copies included.
//
// Scored (il_kv_attend_scored): logits are capped and biased between the two products, and a row may begin at a later token.
// The plain kernels have none of it.
//
// Measured (GB300, 32 query heads on 8 K/V heads of 128, device time): bf16, 128 sequences of 4096 tokens 315 us, 6.8 TB/s
// (the rate of a plain copy); 32 of 0 to 8192 86 us, 6.0 TB/s; one of 512 8.1 us.  Q8, 64 of 1 to 8192 106 us, 5.6 TB/s,
// one of 131071 59 us, 5.2 TB/s.  What bounds it: HBM at bf16 (64 sequences of 8192: 317 us, 263 us with pages that stay in
// L2); at Q8 no unit (207 us either way; issue slots
// 50 % used, ALU 44 %, tensor pipe 27 %, DRAM 65 %) but the chain of a tile in a warp -- q K^T, maximum, exp2, split, p V -- at
// two warps a scheduler, about 520 instructions per 16 tokens; A4, 64 of 1 to 8192 (another draw, 316,517 tokens) 94 us, 4.3 TB/s, one of
// 131071 45 us, one of 512 9.0 us: the same chain at three warps a scheduler, which use 64 % of the issue slots (ALU 54 %, tensor
// pipe 20 %, DRAM 53 %); at HBM's rate a tile would have 848 slots for its 875 instructions.  With two blocks of 4 heads A4 has two warps a
// scheduler and twice the splits and products: 8 heads on one of 256, 64 of 8192, 79 us (Q8 66), 64 on 8 of 128, 64 of 4096, 123 us
// (Q8 110).  Of a short call the latencies before the first tile and in the joins.  Scored: bf16, 16 of 1000 to 16384 under a window of 4096, 16 heads of 256 on 8, 83 us, 5.7 TB/s; Q8, 32 of up to
// 4096, 32 heads on 32, 56 us, 4.1 TB/s.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "il_internal.cuh"
#include "il_ptx.cuh"
#include "kv_a4.cuh"

namespace il {

// What the host adds to KvAttendArgs for the kernel.
struct KvAttendPlan {
  KvAttendArgs a;
  int cap;                // longest length: table_width * page_size, at most 2^31 - 1
  int window;             // 0: all
  FastDiv by_page;        // t / page_size
  FastDiv by_blocks;      // row of a sequence / blocks
  int group;              // query heads of a K/V head
  int blocks;             // blocks of 8 R query heads of a K/V head
  float q_scale;          // scale * log2(e), or scale / cap
  float cap_log2;         // cap * log2(e); 0: none
  int simple;             // pages hold whole groups, the strides below fit, (Q8) scales allow the widest copies
  uint32_t page_bytes, token_bytes, head_bytes;     // strides of k and v (A4: in 16 bytes)
  uint32_t spage_bytes, stoken_bytes, shead_bytes;  // of the scales (A4: in pairs)
  unsigned* arrived;      // one counter a CTA, zero before and after
  float* parts;           // two parts a CTA
};

namespace attend {

constexpr int kGroup = 16;          // tokens of a product's step; pages of whole groups are copied the simple way
constexpr int kSmemLimit = 232448;  // 227 KB
constexpr int kMaxCtas = 256;       // of a grid, one an SM
constexpr int kQ8Columns = 16 + IL_Q8;  // IL_Q8 with query heads in the MMAs' columns, as A4 has them

// F: format of the cache, or kQ8Columns.  W columns of a head in a warp, H warps a head (H * W >= head_dim), R blocks of 8
// (heads in columns: of 4) query heads.
template <int F, int W, int R, int H>
struct Config {
  static constexpr bool kA4 = F == IL_A4, kQ8 = F == IL_Q8, kCols = kA4 || F == kQ8Columns;
  static constexpr int kRows = (kCols ? 4 : 8) * R;  // query heads of a block
  static constexpr int kBlocks = W / 32;           // 32-element blocks of a warp's columns
  static constexpr int kPart = kRows * (W + 2);    // floats of a part: sums, maxima, sums of p
  // Tokens of a tile: 32 where a row is short in bytes, so that what a tile costs beside its bytes counts half
  static constexpr int kTile = kCols || (R == 1 && (kQ8 || W == 64)) ? 32 : 16;
  static constexpr int kValues = kTile / (kCols ? 8 : 4);  // of s, of a softmax row in a lane
  static constexpr int kRowBytes = kA4 ? W / 2 : F == IL_BF16 ? 2 * W : W;
  static constexpr int kChunk = 16 * W / kRowBytes;                    // elements of 16 bytes
  static constexpr int kPool = kTile * kRowBytes;                      // K or V of a tile
  static constexpr int kScales = F != IL_BF16 ? kTile * kBlocks * 4 : 0;  // its scales
  static constexpr int kStage = 2 * (kPool + kScales);
  // (A4, measured with 8, 12 and 16 warps, 64 ragged sequences as the kernel was then: heads of 128 116, 102, 137 us, of 64
  // 133, 112, 97 us)
  static constexpr int kWarps = kA4 ? (R == 2 ? (W == 64 ? 12 : 8) : W == 64 ? 16 : 12) : F != IL_BF16 && R == 1 && W == 64 ? 12 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kWorkers = kWarps / H;    // runs of tiles in a CTA
  static constexpr uint32_t kWhole = 2 * kWorkers;  // tiles of a row that is not cut over CTAs
  static constexpr int kFixed = kThreads * 8 + kWorkers * 48 + 32;
  // Two stages, one on its way while the other is used, are 70 KB in flight an SM.  More cost DRAM efficiency: with
  // three, 128 x 4096 tokens bf16 took 332 us instead of 317, heads of 64 92.3 instead of 89.5 (Q8 70.7, 69.1).
  static constexpr int kStages = kA4 && W == 64 ? 4 : 2;
  static constexpr int kRing = kStages * kStage;
  static constexpr size_t kSmem = (size_t)kFixed + kWarps * (kPart * 4 + kRing);
  static_assert(kStages >= 2 && kSmem <= kSmemLimit, "the ring does not fit");
  static_assert(kRing >= kPart * 4, "a part must fit the warp's ring");
  static_assert(kWorkers * 48 >= kWarps * 8, "the sums over sequences are kept where the workers' parts are described");
  static_assert(H == 1 || kPool >= 128 * kValues * R, "s is traded through the tile of K");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool use, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(use ? 16 : 0),
               "l"(policy)
               : "memory");
}
// The same without a policy, which costs two instructions a copy.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool use) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(use ? 16 : 0) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void cp_small(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void cp_small(uint32_t dst, const void* src, bool use, uint64_t policy) {
  if constexpr (BYTES == 16)
    cp16(dst, src, use, policy);
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(use ? BYTES : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

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
template <int N>  // N = 2 or 4 floats
__device__ __forceinline__ void lds_floats(float (&f)[N], uint32_t at) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]) : "r"(at));
  else
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(f[0]), "=f"(f[1]) : "r"(at));
}
__device__ __forceinline__ void sts128(uint32_t at, const float (&f)[4]) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}

// Four floats of a part in the workspace, past this SM's L1 (other SMs write it), or zeros: a load without a
// branch, so that several are on their way at once.
__device__ __forceinline__ float4 load_part4(const float* p, bool use) {
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  asm volatile(
      "{\n.reg .pred use;\nsetp.ne.b32 use, %5, 0;\n@use ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];\n}\n"
      : "+f"(x.x), "+f"(x.y), "+f"(x.z), "+f"(x.w)
      : "l"(p), "r"((int)use)
      : "memory");
  return x;
}

// c = A B, or c += A B.  The first has its zeros in the instruction, not in registers set to 0.
#define IL_MMA(TYPE, C0, C1, C2, C3) \
  "mma.sync.aligned.m16n8k16.row.col.f32." TYPE "." TYPE ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {" C0 "," C1 "," C2 "," C3 "};"
template <bool F16>
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  if constexpr (F16)
    asm(IL_MMA("f16", "%10", "%10", "%10", "%10")
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm(IL_MMA("bf16", "%10", "%10", "%10", "%10")
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// d = c + A B (fp16)
__device__ __forceinline__ void mma_from(float (&d)[4], float c0, float c1, float c2, float c3, uint32_t a0, uint32_t a1,
                                         uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(IL_MMA("f16", "%10", "%11", "%12", "%13")
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (F16)
    asm(IL_MMA("f16", "%0", "%1", "%2", "%3")
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm(IL_MMA("bf16", "%0", "%1", "%2", "%3")
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
#undef IL_MMA

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float pow2_biased(int e) { return __int_as_float(e << 23); }  // 2^(e - 127), 0 < e < 255

// K's bytes u = q + 128 (0 .. 255) as fp16: the bit pattern 00uu is u 2^-24, a subnormal, exactly.  The products
// with the 128 are taken off by where the sums start.  (V's become exact q: a sum over tokens may
// meet nothing but small q, which 128 times the sum of p would drown.)
__device__ __forceinline__ void bytes_to_f16x2(uint32_t w, uint32_t& p01, uint32_t& p23) {
  const uint32_t u = w ^ 0x80808080u;
  p01 = __byte_perm(u, 0u, 0x4140);
  p23 = __byte_perm(u, 0u, 0x4342);
}

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
  int hk, block;  // K/V head, block of its query heads
  uint32_t tile;  // of the row
  Seq q;
};

// a / b, the quotient of 64 bits only where it has to be: that one takes 0.3 us at the start of a launch.
static __device__ __noinline__ unsigned long long divide_wide(unsigned long long a, uint32_t b) { return a / b; }
__device__ __forceinline__ unsigned long long divide(unsigned long long a, uint32_t b) {
  return a >> 32 == 0 ? (unsigned long long)((uint32_t)a / b) : divide_wide(a, b);
}

template <int T, bool SCORED, int LEAD>
__device__ __forceinline__ Seq seq_of(const KvAttendPlan& P, int s) {
  Seq q;
  const int len = min(max(P.a.lens[s], 0), P.cap);
  q.len = (uint32_t)len;
  q.begin = P.window > 0 ? (uint32_t)max(len - P.window, 0) : 0u;
  if (SCORED && P.a.starts != nullptr) q.begin = max(q.begin, (uint32_t)min(max(P.a.starts[s], 0), len));
  q.first = q.begin / T;
  q.tiles = len == 0 || (SCORED && q.begin == q.len) ? 0u : (q.len + T - 1) / T - q.first + LEAD;
  return q;
}

template <int T, bool SCORED, int LEAD>
__device__ __forceinline__ void advance(Walk& w, const KvAttendPlan& P) {
  if (++w.tile < w.q.tiles) return;
  w.tile = 0;
  if (++w.block < P.blocks) return;
  w.block = 0;
  if (++w.hk < P.a.kv.n_heads) return;
  w.hk = 0;
  do w.q = seq_of<T, SCORED, LEAD>(P, ++w.s);
  while (w.q.tiles == 0 && w.s + 1 < P.a.n_seq);
}

// What a worker leaves for the CTA: part 0, the end (or all) of a row begun before its run, and
// part 1, the beginning of a row that goes on behind it.
struct Left {
  int s0, hk0, block0;
  int s1, hk1, block1;
  uint32_t tiles0, tiles1;
  long long row0, row1;  // first tiles of the rows in the list
};
static_assert(sizeof(Left) == 48, "see Config::kFixed");

template <int F, bool SCORED, int W, int R, int H>
__global__ void __launch_bounds__(Config<F, W, R, H>::kThreads, 1) kv_attend_kernel(const KvAttendPlan P) {
  using C = Config<F, W, R, H>;
  constexpr bool Q8 = C::kQ8, A4 = C::kA4, COLS = C::kCols, BLOCKED = F != IL_BF16;  // scales of 32 elements
  constexpr int NV = C::kValues;
  // Empty tiles before each row's, for what its start and end cost beside its tiles (q, parts, result).  One: 1024 biased Q8
  // rows of 1 to 108 tiles, from the oldest on, 78.9 -> 60.5 us (two 61.5, four 65.3), 64 ragged A4 sequences 94.0 -> 93.4, 256 of 50 to 150
  // tokens 20.8 -> 19.9.  Not where rows of few bytes or pairs of warps lose: A4 heads of 64 90.3 -> 94.4, capped heads of
  // 256 83.0 -> 84.0.  (A pair of warps meets at every tile's barrier: none of its tiles may be empty.)
  constexpr int LEAD = H == 1 && (SCORED || (A4 && W == 128)) ? 1 : 0;
  // Rows from the newest tile back: a steep bias then leaves tiles that weigh nothing beside the newest, whose V is not used,
  // and few whose p lie far apart.  (The first CTAs took 42 us and those of the steep heads 55.)  32 heads on 32, 32 sequences
  // of up to 4096 tokens: Q8 with document starts, 25,000 tokens seen, 60.6 -> 56.2 us, A4 without, 59,000 seen, 119 -> 102; 32 on 8,
  // 64 of up to 8192: Q8 143 -> 134, A4 140 -> 135; capped
  // without a bias Q8 119.7 -> 122.6, A4 104.5 -> 103.5.  Rows of bf16 are bound by HBM either way.
  constexpr bool BACK = SCORED && COLS;
  constexpr int T = C::kTile, NN = T / 8, GR = T / kGroup;  // tokens of a tile, in eights, in groups
  constexpr int NB = C::kBlocks, NT = C::kThreads, NW = C::kWarps, NK = C::kWorkers, S = C::kStages, ROWS = C::kRows;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* const ring_mem = smem;
  float* const part_mem = reinterpret_cast<float*>(smem + (size_t)NW * C::kRing);
  long long* const s_before = reinterpret_cast<long long*>(reinterpret_cast<uint8_t*>(part_mem) + NW * C::kPart * 4);
  Left* const s_left = reinterpret_cast<Left*>(s_before + NT);
  long long* const s_warp = reinterpret_cast<long long*>(s_left);  // at the start, of the sums over sequences
  int* const s_flag = reinterpret_cast<int*>(s_left + NK);  // of the two rows that may cross CTAs: parts to join, first CTA
  unsigned* const s_mask = reinterpret_cast<unsigned*>(s_flag + 4);  // workers with a part 0, whose row ends in it, with a part 1

  const KvAttendArgs& a = P.a;
  const KvView& kv = a.kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q4 = lane & 3;
  const int worker = warp / H, col0 = H == 1 ? 0 : (warp % H) * W;  // first column of this warp
  const int rows_per_seq = kv.n_heads * P.blocks, D = kv.head_dim;
  grid_dep_launch();
  {
    // the table and q into L2 while the launch before this one drains (both are read soon after the wait;
    // whatever that launch still writes to them goes to the same L2 lines)
    const int64_t at = ((int64_t)blockIdx.x * NT + tid) * 32, step = (int64_t)gridDim.x * NT * 32;
    const int64_t tn = (int64_t)(a.n_seq - 1) * a.table_stride + a.table_width;
    if (at < tn) prefetch_l2(a.table + at);
    const int64_t qn = (int64_t)(a.n_seq - 1) * a.q_stride + (int64_t)a.n_q_heads * D;
#pragma unroll 1
    for (int64_t i = at; i < min(qn, 4 * step); i += step) prefetch_l2(a.q + i);
  }
  grid_dep_wait();

  // ---- tiles before each run of sequences; sequences without tokens get their zeros
  const int run = (a.n_seq + NT - 1) / NT;
  long long mine = 0;
  bool short_rows = false;
#pragma unroll 1
  for (int k = 0; k < run; ++k) {
    const int s = tid * run + k;
    const bool in = s < a.n_seq;
    const Seq q = in ? seq_of<T, SCORED, LEAD>(P, s) : Seq{0, 0, 0, 0};
    mine += q.tiles;
    short_rows |= q.tiles - 1 < C::kWhole;
    unsigned none = __ballot_sync(~0u, in && q.tiles == 0 && s % gridDim.x == blockIdx.x);
    while (none != 0) {
      const int src = __ffs(none) - 1;
      none &= none - 1;
      const int64_t z = __shfl_sync(~0u, s, src);
#pragma unroll 1
      for (int i = lane; i < a.n_q_heads * D / 4; i += 32)
        reinterpret_cast<float4*>(a.out + z * a.out_stride)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (a.lse != nullptr)
#pragma unroll 1
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
  if (tid < 3) s_mask[tid] = 0;
  __syncthreads();
  long long total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const long long t = s_warp[w];
    if (w < warp) before += t;
    total += t;
  }
  s_before[tid] = before + incl - mine;
  short_rows = __syncthreads_or(short_rows);

  // ---- this CTA's range of the list, and this worker's run of it.  Ranges are equal but for one tile, except that
  // a boundary inside a short row (up to kWhole tiles) moves to the row's nearer end: at most two more tiles for a worker
  // (1 us each where they do not overlap) against a join across CTAs (3 us after the last tile); 64 sequences of
  // 100 to 200 tokens 18.1 -> 15.2 us, 256 of 50 to 100 25.7 -> 21.8 us.
  const long long units = total * rows_per_seq;
  const int ctas = (int)min((long long)gridDim.x, (units + NK - 1) / NK);
  if ((int)blockIdx.x >= ctas) return;
  const long long share = (long long)divide(units, ctas);
  const int more = (int)(units - share * ctas);
  auto begin_of = [&](int cta) { return cta * share + min(cta, more); };  // before boundaries move
  Walk in;                                                                 // next tile to be fetched
  long long from = begin_of(blockIdx.x), to = begin_of(blockIdx.x + 1);  // the CTA's tiles
  long long u0 = lane < 16 ? from : to;                                  // first its boundaries, one in each half of the warp
  int n = 0;                                                             // tiles of this worker
#pragma unroll 1
  for (int pass = short_rows ? 0 : 1; pass < 2; ++pass) {
    if (pass == 1) {  // then the worker's first tile
      const uint32_t all = (uint32_t)(to - from);  // 2^32 tiles would be 10^5 GB of cache
      const int per = all / NK, extra = all % NK;
      n = per + (worker < extra);
      u0 = from + (long long)worker * per + min(worker, extra);
      if (n == 0) break;
    }
    // the place of tile u0 (of the last one for u0 = units): the last run of sequences with no more tiles before it, by
    // counting in each half of the warp
    const long long target = min(u0, units - 1), tiles_before = (long long)divide(target, rows_per_seq);
    int runs = 0;
#pragma unroll
    for (int k = 0; k < NT / 16; ++k) runs += s_before[k * 16 + (lane & 15)] <= tiles_before;
#pragma unroll
    for (int by = 8; by > 0; by /= 2) runs += __shfl_xor_sync(~0u, runs, by);
    const int lo = runs - 1;
    long long off = target - s_before[lo] * rows_per_seq;
    in.s = lo * run;
    in.q = seq_of<T, SCORED, LEAD>(P, in.s);
    while (off >= (long long)in.q.tiles * rows_per_seq && in.s + 1 < a.n_seq) {
      off -= (long long)in.q.tiles * rows_per_seq;
      in.q = seq_of<T, SCORED, LEAD>(P, ++in.s);
    }
    const int row = (int)divide(off, in.q.tiles);
    in.tile = (uint32_t)(off - (long long)row * in.q.tiles);
    in.hk = (int)P.by_blocks.of(row);
    in.block = row - in.hk * P.blocks;
    if (pass == 0) {
      if (u0 < units && in.q.tiles <= C::kWhole) u0 += 2 * in.tile < in.q.tiles ? -(int)in.tile : (int)(in.q.tiles - in.tile);
      from = __shfl_sync(~0u, u0, 0);
      to = __shfl_sync(~0u, u0, 16);
    }
  }

  Left left;
  bool has0 = false, end0 = false, has1 = false;  // part 0, its row's end in it, part 1
  if (n > 0) {
    Walk at = in;  // tile being used
    const uint32_t ring = smem_u32(ring_mem) + warp * C::kRing;
    // K and V pass once, so that they need not push the rest (code, table, parts) out of L2: about 1 % of a long call.
    // Where several blocks of query heads read them they are ordinary lines.
    uint64_t policy = policy_evict_first();
    if (P.blocks > 1) asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));

    // 16-byte chunks of a row, rows of one copy instruction, this lane's chunk
    constexpr int ES = BLOCKED ? 1 : 2, CPR = C::kRowBytes / 16, PER = 32 / CPR;  // ES: bytes of what strides count
    const int chunk = lane % CPR, sub = lane / CPR;
    const bool in_row = col0 + chunk * C::kChunk < D;
    const int col_bytes = A4 ? col0 / 2 : col0 * ES;
    const uint32_t lane_off = sub * P.token_bytes + col_bytes + chunk * 16, row_step = PER * P.token_bytes;
    // scales: the widest copy of a token's scales; a lane copies K's (lanes 0-15) or V's
    constexpr int SB = NB * 4 > 16 ? 16 : NB * 4;

    auto token_of = [&](const Walk& w) {
      return (w.q.first + (BACK ? w.q.tiles - 1 - w.tile : w.tile - LEAD)) * T + (lane & (T - 1));
    };
    auto empty = [&](const Walk& w) { return LEAD > 0 && w.tile < LEAD; };
    auto column_of = [&](uint32_t t) { return P.by_page.of(t); };
    // Heads in columns: of the tile to be copied next, this lane's token's place in its page (units of `fetch` below),
    // and which tokens are wanted
    uint32_t in_page_off = 0, in_page_soff = 0, wanted = 0;
    auto page_of = [&](const Walk& w) {  // page of this lane's token of the tile (of 16 tokens, lanes 16-31 repeat 0-15)
      const uint32_t t = token_of(w);
      if (empty(w)) return -1;
      if constexpr (COLS) {
        const bool want = t >= w.q.begin && t < w.q.len;
        const uint32_t col = column_of(t), in_page = t - col * (uint32_t)kv.page_size;
        in_page_off = in_page * P.token_bytes + w.hk * P.head_bytes;
        in_page_soff = in_page * P.stoken_bytes + w.hk * P.shead_bytes;
        wanted = __ballot_sync(~0u, want);
        return want ? a.table[(int64_t)w.s * (int)a.table_stride + col] : -1;
      }
      return t >= w.q.begin && t < w.q.len ? a.table[w.s * a.table_stride + column_of(t)] : -1;
    };
    // Positions of the chunks of a row in shared memory, without bank conflicts in the reads below.
    auto k_at = [&](int row) {
      if (COLS) return (int)a4::chunk_at<CPR>(row, chunk);
      return row * C::kRowBytes +
             ((Q8 ? chunk ^ ((W == 64 ? (row >> 1) & 1 : row & 3) << 1) : chunk ^ ((row & 1) << 2)) << 4);
    };
    auto v_at = [&](int row) {
      if (COLS) return (int)a4::chunk_at<CPR>(row, chunk);
      if (!Q8) return row * C::kRowBytes + ((chunk ^ (row & 7)) << 4);
      if (W == 64) row = (row & ~15) | ((row >> 1) & 7) | ((row & 1) << 3);
      return row * C::kRowBytes + ((chunk ^ (((row >> 1) & (W == 64 ? 1 : 3)) << 1)) << 4);
    };
    // Copies the tile at `w`; gives the mask of its tokens that exist.
    auto fetch = [&](const Walk& w, int page, int stage) -> uint32_t {
      if (empty(w)) return 0u;
      if constexpr (COLS) {
        const uint32_t to = ring + stage * C::kStage;
        if (P.simple && wanted == ~0u && __all_sync(~0u, (uint32_t)page < (uint32_t)kv.n_pages)) {
          // offsets in units of 16 bytes (and of a pair of steps): 32 bits, computed for one token a lane
          const uint32_t off = (uint32_t)page * P.page_bytes + in_page_off, soff = (uint32_t)page * P.spage_bytes + in_page_soff;
          const uint8_t *const kb = kv.k + (col_bytes + chunk * 16), *const vb = kv.v + (col_bytes + chunk * 16);
          const uint32_t first = to + a4::chunk_at<CPR>(sub, chunk);
#pragma unroll
          for (int i = 0; i < T / PER; ++i) {
            const uint64_t o = (uint64_t)__shfl_sync(~0u, off, i * PER + sub) * 16;
            // A4: rows PER further lie as far apart, whatever the chunk
            const uint32_t at = A4 ? first + i * 512 : to + a4::chunk_at<CPR>(i * PER + sub, chunk);
            cp16(at, kb + o, in_row);
            cp16(at + C::kPool, vb + o, in_row);
          }
          const uint32_t st = to + 2 * C::kPool + lane * NB * 4;
#pragma unroll
          for (int i = 0; i < NB * 4 / SB; ++i) {
            cp_small<SB>(st + i * SB, reinterpret_cast<const uint8_t*>(kv.k_scale + soff) + col0 / 8 + i * SB);
            cp_small<SB>(st + C::kScales + i * SB, reinterpret_cast<const uint8_t*>(kv.v_scale + soff) + col0 / 8 + i * SB);
          }
          return ~0u;
        }
      }
      const uint32_t t = token_of(w), t0 = t - (lane & (T - 1));
      const uint32_t to = ring + stage * C::kStage;
      const bool want = t >= w.q.begin && t < w.q.len, ok = want && (uint32_t)page < (uint32_t)kv.n_pages;
      const uint32_t mask = __ballot_sync(~0u, ok) & (uint32_t)((1ull << T) - 1);
      if (!COLS && P.simple && mask == (uint32_t)((1ull << T) - 1)) {
#pragma unroll
        for (int k = 0; k < GR; ++k) {
          const uint32_t first = t0 + k * kGroup, pg = GR == 1 ? (uint32_t)page : (uint32_t)__shfl_sync(~0u, page, k * kGroup);
          const uint32_t in_page = first - column_of(first) * (uint32_t)kv.page_size;
          const uint64_t off = (uint64_t)pg * P.page_bytes + (in_page * P.token_bytes + w.hk * P.head_bytes + lane_off);
          const uint8_t *kp = kv.k + off, *vp = kv.v + off;
#pragma unroll
          for (int i = 0; i < kGroup / PER; ++i) {
            const int row = k * kGroup + i * PER + sub;
            cp16(to + k_at(row), kp, in_row, policy);
            cp16(to + C::kPool + v_at(row), vp, in_row, policy);
            kp += row_step;
            vp += row_step;
          }
          if constexpr (Q8) {
            const uint8_t* const sc = reinterpret_cast<const uint8_t*>(lane < 16 ? kv.k_scale : kv.v_scale) +
                                      ((uint64_t)pg * P.spage_bytes + ((in_page + (lane & 15)) * P.stoken_bytes +
                                                                       w.hk * P.shead_bytes + col0 / 8));
            const uint32_t st = to + 2 * C::kPool + (lane < 16 ? 0 : C::kScales) + (k * kGroup + (lane & 15)) * NB * 4;
#pragma unroll
            for (int i = 0; i < NB * 4 / SB; ++i) cp_small<SB>(st + i * SB, sc + i * SB, true, policy);
          }
        }
      } else {
        if (want && !ok) atomicOr(a.status, kStatusBadSlot);
        const uint32_t in_page = t - column_of(t) * (uint32_t)kv.page_size;
        long long off = 0, soff = 0;
        if (ok) off = page * kv.page + in_page * kv.token + w.hk * kv.head + (A4 ? col_bytes : col0);
        if (BLOCKED && ok) soff = page * kv.spage + in_page * kv.stoken + w.hk * kv.shead + col0 / 32;
#pragma unroll 1
        for (int i = 0; i < T / PER; ++i) {
          const int row = i * PER + sub;
          const long long o = __shfl_sync(~0u, off, row);
          const bool use = ((mask >> row) & 1) && in_row;
          const long long src = use ? o * ES + chunk * 16 : 0;
          cp16(to + k_at(row), kv.k + src, use, policy);
          cp16(to + C::kPool + v_at(row), kv.v + src, use, policy);
        }
        if constexpr (BLOCKED) {
          const uint32_t st = to + 2 * C::kPool;
#pragma unroll 1
          for (int i = 0; i < T * NB / 32; ++i) {
            const int row = (i * 32 + lane) / NB, b = (i * 32 + lane) % NB;
            const long long so = __shfl_sync(~0u, soff, row);
            const bool use = ((mask >> row) & 1) && col0 + b * 32 < D;
            const long long src = use ? so + b : 0;
            cp_small<4>(st + (i * 32 + lane) * 4, kv.k_scale + src, use, policy);
            cp_small<4>(st + C::kScales + (i * 32 + lane) * 4, kv.v_scale + src, use, policy);
          }
        }
      }
      return mask;
    };

    // Position of this lane's token of the tile, for the bias by distance.
    auto position_of = [&](const Walk& w) {
      const uint32_t t = token_of(w);
      if (a.positions == nullptr || empty(w) || !(t >= w.q.begin && t < w.q.len)) return (int)t;
      return (int)a.positions[w.s * a.positions_stride + t];
    };

    uint32_t chunks[CPR / 2];  // heads in columns: of ldmatrix's rows in 16 tokens, for chunks 2 i and 2 i + 1
    if constexpr (COLS) {
#pragma unroll
      for (int i = 0; i < CPR / 2; ++i) chunks[i] = a4::chunk_at<CPR>(lane & 15, 2 * i + (lane >> 4));
    }

    int page = page_of(in);
    uint32_t masks[S];  // of the tiles in the ring, the tile being used first
    int place = SCORED ? position_of(in) : 0, places[SCORED ? S : 1];

    // ---- the row being worked on
    constexpr int QR = COLS ? 1 : Q8 ? 4 * R : 6 * R;  // registers of q for 16 elements
    constexpr int OX = COLS ? 2 * R : 4 * R;
    uint32_t qf[2 * NB][QR];
    float q_back[R];      // Q8: what s is to be multiplied by for the scaling of q and the bytes' unit; -2^-64 times it if above 2^127
    float q_start[R][NB];  // Q8: -128 units times the sum of q over a block
    // sums of p V, transposed: o[i][4 r + x] of MMA rows (columns of the head) g (x = 0, 1) or g + 8 (2, 3) of step i
    // and of query heads 8 r + 2 q4 + (x & 1).  Heads in columns: o[2 b + j][2 r + x] of head 4 r + q4,
    // element 32 b + 4 g + 2 j + x (A4) or 32 b + 16 j + 2 g + x (Q8)
    float o[W / 16][OX], m[R], l[R];
    typename std::conditional<A4, a4::Query<A4 ? NB : 1, R>, a4::Query8<COLS ? NB : 1, R>>::type cq;
    float om[A4 ? R : 1][A4 ? NB : 1];  // A4: this lane's tokens' part of sum p (m + 8 d), of block b
    float slope[SCORED ? R : 1];        // of this lane's softmax rows, times log2(e)
    int newest = 0;                     // position of the row's last token
    // Q8: the largest s so far (m may lie below it), the biased exponent of the largest V scale so far, and that of
    // the sums' unit: the same but inside a tile
    float highest[R];
    int v_exp = 14, o_exp = 14;

    auto load_q = [&]() {
      // this lane's eight elements of a block: 8 q4 .., or (Q8 in columns) 4 q4 .. of both its chunks
      constexpr bool CHUNKS = COLS && !A4;
      if constexpr (SCORED) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int in_group = at.block * ROWS + (COLS ? 4 * r + q4 : 8 * r + g);
          slope[r] = a.slopes != nullptr && in_group < P.group
                         ? a.slopes[(int64_t)at.hk * P.group + in_group] * 1.4426950408889634f
                         : 0.f;
        }
        newest = a.positions != nullptr ? a.positions[at.s * a.positions_stride + at.q.len - 1] : (int)at.q.len - 1;
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int in_group = at.block * ROWS + (COLS ? r * 4 + g / 2 : r * 8 + g);
        const bool use = in_group < P.group;
        const float* src = a.q + at.s * a.q_stride + (int64_t)(at.hk * P.group + in_group) * D + col0 + (CHUNKS ? 4 : 8) * q4;
        float x[NB][8];
        float top = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const bool here = use && col0 + 32 * b + 8 * q4 < D;
          const float4 u = here ? *reinterpret_cast<const float4*>(src + 32 * b) : make_float4(0.f, 0.f, 0.f, 0.f);
          const float4 v = here ? *reinterpret_cast<const float4*>(src + 32 * b + (CHUNKS ? 16 : 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
          x[b][0] = u.x, x[b][1] = u.y, x[b][2] = u.z, x[b][3] = u.w;
          x[b][4] = v.x, x[b][5] = v.y, x[b][6] = v.z, x[b][7] = v.w;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[b][i] *= P.q_scale;
            if (BLOCKED) top = fmaxf(top, fabsf(x[b][i]));
          }
        }
        if constexpr (BLOCKED) {
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        }
        if constexpr (COLS) {
          cq.take(r, x, top, lane);
          if constexpr (A4)
#pragma unroll
            for (int b = 0; b < NB; ++b) om[r][b] = 0.f;
        } else if constexpr (Q8) {
          const int e = max((int)(__float_as_uint(top) >> 23), 14);
          const float up = pow2_biased(267 - e);  // the row's largest |q| becomes 2^13 .. 2^14
          q_back[r] = e + 11 < 255 ? pow2_biased(e + 11) : -pow2_biased(e + 11 - 64);
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
        m[r] = highest[r] = -INFINITY;
        l[r] = 0.f;
      }
      if constexpr (Q8) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {  // products with 0x8080, -2^-17 = -128 units
          const uint32_t(&x)[QR] = qf[2 * b];
          const uint32_t(&y)[QR] = qf[2 * b + 1];
          constexpr uint32_t k = 0x80808080u;
          float c[4];
          if constexpr (R == 1) {
            mma_first<true>(c, x[0], x[1], x[2], x[3], k, k);
            mma<true>(c, y[0], y[1], y[2], y[3], k, k);
            q_start[0][b] = c[0] + c[2];
          } else {
            mma_first<true>(c, x[0], x[1], x[4], x[5], k, k);
            mma<true>(c, y[0], y[1], y[4], y[5], k, k);
            mma<true>(c, x[2], x[3], x[6], x[7], k, k);
            mma<true>(c, y[2], y[3], y[6], y[7], k, k);
            q_start[0][b] = c[0];
            q_start[R - 1][b] = c[2];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < W / 16; ++i)
#pragma unroll
        for (int x = 0; x < OX; ++x) o[i][x] = 0.f;
      v_exp = o_exp = 14;
    };

    // Tile i is used while tile i + S - 1 is on its way; the loop starts S - 1 tiles early, so that its
    // body exists once (the code of a launch is read from L2, past the cache stream, and has to be short).
    bool begun_here = at.tile == 0, fresh = true;
    int stage = 0, ahead = 0;  // of tile i and of tile i + S - 1
#pragma unroll 1
    for (int i = 1 - S; i < n; ++i) {
      // the stage used by the tile before this one takes the tile S - 1 ahead
      auto fetch_ahead = [&]() {
#pragma unroll
        for (int k = 0; k + 1 < S; ++k) {
          masks[k] = masks[k + 1];
          if (SCORED) places[k] = places[k + 1];
        }
        if (i + S - 1 < n) {
          masks[S - 1] = fetch(in, page, ahead);
          if (SCORED) places[S - 1] = place;
          if (i + S < n) {
            advance<T, SCORED, LEAD>(in, P);
            page = page_of(in);
            if (SCORED) place = position_of(in);
          }
        }
        cp_commit();
        ahead = ahead + 1 == S ? 0 : ahead + 1;
      };
      if (i >= 0) {
        if (fresh) {
          fresh = false;
          load_q();
        }
        cp_wait<S - 2>();
        __syncwarp();
      }
      if (H == 1) {
        fetch_ahead();
        if (i < 0) continue;
      }
      const uint32_t from = ring + stage * C::kStage;

      // ---- s = q K^T: s[r][2 nt + c] of head row g + 8 r, token 8 nt + 2 q4 + c (in columns: s[r][c] of head 4 r + q4,
      // token 8 c + g)
      float s[R][NV];
      auto token_at = [&](int c) { return COLS ? 8 * c + g : 8 * (c / 2) + 2 * q4 + c % 2; };
      if ((H == 1 || i >= 0) && !empty(at)) {
        if constexpr (COLS) {
#pragma unroll
          for (int k = 0; k < GR; ++k) {
            float c[R][2];
            cq.dot(c, from + 16 * k * C::kRowBytes, from + 2 * C::kPool + 16 * k * NB * 4, chunks, lane);
#pragma unroll
            for (int r = 0; r < R; ++r) s[r][2 * k] = c[r][0], s[r][2 * k + 1] = c[r][1];
          }
        } else if constexpr (Q8) {
#pragma unroll
          for (int nt = 0; nt < NN; ++nt) {
            float d0[NB], d1[NB];  // K's scales of tokens 8 nt + 2 q4, and the next
            const uint32_t sc = from + 2 * C::kPool + (8 * nt + 2 * q4) * NB * 4;
            lds_floats(d0, sc);
            lds_floats(d1, sc + NB * 4);
#pragma unroll
            for (int r = 0; r < R; ++r) s[r][2 * nt] = s[r][2 * nt + 1] = 0.f;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              const int row = 8 * nt + g;
              // element order inside a block: lane q4 holds 8 q4 .. 8 q4 + 7, as q does
              const int seg = b ^ (W == 64 ? (row >> 1) & 1 : row & 3);
              uint32_t w0, w1, b0, b1, b2, b3;
              lds64(w0, w1, from + row * C::kRowBytes + seg * 32 + q4 * 8);
              bytes_to_f16x2(w0, b0, b1);
              bytes_to_f16x2(w1, b2, b3);
              float c[4];
              const uint32_t(&x)[QR] = qf[2 * b];
              const uint32_t(&y)[QR] = qf[2 * b + 1];
              if constexpr (R == 1) {
                mma_from(c, q_start[0][b], q_start[0][b], 0.f, 0.f, x[0], x[1], x[2], x[3], b0, b1);
                mma<true>(c, y[0], y[1], y[2], y[3], b2, b3);
                s[0][2 * nt] = fmaf(c[0] + c[2], d0[b], s[0][2 * nt]);
                s[0][2 * nt + 1] = fmaf(c[1] + c[3], d1[b], s[0][2 * nt + 1]);
              } else {
                mma_from(c, q_start[0][b], q_start[0][b], q_start[R - 1][b], q_start[R - 1][b], x[0], x[1], x[4], x[5], b0, b1);
                mma<true>(c, y[0], y[1], y[4], y[5], b2, b3);
                mma<true>(c, x[2], x[3], x[6], x[7], b0, b1);
                mma<true>(c, y[2], y[3], y[6], y[7], b2, b3);
                s[0][2 * nt] = fmaf(c[0], d0[b], s[0][2 * nt]);
                s[0][2 * nt + 1] = fmaf(c[1], d1[b], s[0][2 * nt + 1]);
                s[R - 1][2 * nt] = fmaf(c[2], d0[b], s[R - 1][2 * nt]);
                s[R - 1][2 * nt + 1] = fmaf(c[3], d1[b], s[R - 1][2 * nt + 1]);
              }
            }
          }
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < 2 * NN; ++c) s[r][c] *= q_back[r];
#pragma unroll
          for (int r = 0; r < R; ++r)
            if (q_back[r] < 0.f)  // |q| of 2^117 and more
#pragma unroll
              for (int c = 0; c < 2 * NN; ++c) s[r][c] *= -18446744073709551616.f;
        } else {
#pragma unroll
          for (int k = 0; k < GR; ++k) {
            float c[2][4], e[2][4];  // of q's first two parts, and of the others
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              uint32_t w[2][4];
#pragma unroll
              for (int nt = 0; nt < 2; ++nt)
                lds128(w[nt], from + (16 * k + 8 * nt + g) * C::kRowBytes + (((4 * b + q4) ^ ((g & 1) << 2)) << 4));
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t(&x)[QR] = qf[2 * b + h];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                  if constexpr (R == 1) {
                    if (b + h == 0) {
                      mma_first<false>(c[nt], x[0], x[1], x[3], x[4], w[nt][0], w[nt][1]);
                      mma_first<false>(e[nt], x[2], 0u, x[5], 0u, w[nt][0], w[nt][1]);
                    } else {
                      mma<false>(c[nt], x[0], x[1], x[3], x[4], w[nt][2 * h], w[nt][2 * h + 1]);
                      mma<false>(e[nt], x[2], 0u, x[5], 0u, w[nt][2 * h], w[nt][2 * h + 1]);
                    }
                  } else {
                    if (b + h == 0) {
                      mma_first<false>(c[nt], x[0], x[1], x[6], x[7], w[nt][0], w[nt][1]);
                      mma_first<false>(e[nt], x[2], x[3], x[8], x[9], w[nt][0], w[nt][1]);
                    } else {
                      mma<false>(c[nt], x[0], x[1], x[6], x[7], w[nt][2 * h], w[nt][2 * h + 1]);
                      mma<false>(e[nt], x[2], x[3], x[8], x[9], w[nt][2 * h], w[nt][2 * h + 1]);
                    }
                    mma<false>(e[nt], x[4], x[5], x[10], x[11], w[nt][2 * h], w[nt][2 * h + 1]);
                  }
                }
              }
            }
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              const int at0 = 4 * k + 2 * nt;
              if constexpr (R == 1) {
                s[0][at0] = c[nt][0] + (c[nt][2] + e[nt][0]);
                s[0][at0 + 1] = c[nt][1] + (c[nt][3] + e[nt][1]);
              } else {
                s[0][at0] = c[nt][0] + e[nt][0];
                s[0][at0 + 1] = c[nt][1] + e[nt][1];
                s[R - 1][at0] = c[nt][2] + e[nt][2];
                s[R - 1][at0 + 1] = c[nt][3] + e[nt][3];
              }
            }
          }
        }
        if constexpr (H == 2) {
          // the pair's halves of s: each puts its own where its tile of K was, both add the two.  The next
          // copy into this stage starts behind the next tile's barrier, when both have read.
          __syncwarp();
          constexpr int NX = NV / 4;
#pragma unroll
          for (int x = 0; x < R * NX; ++x) {
            const float(&v)[NV] = s[x / NX];
            const float part[4] = {v[4 * (x % NX)], v[4 * (x % NX) + 1], v[4 * (x % NX) + 2], v[4 * (x % NX) + 3]};
            sts128(from + (x * 32 + lane) * 16, part);
          }
          asm volatile("bar.sync %0, 64;" ::"r"(worker + 1) : "memory");
          const uint32_t other = from + (warp % 2 == 0 ? C::kRing : -C::kRing);
#pragma unroll
          for (int x = 0; x < R * NX; ++x) {
            float part[4];
            lds_floats(part, other + (x * 32 + lane) * 16);
#pragma unroll
            for (int c = 0; c < 4; ++c) s[x / NX][4 * (x % NX) + c] += part[c];
          }
        }
      }
      if (H == 2) {
        fetch_ahead();
        if (i < 0) continue;
      }

      const uint32_t mk = masks[0];
      float low[R], top[R];
      bool idle = false;
      if (!empty(at)) {
        // ---- capped and biased
        if constexpr (SCORED) {
          if (P.cap_log2 > 0.f) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int c = 0; c < NV; ++c) s[r][c] = P.cap_log2 * tanhf(s[r][c]);
          }
          if (a.slopes != nullptr) {
#pragma unroll
            for (int c = 0; c < NV; ++c) {
              const float far = (float)(__shfl_sync(~0u, places[0], token_at(c)) - newest);
#pragma unroll
              for (int r = 0; r < R; ++r) s[r][c] = fmaf(slope[r], far, s[r][c]);
            }
          }
        }

        if constexpr (BLOCKED) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            low[r] = s[r][0];
#pragma unroll
            for (int c = 1; c < NV; ++c) low[r] = fminf(low[r], s[r][c]);
          }
        }
        if (mk != (uint32_t)((1ull << T) - 1)) {
#pragma unroll
          for (int c = 0; c < NV; ++c)
            if (!((mk >> token_at(c)) & 1))
#pragma unroll
              for (int r = 0; r < R; ++r) s[r][c] = -INFINITY;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          top[r] = s[r][0];
#pragma unroll
          for (int c = 1; c < NV; ++c) top[r] = fmaxf(top[r], s[r][c]);
          if constexpr (COLS) {
            top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 4));
            top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 8));
            top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 16));
          } else {
            top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 1));
            top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 2));
          }
        }
        if (BACK && a.slopes != nullptr) {
          // A head's tile of which every p is below 2^-104 adds nothing (but a NaN)
          idle = true;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const bool gone = top[r] < highest[r] - 104.f;
            idle &= gone || at.block * ROWS + 4 * r + q4 >= P.group;
            if (gone) low[r] = INFINITY;
#pragma unroll
            for (int c = 0; c < NV; ++c)
              if (gone && s[r][c] == s[r][c]) s[r][c] = -INFINITY;
          }
          idle = __all_sync(~0u, idle);
          if (idle) {
            uint32_t dm[NB];
            bool number = true;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int c = 0; c < NV; ++c) number &= s[r][c] == s[r][c];
#pragma unroll
            for (int half = 0; half < H; ++half) {  // (both warps of a pair decide alike)
              const uint32_t there = half == 0 ? from : from + (warp % 2 == 0 ? C::kRing : -C::kRing);
              a4::load_steps<NB>(dm, there + 2 * C::kPool + C::kScales + lane * NB * 4);
#pragma unroll
              for (int b = 0; b < NB; ++b)
                number &= (dm[b] & 0x7f800000u) != 0x7f800000u && (!A4 || (dm[b] & 0x7f80u) != 0x7f80u);
            }
            idle = __all_sync(~0u, number);
          }
        }
      }

      if (!empty(at) && !idle) {
        // ---- softmax: p = 2^(s - m) and the factor of what came before.
        // bf16 parts of p have fp32's range: m is the maximum so far.  fp16 parts keep 12 bits or more of p only
        // above 2^-26, so that m follows the tile's own maximum, down to 2^-24 (or 2^-64) of the largest p; a tile with
        // smaller p all the same (`wide`) takes its products in classes of 2^-26 (below).
        bool wide = false;
        float next[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if constexpr (Q8) {
            highest[r] = fmaxf(highest[r], top[r]);
            next[r] = fmaxf(top[r], highest[r] - 24.f);
            wide |= next[r] - low[r] > 26.f;
          } else if constexpr (COLS) {
            // (from the newest back most tiles lie below.  2^64 leaves Q8's sums of 2^31 tokens numbers, A4's of m + 8 d have no
            // unit that would)
            highest[r] = fmaxf(highest[r], top[r]);
            next[r] = fmaxf(top[r], highest[r] - (BACK && !A4 ? 64.f : 24.f));
            wide |= next[r] - low[r] > 26.f;
          } else {
            next[r] = fmaxf(m[r], top[r]);
          }
        }
        const uint32_t sv = from + 2 * C::kPool + C::kScales;  // V's steps
        // Of this lane's token, |d| as the bits of a float and 2^23 more: infinities and NaN, which are for their own 32 columns and
        // set no unit for the others, become negative.
        constexpr int kOne = 1 << 23;
        auto steps_of_one = [&](int (&one)[NB]) {
          static_assert(!COLS || T == 32, "a lane looks at one token's steps");
          uint32_t step[NB];
          a4::load_steps<NB>(step, sv + lane * NB * 4);
#pragma unroll
          for (int b = 0; b < NB; ++b) one[b] = (int)((A4 ? (step[b] & 0x7fffu) * 65536u : step[b] & 0x7fffffffu) + kOne);
        };
        if constexpr (COLS) {
          int one[NB], most = 0;
          steps_of_one(one);
#pragma unroll
          for (int b = 0; b < NB; ++b) most = max(most, one[b]);
          v_exp = max(v_exp, (__reduce_max_sync(~0u, most) >> 23) - 1);
          const int little = (v_exp - 12) * kOne;
#pragma unroll
          for (int b = 0; b < NB; ++b) wide |= one[b] > kOne && one[b] < little + kOne;
        }
        if (Q8 || COLS) wide = __any_sync(~0u, wide);
        float keep[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if ((Q8 || COLS) && wide) next[r] = highest[r];  // the classes' factors leave no room for 2^24 more
          const float base = next[r] == -INFINITY ? 0.f : next[r];
          keep[r] = exp2_fast(m[r] - base);
          m[r] = next[r];
          float sum = 0.f;
#pragma unroll
          for (int c = 0; c < NV; c += 2) {
            s[r][c] = exp2_fast(s[r][c] - base);
            s[r][c + 1] = exp2_fast(s[r][c + 1] - base);
            sum += s[r][c] + s[r][c + 1];
          }
          l[r] = fmaf(l[r], keep[r], sum);
        }

        // ---- o^T = o^T keep + V^T p^T: p is the B operand as it stands, its parts add up in the accumulators
        const uint32_t fv = from + C::kPool;
        float kept[2 * R];  // keep of the heads that this lane's sums are of
#pragma unroll
        for (int r = 0; r < (COLS ? 0 : R); ++r) {
          kept[2 * r] = __shfl_sync(~0u, keep[r], 8 * q4);
          kept[2 * r + 1] = __shfl_sync(~0u, keep[r], 8 * q4 + 4);
        }
        auto join = [&](float (&acc)[OX], const float (&c)[R][4]) {
#pragma unroll
          for (int x = 0; x < 4 * R; ++x) acc[x] = fmaf(acc[x], kept[2 * (x / 4) + x % 2], c[x / 4][x % 4]);
        };
        if constexpr (COLS) {
          const float up = pow2_biased(267 - v_exp);  // the largest d becomes 2^13 .. 2^14
          const uint32_t v_at = from + C::kPool, steps = sv + g * NB * 4;
          float gap_up[NB];
          // Products of weights p (ps: p up), with what came before times `keep`, and the sums' unit moved by `shift` too.
          auto products = [&](auto is_wide, const float (&ps)[R][NV], const float (&p)[R][NV], float shift) {
            constexpr bool WIDE = decltype(is_wide)::value;
            uint32_t dm[NV][2], z[GR][4];
            float d[NV];  // of block b
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              if constexpr (!A4) {
                // V of tokens 2 q4, 2 q4 + 1 and 8 further of 16, bytes 2 g and 2 g + 1 of the block's two chunks
#pragma unroll
                for (int c = 0; c < NV; ++c) {
                  d[c] = __uint_as_float(lds32(steps + (8 * c * NB + b) * 4));
                  if constexpr (WIDE) d[c] *= gap_up[b];
                }
#pragma unroll
                for (int k = 0; k < GR; ++k) a4::ldmatrix4_trans(z[k], v_at + 16 * k * C::kRowBytes + chunks[b]);
              } else if (b % 2 == 0) {
                // {d, m} of the lane's tokens, of blocks b and b + 1; V of tokens 2 q4, 2 q4 + 1 and 8 further of 16,
                // elements 4 g .. 4 g + 3
#pragma unroll
                for (int c = 0; c < NV; ++c) lds64(dm[c][0], dm[c][1], steps + (8 * c * NB + b) * 4);
#pragma unroll
                for (int k = 0; k < GR; ++k) a4::ldmatrix4_trans(z[k], v_at + 16 * k * C::kRowBytes + chunks[b / 2]);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                  for (int x = 0; x < 2; ++x) {
                    float sum = p[r][0] * a4::middle_of(dm[0][x]);
#pragma unroll
                    for (int c = 1; c < NV; ++c) sum = fmaf(p[r][c], a4::middle_of(dm[c][x]), sum);
                    om[r][b + x] = fmaf(om[r][b + x], keep[r], sum);
                  }
                if constexpr (WIDE) {
#pragma unroll
                  for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int c = 0; c < NV; ++c) dm[c][x] = __float_as_uint(a4::step_of(dm[c][x]) * gap_up[b + x]) >> 16;
                }
              }
              if constexpr (A4)
#pragma unroll
                for (int c = 0; c < NV; ++c) d[c] = a4::step_of(dm[c][b % 2]);
              uint32_t w[GR][R][2];
#pragma unroll
              for (int k = 0; k < GR; ++k)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                  a4::split2(a4::mul2(make_float2(ps[r][2 * k], ps[r][2 * k + 1]), make_float2(d[2 * k], d[2 * k + 1])),
                             w[k][r][0], w[k][r][1]);
                  w[k][r][0] = a4::movmatrix(w[k][r][0]);
                  w[k][r][1] = a4::movmatrix(w[k][r][1]);
                }
              float c[2][R][4];  // MMA rows g, g + 8 of step j: elements as in o
#pragma unroll
              for (int k = 0; k < GR; ++k) {
                uint32_t x[4], y[4];
                if constexpr (A4) {
                  a4::nibbles_less_8(z[k][2 * (b % 2)], x);
                  a4::nibbles_less_8(z[k][2 * (b % 2) + 1], y);
                } else {
#pragma unroll
                  for (int j = 0; j < 2; ++j) {
                    a4::bytes_of_pairs(z[k][2 * j], x[2 * j], x[2 * j + 1]);
                    a4::bytes_of_pairs(z[k][2 * j + 1], y[2 * j], y[2 * j + 1]);
                  }
                }
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                  for (int j = 0; j < 2; ++j) {
                    if (k == 0)
                      a4::mma_first(c[j][r], x[2 * j], x[2 * j + 1], y[2 * j], y[2 * j + 1], w[k][r][0], w[k][r][1]);
                    else
                      a4::mma(c[j][r], x[2 * j], x[2 * j + 1], y[2 * j], y[2 * j + 1], w[k][r][0], w[k][r][1]);
                  }
              }
              const float back = WIDE ? pow2_biased(254 - (int)(__float_as_uint(gap_up[b]) >> 23)) : 1.f;
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                  const float f = keep[r] * shift;
#pragma unroll
                  for (int x = 0; x < 2; ++x) {
                    float sum = fmaf(c[j][r][2 * x + 1], a4::kLoUnit, c[j][r][2 * x]);
                    if constexpr (WIDE) sum *= back;
                    o[2 * b + j][2 * r + x] = fmaf(o[2 * b + j][2 * r + x], f, sum);
                  }
                }
            }
          };
          float ps[R][NV];
          if (!wide) {
            float shift = 1.f;
            if (o_exp != v_exp) {
              shift = o_exp - v_exp < -126 ? 0.f : pow2_biased(127 + o_exp - v_exp);
              o_exp = v_exp;
            }
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int c = 0; c < NV; ++c) ps[r][c] = s[r][c] * up;
            products(std::false_type{}, ps, s, shift);
          } else {
            // A tile with p below 2^-26, or a d below 2^-12 of the largest, takes its products in classes of p, class k
            // being 2^(-26 (k + 1)) <= p < 2^(-26 k) (p = 1 in class 0; p below 2^-104 is 0), and with each block's steps brought up to
            // the largest.  Class k is multiplied by 2^(26 k), and the sums' unit goes down as far until the last class is in.
            constexpr float kClass = 67108864.f;  // 2^26
            int one[NB];
            steps_of_one(one);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              const int e = (__reduce_max_sync(~0u, one[b]) >> 23) - 1;
              // (e is at most v_exp.  Up to 2^120, so that it and its inverse are numbers, for steps of 0 too; p d below 2^-104 is 0 anyway)
              gap_up[b] = pow2_biased(127 + min(v_exp - max(e, 14), 120));
            }
            uint32_t classes = 0;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int c = 0; c < NV; ++c) {
                const int k = (126 - (int)(__float_as_uint(s[r][c]) >> 23)) / 26;
                if (s[r][c] > 0.f && k < 4) classes |= 1u << k;
              }
            classes = max(__reduce_or_sync(~0u, classes), 1u);  // one at least: what came before takes its factor there
#pragma unroll 1
            while (classes != 0) {
              const int k26 = 26 * (31 - __clz(classes));
              classes &= ~(1u << (k26 / 26));
              const int change = o_exp - (v_exp - k26);
              o_exp = v_exp - k26;
              const float class_up = pow2_biased(127 + k26);
              float p[R][NV];
#pragma unroll
              for (int r = 0; r < R; ++r)
#pragma unroll
                for (int c = 0; c < NV; ++c) {
                  const float x = s[r][c] * class_up;  // of a higher class: 2^26 or more above 1; of a lower: under 2^-26
                  const bool in_class = x >= 1.f / kClass && (x < 1.f || k26 == 0);
                  p[r][c] = in_class ? s[r][c] : 0.f, ps[r][c] = in_class ? x * up : 0.f;
                }
              products(std::true_type{}, ps, p, change < -126 ? 0.f : pow2_biased(127 + change));
#pragma unroll
              for (int r = 0; r < R; ++r) keep[r] = 1.f;  // of a class still to come
            }
          }
          if (o_exp != v_exp) {
            const float again = pow2_biased(127 + o_exp - v_exp);  // from the last class's unit
            o_exp = v_exp;
#pragma unroll
            for (int k = 0; k < W / 16; ++k)
#pragma unroll
              for (int x = 0; x < OX; ++x) o[k][x] *= again;
          }
        } else if constexpr (Q8) {
          float d[2 * NN][NB];  // V's scales of the lane's tokens
          const uint32_t sv = from + 2 * C::kPool + C::kScales + 2 * q4 * NB * 4;
          float vs[NB];  // of one token
          int most = 0;  // as in steps_of_one: an infinity sets no unit
          lds_floats(vs, from + 2 * C::kPool + C::kScales + (lane & (T - 1)) * NB * 4);
#pragma unroll
          for (int b = 0; b < NB; ++b) most = max(most, (int)(__float_as_uint(fabsf(vs[b])) + kOne));
          v_exp = max(v_exp, (__reduce_max_sync(~0u, most) >> 23) - 1);
          // fp16 parts of p d keep 2^-38 of the largest scale: 2^-26 of one that lies 2^12 below it.  A tile with smaller
          // ones takes its products in classes too, with each block's scales brought up to the largest (64 x 8192 tokens whose
          // blocks lie further apart: 267 us, else 207).
          const float little = pow2_biased(v_exp - 12);
#pragma unroll
          for (int b = 0; b < NB; ++b) wide |= fabsf(vs[b]) < little && vs[b] != 0.f;
          wide = __any_sync(~0u, wide);
#pragma unroll
          for (int c = 0; c < 2 * NN; ++c) lds_floats(d[c], sv + (8 * (c / 2) + c % 2) * NB * 4);
          const float up = pow2_biased(267 - v_exp);  // the largest scale becomes 2^13 .. 2^14
          // Products of weights w, with the sums' unit moved to the biased exponent `unit`; back(b) undoes what d[.][b] was
          // multiplied by.
          auto products = [&](const float (&w)[R][2 * NN], int unit, auto back) {
            const int change = o_exp - unit;
            const float shift = change < -126 ? 0.f : pow2_biased(127 + change);
            o_exp = unit;
#pragma unroll
            for (int x = 0; x < 2 * R; ++x) kept[x] *= shift;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              float c[2][R][4];  // MMA rows g, g + 8 of step j: elements 32 b + 4 g + 2 j, and the next
#pragma unroll
              for (int k = 0; k < GR; ++k) {
                uint32_t f[2][4];  // V of tokens (2 q4, 2 q4 + 1) and 8 further, elements 32 b + 4 g + 0..3
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  auto word = [&](int t) {
                    const int vrow = W == 64 ? (t & ~15) | ((t >> 1) & 7) | ((t & 1) << 3) : t;
                    const int seg = b ^ ((vrow >> 1) & (W == 64 ? 1 : 3));
                    return lds32(fv + vrow * C::kRowBytes + seg * 32 + g * 4) ^ 0x80808080u;
                  };
                  const uint32_t x = word(16 * k + 8 * h + 2 * q4), y = word(16 * k + 8 * h + 2 * q4 + 1);
                  q8_word_to_f16x2(__byte_perm(x, y, 0x5140), f[h][0], f[h][1]);
                  q8_word_to_f16x2(__byte_perm(x, y, 0x7362), f[h][2], f[h][3]);
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                  uint32_t hi[2], lo[2];
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    const int t = 4 * k + 2 * h;
                    split2(w[r][t] * d[t][b], w[r][t + 1] * d[t + 1][b], hi[h], lo[h]);
                  }
#pragma unroll
                  for (int j = 0; j < 2; ++j) {
                    if (k == 0)
                      mma_first<true>(c[j][r], f[0][2 * j], f[0][2 * j + 1], f[1][2 * j], f[1][2 * j + 1], hi[0], hi[1]);
                    else
                      mma<true>(c[j][r], f[0][2 * j], f[0][2 * j + 1], f[1][2 * j], f[1][2 * j + 1], hi[0], hi[1]);
                    mma<true>(c[j][r], f[0][2 * j], f[0][2 * j + 1], f[1][2 * j], f[1][2 * j + 1], lo[0], lo[1]);
                  }
                }
              }
#pragma unroll
              for (int x = 0; x < 8 * R; ++x) c[x / (4 * R)][x / 4 % R][x % 4] *= back(b);
              join(o[2 * b], c[0]);
              join(o[2 * b + 1], c[1]);
            }
          };
          float w[R][2 * NN];
          if (!wide) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int c = 0; c < 2 * NN; ++c) w[r][c] = s[r][c] * up;
            products(w, v_exp, [](int) { return 1.f; });
          } else {
            // Classes of p, class k being 2^(-26 (k + 1)) <= p < 2^(-26 k) (p = 1 in class 0); p below 2^-104 is 0.  Class k is
            // multiplied by 2^(26 k), and the sums' unit goes down as far, until the last class is in.
            constexpr float kClass = 67108864.f;  // 2^26
            float back[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              const int e = (int)(__reduce_max_sync(~0u, __float_as_uint(fabsf(vs[b]))) >> 23);
              const int gap = min(max(v_exp - e, 0), 120);  // (a NaN's e is 255)
              back[b] = pow2_biased(127 - gap);
#pragma unroll
              for (int c = 0; c < 2 * NN; ++c) d[c][b] *= pow2_biased(127 + gap);
            }
            uint32_t classes = 0;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int c = 0; c < 2 * NN; ++c) {
                const int k = (126 - (int)(__float_as_uint(s[r][c]) >> 23)) / 26;
                if (s[r][c] > 0.f && k < 4) classes |= 1u << k;
              }
            classes = max(__reduce_or_sync(~0u, classes), 1u);  // one at least: what came before takes its factor there
#pragma unroll 1
            while (classes != 0) {
              const int k = 31 - __clz(classes);
              classes ^= 1u << k;
              float factor = 1.f;
              for (int i26 = 0; i26 < k; ++i26) factor *= kClass;
#pragma unroll
              for (int r = 0; r < R; ++r)
#pragma unroll
                for (int c = 0; c < 2 * NN; ++c) {
                  const float x = s[r][c] * factor;  // of a higher class: 2^26 or more above 1; of a lower: under 2^-26
                  w[r][c] = x >= 1.f / kClass && (x < 1.f || k == 0) ? x * up : 0.f;
                }
              products(w, v_exp - 26 * k, [&](int b) { return back[b]; });
#pragma unroll
              for (int x = 0; x < 2 * R; ++x) kept[x] = 1.f;  // of a class still to come
            }
            const float up_again = pow2_biased(127 + o_exp - v_exp);  // from the last class's unit
            o_exp = v_exp;
#pragma unroll
            for (int k = 0; k < W / 16; ++k)
#pragma unroll
              for (int x = 0; x < 4 * R; ++x) o[k][x] *= up_again;
          }
        } else {
          uint32_t hi[R][NN], mid[R][NN], lo[R][NN];  // of tokens 8 nt + 2 q4, and the next
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int nt = 0; nt < NN; ++nt)
              split3(s[r][2 * nt], s[r][2 * nt + 1], hi[r][nt], mid[r][nt], lo[r][nt]);
#pragma unroll
          for (int i16 = 0; i16 < W / 16; ++i16) {  // MMA rows g, g + 8: elements 16 i16 + g, and 8 further
            float c[R][4];
#pragma unroll
            for (int k = 0; k < GR; ++k) {
              uint32_t w[4];
              const int t = 16 * k + (lane & 15);
              ldmatrix4_trans(w, fv + t * C::kRowBytes + (((2 * i16 + (lane >> 4)) ^ (t & 7)) << 4));
#pragma unroll
              for (int r = 0; r < R; ++r) {
                if (k == 0)
                  mma_first<false>(c[r], w[0], w[2], w[1], w[3], hi[r][0], hi[r][1]);
                else
                  mma<false>(c[r], w[0], w[2], w[1], w[3], hi[r][2 * k], hi[r][2 * k + 1]);
                mma<false>(c[r], w[0], w[2], w[1], w[3], mid[r][2 * k], mid[r][2 * k + 1]);
                mma<false>(c[r], w[0], w[2], w[1], w[3], lo[r][2 * k], lo[r][2 * k + 1]);
              }
            }
            join(o[i16], c);
          }
        }
      }

      // ---- the row's or the run's end
      const bool row_ends = at.tile + 1 == at.q.tiles;
      if (row_ends || i + 1 == n) {
        float unit = Q8 ? pow2_biased(o_exp - 13) : 1.f;  // (in columns: below)
        if (Q8 && o_exp < 80) {  // unit / sum may be below 2^-126: two factors
#pragma unroll
          for (int k = 0; k < W / 16; ++k)
#pragma unroll
            for (int x = 0; x < OX; ++x) o[k][x] *= unit;
          unit = 1.f;
        }
        const bool alone = begun_here && row_ends;
        float* part = nullptr;
        if (!alone) {
          const long long row = u0 + i - at.tile;
          if (!begun_here) {
            Left& to = COLS ? s_left[worker] : left;  // (in columns: not kept in registers meanwhile)
            has0 = true, end0 = row_ends, to.s0 = at.s, to.hk0 = at.hk, to.block0 = at.block;
            to.tiles0 = at.q.tiles, to.row0 = row;
            part = part_mem + warp * C::kPart;
          } else {  // the run's last tile: nothing is in flight into the ring any more
            Left& to = COLS ? s_left[worker] : left;
            has1 = true, to.s1 = at.s, to.hk1 = at.hk, to.block1 = at.block;
            to.tiles1 = at.q.tiles, to.row1 = row;
            part = reinterpret_cast<float*>(ring_mem + (size_t)warp * C::kRing);
            cp_wait<0>();
            __syncwarp();
            // and the other warp of a pair has read this warp's half of s
            if (H == 2) asm volatile("bar.sync %0, 64;" ::"r"(worker + 1) : "memory");
          }
        }
        if constexpr (COLS) {
          const int exp = o_exp - 140, half = exp >> 1;  // the sums' unit is 2^exp, as two factors
          const float ua = pow2_biased(127 + half), ub = pow2_biased(127 + exp - half);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            // from m to the maximum: m may lie 2^64 below it, and the warps of a pair, whose V differ, have one only of that
            const float down = highest[r] == -INFINITY ? 1.f : exp2_fast(m[r] - highest[r]);
            float sum = l[r] * down;
#pragma unroll
            for (int by = 4; by < 32; by *= 2) {
              sum += __shfl_xor_sync(~0u, sum, by);
              if constexpr (A4)
#pragma unroll
                for (int b = 0; b < NB; ++b) om[r][b] += __shfl_xor_sync(~0u, om[r][b], by);
            }
            const int row = 4 * r + q4, of_group = at.block * ROWS + row;
            if (of_group >= P.group) continue;
            if (g == 0) {
              if (!alone) {
                part[ROWS * W + row] = highest[r];
                part[ROWS * W + ROWS + row] = sum;
              } else if (a.lse != nullptr && col0 == 0) {
                a.lse[(int64_t)at.s * a.n_q_heads + (int64_t)at.hk * P.group + of_group] =
                    sum == 0.f ? -INFINITY : (highest[r] + __log2f(sum)) * 0.6931471805599453f;
              }
            }
            const float f = !alone ? down : sum == 0.f ? 0.f : __fdividef(down, sum);
            float* const to = alone ? a.out + at.s * a.out_stride + ((int64_t)at.hk * P.group + of_group) * D + col0 : part + row * W;
            auto value = [&](int b, int e) {
              const float x = o[2 * b + e / 2][2 * r + e % 2] * f * ua;
              if constexpr (A4) return fmaf(x, ub, om[r][b] * f);
              return x * ub;
            };
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              if (col0 + 32 * b >= D) continue;
              if constexpr (A4) {
                *reinterpret_cast<float4*>(to + 32 * b + 4 * g) = make_float4(value(b, 0), value(b, 1), value(b, 2), value(b, 3));
              } else {
                *reinterpret_cast<float2*>(to + 32 * b + 2 * g) = make_float2(value(b, 0), value(b, 1));
                *reinterpret_cast<float2*>(to + 32 * b + 16 + 2 * g) = make_float2(value(b, 2), value(b, 3));
              }
            }
          }
        }
#pragma unroll
        for (int r = 0; r < (COLS ? 0 : R); ++r) {
          float sum = l[r];
          sum += __shfl_xor_sync(~0u, sum, 1);
          sum += __shfl_xor_sync(~0u, sum, 2);
          const int in_group = at.block * ROWS + 8 * r + g;  // of the softmax row
          if (q4 == 0 && in_group < P.group) {
            if (!alone) {
              part[ROWS * W + 8 * r + g] = m[r];
              part[ROWS * W + ROWS + 8 * r + g] = sum;
            } else if (a.lse != nullptr && col0 == 0) {
              a.lse[(int64_t)at.s * a.n_q_heads + (int64_t)at.hk * P.group + in_group] =
                  sum == 0.f ? -INFINITY : (m[r] + __log2f(sum)) * 0.6931471805599453f;
            }
          }
          const float f = alone ? (sum == 0.f ? 0.f : __fdividef(unit, sum)) : unit;
#pragma unroll
          for (int x = 0; x < 2; ++x) {  // the heads of this lane's sums
            const float fx = __shfl_sync(~0u, f, 8 * q4 + 4 * x);
            const int row = 8 * r + 2 * q4 + x, of_group = at.block * ROWS + row;
            float* to = alone ? a.out + at.s * a.out_stride + ((int64_t)at.hk * P.group + of_group) * D + col0 : part + row * W;
            if (of_group >= P.group) continue;
            if constexpr (Q8) {
#pragma unroll
              for (int b = 0; b < NB; ++b)
                if (col0 + 32 * b < D)
                  *reinterpret_cast<float4*>(to + 32 * b + 4 * g) =
                      make_float4(o[2 * b][4 * r + x] * fx, o[2 * b][4 * r + x + 2] * fx, o[2 * b + 1][4 * r + x] * fx,
                                  o[2 * b + 1][4 * r + x + 2] * fx);
            } else {
#pragma unroll
              for (int c8 = 0; c8 < W / 8; ++c8)
                if (col0 + 8 * c8 < D) to[8 * c8 + g] = o[c8 / 2][4 * r + x + 2 * (c8 % 2)] * fx;
            }
          }
        }
      }
      stage = stage + 1 == S ? 0 : stage + 1;
      if (i + 1 < n) {
        advance<T, SCORED, LEAD>(at, P);
        if (at.tile == 0) begun_here = fresh = true;
      }
    }
    cp_wait<0>();
  }
  if (lane == 0 && col0 == 0) {
    if (!COLS) s_left[worker] = left;
    if (has0) atomicOr(s_mask, 1u << worker);
    if (has0 && end0) atomicOr(s_mask + 1, 1u << worker);
    if (has1) atomicOr(s_mask + 2, 1u << worker);
  }
  __syncthreads();

  // ---- parts of rows: added up with weights 2^(m_i - max m), to the output where the row is complete, else to a
  // part in the workspace.  A chain is the parts of one row in this CTA: part 1 of the worker that left the
  // row open (w; -1: the row came into the CTA) and parts 0 of the workers behind it; the warps of a
  // chain's workers share its float4s.
  auto global_part = [&](int cta, int which) { return P.parts + ((int64_t)cta * 2 + which) * (H * C::kPart); };
  auto finish = [&](int s, int64_t head, int c, const float4& x, float M, float L) {
    const float f = L == 0.f ? 0.f : __fdividef(1.f, L);
    *reinterpret_cast<float4*>(a.out + s * a.out_stride + head * D + c) = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
    if (c == 0 && a.lse != nullptr)
      a.lse[(int64_t)s * a.n_q_heads + head] = L == 0.f ? -INFINITY : (M + __log2f(L)) * 0.6931471805599453f;
  };
  auto add = [](float4& x, const float4& y, float f) {
    x.x = fmaf(y.x, f, x.x), x.y = fmaf(y.y, f, x.y), x.z = fmaf(y.z, f, x.z), x.w = fmaf(y.w, f, x.w);
  };
  const unsigned parts0 = s_mask[0], ends0 = s_mask[1], parts1 = s_mask[2];
  // End of the chain of w (exclusive), and whether its row ends there.
  auto end_of = [&](int w, bool& ends) {
    const unsigned stop = ends0 >> (w + 1);
    ends = stop != 0;
    return w + 1 + (ends ? __ffs(stop) : __ffs(~(parts0 >> (w + 1))) - 1);
  };
#pragma unroll 1
  for (int own = 0; own < 2; ++own) {  // the chain that this worker's part 0 is in, then the one that it began
    if ((((own ? parts1 : parts0) >> worker) & 1) == 0) continue;
    const int w = own ? worker : 31 - __clz(parts1 & ((1u << worker) - 1));
    bool ends;
    const int first = max(w, 0), count = end_of(w, ends) - first;
    const Left& by = s_left[first];
    const int s = w < 0 ? by.s0 : by.s1, hk = w < 0 ? by.hk0 : by.hk1, block = w < 0 ? by.block0 : by.block1;
    const int rows = min(ROWS, P.group - block * ROWS);
    constexpr int kNext = H * C::kPart;
    const int wp = first * H + warp % H;  // the first worker's warp of this warp's columns
    const float* const rest = part_mem + wp * C::kPart;
    const float* const head = w < 0 ? rest : reinterpret_cast<const float*>(ring_mem + (size_t)wp * C::kRing);
    float* const to = global_part(blockIdx.x, w < 0 ? 0 : 1) + (warp % H) * C::kPart;
#pragma unroll 1
    for (int e = (worker - first) * 32 + lane; e < rows * (W / 4); e += count * 32) {
      const int row = e / (W / 4), c = 4 * (e % (W / 4));
      const float* const hm = head + ROWS * W + row;
      const float* const rm = rest + ROWS * W + row;
      float M = *hm, L;
#pragma unroll 4
      for (int i = 1; i < count; ++i) M = fmaxf(M, rm[i * kNext]);
      const float base = M == -INFINITY ? 0.f : M;
      const float f0 = exp2_fast(*hm - base);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      add(x, *reinterpret_cast<const float4*>(head + row * W + c), f0);
      L = hm[ROWS] * f0;
#pragma unroll 4
      for (int i = 1; i < count; ++i) {
        const float f = exp2_fast(rm[i * kNext] - base);
        add(x, *reinterpret_cast<const float4*>(rest + i * kNext + row * W + c), f);
        L = fmaf(rm[i * kNext + ROWS], f, L);
      }
      if (w >= 0 && ends) {
        if (col0 + c < D) finish(s, (int64_t)hk * P.group + block * ROWS + row, col0 + c, x, M, L);
      } else {
        *reinterpret_cast<float4*>(to + row * W + c) = x;
        if (c == 0) to[ROWS * W + row] = M, to[ROWS * W + ROWS + row] = L;
      }
    }
  }

  // ---- rows that cross CTAs: the last CTA to arrive adds them up in CTA order.  Of a CTA's rows only the one that
  // came in (0) and the last one left open (1) can cross.
  const int open = 31 - __clz(parts1);
  bool crosses[2] = {(parts0 & 1) != 0, false};
  if (open >= 0) {
    end_of(open, crosses[1]);
    crosses[1] = !crosses[1];
  }
  if (!crosses[0] && !crosses[1]) return;
  __syncthreads();
  if (tid < 2) {
    int joined = 0, c0 = 0;
    if (tid == 0 ? crosses[0] : crosses[1]) {
      const Left& r = s_left[tid == 0 ? 0 : open];
      const long long row0 = tid == 0 ? r.row0 : r.row1, row1 = row0 + (tid == 0 ? r.tiles0 : r.tiles1) - 1;
      const float per_tile = (float)ctas / (float)units;
      auto owner = [&](long long u) {  // CTA of tile u (in a row that boundaries cut, they have not moved): an estimate, set right
        int c = min((int)((float)u * per_tile), ctas - 1);
        while (begin_of(c) > u) --c;
        while (c + 1 < ctas && begin_of(c + 1) <= u) ++c;
        return c;
      };
      c0 = owner(row0);
      const int count = owner(row1) - c0 + 1;
      __threadfence();
      const unsigned seen = atomicAdd(P.arrived + c0, 1u);
      __threadfence();
      if (seen == (unsigned)count - 1) {
        joined = count;
        P.arrived[c0] = 0;
      }
    }
    s_flag[tid] = joined;
    s_flag[2 + tid] = c0;
  }
  __syncthreads();
  // The CTA that ends last is often the last of both its rows: then half of the warps take each.
  {
    const bool both = s_flag[0] != 0 && s_flag[1] != 0;
    const int team = both ? NT / 2 : NT, which = both ? tid / (NT / 2) : s_flag[0] != 0 ? 0 : 1, tt = both ? tid % (NT / 2) : tid;
    const int team_warp = tt / 32, team_warps = team / 32;
    auto sync = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(both ? 14 + which : 0), "r"(team) : "memory"); };
    const int count = s_flag[which], c0 = s_flag[2 + which];
    if (count == 0) return;
    const Left& by = s_left[which == 0 ? 0 : open];
    const int s = which == 0 ? by.s0 : by.s1, hk = which == 0 ? by.hk0 : by.hk1;
    const int block = which == 0 ? by.block0 : by.block1, rows = min(ROWS, P.group - block * ROWS);
    constexpr int kNext = 2 * H * C::kPart, WIDE = H * W / 4;
    constexpr int kJoin = 32768;  // bytes of a row's join: weights of up to kMaxCtas parts, and the groups' sums
    static_assert(ROWS * (kMaxCtas + 2) * 4 + 16 + NT * 16 <= kJoin && 2 * kJoin <= NW * (C::kRing + C::kPart * 4),
                  "two joins must fit what the ring and the parts took");
    const float* const rest = global_part(c0, 0);  // part i: of the row that came into CTA c0 + i
    const float* const head = global_part(c0, 1);  // part 0: of the row that CTA c0 left open
    // The row's float4s over groups of threads; a group takes every groups-th part, 12 loads at a time.  As many groups as
    // half a CTA has, also for a whole one: the order of the sums, and with it the bits, must not depend on who arrives last.
    const int wide = rows * WIDE, groups = wide <= NT / 4 ? NT / 2 / wide : 1, grp = groups == 1 ? 0 : tt / wide;
    float* const weight = reinterpret_cast<float*>(ring_mem + which * kJoin);  // [rows][count]
    float* const stat = weight + rows * count;                 // [rows][2]: max, sum
    float4* const sums = reinterpret_cast<float4*>(weight + ((rows * (count + 2) + 3) & ~3));
    auto part_of = [&](int i) { return i == 0 ? head : rest + (int64_t)i * kNext; };
    bool weighed = false;
    float m1 = -INFINITY, l1 = 0.f;  // of the first part whose weight this lane computes
    if (team_warp < rows && lane < count) {
      m1 = __ldcg(part_of(lane) + ROWS * W + team_warp);
      l1 = __ldcg(part_of(lane) + ROWS * W + ROWS + team_warp);
    }
#pragma unroll 1
    for (int e = tt - grp * wide; e - tt + grp * wide < wide; e += team) {
      const bool mine = e < wide && grp < groups;
      const int row = mine ? e / WIDE : 0, c = 4 * (e % WIDE);
      const int at = (c / W) * C::kPart + row * W + c % W;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int i0 = grp; i0 - grp < count; i0 += 12 * groups) {
        float4 y[12];
#pragma unroll
        for (int k = 0; k < 12; ++k) {
          const int i = i0 + k * groups;
          y[k] = load_part4(part_of(i) + at, mine && i < count);
        }
        if (!weighed) {
          // while those are on their way: the weights, a warp a head row
          weighed = true;
#pragma unroll 1
          for (int r = team_warp; r < rows; r += team_warps) {
            float M = -INFINITY, L = 0.f;
#pragma unroll 1
            for (int i = lane; i < count; i += 32) {
              if (r != team_warp || i != lane) {
                m1 = __ldcg(part_of(i) + ROWS * W + r);
                l1 = __ldcg(part_of(i) + ROWS * W + ROWS + r);
              }
              weight[r * count + i] = m1;
              const float now = fmaxf(M, m1), b = now == -INFINITY ? 0.f : now;
              L = fmaf(L, exp2_fast(M - b), l1 * exp2_fast(m1 - b));
              M = now;
            }
            float top = M;
#pragma unroll
            for (int by = 16; by > 0; by /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, by));
            const float b = top == -INFINITY ? 0.f : top;
            L *= exp2_fast(M - b);
#pragma unroll
            for (int by = 16; by > 0; by /= 2) L += __shfl_xor_sync(~0u, L, by);
#pragma unroll 1
            for (int i = lane; i < count; i += 32) weight[r * count + i] = exp2_fast(weight[r * count + i] - b);
            if (lane == 0) stat[2 * r] = top, stat[2 * r + 1] = L;
          }
          sync();
        }
#pragma unroll
        for (int k = 0; k < 12; ++k) {
          const int i = min(i0 + k * groups, count - 1);  // past the last, y is 0
          add(x, y[k], weight[row * count + i]);
        }
      }
      if (groups > 1) {  // the groups' sums in order
        if (mine) sums[tt] = x;
        sync();
#pragma unroll 1
        for (int k = 1; k < groups && grp == 0; ++k) add(x, sums[tt + k * wide], 1.f);
      }
      if (mine && grp == 0 && c < D)
        finish(s, (int64_t)hk * P.group + block * ROWS + row, c, x, stat[2 * row], stat[2 * row + 1]);
    }
  }
}

template <int F, bool SCORED, int W, int R, int H>
cudaError_t prepare_variant(const KvAttendPlan& p, int ctas, Launch* out) {
  using C = Config<F, W, R, H>;
  static std::atomic<unsigned long long> attr_set{0};  // one bit per device (setting it twice is harmless)
  const void* fn = reinterpret_cast<const void*>(kv_attend_kernel<F, SCORED, W, R, H>);
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

// The variant of a cache: heads of up to 64, 128 or (a pair of warps) 256 elements, in blocks of kRows query heads (R blocks of 8
// or, in columns, of 4).
template <int F, bool SCORED>
cudaError_t prepare_format(const KvAttendPlan& p, int dim, int blocks, int ctas, Launch* out) {
  auto of = [&](auto w, auto h) {
    constexpr int W = decltype(w)::value, H = decltype(h)::value;
    return blocks == 2 ? prepare_variant<F, SCORED, W, 2, H>(p, ctas, out) : prepare_variant<F, SCORED, W, 1, H>(p, ctas, out);
  };
  using std::integral_constant;
  if (dim == 256) return of(integral_constant<int, 128>{}, integral_constant<int, 2>{});
  if (dim == 128) return of(integral_constant<int, 128>{}, integral_constant<int, 1>{});
  return of(integral_constant<int, 64>{}, integral_constant<int, 1>{});
}

}  // namespace attend

// One translation unit each.
cudaError_t prepare_kv_attend_bf16(const KvAttendPlan& p, int dim, int blocks, int ctas, Launch* out);
cudaError_t prepare_kv_attend_q8(const KvAttendPlan& p, int dim, int blocks, int ctas, Launch* out);
cudaError_t prepare_kv_attend_a4(const KvAttendPlan& p, int dim, int blocks, int ctas, Launch* out);
cudaError_t prepare_kv_attend_bf16_scored(const KvAttendPlan& p, int dim, int blocks, int ctas, Launch* out);
cudaError_t prepare_kv_attend_q8_scored(const KvAttendPlan& p, int dim, int blocks, int ctas, Launch* out);
cudaError_t prepare_kv_attend_a4_scored(const KvAttendPlan& p, int dim, int blocks, int ctas, Launch* out);

}  // namespace il
