// kv_a4.cuh -- products with 4-bit rows of the cache (IL_A4: value d u + m, u of 0 .. 15) on m16n8k16 MMAs, for il_kv_attend
// (kv_attend.cuh) and il_kv_weigh; with 8-bit rows for il_kv_attend_scored and il_kv_weigh.
//
// Tokens (for q K^T) or elements of V (for p V) are the rows of an MMA, and each query head has two columns: the hi and the lo
// part of its fp32 operand, x = hi + lo 2^-11 in fp16.  The parts have accumulators of their own, so that lo is kept 2^11
// times as large: x keeps 22 bits down to 2^-27 of the largest and is cut at 2^-49 of it.  With four heads a K/V head nothing of
// an MMA is idle, a lane's accumulators are of one head (that of column pair q4 = lane % 4), and a softmax value is in one lane.
//
// Decoding K costs 6 instructions for 8 elements: nibbles at bits 2-5 and 6-9 of a 16-bit half are fp16 subnormals, 4 u 2^-24
// and 64 u 2^-24, exactly; two shifts bring all four there.  The factor 16 is taken from q.  (One shift would do for bits 0-3 and
// 4-7, but the MMAs line products up by the exponents as written and cut 25 bits below the largest: what subnormals lead with in
// zeros is lost.  A logit was off by 1e-6, now by 3e-7; higher bits gain nothing more, since q has 22.)  d multiplies a
// block's fp32 sum; the m of four blocks meet the sums of q over them, three bf16 parts each, in one MMA.
// V is taken as d (u - 8) + (m + 8 d), d multiplying p: sums of d u and of m over many tokens would each be far larger than the
// sum of V, and lose it (1e-5 of the result for 512 tokens; 6e-6 with sums that start at -8 times the weights').  u - 8
// costs 9 instructions for 8 elements, the sum of p (m + 8 d) 8 FMAs for 16 tokens.
#pragma once

#include "il_internal.cuh"

namespace il {
namespace a4 {

constexpr float kLoUnit = 1.f / 2048.f;  // of the lo part

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
// Transpose of an 8 x 8 matrix of 16-bit elements, one row in the four lanes of a quad.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Nibbles 0, 1, 2, 3 of both halves of w, as fp16 pairs of u 2^-22 (even) and 16 u 2^-22 (odd).
__device__ __forceinline__ void nibbles(uint32_t w, uint32_t (&p)[4]) {
  const uint32_t low = w << 2, high = w >> 6;
  p[0] = low & 0x003c003cu;
  p[1] = low & 0x03c003c0u;
  p[2] = high & 0x003c003cu;
  p[3] = high & 0x03c003c0u;
}

// The same nibbles as fp16 pairs of u - 8, by the known way with the exponent of 1024: the bits 64uu are 1024 + u, 6400 + 16 u are
// 1024 + 16 u.
__device__ __forceinline__ void nibbles_less_8(uint32_t w, uint32_t (&p)[4]) {
  const __half2 low = __floats2half2_rn(-1032.f, -1032.f), high = __floats2half2_rn(-72.f, -72.f);
  const __half2 sixteenth = __floats2half2_rn(0.0625f, 0.0625f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t u;  // (w & mask) | 0x64006400
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;"
        : "=r"(u)
        : "r"(i < 2 ? w : w >> 8), "r"(i % 2 == 0 ? 0x000f000fu : 0x00f000f0u), "r"(0x64006400u));
    const __half2 h = *reinterpret_cast<const __half2*>(&u);
    const __half2 v = i % 2 == 0 ? __hadd2(h, low) : __hfma2(h, sixteenth, high);
    p[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// c = A B of bf16, or c += A B; A's rows g and g + 8 hold pairs x, y in columns 2 q4 and 2 q4 + 8.
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t x0, uint32_t x1, uint32_t y0, uint32_t y1, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(x0), "r"(x1), "r"(y0), "r"(y1), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float step_of(uint32_t dm) { return __uint_as_float(dm << 16); }
__device__ __forceinline__ float least_of(uint32_t dm) { return __uint_as_float(dm & 0xffff0000u); }
__device__ __forceinline__ float middle_of(uint32_t dm) { return fmaf(8.f, step_of(dm), least_of(dm)); }

// Pairs of fp32 in one instruction each.
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(*reinterpret_cast<const uint64_t*>(&x)), "l"(*reinterpret_cast<const uint64_t*>(&y)));
  return *reinterpret_cast<const float2*>(&r);
}
__device__ __forceinline__ float2 sub2(float2 x, float2 y) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(*reinterpret_cast<const uint64_t*>(&x)), "l"(*reinterpret_cast<const uint64_t*>(&y)));
  return *reinterpret_cast<const float2*>(&r);
}

// u = {hi, lo 2^11} of x's first number, v of its second.
__device__ __forceinline__ void split2(float2 x, uint32_t& u, uint32_t& v) {
  const __half2 h = __floats2half2_rn(x.x, x.y);
  const float2 rest = mul2(sub2(x, __half22float2(h)), make_float2(2048.f, 2048.f));
  const __half2 l = __floats2half2_rn(rest.x, rest.y);
  const uint32_t hi = *reinterpret_cast<const uint32_t*>(&h), lo = *reinterpret_cast<const uint32_t*>(&l);
  u = __byte_perm(hi, lo, 0x5410);
  v = __byte_perm(hi, lo, 0x7632);
}

// The {d, m} of one token: NB of them in shared memory, 4 NB-byte aligned.
template <int NB>
__device__ __forceinline__ void load_steps(uint32_t (&dm)[NB], uint32_t at) {
  if constexpr (NB == 2) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(dm[0]), "=r"(dm[1]) : "r"(at));
  } else {
#pragma unroll
    for (int b = 0; b < NB; b += 4)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(dm[b]), "=r"(dm[b + 1]), "=r"(dm[b + 2]), "=r"(dm[b + 3])
                   : "r"(at + 4 * b));
  }
}

// Where 16-byte chunk `c` of row `row` is in a tile whose rows have CPR of them: eight rows of one chunk cover the banks.
template <int CPR>
__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
  return row * (16 * CPR) + ((c ^ (CPR >= 8 ? row & 7 : CPR == 4 ? (row >> 1) & 3 : (row >> 2) & 1)) << 4);
}

// Query heads of 4 R columns as B operands, scaled so that the largest of a head becomes 2^13 .. 2^14.
// FMAS: m by FMAs, 2 NB a head block, and not by an MMA.  What is faster depends on the kernel around it: il_kv_weigh, 64 ragged
// sequences, 45.7 us (by MMA 47.4), il_kv_attend 93.7 (93.1), two blocks of 4 heads 122.7 (117.3 when it was chosen, 123 now).
template <int NB, int R, bool FMAS = false>
struct Query {
  uint32_t f[R][4 * NB];  // of head 4 r + g / 2, its hi (g even) or lo part: elements 8 q4 .. 8 q4 + 7 of each block
  // The sums over the blocks, in the products' unit.  FMAS: of head 4 r + q4.  Else as a B operand whose rows are the same four
  // blocks' times three bf16 parts (in the lanes of a quad; hi's column only): blocks 4 i, 4 i + 1 in [2 i], and the next two
  uint32_t sum[R][FMAS ? NB : (NB + 1) / 2];
  float back[R][2];       // of head 4 r + q4: the unit, as two factors

  // Elements x[b][0 .. 7] = 8 q4 .. of block b, of head 4 r + g / 2; `top`: their largest magnitude over the whole head.
  __device__ __forceinline__ void take(int r, const float (&x)[NB][8], float top, int lane) {
    const int q4 = lane & 3, head_lane = q4 * 8;  // a lane with g / 2 = q4
    const bool lo_part = (lane >> 2) & 1;
    const int e = max((int)(__float_as_uint(top) >> 23), 14);
    const float up = __int_as_float((267 - e) << 23);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float total = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // nibble j of both halves of the lane's word: elements j, j + 4
        const float y = x[b][j] * up, z = x[b][j + 4] * up, sixteenth = j % 2 == 0 ? 1.f : 0.0625f;
        uint32_t u, v;
        split2(make_float2(y * sixteenth, z * sixteenth), u, v);
        f[r][4 * b + j] = lo_part ? __byte_perm(u, v, 0x7632) : __byte_perm(u, v, 0x5410);
        total += y + z;
      }
      total += __shfl_xor_sync(~0u, total, 1);
      total += __shfl_xor_sync(~0u, total, 2);
      total *= 2.384185791015625e-07f;  // 2^-22
      if constexpr (FMAS) {
        sum[r][b] = __float_as_uint(__shfl_sync(~0u, total, head_lane));
      } else {
        float part = 0.f;  // hi, mid or lo of it
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const float p = __bfloat162float(__float2bfloat16_rn(total));
          if (k == q4) part = p;
          total -= p;
        }
        const uint32_t bits = lo_part ? 0u : __float_as_uint(part);
        sum[r][b / 2] = b % 2 == 0 ? bits >> 16 : sum[r][b / 2] | bits;
      }
    }
    const int unit = __shfl_sync(~0u, e, head_lane) - 118, half = unit >> 1;  // 2^unit = 2^22 / up
    back[r][0] = __int_as_float((half + 127) << 23);
    back[r][1] = __int_as_float((unit - half + 127) << 23);
  }

  // s[r][h]: the product of head 4 r + q4 with token 8 h + g of 16, whose rows of K are at `tile` and steps at `steps`;
  // chunks[i]: where the lane's row of blocks 2 i and 2 i + 1 for ldmatrix lies from there, chunk_at(lane % 16, 2 i + lane / 16).
  __device__ __forceinline__ void dot(float (&s)[R][2], uint32_t tile, uint32_t steps, const uint32_t (&chunks)[NB / 2],
                                      int lane) const {
    const int g = lane >> 2;
    uint32_t d[2][NB];
    load_steps<NB>(d[0], steps + g * (4 * NB));
    load_steps<NB>(d[1], steps + (8 + g) * (4 * NB));
    auto pair = [&](int t, int b) { return b < NB ? __byte_perm(d[t][b], d[t][b + 1], 0x7632) : 0u; };  // {m, m}
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if constexpr (FMAS) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          s[r][t] = 0.f;
#pragma unroll
          for (int b = 0; b < NB; ++b) s[r][t] = fmaf(__uint_as_float(sum[r][b]), least_of(d[t][b]), s[r][t]);
        }
      } else {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int b = 0; b < NB; b += 4)
          mma_bf16(c, pair(0, b), pair(1, b), pair(0, b + 2), pair(1, b + 2), sum[r][b / 2], b + 2 < NB ? sum[r][b / 2 + 1] : 0u);
        s[r][0] = c[0], s[r][1] = c[2];
      }
    }
#pragma unroll
    for (int i = 0; i < NB / 2; ++i) {
      uint32_t w[4];  // tokens g and g + 8 of blocks 2 i and 2 i + 1
      ldmatrix4(w, tile + chunks[i]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int b = 2 * i + h;
        uint32_t x[4], y[4];
        nibbles(w[2 * h], x);
        nibbles(w[2 * h + 1], y);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float c[4];
          mma_first(c, x[0], y[0], x[1], y[1], f[r][4 * b], f[r][4 * b + 1]);
          mma(c, x[2], y[2], x[3], y[3], f[r][4 * b + 2], f[r][4 * b + 3]);
#pragma unroll
          for (int t = 0; t < 2; ++t) s[r][t] = fmaf(fmaf(c[2 * t + 1], kLoUnit, c[2 * t]), step_of(d[t][b]), s[r][t]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < 2; ++t) s[r][t] = s[r][t] * back[r][0] * back[r][1];
  }
};

// V's 8-bit elements 2 g and 2 g + 1 of a token pair (its bytes 0, 1 and 2, 3) as fp16 pairs over the tokens, exactly q.
__device__ __forceinline__ void bytes_of_pairs(uint32_t w, uint32_t& even, uint32_t& odd) {
  const uint32_t u = w ^ 0x80808080u;  // q + 128; the bits 64uu are 1024 + u
  const __half2 low = __floats2half2_rn(-1152.f, -1152.f);
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4240), b = __byte_perm(u, 0x64646464u, 0x4341);
  const __half2 x = __hadd2(*reinterpret_cast<const __half2*>(&a), low), y = __hadd2(*reinterpret_cast<const __half2*>(&b), low);
  even = *reinterpret_cast<const uint32_t*>(&x);
  odd = *reinterpret_cast<const uint32_t*>(&y);
}

// The same for 8-bit rows (IL_Q8: value d q), whose bytes u = q + 128 are fp16 subnormals u 2^-24 as they stand; the products with
// the 128 are taken off by where the sums start.
template <int NB, int R>
struct Query8 {
  // Of head 4 r + g / 2, its hi or lo part: of 16-element chunk i elements 4 q4, 4 q4 + 1 in [2 i], then the next two
  uint32_t f[R][4 * NB];
  float start[R][NB];     // of head 4 r + q4: -128 times the sum over a block, in the products' unit
  float back[R][2];

  // Elements x[b][0 .. 3] = 4 q4 .. of the first chunk of block b, x[b][4 .. 7] of the second.
  __device__ __forceinline__ void take(int r, const float (&x)[NB][8], float top, int lane) {
    const int q4 = lane & 3, head_lane = q4 * 8;
    const bool lo_part = (lane >> 2) & 1;
    const int e = max((int)(__float_as_uint(top) >> 23), 14);
    const float up = __int_as_float((267 - e) << 23);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float total = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float y = x[b][2 * j] * up, z = x[b][2 * j + 1] * up;
        uint32_t u, v;
        split2(make_float2(y, z), u, v);
        f[r][4 * b + j] = lo_part ? __byte_perm(u, v, 0x7632) : __byte_perm(u, v, 0x5410);
        total += y + z;
      }
      total += __shfl_xor_sync(~0u, total, 1);
      total += __shfl_xor_sync(~0u, total, 2);
      start[r][b] = __shfl_sync(~0u, total, head_lane) * -7.62939453125e-06f;  // -128 2^-24
    }
    const int unit = __shfl_sync(~0u, e, head_lane) - 116, half = unit >> 1;  // 2^unit = 2^24 / up
    back[r][0] = __int_as_float((half + 127) << 23);
    back[r][1] = __int_as_float((unit - half + 127) << 23);
  }

  __device__ __forceinline__ void dot(float (&s)[R][2], uint32_t tile, uint32_t steps, const uint32_t (&chunks)[NB], int lane) const {
    const int g = lane >> 2;
    uint32_t d[2][NB];
    load_steps<NB>(d[0], steps + g * (4 * NB));
    load_steps<NB>(d[1], steps + (8 + g) * (4 * NB));
#pragma unroll
    for (int r = 0; r < R; ++r) s[r][0] = s[r][1] = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint32_t w[4];  // tokens g and g + 8 of chunk 2 b, then of 2 b + 1
      ldmatrix4(w, tile + chunks[b]);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] ^= 0x80808080u;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float c[4] = {start[r][b], 0.f, start[r][b], 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h)
          mma(c, __byte_perm(w[2 * h], 0u, 0x4140), __byte_perm(w[2 * h + 1], 0u, 0x4140), __byte_perm(w[2 * h], 0u, 0x4342),
              __byte_perm(w[2 * h + 1], 0u, 0x4342), f[r][4 * b + 2 * h], f[r][4 * b + 2 * h + 1]);
#pragma unroll
        for (int t = 0; t < 2; ++t) s[r][t] = fmaf(fmaf(c[2 * t + 1], kLoUnit, c[2 * t]), __uint_as_float(d[t][b]), s[r][t]);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < 2; ++t) s[r][t] = s[r][t] * back[r][0] * back[r][1];
  }
};

}  // namespace a4
}  // namespace il
