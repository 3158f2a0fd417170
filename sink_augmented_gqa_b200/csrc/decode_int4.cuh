// One-token decode over an INT4 cache (int4.cuh). As in decode_kernel
// (decode.cuh) a producer warp streams the rows through a ring of stages and
// the consumer warps attend them, but with 4.5 bits an element the arithmetic
// per byte is about four times that of a bf16 cache: of all units the issue
// slots and the ALU pipe (half their rate) are the busiest, at about 60 % with
// the four or five warps a scheduler has to hide latency with, and memory after
// them. So the codes go to the tensor cores with as few instructions as
// possible, and every SM gets the same number of rows. 16 sequences of 65,536
// rows, 64 query and 8 KV heads of 64: 127 us back to back (4.7 TB/s).
//
// One CTA per SM, 16 consumer warps (d = 128: 12) that take 32 rows each of a
// 512-row (384-row) stage (with two CTAs of 8 per SM the scheduler's older one
// ran ahead and left the other half of the SM's warps for the last fifth of the
// time). A (sequence,
// KV head) pair's rows count in units of 128. Where the CTAs can be dealt out
// to the pairs evenly, each pair gets S of them; else the units of all pairs
// lie in one row and every CTA takes an equal, contiguous share (plan_decode
// chooses). A share can end one pair, span several and begin another. Nothing
// of that holds up the rows: the producer streams on across the border, and
// three warps beside it make the next pair's queries into fragments, quantise
// the new row, and merge what the consumers left of the last pair
// (decode_finish). The last pair of a CTA, with nothing behind it, the
// consumers merge themselves.
//
// S^T = K Q^T, m16n8k16 in f16, 16 keys on the M side, the group's heads on the
// N side: a code word w (8 nibbles) gives four f16 pairs by masks and one
//   shift: w & 0x000F000F as f16 are the subnormals u 2^-24 of nibbles 0 and 4,
//   w & 0x00F000F0 those of nibbles 1 and 5 times 16, and the same of w >> 8.
//   The queries' fragments take that order, 1/16 in every second register;
//   they are f16 after a power-of-two scaling per head, exact for bf16 queries
//   down to 2^-25 of the largest. A block's scale multiplies its partial sums
//   afterwards in fp32. The codes' offset of 8, scale * (-8 sum of q) over the
//   blocks, is one more product in bf16 (the scales as stored against the
//   queries' sums in three bf16 parts) and what the fp32 sums start from.
//   (m16n8k32 in e4m3 reads a byte 0000uuuu as u 2^-9 and needs half of the
//   masks, but runs here as conversions and two f16 products and was no faster:
//   166 us against 160 of f16 at 16 sequences of 65,536 rows, in an earlier form
//   of this kernel.)
// O^T += V^T P'^T, m16n8k16 in f16, P' = p * scale_v, transposed by movmatrix:
//   ldmatrix.trans over 16-bit units hands a lane the same 4 codes of two
//   neighbouring keys; x & 0x000F000F as f16 are the subnormals u 2^-24 of
//   the first, x & 0x00F000F0 16 times those of the second, and x >> 8 gives
//   the other two: 5 instructions for 8 codes (bf16, whose 7 fraction bits
//   hold one code, takes 7). The offset of 8 goes out at the end, by the sums
//   of P' in fp32: of P' as rounded to f16, so that a key whose P' is rounded
//   (to nothing, even) is wrong by that much of its value and no more.
// p is relative to 2^ref, ref a score of the head that no score so far has
//   exceeded by more than 8 (log2 units); the sum of p, the merge and the lse
//   know nothing of V. P' has a power of two of its own for each block of 32
//   elements and each head, f = 2^(6 - E): blocks and heads do not share one,
//   since what is large in one may be nothing in another. 2^E is 16 times the
//   largest p |scale_v| (rounded down to a power of two) found where E last
//   moved, so a row of negligible weight does not set it, however large; it
//   moves with ref, up and down, and up where a |scale_v| exceeds 2^(E + 1).
//   In a tile where none does, P' < 2^(8 + E + 1) f = 2^15, which f16 holds;
//   in one where E moves, P' is at most 2^3. Scales that are no numbers move
//   nothing: p times such a scale carries the NaN to its own block. f16's 11
//   bits reach down to 2^-16 of the largest product, its last one to 2^-26.
//   ref and E move only when a tile breaks one of the two bounds, so a tile needs
//   no maximum across lanes, only a vote.
#pragma once

#include <math.h>

#include "decode.cuh"
#include "int4.cuh"

namespace sa {

template <int D>
struct DecodeI4Cfg {
  // Consumer warps, 32 rows of a stage each. d = 128 holds 16 registers of sums and
  // queries for each of four blocks: 12 warps of 144 registers (16 sequences of
  // 16,384 rows, 64 / 8 heads: 71.8 us) rather than 16 of 104, which spill (103).
  // d = 64 the other way round: 16 of 65,536 rows 138 us with 16 warps, 150 with
  // 12. d = 96 has room in 104: 16 of 30,000 rows, 16 / 4 heads, 54.8 against 55.5.
  static constexpr int NCW = D == 128 ? 12 : 16;
  static constexpr int UNIT = 128;              // rows that shares count in
  static constexpr int R = 32 * NCW;            // rows per stage
  static constexpr int NB = D / kI4Block;       // blocks per row
  static constexpr int ROWB = D / 2;            // code bytes per row
  static constexpr uint32_t STAGE_BYTES = R * ROWB;
  static constexpr uint32_t SC_BYTES = R * NB * 2;   // K (or V) scales of one stage
  static constexpr int NS = (D == 64) ? 5 : 3;
  static constexpr uint32_t STAGE_TX = 2 * (STAGE_BYTES + SC_BYTES);
  // warpgroups of consumers, and one of the producer and the three warps beside
  // it, which gives registers to the others (640 * 96 at launch, 512 * 104 + 128
  // * 64 after; d = 128: 512 * 128, 384 * 144 + 128 * 64)
  static constexpr int NUM_THREADS = 32 * (NCW + 4);
  static constexpr int HELPERS = 96;
  static constexpr int REGS_CONSUMER = D == 128 ? 144 : 104, REGS_PRODUCER = 64;
  // K codes of the stages, then a tile of 32 rows for the new row (row 0
  // valid); the same of V; scales likewise ([R][NB] bf16 a stage)
  static constexpr uint32_t XTILE = (32 * ROWB + 1023) / 1024 * 1024;
  static constexpr uint32_t XSC = 32 * NB * 2;
  static constexpr uint32_t OFF_K = 0;
  static constexpr uint32_t OFF_XK = NS * STAGE_BYTES;
  static constexpr uint32_t OFF_V = OFF_XK + XTILE;
  static constexpr uint32_t OFF_XV = OFF_V + NS * STAGE_BYTES;
  static constexpr uint32_t RING_BYTES = OFF_XK;                 // K's: takes the records of the last merge
  static constexpr uint32_t OFF_KS = OFF_XV + XTILE;
  static constexpr uint32_t OFF_XS = OFF_KS + NS * SC_BYTES;
  static constexpr uint32_t OFF_VS = OFF_XS + XSC;
  static constexpr uint32_t OFF_XVS = OFF_VS + NS * SC_BYTES;
  // [NCW warps][8 m | 8 l | 8*D O] fp32, then the records of a merge
  static constexpr uint32_t RED_WARP = (16 + 8 * D) * 4;
  static constexpr uint32_t OFF_RED = OFF_XVS + XSC;
  static constexpr uint32_t RED_BYTES = NCW * RED_WARP;
  // two pairs' queries: fragment words [8][D / 8] uint4, the sums of their 8
  // elements [8][D / 8] fp32, score scales [8], sinks [8]
  static constexpr uint32_t OFF_Q = OFF_RED + RED_BYTES;
  static constexpr uint32_t Q_SUM = 8 * D * 2, Q_HS = Q_SUM + D * 4, Q_SINK = Q_HS + 32, Q_BYTES = Q_SINK + 32;
  static constexpr uint32_t OFF_XROW = OFF_Q + 2 * Q_BYTES;      // the new K row, rotated, bf16
  static constexpr uint32_t OFF_BAR = OFF_XROW + D * 2;
  static constexpr uint32_t OFF_FLAG = OFF_BAR + 8 * (2 * NS + 7);
  static constexpr uint32_t SMEM_BYTES = OFF_FLAG + 16 + 1024;
  static_assert(SMEM_BYTES <= 232448, "dynamic shared memory per block");
  static_assert(9 * 8 <= HELPERS && D / 16 <= 8, "the helpers rotate the rows, eight lanes each");
  static_assert(STAGE_BYTES % 1024 == 0, "swizzled tiles start on a multiple of their pattern");
  static_assert(OFF_BAR % 16 == 0 && OFF_KS % 16 == 0 && OFF_VS % 16 == 0 && SC_BYTES % 16 == 0 && OFF_RED % 16 == 0,
                "barriers and bulk copies");
  static_assert(OFF_XV - OFF_XK == OFF_V - OFF_K && OFF_XVS - OFF_XS == OFF_VS - OFF_KS, "the new row's tile");
  static_assert(OFF_Q % 16 == 0 && Q_BYTES % 16 == 0 && OFF_BAR % 8 == 0, "alignment");
};

// Byte offset of 16-byte block blk of a row in a tile. The rows lie end to
// end in 128-byte lines, which TMA brings as such (a box of 32- to 64-byte
// rows moves a third as fast: 253 us against 115 for 16 sequences of 65,536
// rows, d = 64): with the 128-byte swizzle for 32- and 64-byte rows, plain
// for 48-byte rows. In each, the eight rows an ldmatrix phase reads lie in
// distinct banks.
template <int D>
__device__ __forceinline__ uint32_t i4_off(int row, int blk) {
  const uint32_t n = (uint32_t)row * (D / 32) + blk;   // 16-byte chunk
  const uint32_t line = n >> 3;
  return line * 128 + (((n & 7) ^ (D == 96 ? 0u : line & 7)) << 4);
}

// d = A B, 16 x 8 x 16, fp32 accumulators.
__device__ __forceinline__ void mma_16816_f16_0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_16816_bf16_0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                 uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// d = A B, bf16, 16 x 8 x 8.
__device__ __forceinline__ void mma_1688_bf16_0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%7, %7, %7, %7};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(b0), "f"(0.f));
}

// Loads at addr + OFF bytes: the offset belongs to the instruction.
template <uint32_t OFF>
__device__ __forceinline__ void ldmatrix_x4_at(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4 + %5];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr), "n"(OFF));
}
template <uint32_t OFF>
__device__ __forceinline__ void ldmatrix_x4_trans_at(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4 + %5];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr), "n"(OFF));
}

// A row's block scales as words (bf16 pairs; the last one's upper half 0 where
// the blocks are odd), and block blk's of them as fp32.
template <int NB, uint32_t OFF>
__device__ __forceinline__ void i4_row_scales(uint32_t addr, uint32_t (&w)[(NB + 1) / 2]) {
  if constexpr (NB == 2) {
    asm volatile("ld.shared.u32 %0, [%1 + %2];" : "=r"(w[0]) : "r"(addr), "n"(OFF));
  } else if constexpr (NB == 4) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2 + %3];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr), "n"(OFF));
  } else {
    uint16_t h[3];
    asm volatile("ld.shared.u16 %0, [%1 + %2];" : "=h"(h[0]) : "r"(addr), "n"(OFF));
    asm volatile("ld.shared.u16 %0, [%1 + %2];" : "=h"(h[1]) : "r"(addr), "n"(OFF + 2));
    asm volatile("ld.shared.u16 %0, [%1 + %2];" : "=h"(h[2]) : "r"(addr), "n"(OFF + 4));
    w[0] = (uint32_t)h[0] | (uint32_t)h[1] << 16;
    w[1] = h[2];
  }
}
// The scales of rows 8 c + r, c < 4, from row r's address on.
template <int NB, uint32_t OFF>
__device__ __forceinline__ void i4_tile_scales(uint32_t addr, uint32_t (&w)[4][(NB + 1) / 2]) {
  i4_row_scales<NB, OFF>(addr, w[0]);
  i4_row_scales<NB, OFF + 16 * NB>(addr, w[1]);
  i4_row_scales<NB, OFF + 32 * NB>(addr, w[2]);
  i4_row_scales<NB, OFF + 48 * NB>(addr, w[3]);
}
__device__ __forceinline__ float i4_scale(const uint32_t* w, int blk) {
  return (blk & 1) ? bf16_hi(w[blk >> 1]) : bf16_lo(w[blk >> 1]);
}

// What a consumer warp keeps of its (b, g). Of heads 2 (lane % 4) + {0, 1}: the
// score scale hs, ref (see the head of this file; 0 while no key has been seen) and
// the unscaled score thr = (ref + 8) / hs that moves it (-inf while none has); the
// running sum l (over this lane's keys), and for each block f and the sum of P',
// ps. qf: the query fragments, qo: the offset's. lim: the blocks' 2^(E + 1), the
// lesser of the two heads', as bf16 pairs like the scales. o[blk][i]: the
// accumulators of d = 32 blk + 4 (lane / 4) + 2 i + {0, 1} (fragment rows g and g +
// 8, the latter times 16), offset included, times f 2^-24.
template <int D>
struct I4State {
  static constexpr int NB = D / kI4Block;
  uint32_t qf[NB][4];
  uint32_t qo[2];
  uint32_t lim[(NB + 1) / 2];
  float hs[2], ref[2], thr[2], l[2];
  float f[NB][2], ps[NB][2], o[NB][2][4];
};

// E within [-120, 126], so that f and 1 / f are normal numbers.
constexpr int kI4MinE = -120, kI4MaxE = 126;

// The largest of x over the lanes with the same heads.
__device__ __forceinline__ float i4_max8(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}

// ref and E after a tile that broke one of the bounds: s its scores, mx their
// largest in this lane, sw its scales of V. E is what the tile's products ask
// for, or what it was less the rise of ref.
template <int D>
__device__ __forceinline__ void i4_move(I4State<D>& z, const float (&s)[2][4], const float (&mx)[2],
                                        const uint32_t (&sw)[4][(D / 32 + 1) / 2]) {
  constexpr int NB = D / 32;
  float p[4][2], down[2];   // down: log2 of what becomes of the sums so far
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float x = i4_max8(mx[e]) * z.hs[e];
    const bool empty = z.thr[e] == -INFINITY;
    const float m = empty ? x : fmaxf(z.ref[e], x);
    const float ref = m == -INFINITY ? 0.f : m;
    down[e] = empty ? 0.f : z.ref[e] - ref;
    z.ref[e] = ref;
    z.thr[e] = __fdividef(m + 8.f, z.hs[e]);
    z.l[e] *= ex2(down[e]);
#pragma unroll
    for (int c = 0; c < 4; ++c) p[c][e] = ex2(fmaf(s[c >> 1][2 * (c & 1) + e], z.hs[e], -ref));
  }
#pragma unroll
  for (int blk = 0; blk < NB; ++blk) {
    float w[2] = {};   // the largest products, of which the upper halves go across the lanes
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float v = fabsf(i4_scale(sw[c], blk));
      w[0] = fmaxf(w[0], p[c][0] * v);   // (a NaN counts for nothing)
      w[1] = fmaxf(w[1], p[c][1] * v);
    }
    uint32_t top = __byte_perm(__float_as_uint(w[0]), __float_as_uint(w[1]), 0x7632);
#pragma unroll
    for (int i = 4; i < 32; i <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, i));
    int E[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int asked = (int)(top >> (16 * e + 7) & 0xFFu) - 123;
      const int was = 133 - (int)(__float_as_uint(z.f[blk][e]) >> 23);
      E[e] = min(max(max(asked, was + __float2int_rn(fmaxf(down[e], -512.f))), kI4MinE), kI4MaxE);
      const float al = ex2(down[e] + (float)(was - E[e]));
      z.f[blk][e] = __uint_as_float((uint32_t)(133 - E[e]) << 23);
      z.ps[blk][e] *= al;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        z.o[blk][i][e] *= al;
        z.o[blk][i][2 + e] *= al;
      }
    }
    const uint32_t lim = (uint32_t)(min(E[0], E[1]) + 128) << 7;
    z.lim[blk >> 1] = (blk & 1) ? z.lim[blk >> 1] | lim << 16 : lim;
  }
}

// One warp's 32 keys of a stage: K codes at kst plus this lane's offsets
// off[blk] (of row `lane`), V codes VC bytes behind; K scales of row lane / 4 at
// ksc, V's VS bytes behind. With MASK, keys below n_first and from n_valid on
// are masked (their scales may hold anything).
template <int D, bool MASK, uint32_t VC, uint32_t VS>
__device__ __forceinline__ void decode_tile_i4(uint32_t kst, const uint32_t (&off)[D / 32], uint32_t ksc, int n_first,
                                               int n_valid, I4State<D>& z, int lane) {
  constexpr int NB = D / 32, NW = (NB + 1) / 2;
  constexpr uint32_t M0 = 0x000F000Fu, M1 = 0x00F000F0u;
  const int r = lane >> 2, t = lane & 3;
  bool ok[4];   // key 8 c + r
#pragma unroll
  for (int c = 0; c < 4; ++c) ok[c] = !MASK || (8 * c + r >= n_first && 8 * c + r < n_valid);
  float s[2][4];   // keys 16 j + r (0, 1) and + 8 (2, 3), heads 2 t + {0, 1}
  uint32_t sw[4][NW];
  i4_tile_scales<NB, 0>(ksc, sw);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if constexpr (NB == 2) {
      mma_1688_bf16_0(s[j], sw[2 * j][0], sw[2 * j + 1][0], z.qo[0]);
      continue;
    }
    const uint32_t a0 = (NW == 2 && (t & 1)) ? sw[2 * j][NW - 1] : sw[2 * j][0];
    const uint32_t a1 = (NW == 2 && (t & 1)) ? sw[2 * j + 1][NW - 1] : sw[2 * j + 1][0];
    mma_16816_bf16_0(s[j], a0, a1, a0, a1, z.qo[0], z.qo[1]);
  }
#pragma unroll
  for (int blk = 0; blk < NB; ++blk) {
    uint32_t w[4];
    ldmatrix_x4_at<0>(kst + off[blk], w);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float a[4];
      const uint32_t w0 = w[2 * j], w1 = w[2 * j + 1];
      mma_16816_f16_0(a, w0 & M0, w1 & M0, w0 & M1, w1 & M1, z.qf[blk][0], z.qf[blk][1]);
      const uint32_t v0 = w0 >> 8, v1 = w1 >> 8;
      mma_16816_f16(a, v0 & M0, v1 & M0, v0 & M1, v1 & M1, z.qf[blk][2], z.qf[blk][3]);
      const float k0 = i4_scale(sw[2 * j], blk), k1 = i4_scale(sw[2 * j + 1], blk);
      s[j][0] = fmaf(a[0], k0, s[j][0]);
      s[j][1] = fmaf(a[1], k0, s[j][1]);
      s[j][2] = fmaf(a[2], k1, s[j][2]);
      s[j][3] = fmaf(a[3], k1, s[j][3]);
    }
  }
  uint32_t mag[NW] = {};   // the largest |scale_v| of each block
  i4_tile_scales<NB, VS>(ksc, sw);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      if (MASK && !ok[c]) sw[c][i] = 0;   // a row never written holds anything
      mag[i] = __vmaxu2(mag[i], sw[c][i] & 0x7FFF7FFFu);
    }
  }
  float mx[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (MASK) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (!ok[c]) s[c >> 1][2 * (c & 1) + e] = -INFINITY;
    }
    mx[e] = fmaxf(max3f(s[0][e], s[0][2 + e], s[1][e]), s[1][2 + e]);
  }
  bool move = mx[0] > z.thr[0] || mx[1] > z.thr[1];
#pragma unroll
  for (int i = 0; i < NW; ++i) move = move || __vmaxu2(mag[i], z.lim[i]) != z.lim[i];
  if (__any_sync(0xffffffffu, move)) i4_move<D>(z, s, mx, sw);
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[j][i] = ex2(fmaf(s[j][i], z.hs[i & 1], -z.ref[i & 1]));
      z.l[i & 1] += s[j][i];
    }
#pragma unroll
  for (int blk = 0; blk < NB; ++blk) {
    uint32_t x[4], pb[4];   // pb: P' of octet c, f16
    ldmatrix_x4_trans_at<VC>(kst + off[blk], x);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      // (in this order: f times the scale of a row without weight may be infinite)
      const float v = i4_scale(sw[c], blk);
      float p0 = s[c >> 1][2 * (c & 1)], p1 = s[c >> 1][2 * (c & 1) + 1];
      mul2(p0, p1, v, v);
      mul2(p0, p1, z.f[blk][0], z.f[blk][1]);
      const uint32_t ph = pack_f16(p0, p1);
      add_f16x2(z.ps[blk][0], z.ps[blk][1], ph);
      pb[c] = movmatrix_trans(ph);
    }
#pragma unroll
    for (int c = 0; c < 4; c += 2) {
      mma_16816_f16(z.o[blk][0], x[c] & M0, x[c] & M1, x[c + 1] & M0, x[c + 1] & M1, pb[c], pb[c + 1]);
      const uint32_t y0 = x[c] >> 8, y1 = x[c + 1] >> 8;
      mma_16816_f16(z.o[blk][1], y0 & M0, y0 & M1, y1 & M0, y1 & M1, pb[c], pb[c + 1]);
    }
  }
}

// fp32 x as three bf16 parts, x = sum of them to 2^-24 of x.
__device__ __forceinline__ void i4_split3(float x, uint32_t (&part)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    part[i] = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(x));
    x -= __uint_as_float(part[i] << 16);
  }
}

// Eight lanes of a warp (ch = lane % 8; those with ch >= D / 16 idle) make one
// query row's fragment words: x1, x2 its rotated elements 8 ch.. and D / 2 + 8
// ch... qw, qsum: the row's entries of 8 elements each. Returns the row's score
// scale.
template <int D>
__device__ __forceinline__ float i4_query(uint4 x1, uint4 x2, int ch, uint4* qw, float* qsum, float scale_log2) {
  float v[2][8];
  const uint32_t w[2][4] = {{x1.x, x1.y, x1.z, x1.w}, {x2.x, x2.y, x2.z, x2.w}};
  float amax = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[h][i] = (i & 1) ? bf16_hi(w[h][i >> 1]) : bf16_lo(w[h][i >> 1]);
      amax = fmaxf(amax, fabsf(v[h][i]));
    }
#pragma unroll
  for (int i = 1; i < 8; i <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, i));
  // the row's largest |q| goes to [2^14, 2^15)
  int eq = 0;
  if (amax > 0.f) {
    eq = (int)((__float_as_uint(amax) >> 23) & 0xFFu) - 127 - 14;
    eq = eq < -100 ? -100 : (eq > 100 ? 100 : eq);
  }
  const float down = __uint_as_float((uint32_t)(127 - eq) << 23);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[h][i] *= down;
      sum += v[h][i];
    }
    if (ch < D / 16) {
      // elements {0, 4}, {1, 5}, {2, 6}, {3, 7}; nibbles 1, 3, 5, 7 enter times 16
      qw[ch + h * (D / 16)] = make_uint4(pack_f16(v[h][0], v[h][4]), pack_f16(v[h][1] * 0.0625f, v[h][5] * 0.0625f),
                                         pack_f16(v[h][2], v[h][6]), pack_f16(v[h][3] * 0.0625f, v[h][7] * 0.0625f));
      qsum[ch + h * (D / 16)] = sum;
    }
  }
  return scale_log2 * __uint_as_float((uint32_t)(127 + eq) << 23) * 0x1p24f;
}

// A warp's share of the rows made by i4_query (B operand: head lane / 4, 8
// elements t = lane % 4 of every block), and empty sums.
template <int D>
__device__ __forceinline__ void i4_start(I4State<D>& z, const uint4* qw, const float* qsum, const float* hs, int QM,
                                         int lane) {
  constexpr int NB = D / kI4Block;
  const int n = lane >> 2, t = lane & 3;
  uint32_t part[4][3] = {};   // of block blk's offset, bf16
#pragma unroll
  for (int blk = 0; blk < NB; ++blk) {
    uint4 u = make_uint4(0, 0, 0, 0);
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (n < QM) {
      u = qw[n * (D / 8) + 4 * blk + t];
      f = *reinterpret_cast<const float4*>(qsum + n * (D / 8) + 4 * blk);
    }
    z.qf[blk][0] = u.x;
    z.qf[blk][1] = u.y;
    z.qf[blk][2] = u.z;
    z.qf[blk][3] = u.w;
    i4_split3(((f.x + f.y) + (f.z + f.w)) * (-8.0f * 0x1p-24f), part[blk]);
  }
  // The offset's B operand against a row's scale words w (A operand): two
  // blocks: lane t has w and part t; more: word t & 1, in register 0 part
  // t >> 1, in register 1 part 2 (t < 2).
  if (NB == 2) {
    z.qo[0] = t == 0 ? part[0][0] | part[1][0] << 16
                     : (t == 1 ? part[0][1] | part[1][1] << 16 : (t == 2 ? part[0][2] | part[1][2] << 16 : 0u));
    z.qo[1] = 0;
  } else {
    uint32_t wp[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) wp[i] = (t & 1) ? part[2][i] | part[3][i] << 16 : part[0][i] | part[1][i] << 16;
    z.qo[0] = t < 2 ? wp[0] : wp[1];
    z.qo[1] = t < 2 ? wp[2] : 0u;
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    z.hs[e] = 2 * t + e < QM ? hs[2 * t + e] : 1.f;
    z.thr[e] = -INFINITY;
    z.ref[e] = 0.f;
    z.l[e] = 0.f;
  }
#pragma unroll
  for (int blk = 0; blk < NB; ++blk) {
    z.lim[blk >> 1] = (uint32_t)(kI4MinE + 128) * 0x00800080u;   // 2^(E + 1), twice
    z.f[blk][0] = z.f[blk][1] = __uint_as_float((uint32_t)(133 - kI4MinE) << 23);
    z.ps[blk][0] = z.ps[blk][1] = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) z.o[blk][i][0] = z.o[blk][i][1] = z.o[blk][i][2] = z.o[blk][i][3] = 0.f;
  }
}

// The warp's partial as decode_finish takes it.
template <int D>
__device__ __forceinline__ void i4_write_partial(const I4State<D>& z, float* rw, int lane) {
  constexpr int NB = D / kI4Block;
  const int t = lane & 3, r = lane >> 2;
  // over the lanes with the same heads
  auto sum8 = [](float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
  };
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float l = sum8(z.l[e]);
    if (r == 0) {
      rw[2 * t + e] = z.thr[e] == -INFINITY ? -INFINITY : z.ref[e];
      rw[8 + 2 * t + e] = l;
    }
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      const float c = -8.f * sum8(z.ps[blk][e]);   // the codes' offset
      const float unit = __uint_as_float((254u << 23) - __float_as_uint(z.f[blk][e]));   // 1 / f
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<float2*>(rw + 16 + (2 * t + e) * D + 32 * blk + 4 * r + 2 * i) =
            make_float2(fmaf(z.o[blk][i][e], 0x1p24f, c) * unit, fmaf(z.o[blk][i][2 + e], 0x1p20f, c) * unit);
    }
  }
}

// tmK / tmV: the codes, dims {128, lines, n_kv, B} bytes, boxes of a stage's
// rows; tmK1 / tmV1: the same with boxes of 128 rows. p.ck, p.cv, p.cks, p.cvs
// hold the cache's code and scale arrays. p.units units of 128 rows in all, per
// pair p.n_blocks (one at least); p.S > 0: S CTAs per pair, else equal shares.
template <int D>
__global__ void __launch_bounds__(DecodeI4Cfg<D>::NUM_THREADS, 1)
    decode_i4_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmK1, const __grid_constant__ CUtensorMap tmV1,
                     const DecodeParams p) {
  using C = DecodeI4Cfg<D>;
  constexpr int NB = C::NB, HALF = D / 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto full_bar = [&](int s) -> uint32_t { return bar0 + 8u * (uint32_t)s; };
  auto empty_bar = [&](int s) -> uint32_t { return bar0 + 8u * (uint32_t)(C::NS + s); };
  // a pair's queries ready (two buffers), its partials written, read again,
  // its new row ready, and the barriers of the two merges' copies
  auto q_bar = [&](int i) -> uint32_t { return bar0 + 8u * (uint32_t)(2 * C::NS + (i & 1)); };
  const uint32_t part_bar = bar0 + 8u * (2 * C::NS + 2), free_bar = part_bar + 8, row_bar = part_bar + 16,
                 merge_bar = part_bar + 24, last_merge_bar = part_bar + 32;
  // flag[0]: a wait ran out, and no rows are brought or attended any more;
  // flag[1], flag[2]: "this CTA merges the pair's records"
  volatile int* flag = reinterpret_cast<volatile int*>(smem + C::OFF_FLAG);
  const float* red = reinterpret_cast<const float*>(smem + C::OFF_RED);
  auto q_buf = [&](int i) -> uint8_t* { return smem + C::OFF_Q + (uint32_t)(i & 1) * C::Q_BYTES; };

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int QM = p.q_mult;
  const int per = p.n_blocks > 0 ? (int)p.n_blocks : 1;   // units of a pair

  // This CTA's units [u0, u1) of the row of all, and who holds unit u.
  const int cta = blockIdx.x, base = p.units / (int)gridDim.x, rem = p.units - base * (int)gridDim.x;
  int u0, u1;
  if (p.S > 0) {
    const int pair = cta / p.S, i = cta - pair * p.S;
    u0 = pair * per + (int)((long long)i * per / p.S);
    u1 = pair * per + (int)((long long)(i + 1) * per / p.S);
  } else {
    u0 = cta * base + min(cta, rem);
    u1 = u0 + base + (cta < rem ? 1 : 0);
  }
  auto holder = [&](int u) -> int {
    const int cut = rem * (base + 1);
    return u < cut ? u / (base + 1) : rem + (u - cut) / base;
  };
  int bg = u0 / per, b = bg / p.n_kv, g = bg - b * p.n_kv;

  // Brings rows [pos, pos + n) of pair (sequence b, KV head g), n > 0, through
  // load(map, row, bytes of codes before, rows of the box) and scales(row,
  // rows before, rows): one box for a whole stage of a linear cache, else
  // boxes of 128 rows. pos is a multiple of 128 on a ring, whose capacity is
  // one too, so that none wraps; scales come in whole groups of 16 rows (cap
  // is a multiple of 16).
  auto for_boxes = [&](long long pos, int n, auto&& load, auto&& scales) {
    if (p.ring_cap == 0) {
      if (n == C::R)
        load(&tmK, &tmV, (int)pos, 0);
      else
        for (int r = 0; r < n; r += 128) load(&tmK1, &tmV1, (int)pos + r, r);
      scales((int)pos, 0, (n + 15) / 16 * 16);
    } else {
      for (int r = 0; r < n; r += 128) {
        const int row = (int)((pos + r) % p.ring_cap);
        load(&tmK1, &tmV1, row, r);
        scales(row, r, 128);
      }
    }
  };
  const char* ksc_g = reinterpret_cast<const char*>(p.cks);
  const char* vsc_g = reinterpret_cast<const char*>(p.cvs);

  // The rows that the helpers rotate for a pair, 16 elements (8 RoPE pairs) a
  // thread, 8 lanes a row: the group's queries, then the new K row.
  const int htid = (int)threadIdx.x - 32 * (C::NCW + 1);
  const int rot_row = htid >> 3, rot_ch = htid & 7;
  const bool rot_in = htid >= 0 && rot_row <= QM && rot_ch < D / 16;
  auto rot_src = [&]() -> const __nv_bfloat16* {
    return 8 * rot_ch + (rot_row < QM ? p.q + b * p.qs0 + (long long)(g * QM + rot_row) * p.qs2
                                      : p.k + b * p.ks0 + (long long)g * p.ks2);
  };
  const float* ctab = p.cos_t + p.off * HALF + 8 * rot_ch;
  const float* stab = p.sin_t + p.off * HALF + 8 * rot_ch;
  auto next_pair = [&]() {
    ++bg;
    if (++g == p.n_kv) {
      g = 0;
      ++b;
    }
  };
  // The pair's CTAs. CTA c's record of pair bg is record c + bg of all: the
  // shares' borders and the pairs' make one staircase.
  auto first_cta = [&]() -> int { return p.S > 0 ? bg * p.S : holder(bg * per); };
  auto last_cta = [&]() -> int { return p.S > 0 ? bg * p.S + p.S - 1 : holder(bg * per + per - 1); };

  // The next launch may take this CTA's slot as soon as it frees up; it does
  // its own set-up there and then waits for this grid to complete.
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), C::NCW);
    }
    mbar_init(q_bar(0), C::HELPERS / 32);
    mbar_init(q_bar(1), C::HELPERS / 32);
    mbar_init(part_bar, C::NCW);
    mbar_init(free_bar, C::HELPERS / 32);
    mbar_init(row_bar, 1);
    mbar_init(merge_bar, 1);
    mbar_init(last_merge_bar, 1);
    flag[0] = 0;
    flag[1] = 0;
    flag[2] = 0;
    fence_barrier_init();
  }
  // The first rows go into L2 while the kernel before this one drains (a
  // prefetch brings nothing into the SM, so it is safe even if that kernel
  // writes some of them: L2 is where its writes land).
  if (rot_in) {
    prefetch_l2(rot_src());
    if (D > 64) prefetch_l2(rot_src() + HALF);
    if (p.rope && rot_row == 0) {
      prefetch_l2(ctab);
      prefetch_l2(stab);
    }
  }
  if (warp == C::NCW && lane == 0 && p.n_blocks > 0) {
    tma_prefetch_desc(&tmK1);
    tma_prefetch_desc(&tmV1);
    const int k0 = u0 - bg * per, k1 = min(per, u1 - bg * per);
    for (int k = k0, i = 0; k < k1 && i < p.pf_stages; k += C::R / C::UNIT, ++i) {
      const long long pos = p.lo + (long long)k * C::UNIT;
      const int n = (int)min(min((long long)C::R, p.off - pos), (long long)(k1 - k) * C::UNIT);
      for_boxes(pos, n,
                [&](const CUtensorMap* mk, const CUtensorMap* mv, int row, int) {
                  tma_prefetch_l2_4d(mk, 0, row / 128 * C::ROWB, g, b);   // 128 rows are ROWB lines
                  tma_prefetch_l2_4d(mv, 0, row / 128 * C::ROWB, g, b);
                },
                [&](int row, int, int rows) {
                  const long long so = ((long long)bg * p.cap + row) * NB * 2;
                  bulk_prefetch_l2(ksc_g + so, (uint32_t)(rows * NB * 2));
                  bulk_prefetch_l2(vsc_g + so, (uint32_t)(rows * NB * 2));
                });
    }
  }
  __syncthreads();
  // Everything below reads or writes global memory that the kernel before
  // this one may still be using.
  griddep_wait();

  if (warp >= C::NCW) {
    regs_dec<C::REGS_PRODUCER>();
    if (warp == C::NCW) {
      // ------------------------------------------------------------ producer
      if (lane != 0) return;
      int it = 0;
      for (int u = u0; u < u1 && !flag[0]; ++it) {
        const int k = u - bg * per;   // unit within the pair
        const int s = it % C::NS;
        if (!mbar_wait_asleep(empty_bar(s), (uint32_t)(((it / C::NS) & 1) ^ 1))) { flag[0] = 1; break; }
        const int units = min(min(C::R / C::UNIT, per - k), u1 - u);
        const long long pos = p.lo + (long long)k * C::UNIT;
        const int n = (int)min((long long)units * C::UNIT, p.off - pos);   // 0: a pair without cached rows
        const int boxes = (n + 127) / 128;
        const int sc = p.ring_cap > 0 ? 128 * boxes : (n + 15) / 16 * 16;
        mbar_arrive_expect_tx(full_bar(s), n > 0 ? 2u * (uint32_t)(128 * boxes * C::ROWB + sc * NB * 2) : 0u);
        if (n > 0)
          for_boxes(pos, n,
                    [&](const CUtensorMap* mk, const CUtensorMap* mv, int row, int r) {
                      const uint32_t co = s * C::STAGE_BYTES + (uint32_t)(r * C::ROWB);
                      tma_load_4d(sbase + C::OFF_K + co, mk, full_bar(s), 0, row / 128 * C::ROWB, g, b);
                      tma_load_4d(sbase + C::OFF_V + co, mv, full_bar(s), 0, row / 128 * C::ROWB, g, b);
                    },
                    [&](int row, int r, int rows) {
                      const long long so = ((long long)bg * p.cap + row) * NB * 2;
                      const uint32_t sd = s * C::SC_BYTES + (uint32_t)(r * NB * 2), bytes = (uint32_t)(rows * NB * 2);
                      bulk_load(sbase + C::OFF_KS + sd, ksc_g + so, bytes, full_bar(s));
                      bulk_load(sbase + C::OFF_VS + sd, vsc_g + so, bytes, full_bar(s));
                    });
        u += units;
        if (k + units == per) next_pair();
      }
      // Copies still in flight keep this CTA, also when the consumers gave up.
      for (int j = (it > C::NS ? it - C::NS : 0); j < it; ++j)
        mbar_wait_drain(full_bar(j % C::NS), (uint32_t)((j / C::NS) & 1));
      return;
    }
    // ------------------------------------------------------------ helpers
    // prepare(i): the queries of this CTA's pair i, which is (b, g), into buffer
    // i, and the new K row, rotated. The buffer's last readers, of pair i - 2,
    // are through: their partials were waited for.
    constexpr int CH = D / 8;   // 8 elements of the new row a lane of the first warp: lanes 0.. K, lanes 16.. V
    const int nch = lane & 15;
    const bool n_is_v = lane >= 16, n_live = htid < 32 && nch < CH;
    __nv_bfloat16* x_sm = reinterpret_cast<__nv_bfloat16*>(smem + C::OFF_XROW);
    auto prepare = [&](int i, bool last) {
      uint8_t* qb = q_buf(i);
      const float sink_in = (htid < QM && p.sinks) ? p.sinks[g * QM + htid] : -INFINITY;
      uint4 x1 = make_uint4(0, 0, 0, 0), x2 = x1;
      if (rot_in && (rot_row < QM || last)) {
        const __nv_bfloat16* src = rot_src();
        x1 = *reinterpret_cast<const uint4*>(src);
        x2 = *reinterpret_cast<const uint4*>(src + HALF);
        if (p.rope) rotate8(x1, x2, ctab, stab);
        if (rot_row == QM) {
          *reinterpret_cast<uint4*>(x_sm + 8 * rot_ch) = x1;
          *reinterpret_cast<uint4*>(x_sm + HALF + 8 * rot_ch) = x2;
        }
      }
      const int row = min(rot_row, 7);   // lanes past the queries write nothing
      const float hs =
          i4_query<D>(x1, x2, rot_row < QM ? rot_ch : 8, reinterpret_cast<uint4*>(qb) + row * (D / 8),
                      reinterpret_cast<float*>(qb + C::Q_SUM) + row * (D / 8), p.scale_log2);
      if (rot_row < QM && rot_ch == 0) reinterpret_cast<float*>(qb + C::Q_HS)[rot_row] = hs;
      if (htid < QM) reinterpret_cast<float*>(qb + C::Q_SINK)[htid] = sink_in * 1.4426950408889634f;
      __syncwarp();
      if (lane == 0) mbar_arrive(q_bar(i));
    };
    // The new row of pair (b, g), quantised, into the cache and into smem as row
    // 0 of a tile (whose other rows are masked). Its last reader, of the pair
    // before, is through.
    auto put_row = [&]() {
      uint4 na = make_uint4(0, 0, 0, 0);
      if (n_live && n_is_v) na = *reinterpret_cast<const uint4*>(p.v + b * p.vs0 + (long long)g * p.vs2 + 8 * nch);
      named_bar_sync(2, C::HELPERS);   // x_sm is written
      if (htid < 32) {
        if (n_live && !n_is_v) na = *reinterpret_cast<const uint4*>(x_sm + 8 * nch);
        uint16_t sc;
        const uint32_t codes = i4_quantise8(na, sc);
        if (n_live) {
          const long long slot = p.ring_cap > 0 ? p.off % p.ring_cap : p.off;
          const long long crow = (long long)bg * p.cap + slot;
          reinterpret_cast<uint32_t*>(n_is_v ? p.cv : p.ck)[crow * CH + nch] = codes;
          *reinterpret_cast<uint32_t*>(smem + (n_is_v ? C::OFF_XV : C::OFF_XK) + i4_off<D>(0, nch / 4) +
                                       4 * (nch & 3)) = codes;
          if ((nch & 3) == 0) {
            reinterpret_cast<uint16_t*>(n_is_v ? p.cvs : p.cks)[crow * NB + nch / 4] = sc;
            reinterpret_cast<uint16_t*>(smem + (n_is_v ? C::OFF_XVS : C::OFF_XS))[nch / 4] = sc;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(row_bar);
      }
    };
    uint32_t merge_phase = 0;
    int end = min(u1, bg * per + per);
    prepare(0, end == bg * per + per);
    if (end == bg * per + per) put_row();
    named_bar_sync(2, C::HELPERS);   // x_sm is read
    for (int i = 0; end < u1; ++i) {
      const int bg_i = bg, b_i = b, g_i = g, c0 = first_cta(), c1 = last_cta();
      next_pair();
      end = min(u1, bg * per + per);
      prepare(i + 1, end == bg * per + per);
      // pair i's partials, merged
      if (!mbar_wait_asleep(part_bar, (uint32_t)(i & 1))) flag[0] = 1;
      if (end == bg * per + per) put_row();
      decode_finish<D, C, C::HELPERS, 2>(p, htid, red, smem + C::OFF_RED, C::RED_BYTES, merge_bar, merge_phase,
                                         flag + 1, reinterpret_cast<const float*>(q_buf(i) + C::Q_SINK), g_i, b_i,
                                         cta - c0, c1 - c0 + 1, p.ws_rec + (long long)(c0 + bg_i) * p.rec_floats);
      named_bar_sync(2, C::HELPERS);   // all have read flag[1], the partials and x_sm
      if (lane == 0) mbar_arrive(free_bar);
    }
    return;
  }

  // ---------------------------------------------------------------- consumers
  regs_inc<C::REGS_CONSUMER>();
  uint32_t off[NB];   // this lane's ldmatrix row (row `lane` of the warp's) in a stage
#pragma unroll
  for (int blk = 0; blk < NB; ++blk) off[blk] = i4_off<D>(32 * warp + lane, blk);
  uint32_t phase = 0;
  int slot = 0, i = 0;
  for (int u = u0;; ++i) {
    const int bg0 = u / per * per;   // the pair's first unit
    const int end = min(u1, bg0 + per);
    if (!mbar_wait_warp(q_bar(i), (uint32_t)((i >> 1) & 1))) flag[0] = 1;
    I4State<D> z;
    i4_start<D>(z, reinterpret_cast<const uint4*>(q_buf(i)), reinterpret_cast<const float*>(q_buf(i) + C::Q_SUM),
                reinterpret_cast<const float*>(q_buf(i) + C::Q_HS), QM, lane);

    // The share's rows of this pair from position pos0 on: the first skip ones
    // lie before the band. left and skip count from this warp's rows of a stage.
    const int k0 = u - bg0, k_end = end - bg0;
    const long long pos0 = p.lo + (long long)k0 * C::UNIT;
    const int rows = (int)(min(p.off, p.lo + (long long)k_end * C::UNIT) - pos0);
    int left = rows - 32 * warp, skip = (int)max(p.lo_mask - pos0, 0LL) - 32 * warp;
    // The stages, and in the CTA with the pair's last unit one warp has the new
    // row's tile as one more: the first that the last stage leaves idle, or where
    // it is full each in its turn (one and the same held the others up: 74.4 us
    // against 70.9 for 64 sequences of 8,192 rows, d = 64).
    const int n_st = (k_end - k0 + C::R / C::UNIT - 1) / (C::R / C::UNIT);
    const int busy = ((rows + 31) / 32) % C::NCW;
    const bool new_row = end == bg0 + per && warp == (busy > 0 ? busy : i % C::NCW);
    const int n_it = __any_sync(0xffffffffu, flag[0]) ? 0 : n_st + (new_row ? 1 : 0);
    for (int j = 0; j < n_it; ++j) {
      // the new row's tile stands to V's as a stage does (off counts from the
      // stage's start: 32 rows are whole patterns of the swizzle)
      uint32_t kt = sbase + C::OFF_XK - (uint32_t)(32 * warp * C::ROWB), ks = sbase + C::OFF_XS;
      if (j < n_st) {
        if (!mbar_wait_warp(full_bar(slot), phase)) { flag[0] = 1; break; }
        kt = sbase + C::OFF_K + slot * C::STAGE_BYTES;
        ks = sbase + C::OFF_KS + slot * C::SC_BYTES + (uint32_t)(32 * warp * NB * 2);
      } else {
        // (every pair of this CTA before this one ended here: use i of row_bar)
        if (!mbar_wait_warp(row_bar, (uint32_t)(i & 1))) { flag[0] = 1; break; }
        left = 1;
        skip = 0;
      }
      ks += (uint32_t)((lane >> 2) * NB * 2);
      if (skip <= 0 && left >= 32)
        decode_tile_i4<D, false, C::OFF_V - C::OFF_K, C::OFF_VS - C::OFF_KS>(kt, off, ks, 0, 32, z, lane);
      else if (skip < min(left, 32))
        decode_tile_i4<D, true, C::OFF_V - C::OFF_K, C::OFF_VS - C::OFF_KS>(kt, off, ks, max(skip, 0), min(left, 32),
                                                                            z, lane);
      if (j < n_st) {
        __syncwarp();
        if (lane == 0) mbar_arrive(empty_bar(slot));
        left -= C::R;
        skip = 0;
        if (++slot == C::NS) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
    // the last pair's partials are read
    if (i > 0 && !mbar_wait_warp(free_bar, (uint32_t)((i - 1) & 1))) flag[0] = 1;
    i4_write_partial<D>(z, reinterpret_cast<float*>(smem + C::OFF_RED) + warp * (C::RED_WARP / 4), lane);
    u = end;
    if (u == u1) break;
    __syncwarp();
    if (lane == 0) mbar_arrive(part_bar);
  }
  named_bar_sync(1, 32 * C::NCW);
  bg = (u1 - 1) / per;
  b = bg / p.n_kv;
  g = bg - b * p.n_kv;
  // The last pair. The ring holds nothing to come: it takes the records.
  uint32_t merge_phase = 0;
  const int c0 = first_cta();
  decode_finish<D, C, 32 * C::NCW, 1>(p, threadIdx.x, red, smem, C::RING_BYTES, last_merge_bar, merge_phase, flag + 2,
                                      reinterpret_cast<const float*>(q_buf(i) + C::Q_SINK), g, b, cta - c0,
                                      last_cta() - c0 + 1, p.ws_rec + (long long)(c0 + bg) * p.rec_floats);
}

}  // namespace sa
