// One-token decode over an INT4 cache (int4.cuh): a producer warp and eight
// consumer warps per CTA, two CTAs per SM, as decode_kernel (decode.cuh), but
// with 4.5 bits an element the arithmetic per byte is about four times that
// of a bf16 cache, so the codes go to the tensor cores with as few
// instructions as possible, and all SMs get the same number of rows:
//
// A (sequence, KV head) pair's rows are cut into stages. Where the CTAs can be
// dealt out to the pairs evenly, each pair gets S of them; else the stages of
// all pairs lie in one row and every CTA takes an equal, contiguous share
// (plan_decode chooses). A share can end one pair, span several and begin
// another: the producer streams on across the border while the consumers
// merge what they have of a pair (decode_finish) and take up the next one's
// queries.
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
//   masks, but runs here as conversions and two f16 products: 219 us against
//   the 166 of f16 at 16 sequences of 65,536 rows.)
// O^T += V^T P'^T, m16n8k16 in f16, P' = p * scale_v, transposed by movmatrix:
//   ldmatrix.trans over 16-bit units hands a lane the same 4 codes of two
//   neighbouring keys; x & 0x000F000F as f16 are the subnormals u 2^-24 of
//   the first, x & 0x00F000F0 16 times those of the second, and x >> 8 gives
//   the other two: 5 instructions for 8 codes (bf16, whose 7 fraction bits
//   hold one code, takes 7). The offset of 8 goes out at the end, by the sums
//   of P', which a lane has in fp32.
// The weights are taken relative to 2^ref with ref = m + E - 6, m a score of the
//   head that no score so far has exceeded by more than 8 (log2 units) and 2^E
//   the power of two below the largest |scale_v| that the warp has seen: then
//   |P'| < 2^15, which f16 holds, with its 11 bits down to 2^-20 of the weight
//   of m and some to 2^-30. m and E move only when a tile breaks one of the two
//   bounds, so a tile needs no maximum across lanes, only a vote. Sums, the
//   merge and the lse go by ref as by a maximum.
#pragma once

#include <math.h>

#include "decode.cuh"
#include "int4.cuh"

namespace sa {

template <int D>
struct DecodeI4Cfg {
  static constexpr int NCW = 8;                 // consumer warps
  // rows per consumer warp and stage, in tiles of 32
  static constexpr int RW = (D == 64) ? 64 : 32;
  static constexpr int R = RW * NCW;
  static constexpr int NB = D / kI4Block;       // blocks per row
  static constexpr int ROWB = D / 2;            // code bytes per row
  static constexpr uint32_t STAGE_BYTES = R * ROWB;
  static constexpr uint32_t SC_BYTES = R * NB * 2;   // K (or V) scales of one stage
  static constexpr int NS = (D == 96) ? 3 : 2;
  static constexpr uint32_t STAGE_TX = 2 * (STAGE_BYTES + SC_BYTES);
  static constexpr int NUM_THREADS = 32 * (NCW + 1);
  static constexpr uint32_t OFF_K = 0;
  static constexpr uint32_t OFF_V = NS * STAGE_BYTES;
  // the new row: a tile of codes and scales, row 0 valid
  static constexpr uint32_t XTILE = 32 * ROWB;
  static constexpr uint32_t OFF_XK = 2 * NS * STAGE_BYTES;
  static constexpr uint32_t OFF_XV = OFF_XK + XTILE;
  static constexpr uint32_t OFF_KS = OFF_XV + XTILE;             // [NS][R][NB] bf16
  static constexpr uint32_t OFF_VS = OFF_KS + NS * SC_BYTES;
  static constexpr uint32_t OFF_XS = OFF_VS + NS * SC_BYTES;     // [2][32][NB] bf16
  // [NCW warps][8 m | 8 l | 8*D O] fp32, then the records of a merge
  static constexpr uint32_t RED_WARP = (16 + 8 * D) * 4;
  static constexpr uint32_t OFF_RED = OFF_XS + 2 * 32 * NB * 2;
  static constexpr uint32_t RED_BYTES = NCW * RED_WARP;
  static constexpr uint32_t OFF_Q = OFF_RED + RED_BYTES;   // 8 query rows and the new K row, rotated, bf16
  static constexpr uint32_t OFF_BAR = OFF_Q + 9 * D * 2;
  static constexpr uint32_t OFF_MBAR = OFF_BAR + 8 * (2 * NS);
  static constexpr uint32_t OFF_FLAG = OFF_MBAR + 8;
  static constexpr uint32_t OFF_SINK = OFF_FLAG + 16;
  static constexpr uint32_t SMEM_BYTES = OFF_SINK + 32 + 1024;
  static_assert(2 * (SMEM_BYTES + 1024) <= 228 * 1024, "two CTAs per SM");
  static_assert(9 * (D / 16) <= 32 * NCW, "one thread per 16 elements of the rows to rotate");
  static_assert(OFF_XK % 1024 == 0 && STAGE_BYTES % 1024 == 0 && (XTILE % 1024 == 0 || D == 96),
                "swizzled tiles start on a multiple of their pattern");
  static_assert(OFF_BAR % 16 == 0 && OFF_KS % 16 == 0 && OFF_RED % 16 == 0, "barriers and bulk copies");
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

// A row's block scales as words (bf16 pairs; the last one's upper half 0 where
// the blocks are odd), and block blk's of them as fp32.
template <int NB>
__device__ __forceinline__ void i4_row_scales(uint32_t addr, uint32_t (&w)[(NB + 1) / 2]) {
  if constexpr (NB == 2) {
    w[0] = ld_shared_u32(addr);
  } else if constexpr (NB == 4) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  } else {
    uint16_t h[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h[i]) : "r"(addr + 2 * i));
    w[0] = (uint32_t)h[0] | (uint32_t)h[1] << 16;
    w[1] = h[2];
  }
}
__device__ __forceinline__ float i4_scale(const uint32_t* w, int blk) {
  return (blk & 1) ? bf16_hi(w[blk >> 1]) : bf16_lo(w[blk >> 1]);
}

// What a consumer warp keeps of its (b, g). Of heads 2 (lane % 4) + {0, 1}: the
// score scale hs, what the sums are relative to (ref, see the head of this
// file; ref = m + er) and the unscaled score thr = (m + 8) / hs that moves it;
// the running sum l and those of P' per block ps (both over this lane's keys).
// qf: the query fragments, qo: the offset's. lim: 2^(E + 1) as a bf16 pair, er =
// E - 6. o[blk][i]: the accumulators of d = 32 blk + 4 (lane / 4) + 2 i + {0, 1}
// (fragment rows g and g + 8, the latter times 16), offset included, times 2^-24.
template <int D>
struct I4State {
  static constexpr int NB = D / kI4Block;
  uint32_t qf[NB][4];
  uint32_t qo[2];
  uint32_t lim;
  float er, hs[2], m[2], ref[2], thr[2], l[2];
  float ps[NB][2], o[NB][2][4];
};

// lim for scales whose magnitudes (bf16 pairs) are at most mag in any lane. E
// is kept within [-90, 125], so that sums of weights stay in range whatever
// the scales. (Rare, so out of the tile's way.)
__device__ __noinline__ uint32_t i4_raise(uint32_t mag) {
  const uint32_t mx = __reduce_max_sync(0xffffffffu, max(mag & 0xFFFFu, mag >> 16));
  const int e = (int)(mx >> 7) - 127;
  const uint32_t top = (uint32_t)((e < -90 ? -90 : (e > 125 ? 125 : e)) + 128) << 7;   // 2^(e + 1)
  return top | top << 16;
}

// One warp's 32 keys of a stage: codes at kst / vst plus this lane's offsets
// off[blk] (of row `lane`), scales of the first row at ksc / vsc. With MASK,
// keys below n_first and from n_valid on are masked (their scales may hold
// anything).
template <int D, bool MASK>
__device__ __forceinline__ void decode_tile_i4(uint32_t kst, uint32_t vst, const uint32_t (&off)[D / 32],
                                               uint32_t ksc, uint32_t vsc, int n_first, int n_valid, I4State<D>& z,
                                               int lane) {
  constexpr int NB = D / 32, NW = (NB + 1) / 2;
  constexpr uint32_t M0 = 0x000F000Fu, M1 = 0x00F000F0u;
  const int r = lane >> 2, t = lane & 3;
  ksc += (uint32_t)(r * NB * 2);
  vsc += (uint32_t)(r * NB * 2);
  bool ok[4];   // key 8 c + r
#pragma unroll
  for (int c = 0; c < 4; ++c) ok[c] = !MASK || (8 * c + r >= n_first && 8 * c + r < n_valid);
  float s[2][4];   // keys 16 j + r (0, 1) and + 8 (2, 3), heads 2 t + {0, 1}
  uint32_t sw[4][NW];
#pragma unroll
  for (int c = 0; c < 4; ++c) i4_row_scales<NB>(ksc + (uint32_t)(8 * c * NB * 2), sw[c]);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t a0 = (NW == 2 && (t & 1)) ? sw[2 * j][NW - 1] : sw[2 * j][0];
    const uint32_t a1 = (NW == 2 && (t & 1)) ? sw[2 * j + 1][NW - 1] : sw[2 * j + 1][0];
    mma_16816_bf16_0(s[j], a0, a1, NW == 1 ? 0u : a0, NW == 1 ? 0u : a1, z.qo[0], z.qo[1]);
  }
#pragma unroll
  for (int blk = 0; blk < NB; ++blk) {
    uint32_t w[4];
    ldmatrix_x4(kst + off[blk], w[0], w[1], w[2], w[3]);
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
  // the scales of V: E over them all
  uint32_t mag = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    i4_row_scales<NB>(vsc + (uint32_t)(8 * c * NB * 2), sw[c]);
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      if (MASK && !ok[c]) sw[c][i] = 0;   // a row never written holds anything
      mag = __vmaxu2(mag, sw[c][i] & 0x7FFF7FFFu);
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
  if (__any_sync(0xffffffffu, mx[0] > z.thr[0] || mx[1] > z.thr[1] || __vmaxu2(mag, z.lim) != z.lim)) {
    z.lim = i4_raise(__vmaxu2(mag, z.lim - 0x00010001u));
    z.er = (float)((int)(z.lim >> 23) - 134);   // E - 6
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 4));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
      const bool empty = z.m[e] == -INFINITY;   // no key so far
      z.m[e] = fmaxf(z.m[e], x * z.hs[e]);
      const float ref = z.m[e] == -INFINITY ? 0.f : z.m[e] + z.er;
      const float al = empty ? 0.f : ex2(z.ref[e] - ref);
      z.ref[e] = ref;
      z.thr[e] = (z.m[e] + 8.f) / z.hs[e];
      z.l[e] *= al;
#pragma unroll
      for (int blk = 0; blk < NB; ++blk) {
        z.ps[blk][e] *= al;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          z.o[blk][i][e] *= al;
          z.o[blk][i][2 + e] *= al;
        }
      }
    }
  }
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
    ldmatrix_x4_trans(vst + off[blk], x[0], x[1], x[2], x[3]);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float v = i4_scale(sw[c], blk);
      const float p0 = s[c >> 1][2 * (c & 1)] * v, p1 = s[c >> 1][2 * (c & 1) + 1] * v;
      z.ps[blk][0] += p0;
      z.ps[blk][1] += p1;
      pb[c] = movmatrix_trans(pack_f16(p0, p1));
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

// Query fragments (B operand) from the group's rotated rows qs [QM][D]: head
// lane / 4, elements 32 blk + 8 t + {0, 4}, {1, 5}, {2, 6}, {3, 7} (t = lane % 4);
// and empty sums.
template <int D>
__device__ __forceinline__ void i4_start(I4State<D>& z, const __nv_bfloat16* qs, int QM, float scale_log2, int lane) {
  constexpr int NB = D / kI4Block;
  const int n = lane >> 2, t = lane & 3;
  float qv[NB][8];
  float amax = 0.f;
#pragma unroll
  for (int blk = 0; blk < NB; ++blk) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (n < QM) u = *reinterpret_cast<const uint4*>(qs + n * D + 32 * blk + 8 * t);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      qv[blk][i] = (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
      amax = fmaxf(amax, fabsf(qv[blk][i]));
    }
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  // the head's largest |q| goes to [2^14, 2^15)
  int eq = 0;
  if (amax > 0.f) {
    eq = (int)((__float_as_uint(amax) >> 23) & 0xFFu) - 127 - 14;
    eq = eq < -100 ? -100 : (eq > 100 ? 100 : eq);
  }
  const float down = __uint_as_float((uint32_t)(127 - eq) << 23);
  const float hs = scale_log2 * __uint_as_float((uint32_t)(127 + eq) << 23) * 0x1p24f;
  z.hs[0] = __shfl_sync(0xffffffffu, hs, 8 * t);
  z.hs[1] = __shfl_sync(0xffffffffu, hs, 8 * t + 4);
  uint32_t part[4][3] = {};   // of block blk's offset, bf16
#pragma unroll
  for (int blk = 0; blk < NB; ++blk) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      qv[blk][i] *= down;
      sum += qv[blk][i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = (i & 1) ? 0.0625f : 1.f;   // nibbles 1, 3, 5, 7 enter times 16
      z.qf[blk][i] = pack_f16(qv[blk][i] * f, qv[blk][i + 4] * f);
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    i4_split3(sum * (-8.0f * 0x1p-24f), part[blk]);
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
  z.er = -96.f;   // E = -90
  z.lim = 0x13001300u;   // 2^-89, twice
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    z.m[e] = z.thr[e] = -INFINITY;
    z.ref[e] = 0.f;
    z.l[e] = 0.f;
  }
#pragma unroll
  for (int blk = 0; blk < NB; ++blk) {
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
      rw[2 * t + e] = z.m[e] == -INFINITY ? -INFINITY : z.ref[e];
      rw[8 + 2 * t + e] = l;
    }
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      const float c = -8.f * sum8(z.ps[blk][e]);   // the codes' offset
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<float2*>(rw + 16 + (2 * t + e) * D + 32 * blk + 4 * r + 2 * i) =
            make_float2(fmaf(z.o[blk][i][e], 0x1p24f, c), fmaf(z.o[blk][i][2 + e], 0x1p20f, c));
    }
  }
}

// tmK / tmV: the codes, dims {128, lines, n_kv, B} bytes. p.ck, p.cv, p.cks,
// p.cvs hold the cache's code and scale arrays. p.units stages in all, per
// pair p.units / (B n_kv); p.S > 0: S CTAs per pair, else equal shares.
template <int D>
__global__ void __launch_bounds__(DecodeI4Cfg<D>::NUM_THREADS, 2)
    decode_i4_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
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
  const uint32_t merge_bar = sbase + C::OFF_MBAR;
  volatile int* flag = reinterpret_cast<volatile int*>(smem + C::OFF_FLAG);
  // flag[0]: abort, flag[1]: "this CTA merges the pair's records"
  float* sink_sm = reinterpret_cast<float*>(smem + C::OFF_SINK);   // [q_mult] sinks, log2 units
  __nv_bfloat16* q_sm = reinterpret_cast<__nv_bfloat16*>(smem + C::OFF_Q);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int QM = p.q_mult;
  const int per = p.n_blocks > 0 ? (int)p.n_blocks : 1;   // stages of a pair

  // This CTA's stages [u0, u1) of the row of all, and who holds stage u.
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

  // Rows of scales to bring for a box of box_rows rows from position pos < off:
  // whole 16-row groups up to the last cached one (cap is a multiple of 16).
  const int box_rows = p.box_rows;
  auto scale_rows = [&](long long pos) -> int {
    if (p.ring_cap > 0) return box_rows;
    const long long n = p.off - pos;
    return n >= box_rows ? box_rows : (int)((n + 15) / 16 * 16);
  };
  const char* ksc_g = reinterpret_cast<const char*>(p.cks);
  const char* vsc_g = reinterpret_cast<const char*>(p.cvs);

  // The rows a pair's CTA rotates into q_sm, 16 elements (8 RoPE pairs) a
  // thread: the group's queries, then the new K row. (sequence b, KV head g)
  const int rot_row = threadIdx.x / (D / 16), rot_ch = threadIdx.x - rot_row * (D / 16);
  auto rot_src = [&]() -> const __nv_bfloat16* {
    return 8 * rot_ch + (rot_row < QM ? p.q + b * p.qs0 + (long long)(g * QM + rot_row) * p.qs2
                                      : p.k + b * p.ks0 + (long long)g * p.ks2);
  };
  const float* ctab = p.cos_t + p.off * HALF + 8 * rot_ch;
  const float* stab = p.sin_t + p.off * HALF + 8 * rot_ch;

  // The next launch may take this CTA's slot as soon as it frees up; it does
  // its own set-up there and then waits for this grid to complete.
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), C::NCW);
    }
    mbar_init(merge_bar, 1);
    flag[0] = 0;
    flag[1] = 0;
    fence_barrier_init();
  }
  // The first rows go into L2 while the kernel before this one drains (a
  // prefetch brings nothing into the SM, so it is safe even if that kernel
  // writes some of them: L2 is where its writes land).
  if (warp < C::NCW && rot_row <= QM) {
    prefetch_l2(rot_src());
    if (D > 64) prefetch_l2(rot_src() + HALF);
    if (p.rope && rot_row == 0) {
      prefetch_l2(ctab);
      prefetch_l2(stab);
    }
  }
  if (warp == C::NCW && lane == 0 && p.n_blocks > 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    int k = u0 - bg * per;
    for (int i = 0; i < p.pf_stages && i < u1 - u0 && k < per; ++i, ++k) {
      const long long pos0 = p.lo + (long long)k * C::R;
      for (int r = 0; r < C::R && pos0 + r < p.off; r += box_rows) {
        const long long pos = pos0 + r;
        const int row = (int)(p.ring_cap > 0 ? pos % p.ring_cap : pos);
        const int line = row / 128 * C::ROWB;   // 128 rows are ROWB lines of 128 bytes
        tma_prefetch_l2_4d(&tmK, 0, line, g, b);
        tma_prefetch_l2_4d(&tmV, 0, line, g, b);
        const uint32_t bytes = (uint32_t)scale_rows(pos) * NB * 2;
        const long long so = ((long long)bg * p.cap + row) * NB * 2;
        bulk_prefetch_l2(ksc_g + so, bytes);
        bulk_prefetch_l2(vsc_g + so, bytes);
      }
    }
  }
  __syncthreads();
  // Everything below reads or writes global memory that the kernel before
  // this one may still be using.
  griddep_wait();

  if (warp == C::NCW) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int k = u0 - bg * per;   // stage within the pair
      const int n = u1 - u0;
      int it = 0;
      for (; it < n && !flag[0]; ++it) {
        const int s = it % C::NS;
        if (!mbar_wait(empty_bar(s), (uint32_t)(((it / C::NS) & 1) ^ 1))) { flag[0] = 1; break; }
        // one box a stage, or on a ring (whose capacity a stage need not divide)
        // boxes of 128 rows that start on multiples of 128: none wraps
        const long long pos0 = p.lo + (long long)k * C::R;
        uint32_t tx = 0;
        for (int r = 0; r < C::R && pos0 + r < p.off; r += box_rows)
          tx += 2u * (uint32_t)(box_rows * C::ROWB + scale_rows(pos0 + r) * NB * 2);
        mbar_arrive_expect_tx(full_bar(s), tx);
        for (int r = 0; r < C::R && pos0 + r < p.off; r += box_rows) {
          const long long pos = pos0 + r;
          const int row = (int)(p.ring_cap > 0 ? pos % p.ring_cap : pos);
          const uint32_t co = s * C::STAGE_BYTES + (uint32_t)(r * C::ROWB);
          const int line = row / 128 * C::ROWB;
          tma_load_4d(sbase + C::OFF_K + co, &tmK, full_bar(s), 0, line, g, b);
          tma_load_4d(sbase + C::OFF_V + co, &tmV, full_bar(s), 0, line, g, b);
          const uint32_t bytes = (uint32_t)scale_rows(pos) * NB * 2;
          const long long so = ((long long)bg * p.cap + row) * NB * 2;
          const uint32_t sd = s * C::SC_BYTES + (uint32_t)(r * NB * 2);
          bulk_load(sbase + C::OFF_KS + sd, ksc_g + so, bytes, full_bar(s));
          bulk_load(sbase + C::OFF_VS + sd, vsc_g + so, bytes, full_bar(s));
        }
        if (++k == per) {
          k = 0;
          ++bg;
          if (++g == p.n_kv) {
            g = 0;
            ++b;
          }
        }
      }
      if (flag[0]) {
        for (int j = (it > C::NS ? it - C::NS : 0); j < it; ++j)
          mbar_wait_drain(full_bar(j % C::NS), (uint32_t)((j / C::NS) & 1));
      }
    }
    return;  // the producer takes no part in the merges (named barriers below count 32*NCW)
  }

  // ---------------------------------------------------------------- consumers
  uint32_t off[NB];   // this lane's ldmatrix row (row `lane` of the warp's first 32) in a stage
#pragma unroll
  for (int blk = 0; blk < NB; ++blk) off[blk] = i4_off<D>(C::RW * warp + lane, blk);
  uint32_t merge_phase = 0;
  int it = 0;
  for (int u = u0; u < u1;) {
    const int bg0 = bg * per;                       // the pair's first stage
    const int end = min(u1, bg0 + per);
    // the CTA with the pair's last stage attends the new row, in warp 0
    const bool last_cta = end == bg0 + per, new_row = last_cta && warp == 0;
    {
      const float sink_in = (threadIdx.x < QM && p.sinks) ? p.sinks[g * QM + threadIdx.x] : -INFINITY;
      if (rot_row < QM || (rot_row == QM && last_cta)) {
        const __nv_bfloat16* src = rot_src();
        uint4 x1 = *reinterpret_cast<const uint4*>(src), x2 = *reinterpret_cast<const uint4*>(src + HALF);
        if (p.rope) rotate8(x1, x2, ctab, stab);
        __nv_bfloat16* dst = q_sm + rot_row * D + 8 * rot_ch;
        *reinterpret_cast<uint4*>(dst) = x1;
        *reinterpret_cast<uint4*>(dst + HALF) = x2;
      }
      if (threadIdx.x < QM) sink_sm[threadIdx.x] = sink_in * 1.4426950408889634f;
    }
    // The new row, 8 elements a lane: lanes 0.. its K, lanes 16.. its V.
    constexpr int CH = D / 8;
    const int nch = lane & 15;                       // this lane's chunk
    const bool n_live = new_row && nch < CH, n_is_v = lane >= 16;
    uint4 na = make_uint4(0, 0, 0, 0);
    if (n_live && n_is_v) na = *reinterpret_cast<const uint4*>(p.v + b * p.vs0 + (long long)g * p.vs2 + 8 * nch);
    named_bar_sync(1, 32 * C::NCW);
    I4State<D> z;
    i4_start<D>(z, q_sm, QM, p.scale_log2, lane);
    // Quantise it, write it to the cache and stage it in smem as row 0 of a
    // tile (the other rows are masked).
    if (new_row) {
      if (n_live && !n_is_v) na = *reinterpret_cast<const uint4*>(q_sm + QM * D + 8 * nch);
      uint16_t sc;
      const uint32_t codes = i4_quantise8(na, sc);
      if (n_live) {
        const long long slot = p.ring_cap > 0 ? p.off % p.ring_cap : p.off;
        const long long crow = (long long)bg * p.cap + slot;
        uint32_t* cc = reinterpret_cast<uint32_t*>(n_is_v ? p.cv : p.ck) + crow * CH + nch;
        uint16_t* cs = reinterpret_cast<uint16_t*>(n_is_v ? p.cvs : p.cks) + crow * NB + nch / 4;
        *cc = codes;
        *reinterpret_cast<uint32_t*>(smem + (n_is_v ? C::OFF_XV : C::OFF_XK) + i4_off<D>(0, nch / 4) +
                                     4 * (nch & 3)) = codes;
        if ((nch & 3) == 0) {
          *cs = sc;
          reinterpret_cast<uint16_t*>(smem + C::OFF_XS)[(n_is_v ? 32 * NB : 0) + nch / 4] = sc;
        }
      }
      __syncwarp();
    }

    // the stages, and for the warp with the new row its tile as one more
    const int k_end = end - bg0;
    for (int k = u - bg0; k < k_end + (new_row ? 1 : 0); ++k) {
      if (flag[0]) break;
      const bool is_new = k == k_end;
      uint32_t kt = sbase + C::OFF_XK, vt = sbase + C::OFF_XV, ks = sbase + C::OFF_XS, vs = ks + 32 * NB * 2;
      int first = 0, last = 1;
      const int s = it % C::NS;
      if (!is_new) {
        if (!mbar_wait(full_bar(s), (uint32_t)((it / C::NS) & 1))) { flag[0] = 1; break; }
        ++it;
        // this warp's rows [first, last) of the stage are valid (the first ones
        // may lie before the band, the last ones behind the cache)
        const int r = C::RW * warp;
        const long long pos = p.lo + (long long)k * C::R + r;
        first = p.lo_mask > pos ? (int)(p.lo_mask - pos) : 0;
        last = p.off - pos < C::RW ? (int)(p.off - pos) : C::RW;
        kt = sbase + C::OFF_K + s * C::STAGE_BYTES;
        vt = sbase + C::OFF_V + s * C::STAGE_BYTES;
        ks = sbase + C::OFF_KS + s * C::SC_BYTES + (uint32_t)(r * NB * 2);
        vs = sbase + C::OFF_VS + s * C::SC_BYTES + (uint32_t)(r * NB * 2);
      }
      // 32 rows are a whole number of the swizzle's 1024-byte patterns (or of
      // plain lines): a tile's offsets are the first one's plus its bytes
      for (int i = 0; i < C::RW && i < last; i += 32) {
        if (first <= i && i + 32 <= last)
          decode_tile_i4<D, false>(kt + i * C::ROWB, vt + i * C::ROWB, off, ks + i * NB * 2, vs + i * NB * 2, 0, 32, z,
                                   lane);
        else if (first < i + 32 && first < last)
          decode_tile_i4<D, true>(kt + i * C::ROWB, vt + i * C::ROWB, off, ks + i * NB * 2, vs + i * NB * 2, first - i,
                                  last - i, z, lane);
      }
      if (!is_new) {
        __syncwarp();
        if (lane == 0) mbar_arrive(empty_bar(s));
      }
    }
    i4_write_partial<D>(z, reinterpret_cast<float*>(smem + C::OFF_RED) + warp * (C::RED_WARP / 4), lane);
    named_bar_sync(1, 32 * C::NCW);

    // The pair's CTAs. CTA c's record of pair bg is record c + bg of all: the
    // shares' borders and the pairs' make one staircase.
    const int c_first = p.S > 0 ? bg * p.S : holder(bg0);
    const int c_last = p.S > 0 ? c_first + p.S - 1 : holder(bg0 + per - 1);
    const bool idle = end == u1;   // the ring holds nothing to come: it takes the records
    decode_finish<D, C>(p, reinterpret_cast<const float*>(smem + C::OFF_RED), smem + (idle ? 0u : C::OFF_RED),
                        idle ? C::OFF_XK : C::RED_BYTES, merge_bar, merge_phase, flag, sink_sm, g, b, cta - c_first,
                        c_last - c_first + 1, p.ws_rec + (long long)(c_first + bg) * p.rec_floats);
    u = end;
    if (u < u1) {
      named_bar_sync(1, 32 * C::NCW);   // the partials, the sinks and flag[1] are free for the next pair
      ++bg;
      if (++g == p.n_kv) {
        g = 0;
        ++b;
      }
    }
  }
}

}  // namespace sa
