// INT4 KV cache: rows stored as 4-bit codes with one bf16 scale per block of
// 32 elements, 4.5 bits an element, and the kernels that write such rows and
// read quantised rows back.
//
// The codes are those of the published Q4_0 scheme (blocks of 32, the step an
// eighth of the largest element with its sign turned); the scale's 5 bits, the
// tie, zeros and NaNs are this library's own. A block of 32 bf16 values x with m its
// element of largest magnitude (the positive one of two opposite ones) is kept as
//   s = -m / 8 rounded to 5 significant bits (nearest, ties to even), bf16
//   u = min(15, floor(x / s + 8.5)),  0 <= u <= 15
// and stands for s (u - 8). The scale carries the sign that sends m to the
// code 0, the one end of the range that has a step more: with the step
// |m| / 8 instead of |m| / 7 the error of the other elements is an eighth
// smaller, and only elements of the opposite sign beyond 7.5 steps (from 7.5 / 8.25
// of m on, where s is rounded down furthest) are clipped, by a step and a quarter at
// most. s has 5 significant bits and u - 8 at most
// 3, so every stored value is exactly a bf16 number: all readers see the
// same rows (decode multiplies codes and scales apart, the read-back returns
// bf16), and rows read back and appended again give the same codes, because
// the element coded 0 stands for -8 s, whose eighth is s.
// A block whose largest magnitude is under 2^-120 is kept as zeros (scale 0,
// codes 8); a block with an infinity or a NaN reads back as 32 NaNs (scale
// NaN, codes 8).
//
// Codes lie in [B][n_kv][cap][d / 2] bytes, element 2 i of a row in the low
// half of byte i and element 2 i + 1 in the high half; scales in
// [B][n_kv][cap][d / 32] bf16.
#pragma once

#include "fp8.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace sa {

constexpr int kI4Block = 32;

// Quantises 8 consecutive elements per lane (bf16 pairs in v); the four lanes
// of an aligned group of four hold one block. Returns the 8 codes as a word,
// element i in bits 4i.., and the block's scale bits (the same on all four).
// Every lane of the warp takes part.
__device__ __forceinline__ uint32_t i4_quantise8(uint4 v, uint16_t& scale) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  // the block's largest and, negated, smallest element (NaN if one is)
  const __nv_bfloat162* x2 = reinterpret_cast<const __nv_bfloat162*>(w);
  __nv_bfloat162 hi = __hmax2_nan(__hmax2_nan(x2[0], x2[1]), __hmax2_nan(x2[2], x2[3]));
  __nv_bfloat162 lo = __hmin2_nan(__hmin2_nan(x2[0], x2[1]), __hmin2_nan(x2[2], x2[3]));
  const uint32_t hb = *reinterpret_cast<const uint32_t*>(&hi), lb = *reinterpret_cast<const uint32_t*>(&lo) ^ 0x80008000u;
  const uint32_t pa = __byte_perm(hb, lb, 0x5410), pb = __byte_perm(hb, lb, 0x7632);
  __nv_bfloat162 top = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&pa),
                                   *reinterpret_cast<const __nv_bfloat162*>(&pb));   // {max, -min}
#pragma unroll
  for (int i = 1; i < 4; i <<= 1) {
    const uint32_t o = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<const uint32_t*>(&top), i);
    top = __hmax2_nan(top, *reinterpret_cast<const __nv_bfloat162*>(&o));
  }
  // |m| is the larger of the two and not negative; m < 0 where that is -min alone
  const uint32_t tb = *reinterpret_cast<const uint32_t*>(&top);
  const bool neg = bf16_hi(tb) > bf16_lo(tb);
  const uint32_t mag = (neg ? tb >> 16 : tb) & 0x7FFFu;
  // |m| / 8 (three off the exponent, exact), then the 7 fraction bits rounded to 4
  uint32_t sb = mag - (3u << 7);
  sb = (sb + 3u + ((sb >> 3) & 1u)) & ~7u;
  sb |= neg ? 0u : 0x8000u;
  // floor(x / s + 8.5) by the reciprocal: x and s have 8 and 5 significant
  // bits, so x / s + 8.5 is an integer or at least 2^-9 away from one (checked
  // over all pairs), while the two products below are off by under 2^-18; with
  // 2^-11 added, rounding x / s + 8 to the nearest integer gives that floor.
  // The first product saturates to [0, 1], which is the clamp to [0, 15].
  const float r = __fdividef(1.0f / 15.0f, __uint_as_float(sb << 16));
  constexpr float MAGIC = 12582912.0f;   // 1.5 * 2^23: its sum's low bits are the rounded integer
  uint32_t word = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    const float x = (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
    const float y = fmaf(__saturatef(fmaf(x, r, (8.0f + 0x1p-11f) / 15.0f)), 15.0f, MAGIC);
    word = (word << 4) + __float_as_uint(y);
  }
  // each term carried MAGIC's own bits 0x4B400000, at shifts 0, 4, .., 28
  constexpr uint32_t EXTRA = [] {
    uint32_t e = 0;
    for (int i = 0; i < 8; ++i) e = (e << 4) + 0x4B400000u;
    return e;
  }();
  // no number to scale by: an infinity or NaN in the block, or |m| < 2^-120
  const bool nan = mag >= 0x7F80u, zero = mag < 0x0380u;
  scale = nan ? 0x7FC0u : (zero ? 0u : (uint16_t)sb);
  return nan || zero ? 0x88888888u : word - EXTRA;
}

// 8 codes (a word, element i in bits 4i..) and their block's scale to bf16
// pairs in order. 0x4300 | u is the bf16 number 128 + u; both packed
// operations after it are exact (see above).
__device__ __forceinline__ uint4 i4_dequantise8(uint32_t w, uint16_t scale) {
  const __nv_bfloat162 s2 = __halves2bfloat162(__ushort_as_bfloat16(scale), __ushort_as_bfloat16(scale));
  const __nv_bfloat162 c2 = __float2bfloat162_rn(-136.0f);
  uint32_t p[4];   // elements (i, i + 4)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 y = __hmul2(__hadd2(*reinterpret_cast<const __nv_bfloat162*>(&b), c2), s2);
    p[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410),
                    __byte_perm(p[0], p[1], 0x7632), __byte_perm(p[2], p[3], 0x7632));
}

// A run of rows [T] of every (sequence, KV head) as bf16, and the cache rows
// they go to or come from: position index t is row (row0 + t), less cap once
// it passes the end of a ring.
struct RowsParams {
  const void* ck;   // codes, or bf16 rows
  const void* cv;
  const void* cks;  // scales: bf16 [..][d / 32] (INT4), fp32 (FP8)
  const void* cvs;
  const __nv_bfloat16* k;   // bf16 rows [B][T][n_kv][d]: the source of an append,
  const __nv_bfloat16* v;   // the destination of a read
  long long ks0, ks1, ks2, vs0, vs1, vs2;
  int T, n_kv, cap;
  int row0;
};

// A thread takes 8 elements of NR rows, K and V together, and has all of
// their loads in flight before it works on the first; a block takes rows of one
// (sequence, KV head), so its codes and scales are one contiguous run and each
// row's 16-byte pieces are adjacent lanes. NR is 4 where that still gives
// every SM four blocks, else 1 (rows_grid).
template <int D>
struct RowsCfg {
  static constexpr int CH = D / 8;             // 8-element chunks of a row
  static constexpr int RB = 256 / CH;          // rows of a block at a time
  static constexpr int NB = D / kI4Block;
};

// Appends T bf16 rows to an INT4 cache. Bound by reading them (4 d bytes a
// position and KV head against 1.1 d written): 8 x 4,096 rows of 4 heads of 96
// in 15.3 us back to back (50 MB read, 14 MB written: 4.2 TB/s; the last of this
// grid's 1.3 waves of blocks is mostly empty), 8,192 rows of 8 heads of 64 in a fused
// qkv in 5.6.
template <int D, int NR>
__global__ void __launch_bounds__(256) kv_append_i4_kernel(const RowsParams p) {
  using C = RowsCfg<D>;
  griddep_launch_dependents();
  griddep_wait();
  const int g = blockIdx.y, b = blockIdx.z;
  const int rb = threadIdx.x / C::CH, ch = threadIdx.x - rb * C::CH;
  const int t0 = blockIdx.x * (C::RB * NR) + rb;
  const long long row_bg = ((long long)b * p.n_kv + g) * p.cap;
  const __nv_bfloat16* k = p.k + b * p.ks0 + g * p.ks2 + 8 * ch;
  const __nv_bfloat16* v = p.v + b * p.vs0 + g * p.vs2 + 8 * ch;
  uint4 kw[NR], vw[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int t = t0 + i * C::RB;
    kw[i] = vw[i] = make_uint4(0, 0, 0, 0);
    if (rb < C::RB && t < p.T) {
      kw[i] = *reinterpret_cast<const uint4*>(k + t * p.ks1);
      vw[i] = *reinterpret_cast<const uint4*>(v + t * p.vs1);
    }
  }
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int t = t0 + i * C::RB;
    uint16_t sk, sv;
    const uint32_t ck = i4_quantise8(kw[i], sk), cv = i4_quantise8(vw[i], sv);
    if (rb >= C::RB || t >= p.T) continue;
    long long row = (long long)p.row0 + t;
    if (row >= p.cap) row -= p.cap;
    const long long at = row_bg + row;
    reinterpret_cast<uint32_t*>(const_cast<void*>(p.ck))[at * C::CH + ch] = ck;
    reinterpret_cast<uint32_t*>(const_cast<void*>(p.cv))[at * C::CH + ch] = cv;
    if ((ch & 3) == 0) {
      reinterpret_cast<uint16_t*>(const_cast<void*>(p.cks))[at * C::NB + ch / 4] = sk;
      reinterpret_cast<uint16_t*>(const_cast<void*>(p.cvs))[at * C::NB + ch / 4] = sv;
    }
  }
}

enum : int { ROWS_BF16 = 0, ROWS_FP8 = 1, ROWS_INT4 = 2 };

// code * scale rounded to bf16 once: the fp32 product towards zero, its last
// bit set where it was not exact (round to odd; 24 bits >= 8 + 2, so rounding
// that to bf16 makes no false tie). The remainder is exact while it is no
// subnormal; scales under 2^-90 go through fp64.
__device__ __forceinline__ float f8_product(float code, float scale) {
  const float p = __fmul_rz(code, scale);
  return __fmaf_rn(code, scale, -p) != 0.f ? __uint_as_float(__float_as_uint(p) | 1u) : p;
}

// A pair of e4m3 codes and their row's scale to a bf16 pair.
__device__ __forceinline__ uint32_t f8_pair_bf16(uint16_t codes, float s) {
  const uint32_t h = f16x2_from_e4m3x2(codes);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  if (s >= 0x1p-90f) return pack_bf16(f8_product(f.x, s), f8_product(f.y, s));
  return bf16_bits_from_f64((double)f.x * (double)s) | bf16_bits_from_f64((double)f.y * (double)s) << 16;
}

// Elements 8 ch.. of cache row `at`: as stored, and as bf16 pairs.
template <int KIND>
struct StoredRow8 {
  uint4 c;   // bf16 pairs, or codes (FP8: x, y; INT4: x)
  float s;   // FP8: the row's scale
  uint16_t h;  // INT4: the block's
};
template <int D, int KIND>
__device__ __forceinline__ StoredRow8<KIND> load_row8(const void* rows, const void* scales, long long at, int ch) {
  using C = RowsCfg<D>;
  StoredRow8<KIND> x;
  if constexpr (KIND == ROWS_BF16) {
    x.c = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(rows) + at * D + 8 * ch);
  } else if constexpr (KIND == ROWS_INT4) {
    x.c.x = static_cast<const uint32_t*>(rows)[at * C::CH + ch];
    x.h = static_cast<const uint16_t*>(scales)[at * C::NB + ch / 4];
  } else {
    const uint2 c = static_cast<const uint2*>(rows)[at * C::CH + ch];
    x.c.x = c.x;
    x.c.y = c.y;
    x.s = static_cast<const float*>(scales)[at];
  }
  return x;
}
template <int KIND>
__device__ __forceinline__ uint4 row8_bf16(const StoredRow8<KIND>& x) {
  if constexpr (KIND == ROWS_BF16) {
    return x.c;
  } else if constexpr (KIND == ROWS_INT4) {
    return i4_dequantise8(x.c.x, x.h);
  } else {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = f8_pair_bf16((uint16_t)((i < 2 ? x.c.x : x.c.y) >> (16 * (i & 1))), x.s);
    return make_uint4(r[0], r[1], r[2], r[3]);
  }
}

// Reads T positions of a cache back as bf16 rows. Bound by writing them, which
// DRAM takes at ~3.8 TB/s where little is read beside them: 131,071 rows of 8 heads
// of 64 from INT4 in 68.6 us (268 MB written, 75 MB read), from FP8 in 77.9, from bf16
// in 93.8 (as many read as written: 5.7 TB/s). Where the rows written stay in L2 (25 MB:
// 3 x 4,099 rows of 4 heads of 128 from FP8 in 9.3 us) it is a launch and one short
// wave of loads.
template <int D, int KIND, int NR>
__global__ void __launch_bounds__(256) kv_read_kernel(const RowsParams p) {
  using C = RowsCfg<D>;
  griddep_launch_dependents();
  griddep_wait();
  const int g = blockIdx.y, b = blockIdx.z;
  const int rb = threadIdx.x / C::CH, ch = threadIdx.x - rb * C::CH;
  if (rb >= C::RB) return;
  const int t0 = blockIdx.x * (C::RB * NR) + rb;
  const long long row_bg = ((long long)b * p.n_kv + g) * p.cap;
  StoredRow8<KIND> kr[NR], vr[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int t = t0 + i * C::RB;
    long long row = (long long)p.row0 + t;
    if (row >= p.cap) row -= p.cap;
    const long long at = row_bg + row;
    if (t < p.T) {
      kr[i] = load_row8<D, KIND>(p.ck, p.cks, at, ch);
      vr[i] = load_row8<D, KIND>(p.cv, p.cvs, at, ch);
    }
  }
  __nv_bfloat16* k = const_cast<__nv_bfloat16*>(p.k) + b * p.ks0 + g * p.ks2 + 8 * ch;
  __nv_bfloat16* v = const_cast<__nv_bfloat16*>(p.v) + b * p.vs0 + g * p.vs2 + 8 * ch;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int t = t0 + i * C::RB;
    if (t < p.T) {
      *reinterpret_cast<uint4*>(k + t * p.ks1) = row8_bf16<KIND>(kr[i]);
      *reinterpret_cast<uint4*>(v + t * p.vs1) = row8_bf16<KIND>(vr[i]);
    }
  }
}

}  // namespace sa
