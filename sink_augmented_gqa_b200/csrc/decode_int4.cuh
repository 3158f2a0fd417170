// One-token decode over an INT4 cache (int4.cuh). The split of the rows over
// CTAs, the ring of stages, the new row and the merge of partials are
// decode_kernel's (decode.cuh); this file is the part that differs: 4.5 bits
// an element leave about a quarter of the issue slots per key that the bf16
// cache leaves, so the codes go to the tensor cores with as few instructions
// as possible.
//
// S = Q K^T, m16n8k16 in f16, queries on the M side and 8 keys on the N side:
//   A code word w (8 nibbles) gives four f16 pairs by masks alone, plus one
//   shift: w & 0x000F000F as f16 are the subnormals u 2^-24 of nibbles 0 and
//   4, w & 0x00F000F0 those of nibbles 1 and 5 times 16, and the same of
//   w >> 8. The queries' fragments take that order, with 1/16 in the second
//   registers; they are f16 after a power-of-two scaling per head, exact for
//   bf16 queries down to 2^-25 of the largest. The codes' offset of 8 is the
//   accumulator's start, -8 2^-24 sum of q over the block, and a block's
//   scale multiplies its 32-element partial sum afterwards, in fp32.
//   Queries on the M side waste half of the instruction (8 of 16 rows) but
//   give a lane the scores of one head at keys 2t, 2t + 1 of each octet, the
//   fragment that O^T = V^T P^T takes as its B operand, so the weights never
//   cross lanes, and a maximum needs two shuffles.
// O^T += V^T P'^T, m16n8k16 in bf16 (the weights p * scale_v span any range):
//   ldmatrix.trans over 16-bit units hands a lane the same 4 codes of two
//   neighbouring keys; 0x4300 | u is the bf16 number 128 + u, and the offset
//   136 goes out by a product of the weights with a constant -136 just before
//   (a running sum of 136 P' beside O would lose what the tensor core's
//   truncation of its sums takes from a number 30 times as large).
#pragma once

#include "decode.cuh"
#include "int4.cuh"

namespace sa {

template <int D>
struct DecodeI4Cfg {
  static constexpr int NCW = 8;                 // consumer warps
  static constexpr int RW = 32;                 // rows per consumer warp and stage
  static constexpr int R = RW * NCW;
  static constexpr int NBOX = R / 128;          // 128-row TMA boxes per stage
  static constexpr int NB = D / kI4Block;       // blocks per row
  static constexpr int ROWB = D / 2;            // code bytes per row
  static constexpr uint32_t STAGE_BYTES = R * ROWB;
  static constexpr uint32_t SC_BYTES = R * NB * 2;   // K (or V) scales of one stage
  static constexpr int NS = (D == 128) ? 2 : 3;
  static constexpr uint32_t STAGE_TX = 2 * (STAGE_BYTES + SC_BYTES);
  static constexpr int NUM_THREADS = 32 * (NCW + 1);
  static constexpr uint32_t OFF_K = 0;
  static constexpr uint32_t OFF_V = NS * STAGE_BYTES;
  static constexpr uint32_t RING_BYTES = 2 * NS * STAGE_BYTES;   // K and V codes
  // the new row: one warp's tile of codes and scales, row 0 valid
  static constexpr uint32_t XTILE = RW * ROWB;
  static constexpr uint32_t OFF_XK = RING_BYTES;
  static constexpr uint32_t OFF_XV = OFF_XK + XTILE;
  static constexpr uint32_t OFF_KS = OFF_XV + XTILE;             // [NS][R][NB] bf16
  static constexpr uint32_t OFF_VS = OFF_KS + NS * SC_BYTES;
  static constexpr uint32_t OFF_XS = OFF_VS + NS * SC_BYTES;     // [2][RW][NB] bf16
  static constexpr uint32_t OFF_RED = OFF_K;
  static constexpr uint32_t RED_WARP = (16 + 8 * D) * 4;
  static_assert(NCW * RED_WARP <= RING_BYTES, "warp partials must fit in the ring");
  static_assert(OFF_XK % 1024 == 0 && STAGE_BYTES % 1024 == 0 && XTILE % 512 == 0,
                "swizzled tiles start on a multiple of their pattern");
  static constexpr uint32_t OFF_BAR = OFF_XS + 2 * RW * NB * 2;
  static constexpr uint32_t OFF_MBAR = OFF_BAR + 8 * (2 * NS);
  static constexpr uint32_t OFF_FLAG = OFF_MBAR + 8;
  static constexpr uint32_t OFF_SINK = OFF_FLAG + 16;
  static constexpr uint32_t OFF_SROW = OFF_SINK + 32;   // [NS] first cache position of each stage
  static constexpr uint32_t SMEM_BYTES = OFF_SROW + 8 * NS + 1024;
  static_assert(OFF_BAR % 16 == 0 && OFF_KS % 16 == 0, "barriers and bulk copies");
};

// Byte offset of 16-byte block blk of a row in a tile of ROWB-byte rows as
// TMA lays it out: 32-byte rows swizzled over 32 bytes, 64-byte rows over 64,
// 48-byte rows plain. In each, the eight rows an ldmatrix phase reads lie in
// distinct banks.
template <int D>
__device__ __forceinline__ uint32_t i4_off(int row, int blk) {
  constexpr int ROWB = D / 2;
  constexpr uint32_t MASK = (ROWB == 32) ? 1 : (ROWB == 64 ? 3 : 0);
  const uint32_t off = (uint32_t)row * ROWB + 16u * blk;
  return off ^ (((off >> 7) & MASK) << 4);
}

// The scales of rows r, r + 1 (r even) as fp32, s[blk] = {row r, row r + 1}.
template <int NB>
__device__ __forceinline__ void i4_scales(uint32_t addr, float (&s)[NB][2]) {
  uint32_t w[NB];
  if constexpr (NB == 2) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  } else if constexpr (NB == 4) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr));
  } else {
#pragma unroll
    for (int i = 0; i < NB; ++i) w[i] = ld_shared_u32(addr + 4 * i);
  }
#pragma unroll
  for (int i = 0; i < 2 * NB; ++i)
    s[i % NB][i / NB] = (i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
}

__device__ __forceinline__ void mma_16816_f16_half(float (&c)[4], uint32_t a0, uint32_t a2, uint32_t b0,
                                                   uint32_t b1) {
  mma_16816_f16(c, a0, 0u, a2, 0u, b0, b1);
}

// One warp's 32 keys of a stage: codes at kst / vst plus this lane's offsets
// off[blk] (row = lane, see the kernel), scales of the warp's first row at
// ksc / vsc. With MASK, keys below n_first and from n_valid on are masked
// (their scales may hold anything). m, l: running maximum (log2 units) and
// sum of head lane / 4; o[blk][i]: the accumulators of d = 32 blk + 4 (lane /
// 4) + 2 i + {0, 1} (fragment rows g and g + 8) for heads 2 (lane % 4) + {0, 1}.
template <int D, bool MASK>
__device__ __forceinline__ void decode_tile_i4(uint32_t kst, uint32_t vst, const uint32_t (&off)[D / 32],
                                               uint32_t ksc, uint32_t vsc, int n_first, int n_valid,
                                               const uint32_t (&qf)[D / 32][4], const float (&qo)[D / 32],
                                               float hs, float& m, float& l, float (&o)[D / 32][2][4], int lane) {
  constexpr int NB = D / 32;
  const int t2 = 2 * (lane & 3);
  float s[4][2];
#pragma unroll
  for (int c = 0; c < 4; ++c) s[c][0] = s[c][1] = 0.f;
  {
    float sk[4][NB][2];
#pragma unroll
    for (int c = 0; c < 4; ++c) i4_scales<NB>(ksc + (uint32_t)((8 * c + t2) * NB * 2), sk[c]);
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      uint32_t w[4];
      ldmatrix_x4(kst + off[blk], w[0], w[1], w[2], w[3]);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float a[4] = {qo[blk], qo[blk], 0.f, 0.f};
        mma_16816_f16_half(a, qf[blk][0], qf[blk][1], w[c] & 0x000F000Fu, w[c] & 0x00F000F0u);
        const uint32_t w8 = w[c] >> 8;
        mma_16816_f16_half(a, qf[blk][2], qf[blk][3], w8 & 0x000F000Fu, w8 & 0x00F000F0u);
        s[c][0] = fmaf(sk[c][blk][0], a[0], s[c][0]);
        s[c][1] = fmaf(sk[c][blk][1], a[1], s[c][1]);
      }
    }
  }
  float mx = -INFINITY;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int key = 8 * c + t2 + e;
      s[c][e] = (!MASK || (key >= n_first && key < n_valid)) ? s[c][e] * hs : -INFINITY;
    }
    mx = max3f(mx, s[c][0], s[c][1]);
  }
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  const float m_new = fmaxf(m, mx);
  const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
  const float alpha = ex2(m - m_use);
  m = m_new;
  // the accumulators move only when some head's maximum grew
  if (__any_sync(0xffffffffu, alpha != 1.f)) {
    l *= alpha;
    const float f0 = __shfl_sync(0xffffffffu, alpha, 4 * t2), f1 = __shfl_sync(0xffffffffu, alpha, 4 * t2 + 4);
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        o[blk][i][0] *= f0;
        o[blk][i][1] *= f1;
        o[blk][i][2] *= f0;
        o[blk][i][3] *= f1;
      }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    s[c][0] = ex2(s[c][0] - m_use);
    s[c][1] = ex2(s[c][1] - m_use);
    l += s[c][0] + s[c][1];
  }
  uint32_t pb[4][NB];   // weights of octet c's keys 2t, 2t + 1 for block blk, bf16
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float sv[NB][2];
    i4_scales<NB>(vsc + (uint32_t)((8 * c + t2) * NB * 2), sv);
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      float p0 = s[c][0] * sv[blk][0], p1 = s[c][1] * sv[blk][1];
      if (MASK) {   // 0, whatever a row never written holds as its scale
        const int key = 8 * c + t2;
        if (!(key >= n_first && key < n_valid)) p0 = 0.f;
        if (!(key + 1 >= n_first && key + 1 < n_valid)) p1 = 0.f;
      }
      pb[c][blk] = pack_bf16(p0, p1);
    }
  }
  constexpr uint32_t NEG136 = 0xC308C308u;   // bf16 -136, twice
  constexpr uint32_t NIB = 0x000F000Fu, BASE = 0x43004300u;
#pragma unroll
  for (int blk = 0; blk < NB; ++blk) {
    uint32_t x[4];
    ldmatrix_x4_trans(vst + off[blk], x[0], x[1], x[2], x[3]);
#pragma unroll
    for (int c = 0; c < 4; c += 2) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mma_16816(o[blk][i], NEG136, NEG136, NEG136, NEG136, pb[c][blk], pb[c + 1][blk]);
        mma_16816(o[blk][i], ((x[c] >> (8 * i)) & NIB) | BASE, ((x[c] >> (8 * i + 4)) & NIB) | BASE,
                  ((x[c + 1] >> (8 * i)) & NIB) | BASE, ((x[c + 1] >> (8 * i + 4)) & NIB) | BASE, pb[c][blk],
                  pb[c + 1][blk]);
      }
    }
  }
}

// tmK / tmV: the codes, dims {D / 2, rows, n_kv, B} bytes. p.ck, p.cv, p.cks,
// p.cvs hold the cache's code and scale arrays.
template <int D>
__global__ void __launch_bounds__(288, 2)
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
  // flag[0]: abort, flag[1]: "this CTA merges the splits"
  float* sink_sm = reinterpret_cast<float*>(smem + C::OFF_SINK);   // [q_mult] sinks, log2 units
  // position of each ring slot's first row, or -1: the producer has no more stages
  volatile long long* srow = reinterpret_cast<volatile long long*>(smem + C::OFF_SROW);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int g = blockIdx.x;
  const int split = blockIdx.y;
  const int b = blockIdx.z;
  const int QM = p.q_mult;
  const long long bg = (long long)b * p.n_kv + g;

  // static stages first, then dynamic ones (decode_kernel)
  const int F = p.static_stages;
  const long long s_begin = (long long)split * F;
  const bool dyn = (long long)p.S * F < p.n_blocks;
  const bool last_split = split == p.S - 1;
  // scale rows of the 128-row box at cache row `row`, position pos: whole
  // 16-row groups up to the last cached one (cap is a multiple of 16)
  auto scale_rows = [&](long long pos) -> int {
    if (p.ring_cap > 0) return 128;
    const long long n = p.off - pos;
    return n <= 0 ? 0 : (n >= 128 ? 128 : (int)((n + 15) / 16 * 16));
  };
  const char* ksc_g = reinterpret_cast<const char*>(p.cks) + bg * p.cap * NB * 2;
  const char* vsc_g = reinterpret_cast<const char*>(p.cvs) + bg * p.cap * NB * 2;

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
  // the first stages go into L2 while the kernel before this one drains
  if (warp == C::NCW && lane == 0 && p.n_blocks > 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    const int pf = F < p.pf_stages ? F : p.pf_stages;
    for (int it = 0; it < pf; ++it) {
#pragma unroll
      for (int bx = 0; bx < C::NBOX; ++bx) {
        const long long pos = p.lo + (s_begin + it) * C::R + 128 * bx;
        const int row = (int)(p.ring_cap > 0 ? pos % p.ring_cap : pos);
        tma_prefetch_l2_4d(&tmK, 0, row, g, b);
        tma_prefetch_l2_4d(&tmV, 0, row, g, b);
        const uint32_t bytes = (uint32_t)scale_rows(pos) * NB * 2;
        if (bytes > 0) {
          bulk_prefetch_l2(ksc_g + (long long)row * NB * 2, bytes);
          bulk_prefetch_l2(vsc_g + (long long)row * NB * 2, bytes);
        }
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
      int* grab = p.ws_grab + bg;
      int pending = dyn ? atomicAdd(grab, 1) : 0;   // the first dynamic stage, asked for early
      int it = 0;
      for (int k = 0; !flag[0]; ++k) {
        long long sidx;
        if (k < F) {
          sidx = s_begin + k;
        } else {
          if (!dyn) break;
          sidx = (long long)p.S * F + pending;
          if (sidx >= p.n_blocks) break;
          pending = atomicAdd(grab, 1);
        }
        const int s = it % C::NS;
        if (!mbar_wait(empty_bar(s), (uint32_t)(((it / C::NS) & 1) ^ 1))) { flag[0] = 1; break; }
        const long long pos0 = p.lo + sidx * C::R;
        srow[s] = pos0;
        uint32_t tx = 2 * C::STAGE_BYTES;
#pragma unroll
        for (int bx = 0; bx < C::NBOX; ++bx) tx += 2u * NB * 2u * (uint32_t)scale_rows(pos0 + 128 * bx);
        mbar_arrive_expect_tx(full_bar(s), tx);
#pragma unroll
        for (int bx = 0; bx < C::NBOX; ++bx) {
          // boxes of 128 rows that start on multiples of 128: none wraps a ring
          const long long pos = pos0 + 128 * bx;
          const int row = (int)(p.ring_cap > 0 ? pos % p.ring_cap : pos);
          const uint32_t boff = (uint32_t)bx * 128u * C::ROWB;
          tma_load_4d(sbase + C::OFF_K + s * C::STAGE_BYTES + boff, &tmK, full_bar(s), 0, row, g, b);
          tma_load_4d(sbase + C::OFF_V + s * C::STAGE_BYTES + boff, &tmV, full_bar(s), 0, row, g, b);
          const uint32_t bytes = (uint32_t)scale_rows(pos) * NB * 2;
          if (bytes > 0) {
            const uint32_t so = s * C::SC_BYTES + (uint32_t)bx * 128u * NB * 2u;
            bulk_load(sbase + C::OFF_KS + so, ksc_g + (long long)row * NB * 2, bytes, full_bar(s));
            bulk_load(sbase + C::OFF_VS + so, vsc_g + (long long)row * NB * 2, bytes, full_bar(s));
          }
        }
        ++it;
      }
      // the end of this CTA's stream: a slot marked -1, completed by a plain arrive
      if (!flag[0]) {
        const int s = it % C::NS;
        if (mbar_wait(empty_bar(s), (uint32_t)(((it / C::NS) & 1) ^ 1))) {
          srow[s] = -1;
          mbar_arrive(full_bar(s));
        } else {
          flag[0] = 1;
        }
      }
      if (flag[0]) {
        for (int j = (it > C::NS ? it - C::NS : 0); j < it; ++j)
          mbar_wait_drain(full_bar(j % C::NS), (uint32_t)((j / C::NS) & 1));
      }
    }
    return;  // the producer takes no part in the merge (named barriers below count 32*NCW)
  }

  // ---------------------------------------------------------------- consumers
  const float sink_in = (threadIdx.x < QM && p.sinks) ? p.sinks[g * QM + threadIdx.x] : -INFINITY;
  const bool new_row = last_split && warp == 0;
  const float* ctab = p.cos_t + p.off * HALF;
  const float* stab = p.sin_t + p.off * HALF;

  // The new row, 8 elements a lane: lanes 0.. its K, lanes 16.. its V.
  constexpr int CH = D / 8;
  const int nch = lane & 15;                       // this lane's chunk
  const bool n_live = new_row && nch < CH, n_is_v = lane >= 16;
  uint4 na = make_uint4(0, 0, 0, 0), nb = na;      // the chunk's RoPE pair (K), or the chunk (V)
  float4 nc0, nc1, ns0, ns1;
  const int nlo = nch < CH / 2 ? nch : nch - CH / 2;
  nc0 = nc1 = ns0 = ns1 = make_float4(0.f, 0.f, 0.f, 0.f);
  if (n_live) {
    if (n_is_v) {
      na = *reinterpret_cast<const uint4*>(p.v + b * p.vs0 + (long long)g * p.vs2 + 8 * nch);
    } else {
      const __nv_bfloat16* krow = p.k + b * p.ks0 + (long long)g * p.ks2;
      na = *reinterpret_cast<const uint4*>(krow + 8 * nlo);
      nb = *reinterpret_cast<const uint4*>(krow + 8 * nlo + HALF);
      if (p.rope) {
        nc0 = *reinterpret_cast<const float4*>(ctab + 8 * nlo);
        nc1 = *reinterpret_cast<const float4*>(ctab + 8 * nlo + 4);
        ns0 = *reinterpret_cast<const float4*>(stab + 8 * nlo);
        ns1 = *reinterpret_cast<const float4*>(stab + 8 * nlo + 4);
      }
    }
  }

  // Query fragments (A operand): row lane / 4 = head, elements 32 blk + 8 t +
  // {0, 4}, {1, 5}, {2, 6}, {3, 7} (t = lane % 4), rotated at position off.
  uint32_t qf[NB][4];
  float qo[NB], hs;
  {
    const int n = lane >> 2, t = lane & 3;
    const bool hv = n < QM;
    const __nv_bfloat16* qrow = p.q + b * p.qs0 + (long long)(g * QM + (hv ? n : 0)) * p.qs2;
    float qv[NB][8];
    float amax = 0.f;
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      const int c0 = 32 * blk + 8 * t;               // this lane's 8 elements of the block
      const int lo = c0 < HALF ? c0 : c0 - HALF;
      uint4 a = *reinterpret_cast<const uint4*>(qrow + lo), c = *reinterpret_cast<const uint4*>(qrow + lo + HALF);
      if (p.rope) rotate8(a, c, ctab + lo, stab + lo);
      const uint4 u = c0 < HALF ? a : c;
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        qv[blk][i] = hv ? ((i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1])) : 0.f;
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
    hs = p.scale_log2 * __uint_as_float((uint32_t)(127 + eq) << 23) * 0x1p24f;
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
        qf[blk][i] = pack_f16(qv[blk][i] * f, qv[blk][i + 4] * f);
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      qo[blk] = sum * (-8.0f * 0x1p-24f);
    }
  }
  if (threadIdx.x < QM) sink_sm[threadIdx.x] = sink_in * 1.4426950408889634f;

  uint32_t off[NB];   // this lane's ldmatrix row (row `lane` of the warp's 32) in a stage
#pragma unroll
  for (int blk = 0; blk < NB; ++blk) off[blk] = i4_off<D>(C::RW * warp + lane, blk);

  float m = -INFINITY, l = 0.f;
  float o[NB][2][4];
#pragma unroll
  for (int blk = 0; blk < NB; ++blk)
#pragma unroll
    for (int i = 0; i < 2; ++i) o[blk][i][0] = o[blk][i][1] = o[blk][i][2] = o[blk][i][3] = 0.f;

  // Quantise the new row, write it to the cache and stage it in smem as row
  // 0 of a tile (the other rows are masked).
  if (new_row) {
    if (!n_is_v) {
      if (p.rope) rotate8_regs(na, nb, nc0, nc1, ns0, ns1);
      if (nch >= CH / 2) na = nb;
    }
    uint16_t sc;
    const uint32_t codes = i4_quantise8(na, sc);
    if (n_live) {
      const long long slot = p.ring_cap > 0 ? p.off % p.ring_cap : p.off;
      const long long crow = bg * p.cap + slot;
      uint32_t* cc = reinterpret_cast<uint32_t*>(n_is_v ? p.cv : p.ck) + crow * CH + nch;
      uint16_t* cs = reinterpret_cast<uint16_t*>(n_is_v ? p.cvs : p.cks) + crow * NB + nch / 4;
      *cc = codes;
      *reinterpret_cast<uint32_t*>(smem + (n_is_v ? C::OFF_XV : C::OFF_XK) + i4_off<D>(0, nch / 4) + 4 * (nch & 3)) =
          codes;
      if ((nch & 3) == 0) {
        *cs = sc;
        reinterpret_cast<uint16_t*>(smem + C::OFF_XS)[(n_is_v ? C::RW * NB : 0) + nch / 4] = sc;
      }
    }
    __syncwarp();
  }

  for (int it = 0;; ++it) {
    const int s = it % C::NS;
    if (!mbar_wait(full_bar(s), (uint32_t)((it / C::NS) & 1))) { flag[0] = 1; break; }
    const long long pos0 = srow[s];
    if (pos0 < 0) break;   // the producer's end mark
    const long long row0 = pos0 + C::RW * warp;
    const long long nv = p.off - row0;
    const long long nf = p.lo_mask - row0;
    if (nv > 0 && nf < C::RW && !flag[0]) {
      const uint32_t kst = sbase + C::OFF_K + s * C::STAGE_BYTES, vst = sbase + C::OFF_V + s * C::STAGE_BYTES;
      const uint32_t so = s * C::SC_BYTES + (uint32_t)(C::RW * warp * NB * 2);
      const uint32_t ks = sbase + C::OFF_KS + so, vs = sbase + C::OFF_VS + so;
      if (nf <= 0 && nv >= C::RW)
        decode_tile_i4<D, false>(kst, vst, off, ks, vs, 0, C::RW, qf, qo, hs, m, l, o, lane);
      else
        decode_tile_i4<D, true>(kst, vst, off, ks, vs, nf > 0 ? (int)nf : 0, nv > C::RW ? C::RW : (int)nv, qf, qo,
                                hs, m, l, o, lane);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty_bar(s));
  }
  if (new_row) {
    uint32_t xo[NB];
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) xo[blk] = i4_off<D>(lane, blk);
    const uint32_t xs = sbase + C::OFF_XS;
    decode_tile_i4<D, true>(sbase + C::OFF_XK, sbase + C::OFF_XV, xo, xs, xs + C::RW * NB * 2, 0, 1, qf, qo, hs, m,
                            l, o, lane);
  }

  // ---------------------------------------------------------------- merge the consumer warps
  named_bar_sync(1, 32 * C::NCW);   // every warp is done reading the K/V ring
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
  {
    float* rw = reinterpret_cast<float*>(smem + C::OFF_RED) + warp * (C::RED_WARP / 4);
    const int t = lane & 3, gq = lane >> 2;
    if (t == 0) {
      rw[gq] = m;
      rw[8 + gq] = l;
    }
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int d0 = 32 * blk + 4 * gq + 2 * i;
        rw[16 + (2 * t) * D + d0] = o[blk][i][0];
        rw[16 + (2 * t + 1) * D + d0] = o[blk][i][1];
        rw[16 + (2 * t) * D + d0 + 1] = o[blk][i][2];
        rw[16 + (2 * t + 1) * D + d0 + 1] = o[blk][i][3];
      }
  }
  named_bar_sync(1, 32 * C::NCW);
  decode_finish<D, C>(p, smem, sbase, merge_bar, flag, sink_sm, g, split, b);
}

}  // namespace sa
