// pa_kv4.cuh -- persistent, warp-specialised paged decode attention over a
// cache held in 4 bits (phase 1; the partitions are combined by pa_combine.cuh).
//
// Cache record of one (block, kv head), BS * (D + 8) bytes (x = min(D, 128)):
//
//   key codes    [D/x][BS][x/2]   two 4-bit codes a byte, the even dim in the low nibble
//   value codes  [D/x][BS][x/2]
//   parameters   [BS][4] of T     key scale, key zero, value scale, value zero of a token
//
// and a code c stands for scale * c + zero.  Neither product therefore needs a
// dequantised element:
//
//   q . k_t        = ks_t (q . c_t) + kz_t sum(q)
//   sum p_t v_t[d] = sum (p_t vs_t) c_t[d] + sum p_t vz_t
//
// The codes enter the tensor cores as fp16 bit patterns: a nibble masked out
// at bits 0-3 of a half is the subnormal c * 2^-24, at bits 4-7 c * 2^-20,
// both exact, so a register of two operands costs one AND (and a shift for
// every second one); no conversion instruction is issued.  The factor 16
// between the two positions is taken out of the query (scores) or of the
// finished accumulator rows (values).
//
// Roundings below 32 bits, besides the codes: the query is scaled by a power
// of two into fp16's range (exact, except for elements more than 2^24 below
// the unit's largest), and the weights p_t vs_t enter the value product as
// fp16.  A weight's rounding error meets the code, whose mean is far from
// zero; it is kept to the spread of the codes (c - 8) by summing the rounded
// weights themselves (one more product, with rows of code 8) and putting
// 8 p_t vs_t back in fp32 with the zeros.  The weights are scaled by the power
// of two 2^7 / vb, vb above every value scale the warp has met (raised, with
// the accumulators, when a larger one comes), so they stay in fp16's range
// whatever the cache's magnitude.
//
// Softmax without a reduction per item: each column keeps a reference (a
// maximum it has met) and raises it only when a score passes it by more than
// 2^8, which one vote per item finds out; weights stay below 2^8, sums and
// accumulators in fp32.  Most items need no shuffle, no rescaling.
//
// Rows and slots.  MMA row i of a 16-token score tile holds token kTok(i):
// 0 7 1 6 2 5 3 4, then 8 more of the same.  The 4-byte words of a token row
// go to the lane quads in contiguous runs (one 16-byte load for D = 128),
// and with this order the rows one load phase touches fall in distinct banks
// for rows of 32 and 64 bytes.  A value word holds 8 dims of one token; words
// of two tokens are interleaved by halves (PRMT), so a masked register is a
// dim's pair of token slots.  Lane group r holds dims 16r .. 16r + 15 of a
// 128-dim slab (8r .. 8r + 7 of D = 64).  Head sizes that are not a multiple
// of 64 run padded: the words past a row's end are other bytes of the record,
// which the zeroed query slots, or leaving the accumulator rows out, ignore
// (every nibble is a finite number).
//
// Work unit = (sequence, partition, kv head, GT of its query rows), taken by a
// team of TW warps of one CTA (TW = 1, 2, 4 ..: as many as make enough teams'
// worth of units, choose_team); each warp takes a contiguous run of the
// partition's tokens.  One CTA of NC equal warps per SM, no producer: a warp
// owns a ring of a few 32-token stages and refills a stage itself, by one bulk
// copy per block, right after it has used it, so no warp waits for another
// while it streams.  What was measured on the way to this: a team of all the
// SM's warps with one warp that merges their states (the scheme of
// pa_kernel.cuh) spends more on set-ups, hand-overs and the merging warp than
// on the tokens, as a 4-bit partition holds a quarter of the bytes.  A warp of
// a team of one writes its unit itself; larger teams meet once per unit, leave
// their states in their rings and each merge a slice of the rows.
#pragma once

#include "pa_common.cuh"
#include "pa_kernel.cuh"

namespace pa {

#ifndef PA_KV4_UNITS
#define PA_KV4_UNITS 5
#endif

// TB: tokens per block.
template <typename T_, int D_, int NT_, int TB_>
struct Kv4 {
  using T = T_;
  static constexpr int D = D_, NT = NT_, GT = 8 * NT_, TB = TB_;
#ifndef PA_KV4_TILES
#define PA_KV4_TILES 4
#endif
  // 16-token tiles per stage (two at head size 256, for three stages in the ring).
  static constexpr int NTI = D_ > 128 && TB_ < 64 ? 2 : PA_KV4_TILES;
  static constexpr int TS = 16 * NTI;            // tokens per stage
  static constexpr int NBLK = TS / TB_;          // blocks per stage
  static_assert(NBLK >= 1, "a stage holds whole blocks");
  static constexpr uint32_t REC = (uint32_t)TB_ * (D_ + 8), STAGE = REC * NBLK;
  // Warps per CTA: as many as the accumulators' registers allow (128 or 255 a thread).
#ifndef PA_KV4_NC
#define PA_KV4_NC 8
#endif
  static constexpr int NC = D_ > 128 && TB_ == 64 ? 4 : (D_ <= 128 && NT_ == 1) ? PA_KV4_NC : 8;
  static_assert((NC & (NC - 1)) == 0, "teams of a power of two");
  static constexpr int THREADS = NC * 32;
  static constexpr int X = D_ < 128 ? D_ : 128;  // dims per slab
  static constexpr int NSLAB = D_ / X;
  static constexpr int XB = X / 2;               // bytes of a token row in a slab
  static_assert(D_ % X == 0 && X % 16 == 0, "whole slabs");
  // 4-byte words of a slab row per lane quad member (keys) and per lane group (values).
  static constexpr int KW = (X / 8 + 3) / 4;
  static constexpr int VW = (X / 8 + 7) / 8;
  static constexpr int NK = NSLAB * KW * 2;      // k-steps of the score product
  static constexpr int MTS = VW * 4;             // 16-dim tiles of a slab's value product
  static constexpr int NMT = NSLAB * MTS;
  static constexpr int NSMAX = 8;                // ring stages per warp
  static constexpr int AROW = D_ + 4;            // floats of a handed-over row (16 bytes past it, for the banks)
  static constexpr uint32_t STATE = GT * AROW * 4 + GT * 2 * 4;
  static constexpr uint32_t SZ_BAR = NC * NSMAX * 8;
  static constexpr uint32_t SZ_PREF = (kMaxSeqsPerLaunch + 1) * 4;
  static constexpr uint32_t FIXED = al16(SZ_BAR) + 64 + 256 + al16(SZ_PREF);
  static constexpr uint32_t BUDGET = 227 * 1024;
  static constexpr uint32_t RING = (BUDGET - FIXED) / NC / 128 * 128;  // bytes per warp
  static constexpr uint32_t OFF_BAR = NC * RING, OFF_FLAGS = OFF_BAR + al16(SZ_BAR), OFF_NEXT = OFF_FLAGS + 64,
                            OFF_PREF = OFF_NEXT + 256, BYTES = OFF_PREF + al16(SZ_PREF);
  static_assert(BYTES <= BUDGET, "shared memory over budget");
  static constexpr int NS = RING / STAGE < NSMAX ? RING / STAGE : NSMAX;  // ring stages per warp
  static_assert(STATE <= RING && NS >= 1, "a warp's state and a stage fit its ring");
};

// What a CTA derives from the launch and the lengths.
struct Kv4Plan {
  int TW;             // warps per unit
  int n_hg;           // units per partition: KH * hg_per_kv
  int total;          // units
};

// Warps per unit: the fewest that give the grid's teams a few units each (an
// even end), but no more than a partition has stages.
template <class K>
__device__ __forceinline__ Kv4Plan make_plan(const KParams& prm, int partitions) {
  Kv4Plan pl;
  pl.n_hg = prm.KH * prm.hg_per_kv;
  pl.total = partitions * pl.n_hg;
  const long long want = (long long)PA_KV4_UNITS * gridDim.x * K::NC;
  int tw = 1;
  while (tw < K::NC && tw * K::TS < prm.P && (long long)pl.total * tw < want) tw *= 2;
  pl.TW = tw;
  return pl;
}

// ---------------------------------------------------------------- small pieces
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t lds_b32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void lds_b64(uint32_t a, uint32_t& x, uint32_t& y) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(a));
}
__device__ __forceinline__ void lds_b128(uint32_t a, uint32_t* v) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(a));
}
// One lane of the warp (the compiler issues what it does from uniform
// registers; copies by several lanes would be a loop over them).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
// fp16 products, accumulated in fp32; `first`: from zero.
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Offsets within a stage (a constant each).
template <class K>
struct Kv4Offsets {
  static constexpr uint32_t slab = K::TB * K::XB;     // slab 1 after slab 0
  static constexpr uint32_t voff = K::TB * K::D / 2;  // value codes in a record
  static constexpr uint32_t poff = K::TB * K::D;      // parameters in a record
  // Tokens 8..15 of a tile after 0..7: codes, parameters.
  static constexpr uint32_t hd = K::TB == 8 ? K::REC : 8 * K::XB;
  static constexpr uint32_t hdp = K::TB == 8 ? K::REC : 64;
  // Tile t.
  __device__ static constexpr uint32_t tile(int t) {
    return (uint32_t)(16 * t / K::TB) * K::REC + (uint32_t)(16 * t % K::TB) * K::XB;
  }
  __device__ static constexpr uint32_t tilep(int t) {
    return (uint32_t)(16 * t / K::TB) * K::REC + (uint32_t)(16 * t % K::TB) * 8;
  }
};

// ---------------------------------------------------------------- a consumer warp's state
template <class K>
struct Kv4State {
  using T = typename K::T;
  static constexpr int NT = K::NT, NK = K::NK, NMT = K::NMT, KW = K::KW, VW = K::VW, NSLAB = K::NSLAB, NTI = K::NTI;
  static constexpr uint32_t LO = 0x000f000fu, HI = 0x00f000f0u;

  uint32_t qb[NT][NK][2];          // Q^T fragments: the query row of column lane / 4
  float ms[NT][2], thr[NT][2];     // reference (0 until set); 8, or -inf until it is set
  float l[NT][2], zs[NT][2];       // sums of weights; of weight * (value zero + 8 value scale)
  float qz[NT][2];                 // scale_log2 * sum(q)
  float acc[NMT][NT][4], acc8[NT][4];
  float kf;                        // score factor: scale_log2 over the operands' powers of two
  float vb, vinv;                  // see the top: a power of two, and 2^7 / vb
  int lim[NT][2], minlim;          // positions the lane's columns see; the warp's least
  // The lane's offsets in a tile: key words, parameters, values of the first
  // and second token of its slots.
  uint32_t ko, po, vo, vo2;

  __device__ __forceinline__ explicit Kv4State(int lane) {
    const int r = lane >> 2, c = lane & 3;
    ko = tok_lo(r) * K::XB + c * (KW * 4);
    po = tok_lo(r) * 8;
    // Slots 2c, 2c + 1 and 2c + 8, 2c + 9 hold tokens c, 7 - c, 8 + c, 15 - c.
    vo = c * K::XB + r * (VW * 4);
    vo2 = (7 - c) * K::XB + r * (VW * 4);
    // (Opaque: kept in registers rather than computed again for every stage,
    // which cost 30 instructions of 500.)
    asm volatile("" : "+r"(ko), "+r"(po), "+r"(vo), "+r"(vo2));
  }

  __device__ __forceinline__ static int tok_lo(int i) { return (i & 1) ? 7 - (i >> 1) : (i >> 1); }

  __device__ __forceinline__ static void key_words(uint32_t a, uint32_t (&w)[KW]) {
    if constexpr (KW == 4 && K::XB % 16 == 0) {
      lds_b128(a, w);
    } else if constexpr (KW % 2 == 0) {
#pragma unroll
      for (int i = 0; i < KW; i += 2) lds_b64(a + 4 * i, w[i], w[i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < KW; ++i) w[i] = lds_b32(a + 4 * i);
    }
  }
  __device__ __forceinline__ static void value_words(uint32_t a, uint32_t (&w)[2]) {
    if constexpr (VW == 2) {
      lds_b64(a, w[0], w[1]);
    } else {
      w[0] = lds_b32(a);
      w[1] = 0u;
    }
  }

  // row(i): the unit's query row i (of nh), in global memory.
  template <class F>
  __device__ __forceinline__ void begin_unit(F row, int nh, float sl2, int lane) {
    const int n = lane >> 2, c = lane & 3;
    // Dims 8w .. 8w + 7 of a slab are word w; this lane holds words c * KW ...
    uint4 v[NT][NSLAB * KW];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const T* q = 8 * t + n < nh ? row(8 * t + n) : nullptr;
#pragma unroll
      for (int sl = 0; sl < NSLAB; ++sl)
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          const int w = c * KW + i;
          v[t][sl * KW + i] = make_uint4(0, 0, 0, 0);
          if (q && w < K::X / 8) v[t][sl * KW + i] = __ldg(reinterpret_cast<const uint4*>(q + sl * K::X + w * 8));
        }
    }
    // The largest |q|, as 16-bit patterns (ordered as the values are).
    uint32_t top = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < NSLAB * KW; ++i) {
        top = __vmaxu2(top, v[t][i].x & 0x7fff7fffu);
        top = __vmaxu2(top, v[t][i].y & 0x7fff7fffu);
        top = __vmaxu2(top, v[t][i].z & 0x7fff7fffu);
        top = __vmaxu2(top, v[t][i].w & 0x7fff7fffu);
      }
    top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
    // 2^s brings the unit's largest |q| below 2^15; zero, subnormal, Inf or
    // NaN leave the query unscaled.
    const int E = (__float_as_int(F16Traits<T>::to_float2(top).x) >> 23) & 0xff;
    const int s = (E == 0 || E == 255) ? 0 : max(-113, min(110, 141 - E));
    const float up = __int_as_float((127 + s) << 23), up16 = up * 0.0625f;
    kf = sl2 * __int_as_float((127 - s) << 23) * 16777216.f;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NSLAB * KW; ++i) {
        float f[8];
        unpack_chunk<T>(v[t][i], f);
        const int ks = 2 * i;
        qb[t][ks][0] = F16Traits<__half>::pack(f[0] * up, f[4] * up);
        qb[t][ks][1] = F16Traits<__half>::pack(f[1] * up16, f[5] * up16);
        qb[t][ks + 1][0] = F16Traits<__half>::pack(f[2] * up, f[6] * up);
        qb[t][ks + 1][1] = F16Traits<__half>::pack(f[3] * up16, f[7] * up16);
      }
      // sum(q): the product with keys of code 1.
      const uint32_t one[4] = {0x00010001u, 0x00010001u, 0x00100010u, 0x00100010u};
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) mma_f16(sum, one, qb[t][ks][0], qb[t][ks][1]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        qz[t][j] = kf * sum[j];
        ms[t][j] = 0.f;
        thr[t][j] = -INFINITY;
        l[t][j] = zs[t][j] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < NMT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[mt][t][i] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc8[t][i] = 0.f;
    }
    vb = 7.888609052210118e-31f;  // 2^-100
    vinv = 128.f / vb;
  }

  template <class F>
  __device__ __forceinline__ void set_limits(F limit_of, int lane) {
    int least = 0x7fffffff;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        lim[t][j] = limit_of(8 * t + (lane & 3) * 2 + j);
        least = min(least, lim[t][j]);
      }
    minlim = __reduce_min_sync(0xffffffffu, least);
  }

  // The stage at `codes`: ntok of its tokens lie before the sequence end, the
  // first is token tok0.
  __device__ __forceinline__ void pass(uint32_t codes, int ntok, int tok0, int lane) {
    using O = Kv4Offsets<K>;
    float y[NTI][NT][4];  // scores, less the columns' references
    float2 pv[NTI][2];    // (value scale, value zero) of the lane's score rows r, r + 8 of each tile
    const uint32_t ka = codes + ko, pa = codes + O::poff + po;
    float dot[NTI][NT][4];
#pragma unroll
    for (int t0 = 0; t0 < NTI; t0 += 2)
#pragma unroll
      for (int sl = 0; sl < NSLAB; ++sl) {
        uint32_t wl[2][KW], wh[2][KW];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          key_words(ka + O::tile(t0 + t) + sl * O::slab, wl[t]);
          key_words(ka + O::tile(t0 + t) + sl * O::slab + O::hd, wh[t]);
        }
        // (Two tiles' chains of dependent products run side by side.)
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          const int ks = (sl * KW + i) * 2;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const uint32_t a[4] = {wl[t][i] & LO, wh[t][i] & LO, wl[t][i] & HI, wh[t][i] & HI};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (ks == 0) mma_f16_first(dot[t0 + t][n], a, qb[n][ks][0], qb[n][ks][1]);
              else mma_f16(dot[t0 + t][n], a, qb[n][ks][0], qb[n][ks][1]);
            }
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const uint32_t xl = wl[t][i] >> 8, xh = wh[t][i] >> 8;
            const uint32_t b[4] = {xl & LO, xh & LO, xl & HI, xh & HI};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(dot[t0 + t][n], b, qb[n][ks + 1][0], qb[n][ks + 1][1]);
          }
        }
      }
#pragma unroll
    for (int t = 0; t < NTI; ++t) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t wk, wv;
        lds_b64(pa + O::tilep(t) + (h ? O::hdp : 0u), wk, wv);
        const float2 k = F16Traits<T>::to_float2(wk);
        pv[t][h] = F16Traits<T>::to_float2(wv);
        const float kx = k.x * kf;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            y[t][n][2 * h + j] = fmaf(kx, dot[t][n][2 * h + j], fmaf(k.y, qz[n][j], -ms[n][j]));
      }
    }
    // Slots past the sequence end hold arbitrary parameters, and causal rows
    // stop earlier: their scores become -inf, and (below) their weights 0.
    const bool full = ntok >= K::TS && tok0 + K::TS <= minlim;
    if (!full) {
      const int trow = tok_lo(lane >> 2);
#pragma unroll
      for (int t = 0; t < NTI; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int tt = 16 * t + 8 * h + trow;
          if (tt >= ntok) pv[t][h] = make_float2(0.f, 0.f);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (tt >= ntok || tok0 + tt >= lim[n][j]) y[t][n][2 * h + j] = -INFINITY;
        }
    }
    float vm = 0.f;
#pragma unroll
    for (int t = 0; t < NTI; ++t) vm = fmaxf(vm, fmaxf(fabsf(pv[t][0].x), fabsf(pv[t][1].x)));
    bool raise = vm >= vb;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) raise |= column_max(y, n, j) > thr[n][j];
    if (__any_sync(0xffffffffu, raise)) raise_bounds(y, pv);
    if (full) weigh<false>(y, pv);
    else weigh<true>(y, pv);
    values(y, codes + O::voff);
  }

  __device__ __forceinline__ static float column_max(const float (&y)[NTI][NT][4], int n, int j) {
    float b = fmaxf(y[0][n][j], y[0][n][j + 2]);
#pragma unroll
    for (int t = 1; t < NTI; ++t) b = fmaxf(b, fmaxf(y[t][n][j], y[t][n][j + 2]));
    return b;
  }

  // New references, and a new bound on the value scales (finite ones: a NaN
  // or Inf goes through to the output whatever the bound is; four times the
  // largest, so that few items raise it); the sums and accumulators follow.
  __device__ __forceinline__ void raise_bounds(float (&y)[NTI][NT][4], const float2 (&pv)[NTI][2]) {
    float vm = 0.f;
#pragma unroll
    for (int t = 0; t < NTI; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float a = fabsf(pv[t][h].x);
        vm = a < INFINITY ? fmaxf(vm, a) : vm;
      }
    const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(vm));
    float down = 1.f;
    if (__uint_as_float(top) >= vb) {
      const float nb = __uint_as_float(min((top >> 23) + 3u, 254u) << 23);
      down = vb / nb;
      vb = nb;
      vinv = 128.f / nb;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float a[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float bm = column_max(y, n, j);
        bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 4));
        bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 8));
        bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 16));
        const bool set = thr[n][j] != -INFINITY;
        a[j] = 1.f;
        // (A row that has seen no position yet stays unset; a set reference only rises.)
        if (bm != -INFINITY && (!set || bm > 0.f)) {
          if (set) a[j] = ex2(-bm);
          ms[n][j] += bm;
          thr[n][j] = 8.f;
#pragma unroll
          for (int t = 0; t < NTI; ++t) {
            y[t][n][j] -= bm;
            y[t][n][j + 2] -= bm;
          }
        }
        l[n][j] *= a[j];
        zs[n][j] *= a[j];
        a[j] *= down;
      }
#pragma unroll
      for (int mt = 0; mt < NMT; ++mt) {
        acc[mt][n][0] *= a[0];
        acc[mt][n][1] *= a[1];
        acc[mt][n][2] *= a[0];
        acc[mt][n][3] *= a[1];
      }
      acc8[n][0] *= a[0];
      acc8[n][1] *= a[1];
      acc8[n][2] *= a[0];
      acc8[n][3] *= a[1];
    }
  }

  // Scores into weights (over the value scales' bound), and their sums.
  template <bool MASK>
  __device__ __forceinline__ void weigh(float (&y)[NTI][NT][4], const float2 (&pv)[NTI][2]) {
#pragma unroll
    for (int t = 0; t < NTI; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float zc = fmaf(8.f, pv[t][h].x, pv[t][h].y), vw = pv[t][h].x * vinv;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float x = y[t][n][2 * h + j];
            const float p = ex2(x);
            l[n][j] += p;
            // A masked position weighs nothing, whatever its parameters hold.
            const bool out = MASK && x == -INFINITY;
            zs[n][j] = out ? zs[n][j] : fmaf(p, zc, zs[n][j]);
            y[t][n][2 * h + j] = out ? 0.f : p * vw;
          }
      }
  }

  __device__ __forceinline__ void values(const float (&w)[NTI][NT][4], uint32_t codes) {
    using O = Kv4Offsets<K>;
#pragma unroll
    for (int t = 0; t < NTI; ++t) {
      uint32_t b0[NT], b1[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        b0[n] = movmatrix_trans(F16Traits<__half>::pack(w[t][n][0], w[t][n][1]));
        b1[n] = movmatrix_trans(F16Traits<__half>::pack(w[t][n][2], w[t][n][3]));
        const uint32_t eight[4] = {0x00080008u, 0x00080008u, 0x00080008u, 0x00080008u};
        mma_f16(acc8[n], eight, b0[n], b1[n]);
      }
      const uint32_t va = codes + vo + O::tile(t), vd = codes + vo2 + O::tile(t);
#pragma unroll
      for (int sl = 0; sl < NSLAB; ++sl) {
        uint32_t wa[2], wb[2], wc[2], wd[2];
        value_words(va + sl * O::slab, wa);
        value_words(vd + sl * O::slab, wb);
        value_words(va + sl * O::slab + O::hd, wc);
        value_words(vd + sl * O::slab + O::hd, wd);
#pragma unroll
        for (int half = 0; half < VW; ++half) {
          // VW = 2: rows r and r + 8 of tile mt hold nibble mt of the two
          // words (nibbles 0-3, then 4-7); VW = 1: nibbles mt and mt + 4 of the one.
          uint32_t x0, x1, x2, x3;
          if constexpr (VW == 2) {
            const uint32_t sel = half ? 0x7632u : 0x5410u;
            x0 = __byte_perm(wa[0], wb[0], sel);
            x1 = __byte_perm(wa[1], wb[1], sel);
            x2 = __byte_perm(wc[0], wd[0], sel);
            x3 = __byte_perm(wc[1], wd[1], sel);
          } else {
            x0 = __byte_perm(wa[0], wb[0], 0x5410u);
            x1 = __byte_perm(wa[0], wb[0], 0x7632u);
            x2 = __byte_perm(wc[0], wd[0], 0x5410u);
            x3 = __byte_perm(wc[0], wd[0], 0x7632u);
          }
          const int mt = sl * K::MTS + half * 4;
          const uint32_t f0[4] = {x0 & LO, x1 & LO, x2 & LO, x3 & LO};
          const uint32_t f1[4] = {x0 & HI, x1 & HI, x2 & HI, x3 & HI};
          x0 >>= 8; x1 >>= 8; x2 >>= 8; x3 >>= 8;
          const uint32_t f2[4] = {x0 & LO, x1 & LO, x2 & LO, x3 & LO};
          const uint32_t f3[4] = {x0 & HI, x1 & HI, x2 & HI, x3 & HI};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_f16(acc[mt][n], f0, b0[n], b1[n]);
            mma_f16(acc[mt + 1][n], f1, b0[n], b1[n]);
            mma_f16(acc[mt + 2][n], f2, b0[n], b1[n]);
            mma_f16(acc[mt + 3][n], f3, b0[n], b1[n]);
          }
        }
      }
    }
  }

  // The warp's state of the unit, four dims at a time: sink(col, d, v) with
  // the sums of column col's dims d .. d + 3, times scale(l), and
  // stat(col, m, l) once per column.
  template <class Scale, class Sink, class Stat>
  __device__ __forceinline__ void finish(Scale scale, Sink sink, Stat stat, int lane) {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float ls = l[n][j], zz = zs[n][j];
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) {
          ls += __shfl_xor_sync(0xffffffffu, ls, k);
          zz += __shfl_xor_sync(0xffffffffu, zz, k);
        }
        const int col = 8 * n + 2 * c + j;
        stat(col, thr[n][j] == -INFINITY ? -INFINITY : ms[n][j], ls);
        // Tiles of odd nibbles carry 2^-20 instead of 2^-24.
        const float e8 = acc8[n][j], e16 = 16.f * e8;
        const float f = scale(ls), vbf = vb * f, zf = zz * f;
#pragma unroll
        for (int sl = 0; sl < NSLAB; ++sl)
#pragma unroll
          for (int h = 0; h < 2; ++h)   // rows r and r + 8
#pragma unroll
            for (int q = 0; q < VW; ++q) {
              // Dims of row half h: VW = 2: 16 r + 8 h + 4 q ..; VW = 1: 8 r + 4 h ..
              const int d = VW == 2 ? 16 * r + 8 * h + 4 * q : 8 * r + 4 * h;
              const int mt = sl * K::MTS + 4 * q;
              float4 v;
              v.x = fmaf((acc[mt][n][2 * h + j] - e8) * 131072.f, vbf, zf);
              v.y = fmaf((acc[mt + 1][n][2 * h + j] - e16) * 8192.f, vbf, zf);
              v.z = fmaf((acc[mt + 2][n][2 * h + j] - e8) * 131072.f, vbf, zf);
              v.w = fmaf((acc[mt + 3][n][2 * h + j] - e16) * 8192.f, vbf, zf);
              if (d < K::X) sink(col, sl * K::X + d, v);
            }
      }
  }
};

// ---------------------------------------------------------------- units
// Cached tokens of sequence s, clamped to what its table row can hold (out of
// range lengths are recorded by the prologue).
__device__ __forceinline__ int kv4_tokens(const KParams& prm, int s, int BS) {
  return min(max(prm.lens[s], 0), prm.MB * BS);
}
// Unit u = (partition, kv head, row group), partitions numbered in batch
// order: sequence s holds pref[s] .. pref[s + 1] - 1.
struct Kv4Unit {
  int s, p, np, L, t0, t1, nb, kv, h0, nh;
};
template <class K>
__device__ __forceinline__ Kv4Unit kv4_unit(const KParams& prm, const Kv4Plan& pl, const int* pref, int u) {
  Kv4Unit U;
  const int pair = u / pl.n_hg, hg = u - pair * pl.n_hg;
  int lo = 0, hi = prm.S;  // pref[lo] <= pair < pref[lo + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pref[mid] <= pair) lo = mid; else hi = mid;
  }
  U.s = lo;
  U.p = pair - pref[lo];
  U.np = pref[lo + 1] - pref[lo];
  U.L = kv4_tokens(prm, lo, K::TB);
  U.t0 = U.p * prm.P;
  U.t1 = min(U.t0 + prm.P, U.L);
  U.nb = (U.t1 - U.t0 + K::TB - 1) / K::TB;
  U.kv = hg / prm.hg_per_kv;
  const int part = hg - U.kv * prm.hg_per_kv;
  U.h0 = U.kv * prm.G + part * K::GT;
  U.nh = min(K::GT, prm.G - part * K::GT);
  return U;
}

// One finished row piece: the partition's normalised output in the workspace,
// or the output itself where the sequence has one partition.
template <class K>
__device__ __forceinline__ void put_row(const KParams& prm, const Kv4Unit& U, int col, int d, const float4& v,
                                        uint64_t keep) {
  using T = typename K::T;
  const int h = U.h0 + col;
  if (U.np == 1) {
    store4<T>(static_cast<T*>(prm.out) + out_row_rt(prm, U.s, h) * K::D + d, v);
  } else {
    const size_t at = ((size_t)U.s * prm.H + h) * prm.Pmax + U.p;
    st_f4_policy(reinterpret_cast<float4*>(prm.ws_o + at * K::D + d), v, keep);
  }
}
__device__ __forceinline__ void put_stat(const KParams& prm, const Kv4Unit& U, int col, float m, float l,
                                         uint64_t keep) {
  const int h = U.h0 + col;
  const size_t at = ((size_t)U.s * prm.H + h) * prm.Pmax + U.p;
  st_f32_policy(prm.ws_m + at, m * kLn2, keep);
  st_f32_policy(prm.ws_l + at, l, keep);
  if (U.np == 1 && prm.lse) prm.lse[out_row_rt(prm, U.s, h)] = m * kLn2 + logf(l);
}
// (A NaN sum stays NaN: only an empty row divides by nothing.)
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }

// Unused partitions: sentinels (m = -inf, l = 0).  Empty sequences: zeros (a
// multi-query sequence is never empty: it holds its new tokens).
template <class K>
__device__ __forceinline__ void kv4_sentinels(const KParams& prm) {
  using T = typename K::T;
  const int S = prm.S, H = prm.H, Pmax = prm.Pmax;
  const long long me = (long long)blockIdx.x * K::THREADS + threadIdx.x, n = (long long)gridDim.x * K::THREADS;
  auto parts_of = [&](int s) { return (kv4_tokens(prm, s, K::TB) + prm.P - 1) / prm.P; };
  for (long long i = me; i < (long long)S * H * Pmax; i += n) {
    const int s = (int)(i / ((long long)H * Pmax)), p = (int)(i % Pmax);
    if (p >= parts_of(s)) {
      prm.ws_m[i] = -INFINITY;
      prm.ws_l[i] = 0.f;
    }
  }
  if (prm.q_len == 1) {
    constexpr int D16 = K::D * 2 / 16;
    uint4* out = static_cast<uint4*>(prm.out);
    for (long long i = me; i < (long long)S * H * D16; i += n)
      if (parts_of((int)(i / ((long long)H * D16))) == 0) out[i] = make_uint4(0, 0, 0, 0);
    if (prm.lse)
      for (long long i = me; i < (long long)S * H; i += n)
        if (parts_of((int)(i / H)) == 0) prm.lse[i] = -INFINITY;
  }
}

// (Out of line: a wait that does not succeed at once has time for a call.)
static __device__ __noinline__ bool kv4_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err_word,
                                           long long timeout_ns, int slot) {
  return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort_flag, err_word, timeout_ns, kSiteFull, slot));
}

// A bulk copy into this CTA's own shared memory (bulk_copy_g2s names its
// destination in the cluster's address space, which costs a few instructions).
__device__ __forceinline__ void bulk_copy_cta(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar,
                                              uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}

// A warp's run of a unit's stages: refills its own ring.  (Everything but the
// ids is the same in all lanes.)
template <class K>
struct Kv4Stream {
  uint32_t in, out;      // byte offsets in the ring of the next stage to fill, and of the next to use
  uint32_t bar_in, bar_out, ph_out;  // their barriers, and the phase of the latter
  int nb, left;          // blocks of the run; those not asked for yet
  int ids, ids_next;     // lane's ids of the current window of 32 blocks, and of the one after
  uint32_t ring, bars;   // shared addresses of the warp's ring and barriers
  const int32_t* row;    // the run's block ids
  const uint8_t* base;   // the kv head's record of block 0
  size_t block_bytes;    // of all kv heads
  uint64_t policy;

  __device__ __forceinline__ Kv4Stream(const KParams& prm, uint32_t r, uint32_t b)
      : in(0), out(0), bar_in(b), bar_out(b), ph_out(0), nb(0), left(0), ring(r), bars(b),
        block_bytes((size_t)prm.KH * K::REC), policy(l2_policy_evict_first()) {}

  __device__ __forceinline__ int fetch(int b0, int lane) const { return b0 + lane < nb ? __ldg(row + b0 + lane) : 0; }

  __device__ __forceinline__ void start(const KParams& prm, const int32_t* table, const uint8_t* cache_kv, int blocks,
                                        int lane) {
    row = table;
    base = cache_kv;
    nb = left = blocks;
    ids = fetch(0, lane);
    ids_next = fetch(32, lane);
    ids = check_block_id(prm, ids);
    for (int i = 0; i < K::NS; ++i) issue(prm, lane);
  }
  // Fills the next stage (it is free: this warp has used it, or never filled it).
  __device__ __forceinline__ void issue(const KParams& prm, int lane) {
    if (left <= 0) return;
    const int b0 = nb - left, w = b0 & 31;
    if (w == 0 && b0 > 0) {
      ids = check_block_id(prm, ids_next);
      ids_next = fetch(b0 + 32, lane);
    }
    int id[K::NBLK];
#pragma unroll
    for (int k = 0; k < K::NBLK; ++k) id[k] = __shfl_sync(0xffffffffu, ids, w + k);
    const int n = min(K::NBLK, left);
    if (elect_one()) {
      mbar_arrive_expect_tx(bar_in, (uint32_t)n * K::REC);
#pragma unroll
      for (int k = 0; k < K::NBLK; ++k)
        if (k < n) bulk_copy_cta(ring + in + k * K::REC, base + (uint32_t)id[k] * block_bytes, K::REC, bar_in, policy);
    }
    left -= K::NBLK;
    in += K::STAGE;
    bar_in += 8;
    if (in == K::NS * K::STAGE) {
      in = 0;
      bar_in = bars;
    }
  }
  // Waits for the next stage to land; false: gave up.
  __device__ __forceinline__ bool wait(const KParams& prm, volatile int* abort_flag) const {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar_out, ph_out))) return true;
    return kv4_wait_slow(bar_out, ph_out, abort_flag, prm.hdr + kHdrError, prm.timeout_ns, (int)(out / K::STAGE));
  }
  __device__ __forceinline__ void used() {
    // The stage is refilled by bulk copies (async proxy): every lane's reads
    // of it are ordered before that by a proxy fence.
    fence_proxy_async_smem();
    __syncwarp();
    out += K::STAGE;
    bar_out += 8;
    if (out == K::NS * K::STAGE) {
      out = 0;
      bar_out = bars;
      ph_out ^= 1u;
    }
  }
  // After a wait that gave up at stage `done` of the run: no copy of this warp
  // stays in flight (bounded).
  __device__ __forceinline__ void drain(int done) {
    const int asked = (nb - max(left, 0) + K::NBLK - 1) / K::NBLK;
    for (; done < asked; ++done) {
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(bar_out, ph_out) && (long long)(global_timer_ns() - t0) < 100000000LL) {
      }
      used();
    }
  }
};

template <class K>
__global__ void __launch_bounds__(K::THREADS, 1) kv4_decode_kernel(const __grid_constant__ KParams prm) {
  using T = typename K::T;
  extern __shared__ __align__(1024) uint8_t smem[];
  // (The warp index by a shuffle: known to be the same in all lanes.)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t sbase = smem_addr(smem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + K::OFF_FLAGS);
  int* bad_len = reinterpret_cast<int*>(smem + K::OFF_FLAGS + 16);
  volatile int* team_next = reinterpret_cast<volatile int*>(smem + K::OFF_NEXT);
  int* pref = reinterpret_cast<int*>(smem + K::OFF_PREF);
  if (tid == 0) {
    *abort_flag = 0;
    *bad_len = 0;
  }
  if (lane < K::NSMAX) mbar_init(sbase + K::OFF_BAR + (warp * K::NSMAX + lane) * 8, 1);
  fence_mbarrier_init();
  __syncthreads();
  // pref[s]: partitions of the sequences before s (an exclusive scan; the warp
  // totals are kept in the ring, not filled yet).
  {
    constexpr int NW = K::NC;
    int* scan = reinterpret_cast<int*>(smem);
    const int S = prm.S, per = (S + K::THREADS - 1) / K::THREADS;
    const int beg = min(tid * per, S), end = min(beg + per, S);
    bool bad = false;
    int sum = 0;
    for (int s = beg; s < end; ++s) {
      // (A multi-query sequence holds its q_len new tokens.)
      bad |= prm.lens[s] < (prm.q_len > 1 ? prm.q_len : 0) || prm.lens[s] > prm.MB * K::TB;
      const int np = (kv4_tokens(prm, s, K::TB) + prm.P - 1) / prm.P;
      pref[s] = sum;
      sum += np;
    }
    if (bad) *bad_len = 1;
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const int v = scan[w];
      if (w < warp) before += v;
      all += v;
    }
    for (int s = beg; s < end; ++s) pref[s] += before + incl - sum;
    if (tid == 0) pref[S] = all;
    fence_proxy_async_smem();  // the ring is filled by bulk copies from here on
  }
  __syncthreads();
  const Kv4Plan pl = make_plan<K>(prm, pref[prm.S]);
  // A programmatic dependent of the kernel that clears the workspace header:
  // nothing below may touch the header before it has completed.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tid == 0 && *bad_len) atomicCAS(prm.hdr + kHdrError, 0, kErrDeviceBounds);

  const int ltw = __ffs(pl.TW) - 1;
  const int teams = K::NC >> ltw, team = warp >> ltw, tw = warp & (pl.TW - 1);
  const uint64_t keep = l2_policy_evict_last();
  Kv4Stream<K> in(prm, sbase + warp * K::RING, sbase + K::OFF_BAR + warp * K::NSMAX * 8);
  Kv4State<K> st(lane);
  // The first units are dealt out over the CTAs; the counter hands out the rest.
  int u = blockIdx.x + (int)gridDim.x * team;
  bool alive = true;
  // The sentinels are written while the first copies fly.
  bool sentinels = false;
  while (u < pl.total) {
    const Kv4Unit U = kv4_unit<K>(prm, pl, pref, u);
    const int nst = (U.nb + K::NBLK - 1) / K::NBLK, per = (nst + pl.TW - 1) >> ltw;
    const int i0 = min(tw * per, nst), b0 = i0 * K::NBLK, nb = min(per * K::NBLK, U.nb - b0);
    int u_next = 0;
    if (tw == 0 && lane == 0) u_next = atomicAdd(prm.hdr + kHdrWork, 1) + (int)gridDim.x * teams;
    const int blocks = alive ? max(nb, 0) : 0, stages = (blocks + K::NBLK - 1) / K::NBLK;
    in.start(prm, prm.bt + (size_t)U.s * prm.MB + U.t0 / K::TB + b0,
             static_cast<const uint8_t*>(prm.kc) + (size_t)U.kv * K::REC, blocks, lane);
    if (!sentinels) {
      sentinels = true;
      kv4_sentinels<K>(prm);
    }
    st.begin_unit([&](int i) { return static_cast<const T*>(prm.q) + out_row_rt(prm, U.s, U.h0 + i) * K::D; }, U.nh,
                  prm.scale_log2, lane);
    if (prm.q_len > 1) st.set_limits([&](int h) { return row_limit<true>(prm, U.L, U.h0 + h); }, lane);
    else st.set_limits([&](int) { return U.L; }, lane);
    int n = U.t1 - U.t0 - i0 * K::TS, tok = U.t0 + i0 * K::TS;  // tokens from the stage on; its first
    for (int i = 0; i < stages; ++i, n -= K::TS, tok += K::TS) {
      if (!in.wait(prm, abort_flag)) {
        in.drain(i);
        alive = false;
        break;
      }
      st.pass(in.ring + in.out, n, tok, lane);
      in.used();
      in.issue(prm, lane);
    }
    if (pl.TW == 1) {
      if (!alive) break;
      st.finish([](float ls) { return inverse(ls); },
          [&](int col, int d, const float4& v) {
            if (col < U.nh) put_row<K>(prm, U, col, d, v, keep);
          },
          [&](int col, float m, float ls) {
            if (lane < 4 && col < U.nh) put_stat(prm, U, col, m, ls, keep);
          },
          lane);
      u = __shfl_sync(0xffffffffu, u_next, 0);
    } else {
      // The team's states, each in its warp's ring (whose stages are all used).
      float* acc = reinterpret_cast<float*>(smem + warp * K::RING);
      float* ml = acc + K::GT * K::AROW;
      st.finish([](float) { return 1.f; },
                [&](int col, int d, const float4& v) { *reinterpret_cast<float4*>(acc + col * K::AROW + d) = v; },
                [&](int col, float m, float ls) {
                  if (lane < 4) {
                    ml[2 * col] = m;
                    ml[2 * col + 1] = ls;
                  }
                },
                lane);
      if (tw == 0 && lane == 0) team_next[team] = *abort_flag ? pl.total : u_next;
      named_barrier_sync(1 + team, pl.TW * 32);
      // A slice of the rows each; the warps' states in warp order.
      const float* first = reinterpret_cast<const float*>(smem + (warp - tw) * K::RING);
      constexpr int D4 = K::D / 4, WR = K::RING / 4;
      for (int i = tw * 32 + lane; i < U.nh * D4; i += pl.TW * 32) {
        const int col = i / D4, d4 = i - col * D4;
        float M = -INFINITY;
        for (int w = 0; w < pl.TW; ++w) M = fmaxf(M, first[w * WR + K::GT * K::AROW + 2 * col]);
        // (A row that sees nothing in this partition has M = -inf: its weights are 0.)
        const float Ms = M == -INFINITY ? 0.f : M;
        float den = 0.f;
        float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < pl.TW; ++w) {
          const float2 s2 = *reinterpret_cast<const float2*>(first + w * WR + K::GT * K::AROW + 2 * col);
          const float f = ex2(s2.x - Ms);
          const float4 v = *reinterpret_cast<const float4*>(first + w * WR + col * K::AROW + 4 * d4);
          den = fmaf(f, s2.y, den);
          num.x = fmaf(f, v.x, num.x);
          num.y = fmaf(f, v.y, num.y);
          num.z = fmaf(f, v.z, num.z);
          num.w = fmaf(f, v.w, num.w);
        }
        const float inv = inverse(den);
        put_row<K>(prm, U, col, 4 * d4, make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv), keep);
        if (d4 == 0) put_stat(prm, U, col, M, den, keep);
      }
      u = team_next[team];
      fence_proxy_async_smem();  // the rings are filled by bulk copies again
      named_barrier_sync(1 + team, pl.TW * 32);
    }
    if (*abort_flag && pl.TW == 1) break;
  }
  if (!sentinels) kv4_sentinels<K>(prm);
  // Phase 2 may be launched once every CTA has said so or ended (it waits for
  // this grid to complete before it reads anything).
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace pa
