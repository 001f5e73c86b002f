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
// the unit's largest finite one), and the weights p_t vs_t enter the value product as
// fp16.  A weight's rounding error meets the code, whose mean is far from
// zero; it is kept to the spread of the codes (c - 8) by summing the rounded
// weights themselves (one more product, with rows of code 8) and putting
// 8 p_t vs_t back in fp32 with the zeros.
//
// Softmax without a reduction per item: each column subtracts a reference from
// its scores that brings the largest p_t vs_t it has met to 2^6, so that what is
// rounded to fp16 has its range whatever the cache's magnitude and however far
// its value scales differ: a large scale at a position of no weight takes nothing
// from the others.  (p_t itself stays below 2^40, and the sums in fp32.)  The
// reference is raised, with the sums and accumulators, only where a product may
// pass 2^15, which one vote per item finds out from a bound (the lane's largest
// p times its largest scale); most items need no shuffle, no rescaling.
// (References of the scores alone and one factor for the scales, above the
// largest met by the warp, cost as much and lost the others' bits: 2^28 below
// that scale nothing was left.)
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
// Work.  A unit is (sequence, partition, kv head, GT of its query rows), a run
// of stages of 64 tokens (32 at head size 256, and where a unit is two kv heads:
// GT = 8 columns of four rows each).  One CTA of NC equal warps per
// SM, no producer: a warp takes whole units from a global counter, owns a ring
// of a few stages and refills a stage itself, by one bulk copy per block, right
// after it has used it; what it asks for runs ahead into its next unit.  Units
// are numbered with the kv heads of a partition next to each other, so the
// records of one block, neighbours in memory, are read at about the same time
// by different SMs (contiguous shares per warp instead, which end together,
// took 160 us where this takes 118 for the copies of a batch alone).  The units
// left over when every warp has taken as many as the others are shared by
// teams of TW warps of a CTA, each a part of the tokens; the team merges the
// parts through shared memory.
//
// Measured (GB300, 2070 MHz; 6766 GB/s is the measured copy rate):
//   128 sequences of 2048 to 8192 tokens, 32 heads over 8 kv heads, D = 128:
//     131 us for 715 MB, 81% of the copy rate (the copies alone, without the
//     arithmetic, 118 us); 140 with eight warps of 255 registers, 158 with one
//     kv head a unit and the units handed out whole (177 with 16 warps of 128
//     registers and 32-token stages), 239 in the scheme of pa_kernel.cuh: a
//     4-bit partition holds a quarter of the bytes, so set-ups, hand-overs and
//     the one merging warp outweigh the tokens.
//   A batch with a few long sequences among short ones, 64 heads over 8:
//     45 us, 76 without teams for the units left over.
//   Four new tokens a sequence, 32 heads over 8 (16 rows a unit): 61 us for
//     160 MB.  The tensor pipe is a third used, the issue slots 37%: two warps a
//     scheduler (255 registers) leave the chains of a tile, scores to weights to
//     values, in the open.  32-token stages 64 to 67 us.  What cost most before
//     that were spilled registers: 227 KB of shared memory leave next to no L1,
//     so they come from L2 (68 us with ten reloads a stage; 10 and 12 warps of
//     168 registers, 13 a tile, 115 and 90; the four to six words a thread that
//     still spill lie outside the tiles, as the references are raised).
//   More rows a kv head than a unit takes (16; 8 at head size 256) read and
//     unpack its records again: 48 sequences as above with 32 rows a kv head 135 us
//     for 177 MB, 64 of 2048 to 8192 tokens with 16 rows a head (64 heads over 4)
//     76 us for 190 MB.
//   Head size 256, 64 sequences of 2048 to 8192 tokens, 8 kv heads, 730 MB: 139 us
//     with one row a head, 143 with four, 150 with eight (8 warps); 166 in blocks of
//     64 tokens (4 warps).  The first batch in blocks of 8 tokens 135 us, of 64 tokens
//     138; with one row a kv head (64 sequences, 32 heads, 735 MB) 125; at head size 64
//     91 us for 393 MB.
#pragma once

#include <type_traits>

#include "pa_common.cuh"
#include "pa_kernel.cuh"

namespace pa {

// TB: tokens per block.  KVU: kv heads per unit; with two (at most four query
// rows each), head u's rows are columns 4u .. 4u + 3, so the softmax and the
// weights of a tile serve both, and a block's copy covers both records.
template <typename T_, int D_, int NT_, int TB_, int KVU_>
struct Kv4 {
  using T = T_;
  static constexpr int D = D_, NT = NT_, GT = 8 * NT_, TB = TB_, KVU = KVU_;
  static_assert(KVU_ == 1 || (KVU_ == 2 && NT_ == 1), "two heads share one column tile");
  // 16-token tiles per stage (two at head size 256 and of two kv heads, for two
  // stages in the ring).
  static constexpr int NTI = TB_ == 64 ? 4 : D_ > 128 || KVU_ == 2 ? 2 : 4;
  static constexpr int TS = 16 * NTI;            // tokens per stage
  static constexpr int NBLK = TS / TB_;          // blocks per stage
  static_assert(NBLK >= 1, "a stage holds whole blocks");
  static constexpr uint32_t REC = (uint32_t)TB_ * (D_ + 8), BLOCK = REC * KVU_, STAGE = BLOCK * NBLK;
  // Warps per CTA: as many as the accumulators' registers allow without a
  // spill: 12 of 168 a thread where a unit has 8 columns, 8 of 255 where it has
  // 16 or the head 256 dims, 4 where two stages of 64-token blocks of such a
  // head fill the ring.  (12 against 8: 128 sequences of 32 heads over 8 133
  // against 138 us, 64 of 64 over 8 74 against 86, long skew 45 against 47; 16
  // columns, spilling: 90 against 60.)
  static constexpr int NC = NT_ == 2 ? 8 : D_ <= 128 ? 12 : TB_ == 64 ? 4 : 8;

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
  static constexpr uint32_t SZ_PREF = (2 * kMaxSeqsPerLaunch + 1) * 4;  // partition prefix, lengths
  static constexpr uint32_t SZ_UNIT = NC * 2 * 48;                      // each warp's unit and the one after it
  static constexpr uint32_t FIXED = al16(SZ_BAR) + 64 + al16(SZ_PREF) + SZ_UNIT;
  static constexpr uint32_t BUDGET = 227 * 1024;
  static constexpr uint32_t RING = (BUDGET - FIXED) / NC / 128 * 128;  // bytes per warp
  static constexpr uint32_t OFF_BAR = NC * RING, OFF_FLAGS = OFF_BAR + al16(SZ_BAR),
                            OFF_PREF = OFF_FLAGS + 64, OFF_UNIT = OFF_PREF + al16(SZ_PREF),
                            BYTES = OFF_UNIT + SZ_UNIT;
  static_assert(BYTES <= BUDGET, "shared memory over budget");
  static constexpr int NS = RING / STAGE < NSMAX ? RING / STAGE : NSMAX;  // ring stages per warp
  static_assert(STATE <= RING && NS >= 2, "a warp's state or two stages fit its ring");
};

// ---------------------------------------------------------------- small pieces
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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
  static constexpr uint32_t hd = K::TB == 8 ? K::BLOCK : 8 * K::XB;
  static constexpr uint32_t hdp = K::TB == 8 ? K::BLOCK : 64;
  // Tile t.
  __device__ static constexpr uint32_t tile(int t) {
    return (uint32_t)(16 * t / K::TB) * K::BLOCK + (uint32_t)(16 * t % K::TB) * K::XB;
  }
  __device__ static constexpr uint32_t tilep(int t) {
    return (uint32_t)(16 * t / K::TB) * K::BLOCK + (uint32_t)(16 * t % K::TB) * 8;
  }
};

// ---------------------------------------------------------------- a consumer warp's state
template <class K>
struct Kv4State {
  using T = typename K::T;
  static constexpr int NT = K::NT, NK = K::NK, NMT = K::NMT, KW = K::KW, VW = K::VW, NSLAB = K::NSLAB;
  static constexpr int NTI = K::NTI, KVU = K::KVU;
  static constexpr uint32_t LO = 0x000f000fu, HI = 0x00f000f0u;

  uint32_t qb[NT][NK][2];          // Q^T fragments: the query row of column lane / 4
  float ms[NT][2];                 // reference (0 until set)
  uint32_t set;                    // bit 2n + j: column j of tile n has one
  float l[NT][2], zs[NT][2];       // sums of weights; of weight * (value zero + 8 value scale)
  float qz[NT][2];                 // scale_log2 * sum(q)
  float acc[NMT][NT][4], acc8[NT][4];
  float kf;                        // score factor: scale_log2 over the operands' powers of two
  // Weights (log2) and their products with the value scales: the most there may
  // be, and where a new reference puts them.
  static constexpr float kTopP = 40.f, kNewP = 36.f, kTopW = 32768.f, kNewW = 6.f;
  // The lane's offsets in a tile: key words, parameters, values of the first
  // and second token of its slots.
  uint32_t ko, po, vo, vo2;

  __device__ __forceinline__ explicit Kv4State(int lane) {
    const int r = lane >> 2, c = lane & 3;
    ko = tok_lo(r) * K::XB + c * (KW * 4);
    po = tok_lo(r) * 8 + (KVU == 2 ? (c >> 1) * K::REC : 0u);  // (of its columns' kv head)
    // Slots 2c, 2c + 1 and 2c + 8, 2c + 9 hold tokens c, 7 - c, 8 + c, 15 - c.
    vo = c * K::XB + r * (VW * 4);
    vo2 = (7 - c) * K::XB + r * (VW * 4);
    // (Opaque: kept in registers rather than computed again for every stage,
    // which cost 30 instructions of 500.)
    asm volatile("" : "+r"(ko), "+r"(po), "+r"(vo), "+r"(vo2));
  }

  __device__ __forceinline__ bool has_ref(int n, int j) const { return (set >> (2 * n + j)) & 1u; }
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

  // Column `col` holds query row row_of(col, nh) of the unit, where it holds
  // one; nh: rows of a kv head.
  __device__ __forceinline__ static bool has_row(int col, int nh) { return (KVU == 2 ? col & 3 : col) < nh; }
  __device__ __forceinline__ static int row_of(int col, int nh) {
    return KVU == 2 ? (col >> 2) * nh + (col & 3) : col;
  }
  __device__ __forceinline__ static int column_of(int row, int nh) {
    return KVU == 2 && row >= nh ? 4 + row - nh : row;
  }

  // The unit's query rows as this lane needs them: row(i) is row i in global
  // memory.  Dims 8w .. 8w + 7 of a slab are word w; this lane holds
  // words c * KW ...
  struct Rows {
    uint4 v[NT][NSLAB * KW];
  };
  template <class F>
  __device__ __forceinline__ static void load_rows(Rows& q, F row, int nh, int lane) {
    const int n = lane >> 2, c = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const T* p = has_row(8 * t + n, nh) ? row(row_of(8 * t + n, nh)) : nullptr;
#pragma unroll
      for (int sl = 0; sl < NSLAB; ++sl)
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          const int w = c * KW + i;
          q.v[t][sl * KW + i] = make_uint4(0, 0, 0, 0);
          if (p && w < K::X / 8) q.v[t][sl * KW + i] = __ldg(reinterpret_cast<const uint4*>(p + sl * K::X + w * 8));
        }
    }
  }
  // The unit's largest |q| (FINITE: of its finite elements) as a pattern.
  static constexpr uint32_t kInf16 = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  template <bool FINITE>
  __device__ __forceinline__ static uint32_t largest(const Rows& q) {
    uint32_t top = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < NSLAB * KW; ++i) {
        const uint32_t w[4] = {q.v[t][i].x, q.v[t][i].y, q.v[t][i].z, q.v[t][i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t a = w[k] & 0x7fff7fffu;
          top = __vmaxu2(top, FINITE ? a & __vcmpltu2(a, kInf16 * 0x10001u) : a);
        }
      }
    return __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
  }
  __device__ __forceinline__ void begin_unit(const Rows& q, float sl2) {
    // The largest |q|, as 16-bit patterns (ordered as the values are); where a
    // row holds infinities or NaN (patterns from kInf16 on), the largest finite
    // one: the scale is the other rows' too.
    uint32_t top = largest<false>(q);
    if (top >= kInf16) top = largest<true>(q);
    // 2^s brings the unit's largest |q| below 2^15; zero or subnormal leave the
    // query unscaled.
    const int E = (__float_as_int(F16Traits<T>::to_float2(top).x) >> 23) & 0xff;
    const int s = E == 0 ? 0 : max(-113, min(110, 141 - E));
    const float up = __int_as_float((127 + s) << 23), up16 = up * 0.0625f;
    kf = sl2 * __int_as_float((127 - s) << 23) * 16777216.f;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NSLAB * KW; ++i) {
        float f[8];
        unpack_chunk<T>(q.v[t][i], f);
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
        l[t][j] = zs[t][j] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < NMT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[mt][t][i] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc8[t][i] = 0.f;
    }
    set = 0;
  }

  // The stage at `codes`: ntok of its tokens lie before the sequence end, the
  // first is token tok0; rows see at least `least` positions, and column `col`
  // sees limit_of(col).
  template <class F>
  __device__ __forceinline__ void pass(uint32_t codes, int ntok, int tok0, int least, F limit_of, int lane) {
    using O = Kv4Offsets<K>;
    float y[NTI][NT][4];  // scores, less the columns' references
    float2 pv[NTI][2];    // (value scale, value zero) of the lane's score rows r, r + 8 of each tile
    const uint32_t ka = codes + ko, pa = codes + O::poff + po;
    const bool second = (lane & 2) != 0;  // KVU = 2: the lane's score columns are the second head's
    float dot[NTI][NT][4];
#pragma unroll
    for (int t0 = 0; t0 < NTI; t0 += 2) {
      float du[KVU][2][NT][4];
#pragma unroll
      for (int sl = 0; sl < NSLAB; ++sl) {
#pragma unroll
        for (int u = 0; u < KVU; ++u) {
          uint32_t wl[2][KW], wh[2][KW];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            key_words(ka + u * K::REC + O::tile(t0 + t) + sl * O::slab, wl[t]);
            key_words(ka + u * K::REC + O::tile(t0 + t) + sl * O::slab + O::hd, wh[t]);
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
                if (ks == 0) mma_f16_first(du[u][t][n], a, qb[n][ks][0], qb[n][ks][1]);
                else mma_f16(du[u][t][n], a, qb[n][ks][0], qb[n][ks][1]);
              }
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const uint32_t xl = wl[t][i] >> 8, xh = wh[t][i] >> 8;
              const uint32_t b[4] = {xl & LO, xh & LO, xl & HI, xh & HI};
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_f16(du[u][t][n], b, qb[n][ks + 1][0], qb[n][ks + 1][1]);
            }
          }
        }
      }
      // (Every column meets both heads' keys; its own head's product counts.)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dot[t0 + t][n][i] = KVU == 2 && second ? du[KVU - 1][t][n][i] : du[0][t][n][i];
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
    const bool full = ntok >= K::TS && tok0 + K::TS <= least;
    if (!full) {
      const int trow = tok_lo(lane >> 2);
      int lim[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) lim[n][j] = limit_of(8 * n + (lane & 3) * 2 + j) - tok0;
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
              if (tt >= ntok || tt >= lim[n][j]) y[t][n][2 * h + j] = -INFINITY;
        }
    }
    float vm = 0.f;
#pragma unroll
    for (int t = 0; t < NTI; ++t) vm = fmaxf(vm, fmaxf(fabsf(pv[t][0].x), fabsf(pv[t][1].x)));
    float top = column_max(y, 0, 0);
#pragma unroll
    for (int i = 1; i < 2 * NT; ++i) top = fmaxf(top, column_max(y, i >> 1, i & 1));
    bool raise = top > kTopP || vm * ex2(top) > kTopW;
    if (set != (1u << (2 * NT)) - 1u) {
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i) raise |= !has_ref(i >> 1, i & 1) && column_max(y, i >> 1, i & 1) > -INFINITY;
    }
    if (__any_sync(0xffffffffu, raise)) raise_references(y, pv);
    if (full) weigh<false>(y, pv);
    else weigh<true>(y, pv);
    values(y, codes + O::voff, lane);
  }

  __device__ __forceinline__ static float column_max(const float (&y)[NTI][NT][4], int n, int j) {
    float b = fmaxf(y[0][n][j], y[0][n][j + 2]);
#pragma unroll
    for (int t = 1; t < NTI; ++t) b = fmaxf(b, fmaxf(y[t][n][j], y[t][n][j + 2]));
    return b;
  }

  // New references for the columns that have none, or whose weights or products
  // pass their bounds; the sums and accumulators follow.  (Scales that are not
  // finite count for nothing here: they go through to the output whatever the
  // reference is.)
  __device__ __forceinline__ void raise_references(float (&y)[NTI][NT][4], const float2 (&pv)[NTI][2]) {
    float lv[NTI][2];
#pragma unroll
    for (int t = 0; t < NTI; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float a = fabsf(pv[t][h].x);
        lv[t][h] = a < INFINITY ? lg2(a) : -INFINITY;
      }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float a[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float top = column_max(y, n, j), prod = -INFINITY;  // log2 of the largest weight, and product
#pragma unroll
        for (int t = 0; t < NTI; ++t) prod = fmaxf(prod, fmaxf(y[t][n][j] + lv[t][0], y[t][n][j + 2] + lv[t][1]));
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) {
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
          prod = fmaxf(prod, __shfl_xor_sync(0xffffffffu, prod, k));
        }
        const bool old = has_ref(n, j);
        a[j] = 1.f;
        // (A row that has seen no position yet stays unset; a set reference only rises.)
        if (top != -INFINITY && (!old || top > kTopP || prod > 15.f)) {
          const float up = fmaxf(prod - kNewW, top - kNewP);
          if (old) a[j] = ex2(-up);
          ms[n][j] += up;
          set |= 1u << (2 * n + j);
#pragma unroll
          for (int t = 0; t < NTI; ++t) {
            y[t][n][j] -= up;
            y[t][n][j + 2] -= up;
          }
        }
        l[n][j] *= a[j];
        zs[n][j] *= a[j];
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

  // Scores into weights, their sums, and their products with the value scales.
  template <bool MASK>
  __device__ __forceinline__ void weigh(float (&y)[NTI][NT][4], const float2 (&pv)[NTI][2]) {
#pragma unroll
    for (int t = 0; t < NTI; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float zc = fmaf(8.f, pv[t][h].x, pv[t][h].y);
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
            y[t][n][2 * h + j] = out ? 0.f : p * pv[t][h].x;
          }
      }
  }

  __device__ __forceinline__ void values(const float (&w)[NTI][NT][4], uint32_t codes, int lane) {
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
#pragma unroll
      for (int u = 0; u < KVU; ++u) {
        // Head u's product takes the weights of its own columns.
        const bool mine = KVU == 1 || (lane >> 4) == u;
        uint32_t m0[NT], m1[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          m0[n] = mine ? b0[n] : 0u;
          m1[n] = mine ? b1[n] : 0u;
        }
        const uint32_t va = codes + vo + u * K::REC + O::tile(t), vd = codes + vo2 + u * K::REC + O::tile(t);
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
              mma_f16(acc[mt][n], f0, m0[n], m1[n]);
              mma_f16(acc[mt + 1][n], f1, m0[n], m1[n]);
              mma_f16(acc[mt + 2][n], f2, m0[n], m1[n]);
              mma_f16(acc[mt + 3][n], f3, m0[n], m1[n]);
            }
          }
        }
      }
    }
  }

  // The unit's sums: its row i at rows + i * stride, over the row's weight sum,
  // and stat(i, reference, weight sum); or, by_column, all columns' sums, and stat
  // by column.  What leaves the warp is relative to a reference that brings the
  // weight sum to [1, 2): those of other warps and partitions may lie far apart,
  // as their value scales do.
  template <class Stat>
  __device__ __forceinline__ void finish(float* rows, size_t stride, int nh, bool by_column, Stat stat, int lane) {
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
        const int col = 8 * n + 2 * c + j, row = by_column ? col : row_of(col, nh);
        if (!by_column && !has_row(col, nh)) continue;
        // (A NaN or infinite sum stays what it is; only an empty row divides by nothing.)
        const int e = ls > 0.f && ls < INFINITY ? (int)(__float_as_uint(ls) >> 23) - 127 : 0;
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        if (r == 0) stat(row, has_ref(n, j) ? ms[n][j] + (float)e : -INFINITY, ls * down);
        const float f = by_column ? down : ls == 0.f ? 0.f : 1.f / ls;
        const float zf = zz * f;
        float* o = rows + row * stride;
        // Tiles of odd nibbles carry 2^-20 instead of 2^-24.
        const float e8 = acc8[n][j], e16 = 16.f * e8;
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
              v.x = fmaf((acc[mt][n][2 * h + j] - e8) * 16777216.f, f, zf);
              v.y = fmaf((acc[mt + 1][n][2 * h + j] - e16) * 1048576.f, f, zf);
              v.z = fmaf((acc[mt + 2][n][2 * h + j] - e8) * 16777216.f, f, zf);
              v.w = fmaf((acc[mt + 3][n][2 * h + j] - e16) * 1048576.f, f, zf);
              if (d < K::X) *reinterpret_cast<float4*>(o + sl * K::X + d) = v;
            }
      }
  }
};

// ---------------------------------------------------------------- units
// Unit u = (partition, head group), partitions numbered in batch order:
// sequence s holds pref[s] .. pref[s + 1] - 1 (pref and the clamped lengths in
// shared memory).
struct __align__(16) Kv4Unit {
  int s, p, np, L, t0, t1;
  int kv, h0, nh, pad;  // first kv head and row head; rows per kv head
  int nb, stages;  // blocks, stages
};
static_assert(sizeof(Kv4Unit) == 48, "units in shared memory");
template <class K>
__device__ __forceinline__ Kv4Unit kv4_unit(const KParams& prm, const int* pref, const int* lens, int u) {
  Kv4Unit U;
  const int n_hg = prm.KH / K::KVU * prm.hg_per_kv, pair = u / n_hg, hg = u - pair * n_hg;
  int lo = 0, hi = prm.S;  // pref[lo] <= pair < pref[lo + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pref[mid] <= pair) lo = mid; else hi = mid;
  }
  U.s = lo;
  U.p = pair - pref[lo];
  U.np = pref[lo + 1] - pref[lo];
  U.L = lens[lo];
  U.t0 = U.p * prm.P;
  U.t1 = min(U.t0 + prm.P, U.L);
  U.nb = (U.t1 - U.t0 + K::TB - 1) / K::TB;
  U.stages = (U.nb + K::NBLK - 1) / K::NBLK;
  if constexpr (K::KVU == 2) {
    U.kv = 2 * hg;
    U.h0 = U.kv * prm.G;
    U.nh = prm.G;
  } else {
    U.kv = prm.hg_per_kv == 1 ? hg : hg / prm.hg_per_kv;
    const int part = hg - U.kv * prm.hg_per_kv;
    U.h0 = U.kv * prm.G + part * K::GT;
    U.nh = min(K::GT, prm.G - part * K::GT);
  }
  return U;
}

// Warps per unit among the `rest` units that are left when every warp of the
// grid has taken the same number: the time of a round falls with the warps, a
// set-up and a merge (about 0.15 of a unit) comes with every round.
template <class K>
__device__ __forceinline__ int tail_team(const KParams& prm, int rest, int warps) {
  int best = 1;
  float cost = 1.f;
#pragma unroll
  for (int tw = 2; tw <= K::NC; tw *= 2) {
    if (K::NC % tw != 0 || (tw / 2) * K::TS >= prm.P) break;
    const float rounds = (float)((rest + warps / tw - 1) / (warps / tw));
    const float c = rounds / tw + 0.15f * rounds;
    if (c < cost) {
      cost = c;
      best = tw;
    }
  }
  return best;
}

// Place of row head h's partition p in the workspace's m and l (o: times D).
__device__ __forceinline__ size_t ws_row(const KParams& prm, int s, int h, int p) {
  return ((size_t)s * prm.H + h) * prm.Pmax + p;
}
__device__ __forceinline__ void put_stat(const KParams& prm, const Kv4Unit& U, int row, float m, float l,
                                         uint64_t keep) {
  const size_t at = ws_row(prm, U.s, U.h0 + row, U.p);
  st_f32_policy(prm.ws_m + at, m * kLn2, keep);
  st_f32_policy(prm.ws_l + at, l, keep);
  if (U.np == 1 && prm.lse) prm.lse[out_row_rt(prm, U.s, U.h0 + row)] = m * kLn2 + logf(l);
}

// Unused partitions: sentinels (m = -inf, l = 0).  Empty sequences: zeros (a
// multi-query sequence is never empty: it holds its new tokens).  A warp takes
// a row (s, h) at a time.
template <class K>
__device__ __forceinline__ void kv4_sentinels(const KParams& prm, const int* lens, int warp, int lane) {
  using T = typename K::T;
  const int rows = prm.S * prm.H, step = gridDim.x * K::NC;
  for (int row = blockIdx.x + gridDim.x * warp; row < rows; row += step) {
    const int np = (lens[row / prm.H] + prm.P - 1) / prm.P;
    for (int p = np + lane; p < prm.Pmax; p += 32) {
      prm.ws_m[(size_t)row * prm.Pmax + p] = -INFINITY;
      prm.ws_l[(size_t)row * prm.Pmax + p] = 0.f;
    }
    if (np == 0 && prm.q_len == 1) {
      uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(prm.out) + (size_t)row * K::D);
      for (int i = lane; i < K::D / 8; i += 32) out[i] = make_uint4(0, 0, 0, 0);
      if (prm.lse && lane == 0) prm.lse[row] = -INFINITY;
    }
  }
}

// (Out of line: a wait that does not succeed at once has time for a call.)
// try_wait sleeps for longer than a copy takes, and the global timer ticks about
// as seldom as copies land: a short limit is met by looking at the barrier and
// the SM's clock (two cycles a nanosecond or so) in turn.
constexpr long long kShortWaitNs = 1 << 20;
static __device__ __noinline__ bool kv4_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                                  int* err_word, long long timeout_ns, int slot) {
  bool ok = true;
  if (timeout_ns >= kShortWaitNs) {
    ok = wait_bounded(bar, parity, abort_flag, err_word, timeout_ns, kSiteFull, slot);
  } else {
    const long long t0 = clock64();
    while (ok && !mbar_test_wait(bar, parity)) {
      ok = !*abort_flag;
      if (ok && clock64() - t0 > 2 * timeout_ns) {
        record_timeout(abort_flag, err_word, kSiteFull, slot);
        ok = false;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
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

// A warp's stages, asked for ahead of their use: those of a run of blocks, then
// those of the run that `queue` named.  (Everything but the ids is the same in
// all lanes.)
template <class K>
struct Kv4Stream {
  struct Run {
    const int32_t* row;  // block ids
    const uint8_t* base; // the kv head's record of block 0
    int blocks;
  };
  const KParams& prm;
  uint32_t in, out;      // byte offsets in the ring of the next stage to fill, and of the next to use
  uint32_t bar_in, bar_out, ph_out;  // their barriers, and the phase of the latter
  uint32_t ring, bars;   // shared addresses of the warp's ring and barriers
  Run cur, next;
  int blk;               // blocks of the current run asked for
  int ahead;             // stages asked for and not used
  int ids, ids_after;    // lane's ids of the current window of 32 blocks, and of the one after
  int ids_next;          // ... and of the next run's first window
  size_t block_bytes;    // of all kv heads
  uint64_t policy;

  __device__ __forceinline__ Kv4Stream(const KParams& p, uint32_t r, uint32_t b)
      : prm(p), in(0), out(0), bar_in(b), bar_out(b), ph_out(0), ring(r), bars(b), cur{nullptr, nullptr, 0},
        next{nullptr, nullptr, 0}, blk(0), ahead(0), ids(0), ids_after(0), ids_next(0),
        block_bytes((size_t)p.KH * K::REC), policy(l2_policy_evict_first()) {}

  __device__ __forceinline__ static int fetch(const Run& r, int b0, int lane) {
    return b0 + lane < r.blocks ? __ldg(r.row + b0 + lane) : 0;
  }
  // The run to follow the current one.
  __device__ __forceinline__ void queue(const Run& r, int lane) {
    next = r;
    ids_next = fetch(r, 0, lane);
  }
  __device__ __forceinline__ void fill(int lane) {
    while (ahead < K::NS && issue(lane)) {
    }
  }
  // Fills the next stage (it is free: this warp has used it, or never filled
  // it); false: nothing is left to ask for.
  __device__ __forceinline__ bool issue(int lane) {
    if (blk >= cur.blocks) {
      if (next.blocks == 0) return false;
      cur = next;
      next.blocks = 0;
      blk = 0;
      ids = check_block_id(prm, ids_next);
      ids_after = fetch(cur, 32, lane);
    } else if ((blk & 31) == 0) {
      ids = check_block_id(prm, ids_after);
      ids_after = fetch(cur, blk + 32, lane);
    }
    int id[K::NBLK];
#pragma unroll
    for (int k = 0; k < K::NBLK; ++k) id[k] = __shfl_sync(0xffffffffu, ids, (blk + k) & 31);
    const int n = min(K::NBLK, cur.blocks - blk);
    if (elect_one()) {
      mbar_arrive_expect_tx(bar_in, (uint32_t)n * K::BLOCK);
#pragma unroll
      for (int k = 0; k < K::NBLK; ++k)
        if (k < n)
          bulk_copy_cta(ring + in + k * K::BLOCK, cur.base + (uint32_t)id[k] * block_bytes, K::BLOCK, bar_in, policy);
    }
    blk += K::NBLK;
    ++ahead;
    in += K::STAGE;
    bar_in += 8;
    if (in == K::NS * K::STAGE) {
      in = 0;
      bar_in = bars;
    }
    return true;
  }
  // Waits for the next stage to land; false: gave up.
  __device__ __forceinline__ bool wait(volatile int* abort_flag) const {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar_out, ph_out))) return true;
    return kv4_wait_slow(bar_out, ph_out, abort_flag, prm.hdr + kHdrError, prm.timeout_ns, (int)(out / K::STAGE));
  }
  __device__ __forceinline__ void used() {
    // The stage is refilled by bulk copies (async proxy): every lane's reads
    // of it are ordered before that by a proxy fence.
    fence_proxy_async_smem();
    __syncwarp();
    --ahead;
    out += K::STAGE;
    bar_out += 8;
    if (out == K::NS * K::STAGE) {
      out = 0;
      bar_out = bars;
      ph_out ^= 1u;
    }
  }
  // After a wait that gave up: nothing more is asked for, and no copy of this
  // warp stays in flight (bounded).
  __device__ __forceinline__ void drain() {
    while (ahead > 0) {
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(bar_out, ph_out) && (long long)(global_timer_ns() - t0) < 100000000LL) {
      }
      used();
    }
    cur.blocks = next.blocks = 0;
  }
};

template <class K>
__global__ void __launch_bounds__(K::THREADS, 1) kv4_decode_kernel(const __grid_constant__ KParams prm) {
  using T = typename K::T;
  using Run = typename Kv4Stream<K>::Run;
  extern __shared__ __align__(1024) uint8_t smem[];
  // (The warp index by a shuffle: known to be the same in all lanes.)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t sbase = smem_addr(smem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + K::OFF_FLAGS);
  int* bad_len = reinterpret_cast<int*>(smem + K::OFF_FLAGS + 16);
  int* pref = reinterpret_cast<int*>(smem + K::OFF_PREF);
  int* lens = pref + kMaxSeqsPerLaunch + 1;
  if (tid == 0) {
    *abort_flag = 0;
    *bad_len = 0;
  }
  if (lane < K::NS) mbar_init(sbase + K::OFF_BAR + (warp * K::NSMAX + lane) * 8, 1);
  fence_mbarrier_init();
  __syncthreads();
  // pref: an exclusive scan (the warp totals are kept in the ring, not filled yet).
  {
    int* scan = reinterpret_cast<int*>(smem);
    const int S = prm.S, per = (S + K::THREADS - 1) / K::THREADS;
    const int beg = min(tid * per, S), end = min(beg + per, S);
    bool bad = false;
    int sum = 0;
    for (int s = beg; s < end; ++s) {
      // (A multi-query sequence holds its q_len new tokens.)
      const int L = prm.lens[s], cap = prm.MB * K::TB;
      bad |= L < (prm.q_len > 1 ? prm.q_len : 0) || L > cap;
      lens[s] = min(max(L, 0), cap);
      pref[s] = sum;
      sum += (lens[s] + prm.P - 1) / prm.P;
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
    for (int w = 0; w < K::NC; ++w) {
      const int v = scan[w];
      if (w < warp) before += v;
      all += v;
    }
    for (int s = beg; s < end; ++s) pref[s] += before + incl - sum;
    if (tid == 0) pref[S] = all;
    fence_proxy_async_smem();  // the ring is filled by bulk copies from here on
  }
  __syncthreads();
  // Units [0, solo) go to single warps, the rest to teams of TW.
  const int total = pref[prm.S] * (prm.KH / K::KVU) * prm.hg_per_kv, warps = (int)gridDim.x * K::NC;
  int solo = total / warps * warps;
  const int TW = tail_team<K>(prm, total - solo, warps);
  if (TW == 1) solo = total;
  // A programmatic dependent of the kernel that clears the workspace header:
  // nothing below may touch the header before it has completed.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tid == 0 && *bad_len) atomicCAS(prm.hdr + kHdrError, 0, kErrDeviceBounds);

  const uint64_t keep = l2_policy_evict_last();
  Kv4Stream<K> in(prm, sbase + warp * K::RING, sbase + K::OFF_BAR + warp * K::NSMAX * 8);
  Kv4State<K> st(lane);
  typename Kv4State<K>::Rows q;
  auto run_of = [&](const Kv4Unit& U, int b0, int blocks) {
    return Run{prm.bt + (size_t)U.s * prm.MB + U.t0 / K::TB + b0,
               static_cast<const uint8_t*>(prm.kc) + (size_t)U.kv * K::REC, blocks};
  };
  auto load_rows = [&](const Kv4Unit& U) {
    st.load_rows(q, [&](int i) { return static_cast<const T*>(prm.q) + out_row_rt(prm, U.s, U.h0 + i) * K::D; }, U.nh,
                 lane);
  };

  // The first units are dealt out over the CTAs; the counter hands out the rest.
  const int ltw = __ffs(TW) - 1, team = warp >> ltw, tw = warp & (TW - 1);
  bool alone = true, alive = true;
  int u = blockIdx.x + (int)gridDim.x * warp;
  // A warp's unit and the next one wait in shared memory while the stages are
  // worked on: registers that spill cost more (beside 227 KB of shared memory
  // little is left of the L1 cache, so a spilled value comes from L2).
  Kv4Unit* at = reinterpret_cast<Kv4Unit*>(smem + K::OFF_UNIT) + 2 * warp;
  int par = 0;
  if (u < solo) {
    const Kv4Unit U = kv4_unit<K>(prm, pref, lens, u);
    at[0] = U;
    in.queue(run_of(U, 0, U.nb), lane);
    in.fill(lane);
    load_rows(U);
  }
  kv4_sentinels<K>(prm, lens, warp, lane);  // (while the first copies fly)
  while (true) {
    if (alone && u >= solo) {
      // On to the teams' units, dealt out like the first ones.
      if (TW == 1) break;
      alone = false;
      u = solo + blockIdx.x + (int)gridDim.x * team;
    }
    if (u >= total) break;
    int i0 = 0, n, u_next = total, tok, end, least;
    {
      Kv4Unit U;
      if (alone) {
        if (lane == 0) u_next = atomicAdd(prm.hdr + kHdrWork, 1) + warps;
        U = at[par];
        n = U.stages;
      } else {
        U = kv4_unit<K>(prm, pref, lens, u);
        at[par] = U;
        const int per = (U.stages + TW - 1) >> ltw;
        i0 = min(tw * per, U.stages);
        n = min(per, U.stages - i0);
        if (alive && n > 0) {
          in.queue(run_of(U, i0 * K::NBLK, min(n * K::NBLK, U.nb - i0 * K::NBLK)), lane);
          in.fill(lane);
        }
        load_rows(U);
        u_next = u + (int)gridDim.x * (K::NC >> ltw);
      }
      tok = U.t0 + i0 * K::TS;
      end = U.t1;
      least = U.L - prm.q_len + 1;
    }
    st.begin_unit(q, prm.scale_log2);
    for (int i = 0; i < n && alive; ++i, tok += K::TS) {
      if (!in.wait(abort_flag)) {
        in.drain();
        alive = false;
        break;
      }
      if (alone && i == (n > 1 ? 1 : 0)) {
        // The claim has been answered: what is asked for runs on into the next unit.
        u_next = __shfl_sync(0xffffffffu, u_next, 0);
        if (u_next < solo) {
          const Kv4Unit V = kv4_unit<K>(prm, pref, lens, u_next);
          at[par ^ 1] = V;
          in.queue(run_of(V, 0, V.nb), lane);
        }
      }
      st.pass(in.ring + in.out, end - tok, tok, least,
              [&](int col) {
                const Kv4Unit& U = at[par];
                if (prm.q_len == 1 || !st.has_row(col, U.nh)) return U.L;
                return row_limit<true>(prm, U.L, U.h0 + st.row_of(col, U.nh));
              },
              lane);
      in.used();
      in.fill(lane);
    }
    const Kv4Unit U = at[par];
    if (alone) {
      if (!alive) {
        u = solo;
        continue;
      }
      // The partition's normalised output, into the workspace; from there on
      // to the output where the sequence has one partition.
      float* rows = prm.ws_o + ws_row(prm, U.s, U.h0, U.p) * K::D;
      const size_t stride = (size_t)prm.Pmax * K::D;
      st.finish(rows, stride, U.nh, false, [&](int col, float m, float l) { put_stat(prm, U, col, m, l, keep); }, lane);
      if (U.np == 1) {
        __syncwarp();
        for (int i = lane; i < U.nh * K::KVU * (K::D / 4); i += 32) {
          const int col = i / (K::D / 4), d = 4 * (i - col * (K::D / 4));
          store4<T>(static_cast<T*>(prm.out) + out_row_rt(prm, U.s, U.h0 + col) * K::D + d,
                    *reinterpret_cast<const float4*>(rows + col * stride + d));
        }
      }
      par ^= 1;
      if (u_next < solo) load_rows(at[par]);
    } else {
      // The team's states, each in its warp's ring (whose stages are all used).
      float* state = reinterpret_cast<float*>(smem + warp * K::RING);
      st.finish(state, K::AROW, U.nh, true,
                [&](int col, float m, float l) {
                  *reinterpret_cast<float2*>(state + K::GT * K::AROW + 2 * col) = make_float2(m, l);
                },
                lane);
      named_barrier_sync(1 + team, TW * 32);
      // A slice of the rows each; the warps' states in warp order.
      const float* first = reinterpret_cast<const float*>(smem + (warp - tw) * K::RING);
      constexpr int D4 = K::D / 4, WR = K::RING / 4;
      for (int i = tw * 32 + lane; i < U.nh * K::KVU * D4; i += TW * 32) {
        const int row = i / D4, d4 = i - row * D4, col = Kv4State<K>::column_of(row, U.nh);
        float M = -INFINITY;
        for (int w = 0; w < TW; ++w) M = fmaxf(M, first[w * WR + K::GT * K::AROW + 2 * col]);
        // (A row that sees nothing in this partition has M = -inf: its weights are 0.)
        const float Ms = M == -INFINITY ? 0.f : M;
        float den = 0.f;
        float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < TW; ++w) {
          const float2 s2 = *reinterpret_cast<const float2*>(first + w * WR + K::GT * K::AROW + 2 * col);
          const float f = ex2(s2.x - Ms);
          const float4 v = *reinterpret_cast<const float4*>(first + w * WR + col * K::AROW + 4 * d4);
          den = fmaf(f, s2.y, den);
          num.x = fmaf(f, v.x, num.x);
          num.y = fmaf(f, v.y, num.y);
          num.z = fmaf(f, v.z, num.z);
          num.w = fmaf(f, v.w, num.w);
        }
        const float inv = den == 0.f ? 0.f : 1.f / den;
        const float4 val = make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv);
        if (U.np == 1) {
          store4<T>(static_cast<T*>(prm.out) + out_row_rt(prm, U.s, U.h0 + row) * K::D + 4 * d4, val);
        } else {
          st_f4_policy(reinterpret_cast<float4*>(prm.ws_o + ws_row(prm, U.s, U.h0 + row, U.p) * K::D) + d4, val, keep);
        }
        if (d4 == 0) put_stat(prm, U, row, M, den, keep);
      }
      fence_proxy_async_smem();  // the rings are filled by bulk copies again
      named_barrier_sync(1 + team, TW * 32);
    }
    u = u_next;
  }
  // Phase 2 may be launched once every CTA has said so or ended (it waits for
  // this grid to complete before it reads anything).
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace pa
