// pa_kv4.cuh -- tensor-core consumer for the paged decode kernel over a cache
// held in 4 bits.
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
// of two 2^12 / vb, vb above every value scale the warp has met (raised, with
// the accumulators, when a larger one comes), so they stay in fp16's range
// whatever the cache's magnitude.
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
#pragma once

#include "pa_common.cuh"

namespace pa {

template <typename T_, int D_, int BS_, int KVU_>
struct Kv4Consumer {
  using T = T_;
  static constexpr bool kTma = false;
  static constexpr bool kRecord = true;  // keys, values and parameters of a block are one run of bytes
  static constexpr int D = D_, BS = BS_, GT = 8;
  static constexpr int KVU = KVU_;  // kv heads per unit (G * KVU <= 8 columns)
  static constexpr bool kMma = true;
  static constexpr bool kCausal = false;
  static constexpr uint32_t X = D_ < 128 ? D_ : 128;  // dims per slab
  static constexpr int NSLAB = D_ / (int)X;
  static constexpr uint32_t XB = X / 2;               // bytes of a token row in a slab
  static constexpr uint32_t SLAB = (uint32_t)BS_ * XB;
  static constexpr uint32_t VOFFSET = (uint32_t)BS_ * D_ / 2;  // value codes in a record
  static constexpr uint32_t POFFSET = (uint32_t)BS_ * D_;      // parameters in a record
  static constexpr uint32_t REC = (uint32_t)BS_ * (D_ + 8);
  static constexpr uint32_t KBLK = (uint32_t)KVU_ * REC;
  static constexpr uint32_t KREGION = 0;
  static constexpr uint32_t STAGE_BYTES = KBLK;
  static constexpr uint32_t STAGE_TX = KBLK;
  static_assert(D_ % (int)X == 0 && X % 16 == 0 && KBLK % 16 == 0, "whole slabs, 16-byte units");
  static constexpr int KV_ESZ = 1;
  static constexpr int kIssueBatch = (KBLK <= 2304) ? 32 : 16;
  static constexpr int kItemBlocks = BS_ <= 16 ? 2 : 1;
  static constexpr int SCRATCH_FLOATS = 0;
  static constexpr int QROW = D_ + 8;
  static constexpr int AROW = D_ + 4;
  // 4-byte words of a slab row per lane quad member (keys) and per lane group (values).
  static constexpr int KW = ((int)X / 8 + 3) / 4;
  static constexpr int VW = ((int)X / 8 + 7) / 8;
  static constexpr int NK = NSLAB * KW * 2;   // k-steps of the score product
  static constexpr int MTS = VW * 4;          // 16-dim tiles of a slab's value product
  static constexpr int NMT = NSLAB * MTS;
  static constexpr uint32_t LO = 0x000f000fu, HI = 0x00f000f0u;

  uint32_t qb[NK][2];  // Q^T fragments: the query row of column lane / 4
  float m[2], l[2];    // columns 2 (lane % 4) and + 1
  float zs[2];         // sum of weight * (value zero + 8 value scale)
  float acc[NMT][4], acc8[4];
  float kf, qz[2];     // score factors: scale_log2 over the operands' powers of two; times sum(q)
  float vb, vinv;      // see above: vb a power of two, vinv = 2^12 / vb
  int lim[2];
  int own[2], ub;      // kv head (0 .. KVU - 1) of the lane's columns, and of column lane / 4

  __device__ __forceinline__ static int tok_lo(int i) { return (i & 1) ? 7 - (i >> 1) : (i >> 1); }

  __device__ __forceinline__ static uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
  }
  __device__ __forceinline__ static void lds64(uint32_t a, uint32_t& x, uint32_t& y) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(a));
  }
  __device__ __forceinline__ static void lds128(uint32_t a, uint32_t* v) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(a));
  }
  // KW words of a key row from word c * KW on (row strides: 32, 40, 48, 56 or 64 bytes).
  __device__ __forceinline__ static void key_words(uint32_t a, uint32_t (&w)[KW]) {
    if constexpr (KW == 4 && XB % 16 == 0) {
      lds128(a, w);
    } else if constexpr (KW % 2 == 0) {
#pragma unroll
      for (int i = 0; i < KW; i += 2) lds64(a + 4 * i, w[i], w[i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < KW; ++i) w[i] = lds32(a + 4 * i);
    }
  }
  __device__ __forceinline__ static float2 params2(uint32_t w) { return F16Traits<T>::to_float2(w); }

  template <class F>
  __device__ __forceinline__ void set_limits(F limit_of, int lane) {
#pragma unroll
    for (int j = 0; j < 2; ++j) lim[j] = limit_of((lane & 3) * 2 + j);
  }

  __device__ __forceinline__ void begin_unit(const T* qs, int nh, float sl2, int lane, int G) {
    const int n = lane >> 2, c = lane & 3;
    ub = KVU_ > 1 ? n / G : 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) own[j] = KVU_ > 1 ? min((2 * c + j) / G, KVU_ - 1) : 0;
    const uint16_t* q16 = reinterpret_cast<const uint16_t*>(qs) + n * QROW;
    // Dims 8w .. 8w + 7 of head n are word w of a slab; this lane holds words
    // c * KW .. of each slab.
    float amax = 0.f, sum = 0.f;
#pragma unroll
    for (int sl = 0; sl < NSLAB; ++sl)
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        const int w = c * KW + i;
        if (n < nh && w < (int)X / 8) {
          const uint4 v = *reinterpret_cast<const uint4*>(q16 + sl * X + w * 8);
          const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = F16Traits<T>::to_float2(e[k]);
            amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
            sum += f.x + f.y;
          }
        }
      }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    // 2^s brings the unit's largest |q| below 2^15; zero, subnormal, Inf or
    // NaN leave the query unscaled.
    const int E = (__float_as_int(amax) >> 23) & 0xff;
    const int s = (E == 0 || E == 255) ? 0 : max(-113, min(110, 141 - E));
    const float up = __int_as_float((127 + s) << 23), up16 = up * 0.0625f;
#pragma unroll
    for (int sl = 0; sl < NSLAB; ++sl)
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        const int w = c * KW + i;
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = 0.f;
        if (n < nh && w < (int)X / 8)
          unpack_chunk<T>(*reinterpret_cast<const uint4*>(q16 + sl * X + w * 8), f);
        const int ks = (sl * KW + i) * 2;
        qb[ks][0] = F16Traits<__half>::pack(f[0] * up, f[4] * up);
        qb[ks][1] = F16Traits<__half>::pack(f[1] * up16, f[5] * up16);
        qb[ks + 1][0] = F16Traits<__half>::pack(f[2] * up, f[6] * up);
        qb[ks + 1][1] = F16Traits<__half>::pack(f[3] * up16, f[7] * up16);
      }
    kf = sl2 * __int_as_float((127 - s) << 23) * 16777216.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      qz[j] = sl2 * __shfl_sync(0xffffffffu, sum, (2 * c + j) * 4);
      m[j] = -INFINITY;
      l[j] = zs[j] = 0.f;
    }
#pragma unroll
    for (int mt = 0; mt < NMT; ++mt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[mt][i] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc8[i] = 0.f;
    vb = 7.888609052210118e-31f;  // 2^-100
    vinv = 4096.f / vb;
  }

  __device__ __forceinline__ void block(const uint8_t* s, const uint8_t*, int ntok, int lane, float*, int tok0) {
    const uint32_t a = smem_addr(s);
    if constexpr (BS == 8) {
      // Half a tile: rows 8..15 read the block again and are masked.
      const uint32_t lo[1] = {a}, hi[1] = {a};
      const int tl[1] = {0}, th[1] = {0};
      tiles<1>(lo, hi, tl, th, ntok, lane, tok0);
    } else {
      constexpr int NTT = BS / 16, NTU = NTT < 2 ? NTT : 2;
#pragma unroll
      for (int h = 0; h < NTT / NTU; ++h) {
        if (h > 0 && ntok <= h * 16 * NTU) break;
        uint32_t lo[NTU], hi[NTU];
        int tl[NTU], th[NTU];
#pragma unroll
        for (int t = 0; t < NTU; ++t) {
          lo[t] = hi[t] = a;
          tl[t] = (h * NTU + t) * 16;
          th[t] = tl[t] + 8;
        }
        tiles<NTU>(lo, hi, tl, th, ntok - h * 16 * NTU, lane, tok0 + h * 16 * NTU);
      }
    }
  }

  __device__ __forceinline__ void block_pair(const uint8_t* sA, const uint8_t*, const uint8_t* sB, const uint8_t*,
                                             int ntok, int lane, int tok0) {
    const uint32_t a = smem_addr(sA), b = smem_addr(sB);
    if constexpr (BS == 8) {
      const uint32_t lo[1] = {a}, hi[1] = {b};
      const int tl[1] = {0}, th[1] = {0};
      tiles<1>(lo, hi, tl, th, ntok, lane, tok0);
    } else {
      static_assert(BS == 8 || BS == 16 || kItemBlocks == 1, "pairs are 8- or 16-token blocks");
      const uint32_t lo[2] = {a, b}, hi[2] = {a, b};
      const int tl[2] = {0, 0}, th[2] = {8, 8};
      tiles<2>(lo, hi, tl, th, ntok, lane, tok0);
    }
  }

  // NT 16-token tiles: tokens 0..7 of tile t are tokens tl[t].. of the record
  // at lo[t], tokens 8..15 tokens th[t].. of the record at hi[t]; ntok of the
  // item's tokens lie before the sequence end, and its first is token tok0.
  template <int NT>
  __device__ __forceinline__ void tiles(const uint32_t (&lo)[NT], const uint32_t (&hi)[NT], const int (&tl)[NT],
                                        const int (&th)[NT], int ntok, int lane, int tok0) {
    const int r = lane >> 2, c = lane & 3;
    const int trow = tok_lo(r);
    float sc[NT][4];
    float2 pv[NT][2][2];  // (value scale, value zero) of the lane's two score rows, per column
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float dot[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < KVU; ++u) {
        float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int sl = 0; sl < NSLAB; ++sl) {
          uint32_t wl[KW], wh[KW];
          key_words(lo[t] + u * REC + sl * SLAB + (tl[t] + trow) * XB + c * (KW * 4), wl);
          key_words(hi[t] + u * REC + sl * SLAB + (th[t] + trow) * XB + c * (KW * 4), wh);
#pragma unroll
          for (int i = 0; i < KW; ++i) {
            const int ks = (sl * KW + i) * 2;
            const uint32_t a[4] = {wl[i] & LO, wh[i] & LO, wl[i] & HI, wh[i] & HI};
            Mma<__half>::run(c0, a, qb[ks][0], qb[ks][1]);
            const uint32_t xl = wl[i] >> 8, xh = wh[i] >> 8;
            const uint32_t b[4] = {xl & LO, xh & LO, xl & HI, xh & HI};
            Mma<__half>::run(c1, b, qb[ks + 1][0], qb[ks + 1][1]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v = c0[i] + c1[i];
          dot[i] = (KVU == 1 || own[i & 1] == u) ? v : dot[i];
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // score rows r and r + 8
        const int tt = t * 16 + 8 * h + trow;
        const uint32_t pa = (h ? hi[t] + (th[t] + trow) * 8 : lo[t] + (tl[t] + trow) * 8) + POFFSET;
        float2 k = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (j == 0 || KVU > 1) {
            uint32_t wk, wv;
            lds64(pa + (KVU > 1 ? own[j] * REC : 0u), wk, wv);
            k = params2(wk);
            pv[t][h][j] = params2(wv);
          } else {
            pv[t][h][1] = pv[t][h][0];
          }
          const float z = fmaf(k.x * kf, dot[2 * h + j], k.y * qz[j]);
          // Slots past the sequence end hold arbitrary parameters: cleared.
          if (tt >= ntok) pv[t][h][j] = make_float2(0.f, 0.f);
          sc[t][2 * h + j] = (tt < ntok && tok0 + tt < lim[j]) ? z : -INFINITY;
        }
      }
    }
    // Weights and running statistics.
    float alpha[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float bm = fmaxf(sc[0][j], sc[0][j + 2]);
#pragma unroll
      for (int t = 1; t < NT; ++t) bm = fmaxf(bm, fmaxf(sc[t][j], sc[t][j + 2]));
      bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 4));
      bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 8));
      bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 16));
      const float mn = fmaxf(m[j], bm);
      const float ms = (mn == -INFINITY) ? 0.f : mn;  // a row that has seen no position yet
      alpha[j] = exp2f(m[j] - ms);
      m[j] = mn;
      float ps = 0.f;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // A row's masked positions weigh nothing, whatever their parameters hold.
          const bool seen = sc[t][2 * h + j] != -INFINITY;
          sc[t][2 * h + j] = exp2f(sc[t][2 * h + j] - ms);
          ps += sc[t][2 * h + j];
          if (!seen) pv[t][h][j] = make_float2(0.f, 0.f);
        }
      l[j] = fmaf(l[j], alpha[j], ps);
      zs[j] *= alpha[j];
    }
    // The value scales' bound (finite scales only: a NaN or Inf goes through
    // to the output whatever the bound is).
    float vm = 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float a = fabsf(pv[t][h][j].x);
          vm = a < INFINITY ? fmaxf(vm, a) : vm;
        }
    float down = 1.f;
    if (__any_sync(0xffffffffu, vm >= vb)) {
      // The power of two above the largest scale (both positive: ordered as integers).
      const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(vm));
      const float nb = __uint_as_float(min((top >> 23) + 1u, 254u) << 23);
      down = vb / nb;
      vb = nb;
      vinv = 4096.f / nb;
    }
    const float a0 = alpha[0] * down, a1 = alpha[1] * down;
#pragma unroll
    for (int mt = 0; mt < NMT; ++mt) {
      acc[mt][0] *= a0;
      acc[mt][1] *= a1;
      acc[mt][2] *= a0;
      acc[mt][3] *= a1;
    }
    acc8[0] *= a0;
    acc8[1] *= a1;
    acc8[2] *= a0;
    acc8[3] *= a1;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float w[4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float p = sc[t][2 * h + j];
          const float2 v = pv[t][h][j];
          zs[j] = fmaf(p, fmaf(8.f, v.x, v.y), zs[j]);
          w[2 * h + j] = p * (v.x * vinv);
        }
      const uint32_t b0 = movmatrix_trans(F16Traits<__half>::pack(w[0], w[1]));
      const uint32_t b1 = movmatrix_trans(F16Traits<__half>::pack(w[2], w[3]));
      const uint32_t eight[4] = {0x00080008u, 0x00080008u, 0x00080008u, 0x00080008u};
      Mma<__half>::run(acc8, eight, b0, b1);
#pragma unroll
      for (int u = 0; u < KVU; ++u) {
        // kv head u's product takes the weight columns of its own query heads.
        const bool mine = KVU == 1 || ub == u;
        const uint32_t m0 = mine ? b0 : 0u, m1 = mine ? b1 : 0u;
#pragma unroll
        for (int sl = 0; sl < NSLAB; ++sl) {
          // Slots 2c, 2c + 1 and 2c + 8, 2c + 9 hold tokens c, 7 - c, 8 + c, 15 - c.
          const uint32_t base = u * REC + VOFFSET + sl * SLAB + r * (VW * 4);
          uint32_t wa[2], wb[2], wc[2], wd[2];
          value_words(lo[t] + base + (tl[t] + c) * XB, wa);
          value_words(lo[t] + base + (tl[t] + 7 - c) * XB, wb);
          value_words(hi[t] + base + (th[t] + c) * XB, wc);
          value_words(hi[t] + base + (th[t] + 7 - c) * XB, wd);
#pragma unroll
          for (int half = 0; half < VW; ++half) {
            // VW = 2: rows r and r + 8 of tile mt hold nibble mt of the two
            // words (nibbles 0-3, then 4-7); VW = 1: nibbles mt and mt + 4 of the one.
            const uint32_t sel = half ? 0x7632u : 0x5410u;
            uint32_t x0, x1, x2, x3;
            if constexpr (VW == 2) {
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
            const int mt = sl * MTS + half * 4;
            const uint32_t f0[4] = {x0 & LO, x1 & LO, x2 & LO, x3 & LO};
            Mma<__half>::run(acc[mt], f0, m0, m1);
            const uint32_t f1[4] = {x0 & HI, x1 & HI, x2 & HI, x3 & HI};
            Mma<__half>::run(acc[mt + 1], f1, m0, m1);
            x0 >>= 8; x1 >>= 8; x2 >>= 8; x3 >>= 8;
            const uint32_t f2[4] = {x0 & LO, x1 & LO, x2 & LO, x3 & LO};
            Mma<__half>::run(acc[mt + 2], f2, m0, m1);
            const uint32_t f3[4] = {x0 & HI, x1 & HI, x2 & HI, x3 & HI};
            Mma<__half>::run(acc[mt + 3], f3, m0, m1);
          }
        }
      }
    }
  }
  __device__ __forceinline__ static void value_words(uint32_t a, uint32_t (&w)[2]) {
    if constexpr (VW == 2) {
      lds64(a, w[0], w[1]);
    } else {
      w[0] = lds32(a);
      w[1] = 0u;
    }
  }

  __device__ __forceinline__ void finish(float* acc_out, float* ml, int lane) {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float ls = l[j], z = zs[j];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        ls += __shfl_xor_sync(0xffffffffu, ls, o);
        z += __shfl_xor_sync(0xffffffffu, z, o);
      }
      if (r == 0) {
        ml[(2 * c + j) * 2] = m[j];
        ml[(2 * c + j) * 2 + 1] = ls;
      }
      float* o = acc_out + (2 * c + j) * AROW;
      // Tiles of odd nibbles carry 2^-20 instead of 2^-24.
      const float e8 = acc8[j], e16 = 16.f * e8;
#pragma unroll
      for (int sl = 0; sl < NSLAB; ++sl)
#pragma unroll
        for (int h = 0; h < 2; ++h)   // rows r and r + 8
#pragma unroll
          for (int q = 0; q < VW; ++q) {
            // Dims of row half h: VW = 2: 16 r + 8 h + 4 q ..; VW = 1: 8 r + 4 h ..
            const int d = VW == 2 ? 16 * r + 8 * h + 4 * q : 8 * r + 4 * h;
            const int mt = sl * MTS + 4 * q;
            float4 v;
            v.x = fmaf((acc[mt][2 * h + j] - e8) * 4096.f, vb, z);
            v.y = fmaf((acc[mt + 1][2 * h + j] - e16) * 256.f, vb, z);
            v.z = fmaf((acc[mt + 2][2 * h + j] - e8) * 4096.f, vb, z);
            v.w = fmaf((acc[mt + 3][2 * h + j] - e16) * 256.f, vb, z);
            if (d < (int)X) *reinterpret_cast<float4*>(o + sl * X + d) = v;
          }
    }
  }
};

}  // namespace pa
