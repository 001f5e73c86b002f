// pa_rows.cuh -- view attention (windows, trees) with many query rows a kv head, on
// the fifth-generation tensor cores (16-bit caches).
//
// The rows of a kv head (query tokens x query heads of its group) are the M = 128
// side of the products, so that a block of the cache is read once for 128 rows,
// where the units of 8 rows of pa_mma.cuh read it once for 8:
//
//   S[rows x tokens] = Q[rows x D] . K^T       tcgen05.mma, Q in tensor memory
//   O[rows x D]     += P[rows x tokens] . V    tcgen05.mma, P in tensor memory
//
// Both operands of the cache are read as they lie in the page layouts.  A key block
// [D/8][BS][8] is a column of core matrices (8 tokens x 16 bytes) for each chunk of
// eight dims; one instruction takes a block's tokens, or the same eight tokens of
// every block of a tile (the stride between rows of core matrices is then that
// between blocks).  (Blocks copied chunk by chunk, to make one column of core
// matrices of a tile, took 450 us where whole blocks took 160: a bulk copy of 256
// bytes takes as long as one of 4 KB.)  A value block [D][BS] is K-major with rows of
// 2 BS bytes: the tensor copy stores it in the swizzle of that width.  Q is in tensor
// memory because a product of N = 32 columns then takes 17 cycles, and 42 with Q in
// shared memory, whose 4 KB it reads every time (measured; N = 128: 65 either way).
//
// One CTA per SM, persistent over units (sequence, partition, kv head, up to 128
// rows), which a producer warp takes from the global counter (as in pa_kernel.cuh)
// and streams through a ring of K and V tiles of 64 tokens; two warps bring Q, a unit
// ahead; one warp issues the scores' products, one those with the values.  Warpgroups of four warps, a row a thread, turn
// scores into weights: two of them (NP = 2) take the tiles in turn, each with its own
// O, joined at the end of the unit; at head size 256 one does all.  Scores are
// computed up to NBUF tiles ahead, into buffers that the weights then take over.
//
// Softmax: scores in fp32; a row keeps a reference (the maximum when it was last
// set) and sets a new one, rescaling O, only where its maximum has grown by more
// than 2^8 over it: weights stay below 2^8, whose sums in fp32 and, for fp16,
// roundings are as exact as those of weights below 1.  fp16 weights are rounded once;
// bf16 ones are the sum of two terms (two products), as in pa_mma.cuh.
//
// A tile that some row does not see whole is masked row by row, 64 tokens at a time;
// values of it that are not finite are cleared in shared memory (their products with
// other rows' zero weights would be NaN).  Such tiles are noted (RowsOdd), and at the
// end of the unit the rows that see them get their values from the cache added.
//
// 8-bit caches: the ring of tiles is filled by warps that widen E4M3 codes to fp16 from a
// ring of codes, into the layouts of a block of 64 tokens whatever the cache's block.
//
// Measured (32 heads over 8 of 128 dims, blocks of 16; whole calls, one after the other): 16
// nodes of 48 sequences of 1001 to 4999 tokens, bf16 108 us (of the cache's bytes: 82), fp16
// 101; 64 nodes of 16 sequences of 2048 to 8192, bf16 119 (blocks of 32: 111; bytes 49, products
// 85 with two terms a weight), fp16 99, E4M3 155; chunks of 128 tokens over a window of 1024,
// fp16 99, E4M3 123 (products 27).  A tile takes about 1100 cycles (fp16) where its products
// are 530: what is left is the way from a tile's scores through its weights to the buffer's
// next scores, three buffers for two warpgroups; and 5700 cycles from a unit to the next one.
// With one infinite value in a node of 16, over one sequence of 8192 tokens: 155 us instead of 30.
#pragma once

#include <type_traits>

#include <cuda_fp8.h>

#include "pa_kernel.cuh"
#include "pa_tc.cuh"

namespace pa {

constexpr int kRowsMaxUnitSeqs = 256;  // sequences per launch (the order's arrays take shared memory)
constexpr uint32_t kRowsSmem = 227u * 1024u;

struct RowsUnit {
  int s, p, kv, t0, t1, nt, np, nh, h0, L, sink_blocks, skip;
};

// What a unit's values that are not finite leave to its end: the partly seen tiles
// where one was cleared, as a set (tile + 1 by linear probing, 0: free), and for
// 8-bit caches, whose NaN codes are cleared in every tile, the dims (bits) with one in
// a tile that every row sees.  Partly seen tiles lie around the end of the first tokens,
// the start of the window and the end of the rows, each over at most the rows' 512
// tokens: fewer than 28.  (`all` is set if there should be more: every tile is gone through.)
struct RowsOdd {
  static constexpr int kTiles = 32;
  int any, all;
  int tile[kTiles];
  uint32_t dims[8];
  __device__ __forceinline__ void clear(int lane) {  // a warp
    for (int i = lane; i < (int)(sizeof(RowsOdd) / 4); i += 32) reinterpret_cast<int*>(this)[i] = 0;
  }
  __device__ __forceinline__ void add_tile(int i) {
    int at = i % kTiles;
    for (int n = 0; n < kTiles; ++n, at = (at + 1) % kTiles) {
      const int was = atomicCAS(&tile[at], 0, i + 1);
      if (was == 0 || was == i + 1) break;
      if (n + 1 == kTiles) *const_cast<volatile int*>(&all) = 1;
    }
    *const_cast<volatile int*>(&any) = 1;
  }
  __device__ __forceinline__ void add_dim(int d) {
    atomicOr(&dims[d >> 5], 1u << (d & 31));
    *const_cast<volatile int*>(&any) = 1;
  }
};

template <typename T_, int D_, int BS_, bool FP8_ = false>
struct RowsConfig {
  using T = T_;
  static constexpr bool kFp8 = FP8_;
  using MT = typename std::conditional<FP8_, __half, T_>::type;  // of the products' operands
  static constexpr int D = D_, BS = BS_;
  static constexpr int NP = D_ <= 128 ? 2 : 1;      // pipelines (warpgroups)
  static constexpr int NBUF = D_ <= 128 ? 3 : 2;    // buffers of scores and weights
  static constexpr int TN = 64;                     // tokens per tile
  static constexpr int GT = 128, KVU = 1;           // rows per unit; (plan_unit) kv heads per unit
  static constexpr int NB = TN / BS, NG = BS / 8;   // blocks of a tile, groups of eight tokens of a block
  static constexpr int MS = FP8_ ? TN : BS_;        // tokens of a block as the products read it
  static constexpr bool kTma = BS_ >= 16 && !FP8_;
  static constexpr bool kBf16 = std::is_same<MT, __nv_bfloat16>::value;
  // An 8-bit cache's query rows of bf16 go to fp16 by a power of two of their own.
  static constexpr bool kQScale = FP8_ && std::is_same<T_, __nv_bfloat16>::value;
  static constexpr uint32_t BLK = (uint32_t)D_ * BS_ * (FP8_ ? 1 : 2);  // a block of the cache
  static constexpr uint32_t SLOT = (uint32_t)TN * D_ * 2, QTILE = 128u * D_ * 2;
  // 8-bit caches: warps that widen the codes, and the ring of tiles of codes.
  static constexpr int CW = !FP8_ ? 0 : D_ <= 128 ? 4 : 2, NR = !FP8_ ? 0 : D_ <= 128 ? 8 : 2;
  static constexpr uint32_t RSLOT = FP8_ ? (uint32_t)TN * D_ : 0;
  static constexpr int LOADERS = FP8_ ? 32 : 64;  // threads that bring Q
  static constexpr int THREADS = NP * 128 + 96 + LOADERS + CW * 32, UQ = 2;
  // A tile's scores take NI instructions a k-step of N columns each: one a block, or
  // (kGroups) one for each group of eight tokens, of every block, whichever are fewer.
  static constexpr bool kGroups = !FP8_ && NG < NB;
  static constexpr int NI = kGroups ? NG : TN / MS, N = TN / NI;
  // Tensor memory columns: the buffers (scores, then weights: bf16 two words of 16 bits
  // a token), Q (two dims a column), O of either pipeline.
  static constexpr uint32_t Q_COL = NBUF * TN, O_COL = 256, O_STEP = 128;
  static_assert(Q_COL + D_ / 2 <= O_COL && O_COL + (NP == 2 ? 256 : D_) <= 512, "tensor memory");
  // Shared memory: the next unit's Q, the ring, then barriers, units, flags, order.
  static constexpr uint32_t QBYTES = QTILE;
  static constexpr uint32_t bars(int ns) { return 2 * ns + 2 * NR + 2 * UQ + 3 * NBUF + 7; }
  static constexpr uint32_t small(int ns) {
    return al16(bars(ns) * 8) + al16(UQ * sizeof(RowsUnit)) + al16(UQ * sizeof(RowsOdd)) + 64 +
           al16((kRowsMaxUnitSeqs + 1) * 4) + al16(kRowsMaxUnitSeqs * 2);
  }
  static constexpr int kFit = (int)((kRowsSmem - small(D_ > 128 ? 8 : 16) - QBYTES - NR * RSLOT) / SLOT);
  // (An even number: keys have the slots of one parity within a unit, values those of the
  // other, in the middle of it, so that who waits for one kind is a phase off at most.  And
  // NR a multiple of CW, for the warps that widen codes.)
  static constexpr int NS = (kFit < 16 ? kFit : 16) & ~1;
  static_assert(!FP8_ || (NR % (FP8_ ? CW : 1) == 0 && NS >= CW), "a warp's waits for a slot are a phase apart at most");
  static_assert(NS >= 2 * NBUF, "the ring holds the keys that are ahead and two tiles' values");
  // The score column of token t of group gi of eight of block bi.
  static constexpr __device__ __forceinline__ int column(int bi, int gi, int t) {
    return kGroups ? (gi * NB + bi) * 8 + t : bi * BS_ + gi * 8 + t;
  }
  static constexpr uint32_t OFF_RING = QBYTES, OFF_CODES = OFF_RING + NS * SLOT, OFF_BAR = OFF_CODES + NR * RSLOT;
  static constexpr uint32_t OFF_INFO = OFF_BAR + al16(bars(NS) * 8);
  static constexpr uint32_t OFF_ODD = OFF_INFO + al16(UQ * sizeof(RowsUnit));
  static constexpr uint32_t OFF_FLAGS = OFF_ODD + al16(UQ * sizeof(RowsOdd));
  static constexpr uint32_t OFF_PREF = OFF_FLAGS + 64;
  static constexpr uint32_t OFF_PERM = OFF_PREF + al16((kRowsMaxUnitSeqs + 1) * 4);
  static constexpr uint32_t BYTES = OFF_PERM + al16(kRowsMaxUnitSeqs * 2);
  static_assert(BYTES <= kRowsSmem && QBYTES % 1024 == 0 && SLOT % 1024 == 0, "shared memory");
  static_assert(NS * SLOT >= kOrderTempBytes, "prologue temporaries fit in the ring");
  // Barriers.
  static constexpr uint32_t FULL = 0, EMPTY = NS, UFULL = 2 * NS, UEMPTY = UFULL + UQ, SFULL = UEMPTY + UQ,
                            PREADY = SFULL + NBUF, PVDONE = PREADY + NBUF, QSTAGED = PVDONE + NBUF,
                            QTAKEN = QSTAGED + 1, QREADY = QTAKEN + 1, QFREE = QREADY + 1, OFREE = QFREE + 1,
                            XBAR = OFREE + 1, XFREE = XBAR + 1, RFULL = XFREE + 1, REMPTY = RFULL + NR;
  static_assert(REMPTY + NR == bars(NS), "barriers");
  // What the producer fills: the ring of tiles, or of tiles of codes.
  static constexpr int PN = FP8_ ? NR : NS;
  static constexpr uint32_t PFULL = FP8_ ? RFULL : FULL, PEMPTY = FP8_ ? REMPTY : EMPTY;
  static constexpr uint32_t OFF_PRING = FP8_ ? OFF_CODES : OFF_RING, PSLOT = FP8_ ? RSLOT : SLOT;
};

// Wait sites of this kernel (see WaitSite).
enum RowsSite {
  kRowsUnitSlot = 20, kRowsRing = 21, kRowsUnit = 22, kRowsQ = 23, kRowsOFree = 24, kRowsFull = 25, kRowsP = 26,
  kRowsS = 27, kRowsPv = 28, kRowsQFree = 29, kRowsX = 30, kRowsCodes = 31
};

template <class C>
struct RowsCta {
  const KParams& prm;
  uint8_t* smem;
  uint32_t sbase, bar0;
  volatile int* abort_flag;
  int* err;

  __device__ __forceinline__ RowsCta(const KParams& p, uint8_t* sm)
      : prm(p), smem(sm), sbase(smem_addr(sm)), bar0(sbase + C::OFF_BAR),
        abort_flag(reinterpret_cast<volatile int*>(sm + C::OFF_FLAGS)), err(p.hdr + kHdrError) {}
  __device__ __forceinline__ uint32_t bar(uint32_t i) const { return bar0 + 8 * i; }
  __device__ __forceinline__ bool wait(uint32_t b, uint32_t phase, int site, int detail) const {
    return wait_bounded(bar(b), phase & 1u, abort_flag, err, prm.timeout_ns, site, detail);
  }
  // Ring items, in the order in which they are done with: keys are NBUF tiles ahead of
  // the values (of three: K0 K1 K2 V0 K3 V1 ..).  The items of tile j of nt.
  static __device__ __forceinline__ uint32_t key_item(int j) { return j < C::NBUF ? j : 2 * j - C::NBUF + 1; }
  static __device__ __forceinline__ uint32_t value_item(int j, int nt) { return min(2 * j + C::NBUF, nt + j); }

  __device__ __forceinline__ uint32_t slot(uint32_t g) const { return g % C::NS; }
  __device__ __forceinline__ uint32_t phase(uint32_t g) const { return g / C::NS; }

  // Tile i of a unit uses buffer i % NBUF; bit b: the parity of the uses of buffer b so
  // far, which is that of the phase of its barriers' next use.
  static __device__ __forceinline__ uint32_t parity_after(uint32_t par, int nt) {  // a unit
#pragma unroll
    for (int b = 0; b < C::NBUF; ++b) par ^= (uint32_t)((nt - b + C::NBUF - 1) / C::NBUF & 1) << b;
    return par;
  }

  __device__ __forceinline__ RowsOdd* odd_of(uint32_t k) const {
    return reinterpret_cast<RowsOdd*>(smem + C::OFF_ODD) + k % C::UQ;
  }

  // Position of block vb of those that the sequence's rows can see.
  static __device__ __forceinline__ int block_pos(int sink_blocks, int skip, int vb) {
    return (vb + (vb < sink_blocks ? 0 : skip)) * C::BS;
  }

  // The unit of a plan, cut to the tokens that some row of it sees.
  __device__ __forceinline__ RowsUnit cut(const UnitPlan& P) const {
    RowsUnit U{P.s, P.p, P.kv, P.t0, P.t1, 0, P.np, P.nh, P.h0, P.L, P.span.sink_blocks, P.span.skip};
    if (!prm.masks) {
      const int l0 = P.h0 - P.kv * prm.G, first = P.L - prm.q_len;
      const int i0 = l0 / prm.Gu, i1 = (l0 + P.nh - 1) / prm.Gu;  // its first and last query token
      const int skip = U.skip * C::BS;
      // (The skipped blocks lie before every row's window, and before its end.)
      U.t1 = min(U.t1, first + i1 + 1 - skip);
      const int lo = first + i0 - prm.window + 1 - skip;
      if (U.t0 >= U.sink_blocks * C::BS && lo > U.t0) {
        // (Without skipped blocks, the first tokens lie where they are.)
        if (U.skip > 0 || U.t0 >= prm.sinks) U.t0 += (lo - U.t0) / C::TN * C::TN;
      }
    }
    U.nt = U.t1 > U.t0 ? (U.t1 - U.t0 + C::TN - 1) / C::TN : 0;
    return U;
  }

  // ---------------------------------------------------------------- producer warp
  // Item i of a unit of nt tiles (the inverse of the two above): true for values.
  static __device__ __forceinline__ bool item_tile(int i, int nt, int* j) {
    const int first = min(nt, C::NBUF), rest = nt - first, p = i - first;
    const bool value = p >= 0 && (p >= 2 * rest || !(p & 1));
    *j = p < 0 ? i : p >= 2 * rest ? p - rest : value ? p >> 1 : first + (p >> 1);
    return value;
  }
  // A lane's block of a group of GI ring items: NB lanes an item.
  struct Lane {
    int j;        // its tile
    bool value, in;  // of the values; there is such an item
    int blocks;   // blocks of the tile
    int id;       // its block, as the table has it
  };
  __device__ __forceinline__ Lane lane_item(const RowsUnit& U, int i, int b) const {
    Lane x{0, false, i < 2 * U.nt, 0, 0};
    if (x.in) {
      x.value = item_tile(i, U.nt, &x.j);
      x.blocks = min(C::NB, (U.t1 - U.t0 - x.j * C::TN + C::BS - 1) / C::BS);
      int j = U.t0 / C::BS + x.j * C::NB + b;
      j += j < U.sink_blocks ? 0 : U.skip;
      if (b < x.blocks) x.id = __ldg(prm.bt + (size_t)U.s * prm.MB + j);
    }
    return x;
  }

  __device__ __forceinline__ void producer(int P, const int* pref, const uint16_t* perm, int lane) {
    // Items issued together: as many as a warp has lanes for, up to half of the ring.
    // (One at a time took the producer 600 cycles an item, as long as its copy.)
    constexpr int NB = C::NB, GI = 32 / NB < C::PN / 2 ? 32 / NB : C::PN / 2;
    RowsUnit* info = reinterpret_cast<RowsUnit*>(smem + C::OFF_INFO);
    const uint64_t pol = l2_policy_evict_first();
    const int total = pref[prm.S] * prm.n_hg;
    const int li = lane / NB, lb = lane - li * NB;  // the lane's item of a group, and block of that
    fence_proxy_async_smem();  // the prologue's temporaries lay in the ring
    uint32_t g = 0, k = 0, hi = 0;  // ring items and units before this unit; items issued
    int u = blockIdx.x;
    bool ok = true;
    while (ok) {
      const bool have = u < total;
      RowsUnit U{};
      if (have) U = cut(plan_unit<C, kView>(prm, P, pref, perm, u));
      else U.s = -1;
      Lane next = lane_item(U, li, lb);  // (no items without a unit)
      // Publish it.
      const uint32_t us = k % C::UQ;
      ok = __shfl_sync(0xffffffffu, lane == 0 ? (int)wait(C::UEMPTY + us, k / C::UQ + 1, kRowsUnitSlot, (int)k) : 0, 0);
      if (!ok) break;
      odd_of(k)->clear(lane);  // (nothing looks at the unit before in this slot any more)
      __syncwarp();
      if (lane == 0) {
        info[us] = U;
        mbar_arrive(bar(C::UFULL + us));
      }
      ++k;
      if (!have) break;
      int claimed = 0;
      if (U.nt == 0 && lane == 0) claimed = atomicAdd(prm.hdr + kHdrWork, 1);
      for (int i0 = 0; i0 < 2 * U.nt && ok; i0 += GI) {
        const int cnt = min(GI, 2 * U.nt - i0);
        Lane x = next;
        x.in = x.in && li < GI;
        // (The next unit is taken while this one's last items are on their way.)
        if (i0 + cnt == 2 * U.nt && lane == 0) claimed = atomicAdd(prm.hdr + kHdrWork, 1);
        next = lane_item(U, i0 + GI + li, lb);
        const uint32_t gi = g + i0 + li, sl = gi % C::PN, ph = gi / C::PN, fb = bar(C::PFULL + sl);
        const size_t row = (size_t)check_block_id(prm, x.id) * prm.KH + U.kv;
        const uint32_t dst = sbase + C::OFF_PRING + sl * C::PSLOT + lb * C::BLK;
        bool done = !x.in;
        uint64_t t_start = 0;
        while (true) {
          if (!done && mbar_test_wait(bar(C::PEMPTY + sl), (ph & 1u) ^ 1u)) {
            if (lb == 0) mbar_arrive_expect_tx(fb, (uint32_t)x.blocks * C::BLK);
            if (lb < x.blocks) {
              if (!x.value || !C::kTma)
                bulk_copy_g2s(dst, static_cast<const uint8_t*>(x.value ? prm.vc : prm.kc) + row * C::BLK, C::BLK, fb, pol);
              else  // (x = 0: the 16-byte alignment rule holds)
                tma_load_3d(dst, &prm.tmv, 0, 0, (int)row, fb, pol);
            }
            done = true;
          }
          if (__all_sync(0xffffffffu, done)) break;
          int stop = 0;
          if (lane == 0) {
            const uint64_t now = global_timer_ns();
            if (t_start == 0) t_start = now;
            if (*abort_flag) {
              stop = 1;
            } else if ((long long)(now - t_start) > prm.timeout_ns) {
              record_timeout(abort_flag, err, kRowsRing, (int)g);
              stop = 1;
            } else {
              __nanosleep(32);
            }
          }
          if (__shfl_sync(0xffffffffu, stop, 0)) {
            // Aborted: this group's copies land before the warp leaves.
            ok = false;
            if (done && x.in) {
              const uint64_t t0 = global_timer_ns();
              while (!mbar_try_wait(fb, ph & 1u) && global_timer_ns() - t0 < 100000000ull) {
              }
            }
            __syncwarp();
            break;
          }
        }
        if (ok) hi = gi - li + cnt;
      }
      if (ok) g += 2 * U.nt;
      u = __shfl_sync(0xffffffffu, claimed, 0) + (int)gridDim.x;
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // Copies in flight land before the CTA ends, whatever the others did: the last one
    // of each slot.
    if (lane < C::PN && hi > (uint32_t)lane) {
      const uint32_t i = hi - 1 - (hi - 1 - lane) % C::PN;
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(bar(C::PFULL + lane), i / C::PN & 1u) && global_timer_ns() - t0 < 100000000ull) {
      }
    }
    __syncwarp();
  }

  // ---------------------------------------------------------------- product warps
  // A whole warp goes through the loops, so that descriptors are made in uniform
  // registers; one lane issues (descriptors made by one diverged lane cost 100 cycles
  // a product, more than the product).
  // Scores of ring slot `sl` into buffer b.
  __device__ __forceinline__ void issue_scores(uint32_t tmem, uint32_t sl, int b, uint32_t idesc) const {
    constexpr uint32_t STEP = C::kGroups ? 128u : C::BLK;    // from one instruction's tokens to the next one's
    constexpr uint32_t STRIDE = C::kGroups ? C::BLK : 128u;  // from eight tokens of an instruction to the next
    constexpr uint32_t LEAD = C::MS * 16u;                   // from a chunk of dims to the next
    const uint32_t ka = desc_lo(sbase + C::OFF_RING + sl * C::SLOT, LEAD);
    const uint32_t d = tmem + b * C::TN, q = tmem + C::Q_COL;
#pragma unroll
    for (int kk = 0; kk < C::D / 16; ++kk)
#pragma unroll
      for (int i = 0; i < C::NI; ++i)
        mma_ts(d + i * C::N, q + kk * 8, ka + (kk * 2 * LEAD + i * STEP) / 16, desc_hi(STRIDE, kSwizzleNone), idesc,
               kk > 0);
  }
  // O[o] (+)= weights of buffer b times the values in slot `sl`, `ks` k-steps.
  template <bool WHOLE>
  __device__ __forceinline__ void issue_values(uint32_t tmem, int o, uint32_t sl, int b, int ks, uint32_t idesc,
                                               bool add) const {
    constexpr int KB = C::MS == 8 ? 1 : C::MS / 16;  // k-steps of a block (of two blocks of eight tokens)
    constexpr uint32_t SW = C::MS == 8 ? kSwizzleNone : C::MS == 16 ? kSwizzle32 : C::MS == 32 ? kSwizzle64 : kSwizzle128;
    constexpr uint32_t HI = desc_hi(C::MS == 8 ? 128 : C::MS * 16, SW);
    const uint32_t va = desc_lo(sbase + C::OFF_RING + sl * C::SLOT, C::MS == 8 ? C::BLK : 16);
    const uint32_t d = tmem + C::O_COL + o * C::O_STEP, p = tmem + b * C::TN;
#pragma unroll
    for (int h = 0; h < (C::kBf16 ? 2 : 1); ++h) {
#pragma unroll
      for (int k = 0; k < C::TN / 16; ++k) {
        if (!WHOLE && k >= ks) break;
        constexpr uint32_t STEP = C::MS == 8 ? 2 * C::BLK : C::BLK;
        mma_ts(d, p + h * (C::TN / 2) + k * 8, va + ((k / KB) * STEP + (k % KB) * 32) / 16, HI, idesc,
               add || h > 0 || k > 0);
      }
    }
  }
  __device__ __forceinline__ bool all(uint32_t b, uint32_t ph, int site, int detail) const {
    return __all_sync(0xffffffffu, wait(b, ph, site, detail)) != 0;
  }
  // What the warp has issued completes before tensor memory is freed.
  __device__ __forceinline__ void drain(uint32_t at) const {
    if (elect_one()) mma_commit(at);
    __syncwarp();
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(at, 0) && global_timer_ns() - t0 < 100000000ull) {
    }
    __syncwarp();
  }
  // One warp issues the scores' products ...
  __device__ __forceinline__ void score_products(uint32_t tmem, int lane) {
    const RowsUnit* info = reinterpret_cast<const RowsUnit*>(smem + C::OFF_INFO);
    const uint32_t id_s = f16_idesc(C::kBf16, C::N);
    uint32_t g = 0, par = 0;  // ring items before this unit; as in the softmax
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      if (!all(C::UFULL + k % C::UQ, k / C::UQ, kRowsUnit, (int)k)) break;
      const RowsUnit* up = info + k % C::UQ;
      // (Shuffles tell the compiler that these are the same in every lane.)
      const int us = __shfl_sync(0xffffffffu, up->s, 0), nt = __shfl_sync(0xffffffffu, up->nt, 0);
      if (lane == 0) mbar_arrive(bar(C::UEMPTY + k % C::UQ));
      if (us < 0) break;
      if (!all(C::QREADY, k, kRowsQ, (int)k)) break;
      // (The last unit's joining used the buffers, and its products are complete; and
      // with this wait neither side is ever more than a unit ahead, so that a parity
      // tells the phases apart.)
      if (!all(C::XFREE, k + 1, kRowsX, (int)k)) break;
      tc_fence_after();
      if (nt == 0) {
        if (elect_one()) mma_commit(bar(C::QFREE));
        __syncwarp();
      }
      for (int i = 0, b = 0; i < nt; ++i, b = b + 1 < C::NBUF ? b + 1 : 0) {
        const uint32_t it = g + key_item(i);
        ok = all(C::FULL + slot(it), phase(it), kRowsFull, (int)it);
        if (ok && i >= C::NBUF) {  // the buffer's weights have been used
          ok = all(C::PVDONE + b, (par >> b) + (i / C::NBUF - 1), kRowsPv, i);
          tc_fence_after();
        }
        if (!ok) break;
        if (elect_one()) {
          issue_scores(tmem, slot(it), b, id_s);
          mma_commit(bar(C::SFULL + b));
          mma_commit(bar(C::EMPTY + slot(it)));
          if (i + 1 == nt) mma_commit(bar(C::QFREE));  // Q may be replaced
        }
        __syncwarp();
      }
      par = parity_after(par, nt);
      g += 2 * nt;
    }
    drain(sbase + C::OFF_FLAGS + 32);
  }
  // ... and one those with the values.  (One warp that did both, wait for wait, took
  // 1800 cycles a tile, of which the products are 530.)
  __device__ __forceinline__ void value_products(uint32_t tmem, int lane) {
    const RowsUnit* info = reinterpret_cast<const RowsUnit*>(smem + C::OFF_INFO);
    const uint32_t id_o = f16_idesc(C::kBf16, C::D);
    uint32_t g = 0, par = 0;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      if (!all(C::UFULL + k % C::UQ, k / C::UQ, kRowsUnit, (int)k)) break;
      const RowsUnit* up = info + k % C::UQ;
      const int us = __shfl_sync(0xffffffffu, up->s, 0), nt = __shfl_sync(0xffffffffu, up->nt, 0);
      const int tokens = __shfl_sync(0xffffffffu, up->t1 - up->t0, 0);
      if (lane == 0) mbar_arrive(bar(C::UEMPTY + k % C::UQ));
      if (us < 0) break;
      if (!all(C::OFREE, k + 1, kRowsOFree, (int)k)) break;  // the last unit's O is read
      for (int i = 0, b = 0; i < nt; ++i, b = b + 1 < C::NBUF ? b + 1 : 0) {
        const uint32_t it = g + value_item(i, nt);
        ok = all(C::FULL + slot(it), phase(it), kRowsFull, (int)it);
        if (ok) ok = all(C::PREADY + b, par >> b, kRowsP, i);
        if (!ok) break;
        par ^= 1u << b;
        tc_fence_after();
        const int o = C::NP == 2 ? i & 1 : 0;
        const int left = tokens - i * C::TN, ks = left >= C::TN ? C::TN / 16 : (left + 15) / 16;
        if (elect_one()) {
          if (ks == C::TN / 16) issue_values<true>(tmem, o, slot(it), b, ks, id_o, i >= C::NP);
          else issue_values<false>(tmem, o, slot(it), b, ks, id_o, i >= C::NP);
          mma_commit(bar(C::PVDONE + b));
          mma_commit(bar(C::EMPTY + slot(it)));
        }
        __syncwarp();
      }
      g += 2 * nt;
    }
    drain(sbase + C::OFF_FLAGS + 40);
  }

  // ---------------------------------------------------------------- Q warps
  // The next unit's rows, as [D/8][128 rows] 16-byte pieces in shared memory; rows past
  // the unit's (up to whole warps): zeros.  Four lanes a row: 64 bytes of it an
  // instruction.
  __device__ __forceinline__ void bring_rows(int tid, int lane) {
    using T = typename C::T;
    const RowsUnit* info = reinterpret_cast<const RowsUnit*>(smem + C::OFF_INFO);
    for (uint32_t k = 0;; ++k) {
      const bool okw = wait(C::UFULL + k % C::UQ, k / C::UQ, kRowsUnit, (int)k);
      if (!__all_sync(0xffffffffu, okw)) break;
      const RowsUnit U = info[k % C::UQ];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::UEMPTY + k % C::UQ));
      if (!__all_sync(0xffffffffu, wait(C::QTAKEN, k + 1, kRowsQFree, (int)k))) break;
      if (U.s < 0) {  // (the softmax looks for the next unit's Q before it knows that there is none)
        mbar_arrive(bar(C::QSTAGED));
        break;
      }
      const int rows = (U.nh + 31) / 32 * 32;
      for (int row = tid >> 2; row < rows; row += C::LOADERS / 4) {
        const bool in = row < U.nh;
        const T* q = static_cast<const T*>(prm.q) + (in ? out_row<kView>(prm, U.s, U.h0 + row) : 0) * C::D;
        const uint32_t dst = sbase + row * 16;
#pragma unroll
        for (int c0 = 0; c0 < C::D / 8; c0 += 4) {
          const int c = c0 + (tid & 3);
          if (c < C::D / 8)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + c * 2048), "l"(q + c * 8),
                         "r"(in ? 16 : 0)
                         : "memory");
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      mbar_arrive(bar(C::QSTAGED));
    }
  }

  // ---------------------------------------------------------------- softmax warpgroups
  // The tokens that a row sees of 64 at positions p .. p + 63, `n` of them there.
  static __device__ __forceinline__ uint64_t first_bits(int n) { return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1ull; }
  __device__ __forceinline__ uint64_t seen64(const RowView& v, int p, int n) const {
    uint64_t m = first_bits(min(v.hi - p, n));
    m &= ~first_bits(v.lo - p) | first_bits(prm.sinks - p);
    if (v.bits && p + 63 >= v.base) {
      // Node j of the row's mask is the token at base + j.
      const int off = p - v.base, i = max(off, 0) >> 5, sh = max(off, 0) & 31;
      uint32_t w[3];
#pragma unroll
      for (int q = 0; q < 3; ++q) w[q] = i + q < prm.words ? __ldg(v.bits + i + q) : 0u;
      const uint64_t b = (uint64_t)__funnelshift_r(w[1], w[2], sh) << 32 | __funnelshift_r(w[0], w[1], sh);
      m &= off >= 0 ? b : b << -off | first_bits(-off);
    }
    return m;
  }

  // Positions [lo, hi) that every row of a unit sees (padding apart).
  struct Full {
    int lo, hi;
  };
  __device__ __forceinline__ Full full_of(int L, int kv, int h0, int nh) const {
    const int first = L - prm.q_len, l0 = h0 - kv * prm.G;
    const int i0 = l0 / prm.Gu, i1 = (l0 + nh - 1) / prm.Gu;
    return Full{prm.window > 0 ? (prm.masks ? L - prm.window : first + i1 - prm.window + 1) : 0,
                prm.masks ? first : first + i0 + 1};
  }
  // A tile of the unit's work, `left` tokens from its start to the unit's end: where it
  // lies, and whether some row of the unit does not see the whole of it.
  struct Tile {
    int p0;        // the position of its first token
    int n;         // its tokens in front of skipped blocks; the others are skip blocks further on
    bool partial;
  };
  __device__ __forceinline__ Tile tile_at(int tile, int left, int sink_blocks, int skip, const Full& full) const {
    const int vb0 = tile / C::BS, p0 = block_pos(sink_blocks, skip, vb0);
    const int p1 = block_pos(sink_blocks, skip, vb0 + (min(left, C::TN) - 1) / C::BS) + C::BS - 1;
    const bool jump = skip > 0 && vb0 < sink_blocks && vb0 + C::NB > sink_blocks;
    return Tile{p0, jump ? (sink_blocks - vb0) * C::BS : C::TN,
                left < C::TN || jump || p1 >= full.hi || (p0 < full.lo && p1 >= prm.sinks)};
  }
  // The tokens of it that a row sees.
  __device__ __forceinline__ uint64_t tile_seen(const RowView& v, const Tile& t, int left, int skip) const {
    uint64_t m = seen64(v, t.p0, left);
    if (t.n < C::TN) m = (m & first_bits(t.n)) | (seen64(v, t.p0 + skip * C::BS, left) & ~first_bits(t.n));
    return m;
  }

  // Byte offset of tokens 8c .. 8c + 7 of dim d in a staged value block.
  static __device__ __forceinline__ uint32_t value_chunk(int d, int c) {
    constexpr uint32_t ROW = C::MS * 2;
    if constexpr (C::MS >= 16) return d * ROW + ((c ^ ((d * ROW >> 7) & (ROW / 16 - 1))) << 4);
    else return d * ROW + c * 16;
  }

  // A tile's values: those past the unit's end, and of the others those that are
  // not finite, are cleared.  128 threads.  True if there was one of the latter.
  __device__ __forceinline__ bool clear_values(uint32_t sl, int left, int tid) const {
    constexpr uint32_t kExp = C::kBf16 ? 0x7f80u : 0x7c00u;
    uint8_t* v = smem + C::OFF_RING + sl * C::SLOT;
    const int groups = min(C::TN / 8, (left + 15) / 16 * 2);
    // (Not finite: the number without its sign is kExp at least, so that adding `up` sets
    // the sign's bit.)
    constexpr uint32_t up = C::kBf16 ? 0x00800080u : 0x04000400u;
    bool found = false;
#pragma unroll 4
    for (int i = tid; i < C::D * groups; i += 128) {
      const int gr = i / C::D, d = i - gr * C::D, b = gr / C::NG, c = gr % C::NG, n = left - gr * 8;
      uint4* at = reinterpret_cast<uint4*>(v + b * C::BLK + value_chunk(d, c));
      const uint4 x = *at;
      uint32_t w[4] = {x.x, x.y, x.z, x.w};
      uint32_t any = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) any |= (w[q] & 0x7fff7fffu) + up;
      if (!(any & 0x80008000u) && n >= 8) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool past = 2 * q + h >= n, odd = ((w[q] >> (16 * h)) & kExp) == kExp;
          if (past || odd) w[q] &= h ? 0xffffu : 0xffff0000u;
          found |= odd && !past;
        }
      *at = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return found;
  }

  // Eight E4M3 codes as fp16 (exact).
  static __device__ __forceinline__ uint4 widen8(uint32_t lo, uint32_t hi) {
    uint4 x;
    asm("{\n\t.reg .b16 a, b, c, d;\n\t"
        "mov.b32 {a, b}, %4;\n\tmov.b32 {c, d}, %5;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t"
        "cvt.rn.f16x2.e4m3x2 %2, c;\n\tcvt.rn.f16x2.e4m3x2 %3, d;\n\t}"
        : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
        : "r"(lo), "r"(hi));
    return x;
  }
  // Value codes of `n` tokens and anything behind them: what is past them, and NaN codes
  // (0x7f, 0xff; `found`), become zeros.
  static __device__ __forceinline__ uint32_t plain_codes(uint32_t w, int n, bool& found) {
    if (n < 4) w = n <= 0 ? 0u : w & (0xffffffffu >> (32 - 8 * n));
    const uint32_t nan = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
    if (nan) {
      found = true;
      w &= ~((nan >> 7) * 0xffu);
    }
    return w;
  }
  // Tile j, whose codes are in ring slot rs, has NaN codes: it is noted, or if every row
  // sees it, the dims that have one.
  __device__ __noinline__ void note_codes(uint32_t k, uint32_t rs, int j, int lane) const {
    const RowsUnit U = reinterpret_cast<const RowsUnit*>(smem + C::OFF_INFO)[k % C::UQ];
    RowsOdd* odd = odd_of(k);
    const int tile = U.t0 + j * C::TN;
    if (tile_at(tile, U.t1 - tile, U.sink_blocks, U.skip, full_of(U.L, U.kv, U.h0, U.nh)).partial) {
      if (lane == 0) odd->add_tile(j);
      return;
    }
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(smem + C::OFF_CODES + rs * C::RSLOT);
    for (int x = lane; x < C::TN * C::D / 4; x += 32) {  // [block][D][BS]
      const uint32_t w = codes[x];
      if (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) odd->add_dim(x * 4 / C::BS % C::D);
    }
  }
  // 8-bit caches: the ring's codes widened to fp16, into the layouts of a block of 64
  // tokens; each of the CW warps takes every CW-th ring item, so that several are on
  // their way and a warp's waits are another warp's work.
  __device__ __forceinline__ void widen(int cw, int lane) {
    const RowsUnit* info = reinterpret_cast<const RowsUnit*>(smem + C::OFF_INFO);
    constexpr int BS = C::BS, D = C::D;
    uint32_t g = 0;
    for (uint32_t k = 0;; ++k) {
      if (!__all_sync(0xffffffffu, wait(C::UFULL + k % C::UQ, k / C::UQ, kRowsUnit, (int)k))) return;
      const RowsUnit* up = info + k % C::UQ;
      const int us = up->s, nt = up->nt, tokens = up->t1 - up->t0;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::UEMPTY + k % C::UQ));
      if (us < 0) return;
      for (int i = (int)((cw + C::CW - g % C::CW) % C::CW); i < 2 * nt; i += C::CW) {
        const uint32_t it = g + i, rs = it % C::NR, sl = slot(it);
        int j;
        const bool value = item_tile(i, nt, &j);
        const int left = tokens - j * C::TN;
        bool found = false;
        bool ok = wait(C::RFULL + rs, it / C::NR, kRowsCodes, (int)it);
        if (ok) ok = wait(C::EMPTY + sl, phase(it) + 1, kRowsRing, (int)it);
        if (!__all_sync(0xffffffffu, ok)) return;
        const uint4* from = reinterpret_cast<const uint4*>(smem + C::OFF_CODES + rs * C::RSLOT);
        uint8_t* to = smem + C::OFF_RING + sl * C::SLOT;
        constexpr int PIECES = C::TN * D / 16;
        if (!value) {
          // [block][D/16][BS][16]: a token's 16 dims are two pieces of the tile's [D/8][64][8].
#pragma unroll 2
          for (int x = lane; x < PIECES; x += 32) {
            const int t = x % BS, c = x / BS % (D / 16), b = x / (BS * (D / 16));
            const uint4 w = from[x];
            uint8_t* at = to + c * 2048 + (b * BS + t) * 16;
            *reinterpret_cast<uint4*>(at) = widen8(w.x, w.y);
            *reinterpret_cast<uint4*>(at + 1024) = widen8(w.z, w.w);
          }
        } else {
          // [block][D][BS]: 16 tokens of a dim (blocks of eight: eight tokens of two dims).
#pragma unroll 2
          for (int x = lane; x < PIECES; x += 32) {
            constexpr int RP = BS >= 16 ? BS / 16 : 1;  // pieces of a dim's row
            const int b = x / (BS * D / 16), y = x % (BS * D / 16);
            const int d = BS >= 16 ? y / RP : 2 * y, t = b * BS + (BS >= 16 ? y % RP * 16 : 0);
            uint4 w = from[x];
            constexpr uint32_t m7 = 0x7f7f7f7fu, one = 0x01010101u;
            const uint32_t nan = ((w.x & m7) + one) | ((w.y & m7) + one) | ((w.z & m7) + one) | ((w.w & m7) + one);
            if (left < C::TN || (nan & 0x80808080u)) {
              const int n = left - t, n2 = BS >= 16 ? n - 8 : n;
              w.x = plain_codes(w.x, n, found);
              w.y = plain_codes(w.y, n - 4, found);
              w.z = plain_codes(w.z, n2, found);
              w.w = plain_codes(w.w, n2 - 4, found);
            }
            *reinterpret_cast<uint4*>(to + value_chunk(d, t / 8)) = widen8(w.x, w.y);
            *reinterpret_cast<uint4*>(to + (BS >= 16 ? value_chunk(d, t / 8 + 1) : value_chunk(d + 1, t / 8))) =
                widen8(w.z, w.w);
          }
          if (__any_sync(0xffffffffu, found)) note_codes(k, rs, j, lane);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(C::FULL + sl));
          mbar_arrive(bar(C::REMPTY + rs));
        }
      }
      g += 2 * nt;
    }
  }

  // Values that are not finite (rare; the cache itself is read): dims [d0, d1) of a
  // row that has been written get those of the tokens it sees added.  `at`: the row's
  // output or state.  (Only the noted tiles: by the latency of its loads one takes as long
  // as a hundred tiles of the unit, which may have thousands.)
  template <typename E>
  __device__ __noinline__ void add_odd(uint32_t k, int qi, int d0, int d1, E* at) const {
    using CT = typename std::conditional<C::kFp8, uint8_t, typename C::T>::type;
    constexpr int PER = 8 / (int)sizeof(CT), BS = C::BS;  // elements of 8 bytes
    constexpr uint32_t kExp = C::kBf16 ? 0x7f80u : 0x7c00u;
    const RowsUnit U = reinterpret_cast<const RowsUnit*>(smem + C::OFF_INFO)[k % C::UQ];
    const RowView v = row_view_of(prm, U.s, U.L, qi);
    const Full full = full_of(U.L, U.kv, U.h0, U.nh);
    const int t0 = U.t0, t1 = U.t1;
    const volatile RowsOdd& o = *odd_of(k);
    const bool all = o.all != 0;
    const int tiles = all ? (t1 - t0 + C::TN - 1) / C::TN : RowsOdd::kTiles;
    for (int q = 0; q < tiles; ++q) {
      const int i = all ? q : o.tile[q] - 1;
      if (i < 0) continue;
      const int tile = t0 + i * C::TN, left = t1 - tile;
      const uint64_t m = tile_seen(v, tile_at(tile, left, U.sink_blocks, U.skip, full), left, U.skip);
      for (int b = 0; b < C::NB; ++b) {
        const uint64_t mb = m >> (b * BS) & first_bits(BS);
        if (mb == 0) continue;
        int id = prm.bt[(size_t)U.s * prm.MB + block_pos(U.sink_blocks, U.skip, tile / BS + b) / BS];
        if ((unsigned)id >= (unsigned)prm.num_blocks) id = 0;
        const CT* rows = static_cast<const CT*>(prm.vc) + ((size_t)id * prm.KH + U.kv) * C::D * BS;
        // (A call whose registers are few: with more of it unrolled the kernel spilled.)
#pragma unroll 1
        for (int d = d0; d < d1; ++d) {
          float sum = 0.f;
          bool any = false;
#pragma unroll 4
          for (int w = 0; w < BS / PER; ++w) {
            const uint2 x = __ldg(reinterpret_cast<const uint2*>(rows + (size_t)d * BS) + w);
#pragma unroll
            for (int e = 0; e < PER; ++e) {
              const uint32_t word = e * (int)sizeof(CT) < 4 ? x.x : x.y;
              bool is;
              float x1 = NAN;
              if constexpr (C::kFp8) {
                is = (word >> (8 * (e & 3)) & 0x7fu) == 0x7fu;
              } else {
                const uint32_t h = word >> (16 * (e & 1)) & 0xffffu;
                is = (h & kExp) == kExp;
                if (h == kExp) x1 = INFINITY;
                if (h == (kExp | 0x8000u)) x1 = -INFINITY;
              }
              if (is && (mb >> (w * PER + e) & 1u)) {
                sum += x1;
                any = true;
              }
            }
          }
          if (any) at[d] = (E)((float)at[d] + sum);
        }
      }
    }
    if constexpr (C::kFp8) {
      for (int d = d0; d < d1; ++d)
        if (o.dims[d >> 5] >> (d & 31) & 1u) at[d] = (E)NAN;
    }
  }

  // The staged Q of unit k into tensor memory (a row a thread, the pipelines' warpgroups
  // in turn), once the products with the one before are complete.  A negative scale's sign goes
  // with it: the softmax works with one that is not negative.
  __device__ __forceinline__ bool take_rows(uint32_t tmem, uint32_t lanes, int wg, int tid, uint32_t k, float& factor) const {
    bool ok = wait(C::QSTAGED, k, kRowsQ, (int)k);
    if (ok) ok = wait(C::QFREE, k + 1, kRowsQFree, (int)k);
    if (!__all_sync(0xffffffffu, ok)) return false;
    tc_fence_after();
    __syncwarp();
    const uint32_t flip = prm.scale_log2 < 0.f ? 0x80008000u : 0u;
    constexpr int W = C::D / 2;  // columns
    // (8-bit caches) bf16 rows in fp16: times the power of two that brings the largest to
    // 2^14 .. 2^15 (rows that are not finite: as they are), which the scores' factor undoes.
    float up = 1.f;
    if constexpr (C::kQScale) {
      uint32_t m = 0;
#pragma unroll
      for (int c = 0; c < C::D / 8; ++c) {
        const uint4 x = *reinterpret_cast<const uint4*>(smem + c * 2048 + tid * 16);
        const uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, max(e[i] & 0x7fffu, e[i] >> 16 & 0x7fffu));
      }
      const int ex = (int)(m >> 7);
      up = __uint_as_float((uint32_t)(ex == 255 ? 127 : min(268 - ex, 254)) << 23);
      factor = 1.f / up;
    }
#pragma unroll
    for (int w0 = 0; w0 < W; w0 += 16) {
      if (C::NP == 2 && (w0 / 16 & 1) != wg) continue;
      uint32_t w[16];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (w0 + 4 * c >= W) break;
        const uint4 x = *reinterpret_cast<const uint4*>(smem + (w0 / 4 + c) * 2048 + tid * 16);
        const uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t v = e[i];
          if constexpr (C::kQScale)
            v = F16Traits<__half>::pack(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xffff0000u) * up);
          w[4 * c + i] = v ^ flip;
        }
      }
      if (w0 + 16 <= W) tmem_st16(tmem + lanes + C::Q_COL + w0, w);
      else tmem_st8(tmem + lanes + C::Q_COL + w0, w);
    }
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(bar(C::QTAKEN));
    mbar_arrive(bar(C::QREADY));
    return true;
  }

  __device__ __forceinline__ void softmax(uint32_t tmem, int wg, int tid) {
    using T = typename C::T;
    using MT = typename C::MT;
    constexpr int TN = C::TN, NB = C::NB, NG = C::NG, D = C::D;
    const RowsUnit* info = reinterpret_cast<const RowsUnit*>(smem + C::OFF_INFO);
    const int lane = tid & 31;
    const uint32_t lanes = (uint32_t)(tid & ~31) << 16;  // this warp's lanes of tensor memory
    // (Not zero: a masked score, -inf, times it is -inf.)
    const float sl2_all = fmaxf(fabsf(prm.scale_log2), 1.17549435e-38f);
    const uint64_t pol_keep = l2_policy_evict_last();
    uint32_t g = 0, k = 0;  // ring items and units before this unit
    uint32_t par = 0;       // of the buffers before the unit
    float factor = 1.f;  // (kQScale) of the row's scores
    if (!take_rows(tmem, lanes, wg, tid, 0, factor)) return;
    // (The unit's description stays in its slot while it is worked on, and what a row
    // sees is worked out where a tile is partly seen and at the end: registers hold
    // the row's scores.)
    while (true) {
      const bool okw = wait(C::UFULL + k % C::UQ, k / C::UQ, kRowsUnit, (int)k);
      if (!__all_sync(0xffffffffu, okw)) break;
      const volatile RowsUnit& U = info[k % C::UQ];
      if (U.s < 0) break;
      const int nh = U.nh, nt = U.nt;
      const int row = tid;  // the thread's row of the unit
      const bool mine = row < nh;
      const int qi = mine ? (U.h0 - U.kv * prm.G + row) / prm.Gu : -1;  // its query token
      const auto view = [&]() { return qi >= 0 ? row_view_of(prm, U.s, U.L, qi) : RowView{0, 0, 0, nullptr}; };
      const bool warp_rows = (row & ~31) < nh;
      const Full full = full_of(U.L, U.kv, U.h0, nh);
      float mref = -INFINITY, l = 0.f, sl2 = sl2_all;
      if constexpr (C::kQScale) sl2 = fmaxf(sl2 * factor, 1.17549435e-38f);
      const int t0 = U.t0, t1 = U.t1, sink_blocks = U.sink_blocks, skip = U.skip;
      bool ok = true;
      for (int i = C::NP == 2 ? wg : 0; i < nt && ok; i += C::NP) {
        const int b = i % C::NBUF;
        const uint32_t use = (par >> b) + i / C::NBUF;  // (its low bit counts)
        const uint32_t sc = tmem + lanes + b * TN;
        const int tile = t0 + i * TN, left = t1 - tile;
        ok = __all_sync(0xffffffffu, wait(C::SFULL + b, use, kRowsS, i));
        if (!ok) break;
        tc_fence_after();
        const Tile place = tile_at(tile, left, sink_blocks, skip, full);
        const bool partial = place.partial;
        if (!C::kFp8 && partial) {
          // (Values: before the weights of the tile are announced.)
          const uint32_t it = g + value_item(i, nt);
          ok = __all_sync(0xffffffffu, wait(C::FULL + slot(it), phase(it), kRowsFull, (int)it));
          if (!ok) break;
          if (clear_values(slot(it), left, tid)) odd_of(k)->add_tile(i);
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (!warp_rows) {  // a warp without rows only keeps the count
          mbar_arrive(bar(C::PREADY + b));
          continue;
        }
        float s[TN];
        __syncwarp();
        tmem_get64(sc, sc + 32, s);
        if (partial) {
          const uint64_t m = tile_seen(view(), place, left, skip);
          const uint32_t mm[2] = {(uint32_t)m, (uint32_t)(m >> 32)};
#pragma unroll
          for (int t = 0; t < TN; ++t)
            if (!(mm[t / 32] >> (t % 32) & 1u)) s[C::column(t / C::BS, t % C::BS / 8, t % 8)] = -INFINITY;
          __syncwarp();
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < TN; ++c) m4[c & 3] = fmaxf(m4[c & 3], s[c]);
        float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sl2;
        const bool first = i < C::NP;
        if (mx > mref + 8.f || (mref == -INFINITY && mx > -INFINITY)) {
          const float alpha = exp2_approx(mref - mx);
          l *= alpha;
          const bool had = mref > -INFINITY;
          mref = mx;
          mx = had ? alpha : 1.f;
        } else {
          mx = 1.f;
        }
        __syncwarp();
        if (!first && __any_sync(0xffffffffu, mx != 1.f)) {
          // O by the rows' factors, once the last product into it is complete.  (Each
          // buffer's products have a barrier: this tile's scores say that all but those of
          // the NBUF - 1 tiles before are complete, so neither is two phases off.)
          const int ip = i - C::NP, pb = ip % C::NBUF;
          ok = __all_sync(0xffffffffu, wait(C::PVDONE + pb, (par >> pb) + ip / C::NBUF, kRowsPv, i));
          if (!ok) break;
          tc_fence_after();
          const uint32_t oc = tmem + lanes + C::O_COL + (C::NP == 2 ? wg : 0) * C::O_STEP;
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            float o[16];
            tmem_get16(oc + c, o);
            uint32_t w[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) w[q] = __float_as_uint(o[q] * mx);
            tmem_st16(oc + c, w);
          }
        }
        const float ref = mref == -INFINITY ? 0.f : mref;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < TN; ++c) {
          s[c] = exp2_approx(fmaf(s[c], sl2, -ref));
          sum[c & 3] += s[c];
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        // Weights, in token order: word w holds tokens 2w, 2w + 1 of the tile.  bf16: the
        // weight cut to its first 8 bits, and what that leaves (exact in fp32) rounded.
#pragma unroll
        for (int w0 = 0; w0 < TN / 2; w0 += 16) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const int t = 2 * (w0 + q), e = C::column(t / C::BS, t % C::BS / 8, t % 8);
            if constexpr (C::kBf16) {
              const uint32_t x = __float_as_uint(s[e]), y = __float_as_uint(s[e + 1]);
              hi[q] = __byte_perm(x, y, 0x7632);
              lo[q] = F16Traits<MT>::pack(s[e] - __uint_as_float(x & 0xffff0000u), s[e + 1] - __uint_as_float(y & 0xffff0000u));
            } else {
              hi[q] = F16Traits<MT>::pack(s[e], s[e + 1]);
            }
          }
          tmem_st16(sc + w0, hi);
          if constexpr (C::kBf16) tmem_st16(sc + TN / 2 + w0, lo);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(C::PREADY + b));
      }
      if (!ok) break;
      // ---- the end of the unit: the next one's Q, then join the pipelines' states (one row
      // a thread) and write.
      if (!take_rows(tmem, lanes, wg, tid, k + 1, factor)) break;
      const uint32_t ob = tmem + lanes + C::O_COL;
      const bool live = view().hi > 0;
      // The last tile of each pipeline (-1: none), whose buffers are free when their
      // products are complete.
      const int last = C::NP == 1 ? nt - 1 : nt - 1 - ((nt - 1 - wg) & 1);
      const int other = C::NP == 1 ? 0 : nt - 1 - ((nt - 1 - (1 - wg)) & 1);
      if (last >= 0) {
        ok = __all_sync(0xffffffffu, wait(C::PVDONE + last % C::NBUF, (par >> last % C::NBUF) + last / C::NBUF, kRowsPv, -1));
        if (!ok) break;
        tc_fence_after();
      }
      // (mref, l) of either warpgroup's thread of a row, by those buffers.
      if constexpr (C::NP == 2) {
        __syncwarp();
        tmem_st2(tmem + lanes + (last >= 0 ? last % C::NBUF : wg) * TN, mref, l);
        tmem_wait_st();
        tc_fence_before();
      }
      if (nt == 0) {  // (nothing of this unit came from the product warp)
        ok = __all_sync(0xffffffffu, wait(C::QFREE, k, kRowsQFree, (int)k));
        if (!ok) break;
      }
      mbar_arrive(bar(C::XBAR));
      ok = __all_sync(0xffffffffu, wait(C::XBAR, k, kRowsX, (int)k));
      if (!ok) break;
      tc_fence_after();
      const bool odd = *const_cast<const volatile int*>(&odd_of(k)->any) != 0;
      float f0 = 1.f, f1 = 0.f;
      bool has0 = nt > 0, has1 = false;  // pipelines with something in O
      int d_lo = 0, d_hi = D;
      if constexpr (C::NP == 2) {
        // Both warpgroups have every row: each writes half of its dims.
        float ml[2];
        tmem_get2(tmem + lanes + (other >= 0 ? other % C::NBUF : 1 - wg) * TN, ml);
        const float m2 = ml[0], l2 = ml[1];
        tc_fence_before();
        mbar_arrive(bar(C::XFREE));
        const float ma = wg ? m2 : mref, la = wg ? l2 : l, mb = wg ? mref : m2, lb = wg ? l : l2;
        const float M = fmaxf(ma, mb), Ms = M == -INFINITY ? 0.f : M;
        f0 = exp2_approx(ma - Ms);
        f1 = exp2_approx(mb - Ms);
        l = f0 * la + f1 * lb;
        mref = M;
        has1 = nt > 1;
        constexpr int HALF = D / 32 * 16;
        d_lo = wg ? HALF : 0;
        d_hi = wg ? D : HALF;
      } else {
        mbar_arrive(bar(C::XFREE));
      }
      if (warp_rows) {
        const bool some = live && l != 0.f;
        const float inv = some ? (C::kFp8 ? prm.v_scale / l : 1.f / l) : 0.f;
        f0 *= inv;
        f1 *= inv;
        const bool single = U.np == 1;
        const size_t sh0 = (size_t)U.s * prm.H + U.h0, sh = sh0 + row;
        const int orow = mine ? (int)out_row<kView>(prm, U.s, U.h0 + row) : 0;  // (below 2^25: 256 sequences)
        uint8_t* to = single ? static_cast<uint8_t*>(prm.out) + (size_t)orow * D * sizeof(T)
                             : reinterpret_cast<uint8_t*>(prm.ws_o + ((sh0 + row) * prm.Pmax + U.p) * D);
        const bool wide = (reinterpret_cast<uintptr_t>(single ? prm.out : static_cast<void*>(prm.ws_o)) & 31) == 0;
        // (Of a pipeline without a tile, O holds anything: it is read, and not used.)
        constexpr int NCH = (D / 2 % 32 == 0 && C::NP == 2) || C::NP == 1 ? 2 : 1;  // pieces of 16 dims at a time
#pragma unroll 1
        for (int c0 = d_lo; c0 < d_hi; c0 += NCH * 16) {
          float o[NCH][16];
          __syncwarp();  // (rows that are not the unit's have left lanes behind)
          if constexpr (C::NP == 2 && NCH == 2) {
            float ab[64];
            tmem_get64(ob + c0, ob + C::O_STEP + c0, ab);
#pragma unroll
            for (int q = 0; q < 32; ++q) o[q / 16][q % 16] = ab[q] * f0;
            if (has1) {
#pragma unroll
              for (int q = 0; q < 32; ++q) o[q / 16][q % 16] = fmaf(ab[32 + q], f1, o[q / 16][q % 16]);
            }
          } else {
            float ab[32];
            tmem_get32(ob + c0, ob + (C::NP == 2 ? C::O_STEP : 16) + c0, ab);
#pragma unroll
            for (int q = 0; q < NCH * 16; ++q) o[q / 16][q % 16] = ab[q] * f0;
            if (C::NP == 2 && has1) {
#pragma unroll
              for (int q = 0; q < 16; ++q) o[0][q] = fmaf(ab[(16 + q) % 32], f1, o[0][q]);
            }
          }
          if (!some || !has0) {
#pragma unroll
            for (int q = 0; q < NCH * 16; ++q) o[q / 16][q % 16] = 0.f;
          }
          if (mine) {
            // (32 bytes of its row a lane: whole sectors.)
#pragma unroll
            for (int h = 0; h < NCH; ++h) {
              if (single) {
                uint32_t w[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) w[q] = F16Traits<T>::pack(o[h][2 * q], o[h][2 * q + 1]);
                st_32b(to + (c0 + 16 * h) * sizeof(T), w, wide);
              } else {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  uint32_t w[8];
#pragma unroll
                  for (int q = 0; q < 8; ++q) w[q] = __float_as_uint(o[h][8 * x + q]);
                  st_32b(to + (c0 + 16 * h + 8 * x) * 4, w, wide);
                }
              }
            }
          }
        }
        if (odd) {
          __syncwarp();
          if (mine && some) {
            if (single)
              add_odd(k, qi, d_lo, d_hi, static_cast<T*>(prm.out) + (size_t)orow * D);
            else
              add_odd(k, qi, d_lo, d_hi, prm.ws_o + (sh * prm.Pmax + U.p) * D);
          }
          __syncwarp();
        }
        if (mine && d_lo == 0) {
          const float mn = some ? mref * kLn2 : -INFINITY;
          if (!single) {
            st_f32_policy(prm.ws_m + sh * prm.Pmax + U.p, mn, pol_keep);
            st_f32_policy(prm.ws_l + sh * prm.Pmax + U.p, some ? l : 0.f, pol_keep);
          } else if (prm.lse) {
            prm.lse[orow] = some ? mn + logf(l) : -INFINITY;
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      mbar_arrive(bar(C::OFREE));
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::UEMPTY + k % C::UQ));
      par = parity_after(par, nt);
      g += 2 * nt;
      ++k;
    }
  }
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) pa_rows_kernel(const __grid_constant__ KParams prm) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  RowsCta<C> cta(prm, smem);
  int* flags = reinterpret_cast<int*>(smem + C::OFF_FLAGS);  // abort, bad length, tensor memory, partition; at 32 two barriers
  int* pref = reinterpret_cast<int*>(smem + C::OFF_PREF);
  uint16_t* perm = reinterpret_cast<uint16_t*>(smem + C::OFF_PERM);
  constexpr int WP = C::NP * 4, WM = WP + 1, WV = WP + 2, WQ = WP + 3;  // producer, product and Q warps
  if (tid == 0) {
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(cta.bar(C::FULL + i), 1);
      mbar_init(cta.bar(C::EMPTY + i), 1);
    }
    for (int i = 0; i < C::NR; ++i) {
      mbar_init(cta.bar(C::RFULL + i), 1);
      mbar_init(cta.bar(C::REMPTY + i), 1);
    }
    for (int i = 0; i < C::UQ; ++i) {
      mbar_init(cta.bar(C::UFULL + i), 1);
      mbar_init(cta.bar(C::UEMPTY + i), C::NP * 4 + 2 + C::LOADERS / 32 + C::CW);
    }
    for (int i = 0; i < C::NBUF; ++i) {
      mbar_init(cta.bar(C::SFULL + i), 1);
      mbar_init(cta.bar(C::PREADY + i), 128);
      mbar_init(cta.bar(C::PVDONE + i), 1);
    }
    mbar_init(cta.bar(C::QSTAGED), C::LOADERS);
    mbar_init(cta.bar(C::QTAKEN), C::NP * 128);
    mbar_init(cta.bar(C::QREADY), C::NP * 128);
    mbar_init(cta.bar(C::QFREE), 1);
    mbar_init(cta.bar(C::OFREE), C::NP * 128);
    mbar_init(cta.bar(C::XBAR), C::NP * 128);
    mbar_init(cta.bar(C::XFREE), C::NP * 128);
    mbar_init(cta.sbase + C::OFF_FLAGS + 32, 1);
    mbar_init(cta.sbase + C::OFF_FLAGS + 40, 1);
    flags[0] = flags[1] = 0;
    fence_mbarrier_init();
  }
  if (warp == WM) tmem_alloc(smem_addr(flags + 2), 512);
  plan_order<kView, C::BS, C::THREADS>(prm, smem + C::OFF_RING, pref, perm, flags + 1, flags + 3);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)flags[2];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tid == 0 && flags[1]) atomicCAS(prm.hdr + kHdrError, 0, kErrDeviceBounds);
  if (tid == 0 && blockIdx.x == 0) prm.hdr[kHdrPart] = flags[3];
  if (warp < WP) {
    // Sequences with too few tokens: zeros.
    constexpr int D16 = C::D / 8;
    for (int s = blockIdx.x; s < prm.S; s += gridDim.x) {
      bool bad = false;
      if (work_tokens<kView>(prm, seq_tokens<kView>(prm, s, prm.MB * C::BS, &bad), C::BS) > 0) continue;
      uint4* o = static_cast<uint4*>(prm.out) + (size_t)s * prm.H * D16;
      for (int i = tid; i < prm.H * D16; i += C::NP * 128) o[i] = make_uint4(0, 0, 0, 0);
      if (prm.lse)
        for (int i = tid; i < prm.H; i += C::NP * 128) prm.lse[(size_t)s * prm.H + i] = -INFINITY;
    }
    __syncwarp();
    cta.softmax(tmem, warp >> 2, tid & 127);
  } else {
    if (warp == WP) {
      cta.producer(flags[3], pref, perm, lane);
    } else if (warp == WM) {
      cta.score_products(tmem, lane);
    } else if (warp == WV) {
      cta.value_products(tmem, lane);
    } else if (warp < WQ + C::LOADERS / 32) {
      cta.bring_rows(tid - WQ * 32, lane);
    } else if constexpr (C::kFp8) {
      cta.widen(warp - WQ - C::LOADERS / 32, lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == WM) tmem_free(tmem, 512);
}

}  // namespace pa
