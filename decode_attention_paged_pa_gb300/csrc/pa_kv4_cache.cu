// pa_kv4_cache.cu -- tokens written into a 4-bit cache and read back
// (include/pa_decode.h: pa_kv4_append, pa_kv4_gather; the record of a block is
// described in pa_kv4.cuh).
//
// One vector is one token's key or value of one kv head: D elements of T next
// to each other in the token rows, D/2 bytes of codes and two parameters in
// the cache.  D/16 lanes (of a power of two, the last ones idle at head sizes
// 80, 96 and 112) take a vector with two 16-byte accesses each on the row side
// and two 4-byte accesses on the cache side, two vectors at a time so that
// enough loads are in flight.  A lane's two groups of 8 elements lie half a
// vector apart: each access is contiguous over the lanes (16 elements next to
// each other and 8-byte codes instead wrote half sectors, 115 us for the
// prompts below where this took 111).  A CTA takes a run of consecutive tokens; its
// first warp finds each token's sequence (a 32-way search of the row offsets
// for the first, steps from there for the others), block and slot, while the
// others' rows are on their way.
//
// Per vector 2 D bytes on the row side and D/2 + 4 on the cache side are touched
// once.  Read-back is bound by memory (loads in flight); the append by issue (76%
// of the slots, 43% of the memory's rate: about seven single-precision
// instructions an element for its code).  A first form with eight elements a
// lane, fp32 minima and a division per element took twice as long; so minima and maxima are taken on packed pairs (they are
// exact in T), the lowest and the negated highest in one word through the
// shuffles; the quotient (x - zero) / scale by a reciprocal, and only where it
// lies so close to a tie that the reciprocal's error could decide, by the
// division that defines the code; and read-back is one packed multiply-add per
// pair (rounded once).
//
// Measured (GB300): chunks of 24 prompts written and their contexts read back
// (8 kv heads, D = 128), 104 us for 542 MB, 77% of the measured copy rate of
// 6766 GB/s (247 in the first form; 137 with a persistent grid whose first warp
// looked ahead: many small CTAs hide the placing as well); alone, the append
// takes 41 us for 164 MB (60% of that rate), the read-back 65 for 406 MB (92%).
// One token each of 128 sequences, written and read back: 7 us, two launches of
// three dependent loads each.
//
// The status check takes a thread a sequence: of a single sequence of thousands
// of blocks it takes longer than the rows do.  One context of 131072 tokens read
// back, D = 128: 143 us with one kv head (floor 12.6), 233 with eight (floor 100),
// blocks of 16; 274 and 414 with twice as many blocks, of 8; written, 196 us with
// eight (floor 100).
#include <cstring>

#include "pa_common.cuh"
#include "pa_decode.h"
#include "pa_launch.h"

namespace pa {
namespace {

struct Kv4Params {
  uint8_t* cache;
  void* row[2];        // key, value rows (append: only read)
  const int32_t* bt;
  const int32_t* lens;
  const int32_t* cu;   // [S + 1], or null: every sequence has `per` tokens
  int* hdr;
  long long stride[2];  // elements between tokens of the key and value rows
  int S, N, per, KH, BS, MB, num_blocks;
  int tpc;             // tokens per CTA
};

constexpr int kWorkers = 128, kThreads = kWorkers + 32;
constexpr int kMaxTokens = 32;   // per CTA
constexpr int kElements = 16384;  // per CTA, about
constexpr int kBatch = 2;       // vectors a lane group has in flight

// New (or wanted) tokens of sequence s: rows [first, first + n) of N.
__device__ __forceinline__ void seq_rows(const Kv4Params& p, int s, int* first, int* n) {
  if (p.cu) {
    *first = p.cu[s];
    *n = p.cu[s + 1] - *first;
  } else {
    *first = s * p.per;
    *n = p.per;
  }
}

// Warp: block (-1: skip the token) and slot of rows t0 + lane (lane < nt).
__device__ __forceinline__ void place(const Kv4Params& p, int t0, int nt, int lane, int* blk, int* slot) {
  *blk = -1;
  *slot = 0;
  const int t = t0 + lane;
  int s = -1;
  if (!p.cu) {
    s = t / p.per;
  } else {
    // The last s in [0, S) with cu[s] <= t0, 32 pivots a step.
    int lo = 0, n = p.S;
    while (true) {
      const int step = (n + 31) / 32;
      const int i = lo + lane * step;
      const bool le = lane * step < n && p.cu[i] <= t0;
      const unsigned m = __ballot_sync(0xffffffffu, le);
      const int k = m ? 31 - __clz(m) : 0;  // (t0 before the first row: from sequence 0 on)
      lo += k * step;
      n = min(step, n - k * step);
      if (step == 1) break;
    }
    if (lane >= nt) return;
    s = lo;
    while (s + 1 < p.S && p.cu[s + 1] <= t) ++s;
  }
  if (lane >= nt || s < 0 || s >= p.S) return;
  int first, n;
  seq_rows(p, s, &first, &n);
  const int i = t - first, L = p.lens[s];
  // Rows behind the last sequence are left alone, and so are those of a sequence
  // that write_status refuses.
  if (i < 0 || i >= n || first < 0 || first + (long long)n > p.N || L < n || L > p.MB * p.BS) return;
  const int pos = L - n + i;
  const int b = p.bt[(size_t)s * p.MB + pos / p.BS];
  if ((unsigned)b >= (unsigned)p.num_blocks) return;
  *blk = b;
  *slot = pos % p.BS;
}

// CTA 0 checks every sequence, a thread each, and leaves the call's status in the
// header, so that no other launch has to clear it.
__device__ __forceinline__ void write_status(const Kv4Params& p) {
  int bad = 0;
  if (p.cu && threadIdx.x == 0 && p.cu[0] < 0) bad = 1;
  for (int s = threadIdx.x; s < p.S; s += kThreads) {
    int first, n;
    seq_rows(p, s, &first, &n);
    const int L = p.lens[s];
    if (n < 0 || first < 0 || first + (long long)n > p.N || L < n || L > p.MB * p.BS) {
      bad = 1;
      continue;
    }
    if (n == 0) continue;
    for (int j = (L - n) / p.BS; j <= (L - 1) / p.BS; ++j)
      bad |= (unsigned)p.bt[(size_t)s * p.MB + j] >= (unsigned)p.num_blocks;
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) p.hdr[kHdrError] = bad ? kErrDeviceBounds : kOk;
}

template <int D>
constexpr int lanes_per_vector() {
  return D <= 64 ? 4 : D <= 128 ? 8 : 16;
}

// Packed pairs of T.
template <typename T> struct Pair;
template <> struct Pair<__half> {
  using V = __half2;
  static constexpr uint32_t kBase = 0x64006400u;  // 1024: a code in the low bits adds exactly
  static constexpr uint32_t kSmallest = 0x0400u;  // smallest normal number
  static constexpr uint32_t kInf = 0x7c007c00u;
  __device__ __forceinline__ static V fma(V a, V b, V c) { return __hfma2(a, b, c); }
};
template <> struct Pair<__nv_bfloat16> {
  using V = __nv_bfloat162;
  static constexpr uint32_t kBase = 0x43004300u;  // 128
  static constexpr uint32_t kSmallest = 0x0080u;
  static constexpr uint32_t kInf = 0x7f807f80u;
  __device__ __forceinline__ static V fma(V a, V b, V c) { return __hfma2(a, b, c); }
};
template <typename V>
__device__ __forceinline__ V as_pair(uint32_t w) { return *reinterpret_cast<V*>(&w); }
template <typename V>
__device__ __forceinline__ uint32_t as_word(V v) { return *reinterpret_cast<uint32_t*>(&v); }

// The codes of 8 elements (element e in bits 4e ..) of a vector of lowest
// value lo and scale s (the scale that is stored: already rounded to T);
// r: about 1 / s.  `fast`: s is a normal number of T.
__device__ __forceinline__ uint32_t quantise8(const float (&f)[8], float lo, float s, float r, bool fast) {
  // x + 1.5 * 2^23 holds the nearest integer to x (ties to even) in its low bits.
  constexpr float kMagic = 12582912.f;
  float far = 0.f;  // largest distance of a quotient from its integer
  uint32_t w = 0;
#pragma unroll
  for (int e = 7; e >= 0; --e) {
    const float t = (f[e] - lo) * r;
    const float m = t + kMagic;
    far = fmaxf(far, fabsf(t - (m - kMagic)));
    w = w * 16u + __float_as_uint(m);
  }
  w -= 0x4b400000u * 0x11111111u;
  // t is within 2^-17 of the quotient (the reciprocal and three roundings at a
  // value below 16), and at most 15.1 as s is rounded to 8 bits or more: a
  // distance that far from a half decides nothing else.
  if (!fast || !(far < 0.5f - 1.f / 65536.f)) {
    w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = s > 0.f ? min(15, __float2int_rn(__fdiv_rn(f[e] - lo, s))) : 0;
      w |= (uint32_t)c << (4 * e);
    }
  }
  return w;
}

template <typename T, int D, bool GATHER>
__global__ void __launch_bounds__(kThreads, GATHER ? 9 : 7) kv4_tokens_kernel(const __grid_constant__ Kv4Params p) {
  using P = Pair<T>;
  using V = typename P::V;
  constexpr int LPV = lanes_per_vector<D>(), NG = kWorkers / LPV;
  constexpr int X = D < 128 ? D : 128, XB = X / 2;
  __shared__ int s_blk[kMaxTokens], s_slot[kMaxTokens];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long t0 = (long long)blockIdx.x * p.tpc;
  const int nt = (int)min((long long)p.tpc, (long long)p.N - t0);
  if (threadIdx.x >= kWorkers) {
    if (nt > 0) {
      int blk, slot;
      place(p, (int)t0, nt, lane, &blk, &slot);
      if (lane < nt) {
        s_blk[lane] = blk;
        s_slot[lane] = slot;
      }
      named_barrier_sync(1, kThreads);
    }
  } else {
    const int grp = threadIdx.x / LPV, gl = threadIdx.x % LPV;
    const bool act = gl < D / 16;
    const int per_tok = 2 * p.KH;
    const uint32_t rec_bytes = (uint32_t)p.BS * (D + 8), half = (uint32_t)p.BS * (D / 2);
    // This lane's two groups of 8 elements (each access is contiguous over the lanes).
    constexpr int HALF = D / 16;
    const uint32_t at0 = (uint32_t)(gl / (X / 8)) * p.BS * XB + (uint32_t)(gl % (X / 8)) * 4;
    const uint32_t at1 = (uint32_t)((gl + HALF) / (X / 8)) * p.BS * XB + (uint32_t)((gl + HALF) % (X / 8)) * 4;
    // This group's next vector: token i, and k = (key or value, head) within it.
    int i = grp / per_tok, k = grp - i * per_tok;
    bool placed = false;
    // The loop bound is the CTA's, not the group's: shuffles take whole warps.
    for (int v0 = 0; v0 < nt * per_tok; v0 += NG * kBatch) {
      uint4 x[kBatch][2];
      T* row[kBatch];
      int vi[kBatch], vk[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int sel = k >= p.KH;
        vi[j] = i;
        vk[j] = k;
        row[j] = static_cast<T*>(p.row[sel]) + (t0 + i) * p.stride[sel] + (k - sel * p.KH) * D + gl * 8;
        if constexpr (!GATHER) {
          x[j][0] = x[j][1] = make_uint4(0, 0, 0, 0);
          if (act && i < nt) {
            x[j][0] = reinterpret_cast<const uint4*>(row[j])[0];
            x[j][1] = reinterpret_cast<const uint4*>(row[j])[HALF];
          }
        }
        for (k += NG; k >= per_tok; k -= per_tok) ++i;
      }
      if (!placed) {
        named_barrier_sync(1, kThreads);
        placed = true;
      }
      // This lane's code words, and the vector's parameters.
      uint8_t *code[kBatch], *par[kBatch];
      bool go[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const bool in = vi[j] < nt;
        const int blk = in ? s_blk[vi[j]] : -1;
        const uint32_t slot = in ? s_slot[vi[j]] : 0, sel = vk[j] >= p.KH;
        uint8_t* rec = p.cache + ((size_t)max(blk, 0) * p.KH + (vk[j] - (int)sel * p.KH)) * rec_bytes;
        code[j] = rec + (sel * half + slot * XB);
        par[j] = rec + (2 * half + slot * 8 + sel * 4);
        go[j] = act && blk >= 0;
      }
      if constexpr (GATHER) {
        uint2 w[kBatch];
        uint32_t sz[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          w[j].x = go[j] ? *reinterpret_cast<const uint32_t*>(code[j] + at0) : 0u;
          w[j].y = go[j] ? *reinterpret_cast<const uint32_t*>(code[j] + at1) : 0u;
          sz[j] = go[j] ? *reinterpret_cast<const uint32_t*>(par[j]) : 0u;
        }
        const V base = as_pair<V>(P::kBase);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const V s = as_pair<V>(__byte_perm(sz[j], 0, 0x1010)), z = as_pair<V>(__byte_perm(sz[j], 0, 0x3232));
          uint32_t o[8];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t c = q ? w[j].y : w[j].x;
            uint32_t v[4];  // elements e and e + 4
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = as_word(P::fma(__hsub2(as_pair<V>(((c >> (4 * e)) & 0x000f000fu) | P::kBase), base), s, z));
            o[4 * q] = __byte_perm(v[0], v[1], 0x5410);
            o[4 * q + 1] = __byte_perm(v[2], v[3], 0x5410);
            o[4 * q + 2] = __byte_perm(v[0], v[1], 0x7632);
            o[4 * q + 3] = __byte_perm(v[2], v[3], 0x7632);
          }
          if (go[j]) {
            reinterpret_cast<uint4*>(row[j])[0] = make_uint4(o[0], o[1], o[2], o[3]);
            reinterpret_cast<uint4*>(row[j])[HALF] = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          // Lowest and highest, a NaN going through (idle lanes: no influence).
          const uint32_t e[8] = {x[j][0].x, x[j][0].y, x[j][0].z, x[j][0].w,
                                 x[j][1].x, x[j][1].y, x[j][1].z, x[j][1].w};
          V lo = as_pair<V>(e[0]), hi = lo;
#pragma unroll
          for (int q = 1; q < 8; ++q) {
            lo = __hmin2_nan(lo, as_pair<V>(e[q]));
            hi = __hmax2_nan(hi, as_pair<V>(e[q]));
          }
          // (low, -high) in one word.
          const uint32_t nh = as_word(hi) ^ 0x80008000u;
          V m = __hmin2_nan(as_pair<V>(__byte_perm(as_word(lo), nh, 0x5410)),
                            as_pair<V>(__byte_perm(as_word(lo), nh, 0x7632)));
          if (!act) m = as_pair<V>(P::kInf);
#pragma unroll
          for (int o = 1; o < LPV; o <<= 1) m = __hmin2_nan(m, as_pair<V>(__shfl_xor_sync(0xffffffffu, as_word(m), o)));
          if (!go[j]) continue;
          const float2 mf = F16Traits<T>::to_float2(as_word(m));
          // scale = (hi - lo) / 15, rounded to T, which the codes are taken
          // against; zero = lo, an element and so exact in T (a zero of either
          // sign is stored as +0).
          const float low = mf.x + 0.f, spread = -mf.y - low;
          uint32_t sz = F16Traits<T>::pack(__fdiv_rn(spread, 15.f), low);
          uint2 w = make_uint2(0, 0);
          if (!(spread < INFINITY)) {
            sz = 0x7fff7fffu;  // NaN in fp16 and in bf16
          } else {
            const float s = F16Traits<T>::to_float2(sz).x;
            float r;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
            const bool fast = (sz & 0xffffu) >= P::kSmallest;
            float f[8];
            unpack_chunk<T>(x[j][0], f);
            w.x = quantise8(f, low, s, r, fast);
            unpack_chunk<T>(x[j][1], f);
            w.y = quantise8(f, low, s, r, fast);
          }
          *reinterpret_cast<uint32_t*>(code[j] + at0) = w.x;
          *reinterpret_cast<uint32_t*>(code[j] + at1) = w.y;
          if (gl == 0) *reinterpret_cast<uint32_t*>(par[j]) = sz;
        }
      }
    }
  }
  if (blockIdx.x == 0) write_status(p);
}

template <typename T, bool GATHER>
cudaError_t launch_tokens(const Kv4Params& p, int D, cudaStream_t st) {
  // Tokens per CTA: one while the call is too small to give every SM eight
  // CTAs, then as many as still do, up to kElements' worth (8 tokens of 8 heads
  // of 128 dims: 104 us for the prompts above, 111 with 16 tokens, 105 with 4;
  // 8 tokens whatever the heads: 162 against 140 us at 32 heads, 122 against 47
  // at one head of 64 dims).
  const int want = device_sm_count() * 8, most = kElements / (2 * p.KH * D);
  Kv4Params q = p;
  q.tpc = max(1, min(min(most, kMaxTokens), p.N / want));
  const int grid = p.N == 0 ? 1 : (int)(((long long)p.N + q.tpc - 1) / q.tpc);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  switch (D) {
    case 64: return cudaLaunchKernelEx(&cfg, kv4_tokens_kernel<T, 64, GATHER>, q);
    case 80: return cudaLaunchKernelEx(&cfg, kv4_tokens_kernel<T, 80, GATHER>, q);
    case 96: return cudaLaunchKernelEx(&cfg, kv4_tokens_kernel<T, 96, GATHER>, q);
    case 112: return cudaLaunchKernelEx(&cfg, kv4_tokens_kernel<T, 112, GATHER>, q);
    case 128: return cudaLaunchKernelEx(&cfg, kv4_tokens_kernel<T, 128, GATHER>, q);
    case 256: return cudaLaunchKernelEx(&cfg, kv4_tokens_kernel<T, 256, GATHER>, q);
    default: return cudaErrorInvalidValue;
  }
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int tokens_impl(bool gather, void* kv_cache, void* key, void* value, const int32_t* block_tables,
                const int32_t* seq_lens, const int32_t* cu_tokens, int num_seqs, int num_tokens, int num_kv_heads,
                int head_size, int block_size, long long key_stride, long long value_stride, int dtype, void* stream,
                int max_blocks_per_seq, int num_blocks, void* workspace, size_t workspace_bytes) {
  const int D = head_size, BS = block_size;
  if (num_seqs < 0 || num_tokens < 0 || num_kv_heads <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 ||
      BS <= 0 || D <= 0 || (long long)max_blocks_per_seq * BS > 0x3fffffff)
    return PA_ERR_INVALID_ARG;
  if (dtype != PA_DTYPE_FP16 && dtype != PA_DTYPE_BF16 && dtype != PA_DTYPE_FP32) return PA_ERR_INVALID_ARG;
  if (dtype == PA_DTYPE_FP32 || pa_kv4_block_bytes(D, BS) == 0) return PA_ERR_UNSUPPORTED;
  if (num_kv_heads > 65535) return PA_ERR_INVALID_ARG;
  if (num_seqs == 0 && num_tokens > 0) return PA_ERR_INVALID_ARG;
  // Uniform rows: every sequence has the same number of tokens.
  if (!cu_tokens && num_seqs > 0 && num_tokens % num_seqs != 0) return PA_ERR_INVALID_ARG;
  const long long width = (long long)num_kv_heads * D;
  if (key_stride < width || value_stride < width || key_stride % 8 != 0 || value_stride % 8 != 0)
    return PA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 16)) return PA_ERR_INVALID_ARG;
  if (workspace_bytes < kHdrInts * sizeof(int)) return PA_ERR_WORKSPACE;
  if (!kv_cache || !aligned(kv_cache, 16)) return PA_ERR_INVALID_ARG;
  if (num_seqs > 0 && (!block_tables || !seq_lens || !aligned(block_tables, 4) || !aligned(seq_lens, 4)))
    return PA_ERR_INVALID_ARG;
  if (cu_tokens && !aligned(cu_tokens, 4)) return PA_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!key || !value || !aligned(key, 16) || !aligned(value, 16))) return PA_ERR_INVALID_ARG;
  Kv4Params p;
  std::memset(&p, 0, sizeof p);
  p.cache = static_cast<uint8_t*>(kv_cache);
  p.row[0] = key;
  p.row[1] = value;
  p.bt = block_tables;
  p.lens = seq_lens;
  p.cu = num_seqs > 0 ? cu_tokens : nullptr;
  p.hdr = static_cast<int*>(workspace);
  p.stride[0] = key_stride;
  p.stride[1] = value_stride;
  p.S = num_seqs;
  p.N = num_tokens;
  p.per = num_seqs > 0 ? num_tokens / num_seqs : 0;
  p.KH = num_kv_heads;
  p.BS = BS;
  p.MB = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (gather)
    e = dtype == PA_DTYPE_FP16 ? launch_tokens<__half, true>(p, D, st) : launch_tokens<__nv_bfloat16, true>(p, D, st);
  else
    e = dtype == PA_DTYPE_FP16 ? launch_tokens<__half, false>(p, D, st)
                               : launch_tokens<__nv_bfloat16, false>(p, D, st);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_kv4_block_bytes(int head_size, int block_size) {
  const int D = head_size, BS = block_size;
  const bool d_ok = D == 64 || D == 80 || D == 96 || D == 112 || D == 128 || D == 256;
  const bool bs_ok = BS == 8 || BS == 16 || BS == 32 || BS == 64;
  return d_ok && bs_ok ? (size_t)BS * (D + 8) : 0;
}

extern "C" int pa_kv4_append(void* kv_cache, const void* key, const void* value, const int32_t* block_tables,
                             const int32_t* seq_lens, const int32_t* cu_tokens, int num_seqs, int num_tokens,
                             int num_kv_heads, int head_size, int block_size, long long key_stride,
                             long long value_stride, int dtype, void* stream, int max_blocks_per_seq,
                             int num_blocks, void* workspace, size_t workspace_bytes) {
  return tokens_impl(false, kv_cache, const_cast<void*>(key), const_cast<void*>(value), block_tables, seq_lens,
                     cu_tokens, num_seqs, num_tokens, num_kv_heads, head_size, block_size, key_stride,
                     value_stride, dtype, stream, max_blocks_per_seq, num_blocks, workspace, workspace_bytes);
}

extern "C" int pa_kv4_gather(void* key_out, void* value_out, const void* kv_cache, const int32_t* block_tables,
                             const int32_t* seq_lens, const int32_t* cu_tokens, int num_seqs, int num_tokens,
                             int num_kv_heads, int head_size, int block_size, long long key_stride,
                             long long value_stride, int dtype, void* stream, int max_blocks_per_seq,
                             int num_blocks, void* workspace, size_t workspace_bytes) {
  return tokens_impl(true, const_cast<void*>(kv_cache), key_out, value_out, block_tables, seq_lens, cu_tokens,
                     num_seqs, num_tokens, num_kv_heads, head_size, block_size, key_stride, value_stride, dtype,
                     stream, max_blocks_per_seq, num_blocks, workspace, workspace_bytes);
}
