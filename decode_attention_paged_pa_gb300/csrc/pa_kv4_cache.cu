// pa_kv4_cache.cu -- tokens written into a 4-bit cache and read back
// (include/pa_decode.h: pa_kv4_append, pa_kv4_gather; the record of a block is
// described in pa_kv4.cuh).
//
// One vector is one token's key or value of one kv head: D elements of T next
// to each other in the token rows, D/2 bytes of codes and two parameters in
// the cache.  D/8 lanes (a power of two of them, the last ones idle at head
// sizes 80, 96 and 112) take a vector with one 16-byte access each on the row
// side and one 4-byte access on the cache side.  A CTA takes a run of
// consecutive tokens; its warps first find each token's sequence (a 32-way
// search of the row offsets), block and slot.
//
// Both kernels are bound by memory: 2 D bytes on the row side and D/2 + 4 on
// the cache side per vector, each touched once.
#include <cstring>

#include "pa_common.cuh"
#include "pa_decode.h"
#include "pa_launch.h"

namespace pa {
namespace {

struct Kv4Params {
  uint8_t* cache;
  const void* in[2];   // key, value rows (append)
  void* out[2];        // key, value rows (gather)
  const int32_t* bt;
  const int32_t* lens;
  const int32_t* cu;   // [S + 1], or null: every sequence has `per` tokens
  int* hdr;
  long long stride[2];  // elements between tokens of the key and value rows
  int S, N, per, KH, BS, MB, num_blocks;
  int tpc;             // tokens per CTA
};

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;  // per CTA

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

// Warp: block (-1: skip the token) and slot of row t.
__device__ __forceinline__ void place(const Kv4Params& p, int t, int lane, int* blk, int* slot) {
  int s = -1;
  if (!p.cu) {
    s = t / p.per;
  } else {
    // The last s in [0, S) with cu[s] <= t, 32 pivots a step.
    int lo = 0, n = p.S;
    while (true) {
      const int step = (n + 31) / 32;
      const int i = lo + lane * step;
      const bool le = lane * step < n && p.cu[i] <= t;
      const unsigned m = __ballot_sync(0xffffffffu, le);
      if (m == 0) break;  // t lies before the first row
      const int k = 31 - __clz(m);
      lo += k * step;
      n = min(step, n - k * step);
      if (step == 1) {
        s = lo;
        break;
      }
    }
  }
  *blk = -1;
  *slot = 0;
  if (s < 0 || s >= p.S) return;
  int first, n;
  seq_rows(p, s, &first, &n);
  const int i = t - first, L = p.lens[s];
  // Rows behind the last sequence (and rows of a malformed offset list) are left alone.
  if (i < 0 || i >= n || L < n || L > p.MB * p.BS) return;
  const int pos = L - n + i;
  const int b = p.bt[(size_t)s * p.MB + pos / p.BS];
  if ((unsigned)b >= (unsigned)p.num_blocks) return;
  *blk = b;
  *slot = pos % p.BS;
}

// CTA 0 checks every sequence and leaves the call's status in the header, so
// that no other launch has to clear it.
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
  return D <= 64 ? 8 : D <= 128 ? 16 : 32;
}

// The codes of 8 elements (element e in bits 4e ..) of a vector of lowest
// value lo and scale s (the scale that is stored: already rounded to T).
__device__ __forceinline__ uint32_t quantise8(const float (&f)[8], float lo, float s) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = s > 0.f ? min(15, __float2int_rn(__fdiv_rn(f[e] - lo, s))) : 0;
    w |= (uint32_t)c << (4 * e);
  }
  return w;
}

template <typename T, int D, bool GATHER>
__global__ void __launch_bounds__(kThreads) kv4_tokens_kernel(const __grid_constant__ Kv4Params p) {
  constexpr int LPV = lanes_per_vector<D>(), NG = kThreads / LPV;
  constexpr int X = D < 128 ? D : 128, XB = X / 2;
  __shared__ int s_blk[kMaxTokens], s_slot[kMaxTokens];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long t0 = (long long)blockIdx.x * p.tpc;
  const int nt = (int)min((long long)p.tpc, (long long)p.N - t0);
  for (int i = warp; i < nt; i += kThreads / 32) {
    int blk, slot;
    place(p, (int)t0 + i, lane, &blk, &slot);
    if (lane == 0) {
      s_blk[i] = blk;
      s_slot[i] = slot;
    }
  }
  __syncthreads();
  const int grp = threadIdx.x / LPV, gl = threadIdx.x % LPV;
  const bool act = gl < D / 8;
  const int per_tok = 2 * p.KH, nv = nt * per_tok;
  const size_t rec_bytes = (size_t)p.BS * (D + 8);
  // The loop bounds are the warp's, not the group's: its shuffles take whole warps.
  for (int v0 = 0; v0 < nv; v0 += NG) {
    const int v = v0 + grp;
    const bool on = v < nv;
    const int i = on ? v / per_tok : 0, k = on ? v - i * per_tok : 0;
    const int sel = k / p.KH, h = k - sel * p.KH;
    const int blk = on ? s_blk[i] : -1, slot = s_slot[i];
    const bool go = act && blk >= 0;
    uint8_t* rec = p.cache + ((size_t)max(blk, 0) * p.KH + h) * rec_bytes;
    uint32_t* code = reinterpret_cast<uint32_t*>(rec + (size_t)sel * p.BS * (D / 2) +
                                                 (size_t)(gl / (X / 8)) * p.BS * XB + (size_t)slot * XB +
                                                 (gl % (X / 8)) * 4);
    uint32_t* par = reinterpret_cast<uint32_t*>(rec + (size_t)p.BS * D + (size_t)slot * 8 + sel * 4);
    const size_t row = (size_t)(t0 + i) * (size_t)p.stride[sel] + (size_t)h * D + gl * 8;
    if constexpr (GATHER) {
      if (!go) continue;
      const uint32_t w = *code;
      const float2 sz = F16Traits<T>::to_float2(*par);
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = F16Traits<T>::pack(fmaf((float)((w >> (8 * e)) & 15u), sz.x, sz.y),
                                  fmaf((float)((w >> (8 * e + 4)) & 15u), sz.x, sz.y));
      *reinterpret_cast<uint4*>(static_cast<T*>(p.out[sel]) + row) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
      float f[8];
      float lo = INFINITY, hi = -INFINITY;
      bool odd = false;  // a NaN or an infinity among the elements
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = 0.f;
      if (go) {
        unpack_chunk<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(p.in[sel]) + row), f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          lo = fminf(lo, f[e]);
          hi = fmaxf(hi, f[e]);
          odd |= !(fabsf(f[e]) < INFINITY);
        }
      }
#pragma unroll
      for (int o = 1; o < LPV; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      }
      const unsigned odds = __ballot_sync(0xffffffffu, odd);
      const unsigned mine = (LPV == 32 ? 0xffffffffu : ((1u << LPV) - 1u) << (lane / LPV * LPV));
      if (!go) continue;
      // scale = (hi - lo) / 15, rounded to T, which the codes are taken
      // against; zero = lo, an element and so exact in T (a zero of either
      // sign is stored as +0).
      lo += 0.f;
      const float spread = hi - lo;
      const bool poison = (odds & mine) || !(spread < INFINITY);
      uint32_t sz = F16Traits<T>::pack(__fdiv_rn(spread, 15.f), lo), w = 0;
      if (poison) sz = 0x7fff7fffu;  // NaN in fp16 and in bf16
      else w = quantise8(f, lo, F16Traits<T>::to_float2(sz).x);
      *code = w;
      if (gl == 0) *par = sz;
    }
  }
  if (blockIdx.x == 0) write_status(p);
}

template <typename T, bool GATHER>
cudaError_t launch_tokens(const Kv4Params& p, int D, cudaStream_t st) {
  // Tokens per CTA: one while the call is too small to give every SM four
  // CTAs, then as many as still do, up to kMaxTokens.
  const int want = device_sm_count() * 4;
  Kv4Params q = p;
  q.tpc = p.N / want < 1 ? 1 : p.N / want > kMaxTokens ? kMaxTokens : p.N / want;
  const int grid = p.N == 0 ? 1 : (p.N + q.tpc - 1) / q.tpc;
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
  p.in[0] = p.out[0] = key;
  p.in[1] = p.out[1] = value;
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
