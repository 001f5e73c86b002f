// pa_cache.cu -- tokens written into paged caches by their slots, and the
// accepted nodes of a tree moved together (include/pa_decode.h: pa_cache_write,
// pa_tree_accept).
//
// A cache has one block of one kv head contiguous: keys [D/x][BS][x] with 16
// bytes a (chunk of dims, token), values [D][BS].  A token's value is therefore D
// elements BS elements apart, and only tokens that follow one another in a block
// make contiguous bytes.
//
// pa_cache_write.  A CTA takes a run of rows of one kv head into shared memory
// (16-byte loads; for an E4M3 cache rounded on the way) and writes them out by
// chunks: rows that follow one another in up to 32 bytes of a value row (CT
// tokens).  A chunk belongs to the CTA that has its first row, which reads on past
// its last row for it, so no chunk is cut by the split into CTAs.  A full chunk's
// values are transposed in registers (CT words of 4 / element-size dims) and
// stored 16 bytes at a time, its keys as runs of 16 bytes a token; of others every
// element is stored by itself.
//
// pa_tree_accept.  A thread takes one column of a kv head (a 16-byte chunk of the
// key, or one dim of the value) along the whole path, up to kBatch moves' loads
// before their stores.  Accepted nodes ascend, so node i of the path lies at or
// behind place i: a store never lands on what a later batch reads.
//
// Measured: one token of 128 sequences (8 kv heads of 128 dims, bf16) 3.9 us a call in a
// graph, a launch's latency; 24 prompts of 257 to 2049 tokens, fp16 rows into E4M3 codes, 41 us
// for 156 MB (3.8 TB/s; 23 at the copy's rate), bound by the instructions of rounding and
// transposing.  The paths of a batch's trees in eight layers 14 us (dependent loads: length,
// path, table, row; nodes that are in their places already are moved like the others).
#include <algorithm>
#include <atomic>
#include <climits>
#include <cstring>
#include <new>

#include <cuda_fp8.h>

#include "pa_common.cuh"
#include "pa_decode.h"
#include "pa_launch.h"

namespace pa {
namespace {

struct WriteParams {
  uint8_t* cache[2];         // keys, values
  const uint8_t* row[2];     // key, value rows
  const long long* slots;    // [N]
  int* hdr;
  long long stride[2];       // bytes between rows
  long long total;           // slots in the pool
  float scale[2];
  int N, KH, D, BS, T;       // T: rows per CTA
  int shift;                 // BS = 1 << shift
};

constexpr int kWriteThreads = 256;

// Source elements of the rows.
enum Source { kCopy, kHalf, kBfloat, kFloat };

// E4M3 codes of x / scale: the quotient in fp32, to nearest even, rounded again to
// nearest even and kept within +-448; NaN stays NaN.  The quotient comes from x times the
// reciprocal in two steps: the first is within an ulp, and from one that is, with the
// reciprocal rounded to nearest, the remainder times it gives the rounded quotient
// (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990).  Two elements an instruction; with x and the reciprocal negated, a
// zero keeps its sign.  Where a quotient is 1024 or more, or the remainders could leave
// fp32's exact range, the division itself.  (One division for each element, and one for
// each index, took 60 us where this takes 45: 24 prompts of 1100 tokens, 8 kv heads of
// 128 dims, fp16.)
struct Divisor {
  uint64_t s2, i2;  // the scale (which is positive) and -1 / scale, twice each
  float scale, most;
  __device__ __forceinline__ static uint64_t both(float a, float b) {
    uint64_t x;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
    return x;
  }
  __device__ __forceinline__ explicit Divisor(float s) {
    const float inv = -1.f / s;
    s2 = both(s, s);
    i2 = both(inv, inv);
    scale = s;
    most = s >= 0x1p-64f && s <= 0x1p64f ? 1024.f * s : -1.f;
  }
};
__device__ __forceinline__ uint32_t e4m3x2_of(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// `a` and `b`: -x of two elements.
__device__ __forceinline__ uint32_t e4m3x2_of(float a, float b, const Divisor& s) {
  const auto fma2 = [](uint64_t x, uint64_t y, uint64_t z) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
    return d;
  };
  const uint64_t x = Divisor::both(a, b);
  uint64_t q;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(x), "l"(s.i2));
#pragma unroll
  for (int i = 0; i < 2; ++i) q = fma2(fma2(q, s.s2, x), s.i2, q);
  float qa, qb;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(qa), "=f"(qb) : "l"(q));
  return e4m3x2_of(qa, qb);
}
template <typename T>
__device__ __noinline__ uint2 e4m3x8_divided(uint4 x, float scale) {
  float f[8];
  unpack_chunk<T>(x, f);
  uint32_t w[2] = {0, 0};
  for (int i = 0; i < 4; ++i)
    w[i / 2] |= e4m3x2_of(__fdiv_rn(f[2 * i], scale), __fdiv_rn(f[2 * i + 1], scale)) << (16 * (i & 1));
  return make_uint2(w[0], w[1]);
}
__device__ __noinline__ uint32_t e4m3x4_divided(uint4 x, float s) {
  return e4m3x2_of(__fdiv_rn(__uint_as_float(x.x), s), __fdiv_rn(__uint_as_float(x.y), s)) |
         e4m3x2_of(__fdiv_rn(__uint_as_float(x.z), s), __fdiv_rn(__uint_as_float(x.w), s)) << 16;
}
// (The largest magnitude of eight elements, NaN if there is one: two of them.)
__device__ __forceinline__ float2 most_of(const uint4& x, __half) {
  const __half2* h = reinterpret_cast<const __half2*>(&x);
  return __half22float2(__hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])), __hmax2_nan(__habs2(h[2]), __habs2(h[3]))));
}
__device__ __forceinline__ float2 most_of(const uint4& x, __nv_bfloat16) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&x);
  return __bfloat1622float2(
      __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])), __hmax2_nan(__habs2(h[2]), __habs2(h[3]))));
}
template <typename T>
__device__ __forceinline__ uint2 e4m3x8_of(const uint4& x, const Divisor& s) {
  const float2 m = most_of(x, T());
  if (!(m.x < s.most && m.y < s.most)) return e4m3x8_divided<T>(x, s.scale);
  float f[8];
  constexpr uint32_t flip = 0x80008000u;
  unpack_chunk<T>(make_uint4(x.x ^ flip, x.y ^ flip, x.z ^ flip, x.w ^ flip), f);
  return make_uint2(e4m3x2_of(f[0], f[1], s) | e4m3x2_of(f[2], f[3], s) << 16,
                    e4m3x2_of(f[4], f[5], s) | e4m3x2_of(f[6], f[7], s) << 16);
}
// 16 bytes of a row as they are held in the cache: copied, or 8 (4) elements rounded.
template <int SRC>
struct Piece {
  using V = uint4;
  static __device__ __forceinline__ V make(const uint4& x, const Divisor&) { return x; }
};
template <>
struct Piece<kHalf> {
  using V = uint2;
  static __device__ __forceinline__ V make(const uint4& x, const Divisor& s) { return e4m3x8_of<__half>(x, s); }
};
template <>
struct Piece<kBfloat> {
  using V = uint2;
  static __device__ __forceinline__ V make(const uint4& x, const Divisor& s) { return e4m3x8_of<__nv_bfloat16>(x, s); }
};
template <>
struct Piece<kFloat> {
  using V = uint32_t;
  static __device__ __forceinline__ V make(const uint4& x, const Divisor& s) {
    const float a = __uint_as_float(x.x), b = __uint_as_float(x.y), c = __uint_as_float(x.z), d = __uint_as_float(x.w);
    if (!(fabsf(a) < s.most && fabsf(b) < s.most && fabsf(c) < s.most && fabsf(d) < s.most))
      return e4m3x4_divided(x, s.scale);
    return e4m3x2_of(-a, -b, s) | e4m3x2_of(-c, -d, s) << 16;
  }
};

// i, i + kWriteThreads, .. as a * n + b: one division for all.
struct Walk {
  int a, b, da, db, n;
  __device__ __forceinline__ Walk(int i, int n_) : a(i / n_), b(i - a * n_), da(kWriteThreads / n_), db(kWriteThreads - da * n_), n(n_) {}
  __device__ __forceinline__ void next() {
    a += da;
    b += db;
    if (b >= n) {
      b -= n;
      ++a;
    }
  }
};

// Elements [first, first + n) of a word's place as one element of E bytes.
template <int E> struct Elem;
template <> struct Elem<1> { using T = uint8_t; };
template <> struct Elem<2> { using T = uint16_t; };
template <> struct Elem<4> { using T = uint32_t; };

// Dim i (of 4 / E) of CT tokens' words w, next to each other: out[q] holds tokens
// q * (4 / E) ...
template <int E, int CT>
__device__ __forceinline__ void gather_dim(const uint32_t (&w)[CT], int i, uint32_t (&out)[CT * E / 4]) {
#pragma unroll
  for (int q = 0; q < CT * E / 4; ++q) {
    if constexpr (E == 4) {
      out[q] = w[q];
    } else if constexpr (E == 2) {
      out[q] = __byte_perm(w[2 * q], w[2 * q + 1], i ? 0x7632 : 0x5410);
    } else {
      const uint32_t sel = 0x40u + 0x11u * (uint32_t)i;  // byte i of each of two words
      const uint32_t lo = __byte_perm(w[4 * q], w[4 * q + 1], sel), hi = __byte_perm(w[4 * q + 2], w[4 * q + 3], sel);
      out[q] = __byte_perm(lo, hi, 0x5410);
    }
  }
}

template <int SRC, int E, int CT>
__global__ void __launch_bounds__(kWriteThreads, 4) cache_write_kernel(const __grid_constant__ WriteParams p) {
  using PV = typename Piece<SRC>::V;
  using EL = typename Elem<E>::T;
  constexpr int SE = SRC == kCopy ? E : SRC == kFloat ? 4 : 2;  // bytes of a row's element
  constexpr int X = 16 / E, DPW = 4 / E;                        // dims of a key chunk, of a 4-byte word
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int s_n, s_end;     // chunks, and the end of the rows that they need
  __shared__ uint32_t s_next[4];  // bit i: row i follows the one before in its chunk
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  if (blockIdx.x == gridDim.x - 1) {
    // The status: slots past the pool (negative ones are rows to be skipped).
    if (blockIdx.y != 0) return;
    int bad = 0;
#pragma unroll 8
    for (int i = tid; i < p.N; i += kWriteThreads) bad |= p.slots[i] >= p.total;
    bad = __syncthreads_or(bad);
    if (tid == 0) p.hdr[kHdrError] = bad ? kErrDeviceBounds : kOk;
    return;
  }
  const int D = p.D, BS = p.BS, T = p.T, kv = blockIdx.y;
  const int r0 = blockIdx.x * T, rows = min(T + CT - 1, p.N - r0);  // (r0 < N < 2^31 - T - CT)
  const int pitch = D * E + 16, ppr = D * SE / 16;                  // 16-byte pieces per row
  uint8_t* tile[2] = {smem, smem + (size_t)(T + CT - 1) * pitch};
  int4* chunk = reinterpret_cast<int4*>(smem + 2 * (size_t)(T + CT - 1) * pitch);  // [T] first row, rows, block, offset in the block
  // The slots of the tile's rows, and on their way with them the rows' first pieces.
  long long s = -2, before = -2;  // (-2 and its successor are no slots)
  if (tid < rows) {
    s = p.slots[r0 + tid];
    if (r0 + tid > 0) before = p.slots[r0 + tid - 1];
  }
  constexpr int LB = 4;  // loads in flight, of keys and of values
  const uint8_t* src[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) src[w] = p.row[w] + (size_t)r0 * p.stride[w] + (size_t)kv * D * SE;
  Walk at(tid, ppr);
  uint4 x[2][LB];
  int where[LB];
  const int own = min(rows, T);
#pragma unroll
  for (int u = 0; u < LB; ++u) {
    where[u] = at.a < own ? at.a * pitch + at.b * (int)sizeof(PV) : -1;
    if (where[u] >= 0)
#pragma unroll
      for (int w = 0; w < 2; ++w) x[w][u] = *reinterpret_cast<const uint4*>(src[w] + (size_t)at.a * p.stride[w] + at.b * 16);
    at.next();
  }
  if (tid == 0) s_n = s_end = 0;
  if (s < 0 || s >= p.total) s = -2;
  if (before < 0 || before >= p.total) before = -2;
  const bool follows = s >= 0 && before + 1 == s && s % CT != 0;
  if (tid < 128) {
    const uint32_t m = __ballot_sync(0xffffffffu, follows);
    if ((tid & 31) == 0) s_next[tid >> 5] = m;
  }
  __syncthreads();
  if (tid < T && s >= 0 && !follows) {
    const int i = tid + 1;  // (T is 64 at most)
    const int n = 1 + __ffs(~__funnelshift_r(s_next[i >> 5], s_next[(i >> 5) + 1], i & 31)) - 1;
    const int k = atomicAdd(&s_n, 1);
    const int blk = (int)((unsigned long long)s >> p.shift);
    chunk[k] = make_int4(tid, n, blk, (int)(s - ((long long)blk << p.shift)));
    atomicMax(&s_end, tid + n);
  }
  __syncthreads();
  const int nch = s_n, need = s_end;
  if (nch == 0) return;
  // (At least one row in front may belong to the CTA before: it is loaded for nothing.)
  const Divisor div[2] = {Divisor(p.scale[0]), Divisor(p.scale[1])};
#pragma unroll
  for (int u = 0; u < LB; ++u)
    if (where[u] >= 0)
#pragma unroll
      for (int w = 0; w < 2; ++w) *reinterpret_cast<PV*>(tile[w] + where[u]) = Piece<SRC>::make(x[w][u], div[w]);
  const int rest = tid + min(own * ppr, LB * kWriteThreads);  // pieces before it are there
  at = Walk(rest, ppr);
  for (int i = rest; i < need * ppr; i += LB * kWriteThreads) {
#pragma unroll
    for (int u = 0; u < LB; ++u) {
      where[u] = at.a < need ? at.a * pitch + at.b * (int)sizeof(PV) : -1;
      if (where[u] >= 0)
#pragma unroll
        for (int w = 0; w < 2; ++w) x[w][u] = *reinterpret_cast<const uint4*>(src[w] + (size_t)at.a * p.stride[w] + at.b * 16);
      at.next();
    }
#pragma unroll
    for (int u = 0; u < LB; ++u)
      if (where[u] >= 0)
#pragma unroll
        for (int w = 0; w < 2; ++w) *reinterpret_cast<PV*>(tile[w] + where[u]) = Piece<SRC>::make(x[w][u], div[w]);
  }
  __syncthreads();
  // Keys: 16 bytes a token and chunk of dims, tokens next to each other.
  const int DC = D / X;
  Walk kat(tid, DC * CT);
  for (; kat.a < nch; kat.next()) {
    const int k = kat.a, j = kat.b % CT, c = kat.b / CT;
    const int4 ch = chunk[k];
    if (j >= ch.y) continue;
    *reinterpret_cast<uint4*>(p.cache[0] + ((((size_t)ch.z * p.KH + kv) * DC + c) * BS + ch.w + j) * 16) =
        *reinterpret_cast<const uint4*>(tile[0] + (ch.x + j) * pitch + c * 16);
  }
  // Values: 4 / E dims a thread.
  const int DW = D / DPW;
  const bool wide = (reinterpret_cast<uintptr_t>(p.cache[1]) & 31) == 0;
  Walk vat(tid, DW);
  for (; vat.a < nch; vat.next()) {
    const int k = vat.a, g = vat.b;
    const int4 ch = chunk[k];
    const int n = ch.y;
    uint8_t* dst = p.cache[1] + ((((size_t)ch.z * p.KH + kv) * D + g * DPW) * BS + ch.w) * E;
    const uint8_t* src = tile[1] + ch.x * pitch + g * 4;
    if (n == CT) {
      uint32_t w[CT];
#pragma unroll
      for (int j = 0; j < CT; ++j) w[j] = *reinterpret_cast<const uint32_t*>(src + j * pitch);
      constexpr int CW = CT * E / 4;  // words of a dim
      if (CW == 4 && BS == CT) {
        // Blocks of one chunk: two dims are 32 bytes.
#pragma unroll
        for (int d = 0; d < DPW; d += 2) {
          uint32_t o[2][CW], both[8];
          gather_dim<E, CT>(w, d, o[0]);
          gather_dim<E, CT>(w, d + (DPW > 1), o[1]);
#pragma unroll
          for (int q = 0; q < 8; ++q) both[q] = o[q / CW % 2][q % CW];
          st_32b(dst + (size_t)d * BS * E, both, wide);
        }
      } else {
#pragma unroll
        for (int d = 0; d < DPW; ++d) {
          uint32_t o[CW];
          gather_dim<E, CT>(w, d, o);
          uint8_t* to = dst + (size_t)d * BS * E;
          if constexpr (CW == 8) st_32b(to, o, wide);
          else if constexpr (CW == 4) *reinterpret_cast<uint4*>(to) = make_uint4(o[0], o[1], o[2], o[3]);
          else *reinterpret_cast<uint2*>(to) = make_uint2(o[0], o[1]);
        }
      }
    } else {
      for (int j = 0; j < n; ++j)
#pragma unroll
        for (int d = 0; d < DPW; ++d)
          *reinterpret_cast<EL*>(dst + ((size_t)d * BS + j) * E) = *reinterpret_cast<const EL*>(src + j * pitch + d * E);
    }
  }
}

template <int SRC, int E, int CT>
cudaError_t launch_write(const WriteParams& prm, cudaStream_t st) {
  WriteParams p = prm;
  // Rows per CTA: as many as still give every SM four CTAs, 2 to 64.
  const long long want = 4ll * device_sm_count();
  p.T = 64;
  while (p.T > 2 && ((long long)p.N + p.T - 1) / p.T * p.KH < want) p.T /= 2;
  const size_t rows = (size_t)p.T + CT - 1;
  const size_t smem = 2 * rows * (p.D * E + 16) + p.T * sizeof(int4);
  const long long tiles = ((long long)p.N + p.T - 1) / p.T;
  static std::atomic<uint64_t> opted_in{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
  if (!bit || !(opted_in.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(cache_write_kernel<SRC, E, CT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    if (e != cudaSuccess) return e;
    opted_in.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles + 1), (unsigned)(tiles > 0 ? p.KH : 1), 1);
  cfg.blockDim = dim3(kWriteThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_write_kernel<SRC, E, CT>, p);
}

// CT: the tokens in 32 bytes of a value row, or the block.
template <int SRC, int E>
cudaError_t by_block(const WriteParams& p, cudaStream_t st) {
  if constexpr (E == 4) {
    return launch_write<SRC, 4, 8>(p, st);
  } else if constexpr (E == 2) {
    return p.BS == 8 ? launch_write<SRC, 2, 8>(p, st) : launch_write<SRC, 2, 16>(p, st);
  } else {
    if (p.BS == 8) return launch_write<SRC, 1, 8>(p, st);
    return p.BS == 16 ? launch_write<SRC, 1, 16>(p, st) : launch_write<SRC, 1, 32>(p, st);
  }
}

// ------------------------------------------------------------------ pa_tree_accept
constexpr int kMaxLayers = 64;      // per launch
constexpr int kAcceptThreads = 256;
constexpr int kBatch = 8;           // moves whose loads are in flight together
constexpr int kMaxPath = 512;

struct AcceptParams {
  const int32_t* bt;
  const int32_t* lens;
  const int32_t* accepted;  // [S, A]
  const int32_t* count;     // [S]
  int32_t* new_lens;        // [S]
  int* hdr;
  int S, n, A, MB, BS, NB, KH, D;
  bool first;               // the launch that writes lengths and status
};
struct AcceptCaches {
  uint8_t* key[kMaxLayers];
  uint8_t* value[kMaxLayers];
};

// Whether a sequence's lengths and path are in range (ids of blocks apart), for
// `threads` threads that look at its path together.
__device__ __forceinline__ bool path_bad(const AcceptParams& p, int s, int i0, int step) {
  const int L = p.lens[s], a = p.count[s];
  if (L < p.n || L > p.MB * p.BS || a < 0 || a > p.A) return true;
  bool bad = false;
  for (int i = i0; i < a; i += step) {
    const int node = p.accepted[(size_t)s * p.A + i];
    const int before = i > 0 ? p.accepted[(size_t)s * p.A + i - 1] : -1;
    // (Each entry by itself: the one before may be anything, and no table entry outside
    // the row is read for what is not a node or a place among the nodes.)
    if (i >= p.n || node < 0 || node <= before || node >= p.n) {
      bad = true;
      continue;
    }
    const int from = p.bt[(size_t)s * p.MB + (L - p.n + node) / p.BS];
    const int to = p.bt[(size_t)s * p.MB + (L - p.n + i) / p.BS];
    bad |= (unsigned)from >= (unsigned)p.NB || (unsigned)to >= (unsigned)p.NB;
  }
  return bad;
}

template <int E>
__global__ void __launch_bounds__(kAcceptThreads)
    tree_accept_kernel(const __grid_constant__ AcceptParams p, const __grid_constant__ AcceptCaches c) {
  using EL = typename Elem<E>::T;
  __shared__ int s_blk[2][kMaxPath], s_off[2][kMaxPath];  // from, to
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int s = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x;
  const int L = p.lens[s];
  const bool bad = __syncthreads_or(path_bad(p, s, tid, kAcceptThreads)) != 0;
  const int a = bad ? 0 : p.count[s], base = L - p.n;
  if (p.first && layer == 0 && blockIdx.z == 0 && tid == 0) p.new_lens[s] = bad ? L : base + a;
  // Where each node of the path is, and where it goes.
  for (int i = tid; i < a; i += kAcceptThreads) {
    const int pos[2] = {base + p.accepted[(size_t)s * p.A + i], base + i};
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      s_blk[w][i] = p.bt[(size_t)s * p.MB + pos[w] / p.BS];
      s_off[w][i] = pos[w] % p.BS;
    }
  }
  __syncthreads();
  const int col = blockIdx.z * kAcceptThreads + tid;
  const int X = 16 / E, DC = p.D / X, keys = p.KH * DC, cols = keys + p.KH * p.D;
  if (a > 0 && col < cols && c.key[layer]) {
    if (col < keys) {
      uint8_t* k = c.key[layer];
      for (int i0 = 0; i0 < a; i0 += kBatch) {
        uint4 v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (i0 + j < a)
            v[j] = *reinterpret_cast<const uint4*>(k + (((size_t)s_blk[0][i0 + j] * keys + col) * p.BS + s_off[0][i0 + j]) * 16);
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (i0 + j < a)
            *reinterpret_cast<uint4*>(k + (((size_t)s_blk[1][i0 + j] * keys + col) * p.BS + s_off[1][i0 + j]) * 16) = v[j];
      }
    } else {
      EL* val = reinterpret_cast<EL*>(c.value[layer]);
      const int d = col - keys, width = p.KH * p.D;
      for (int i0 = 0; i0 < a; i0 += kBatch) {
        EL v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (i0 + j < a) v[j] = val[((size_t)s_blk[0][i0 + j] * width + d) * p.BS + s_off[0][i0 + j]];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (i0 + j < a) val[((size_t)s_blk[1][i0 + j] * width + d) * p.BS + s_off[1][i0 + j]] = v[j];
      }
    }
  }
  if (p.first && s == 0 && layer == 0 && blockIdx.z == 0) {
    // The status: every sequence looked at by this CTA, a thread each, so that no
    // other launch has to clear it.
    bool any = false;
    for (int i = tid; i < p.S; i += kAcceptThreads) any |= path_bad(p, i, 0, 1);
    any = __syncthreads_or(any) != 0;
    if (tid == 0) p.hdr[kHdrError] = any ? kErrDeviceBounds : kOk;
  }
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na > 0 && nb > 0 && x < y + nb && y < x + na;
}

// Whether any two of the caches, `bytes` each, overlap.
bool caches_overlap(void* const* keys, void* const* values, int n, size_t bytes) {
  uintptr_t few[256], *at = few;
  if (2 * (size_t)n > sizeof few / sizeof *few) at = new (std::nothrow) uintptr_t[2 * (size_t)n];
  if (!at) return true;
  for (int i = 0; i < n; ++i) {
    at[2 * i] = reinterpret_cast<uintptr_t>(keys[i]);
    at[2 * i + 1] = reinterpret_cast<uintptr_t>(values[i]);
  }
  std::sort(at, at + 2 * (size_t)n);
  bool found = false;
  for (int i = 1; i < 2 * n; ++i) found |= at[i] - at[i - 1] < bytes;
  if (at != few) delete[] at;
  return found;
}

bool head_size_ok(int D) { return D == 64 || D == 80 || D == 96 || D == 112 || D == 128 || D == 256; }
bool block_size_ok(int BS) { return BS == 8 || BS == 16 || BS == 32 || BS == 64; }

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" int pa_cache_write(void* key_cache, void* value_cache, const void* key, const void* value,
                              const int64_t* slots, float k_scale, float v_scale, int num_tokens,
                              int num_kv_heads, int head_size, int block_size, long long key_stride,
                              long long value_stride, int dtype, int cache_dtype, void* stream, int num_blocks,
                              void* workspace, size_t workspace_bytes) {
  const int D = head_size, BS = block_size;
  if (num_tokens < 0 || num_tokens > INT_MAX - 4096 || num_kv_heads <= 0 || num_kv_heads > 65535 || D <= 0 ||
      BS <= 0 || num_blocks <= 0)
    return PA_ERR_INVALID_ARG;
  if (dtype != PA_DTYPE_FP16 && dtype != PA_DTYPE_BF16 && dtype != PA_DTYPE_FP32) return PA_ERR_INVALID_ARG;
  if (cache_dtype != dtype && cache_dtype != PA_DTYPE_E4M3) return PA_ERR_INVALID_ARG;
  const bool fp8 = cache_dtype == PA_DTYPE_E4M3;
  const auto scale_ok = [](float s) { return s > 0.f && s < INFINITY; };
  if (fp8 ? !scale_ok(k_scale) || !scale_ok(v_scale) : k_scale != 1.f || v_scale != 1.f) return PA_ERR_INVALID_ARG;
  if (!head_size_ok(D) || !block_size_ok(BS)) return PA_ERR_UNSUPPORTED;
  const int esz = dtype == PA_DTYPE_FP32 ? 4 : 2, E = fp8 ? 1 : esz;
  const long long width = (long long)num_kv_heads * D;
  if (key_stride < width || value_stride < width || key_stride * esz % 16 != 0 || value_stride * esz % 16 != 0 ||
      key_stride > LLONG_MAX / 8 || value_stride > LLONG_MAX / 8)
    return PA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 16)) return PA_ERR_INVALID_ARG;
  if (workspace_bytes < kHdrInts * sizeof(int)) return PA_ERR_WORKSPACE;
  if (!key_cache || !value_cache || !aligned(key_cache, 16) || !aligned(value_cache, 16)) return PA_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!key || !value || !slots || !aligned(key, 16) || !aligned(value, 16) || !aligned(slots, 8)))
    return PA_ERR_INVALID_ARG;
  const size_t N = (size_t)num_tokens, cache = (size_t)num_blocks * BS * (size_t)width * E, hdr = kHdrInts * sizeof(int);
  const auto rows = [&](long long stride) { return N > 0 ? ((N - 1) * (size_t)stride + (size_t)width) * esz : 0; };
  // (The first three are written.)
  const struct { const void* p; size_t n; } a[] = {{key_cache, cache},        {value_cache, cache},        {workspace, hdr},
                                                   {key, rows(key_stride)}, {value, rows(value_stride)}, {slots, 8 * N}};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 6; ++j)
      if (overlap(a[i].p, a[i].n, a[j].p, a[j].n)) return PA_ERR_INVALID_ARG;
  WriteParams p = {};
  p.cache[0] = static_cast<uint8_t*>(key_cache);
  p.cache[1] = static_cast<uint8_t*>(value_cache);
  p.row[0] = static_cast<const uint8_t*>(key);
  p.row[1] = static_cast<const uint8_t*>(value);
  p.slots = reinterpret_cast<const long long*>(slots);
  p.hdr = static_cast<int*>(workspace);
  p.stride[0] = key_stride * esz;
  p.stride[1] = value_stride * esz;
  p.total = (long long)num_blocks * BS;
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.N = num_tokens;
  p.KH = num_kv_heads;
  p.D = D;
  p.BS = BS;
  p.shift = BS == 8 ? 3 : BS == 16 ? 4 : BS == 32 ? 5 : 6;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (!fp8) e = E == 2 ? by_block<kCopy, 2>(p, st) : by_block<kCopy, 4>(p, st);
  else if (dtype == PA_DTYPE_FP16) e = by_block<kHalf, 1>(p, st);
  else if (dtype == PA_DTYPE_BF16) e = by_block<kBfloat, 1>(p, st);
  else e = by_block<kFloat, 1>(p, st);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

extern "C" int pa_tree_accept(int32_t* new_lens, void* const* key_caches, void* const* value_caches,
                              int num_caches, const int32_t* block_tables, const int32_t* seq_lens,
                              const int32_t* accepted, const int32_t* num_accepted, int num_seqs, int num_nodes,
                              int max_accepted, int num_kv_heads, int head_size, int block_size, int cache_dtype,
                              void* stream, int max_blocks_per_seq, int num_blocks, void* workspace,
                              size_t workspace_bytes) {
  const int D = head_size, BS = block_size, S = num_seqs;
  if (S < 0 || num_nodes < 1 || num_nodes > kMaxPath || max_accepted < 0 || max_accepted > kMaxPath ||
      num_kv_heads <= 0 || num_kv_heads > 65535 || D <= 0 || BS <= 0 || max_blocks_per_seq <= 0 ||
      num_blocks <= 0 || num_caches < 0 || (long long)max_blocks_per_seq * BS > INT_MAX / 2)
    return PA_ERR_INVALID_ARG;
  if (cache_dtype != PA_DTYPE_FP16 && cache_dtype != PA_DTYPE_BF16 && cache_dtype != PA_DTYPE_FP32 &&
      cache_dtype != PA_DTYPE_E4M3)
    return PA_ERR_INVALID_ARG;
  if (!head_size_ok(D) || !block_size_ok(BS)) return PA_ERR_UNSUPPORTED;
  if (!workspace || !aligned(workspace, 16)) return PA_ERR_INVALID_ARG;
  if (workspace_bytes < kHdrInts * sizeof(int)) return PA_ERR_WORKSPACE;
  if (num_caches > 0 && (!key_caches || !value_caches)) return PA_ERR_INVALID_ARG;
  for (int i = 0; i < num_caches; ++i)
    if (!key_caches[i] || !value_caches[i] || !aligned(key_caches[i], 16) || !aligned(value_caches[i], 16))
      return PA_ERR_INVALID_ARG;
  if (S == 0) return PA_OK;
  if (!new_lens || !block_tables || !seq_lens || !num_accepted || !aligned(new_lens, 4) ||
      !aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(num_accepted, 4) ||
      (max_accepted > 0 && (!accepted || !aligned(accepted, 4))))
    return PA_ERR_INVALID_ARG;
  const size_t s4 = 4 * (size_t)S;
  const struct { const void* p; size_t n; } a[] = {
      {block_tables, s4 * max_blocks_per_seq}, {seq_lens, s4}, {accepted, s4 * max_accepted}, {num_accepted, s4},
      {workspace, kHdrInts * sizeof(int)}};
  for (const auto& x : a)
    if (overlap(new_lens, s4, x.p, x.n) || (x.p != workspace && overlap(workspace, kHdrInts * sizeof(int), x.p, x.n)))
      return PA_ERR_INVALID_ARG;
  const int E = cache_dtype == PA_DTYPE_E4M3 ? 1 : cache_dtype == PA_DTYPE_FP32 ? 4 : 2;
  const size_t bytes = (size_t)num_blocks * num_kv_heads * D * BS * E;
  if (caches_overlap(key_caches, value_caches, num_caches, bytes)) return PA_ERR_INVALID_ARG;
  for (int i = 0; i < num_caches; ++i)
    for (const void* c : {key_caches[i], value_caches[i]}) {
      if (overlap(new_lens, s4, c, bytes)) return PA_ERR_INVALID_ARG;
      for (const auto& x : a)
        if (overlap(c, bytes, x.p, x.n)) return PA_ERR_INVALID_ARG;
    }
  AcceptParams p = {};
  p.bt = block_tables;
  p.lens = seq_lens;
  p.accepted = accepted;
  p.count = num_accepted;
  p.new_lens = new_lens;
  p.hdr = static_cast<int*>(workspace);
  p.S = S;
  p.n = num_nodes;
  p.A = max_accepted;
  p.MB = max_blocks_per_seq;
  p.BS = BS;
  p.NB = num_blocks;
  p.KH = num_kv_heads;
  p.D = D;
  const long long cols = (long long)num_kv_heads * (D * E / 16 + D);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kAcceptThreads, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  for (int c0 = 0; c0 == 0 || c0 < num_caches; c0 += kMaxLayers) {
    AcceptCaches c;
    std::memset(&c, 0, sizeof c);
    const int n = num_caches - c0 < kMaxLayers ? num_caches - c0 : kMaxLayers;
    for (int i = 0; i < n; ++i) {
      c.key[i] = static_cast<uint8_t*>(key_caches[c0 + i]);
      c.value[i] = static_cast<uint8_t*>(value_caches[c0 + i]);
    }
    p.first = c0 == 0;
    cfg.gridDim = dim3((unsigned)S, (unsigned)(n > 0 ? n : 1), (unsigned)((cols + kAcceptThreads - 1) / kAcceptThreads));
    const cudaError_t e = E == 1   ? cudaLaunchKernelEx(&cfg, tree_accept_kernel<1>, p, c)
                          : E == 2 ? cudaLaunchKernelEx(&cfg, tree_accept_kernel<2>, p, c)
                                   : cudaLaunchKernelEx(&cfg, tree_accept_kernel<4>, p, c);
    if (e != cudaSuccess) return PA_ERR_CUDA;
  }
  return PA_OK;
}
