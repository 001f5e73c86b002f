// pa_pages.cu -- pages of a cache pool: sequences forked, grown, truncated and
// freed, and the pool compacted (include/pa_decode.h: pa_pages_fork,
// pa_pages_resize, pa_pages_compact).
//
// The state of a pool is one count per block, the table rows that hold it; a
// block of count 0 is free.  Every call is two launches:
//
//   plan   one thread-block cluster.  Its first CTA works out what each row
//          needs and numbers the needs in row order (a block scan); the whole
//          cluster looks through the counts, 32 ids a thread as a bit mask,
//          numbers the free ids (counts exchanged through distributed shared
//          memory) and lists the lowest ones.  It stops at the last id needed.
//          It also leaves the call's status: a call that the pool cannot serve
//          changes nothing.
//   apply  the whole GPU: table entries and counts, 256 entries a warp, and
//          the pages to be copied, 4 KB a warp and step.
//
// What bounds them: a call that copies many pages, the memory (each page read
// and written once); a call that copies few, the two launches and the
// dependent loads of the plan.
#include <cooperative_groups.h>

#include <climits>
#include <cstring>

#include "pa_common.cuh"
#include "pa_decode.h"
#include "pa_launch.h"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kErrNoBlocks = 7;
static_assert(kErrNoBlocks == PA_ERR_NO_BLOCKS, "status codes");

// Header words after the error word.
constexpr int kHdrGo = 8;      // 1: apply the plan
constexpr int kHdrCopies = 9;  // pages to copy
constexpr int kHdrUsed = 10;   // compact: blocks in use

enum Mode { kFork, kResize, kCompact };

constexpr int kCluster = 8, kPlanThreads = 1024;
constexpr int kApplyThreads = 256;
constexpr int kEntries = 256;                     // table entries per warp job
constexpr int kCopyUnroll = 8;                    // 16-byte words per lane and job
constexpr uint32_t kCopyBytes = 32 * 16 * kCopyUnroll;
constexpr int kMaxCaches = 128;                   // per launch

struct PagesParams {
  int32_t* bt;          // [S, MB]
  int32_t* lens;        // [S]
  const int32_t* arg;   // fork: parents [rows]; resize: new lengths [rows]
  int32_t* bt_out;      // fork: [rows, MB]
  int32_t* lens_out;    // fork: [rows]
  int32_t* refs;        // [NB]
  int32_t* new_ids;     // compact: [NB] or null
  int* hdr;
  int* row_old;         // [rows] length before the call (resize: -1 for a row left alone)
  int* row_first;       // [rows] number of the row's first new block
  int* row_cow;         // [rows] 1: its partly filled block is replaced by a copy
  int* copy_rank;       // [copies] number of the destination
  int* copy_src;        // [copies]
  int* ids;             // listed free blocks, lowest first
  int* rank_of;         // compact: [NB] number of the move of a block at or above `used`
  int S, rows, MB, BS, NB;
};

struct CopyParams {
  uint8_t* base[kMaxCaches];
  unsigned long long bytes[kMaxCaches];  // per page
  uint32_t first[kMaxCaches + 1];        // warp jobs of a page before this cache
  int n;
};

__device__ __forceinline__ void record(const PagesParams& p) {
  atomicCAS(p.hdr + kHdrError, 0, kErrDeviceBounds);
}

// Exclusive scan over the CTA; *total is its sum.  `tmp`: 33 words of shared memory.
template <typename V>
__device__ __forceinline__ V block_scan(V v, V* total, V* tmp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  V incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  __syncthreads();  // tmp is free
  if (lane == 31) tmp[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const V t = tmp[lane];
    V ti = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const V n = __shfl_up_sync(0xffffffffu, ti, o);
      if (lane >= o) ti += n;
    }
    tmp[lane] = ti - t;
    if (lane == 31) tmp[32] = ti;
  }
  __syncthreads();
  *total = tmp[32];
  return tmp[warp] + incl - v;
}

// Bit i: block id0 + i exists and is in use.
__device__ __forceinline__ uint32_t used_mask(const PagesParams& p, long long id0) {
  uint32_t m = 0;
  if (id0 + 32 <= p.NB && (reinterpret_cast<uintptr_t>(p.refs) & 15) == 0) {
    int4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = reinterpret_cast<const int4*>(p.refs + id0)[i];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      m |= (uint32_t)(v[i].x > 0) << (4 * i) | (uint32_t)(v[i].y > 0) << (4 * i + 1) |
           (uint32_t)(v[i].z > 0) << (4 * i + 2) | (uint32_t)(v[i].w > 0) << (4 * i + 3);
  } else {
    for (int i = 0; i < 32 && id0 + i < p.NB; ++i) m |= (uint32_t)(p.refs[id0 + i] > 0) << i;
  }
  return m;
}
// Bit i: block id0 + i exists.
__device__ __forceinline__ uint32_t valid_mask(const PagesParams& p, long long id0) {
  const long long n = p.NB - id0;
  return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

// What row i needs: *n new blocks, *src the block to copy (-1: none).
// Returns false for a row that is refused.
template <int MODE>
__device__ __forceinline__ bool plan_row(const PagesParams& p, int i, int* n, int* src) {
  const int cap = p.MB * p.BS;
  *n = 0;
  *src = -1;
  if constexpr (MODE == kFork) {
    const int par = p.arg[i];
    p.row_old[i] = 0;
    if (par == -1) return true;  // an empty row
    if (par < -1 || par >= p.S) return false;
    const int L = p.lens[par];
    if (L < 0 || L > cap) return false;
    if (L % p.BS != 0) {
      const int b = p.bt[(size_t)par * p.MB + L / p.BS];
      if ((unsigned)b >= (unsigned)p.NB) return false;
      *n = 1;
      *src = b;
    }
    p.row_old[i] = L;
    return true;
  } else {
    const int L = p.lens[i], N = p.arg[i];
    p.row_old[i] = -1;
    if (L < 0 || L > cap || N < 0 || N > cap) return false;
    const int keep = min(L, N), oldB = (L + p.BS - 1) / p.BS, newB = (N + p.BS - 1) / p.BS;
    if (keep % p.BS != 0) {
      const int b = p.bt[(size_t)i * p.MB + keep / p.BS];
      if ((unsigned)b >= (unsigned)p.NB) return false;
      if (p.refs[b] > 1) {
        *src = b;
        *n = 1;
      }
    }
    *n += max(0, newB - oldB);
    p.row_old[i] = L;
    return true;
  }
}

template <int MODE>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads, 1)
    pages_plan_kernel(const __grid_constant__ PagesParams p) {
  __shared__ unsigned long long tmp[33];
  __shared__ unsigned long long shared_count[2];
  __shared__ long long shared_need;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), tid = threadIdx.x;
  const long long round = (long long)kCluster * kPlanThreads * 32;

  if constexpr (MODE != kCompact) {
    int bad = 0, copies = 0;
    if (rank == 0) {
      long long need = 0;
      for (int r0 = 0; r0 < p.rows; r0 += kPlanThreads) {
        const int i = r0 + tid;
        int n = 0, src = -1;
        if (i < p.rows) bad |= !plan_row<MODE>(p, i, &n, &src);
        // Needs and copies in one scan (a row needs at most 2^30 / BS + 1 blocks).
        unsigned long long total;
        const unsigned long long mine = (unsigned long long)n << 20 | (src >= 0 ? 1u : 0u);
        const unsigned long long before = block_scan(mine, &total, tmp);
        if (i < p.rows) {
          const long long first = need + (long long)(before >> 20);
          p.row_first[i] = (int)min(first, (long long)INT_MAX);
          p.row_cow[i] = src >= 0;
          if (src >= 0) {
            const int k = copies + (int)(before & 0xfffffu);
            p.copy_src[k] = src;
            p.copy_rank[k] = (int)min(first, (long long)INT_MAX);
          }
        }
        need += (long long)(total >> 20);
        copies += (int)(total & 0xfffffu);
      }
      if (tid == 0) shared_need = need;
      bad = __syncthreads_or(bad);
    }
    cl.sync();
    const long long need = *cl.map_shared_rank(&shared_need, 0);
    long long found = 0;
    int par = 0;
    for (long long base = 0; base < p.NB && found < need; base += round, par ^= 1) {
      const long long id0 = base + ((long long)rank * kPlanThreads + tid) * 32;
      uint32_t m = id0 < p.NB ? ~used_mask(p, id0) & valid_mask(p, id0) : 0u;
      unsigned long long total;
      const unsigned long long before = block_scan((unsigned long long)__popc(m), &total, tmp);
      if (tid == 0) shared_count[par] = total;
      cl.sync();
      long long pos = found + (long long)before;
      for (int q = 0; q < kCluster; ++q) {
        const long long c = (long long)*cl.map_shared_rank(&shared_count[par], q);
        if (q < rank) pos += c;
        found += c;
      }
      for (; m && pos < need; m &= m - 1, ++pos) p.ids[pos] = (int)(id0 + __ffs(m) - 1);
    }
    if (rank == 0 && tid == 0) {
      const bool enough = found >= need;
      p.hdr[kHdrError] = !enough ? kErrNoBlocks : bad ? kErrDeviceBounds : kOk;
      p.hdr[kHdrGo] = enough;
      p.hdr[kHdrCopies] = enough ? copies : 0;
    }
  } else {
    // Blocks in use, then the free ids below that number and the used ones
    // from it on (equally many), both ascending.
    unsigned long long n = 0, total;
    for (long long id0 = ((long long)rank * kPlanThreads + tid) * 32; id0 < p.NB; id0 += round)
      n += __popc(used_mask(p, id0));
    block_scan(n, &total, tmp);
    if (tid == 0) shared_count[1] = total;
    cl.sync();
    long long used = 0;
    for (int q = 0; q < kCluster; ++q) used += (long long)*cl.map_shared_rank(&shared_count[1], q);
    long long below = 0, above = 0;
    int par = 0;
    for (long long base = 0; base < p.NB; base += round, par ^= 1) {
      const long long id0 = base + ((long long)rank * kPlanThreads + tid) * 32;
      const uint32_t valid = valid_mask(p, id0), u = id0 < p.NB ? used_mask(p, id0) : 0u;
      const long long nb = used - id0;
      const uint32_t front = nb >= 32 ? 0xffffffffu : nb <= 0 ? 0u : (1u << nb) - 1u;  // ids below `used`
      uint32_t holes = ~u & valid & front, movers = u & ~front;
      const unsigned long long mine = (unsigned long long)__popc(holes) << 32 | __popc(movers);
      const unsigned long long before = block_scan(mine, &total, tmp);
      if (tid == 0) shared_count[par] = total;
      cl.sync();
      long long h = below + (long long)(before >> 32), m = above + (long long)(before & 0xffffffffu);
      for (int q = 0; q < kCluster; ++q) {
        const unsigned long long c = *cl.map_shared_rank(&shared_count[par], q);
        if (q < rank) {
          h += (long long)(c >> 32);
          m += (long long)(c & 0xffffffffu);
        }
        below += (long long)(c >> 32);
        above += (long long)(c & 0xffffffffu);
      }
      for (; holes; holes &= holes - 1) p.ids[h++] = (int)(id0 + __ffs(holes) - 1);
      for (int i = 0; i < 32 && id0 + i < p.NB; ++i) {
        const bool is_used = (u >> i) & 1u, is_front = (front >> i) & 1u;
        if (!is_front) p.rank_of[id0 + i] = is_used ? (int)m : -1;
        if (p.new_ids && (is_front || !is_used)) p.new_ids[id0 + i] = is_used ? (int)(id0 + i) : -1;
        if (!is_front && is_used) p.copy_src[m++] = (int)(id0 + i);
      }
    }
    if (rank == 0 && tid == 0) {
      p.hdr[kHdrError] = kOk;
      p.hdr[kHdrGo] = 1;
      p.hdr[kHdrCopies] = (int)above;
      p.hdr[kHdrUsed] = (int)used;
    }
  }
  cl.sync();  // no CTA leaves while its shared memory may be read
}

// One table row's job: entries [j0, j0 + kEntries) of what the row changes.
template <int MODE>
__device__ __forceinline__ void apply_row(const PagesParams& p, int i, int j0, int lane) {
  if constexpr (MODE == kFork) {
    const int L = p.row_old[i], full = L / p.BS, part = L % p.BS != 0;
    if (j0 == 0 && lane == 0) p.lens_out[i] = L;
    if (j0 >= full + part) return;
    const int32_t* src = p.bt + (size_t)p.arg[i] * p.MB;
    int32_t* dst = p.bt_out + (size_t)i * p.MB;
    int id[kEntries / 32];
#pragma unroll
    for (int k = 0; k < kEntries / 32; ++k) {
      const int j = j0 + k * 32 + lane;
      id[k] = j < full ? src[j] : 0;
    }
#pragma unroll
    for (int k = 0; k < kEntries / 32; ++k) {
      const int j = j0 + k * 32 + lane;
      if (j < full) {
        if ((unsigned)id[k] < (unsigned)p.NB) atomicAdd(p.refs + id[k], 1);
        else record(p);
        dst[j] = id[k];
      } else if (j == full && part) {
        const int b = p.ids[p.row_first[i]];
        p.refs[b] = 1;
        dst[j] = b;
      }
    }
  } else if constexpr (MODE == kResize) {
    const int L = p.row_old[i];
    if (L < 0) return;
    const int N = p.arg[i], cow = p.row_cow[i], first = p.row_first[i];
    if (j0 == 0 && lane == 0) p.lens[i] = N;
    const int oldB = (L + p.BS - 1) / p.BS, newB = (N + p.BS - 1) / p.BS;
    const int lo = min(oldB, newB) - cow, hi = max(oldB, newB);
    int32_t* row = p.bt + (size_t)i * p.MB;
    for (int j = lo + j0 + lane; j < min(hi, lo + j0 + kEntries); j += 32) {
      const bool edge = cow && j == lo;
      if (edge || j < oldB) {  // given back
        const int b = row[j];
        if ((unsigned)b >= (unsigned)p.NB) {
          record(p);
        } else if (atomicSub(p.refs + b, 1) <= 0) {
          atomicAdd(p.refs + b, 1);
          record(p);
        }
      }
      if (edge || j >= oldB) {  // taken
        const int b = p.ids[first + (edge ? 0 : cow + j - oldB)];
        p.refs[b] = 1;
        row[j] = b;
      }
    }
  } else {
    const int used = p.hdr[kHdrUsed], L = p.lens[i], cap = p.MB * p.BS;
    if ((L < 0 || L > cap) && j0 == 0 && lane == 0) record(p);
    const int n = (min(max(L, 0), cap) + p.BS - 1) / p.BS;
    int32_t* row = p.bt + (size_t)i * p.MB;
    for (int j = j0 + lane; j < min(n, j0 + kEntries); j += 32) {
      const int b = row[j];
      if ((unsigned)b >= (unsigned)p.NB) {
        record(p);
      } else if (b >= used) {
        const int r = p.rank_of[b];
        if (r < 0) record(p);  // a table holds a free block
        else row[j] = p.ids[r];
      }
    }
  }
}

// `books`: also the tables and counts (the first launch of a call; further
// ones copy the pages of caches past kMaxCaches).
template <int MODE>
__global__ void __launch_bounds__(kApplyThreads)
    pages_apply_kernel(const __grid_constant__ PagesParams p, const __grid_constant__ CopyParams c, bool books) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!p.hdr[kHdrGo]) return;
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (kApplyThreads / 32);
  const long long w = (long long)blockIdx.x * (kApplyThreads / 32) + (threadIdx.x >> 5);
  const int copies = p.hdr[kHdrCopies];
  if (books) {
    const int chunks = (p.MB + kEntries - 1) / kEntries;
    for (long long job = w; job < (long long)p.rows * chunks; job += warps)
      apply_row<MODE>(p, (int)(job / chunks), (int)(job % chunks) * kEntries, lane);
    if constexpr (MODE == kCompact) {
      for (long long k = w * 32 + lane; k < copies; k += warps * 32) {
        const int src = p.copy_src[k], dst = p.ids[k];
        p.refs[dst] = p.refs[src];
        p.refs[src] = 0;
        if (p.new_ids) p.new_ids[src] = dst;
      }
    }
  }
  const uint32_t per = c.first[c.n];
  // The copies start at the far end of the grid's warps: those have no row.
  for (long long job = warps - 1 - w; job < (long long)copies * per; job += warps) {
    const int k = (int)(job / per);
    const uint32_t r = (uint32_t)(job - (long long)k * per);
    int lo = 0, hi = c.n;  // first[lo] <= r < first[lo + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (c.first[mid] <= r) lo = mid; else hi = mid;
    }
    const unsigned long long page = c.bytes[lo];
    const unsigned long long at = (unsigned long long)(r - c.first[lo]) * kCopyBytes + lane * 16;
    const int dst = MODE == kCompact ? p.ids[k] : p.ids[p.copy_rank[k]];
    const uint8_t* s = c.base[lo] + (unsigned long long)p.copy_src[k] * page;
    uint8_t* d = c.base[lo] + (unsigned long long)dst * page;
    uint4 v[kCopyUnroll];
#pragma unroll
    for (int i = 0; i < kCopyUnroll; ++i)
      if (at + i * 512 < page) v[i] = *reinterpret_cast<const uint4*>(s + at + i * 512);
#pragma unroll
    for (int i = 0; i < kCopyUnroll; ++i)
      if (at + i * 512 < page) *reinterpret_cast<uint4*>(d + at + i * 512) = v[i];
  }
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

struct PagesLayout {
  size_t old, first, cow, rank, src, ids, rank_of, total;
};
bool pages_layout(int rows, int MB, int NB, PagesLayout* l) {
  if (rows < 0 || MB <= 0 || NB <= 0) return false;
  const size_t r = align_up((size_t)rows * 4), b = align_up((size_t)NB * 4);
  l->old = kHdrInts * sizeof(int);
  l->first = l->old + r;
  l->cow = l->first + r;
  l->rank = l->cow + r;
  l->src = l->rank + r;
  l->ids = l->src + (r > b ? r : b);
  l->rank_of = l->ids + b;
  l->total = l->rank_of + b;
  return true;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

template <int MODE>
int pages_impl(PagesParams p, void* const* caches, const size_t* page_bytes, int num_caches, void* stream,
               void* workspace, size_t workspace_bytes) {
  if (p.S < 0 || p.rows < 0 || p.MB <= 0 || p.BS <= 0 || p.NB <= 0 || num_caches < 0 ||
      (long long)p.MB * p.BS > INT_MAX / 2 || p.rows >= (1 << 24))
    return PA_ERR_INVALID_ARG;
  if (!p.refs || !aligned(p.refs, 4) || (p.new_ids && !aligned(p.new_ids, 4))) return PA_ERR_INVALID_ARG;
  if (p.S > 0 && (!p.bt || !p.lens || !aligned(p.bt, 4) || !aligned(p.lens, 4))) return PA_ERR_INVALID_ARG;
  if (MODE != kCompact && p.rows > 0 && (!p.arg || !aligned(p.arg, 4))) return PA_ERR_INVALID_ARG;
  if (MODE == kFork && p.rows > 0) {
    if (!p.bt_out || !p.lens_out || !aligned(p.bt_out, 4) || !aligned(p.lens_out, 4)) return PA_ERR_INVALID_ARG;
    const size_t row = (size_t)p.MB * 4;
    if (p.S > 0 && (overlap(p.bt, p.S * row, p.bt_out, p.rows * row) ||
                    overlap(p.lens, (size_t)p.S * 4, p.lens_out, (size_t)p.rows * 4)))
      return PA_ERR_INVALID_ARG;
  }
  if (num_caches > 0 && (!caches || !page_bytes)) return PA_ERR_INVALID_ARG;
  for (int i = 0; i < num_caches; ++i)
    if (!caches[i] || !aligned(caches[i], 16) || page_bytes[i] == 0 || page_bytes[i] % 16 != 0 ||
        page_bytes[i] > (size_t)1 << 36)
      return PA_ERR_INVALID_ARG;
  PagesLayout l;
  if (!pages_layout(p.rows, p.MB, p.NB, &l)) return PA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 16)) return PA_ERR_INVALID_ARG;
  if (workspace_bytes < l.total) return PA_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.hdr = reinterpret_cast<int*>(ws);
  p.row_old = reinterpret_cast<int*>(ws + l.old);
  p.row_first = reinterpret_cast<int*>(ws + l.first);
  p.row_cow = reinterpret_cast<int*>(ws + l.cow);
  p.copy_rank = reinterpret_cast<int*>(ws + l.rank);
  p.copy_src = reinterpret_cast<int*>(ws + l.src);
  p.ids = reinterpret_cast<int*>(ws + l.ids);
  p.rank_of = reinterpret_cast<int*>(ws + l.rank_of);

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(kCluster, 1, 1);
  cfg.blockDim = dim3(kPlanThreads, 1, 1);
  if (cudaLaunchKernelEx(&cfg, pages_plan_kernel<MODE>, p) != cudaSuccess) return PA_ERR_CUDA;
  cfg.gridDim = dim3((unsigned)device_sm_count() * 4, 1, 1);
  cfg.blockDim = dim3(kApplyThreads, 1, 1);
  for (int c0 = 0; c0 == 0 || c0 < num_caches; c0 += kMaxCaches) {
    CopyParams c;
    std::memset(&c, 0, sizeof c);
    c.n = num_caches - c0 < kMaxCaches ? num_caches - c0 : kMaxCaches;
    for (int i = 0; i < c.n; ++i) {
      c.base[i] = static_cast<uint8_t*>(caches[c0 + i]);
      c.bytes[i] = page_bytes[c0 + i];
      c.first[i + 1] = c.first[i] + (uint32_t)((page_bytes[c0 + i] + kCopyBytes - 1) / kCopyBytes);
    }
    if (cudaLaunchKernelEx(&cfg, pages_apply_kernel<MODE>, p, c, c0 == 0) != cudaSuccess) return PA_ERR_CUDA;
  }
  return PA_OK;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_pages_workspace_bytes(int num_rows, int max_blocks_per_seq, int num_blocks) {
  PagesLayout l;
  return pages_layout(num_rows, max_blocks_per_seq, num_blocks, &l) ? l.total : 0;
}

extern "C" int pa_pages_fork(int32_t* block_tables_out, int32_t* seq_lens_out, const int32_t* block_tables,
                             const int32_t* seq_lens, const int32_t* parents, int32_t* refcounts,
                             void* const* caches, const size_t* page_bytes, int num_caches, int num_seqs,
                             int num_children, int max_blocks_per_seq, int block_size, int num_blocks,
                             void* stream, void* workspace, size_t workspace_bytes) {
  PagesParams p = {};
  p.bt = const_cast<int32_t*>(block_tables);
  p.lens = const_cast<int32_t*>(seq_lens);
  p.arg = parents;
  p.bt_out = block_tables_out;
  p.lens_out = seq_lens_out;
  p.refs = refcounts;
  p.S = num_seqs;
  p.rows = num_children;
  p.MB = max_blocks_per_seq;
  p.BS = block_size;
  p.NB = num_blocks;
  return pages_impl<kFork>(p, caches, page_bytes, num_caches, stream, workspace, workspace_bytes);
}

extern "C" int pa_pages_resize(int32_t* block_tables, int32_t* seq_lens, const int32_t* new_lens,
                               int32_t* refcounts, void* const* caches, const size_t* page_bytes, int num_caches,
                               int num_seqs, int max_blocks_per_seq, int block_size, int num_blocks, void* stream,
                               void* workspace, size_t workspace_bytes) {
  PagesParams p = {};
  p.bt = block_tables;
  p.lens = seq_lens;
  p.arg = new_lens;
  p.refs = refcounts;
  p.S = p.rows = num_seqs;
  p.MB = max_blocks_per_seq;
  p.BS = block_size;
  p.NB = num_blocks;
  return pages_impl<kResize>(p, caches, page_bytes, num_caches, stream, workspace, workspace_bytes);
}

extern "C" int pa_pages_compact(int32_t* block_tables, const int32_t* seq_lens, int32_t* refcounts,
                                int32_t* new_ids, void* const* caches, const size_t* page_bytes, int num_caches,
                                int num_seqs, int max_blocks_per_seq, int block_size, int num_blocks, void* stream,
                                void* workspace, size_t workspace_bytes) {
  PagesParams p = {};
  p.bt = block_tables;
  p.lens = const_cast<int32_t*>(seq_lens);
  p.refs = refcounts;
  p.new_ids = new_ids;
  p.S = p.rows = num_seqs;
  p.MB = max_blocks_per_seq;
  p.BS = block_size;
  p.NB = num_blocks;
  return pages_impl<kCompact>(p, caches, page_bytes, num_caches, stream, workspace, workspace_bytes);
}
