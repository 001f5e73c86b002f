// pa_pages.cu -- pages of a cache pool: sequences forked, grown, truncated and
// freed, and the pool compacted (include/pa_decode.h: pa_pages_fork,
// pa_pages_resize, pa_pages_compact).
//
// The state of a pool is one count per block, the table rows that hold it; a
// block of count 0 is free.  Every call is two launches:
//
//   plan   one thread-block cluster.  Its first CTA works out what each row
//          needs and numbers the needs in row order (a block scan); the whole
//          cluster looks through the counts, up to 1024 ids a warp as bit masks
//          of 32 (one a lane), numbers the free ids (counts exchanged through
//          distributed shared memory) and lists the lowest ones, a warp a mask
//          at a time so that what it writes is contiguous.  It stops at the
//          last id needed.  The counts are on their way while the rows are
//          looked at.  It also leaves the call's status: a call that the pool
//          cannot serve changes nothing.
//   apply  the whole GPU: table entries and counts, 128 entries a warp, and
//          the pages to be copied, 2 KB a warp and step.
//
// What bounds them: a call that copies many pages, the memory (each page read
// and written once); a call that copies few, the two launches and the
// dependent loads of the plan.  Measured (GB300): 4 GB of pages of eight caches
// compacted, 325 us for 1.97 GB read and written, 90% of the measured copy rate
// (6766 GB/s); 512 rows resized in a pool of 262144 blocks 23 us, 37 with the
// ids listed by one lane each.
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
constexpr int kPer = 4, kEntries = 32 * kPer;      // table entries per lane and warp job
constexpr int kCopyUnroll = 4;                    // 16-byte words per lane and job
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
  uint32_t first[kMaxCaches + 1];        // warp jobs of a page before this cache (pages_impl bounds a page)
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

// Ids are looked through in rounds; in a round a warp has `steps` groups of 32
// ids from its first on, and lane l < steps holds group l's mask (bit i: the
// i-th block is in use).  Eight groups' counts are loaded at a time.
struct Groups {
  int steps;
  __device__ __forceinline__ explicit Groups(int NB) {
    constexpr int warps = kCluster * kPlanThreads / 32;
    steps = min(32, max(1, (NB + warps * 32 - 1) / (warps * 32)));
  }
  __device__ __forceinline__ long long ids_per_warp() const { return 32ll * steps; }
  __device__ __forceinline__ void load(const PagesParams& p, long long first, int s0, int lane, int (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const long long id = first + 32 * (s0 + j) + lane;
      v[j] = s0 + j < steps && id < p.NB ? p.refs[id] : 0;
    }
  }
  // (v: the first eight groups, loaded already, or null.)
  __device__ __forceinline__ uint32_t used(const PagesParams& p, long long first, int lane,
                                           const int (*ready)[8]) const {
    uint32_t m = 0;
    for (int s0 = 0; s0 < steps; s0 += 8) {
      int v[8];
      if (ready && s0 == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (*ready)[j];
      } else {
        load(p, first, s0, lane, v);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t b = __ballot_sync(0xffffffffu, v[j] > 0);
        if (lane == s0 + j) m = b;
      }
    }
    return m;
  }
  // Bit i: the lane's group has an i-th block.
  __device__ __forceinline__ uint32_t valid(const PagesParams& p, long long first, int lane) const {
    const long long n = lane < steps ? p.NB - (first + 32 * lane) : 0;
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
  }
  // Warp: the ids of the lanes' masks into list[number], the lane's first one
  // being number `pos`, numbers below `end` only.
  __device__ __forceinline__ void list(int* out, uint32_t mask, long long pos, long long end, long long first,
                                       int lane) const {
    const uint32_t before = (1u << lane) - 1u;
    for (uint32_t left = __ballot_sync(0xffffffffu, mask != 0); left; left &= left - 1) {
      const int l = __ffs(left) - 1;
      const uint32_t m = __shfl_sync(0xffffffffu, mask, l);
      const long long at = __shfl_sync(0xffffffffu, pos, l);
      if (at >= end) break;
      const long long k = at + __popc(m & before);
      if (((m >> lane) & 1u) && k < end) out[k] = (int)first + 32 * l + lane;
    }
  }
};

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
  __shared__ long long shared_need;  // (of the first CTA)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), tid = threadIdx.x, lane = tid & 31;
  const Groups groups(p.NB);
  const long long round = groups.ids_per_warp() * (kCluster * kPlanThreads / 32);
  const long long warp_first = groups.ids_per_warp() * (rank * (kPlanThreads / 32) + (tid >> 5));
  int ready[8];
  groups.load(p, warp_first, 0, lane, ready);

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
    long long need = LLONG_MAX, found = 0;
    int par = 0;
    for (long long base = 0; base < p.NB && found < need; base += round, par ^= 1) {
      const long long first = base + warp_first;
      const uint32_t m = ~groups.used(p, first, lane, base == 0 ? &ready : nullptr) & groups.valid(p, first, lane);
      unsigned long long total;
      const unsigned long long before = block_scan((unsigned long long)__popc(m), &total, tmp);
      if (tid == 0) shared_count[par] = total;
      cl.sync();
      need = *cl.map_shared_rank(&shared_need, 0);
      long long pos = found + (long long)before;
#pragma unroll
      for (int q = 0; q < kCluster; ++q) {
        const long long c = (long long)*cl.map_shared_rank(&shared_count[par], q);
        if (q < rank) pos += c;
        found += c;
      }
      groups.list(p.ids, m, pos, need, first, lane);
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
    const uint32_t u_first = groups.used(p, warp_first, lane, &ready);
    unsigned long long n = __popc(u_first), total;
    for (long long base = round; base < p.NB; base += round)
      n += __popc(groups.used(p, base + warp_first, lane, nullptr));
    block_scan(n, &total, tmp);
    if (tid == 0) shared_count[1] = total;
    cl.sync();
    long long used = 0;
#pragma unroll
    for (int q = 0; q < kCluster; ++q) used += (long long)*cl.map_shared_rank(&shared_count[1], q);
    long long below = 0, above = 0;
    int par = 0;
    for (long long base = 0; base < p.NB; base += round, par ^= 1) {
      const long long first = base + warp_first;
      const uint32_t u = base == 0 ? u_first : groups.used(p, first, lane, nullptr);
      const long long nb = used - (first + 32 * lane);
      const uint32_t front = nb >= 32 ? 0xffffffffu : nb <= 0 ? 0u : (1u << nb) - 1u;  // ids below `used`
      const uint32_t holes = ~u & groups.valid(p, first, lane) & front, movers = u & ~front;
      const unsigned long long mine = (unsigned long long)__popc(holes) << 32 | __popc(movers);
      const unsigned long long before = block_scan(mine, &total, tmp);
      if (tid == 0) shared_count[par] = total;
      cl.sync();
      long long h = below + (long long)(before >> 32), m = above + (long long)(before & 0xffffffffu);
#pragma unroll
      for (int q = 0; q < kCluster; ++q) {
        const unsigned long long c = *cl.map_shared_rank(&shared_count[par], q);
        if (q < rank) {
          h += (long long)(c >> 32);
          m += (long long)(c & 0xffffffffu);
        }
        below += (long long)(c >> 32);
        above += (long long)(c & 0xffffffffu);
      }
      groups.list(p.ids, holes, h, LLONG_MAX, first, lane);
      groups.list(p.copy_src, movers, m, LLONG_MAX, first, lane);
      // Numbers of the moves, and (but for the moved blocks) the new ids.
      for (int l = 0; l < groups.steps && first + 32 * l < p.NB; ++l) {
        if (!p.new_ids && first + 32 * l + 31 < used) continue;
        const long long id = first + 32 * l + lane;
        const uint32_t mv = __shfl_sync(0xffffffffu, movers, l), us = __shfl_sync(0xffffffffu, u, l);
        const long long at = __shfl_sync(0xffffffffu, m, l);
        if (id >= p.NB) continue;
        const bool is_used = (us >> lane) & 1u;
        if (id >= used) p.rank_of[id] = is_used ? (int)at + __popc(mv & ((1u << lane) - 1u)) : -1;
        if (p.new_ids && !(id >= used && is_used)) p.new_ids[id] = is_used ? (int)id : -1;
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
    int id[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int j = j0 + k * 32 + lane;
      id[k] = j < full ? src[j] : 0;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
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
    if (lo + j0 >= hi) return;
    int32_t* row = p.bt + (size_t)i * p.MB;
    // (The loads of all entries first.)
    int old[kPer], fresh[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int j = lo + j0 + k * 32 + lane;
      const bool edge = cow && j == lo;
      old[k] = j < hi && (edge || j < oldB) ? row[j] : -2;                                   // given back
      fresh[k] = j < hi && (edge || j >= oldB) ? p.ids[first + (edge ? 0 : cow + j - oldB)] : -1;  // taken
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int j = lo + j0 + k * 32 + lane;
      const bool edge = cow && j == lo;
      if (j < hi && (edge || j < oldB)) {
        const int b = old[k];
        if ((unsigned)b >= (unsigned)p.NB) {
          record(p);
        } else if (atomicSub(p.refs + b, 1) <= 0) {
          atomicAdd(p.refs + b, 1);
          record(p);
        }
      }
      if (fresh[k] >= 0) {
        p.refs[fresh[k]] = 1;
        row[j] = fresh[k];
      }
    }
  } else {
    const int used = p.hdr[kHdrUsed], L = p.lens[i], cap = p.MB * p.BS;
    if ((L < 0 || L > cap) && j0 == 0 && lane == 0) record(p);
    const int n = (min(max(L, 0), cap) + p.BS - 1) / p.BS;
    int32_t* row = p.bt + (size_t)i * p.MB;
    if (j0 >= n) return;
    int b[kPer], r[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int j = j0 + k * 32 + lane;
      b[k] = j < n ? row[j] : 0;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int j = j0 + k * 32 + lane;
      const bool in = (unsigned)b[k] < (unsigned)p.NB;
      r[k] = j < n && in && b[k] >= used ? p.rank_of[b[k]] : -2;
      // An id outside the pool, or a free block.
      if (j < n && (!in || r[k] == -1)) record(p);
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (r[k] >= 0) row[j0 + k * 32 + lane] = p.ids[r[k]];
  }
}

// `books`: also the tables and counts (the first launch of a call; further
// ones copy the pages of caches past kMaxCaches).
template <int MODE>
__global__ void __launch_bounds__(kApplyThreads, 6)
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

struct Span {
  const void* p;
  size_t n;      // bytes
  bool written;  // by the call
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.n > 0 && b.n > 0 && x < y + b.n && y < x + a.n;
}

// Whether something that the call writes lies in another of its arrays.  The
// plan is checked, and applied by a second launch that reads the lengths,
// parents and tables again: they must not change in between.
template <int MODE>
bool written_overlaps(const PagesParams& p, void* const* caches, const size_t* page_bytes, int num_caches,
                      const void* workspace, size_t workspace_bytes) {
  const size_t row = (size_t)p.MB * 4, S = (size_t)p.S, rows = (size_t)p.rows, NB = (size_t)p.NB;
  const Span spans[] = {{p.bt, S * row, MODE != kFork},
                        {p.lens, S * 4, MODE == kResize},
                        {p.arg, MODE == kCompact ? 0 : rows * 4, false},
                        {p.bt_out, MODE == kFork ? rows * row : 0, true},
                        {p.lens_out, MODE == kFork ? rows * 4 : 0, true},
                        {p.refs, NB * 4, true},
                        {p.new_ids, p.new_ids ? NB * 4 : 0, true},
                        {workspace, workspace_bytes, true}};
  constexpr int n = sizeof spans / sizeof spans[0];
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < i; ++j) {
      // (New lengths that are the lengths: every row keeps its own, and is written as it is.)
      if (MODE == kResize && i == 2 && j == 1 && p.arg == p.lens) continue;
      if ((spans[i].written || spans[j].written) && overlap(spans[i], spans[j])) return true;
    }
  for (int k = 0; k < num_caches; ++k)
    for (int i = 0; i < n; ++i)
      if (overlap(Span{caches[k], NB * page_bytes[k], true}, spans[i])) return true;
  return false;
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
  }
  if (num_caches > 0 && (!caches || !page_bytes)) return PA_ERR_INVALID_ARG;
  for (int i = 0; i < num_caches; ++i)
    if (!caches[i] || !aligned(caches[i], 16) || page_bytes[i] == 0 || page_bytes[i] % 16 != 0 ||
        page_bytes[i] > (size_t)1 << 35)
      return PA_ERR_INVALID_ARG;
  PagesLayout l;
  if (!pages_layout(p.rows, p.MB, p.NB, &l)) return PA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 16)) return PA_ERR_INVALID_ARG;
  if (workspace_bytes < l.total) return PA_ERR_WORKSPACE;
  if (written_overlaps<MODE>(p, caches, page_bytes, num_caches, workspace, l.total)) return PA_ERR_INVALID_ARG;
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
  cfg.blockDim = dim3(kApplyThreads, 1, 1);
  const int sms = device_sm_count();
  // Pages that may have to be copied (how many are is known on the device).
  const long long most = MODE == kCompact ? p.NB / 2 : p.rows;
  for (int c0 = 0; c0 == 0 || c0 < num_caches; c0 += kMaxCaches) {
    CopyParams c;
    std::memset(&c, 0, sizeof c);
    c.n = num_caches - c0 < kMaxCaches ? num_caches - c0 : kMaxCaches;
    for (int i = 0; i < c.n; ++i) {
      c.base[i] = static_cast<uint8_t*>(caches[c0 + i]);
      c.bytes[i] = page_bytes[c0 + i];
      c.first[i + 1] = c.first[i] + (uint32_t)((page_bytes[c0 + i] + kCopyBytes - 1) / kCopyBytes);
    }
    // Four CTAs an SM where the copies are few (an idle CTA costs its launch),
    // up to 32 where they are many: CTAs that end and make room for the next
    // keep a run of addresses together (4 GB of pages compacted: 344 us with 4,
    // 329 with 32).
    const long long jobs = most * c.first[c.n] / (kApplyThreads / 32);
    cfg.gridDim = dim3((unsigned)(sms * (jobs < 4 * sms ? 4 : jobs > 32 * sms ? 32 : jobs / sms)), 1, 1);
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
