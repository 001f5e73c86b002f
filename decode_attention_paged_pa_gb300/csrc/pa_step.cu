// pa_step.cu -- the rows of a step, numbered on the device (include/pa_decode.h:
// pa_pages_slots, pa_tree_masks).
//
// pa_pages_slots.  Row r of the step belongs to the sequence s with cu[s] <= r <
// cu[s + 1], where cu is the running sum of the new tokens; it is at position
// seq_lens[s] - num_new[s] + r - cu[s], and its slot follows from the table.  A
// CTA takes kRows rows.  It sums up the counts itself (a block scan over 2048
// sequences at a time; no CTA waits for another), leaves each sequence's number
// at the row where it starts, and a running maximum over the rows then gives
// every row its sequence: prompts of thousands of rows and single tokens take the
// same time.
//
// pa_tree_masks.  A thread walks up from its node and sets the bits of its
// ancestors in its own words of shared memory.
//
// Both move a few bytes a row and are bound by their chains of dependent loads
// (counts, scan, lengths, table: about four) and their launches: a step of up to
// kRows rows is one launch, whose only CTA also leaves the status; larger ones
// have the workspace's header cleared by a launch before.  Measured (calls in
// a graph): 128 sequences of one new token 3.1 us, 512 of up to 256 (1.1 MB written and read) 4.0.
#include <climits>
#include <cstring>

#include "pa_common.cuh"
#include "pa_decode.h"
#include "pa_launch.h"

namespace pa {
namespace {

struct SlotsParams {
  long long* slots;    // [N]
  int32_t* positions;  // [N] or null
  int32_t* seq_ids;    // [N] or null
  int32_t* cu;         // [S + 1]
  const int32_t* bt;
  const int32_t* lens;
  const int32_t* num_new;
  int* hdr;
  int S, N, MB, BS;
};

constexpr int kRows = 512;      // rows, and threads, per CTA
constexpr int kPerThread = 4;   // sequences a thread sums up at a time
constexpr int kWarps = kRows / 32;

__device__ __forceinline__ long long warp_scan_add(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  return v;
}

__global__ void __launch_bounds__(kRows) pages_slots_kernel(const __grid_constant__ SlotsParams p) {
  // A row's sequence and the row where that starts (both ascend over the rows).
  __shared__ unsigned long long mark[kRows];
  __shared__ long long tot[kWarps];
  __shared__ unsigned long long top[kWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long r0 = (long long)blockIdx.x * kRows;
  const bool first = blockIdx.x == 0;  // this CTA writes cu, and looks at every sequence
  mark[tid] = 0;
  int bad = 0;
  long long carry = 0;  // rows before the sequences at hand
  for (int s0 = 0; s0 < p.S && (first || carry < r0 + kRows); s0 += kRows * kPerThread) {
    int n[kPerThread];
    long long sum = 0;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const int s = s0 + tid * kPerThread + j;
      n[j] = s < p.S ? p.num_new[s] : 0;
      if (n[j] < 0) {
        bad = 1;
        n[j] = 0;
      }
      sum += n[j];
    }
    const long long incl = warp_scan_add(sum, lane);
    __syncthreads();  // tot is free, mark is cleared
    if (lane == 31) tot[warp] = incl;
    __syncthreads();
    long long at = carry + incl - sum, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += tot[w];
      all += tot[w];
    }
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const int s = s0 + tid * kPerThread + j;
      if (first && s < p.S) p.cu[s] = (int)min(at, (long long)INT_MAX);
      if (n[j] > 0 && at < r0 + kRows && at + n[j] > r0) {
        // (Rows past N are never looked at, so a start that matters fits 32 bits.)
        mark[at > r0 ? (int)(at - r0) : 0] = (unsigned long long)(s + 1) << 32 | (unsigned)at;
      }
      at += n[j];
    }
    carry += all;
  }
  if (first && tid == 0) p.cu[p.S] = (int)min(carry, (long long)INT_MAX);
  if (carry > p.N && first) bad = 1;
  // (The last CTA with sequences may have left the loop early: it has seen all rows it needs.)
  __syncthreads();
  unsigned long long m = mark[tid];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long v = __shfl_up_sync(0xffffffffu, m, o);
    if (lane >= o && v > m) m = v;
  }
  if (lane == 31) top[warp] = m;
  __syncthreads();
  for (int w = 0; w < warp; ++w) m = max(m, top[w]);
  const long long r = r0 + tid;
  if (r < p.N) {
    const int s = (int)(m >> 32) - 1;
    long long slot = -1;
    int pos = -1, seq = -1;
    if (s >= 0) {
      const int n = p.num_new[s], L = p.lens[s];
      const int i = (int)(r - (long long)(unsigned)m);
      if (i < n) {
        seq = s;
        if (L < n || L > p.MB * p.BS) {
          bad = 1;
        } else {
          pos = L - n + i;
          const int b = p.bt[(size_t)s * p.MB + pos / p.BS];
          if (b >= 0) slot = (long long)b * p.BS + pos % p.BS;
          else bad = 1;
        }
      }
    }
    p.slots[r] = slot;
    if (p.positions) p.positions[r] = pos;
    if (p.seq_ids) p.seq_ids[r] = seq;
  }
  bad = __syncthreads_or(bad);
  if (tid == 0) {
    if (gridDim.x == 1) p.hdr[kHdrError] = bad ? kErrDeviceBounds : kOk;
    else if (bad) atomicCAS(p.hdr + kHdrError, 0, kErrDeviceBounds);
  }
}

struct MasksParams {
  uint32_t* masks;     // [S, n, words]
  int32_t* positions;  // [S, n] or null
  const int32_t* parents;
  const int32_t* lens;
  int* hdr;
  int S, n, words, per_cta;  // sequences per CTA
};

constexpr int kMaskThreads = 512;

__global__ void __launch_bounds__(kMaskThreads) tree_masks_kernel(const __grid_constant__ MasksParams p) {
  extern __shared__ uint32_t bits[];  // [threads][words], then the parents [threads]
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, W = p.words, n = p.n;
  int32_t* par = reinterpret_cast<int32_t*>(bits + kMaskThreads * W);
  const long long node0 = (long long)blockIdx.x * p.per_cta * n, nodes = (long long)p.S * n;
  const int live = (int)min((long long)p.per_cta * n, nodes - node0);
  const int i = tid % n, base = tid - i;  // the node within its tree, and the tree's first thread
  int bad = 0;
  if (tid < live) par[tid] = p.parents[node0 + tid];
  for (int w = 0; w < W; ++w) bits[tid * W + w] = 0;
  __syncthreads();
  if (tid < live) {
    uint32_t* mine = bits + tid * W;
    int j = i, depth = 0;
    bool ok = true;
    // Every step goes to a lower node: at most n of them.
    while (true) {
      const int q = par[base + j];
      if (q < -1 || q >= j) {  // padding, or no parent that a node can have
        ok = false;
        bad |= q >= j || j != i;  // (a child of padding is refused too)
        break;
      }
      mine[j >> 5] |= 1u << (j & 31);
      ++depth;
      if (q < 0) break;
      j = q;
    }
    const int L = p.lens[(node0 + tid) / n];
    if (L < n) bad = 1;
    for (int w = 0; w < W; ++w) p.masks[(node0 + tid) * W + w] = ok ? mine[w] : 0u;
    if (p.positions) p.positions[node0 + tid] = ok && L >= n ? L - n + depth - 1 : -1;
  }
  bad = __syncthreads_or(bad);
  if (tid == 0) {
    if (gridDim.x == 1) p.hdr[kHdrError] = bad ? kErrDeviceBounds : kOk;
    else if (bad) atomicCAS(p.hdr + kHdrError, 0, kErrDeviceBounds);
  }
}

__global__ void __launch_bounds__(32) clear_status_kernel(int* hdr) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) hdr[kHdrError] = kOk;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na > 0 && nb > 0 && x < y + nb && y < x + na;
}

template <class P>
int launch(void (*kern)(P), const P& p, long long grid, int threads, size_t smem, cudaStream_t st) {
  if (grid > INT_MAX) return PA_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (grid > 1) {
    cfg.gridDim = dim3(1, 1, 1);
    cfg.blockDim = dim3(32, 1, 1);
    if (cudaLaunchKernelEx(&cfg, clear_status_kernel, p.hdr) != cudaSuccess) return PA_ERR_CUDA;
  }
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" int pa_pages_slots(int64_t* slots, int32_t* positions, int32_t* seq_ids, int32_t* cu_tokens,
                              const int32_t* block_tables, const int32_t* seq_lens, const int32_t* num_new,
                              int num_seqs, int num_tokens, int max_blocks_per_seq, int block_size, void* stream,
                              void* workspace, size_t workspace_bytes) {
  if (num_seqs < 0 || num_tokens < 0 || max_blocks_per_seq <= 0 || block_size <= 0 ||
      (long long)max_blocks_per_seq * block_size > INT_MAX / 2 || num_seqs > (1 << 24))
    return PA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 16)) return PA_ERR_INVALID_ARG;
  if (workspace_bytes < kHdrInts * sizeof(int)) return PA_ERR_WORKSPACE;
  if (!cu_tokens || !aligned(cu_tokens, 4)) return PA_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!slots || !aligned(slots, 8))) return PA_ERR_INVALID_ARG;
  if ((positions && !aligned(positions, 4)) || (seq_ids && !aligned(seq_ids, 4))) return PA_ERR_INVALID_ARG;
  if (num_seqs > 0 && (!block_tables || !seq_lens || !num_new || !aligned(block_tables, 4) ||
                       !aligned(seq_lens, 4) || !aligned(num_new, 4)))
    return PA_ERR_INVALID_ARG;
  const size_t N = (size_t)num_tokens, S = (size_t)num_seqs;
  struct { const void* p; size_t n; bool written; } a[] = {
      {slots, 8 * N, true}, {positions, 4 * N, true}, {seq_ids, 4 * N, true}, {cu_tokens, 4 * (S + 1), true},
      {workspace, kHdrInts * sizeof(int), true}, {block_tables, 4 * S * (size_t)max_blocks_per_seq, false},
      {seq_lens, 4 * S, false}, {num_new, 4 * S, false}};
  for (int i = 0; i < 8; ++i)
    for (int j = 0; j < i; ++j)
      if ((a[i].written || a[j].written) && overlap(a[i].p, a[i].n, a[j].p, a[j].n)) return PA_ERR_INVALID_ARG;
  SlotsParams p = {};
  p.slots = reinterpret_cast<long long*>(slots);
  p.positions = positions;
  p.seq_ids = seq_ids;
  p.cu = cu_tokens;
  p.bt = block_tables;
  p.lens = seq_lens;
  p.num_new = num_new;
  p.hdr = static_cast<int*>(workspace);
  p.S = num_seqs;
  p.N = num_tokens;
  p.MB = max_blocks_per_seq;
  p.BS = block_size;
  const long long grid = num_tokens > 0 ? ((long long)num_tokens + kRows - 1) / kRows : 1;
  return launch(pages_slots_kernel, p, grid, kRows, 0, static_cast<cudaStream_t>(stream));
}

extern "C" int pa_tree_masks(int32_t* masks, int32_t* positions, const int32_t* parents, const int32_t* seq_lens,
                             int num_seqs, int num_nodes, void* stream, void* workspace, size_t workspace_bytes) {
  if (num_seqs < 0 || num_nodes < 1 || num_nodes > kMaxSeqsPerLaunch) return PA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 16)) return PA_ERR_INVALID_ARG;
  if (workspace_bytes < kHdrInts * sizeof(int)) return PA_ERR_WORKSPACE;
  if (num_seqs > 0 && (!masks || !parents || !seq_lens || !aligned(masks, 4) || !aligned(parents, 4) ||
                       !aligned(seq_lens, 4)))
    return PA_ERR_INVALID_ARG;
  if (positions && !aligned(positions, 4)) return PA_ERR_INVALID_ARG;
  MasksParams p = {};
  p.words = (num_nodes + 31) / 32;
  const size_t S = (size_t)num_seqs, n = (size_t)num_nodes;
  struct { const void* p; size_t n; bool written; } a[] = {
      {masks, 4 * S * n * p.words, true}, {positions, 4 * S * n, true},
      {workspace, kHdrInts * sizeof(int), true}, {parents, 4 * S * n, false}, {seq_lens, 4 * S, false}};
  for (int i = 0; i < 5; ++i)
    for (int j = 0; j < i; ++j)
      if ((a[i].written || a[j].written) && overlap(a[i].p, a[i].n, a[j].p, a[j].n)) return PA_ERR_INVALID_ARG;
  p.masks = reinterpret_cast<uint32_t*>(masks);
  p.positions = positions;
  p.parents = parents;
  p.lens = seq_lens;
  p.hdr = static_cast<int*>(workspace);
  p.S = num_seqs;
  p.n = num_nodes;
  p.per_cta = kMaskThreads / num_nodes;  // whole trees
  const long long grid = num_seqs > 0 ? ((long long)num_seqs + p.per_cta - 1) / p.per_cta : 1;
  return launch(tree_masks_kernel, p, grid, kMaskThreads, (size_t)kMaskThreads * (p.words + 1) * 4,
                static_cast<cudaStream_t>(stream));
}
