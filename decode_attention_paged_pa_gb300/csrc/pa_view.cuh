// pa_view.cuh -- what the rows of windowed and tree attention see
// (include/pa_decode.h: pa_decode_v2_window, pa_decode_v2_tree).
#pragma once

#include <stdint.h>

namespace pa {

// The blocks of a sequence that some view row can see are its first ones and
// those from the window's start on; the ones between are skipped: no row is
// charged for them, and their table entries are never read.  The kernel works
// on the tokens that are left: token t of them is at position t where it lies in
// the first `sink_blocks` blocks, skip * BS further on otherwise (skip = 0
// without a window, or where the window reaches the first tokens).
struct ViewSpan {
  int sink_blocks, skip;
};
__device__ __forceinline__ ViewSpan view_span(int L, int q_len, int window, int sinks, int BS) {
  ViewSpan v{0, 0};
  const int low = L - q_len + 1 - window;  // the first row's window starts here
  if (window > 0 && low > 0) {
    const int wb = low / BS;
    v.sink_blocks = min((sinks + BS - 1) / BS, wb);
    v.skip = wb - v.sink_blocks;
  }
  return v;
}
// Of a sequence of L tokens (out of range: clamped): the tokens the kernel
// works on, none where it has fewer than q_len.
__device__ __forceinline__ int view_tokens(int L, int q_len, int window, int sinks, int BS) {
  return L < q_len ? 0 : L - view_span(L, q_len, window, sinks, BS).skip * BS;
}

// Tokens of a partition of a launch of view rows, which has `sum` tokens to work on, `most`
// of one sequence: partitions of P are taken together, in powers of two, as long as no unit
// (of n_hg a partition) gets longer than one of `units` equal ones would be (0: never).  Each
// unit has its start and its end, and states that are joined; but the longest one is what
// the call may wait for, whatever the room in the tables.  Both phases work it out from
// the lengths.
__device__ __forceinline__ int joined_partition(unsigned long long sum, int most, int P, int units, int n_hg,
                                                int max_len) {
  if (units > 0) {
    const unsigned long long work = sum * n_hg;  // (below 2^9 * 2^30 * 2^16)
    while (P < most && (unsigned long long)min(2ll * P, (long long)most) * units <= work)
      P = (int)min(2ll * P, (long long)max_len);
  }
  return P;
}
// `sum` and `most` over a warp; a thread's sum is of a few sequences, below 2^32.
__device__ __forceinline__ void reduce_lengths(unsigned long long& sum, int& most) {
  const unsigned lo = __reduce_add_sync(0xffffffffu, (unsigned)sum & 0xffffu);
  const unsigned hi = __reduce_add_sync(0xffffffffu, (unsigned)sum >> 16);
  sum = ((unsigned long long)hi << 16) + lo;
  most = __reduce_max_sync(0xffffffffu, most);
}

// What row head h of sequence s (of L tokens) sees: position t where
//   t < hi  and  (t >= lo or t < sinks)  and  (t < base or bit t - base of `bits`).
// A window row at position p has lo = p - window + 1 and hi = base = p + 1.  A
// tree's row is a node among the sequence's last q_len tokens (base: the first of
// them); its mask has a bit for itself and for each of its ancestors, and so its
// position, for the window, is base + bits - 1.  A node without a bit is padding:
// hi = 0, it sees nothing.  (window >= q_len for trees, so no ancestor lies
// before the window.)
struct RowView {
  int lo, hi, base;
  const uint32_t* bits;
};

}  // namespace pa
