// pa_combine.cu -- launches of the phase-2 combine kernel (pa_combine.cuh), one
// instance per output element type and head size.
#include "pa_combine.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

template <typename T, int D, bool VIEW>
cudaError_t go(const CParams& prm, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = 0;
  cfg.stream = st;
  // A programmatic dependent of the phase-1 launch just before it on the
  // stream: it may start as soon as every phase-1 CTA has run out of work,
  // and waits (griddepcontrol.wait) for phase 1 to complete before it reads.
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (prm.S <= kRowsMaxSeqs && prm.Pmax > 16) {
    // Rows that a single warp would take in two batches or more: one
    // persistent CTA per SM (no more than the batch's rows could need).  With
    // short rows only, the per-sequence grid is as good (its CTAs, 8 rows of
    // one warp each, are short) and the persistent one lost 0.2-0.9%.
    const long long rows = (long long)prm.S * prm.H;
    const int sms = device_sm_count();
    cfg.gridDim = dim3((unsigned)(rows < sms ? rows : sms), 1, 1);
    cfg.blockDim = dim3(kRowsWarps * 32, 1, 1);
    return cudaLaunchKernelEx(&cfg, pa_combine_rows_kernel<T, D, VIEW>, prm);
  }
  // CTAs of 4 warps where a row takes at most 4 (five CTAs of a 98-register
  // kernel fit an SM where two of 8 warps did: 20 warps in flight, not 16).
  const int nw = prm.wpr <= 4 ? 4 : kCombineWarps;
  const int rpc = nw / prm.wpr;
  unsigned groups = (unsigned)((prm.H + rpc - 1) / rpc);
  if constexpr (VIEW) {
    // Often no sequence has two partitions, which is known on the device only: no more
    // CTAs than run at once (five an SM) find that out.
    const unsigned most = (unsigned)(5 * device_sm_count() / prm.S);
    groups = groups < most ? groups : most > 1 ? most : 1;
  }
  cfg.gridDim = dim3((unsigned)prm.S, groups, 1);
  cfg.blockDim = dim3(nw * 32, 1, 1);
  if constexpr (VIEW) {
    return cudaLaunchKernelEx(&cfg, pa_combine_kernel<T, D, 4, true>, prm);  // (Pmax is 16 at most: one warp a row)
  } else {
    if (nw == 4) return cudaLaunchKernelEx(&cfg, pa_combine_kernel<T, D, 4, false>, prm);
    return cudaLaunchKernelEx(&cfg, pa_combine_kernel<T, D, kCombineWarps, false>, prm);
  }
}

template <typename T, bool VIEW>
cudaError_t by_head_size(const CParams& prm, int D, cudaStream_t st) {
  switch (D) {
    case 64: return go<T, 64, VIEW>(prm, st);
    case 80: return go<T, 80, VIEW>(prm, st);
    case 96: return go<T, 96, VIEW>(prm, st);
    case 112: return go<T, 112, VIEW>(prm, st);
    case 128: return go<T, 128, VIEW>(prm, st);
    case 256: return go<T, 256, VIEW>(prm, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_combine(const CParams& prm, int elem_bytes, bool bf16, int D, cudaStream_t st) {
  if (prm.view) {
    if (elem_bytes == 4) return by_head_size<float, true>(prm, D, st);
    return bf16 ? by_head_size<__nv_bfloat16, true>(prm, D, st) : by_head_size<__half, true>(prm, D, st);
  }
  if (elem_bytes == 4) return by_head_size<float, false>(prm, D, st);
  return bf16 ? by_head_size<__nv_bfloat16, false>(prm, D, st) : by_head_size<__half, false>(prm, D, st);
}

}  // namespace pa
