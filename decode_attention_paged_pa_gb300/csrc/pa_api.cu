// pa_api.cu -- C ABI of the paged decode attention library (include/pa_decode.h):
// argument validation, workspace layout, kernel-family choice and launches.
#include <climits>
#include <cstdint>
#include <cstring>

#include "pa_decode.h"
#include "pa_launch.h"

namespace pa {

int device_sm_count() {
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev < 0 || dev >= 64) {
    int n = 1;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
  }
  if (cache[dev] == 0) {
    int n = 1;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    cache[dev] = n;
  }
  return cache[dev];
}

// Clears header words [first, first + count) of the workspace before a phase-1
// launch.  It is itself launched as a programmatic dependent of whatever
// precedes it on the stream, so its launch overlaps that work's end: it first
// waits for that work to complete (its writes -- the caller's inputs among
// them -- visible), and only then lets phase 1, its own programmatic
// dependent, be scheduled; phase 1 waits for this kernel before it touches
// the header.
__global__ void __launch_bounds__(64) pa_clear_header_kernel(int* hdr, int first, int count) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = threadIdx.x; i < count; i += blockDim.x) hdr[first + i] = 0;
}

// The header clear, launched as described above.
static cudaError_t launch_clear_header(int* hdr, int first, int count, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, 1, 1);
  cfg.blockDim = dim3(64, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pa_clear_header_kernel, hdr, first, count);
}

namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

struct WsLayout {
  size_t hdr, m, l, o, total;
  int pmax;
};

bool valid_sizes(int S, int H, int KH, int D, int MB, int BS, int P) {
  if (S < 0 || H <= 0 || KH <= 0 || H % KH != 0 || MB <= 0 || BS <= 0 || P <= 0 || D <= 0) return false;
  if ((long long)MB * BS > INT_MAX / 2) return false;
  return true;
}

size_t elem_bytes(int dtype) { return dtype == PA_DTYPE_FP32 ? 4 : 2; }

// Shapes every kernel family handles; the tensor-core family also takes head
// sizes 80, 96, 112 and 8- or 64-token blocks.
bool base_shape(int D, int BS) {
  return (D == 64 || D == 128 || D == 256) && (BS == 16 || BS == 32);
}

// The CUDA-core family's further shapes: head sizes 80, 96, 112 with
// blocks of 16, 32 or 64 tokens, and 64-token blocks at head sizes 64, 128.
bool simt_extra_shape(int D, int BS) {
  return ((D == 80 || D == 96 || D == 112) && (BS == 16 || BS == 32 || BS == 64)) ||
         ((D == 64 || D == 128) && BS == 64);
}

bool supported(int D, int BS, int P) {
  const bool d_ok = D == 64 || D == 80 || D == 96 || D == 112 || D == 128 || D == 256;
  const bool bs_ok = BS == 8 || BS == 16 || BS == 32 || BS == 64;
  return d_ok && bs_ok && P % BS == 0;
}

bool ws_layout(int S, int H, int KH, int D, int MB, int BS, int P, WsLayout* w) {
  if (!valid_sizes(S, H, KH, D, MB, BS, P)) return false;
  const long long pmax = ((long long)MB * BS + P - 1) / P;
  if (pmax > INT_MAX) return false;
  w->pmax = (int)pmax;
  const size_t shp = (size_t)S * H * (size_t)pmax;
  w->hdr = 0;
  w->m = align_up(kHdrInts * sizeof(int));
  w->l = align_up(w->m + shp * sizeof(float));
  w->o = align_up(w->l + shp * sizeof(float));
  w->total = align_up(w->o + shp * (size_t)D * sizeof(float));
  return true;
}

// Blocks of a sequence that view rows (pa_decode_v2_window, pa_decode_v2_tree) can
// be worked on in one call: all of the table, or the first tokens' and as many as
// a window and the rows behind its start can touch.
int view_blocks(int q_len, int MB, int BS, int window, int sinks) {
  if (window <= 0) return MB;
  const long long n = ((long long)sinks + BS - 1) / BS + ((long long)window + q_len - 1 + BS - 1) / BS + 1;
  return n < MB ? (int)n : MB;
}

// What view rows see (null in decode_impl: plain decode).
struct ViewArgs {
  int window, sinks;
  const int32_t* masks;
  bool tree;
};

// The view kernels' launch.
cudaError_t launch_views(const KParams& prm, int dtype, bool kv_fp8, bool pairs, int D, int BS, int max_ctas,
                         cudaStream_t st) {
  const bool half = dtype == PA_DTYPE_FP16, b = BS == 8 || BS == 64;
  if (dtype == PA_DTYPE_FP32) return b ? launch_view_x_f32(prm, D, BS, max_ctas, st) : launch_view_f32(prm, D, BS, max_ctas, st);
  if (kv_fp8 && pairs) return half ? launch_view8_g_f16(prm, D, BS, max_ctas, st) : launch_view8_g_bf16(prm, D, BS, max_ctas, st);
  if (kv_fp8 && b) return half ? launch_view8_b_f16(prm, D, BS, max_ctas, st) : launch_view8_b_bf16(prm, D, BS, max_ctas, st);
  if (kv_fp8) return half ? launch_view8_f16(prm, D, BS, max_ctas, st) : launch_view8_bf16(prm, D, BS, max_ctas, st);
  if (pairs) return half ? launch_view_g_f16(prm, D, BS, max_ctas, st) : launch_view_g_bf16(prm, D, BS, max_ctas, st);
  if (b) return half ? launch_view_b_f16(prm, D, BS, max_ctas, st) : launch_view_b_bf16(prm, D, BS, max_ctas, st);
  return half ? launch_view_f16(prm, D, BS, max_ctas, st) : launch_view_bf16(prm, D, BS, max_ctas, st);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The 4-bit family's launch, dispatched on the head size.
cudaError_t launch_kv4_f16(const KParams& prm, int D, int BS, int nt, int kvu, int max_ctas, cudaStream_t st) {
  switch (D) {
    case 64: return launch_kv4_d64_f16(prm, BS, nt, kvu, max_ctas, st);
    case 80: return launch_kv4_d80_f16(prm, BS, nt, kvu, max_ctas, st);
    case 96: return launch_kv4_d96_f16(prm, BS, nt, kvu, max_ctas, st);
    case 112: return launch_kv4_d112_f16(prm, BS, nt, kvu, max_ctas, st);
    case 128: return launch_kv4_d128_f16(prm, BS, nt, kvu, max_ctas, st);
    case 256: return launch_kv4_d256_f16(prm, BS, nt, kvu, max_ctas, st);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_kv4_bf16(const KParams& prm, int D, int BS, int nt, int kvu, int max_ctas, cudaStream_t st) {
  switch (D) {
    case 64: return launch_kv4_d64_bf16(prm, BS, nt, kvu, max_ctas, st);
    case 80: return launch_kv4_d80_bf16(prm, BS, nt, kvu, max_ctas, st);
    case 96: return launch_kv4_d96_bf16(prm, BS, nt, kvu, max_ctas, st);
    case 112: return launch_kv4_d112_bf16(prm, BS, nt, kvu, max_ctas, st);
    case 128: return launch_kv4_d128_bf16(prm, BS, nt, kvu, max_ctas, st);
    case 256: return launch_kv4_d256_bf16(prm, BS, nt, kvu, max_ctas, st);
    default: return cudaErrorInvalidValue;
  }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                  CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once through the runtime (the
// library does not link the driver library itself).
EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiledFn>(nullptr);
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// Tensor map of a 16-bit paged value cache for the tensor-core kernels:
// value_cache [NB, KH, D, BS] as a 3-D tensor [NB*KH][D][BS] with a box of one
// whole block ([1][D][BS]), stored in shared memory in the swizzle of the
// rows' width (BS * 2 bytes: 32, 64 or 128).
// kvu: kv heads per box (the unit's consecutive kv heads of one block).
bool encode_value_map(KParams* prm, const void* value_cache, int num_blocks, int KH, int D, int BS, int kvu) {
  const EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const CUtensorMapSwizzle sw = BS == 16 ? CU_TENSOR_MAP_SWIZZLE_32B
                                : BS == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                           : CU_TENSOR_MAP_SWIZZLE_128B;
  const cuuint32_t unit[3] = {1, 1, 1};
  const cuuint64_t vdim[3] = {(cuuint64_t)BS, (cuuint64_t)D, (cuuint64_t)num_blocks * (cuuint64_t)KH};
  const cuuint64_t vstride[2] = {(cuuint64_t)BS * 2, (cuuint64_t)D * BS * 2};
  const cuuint32_t vbox[3] = {(cuuint32_t)BS, (cuuint32_t)D, (cuuint32_t)kvu};
  return enc(&prm->tmv, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(value_cache), vdim, vstride, vbox,
             unit, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode_v2_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads,
                                               int head_size, int max_blocks_per_seq, int block_size,
                                               int partition_size) {
  WsLayout w;
  if (!ws_layout(num_seqs, num_heads, num_kv_heads, head_size, max_blocks_per_seq, block_size,
                 partition_size, &w))
    return 0;
  return w.total;
}

extern "C" int pa_decode_v2_workspace_layout(int num_seqs, int num_heads, int num_kv_heads, int head_size,
                                             int max_blocks_per_seq, int block_size, int partition_size,
                                             size_t offsets[5], int* max_partitions) {
  WsLayout w;
  if (!offsets || !ws_layout(num_seqs, num_heads, num_kv_heads, head_size, max_blocks_per_seq,
                             block_size, partition_size, &w))
    return PA_ERR_INVALID_ARG;
  offsets[0] = w.m;
  offsets[1] = w.l;
  offsets[2] = w.o;
  offsets[3] = w.hdr;
  offsets[4] = w.total;
  if (max_partitions) *max_partitions = w.pmax;
  return PA_OK;
}

namespace {

int decode_impl(void* out, float* lse, const void* query, const void* key_cache,
                const void* value_cache, const int32_t* block_tables, const int32_t* seq_lens,
                float scale, int num_seqs, int q_len, int num_heads, int num_kv_heads, int head_size,
                int block_size, int partition_size, int dtype, void* stream, int max_blocks_per_seq,
                int num_blocks, void* workspace, size_t workspace_bytes, int variant, int max_ctas,
                long long timeout_ns, bool kv_fp8 = false, float k_scale = 1.f, float v_scale = 1.f,
                bool kv4 = false, const ViewArgs* view = nullptr) {
  // Multi-query: the kernel sees q_len "row heads" per caller head (H below
  // counts them), q_len * G per kv head, all sharing the kv head's blocks.
  if (q_len < 1 || q_len > kMaxSeqsPerLaunch || num_heads <= 0 ||
      (long long)num_heads * q_len > 65535)
    return PA_ERR_INVALID_ARG;
  const int S = num_seqs, H = num_heads * q_len, KH = num_kv_heads, D = head_size, BS = block_size,
            P = partition_size, MB = max_blocks_per_seq;
  if (!valid_sizes(S, H, KH, D, MB, BS, P) || num_heads % KH != 0 || num_blocks <= 0) return PA_ERR_INVALID_ARG;
  if (dtype != PA_DTYPE_FP16 && dtype != PA_DTYPE_BF16 && dtype != PA_DTYPE_FP32) return PA_ERR_INVALID_ARG;
  if (variant < PA_VARIANT_AUTO || variant > PA_VARIANT_MMA || max_ctas < 0 || timeout_ns < 0)
    return PA_ERR_INVALID_ARG;
  if (!(scale == scale) || scale == INFINITY || scale == -INFINITY) return PA_ERR_INVALID_ARG;
  if (!(k_scale == k_scale) || k_scale == INFINITY || k_scale == -INFINITY || !(v_scale == v_scale) ||
      v_scale == INFINITY || v_scale == -INFINITY)
    return PA_ERR_INVALID_ARG;
  if (view) {
    // (A tree's ancestors never lie before its window.)
    if (view->sinks < 0 || view->window < (view->tree ? 0 : 1) ||
        (view->tree && view->window > 0 && view->window < q_len))
      return PA_ERR_INVALID_ARG;
  }
  if (!supported(D, BS, P)) return PA_ERR_UNSUPPORTED;
  if (kv_fp8 && variant == PA_VARIANT_SIMT) return PA_ERR_UNSUPPORTED;  // fp8 runs on tensor cores
  // (8-token blocks on the CUDA cores: fp32 only; the 16-bit types take the tensor cores there.)
  const bool simt_ok = base_shape(D, BS) || simt_extra_shape(D, BS) || (dtype == PA_DTYPE_FP32 && BS == 8);
  if (variant == PA_VARIANT_SIMT && !simt_ok) return PA_ERR_UNSUPPORTED;
  // fp32 runs on the CUDA-core family only (its shapes; multi-query rows on
  // its causal instances).
  if (dtype == PA_DTYPE_FP32 && (kv_fp8 || kv4 || variant == PA_VARIANT_MMA || !simt_ok))
    return PA_ERR_UNSUPPORTED;
  if (S == 0) return PA_OK;
  if (!out || !query || !key_cache || !value_cache || !block_tables || !seq_lens)
    return PA_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(query, 16) || !aligned(key_cache, 16) ||
      !aligned(value_cache, 16) || !aligned(block_tables, 4) || !aligned(seq_lens, 4) ||
      (workspace && !aligned(workspace, 16)) || (lse && !aligned(lse, 4)))
    return PA_ERR_INVALID_ARG;
  if (view && view->tree && (!view->masks || !aligned(view->masks, 4))) return PA_ERR_INVALID_ARG;
  WsLayout w;
  if (!ws_layout(S, H, KH, D, view ? view_blocks(q_len, MB, BS, view->window, view->sinks) : MB, BS, P, &w))
    return PA_ERR_INVALID_ARG;
  if (workspace && workspace_bytes < w.total) return PA_ERR_WORKSPACE;

  const int G = H / KH;
  if (variant == PA_VARIANT_AUTO)
    variant = view ? (dtype == PA_DTYPE_FP32 ? PA_VARIANT_SIMT : PA_VARIANT_MMA)
              : ((G == 1 || dtype == PA_DTYPE_FP32) && !kv_fp8 && !kv4 && simt_ok) ? PA_VARIANT_SIMT : PA_VARIANT_MMA;
  // More than 8 query rows per kv head: the tensor-core instances for units
  // of 16 rows (the rows on the M side of the products) read each K/V block
  // once for 16 rows (head sizes 64 and 128, blocks of 16 or 32 tokens,
  // 16-bit caches).
  const bool wide = !view && variant == PA_VARIANT_MMA && G > kMmaGroup && !kv_fp8 && !kv4 && D <= 128 &&
                    base_shape(D, BS);
  // Over a 4-bit cache, 16 rows a unit where a kv head has more than 8: its
  // codes are unpacked once for both halves.
  const int nt = kv4 && G > kMmaGroup && D <= 128 ? 2 : 1;
  const int gt = view && variant == PA_VARIANT_MMA && G > kMmaGroup ? kRowsPerUnit
                 : kv4 ? nt * kMmaGroup : (variant == PA_VARIANT_MMA) ? (wide ? kMmaGroupWide : kMmaGroup) : kSimtGroup;
  // View rows: with more than eight a kv head, 128 of them a unit on the
  // fifth-generation tensor cores (pa_rows.cuh).
  const bool many = view && variant == PA_VARIANT_MMA && G > kMmaGroup;
  // Four query rows per kv head (query heads, or multi-query row heads): a
  // unit's 8 columns take two kv heads (one block copy each for keys and
  // values covers both), head sizes up to 128 and blocks of 8, 16 or 32 tokens.
  const bool pairs = variant == PA_VARIANT_MMA && !wide && G * 2 == kMmaGroup && KH % 2 == 0 &&
                     D <= 128 && (BS == 8 || BS == 16 || BS == 32) && !kv4;
  // Over a 4-bit cache, two kv heads a unit where each has at most four rows
  // (head sizes up to 128, blocks of up to 32 tokens: two stages of both heads
  // fit a warp's ring).
  const bool kv4_pairs = kv4 && G * 2 <= kMmaGroup && KH % 2 == 0 && D <= 128 && BS <= 32;
  const int kvu = pairs || kv4_pairs ? 2 : 1;
  // View rows on the tensor cores: partitions are taken together where the lengths leave
  // every SM its share without them (joined_partition): units of which three make an SM's
  // work, or with many rows a quarter more than it.  (Partitions of 512 as they are, units
  // for four, two and one an SM: 16 nodes, 48 sequences of 3000 tokens: 218, 129, 118, 118
  // us; 64 nodes, 16 sequences of 5000: 155 with four, 136, 122; 32 nodes, 4 sequences of 3000:
  // 33 with two, 27.  One row, 128 sequences, a window of 1024: 108 as they are, 95 for three
  // or two; 40 such sequences: 45 for three, 49 for two.)
  const bool joined = view && variant == PA_VARIANT_MMA;
  const int units = !joined ? 0 : many ? (device_sm_count() * 4 + 4) / 5 : 3 * device_sm_count();
  const int hg_per_kv = (G + gt - 1) / gt;
  const int n_hg = KH * hg_per_kv / kvu;
  const int rows_per_launch = many ? kRowsSeqsPerLaunch : kMaxSeqsPerLaunch;  // sequences per launch
  const int chunk = S < rows_per_launch ? S : rows_per_launch;
  // (Joined partitions are longer than half of the share of one of `units`, or one a sequence.)
  if ((long long)chunk * (joined ? 1 : w.pmax) * n_hg > INT_MAX / 2) return PA_ERR_UNSUPPORTED;
  // The tensor-core kernels over 16-bit caches in blocks of 16 tokens or more
  // stage value blocks by swizzled tensor copies (z coordinates are int32).
  const bool tma_values = variant == PA_VARIANT_MMA && !kv_fp8 && !kv4 && BS >= 16;
  KParams maps;
  std::memset(&maps, 0, sizeof maps);
  if (tma_values) {
    if ((long long)num_blocks * KH > INT_MAX) return PA_ERR_UNSUPPORTED;
    if (!encode_value_map(&maps, value_cache, num_blocks, KH, D, BS, kvu)) return PA_ERR_CUDA;
  }

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  bool own = false;
  if (!ws) {
    if (cudaMallocAsync(reinterpret_cast<void**>(&ws), w.total, st) != cudaSuccess) return PA_ERR_CUDA;
    own = true;
  }
  int status = PA_OK;
  const size_t esz = elem_bytes(dtype);
  // Phase 2 over sequences s0 .. s0 + n - 1 (no sequence has more than one
  // partition if the table holds at most P tokens).  Warps per row: enough that a
  // warp takes at most 16 partitions (one batch of loads), up to 8.
  const auto combine = [&](int s0, int n) {
    if (w.pmax <= 1) return cudaSuccess;
    const size_t rows = (size_t)s0 * H;
    CParams cp;
    std::memset(&cp, 0, sizeof cp);
    cp.out = static_cast<uint8_t*>(out) + rows * D * esz;
    cp.lse = lse ? lse + rows : nullptr;
    cp.ws_m = reinterpret_cast<const float*>(ws + w.m) + rows * w.pmax;
    cp.ws_l = reinterpret_cast<const float*>(ws + w.l) + rows * w.pmax;
    cp.ws_o = reinterpret_cast<const float*>(ws + w.o) + rows * w.pmax * D;
    cp.lens = seq_lens + s0;
    cp.S = n;
    cp.H = H;
    cp.Pmax = w.pmax;
    cp.P = view && P > MB * BS ? MB * BS : P;
    cp.max_len = MB * BS;
    cp.BS = BS;
    if (view) {
      cp.view = 1;
      cp.window = view->window;
      cp.sinks = view->sinks;
      cp.units = units;
      cp.n_hg = n_hg;
    }
    cp.wpr = w.pmax > 64 ? 8 : w.pmax > 32 ? 4 : w.pmax > 16 ? 2 : 1;
    cp.q_len = q_len;
    cp.Hu = num_heads;
    cp.Gu = num_heads / KH;
    cp.G = G;
    return launch_combine(cp, (int)esz, dtype == PA_DTYPE_BF16, D, st);
  };
  for (int s0 = 0; s0 < S && status == PA_OK; s0 += rows_per_launch) {
    const int n = (S - s0) < rows_per_launch ? (S - s0) : rows_per_launch;
    // The header (error word, work counter, timeout record) starts at zero;
    // a later launch of the same call restarts the work counter only.
    if (launch_clear_header(reinterpret_cast<int*>(ws + w.hdr), s0 == 0 ? 0 : kHdrWork,
                            s0 == 0 ? kHdrInts : 1, st) != cudaSuccess) {
      status = PA_ERR_CUDA;
      break;
    }
    KParams prm;
    std::memset(&prm, 0, sizeof prm);
    prm.tmv = maps.tmv;
    prm.out = static_cast<uint8_t*>(out) + (size_t)s0 * H * D * esz;
    prm.q = static_cast<const uint8_t*>(query) + (size_t)s0 * H * D * esz;
    prm.kc = key_cache;
    prm.vc = value_cache;
    prm.bt = block_tables + (size_t)s0 * MB;
    prm.lens = seq_lens + s0;
    prm.q_len = q_len;
    prm.Hu = num_heads;
    prm.Gu = num_heads / KH;
    prm.ws_m = reinterpret_cast<float*>(ws + w.m) + (size_t)s0 * H * w.pmax;
    prm.ws_l = reinterpret_cast<float*>(ws + w.l) + (size_t)s0 * H * w.pmax;
    prm.ws_o = reinterpret_cast<float*>(ws + w.o) + (size_t)s0 * H * w.pmax * D;
    prm.hdr = reinterpret_cast<int*>(ws + w.hdr);
    prm.lse = lse ? lse + (size_t)s0 * H : nullptr;
    prm.scale_log2 = scale * k_scale * kLog2e;
    prm.v_scale = v_scale;
    prm.S = n;
    prm.H = H;
    prm.KH = KH;
    prm.G = G;
    prm.MB = MB;
    prm.num_blocks = num_blocks;
    // (A partition past the table's capacity is the capacity: sums of lengths
    // and partition sizes stay in 32 bits.)
    prm.P = (view || kv4) && P > MB * BS ? MB * BS : P;
    prm.units = units;
    prm.Pmax = w.pmax;
    prm.hg_per_kv = hg_per_kv;
    prm.n_hg = n_hg;
    prm.timeout_ns = timeout_ns > 0 ? timeout_ns : (1LL << 31);
    if (view) {
      prm.window = view->window;
      prm.sinks = view->sinks;
      prm.words = (q_len + 31) / 32;
      prm.masks = view->tree ? reinterpret_cast<const uint32_t*>(view->masks) + (size_t)s0 * q_len * prm.words : nullptr;
    }
    cudaError_t e;
    if (many && kv_fp8)
      e = dtype == PA_DTYPE_FP16 ? launch_rows8_f16(prm, D, BS, max_ctas, st) : launch_rows8_bf16(prm, D, BS, max_ctas, st);
    else if (many)
      e = dtype == PA_DTYPE_FP16 ? launch_rows_f16(prm, D, BS, max_ctas, st) : launch_rows_bf16(prm, D, BS, max_ctas, st);
    else if (view)
      e = launch_views(prm, dtype, kv_fp8, pairs, D, BS, max_ctas, st);
    else if (kv4)
      e = dtype == PA_DTYPE_FP16 ? launch_kv4_f16(prm, D, BS, nt, kvu, max_ctas, st)
                                 : launch_kv4_bf16(prm, D, BS, nt, kvu, max_ctas, st);
    else if (kv_fp8 && pairs && BS == 8)
      e = dtype == PA_DTYPE_FP16 ? launch_mma8_gb8_f16(prm, D, max_ctas, st)
                                 : launch_mma8_gb8_bf16(prm, D, max_ctas, st);
    else if (kv_fp8 && pairs && (D == 64 || D == 128))
      e = dtype == PA_DTYPE_FP16 ? launch_mma8_g_f16(prm, D, BS, max_ctas, st)
                                 : launch_mma8_g_bf16(prm, D, BS, max_ctas, st);
    else if (kv_fp8 && pairs)
      e = dtype == PA_DTYPE_FP16 ? launch_mma8_gx_f16(prm, D, BS, max_ctas, st)
                                 : launch_mma8_gx_bf16(prm, D, BS, max_ctas, st);
    else if (kv_fp8 && BS == 8)
      e = dtype == PA_DTYPE_FP16 ? launch_mma8_b8_f16(prm, D, max_ctas, st)
                                 : launch_mma8_b8_bf16(prm, D, max_ctas, st);
    else if (kv_fp8 && BS == 64)
      e = dtype == PA_DTYPE_FP16 ? launch_mma8_b64_f16(prm, D, max_ctas, st)
                                 : launch_mma8_b64_bf16(prm, D, max_ctas, st);
    else if (kv_fp8 && base_shape(D, BS))
      e = dtype == PA_DTYPE_FP16 ? launch_mma8_f16(prm, D, BS, max_ctas, st)
                                 : launch_mma8_bf16(prm, D, BS, max_ctas, st);
    else if (kv_fp8)
      e = dtype == PA_DTYPE_FP16 ? launch_mma8_x_f16(prm, D, BS, max_ctas, st)
                                 : launch_mma8_x_bf16(prm, D, BS, max_ctas, st);
    else if (wide)
      e = dtype == PA_DTYPE_FP16 ? launch_mma16_f16(prm, D, BS, max_ctas, st)
                                 : launch_mma16_bf16(prm, D, BS, max_ctas, st);
    else if (pairs && BS == 8)
      e = dtype == PA_DTYPE_FP16 ? launch_mma_g8_f16(prm, D, max_ctas, st) : launch_mma_g8_bf16(prm, D, max_ctas, st);
    else if (pairs && BS == 16)
      e = dtype == PA_DTYPE_FP16 ? launch_mma_g16_f16(prm, D, max_ctas, st) : launch_mma_g16_bf16(prm, D, max_ctas, st);
    else if (pairs)
      e = dtype == PA_DTYPE_FP16 ? launch_mma_g32_f16(prm, D, max_ctas, st) : launch_mma_g32_bf16(prm, D, max_ctas, st);
    else if (variant == PA_VARIANT_MMA && BS == 8)
      e = dtype == PA_DTYPE_FP16 ? launch_mma_b8_f16(prm, D, max_ctas, st)
                                 : launch_mma_b8_bf16(prm, D, max_ctas, st);
    else if (variant == PA_VARIANT_MMA && BS == 64)
      e = dtype == PA_DTYPE_FP16 ? launch_mma_b64_f16(prm, D, max_ctas, st)
                                 : launch_mma_b64_bf16(prm, D, max_ctas, st);
    else if (variant == PA_VARIANT_MMA && !base_shape(D, BS))
      e = dtype == PA_DTYPE_FP16 ? launch_mma_xd_f16(prm, D, BS, max_ctas, st)
                                 : launch_mma_xd_bf16(prm, D, BS, max_ctas, st);
    else if (variant == PA_VARIANT_MMA)
      e = dtype == PA_DTYPE_FP16 ? launch_mma_f16(prm, D, BS, max_ctas, st)
                                 : launch_mma_bf16(prm, D, BS, max_ctas, st);
    else if (dtype == PA_DTYPE_FP32 && BS == 8)
      e = launch_simt_b8_f32(prm, D, max_ctas, st);
    else if (dtype == PA_DTYPE_FP32 && q_len > 1)
      e = base_shape(D, BS) ? launch_simt_mq_f32(prm, D, BS, max_ctas, st)
                            : launch_simtx_mq_f32(prm, D, BS, max_ctas, st);
    else if (dtype == PA_DTYPE_FP32)
      e = base_shape(D, BS) ? launch_simt_f32(prm, D, BS, max_ctas, st)
                            : launch_simtx_f32(prm, D, BS, max_ctas, st);
    else if (!base_shape(D, BS))
      e = dtype == PA_DTYPE_FP16 ? launch_simtx_f16(prm, D, BS, max_ctas, st)
                                 : launch_simtx_bf16(prm, D, BS, max_ctas, st);
    else
      e = dtype == PA_DTYPE_FP16 ? launch_simt_f16(prm, D, BS, max_ctas, st)
                                 : launch_simt_bf16(prm, D, BS, max_ctas, st);
    // (View rows: the next launch has partitions of its own.)
    if (e == cudaSuccess && view) e = combine(s0, n);
    if (e != cudaSuccess) status = PA_ERR_CUDA;
  }
  if (status == PA_OK && !view && combine(0, S) != cudaSuccess) status = PA_ERR_CUDA;
  if (own && cudaFreeAsync(ws, st) != cudaSuccess && status == PA_OK) status = PA_ERR_CUDA;
  return status;
}

}  // namespace

extern "C" int pa_decode_v2_kv4(void* out, float* lse, const void* query, const void* kv_cache,
                                const int32_t* block_tables, const int32_t* seq_lens, float scale,
                                int num_seqs, int num_heads, int num_kv_heads, int head_size,
                                int block_size, int partition_size, int dtype, void* stream,
                                int max_blocks_per_seq, int num_blocks, void* workspace,
                                size_t workspace_bytes) {
  return pa_decode_v2_mq_kv4(out, lse, query, kv_cache, block_tables, seq_lens, scale, num_seqs, 1, num_heads,
                             num_kv_heads, head_size, block_size, partition_size, dtype, stream,
                             max_blocks_per_seq, num_blocks, workspace, workspace_bytes);
}

extern "C" int pa_decode_v2_mq_kv4(void* out, float* lse, const void* query, const void* kv_cache,
                                   const int32_t* block_tables, const int32_t* seq_lens, float scale,
                                   int num_seqs, int q_len, int num_heads, int num_kv_heads, int head_size,
                                   int block_size, int partition_size, int dtype, void* stream,
                                   int max_blocks_per_seq, int num_blocks, void* workspace,
                                   size_t workspace_bytes) {
  return pa_decode_v2_kv4_ex(out, lse, query, kv_cache, block_tables, seq_lens, scale, num_seqs, q_len, num_heads,
                             num_kv_heads, head_size, block_size, partition_size, dtype, stream,
                             max_blocks_per_seq, num_blocks, workspace, workspace_bytes, 0, 0);
}

extern "C" int pa_decode_v2_kv4_ex(void* out, float* lse, const void* query, const void* kv_cache,
                                   const int32_t* block_tables, const int32_t* seq_lens, float scale,
                                   int num_seqs, int q_len, int num_heads, int num_kv_heads, int head_size,
                                   int block_size, int partition_size, int dtype, void* stream,
                                   int max_blocks_per_seq, int num_blocks, void* workspace,
                                   size_t workspace_bytes, int max_ctas, long long timeout_ns) {
  return decode_impl(out, lse, query, kv_cache, kv_cache, block_tables, seq_lens, scale, num_seqs, q_len,
                     num_heads, num_kv_heads, head_size, block_size, partition_size, dtype, stream,
                     max_blocks_per_seq, num_blocks, workspace, workspace_bytes, PA_VARIANT_AUTO, max_ctas,
                     timeout_ns, false, 1.f, 1.f, true);
}

namespace {

// Lengths stay far below 2^30: a longer window, or more first tokens, is all of them.
int view_tokens_arg(int n) { return n < (1 << 30) ? n : 1 << 30; }

}  // namespace

extern "C" size_t pa_decode_v2_view_workspace_bytes(int num_seqs, int q_len, int num_heads, int num_kv_heads,
                                                    int head_size, int max_blocks_per_seq, int block_size,
                                                    int partition_size, int window, int sinks) {
  WsLayout w;
  if (q_len < 1 || q_len > kMaxSeqsPerLaunch || num_heads <= 0 || (long long)num_heads * q_len > 65535 ||
      num_kv_heads <= 0 || num_heads % num_kv_heads != 0 || window < 0 || sinks < 0 || block_size <= 0)
    return 0;
  if (!ws_layout(num_seqs, num_heads * q_len, num_kv_heads, head_size,
                 view_blocks(q_len, max_blocks_per_seq, block_size, window, sinks), block_size, partition_size, &w))
    return 0;
  return w.total;
}

extern "C" int pa_decode_v2_view_ex(void* out, float* lse, const void* query, const void* key_cache,
                                    const void* value_cache, const int32_t* block_tables, const int32_t* seq_lens,
                                    const int32_t* masks, float scale, float k_scale, float v_scale, int window,
                                    int sinks, int num_seqs, int q_len, int num_heads, int num_kv_heads, int head_size,
                                    int block_size, int partition_size, int dtype, int tree, int fp8, void* stream,
                                    int max_blocks_per_seq, int num_blocks, void* workspace, size_t workspace_bytes,
                                    int max_ctas, long long timeout_ns) {
  if (!fp8 && (k_scale != 1.f || v_scale != 1.f)) return PA_ERR_INVALID_ARG;
  const ViewArgs view = {view_tokens_arg(window), view_tokens_arg(sinks), masks, tree != 0};
  return decode_impl(out, lse, query, key_cache, value_cache, block_tables, seq_lens, scale, num_seqs, q_len,
                     num_heads, num_kv_heads, head_size, block_size, partition_size, dtype, stream,
                     max_blocks_per_seq, num_blocks, workspace, workspace_bytes, PA_VARIANT_AUTO, max_ctas, timeout_ns,
                     fp8 != 0, k_scale, v_scale, false, &view);
}

extern "C" int pa_decode_v2_window(void* out, float* lse, const void* query, const void* key_cache,
                                   const void* value_cache, const int32_t* block_tables, const int32_t* seq_lens,
                                   float scale, int window, int sinks, int num_seqs, int q_len, int num_heads,
                                   int num_kv_heads, int head_size, int block_size, int partition_size, int dtype,
                                   void* stream, int max_blocks_per_seq, int num_blocks, void* workspace,
                                   size_t workspace_bytes) {
  return pa_decode_v2_view_ex(out, lse, query, key_cache, value_cache, block_tables, seq_lens, nullptr, scale, 1.f, 1.f,
                              window, sinks, num_seqs, q_len, num_heads, num_kv_heads, head_size, block_size,
                              partition_size, dtype, 0, 0, stream, max_blocks_per_seq, num_blocks, workspace,
                              workspace_bytes, 0, 0);
}

extern "C" int pa_decode_v2_window_fp8(void* out, float* lse, const void* query, const void* key_cache,
                                       const void* value_cache, const int32_t* block_tables,
                                       const int32_t* seq_lens, float scale, float k_scale, float v_scale,
                                       int window, int sinks, int num_seqs, int q_len, int num_heads,
                                       int num_kv_heads, int head_size, int block_size, int partition_size,
                                       int dtype, void* stream, int max_blocks_per_seq, int num_blocks,
                                       void* workspace, size_t workspace_bytes) {
  return pa_decode_v2_view_ex(out, lse, query, key_cache, value_cache, block_tables, seq_lens, nullptr, scale, k_scale,
                              v_scale, window, sinks, num_seqs, q_len, num_heads, num_kv_heads, head_size, block_size,
                              partition_size, dtype, 0, 1, stream, max_blocks_per_seq, num_blocks, workspace,
                              workspace_bytes, 0, 0);
}

extern "C" int pa_decode_v2_tree(void* out, float* lse, const void* query, const void* key_cache,
                                 const void* value_cache, const int32_t* block_tables, const int32_t* seq_lens,
                                 const int32_t* masks, float scale, int window, int sinks, int num_seqs,
                                 int num_nodes, int num_heads, int num_kv_heads, int head_size, int block_size,
                                 int partition_size, int dtype, void* stream, int max_blocks_per_seq,
                                 int num_blocks, void* workspace, size_t workspace_bytes) {
  return pa_decode_v2_view_ex(out, lse, query, key_cache, value_cache, block_tables, seq_lens, masks, scale, 1.f, 1.f,
                              window, sinks, num_seqs, num_nodes, num_heads, num_kv_heads, head_size, block_size,
                              partition_size, dtype, 1, 0, stream, max_blocks_per_seq, num_blocks, workspace,
                              workspace_bytes, 0, 0);
}

extern "C" int pa_decode_v2_tree_fp8(void* out, float* lse, const void* query, const void* key_cache,
                                     const void* value_cache, const int32_t* block_tables,
                                     const int32_t* seq_lens, const int32_t* masks, float scale, float k_scale,
                                     float v_scale, int window, int sinks, int num_seqs, int num_nodes,
                                     int num_heads, int num_kv_heads, int head_size, int block_size,
                                     int partition_size, int dtype, void* stream, int max_blocks_per_seq,
                                     int num_blocks, void* workspace, size_t workspace_bytes) {
  return pa_decode_v2_view_ex(out, lse, query, key_cache, value_cache, block_tables, seq_lens, masks, scale, k_scale,
                              v_scale, window, sinks, num_seqs, num_nodes, num_heads, num_kv_heads, head_size,
                              block_size, partition_size, dtype, 1, 1, stream, max_blocks_per_seq, num_blocks,
                              workspace, workspace_bytes, 0, 0);
}

extern "C" int pa_decode_v2_ex(void* out, const void* query, const void* key_cache,
                               const void* value_cache, const int32_t* block_tables,
                               const int32_t* seq_lens, float scale, int num_seqs, int num_heads,
                               int num_kv_heads, int head_size, int block_size, int partition_size,
                               int dtype, void* stream, int max_blocks_per_seq, int num_blocks,
                               void* workspace, size_t workspace_bytes, int variant, int max_ctas,
                               long long timeout_ns) {
  return decode_impl(out, nullptr, query, key_cache, value_cache, block_tables, seq_lens, scale,
                     num_seqs, 1, num_heads, num_kv_heads, head_size, block_size, partition_size,
                     dtype, stream, max_blocks_per_seq, num_blocks, workspace, workspace_bytes,
                     variant, max_ctas, timeout_ns);
}

extern "C" int pa_decode_v2_lse(void* out, float* lse, const void* query, const void* key_cache,
                                const void* value_cache, const int32_t* block_tables,
                                const int32_t* seq_lens, float scale, int num_seqs, int num_heads,
                                int num_kv_heads, int head_size, int block_size, int partition_size,
                                int dtype, void* stream, int max_blocks_per_seq, int num_blocks,
                                void* workspace, size_t workspace_bytes) {
  return decode_impl(out, lse, query, key_cache, value_cache, block_tables, seq_lens, scale,
                     num_seqs, 1, num_heads, num_kv_heads, head_size, block_size, partition_size,
                     dtype, stream, max_blocks_per_seq, num_blocks, workspace, workspace_bytes,
                     PA_VARIANT_AUTO, 0, 0);
}

extern "C" int pa_decode_v2_fp8(void* out, float* lse, const void* query, const void* key_cache,
                                const void* value_cache, const int32_t* block_tables,
                                const int32_t* seq_lens, float scale, float k_scale, float v_scale,
                                int num_seqs, int num_heads, int num_kv_heads, int head_size,
                                int block_size, int partition_size, int dtype, void* stream,
                                int max_blocks_per_seq, int num_blocks, void* workspace,
                                size_t workspace_bytes) {
  return decode_impl(out, lse, query, key_cache, value_cache, block_tables, seq_lens, scale,
                     num_seqs, 1, num_heads, num_kv_heads, head_size, block_size, partition_size,
                     dtype, stream, max_blocks_per_seq, num_blocks, workspace, workspace_bytes,
                     PA_VARIANT_AUTO, 0, 0, true, k_scale, v_scale);
}

extern "C" int pa_decode_v2_mq(void* out, float* lse, const void* query, const void* key_cache,
                               const void* value_cache, const int32_t* block_tables,
                               const int32_t* seq_lens, float scale, int num_seqs, int q_len,
                               int num_heads, int num_kv_heads, int head_size, int block_size,
                               int partition_size, int dtype, void* stream, int max_blocks_per_seq,
                               int num_blocks, void* workspace, size_t workspace_bytes) {
  return decode_impl(out, lse, query, key_cache, value_cache, block_tables, seq_lens, scale,
                     num_seqs, q_len, num_heads, num_kv_heads, head_size, block_size,
                     partition_size, dtype, stream, max_blocks_per_seq, num_blocks, workspace,
                     workspace_bytes, PA_VARIANT_AUTO, 0, 0);
}

extern "C" int pa_decode_v2_mq_fp8(void* out, float* lse, const void* query, const void* key_cache,
                                   const void* value_cache, const int32_t* block_tables,
                                   const int32_t* seq_lens, float scale, float k_scale, float v_scale,
                                   int num_seqs, int q_len, int num_heads, int num_kv_heads, int head_size,
                                   int block_size, int partition_size, int dtype, void* stream,
                                   int max_blocks_per_seq, int num_blocks, void* workspace,
                                   size_t workspace_bytes) {
  return decode_impl(out, lse, query, key_cache, value_cache, block_tables, seq_lens, scale,
                     num_seqs, q_len, num_heads, num_kv_heads, head_size, block_size,
                     partition_size, dtype, stream, max_blocks_per_seq, num_blocks, workspace,
                     workspace_bytes, PA_VARIANT_AUTO, 0, 0, true, k_scale, v_scale);
}

extern "C" int pa_decode_v2(void* out, const void* query, const void* key_cache, const void* value_cache,
                            const int32_t* block_tables, const int32_t* seq_lens, float scale,
                            int num_seqs, int num_heads, int num_kv_heads, int head_size,
                            int block_size, int partition_size, int dtype, void* stream,
                            int max_blocks_per_seq, int num_blocks, void* workspace,
                            size_t workspace_bytes) {
  return pa_decode_v2_ex(out, query, key_cache, value_cache, block_tables, seq_lens, scale, num_seqs,
                         num_heads, num_kv_heads, head_size, block_size, partition_size, dtype, stream,
                         max_blocks_per_seq, num_blocks, workspace, workspace_bytes, PA_VARIANT_AUTO, 0, 0);
}

namespace {
// Staging for the host-I/O entry point, placed after the regular workspace.
struct HostIoLayout {
  size_t q, out, bt, lens, total;
};
bool host_io_layout(int S, int H, int KH, int D, int MB, int BS, int P, HostIoLayout* h, WsLayout* w) {
  if (!ws_layout(S, H, KH, D, MB, BS, P, w)) return false;
  const size_t qbytes = (size_t)S * H * D * 4;  // room for the widest element type
  h->q = w->total;
  h->out = align_up(h->q + qbytes);
  h->bt = align_up(h->out + qbytes);
  h->lens = align_up(h->bt + (size_t)S * MB * sizeof(int32_t));
  h->total = align_up(h->lens + (size_t)S * sizeof(int32_t));
  return true;
}
}  // namespace

extern "C" size_t pa_decode_v2_host_io_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads,
                                                       int head_size, int max_blocks_per_seq,
                                                       int block_size, int partition_size) {
  HostIoLayout h;
  WsLayout w;
  if (!host_io_layout(num_seqs, num_heads, num_kv_heads, head_size, max_blocks_per_seq, block_size,
                      partition_size, &h, &w))
    return 0;
  return h.total;
}

extern "C" int pa_decode_v2_host_io(void* out_host, const void* query_host, const void* key_cache,
                                    const void* value_cache, const int32_t* block_tables_host,
                                    const int32_t* seq_lens_host, float scale, int num_seqs,
                                    int num_heads, int num_kv_heads, int head_size, int block_size,
                                    int partition_size, int dtype, void* stream,
                                    int max_blocks_per_seq, int num_blocks, void* workspace,
                                    size_t workspace_bytes) {
  const int S = num_seqs, H = num_heads, D = head_size, MB = max_blocks_per_seq;
  HostIoLayout h;
  WsLayout w;
  if (!host_io_layout(S, H, num_kv_heads, D, MB, block_size, partition_size, &h, &w))
    return PA_ERR_INVALID_ARG;
  if (S == 0) return PA_OK;
  if (!out_host || !query_host || !block_tables_host || !seq_lens_host || !workspace)
    return PA_ERR_INVALID_ARG;
  if (!aligned(workspace, 16)) return PA_ERR_INVALID_ARG;
  if (workspace_bytes < h.total) return PA_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype != PA_DTYPE_FP16 && dtype != PA_DTYPE_BF16 && dtype != PA_DTYPE_FP32) return PA_ERR_INVALID_ARG;
  const size_t qbytes = (size_t)S * H * D * elem_bytes(dtype);
  if (cudaMemcpyAsync(ws + h.q, query_host, qbytes, cudaMemcpyHostToDevice, st) != cudaSuccess ||
      cudaMemcpyAsync(ws + h.bt, block_tables_host, (size_t)S * MB * sizeof(int32_t),
                      cudaMemcpyHostToDevice, st) != cudaSuccess ||
      cudaMemcpyAsync(ws + h.lens, seq_lens_host, (size_t)S * sizeof(int32_t), cudaMemcpyHostToDevice,
                      st) != cudaSuccess)
    return PA_ERR_CUDA;
  const int status = pa_decode_v2(ws + h.out, ws + h.q, key_cache, value_cache,
                                  reinterpret_cast<const int32_t*>(ws + h.bt),
                                  reinterpret_cast<const int32_t*>(ws + h.lens), scale, S, H,
                                  num_kv_heads, D, block_size, partition_size, dtype, stream, MB,
                                  num_blocks, ws, w.total);
  if (status != PA_OK) return status;
  if (cudaMemcpyAsync(out_host, ws + h.out, qbytes, cudaMemcpyDeviceToHost, st) != cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
}

extern "C" int pa_decode_v2_device_status(const void* workspace, void* stream, int* status) {
  if (!workspace || !status) return PA_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int v = 0;
  if (cudaMemcpyAsync(&v, workspace, sizeof v, cudaMemcpyDeviceToHost, st) != cudaSuccess) return PA_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return PA_ERR_CUDA;
  *status = v;
  return PA_OK;
}

extern "C" const char* pa_decode_v2_status_string(int status) {
  switch (status) {
    case PA_OK: return "ok";
    case PA_ERR_INVALID_ARG: return "invalid argument";
    case PA_ERR_UNSUPPORTED: return "unsupported configuration";
    case PA_ERR_WORKSPACE: return "workspace too small";
    case PA_ERR_CUDA: return "CUDA runtime error";
    case PA_ERR_DEVICE_BOUNDS: return "device-side bounds violation (block id or sequence length)";
    case PA_ERR_TIMEOUT: return "device-side wait timed out";
    case PA_ERR_NO_BLOCKS: return "too few free blocks in the pool";
    default: return "unknown status";
  }
}
