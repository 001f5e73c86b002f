// pa_launch.h -- internal interface between the C ABI (pa_api.cu) and the
// kernel instantiation units.
#pragma once

#include <cuda_runtime.h>

#include "pa_combine.cuh"
#include "pa_kernel.cuh"

namespace pa {

// Query heads per work unit of each kernel family (the tensor-core family
// takes 16 where a kv head has more than 8 query rows).
constexpr int kSimtGroup = 1;
constexpr int kMmaGroup = 8;
constexpr int kMmaGroupWide = 16;

// Launch the persistent kernel for one chunk of sequences.  Returns a cudaError_t.
cudaError_t launch_simt_f16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_simt_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_simt_f32(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
// CUDA-core instances of head sizes 80, 96, 112 (blocks of 16, 32, 64) and of
// 64-token blocks at head sizes 64, 128 (fp16 / bf16).
cudaError_t launch_simtx_f16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_simtx_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_simtx_f32(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
// Multi-query rows with fp32 elements: the causal instances, base and further shapes.
cudaError_t launch_simt_mq_f32(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_simtx_mq_f32(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
// fp32 caches in 8-token blocks, single- and multi-query.
cudaError_t launch_simt_b8_f32(const KParams& prm, int D, int max_ctas, cudaStream_t st);
cudaError_t launch_mma_f16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_mma_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_mma16_f16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_mma16_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
// Tensor-core instances of the other shapes: head sizes 80, 96, 112 (block
// sizes 16, 32), and 8- or 64-token blocks (head sizes 64, 80, 96, 112, 128, 256).
cudaError_t launch_mma_xd_f16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_mma_xd_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_mma_b8_f16(const KParams& prm, int D, int max_ctas, cudaStream_t st);
cudaError_t launch_mma_b8_bf16(const KParams& prm, int D, int max_ctas, cudaStream_t st);
cudaError_t launch_mma_b64_f16(const KParams& prm, int D, int max_ctas, cudaStream_t st);
cudaError_t launch_mma_b64_bf16(const KParams& prm, int D, int max_ctas, cudaStream_t st);
// Tensor-core instances over pairs of kv heads (4 query heads per kv head,
// head sizes up to 128), in 8-, 16- and 32-token blocks.
cudaError_t launch_mma_g8_f16(const KParams& prm, int D, int max_ctas, cudaStream_t st);
cudaError_t launch_mma_g8_bf16(const KParams& prm, int D, int max_ctas, cudaStream_t st);
cudaError_t launch_mma_g16_f16(const KParams& prm, int D, int max_ctas, cudaStream_t st);
cudaError_t launch_mma_g16_bf16(const KParams& prm, int D, int max_ctas, cudaStream_t st);
cudaError_t launch_mma_g32_f16(const KParams& prm, int D, int max_ctas, cudaStream_t st);
cudaError_t launch_mma_g32_bf16(const KParams& prm, int D, int max_ctas, cudaStream_t st);
// The same over an fp8 (E4M3) KV cache, queries and output fp16 / bf16.
cudaError_t launch_mma8_f16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_mma8_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
// (head sizes 64, 128, 256 with 16- or 32-token blocks), at head sizes 80, 96,
// 112 with 16- or 32-token blocks (_x), and in 8- or 64-token blocks (_b8, _b64).
cudaError_t launch_mma8_x_f16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_mma8_x_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_mma8_b8_f16(const KParams& prm, int D, int max_ctas, cudaStream_t st);
cudaError_t launch_mma8_b8_bf16(const KParams& prm, int D, int max_ctas, cudaStream_t st);
cudaError_t launch_mma8_b64_f16(const KParams& prm, int D, int max_ctas, cudaStream_t st);
cudaError_t launch_mma8_b64_bf16(const KParams& prm, int D, int max_ctas, cudaStream_t st);
// ... and over pairs of kv heads (4 query heads per kv head): head sizes 64
// and 128 with 16- or 32-token blocks, 80, 96, 112 with 16- or 32-token
// blocks (_gx), and every head size up to 128 in 8-token blocks (_gb8).
cudaError_t launch_mma8_g_f16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_mma8_g_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_mma8_gx_f16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_mma8_gx_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_mma8_gb8_f16(const KParams& prm, int D, int max_ctas, cudaStream_t st);
cudaError_t launch_mma8_gb8_bf16(const KParams& prm, int D, int max_ctas, cudaStream_t st);

// View rows (windows, trees): 16-bit caches by units of one kv head, in blocks of
// 16 or 32 tokens, of 8 or 64 (_b), and of pairs of kv heads (_g: up to 128 dims,
// blocks of up to 32 tokens); the same over E4M3 caches (8); fp32 caches.
cudaError_t launch_view_f16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_view_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_view_b_f16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_view_b_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_view_g_f16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_view_g_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_view8_f16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_view8_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_view8_b_f16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_view8_b_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_view8_g_f16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_view8_g_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_view_f32(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_view_x_f32(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
// ... and with many rows a kv head (rows8: over E4M3 caches; _x: head sizes from 112).
cudaError_t launch_rows_f16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_rows_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_rows_x_f16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_rows_x_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_rows8_f16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_rows8_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_rows8_x_f16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
cudaError_t launch_rows8_x_bf16(const KParams& prm, int D, int BS, int max_ctas, cudaStream_t st);
// Sequences of a launch, and rows of a unit.
constexpr int kRowsSeqsPerLaunch = 256;
constexpr int kRowsPerUnit = 128;

// Over a 4-bit cache (queries and output fp16 / bf16), by head size: blocks of
// 8, 16, 32 or 64 tokens, units of nt * 8 query rows of a kv head, or (kvu = 2, up
// to four rows each) of two kv heads; either 2: head sizes up to 128, and kvu = 2:
// blocks of up to 32 tokens.
cudaError_t launch_kv4_d64_f16(const KParams& prm, int BS, int nt, int kvu, int max_ctas, cudaStream_t st);
cudaError_t launch_kv4_d64_bf16(const KParams& prm, int BS, int nt, int kvu, int max_ctas, cudaStream_t st);
cudaError_t launch_kv4_d80_f16(const KParams& prm, int BS, int nt, int kvu, int max_ctas, cudaStream_t st);
cudaError_t launch_kv4_d80_bf16(const KParams& prm, int BS, int nt, int kvu, int max_ctas, cudaStream_t st);
cudaError_t launch_kv4_d96_f16(const KParams& prm, int BS, int nt, int kvu, int max_ctas, cudaStream_t st);
cudaError_t launch_kv4_d96_bf16(const KParams& prm, int BS, int nt, int kvu, int max_ctas, cudaStream_t st);
cudaError_t launch_kv4_d112_f16(const KParams& prm, int BS, int nt, int kvu, int max_ctas, cudaStream_t st);
cudaError_t launch_kv4_d112_bf16(const KParams& prm, int BS, int nt, int kvu, int max_ctas, cudaStream_t st);
cudaError_t launch_kv4_d128_f16(const KParams& prm, int BS, int nt, int kvu, int max_ctas, cudaStream_t st);
cudaError_t launch_kv4_d128_bf16(const KParams& prm, int BS, int nt, int kvu, int max_ctas, cudaStream_t st);
cudaError_t launch_kv4_d256_f16(const KParams& prm, int BS, int nt, int kvu, int max_ctas, cudaStream_t st);
cudaError_t launch_kv4_d256_bf16(const KParams& prm, int BS, int nt, int kvu, int max_ctas, cudaStream_t st);
// Phase 2: the cross-partition combine of every multi-partition row, launched
// as a programmatic dependent of the phase-1 launch before it on `st`.
cudaError_t launch_combine(const CParams& prm, int elem_bytes, bool bf16, int D, cudaStream_t st);

// SM count of the current device (cached per device).
int device_sm_count();

}  // namespace pa
