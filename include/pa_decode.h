/*
 * pa_decode.h -- C ABI of a GB300 (sm_103a) paged decode attention library
 * ("PagedAttention V2": partitioned online softmax followed by a
 * cross-partition log-sum-exp combine): single-query decode (pa_decode_v2,
 * pa_decode_v2_ex, pa_decode_v2_lse), multi-query decode (pa_decode_v2_mq),
 * sliding windows (pa_decode_v2_window), trees of drafted tokens
 * (pa_decode_v2_tree; pa_tree_masks, pa_tree_accept), slot maps and the writing of
 * new tokens (pa_pages_slots, pa_cache_write),
 * E4M3 (fp8) caches (pa_decode_v2_fp8), 4-bit caches (pa_decode_v2_kv4,
 * pa_decode_v2_mq_kv4; written and read back with pa_kv4_append and
 * pa_kv4_gather), the pages of a pool managed on the device (pa_pages_fork,
 * pa_pages_resize, pa_pages_compact), host-resident per-step inputs
 * (pa_decode_v2_host_io) and a no-allocation variant
 * (pa_decode_v2_static_scratch).
 *
 * What it computes, per sequence s and query head h (the page
 * "paged_attention_v2_triton.py -- Triton PagedAttention V2 for BI-V100",
 * kernels `_paged_attn_v2_partition_kernel` and `_paged_attn_v2_reduce_kernel`
 * and the module docstring's Phase 2 formula):
 *
 *   kv   = h / (num_heads / num_kv_heads)                 (consecutive GQA groups)
 *   for t < L = seq_lens[s]:  b = block_tables[s, t / block_size], o = t % block_size
 *       K_t[d] = key_cache  [b, kv, d / x, o, d % x]      x = 16 / sizeof(element):
 *                                                         8 (fp16/bf16), 4 (fp32), 16 (E4M3)
 *       V_t[d] = value_cache[b, kv, d, o]
 *       z_t    = scale * sum_d query[s, h, d] * K_t[d]    (fp32)
 *   out[s, h, :] = sum_t softmax(z)_t * V_t               rounded to the element type
 *
 * computed in partitions of `partition_size` tokens: partition p holds tokens
 * [p*P, min((p+1)*P, L)) and yields (m_p, l_p, o_p) = (max z, sum e^(z - m_p),
 * normalised weighted V) -- phase 1, one persistent kernel; the partitions
 * are then combined with M = max m_p, w_p = e^(m_p - M) l_p / sum_q e^(m_q - M)
 * l_q, out = sum w_p o_p -- phase 2, a second kernel launched as a
 * programmatic dependent of the first (it starts while the first finishes and
 * waits for its results).  A sequence that fits in one partition is written
 * directly by phase 1 (single pass); a call in which no sequence can have two
 * partitions launches phase 1 only.
 * L = 0 yields zeros (the "flash_attention.metal" page's forward kernel takes
 * 1/l as 0 when l = 0).
 *
 * Memory: every pointer argument of pa_decode_v2 is a DEVICE pointer on the
 * current CUDA device; tensors are contiguous row-major.  The caller owns all
 * buffers.  The library reads query, caches, tables and lengths, and writes
 * `out` and `workspace` only.  Calls are enqueued on `stream` (a cudaStream_t,
 * NULL = legacy default stream) and never synchronise; results are ready when
 * the stream reaches that point.  Concurrent calls must not share a workspace.
 *
 * Errors: argument problems are reported by the return value before anything
 * is enqueued.  Problems only visible on the device (a block id outside
 * [0, num_blocks), seq_lens[s] outside [0, max_blocks_per_seq*block_size], a
 * bounded wait that ran out) are recorded in the workspace's error word, read
 * with pa_decode_v2_device_status(); the kernel never traps and never reads
 * outside the caches when it records a bad block id.
 */
#ifndef PA_DECODE_H
#define PA_DECODE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of query, caches and output. */
enum { PA_DTYPE_FP16 = 0, PA_DTYPE_BF16 = 1, PA_DTYPE_FP32 = 2 };
/* ... and of caches alone (pa_cache_write, pa_tree_accept). */
enum { PA_DTYPE_E4M3 = 3 };

/* Status codes. */
enum {
    PA_OK = 0,
    PA_ERR_INVALID_ARG = 1,   /* null/misaligned pointer, negative size, H % KH != 0, ... */
    PA_ERR_UNSUPPORTED = 2,   /* head_size not 64/80/96/112/128/256, block_size not
                                 8/16/32/64, partition_size not a positive multiple of
                                 block_size; a shape outside the chosen family (see
                                 pa_decode_v2_ex and pa_decode_v2_fp8) */
    PA_ERR_WORKSPACE = 3,     /* workspace smaller than pa_decode_v2_workspace_bytes() */
    PA_ERR_CUDA = 4,          /* a CUDA runtime call failed (launch, memset, ...) */
    PA_ERR_DEVICE_BOUNDS = 5, /* device-side: bad block id or sequence length */
    PA_ERR_TIMEOUT = 6,       /* device-side: a bounded wait gave up */
    PA_ERR_NO_BLOCKS = 7      /* device-side: the pool has too few free blocks */
};

/* Kernel families (pa_decode_v2_ex's `variant`). */
enum {
    PA_VARIANT_AUTO = 0,      /* SIMT when each kv head serves one query head (MHA), MMA otherwise */
    PA_VARIANT_SIMT = 1,      /* CUDA-core dot products and warp-shuffle reductions */
    PA_VARIANT_MMA = 2        /* mma.sync m16n8k16 over the [group x D] . [D x tokens] contraction */
};

/*
 * Bytes of device workspace pa_decode_v2 needs for these sizes: a 256-byte
 * header (error word, work counter, where a bounded wait gave up) and the
 * phase-1 partition states of the page's launcher -- max_logits
 * [S, H, Pmax] f32, exp_sums [S, H, Pmax] f32 and tmp_output
 * [S, H, Pmax, head_size] f32, with
 * Pmax = ceil(max_blocks_per_seq * block_size / partition_size).
 * Returns 0 for invalid sizes.
 */
size_t pa_decode_v2_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_size,
                                    int max_blocks_per_seq, int block_size, int partition_size);

/*
 * Byte offsets of the workspace regions (for inspection in tests):
 * offsets[0] = max_logits (m_p, natural-log units, -inf for unused partitions),
 * offsets[1] = exp_sums (l_p, 0 for unused partitions),
 * offsets[2] = tmp_output (o_p, normalised; written only for sequences with
 *              more than one partition), offsets[3] = header (int32 error word
 *              at index 0), offsets[4] = total bytes.  *max_partitions = Pmax.
 * Returns PA_OK or PA_ERR_INVALID_ARG.
 */
int pa_decode_v2_workspace_layout(int num_seqs, int num_heads, int num_kv_heads, int head_size,
                                  int max_blocks_per_seq, int block_size, int partition_size,
                                  size_t offsets[5], int* max_partitions);

/*
 * Paged decode attention (see the top of this file).
 *   out          [num_seqs, num_heads, head_size]                      dtype, written
 *   query        [num_seqs, num_heads, head_size]                      dtype
 *   key_cache    [num_blocks, num_kv_heads, head_size/x, block_size, x] dtype,
 *                x = 16 / sizeof(element): 8 for fp16/bf16, 4 for fp32
 *   value_cache  [num_blocks, num_kv_heads, head_size, block_size]      dtype
 *   block_tables [num_seqs, max_blocks_per_seq] int32; entries past
 *                ceil(seq_lens[s]/block_size) are never read
 *   seq_lens     [num_seqs] int32, each in [0, max_blocks_per_seq*block_size]
 *   scale        softmax scale applied to q.k (fp32)
 *   dtype        PA_DTYPE_FP16, PA_DTYPE_BF16 or PA_DTYPE_FP32 (fp32 runs on the
 *                CUDA-core family, one query head per pass, every head size
 *                and block size, single- and multi-query; PA_ERR_UNSUPPORTED
 *                for the tensor-core variant and fp8 caches)
 *   stream       cudaStream_t to enqueue on
 *   max_blocks_per_seq  row stride of block_tables (the page's launcher reads
 *                it from the tensor's shape; a C ABI has to be told)
 *   num_blocks   number of physical blocks in each cache (bounds checks)
 *   workspace    device buffer of >= pa_decode_v2_workspace_bytes() bytes,
 *                16-byte aligned; NULL makes the call allocate and free one
 *                stream-ordered (cudaMallocAsync / cudaFreeAsync).  Its
 *                contents on entry do not matter: the call writes every byte
 *                of it that it reads.
 * out, query and the caches must be 16-byte aligned; tables 4-byte aligned.
 * With a workspace given, a call only enqueues kernels on `stream` (no
 * allocation, no synchronisation), so it can be captured into a CUDA graph
 * and replayed with new contents in its buffers (lengths up to the table's
 * capacity); the first call for a given shape should come before the capture.
 */
int pa_decode_v2(void* out, const void* query, const void* key_cache, const void* value_cache,
                 const int32_t* block_tables, const int32_t* seq_lens, float scale,
                 int num_seqs, int num_heads, int num_kv_heads, int head_size,
                 int block_size, int partition_size, int dtype, void* stream,
                 int max_blocks_per_seq, int num_blocks, void* workspace, size_t workspace_bytes);

/*
 * pa_decode_v2 with tuning controls, for tests and measurement.
 *   variant     PA_VARIANT_*; SIMT takes one query head per pass over the
 *               kv head's blocks (a group of G query heads takes G passes),
 *               MMA up to 8 query heads per pass (with G = 4, those of two kv
 *               heads, one block of each per pass; head sizes up to 128,
 *               blocks of 8, 16 or 32 tokens, an even kv-head count).  SIMT handles head sizes
 *               64/128/256 with blocks of 16 or 32 tokens, 80/96/112 with
 *               blocks of 16, 32 or 64, and 64/128 with blocks of 64, and
 *               fp32 in 8-token blocks at every head size (16-bit types in
 *               8-token blocks: PA_ERR_UNSUPPORTED); MMA every supported
 *               shape of the 16-bit types.  AUTO picks SIMT for G = 1 or fp32 where it
 *               applies, MMA otherwise.
 *   max_ctas    upper bound on the persistent grid (0 = one CTA per SM).
 *   timeout_ns  bound on every device-side wait (0 = 2^31 ns).
 * Results do not depend on variant-independent choices: for a fixed variant
 * the output is bitwise identical for every max_ctas.
 */
int pa_decode_v2_ex(void* out, const void* query, const void* key_cache, const void* value_cache,
                    const int32_t* block_tables, const int32_t* seq_lens, float scale,
                    int num_seqs, int num_heads, int num_kv_heads, int head_size,
                    int block_size, int partition_size, int dtype, void* stream,
                    int max_blocks_per_seq, int num_blocks, void* workspace, size_t workspace_bytes,
                    int variant, int max_ctas, long long timeout_ns);

/*
 * pa_decode_v2 that also returns, per (sequence, head), the log-sum-exp of
 * the scaled scores:
 *     lse[s * num_heads + h] = log( sum_t exp(scale * q[s,h] . k_t) )
 * over the sequence's seq_lens[s] tokens, natural log, fp32; -INFINITY for a
 * sequence with no tokens.  It is the value the forward kernel of the page
 * "flash_attention.metal -- Flash Attention Metal Shaders" stores beside its
 * output (its running maximum plus the log of its running sum, "log-sum-exp
 * for backward pass"), reached here by the same cross-partition combine as
 * the output (page "paged_attention_v2_triton.py -- Triton PagedAttention V2
 * for BI-V100", module docstring: M = max m_p, total = sum exp(m_p - M) l_p,
 * lse = M + log total).  With it, outputs computed over disjoint token sets
 * (for example the two halves of a sequence split across calls or devices)
 * merge exactly: out = sum_i exp(lse_i - LSE) out_i, LSE = log sum_i exp(lse_i).
 *   lse   DEVICE buffer of num_seqs * num_heads floats, 4-byte aligned, written
 *         (NULL: behaves as pa_decode_v2).
 * Every other argument, the ownership and the errors are those of
 * pa_decode_v2 (the kernel family is chosen as PA_VARIANT_AUTO); a misaligned
 * lse is PA_ERR_INVALID_ARG.
 */
int pa_decode_v2_lse(void* out, float* lse, const void* query, const void* key_cache,
                     const void* value_cache, const int32_t* block_tables, const int32_t* seq_lens,
                     float scale, int num_seqs, int num_heads, int num_kv_heads, int head_size,
                     int block_size, int partition_size, int dtype, void* stream,
                     int max_blocks_per_seq, int num_blocks, void* workspace, size_t workspace_bytes);

/*
 * pa_decode_v2_lse over an fp8 KV cache.  The launcher of page
 * "paged_attention_v2_triton.py -- Triton PagedAttention V2 for BI-V100" takes
 * kv_cache_dtype, k_scale and v_scale (and ignores them); here the caches hold
 * E4M3 codes ("e4m3fn": sign, 4 exponent bits with bias 7, 3 fraction bits,
 * no infinities, code 0x7f/0xff NaN) and the real keys and values are
 * k_scale * K and v_scale * V.  With one-byte elements the key layout's x is
 * 16 (16 bytes per chunk, as the launcher's x_pack = key_cache.shape[-1]):
 *   key_cache    [num_blocks, num_kv_heads, head_size/16, block_size, 16] uint8
 *   value_cache  [num_blocks, num_kv_heads, head_size, block_size]        uint8
 *   query, out   [num_seqs, num_heads, head_size]   dtype (fp16 or bf16)
 *   k_scale, v_scale   finite fp32 multipliers (PA_ERR_INVALID_ARG otherwise)
 * Every other argument, the workspace, ownership and errors are those of
 * pa_decode_v2_lse.  The tensor-core kernel family runs every group size
 * and every shape pa_decode_v2 takes: head_size 64, 80, 96, 112, 128 or 256,
 * block_size 8, 16, 32 or 64 (PA_ERR_UNSUPPORTED otherwise).
 */
int pa_decode_v2_fp8(void* out, float* lse, const void* query, const void* key_cache,
                     const void* value_cache, const int32_t* block_tables, const int32_t* seq_lens,
                     float scale, float k_scale, float v_scale, int num_seqs, int num_heads,
                     int num_kv_heads, int head_size, int block_size, int partition_size, int dtype,
                     void* stream, int max_blocks_per_seq, int num_blocks, void* workspace,
                     size_t workspace_bytes);

/*
 * Multi-query decode: q_len new tokens per sequence (speculative or
 * multi-token-prediction verification), each query row attending causally.
 * The decode of page "paged_attention_v2_triton.py -- Triton PagedAttention V2
 * for BI-V100" is its one-row case (module docstring: "For decode
 * (BLOCK_M=1), the Q tile is just one vector"); q_len > 1 rows follow the
 * causal rule of the prefix-prefill kernel its paged gather comes from: the
 * sequence's last q_len cached tokens are the new ones, and query row i sits
 * at position L - q_len + i (L = seq_lens[s]) and attends to positions
 * 0 .. L - q_len + i.  Their K and V must already be in the cache.
 *   query, out  [num_seqs, q_len, num_heads, head_size]   dtype
 *   lse         NULL, or DEVICE [num_seqs, q_len, num_heads] fp32 (as in
 *               pa_decode_v2_lse), written
 *   seq_lens    [num_seqs] int32, each in [q_len, max_blocks_per_seq*block_size]
 *               (a length below q_len is recorded as PA_ERR_DEVICE_BOUNDS)
 *   q_len       1 .. 1024 (q_len = 1 is pa_decode_v2_lse)
 *   workspace   >= pa_decode_v2_workspace_bytes(num_seqs * q_len, ...) bytes, or NULL
 * The other arguments, ownership and errors are those of pa_decode_v2 (kernel
 * family chosen as PA_VARIANT_AUTO).  The q_len query rows of a sequence share
 * its K/V loads: each kv head's q_len * (num_heads / num_kv_heads) rows are
 * the rows of the tensor-core product (8 or 16 per work unit), each masked to
 * the positions it may see; fp32 rows run on the CUDA-core family, one row
 * per pass.
 */
int pa_decode_v2_mq(void* out, float* lse, const void* query, const void* key_cache,
                    const void* value_cache, const int32_t* block_tables, const int32_t* seq_lens,
                    float scale, int num_seqs, int q_len, int num_heads, int num_kv_heads,
                    int head_size, int block_size, int partition_size, int dtype, void* stream,
                    int max_blocks_per_seq, int num_blocks, void* workspace, size_t workspace_bytes);

/*
 * Multi-query decode over an fp8 (E4M3) KV cache: the q_len causal query rows
 * of pa_decode_v2_mq (row i of sequence s sits at position L - q_len + i and
 * sees positions 0 .. L - q_len + i) with the caches, scales and element
 * reading of pa_decode_v2_fp8 (the launcher of "paged_attention_v2_triton.py
 * -- Triton PagedAttention V2 for BI-V100" takes kv_cache_dtype, k_scale and
 * v_scale whatever the query rows).
 *   query, out   [num_seqs, q_len, num_heads, head_size]   dtype (fp16 or bf16)
 *   key_cache    [num_blocks, num_kv_heads, head_size/16, block_size, 16] uint8
 *   value_cache  [num_blocks, num_kv_heads, head_size, block_size]        uint8
 *   lse          NULL, or DEVICE [num_seqs, q_len, num_heads] fp32, written
 *   k_scale, v_scale   finite fp32 multipliers (PA_ERR_INVALID_ARG otherwise)
 *   seq_lens     each in [q_len, max_blocks_per_seq*block_size]
 *   workspace    >= pa_decode_v2_workspace_bytes(num_seqs * q_len, ...) bytes, or NULL
 * Shapes as for pa_decode_v2_fp8 (PA_ERR_UNSUPPORTED otherwise); every other
 * argument, the ownership and the errors are those of pa_decode_v2_mq.
 */
int pa_decode_v2_mq_fp8(void* out, float* lse, const void* query, const void* key_cache,
                        const void* value_cache, const int32_t* block_tables, const int32_t* seq_lens,
                        float scale, float k_scale, float v_scale, int num_seqs, int q_len,
                        int num_heads, int num_kv_heads, int head_size, int block_size,
                        int partition_size, int dtype, void* stream, int max_blocks_per_seq,
                        int num_blocks, void* workspace, size_t workspace_bytes);

/*
 * Attention to a sliding window and to the first tokens, for layers that look
 * back a fixed number of tokens.  Rows, tables and lengths are those of
 * pa_decode_v2_mq (q_len = 1: of pa_decode_v2_lse): row i of sequence s is at
 * position p = L - q_len + i, and sees position t where
 *     t <= p   and   (t > p - window  or  t < sinks)
 * so a window counts the row's own token.  A window of L or more is
 * pa_decode_v2_mq's rule.
 *   window      1 or more
 *   sinks       first tokens that stay visible, 0 or more
 *   seq_lens    [num_seqs] int32, each in [q_len, max_blocks_per_seq*block_size];
 *               a single row (q_len = 1) also takes 0.  Other lengths are recorded
 *               as PA_ERR_DEVICE_BOUNDS; a length below q_len then gives zeros and
 *               -INFINITY, as an empty sequence does.
 *   block_tables  only the entries of blocks with a position that some row of
 *               the sequence sees are read: blocks between the first tokens and
 *               the window may have been given back
 *   q_len       1 .. 512
 *   workspace   >= pa_decode_v2_view_workspace_bytes(num_seqs, q_len, ...) bytes,
 *               or NULL.  Partitions count the visible blocks only.  Over 16-bit
 *               and E4M3 caches several are taken together where the lengths leave
 *               every SM its share of the work without them: on the device, from the
 *               lengths of the call (of each 256 or 512 sequences of it), whatever
 *               room the tables have.
 * Elements, shapes, lse, ownership and errors are those of pa_decode_v2_mq (fp32:
 * not blocks of 64 tokens at head size 256, PA_ERR_UNSUPPORTED).  A key or value
 * that is not finite reaches the rows that see it, no others: they are not finite
 * where they would be by the formula (an infinite value may give NaN, where its
 * weight is 0 or is held in two terms).
 */
int pa_decode_v2_window(void* out, float* lse, const void* query, const void* key_cache,
                        const void* value_cache, const int32_t* block_tables, const int32_t* seq_lens,
                        float scale, int window, int sinks, int num_seqs, int q_len, int num_heads,
                        int num_kv_heads, int head_size, int block_size, int partition_size, int dtype,
                        void* stream, int max_blocks_per_seq, int num_blocks, void* workspace,
                        size_t workspace_bytes);

/* pa_decode_v2_window over an E4M3 cache (caches and scales of pa_decode_v2_mq_fp8). */
int pa_decode_v2_window_fp8(void* out, float* lse, const void* query, const void* key_cache,
                            const void* value_cache, const int32_t* block_tables, const int32_t* seq_lens,
                            float scale, float k_scale, float v_scale, int window, int sinks, int num_seqs,
                            int q_len, int num_heads, int num_kv_heads, int head_size, int block_size,
                            int partition_size, int dtype, void* stream, int max_blocks_per_seq,
                            int num_blocks, void* workspace, size_t workspace_bytes);

/*
 * Attention for a tree of drafted tokens.  The last num_nodes cached tokens of
 * each sequence are the nodes (their K and V are in the cache, in any order that
 * puts a parent before its children): node i's K and V are those of position
 * L - num_nodes + i.  Node i sees
 *     position t < L - num_nodes: the tokens before the tree, and
 *     node j where bit j % 32 of masks[s][i][j / 32] is set
 * and a node whose mask has no bit is padding: it sees nothing, its row is zeros
 * and its lse -INFINITY.  A chain (node i sees nodes 0 .. i) is pa_decode_v2_mq.
 * With a window, node i is at position p = L - num_nodes + (bits of its mask) - 1
 * (its depth in the tree) and sees of the tokens before the tree those with
 * t > p - window or t < sinks.
 *   query, out  [num_seqs, num_nodes, num_heads, head_size]   dtype
 *   lse         NULL, or DEVICE [num_seqs, num_nodes, num_heads] fp32
 *   masks       DEVICE [num_seqs, num_nodes, ceil(num_nodes / 32)] int32, as
 *               pa_tree_masks makes them (once for all layers of a step).  Any masks
 *               will do; bits past num_nodes have to be 0.
 *   window      0: no window (sinks then says nothing), or num_nodes or more
 *   seq_lens    each in [num_nodes, max_blocks_per_seq*block_size] (others:
 *               PA_ERR_DEVICE_BOUNDS; below num_nodes: zeros)
 *   num_nodes   1 .. 512
 *   block_tables  the entries of the nodes' blocks and of those that a child of the
 *               tokens before the tree sees are read, whatever the masks
 *   workspace   >= pa_decode_v2_view_workspace_bytes(num_seqs, num_nodes, ...)
 * All else is as for pa_decode_v2_window.
 */
int pa_decode_v2_tree(void* out, float* lse, const void* query, const void* key_cache,
                      const void* value_cache, const int32_t* block_tables, const int32_t* seq_lens,
                      const int32_t* masks, float scale, int window, int sinks, int num_seqs, int num_nodes,
                      int num_heads, int num_kv_heads, int head_size, int block_size, int partition_size,
                      int dtype, void* stream, int max_blocks_per_seq, int num_blocks, void* workspace,
                      size_t workspace_bytes);

/* pa_decode_v2_tree over an E4M3 cache (caches and scales of pa_decode_v2_mq_fp8). */
int pa_decode_v2_tree_fp8(void* out, float* lse, const void* query, const void* key_cache,
                          const void* value_cache, const int32_t* block_tables, const int32_t* seq_lens,
                          const int32_t* masks, float scale, float k_scale, float v_scale, int window,
                          int sinks, int num_seqs, int num_nodes, int num_heads, int num_kv_heads,
                          int head_size, int block_size, int partition_size, int dtype, void* stream,
                          int max_blocks_per_seq, int num_blocks, void* workspace, size_t workspace_bytes);

/*
 * pa_decode_v2_window (tree 0; masks are not used) and pa_decode_v2_tree (tree 1), over
 * E4M3 caches where fp8 is 1 (else k_scale and v_scale are 1), with the controls of
 * pa_decode_v2_ex, for tests and measurement: max_ctas bounds the persistent grid (0 =
 * one CTA per SM), timeout_ns every device-side wait (0 = 2^31 ns); a wait that runs out
 * is recorded as PA_ERR_TIMEOUT, and the output is then not complete.
 */
int pa_decode_v2_view_ex(void* out, float* lse, const void* query, const void* key_cache,
                         const void* value_cache, const int32_t* block_tables, const int32_t* seq_lens,
                         const int32_t* masks, float scale, float k_scale, float v_scale, int window, int sinks,
                         int num_seqs, int q_len, int num_heads, int num_kv_heads, int head_size,
                         int block_size, int partition_size, int dtype, int tree, int fp8, void* stream,
                         int max_blocks_per_seq, int num_blocks, void* workspace, size_t workspace_bytes,
                         int max_ctas, long long timeout_ns);

/*
 * Bytes of workspace for pa_decode_v2_window and pa_decode_v2_tree (q_len:
 * num_nodes; window 0: a tree without one).  0 for invalid sizes.
 */
size_t pa_decode_v2_view_workspace_bytes(int num_seqs, int q_len, int num_heads, int num_kv_heads,
                                         int head_size, int max_blocks_per_seq, int block_size,
                                         int partition_size, int window, int sinks);

/*
 * The masks of trees given by their nodes' parents:
 *   parents     [num_seqs, num_nodes] int32: the parent's number, below the node's
 *               own; -1 for a child of the tokens before the tree; below -1 for
 *               padding
 *   masks       [num_seqs, num_nodes, ceil(num_nodes / 32)] int32, written: a
 *               node's bits are its own and its ancestors'; padding has none
 *   positions   NULL, or [num_seqs, num_nodes] int32, written: seq_lens[s] -
 *               num_nodes + depth (a child of the tokens before the tree has
 *               depth 0), for rotary embeddings; -1 for padding
 *   seq_lens    [num_seqs] int32, counting the nodes
 *   num_nodes   1 .. 512
 *   workspace   >= 256 bytes, 16-byte aligned, required; holds the status, whatever
 *               it held before
 * A parent that is not below its node, a child of padding (both become padding),
 * and a length below num_nodes (positions of -1) are recorded as
 * PA_ERR_DEVICE_BOUNDS.  What is written may not overlap another array
 * (PA_ERR_INVALID_ARG).
 */
int pa_tree_masks(int32_t* masks, int32_t* positions, const int32_t* parents, const int32_t* seq_lens,
                  int num_seqs, int num_nodes, void* stream, void* workspace, size_t workspace_bytes);

/*
 * After verification: the accepted nodes' K and V move to the front of the tree's
 * part of the cache, in the caches of every layer, and lengths follow.  Sequence
 * s keeps nodes accepted[s][0 .. num_accepted[s]), ascending: node accepted[s][i]
 * goes to position L - num_nodes + i, and new_lens[s] = L - num_nodes +
 * num_accepted[s] (what pa_pages_resize takes).  Positions from there on hold
 * what they held or a moved token.
 *   key_caches, value_caches   HOST arrays of num_caches DEVICE pointers, 16-byte
 *               aligned: caches of one shape and element type (layouts of
 *               pa_decode_v2 and pa_decode_v2_fp8), each named once: none may overlap
 *               another one or any other array (PA_ERR_INVALID_ARG); the two arrays
 *               are read before the call returns
 *   accepted    [num_seqs, max_accepted] int32 (entries past num_accepted are not
 *               read); max_accepted 0 .. 512
 *   num_accepted  [num_seqs] int32, each in [0, max_accepted]
 *   new_lens    [num_seqs] int32, written; may not overlap another array
 *   num_nodes   1 .. 512
 *   cache_dtype PA_DTYPE_FP16, _BF16, _FP32 or _E4M3
 *   workspace   >= 256 bytes, 16-byte aligned, required; holds the status
 * The positions from L - num_nodes on must not be shared with another sequence (as
 * pa_pages_resize leaves them).  A length out of range, a count or path that is
 * not as above, and block ids outside the pool are recorded as
 * PA_ERR_DEVICE_BOUNDS: such a sequence keeps its cache, and new_lens[s] is L.
 * One launch (one more per further 64 caches).
 */
int pa_tree_accept(int32_t* new_lens, void* const* key_caches, void* const* value_caches, int num_caches,
                   const int32_t* block_tables, const int32_t* seq_lens, const int32_t* accepted,
                   const int32_t* num_accepted, int num_seqs, int num_nodes, int max_accepted,
                   int num_kv_heads, int head_size, int block_size, int cache_dtype, void* stream,
                   int max_blocks_per_seq, int num_blocks, void* workspace, size_t workspace_bytes);

/*
 * The rows of a step, numbered from its requests' lengths.  Sequence s has
 * num_new[s] new tokens, its last ones (seq_lens counts them already, as after
 * pa_pages_resize).  With cu[s] the sum of num_new before s, row cu[s] + i of the
 * step is sequence s at position seq_lens[s] - num_new[s] + i.
 *   cu_tokens   [num_seqs + 1] int32, written: cu (at most 2^31 - 1), as
 *               pa_kv4_append takes it
 *   slots       [num_tokens] int64, written: block * block_size + offset of each
 *               row, as pa_cache_write takes it; -1 for rows of no sequence
 *   positions, seq_ids   NULL, or [num_tokens] int32, written: -1 for rows of no
 *               sequence
 *   num_tokens  rows there is room for: more than the step has, where a captured
 *               graph keeps its size
 *   block_size  any positive number
 *   workspace   >= 256 bytes, 16-byte aligned, required; holds the status
 * A negative count (taken as 0), more rows than num_tokens (those behind are left
 * out), of a sequence with rows a length below its count or above the table's
 * capacity (slots and positions of -1), and a row's negative block id (a slot of -1)
 * are recorded as PA_ERR_DEVICE_BOUNDS.  What is written may not overlap another array
 * (PA_ERR_INVALID_ARG).
 */
int pa_pages_slots(int64_t* slots, int32_t* positions, int32_t* seq_ids, int32_t* cu_tokens,
                   const int32_t* block_tables, const int32_t* seq_lens, const int32_t* num_new,
                   int num_seqs, int num_tokens, int max_blocks_per_seq, int block_size, void* stream,
                   void* workspace, size_t workspace_bytes);

/*
 * Writes new tokens into the caches that pa_decode_v2 and pa_decode_v2_fp8 read.
 *   key, value   [num_tokens, num_kv_heads, head_size] dtype (fp16, bf16 or fp32),
 *                rows key_stride / value_stride elements apart (whole 16 bytes, at
 *                least num_kv_heads * head_size), 16-byte aligned
 *   slots        [num_tokens] int64: row r goes to offset slots[r] % block_size of
 *                block slots[r] / block_size; a negative slot skips the row.  Slots
 *                of a call differ (of two rows with one slot, either's bytes may
 *                stay).  Slots past the pool are recorded as PA_ERR_DEVICE_BOUNDS and
 *                skipped.
 *   cache_dtype  dtype: rows are copied (k_scale and v_scale are 1); or
 *                PA_DTYPE_E4M3: codes of x / k_scale and x / v_scale, computed in
 *                fp32, rounded to the nearest E4M3 (ties to even) and kept within
 *                +-448 (infinities too; NaN becomes NaN), so that a code c stands for
 *                scale * c as pa_decode_v2_fp8 reads it; scales positive and finite
 *   workspace    >= 256 bytes, 16-byte aligned, required; holds the status
 * Only the rows' slots are written.  The caches and the workspace may not overlap
 * one another nor what is read (PA_ERR_INVALID_ARG).  One launch on `stream`; it can be
 * captured into a CUDA graph.
 */
int pa_cache_write(void* key_cache, void* value_cache, const void* key, const void* value,
                   const int64_t* slots, float k_scale, float v_scale, int num_tokens, int num_kv_heads,
                   int head_size, int block_size, long long key_stride, long long value_stride, int dtype,
                   int cache_dtype, void* stream, int num_blocks, void* workspace, size_t workspace_bytes);

/*
 * Caches held in 4 bits.  The pages' launcher takes a kv_cache_dtype (page
 * "paged_attention_v2_triton.py -- Triton PagedAttention V2 for BI-V100"); the
 * format here is this library's own: a block of one kv head is one record of
 * pa_kv4_block_bytes(head_size, block_size) = block_size * (head_size + 8)
 * bytes, and the cache is
 *   kv_cache [num_blocks, num_kv_heads, block_size * (head_size + 8)] uint8
 * A record holds, with x = min(head_size, 128),
 *   key codes    [head_size/x][block_size][x/2]   two codes a byte, the even
 *                                                 dim in the low four bits
 *   value codes  [head_size/x][block_size][x/2]
 *   parameters   [block_size][4] of the dtype     key scale, key zero, value
 *                                                 scale, value zero of a token
 * and a code c stands for scale * c + zero.  The dtype (fp16 or bf16) is that
 * of the queries and of the rows that are written: a cache is used with one.
 * Returns 0 for a head or block size outside the supported ones (head_size 64,
 * 80, 96, 112, 128 or 256, block_size 8, 16, 32 or 64).
 */
size_t pa_kv4_block_bytes(int head_size, int block_size);

/*
 * Decode attention over a 4-bit cache: pa_decode_v2_lse with
 *   K_t[d] = k_scale_t * ck_t[d] + k_zero_t,  V_t[d] = v_scale_t * cv_t[d] + v_zero_t
 * of the sequence's cached tokens (nothing is rounded to the dtype before the
 * products).  lse may be NULL.  dtype PA_DTYPE_FP16 or PA_DTYPE_BF16
 * (PA_ERR_UNSUPPORTED for fp32); head sizes, block sizes, partitions, the
 * workspace (pa_decode_v2_workspace_bytes), ownership and errors are those of
 * pa_decode_v2; but the m_p left in the workspace is not the partition's
 * maximum: it lies near the log of its sum, l_p between 1 and 16.
 * Value scales may differ by any factor: a token's precision depends on what it
 * adds to a row, not on other tokens' scales.  For full precision |scale * query|
 * is expected below 2^100, the largest elements of the query rows of a kv head
 * and its neighbour within 2^16 of one another, and in bf16 caches value scales
 * of 2^-50 or more (or 0) and value zeros below 2^64.  A query row with an
 * infinity or NaN leaves the other rows' results alone.
 */
int pa_decode_v2_kv4(void* out, float* lse, const void* query, const void* kv_cache,
                     const int32_t* block_tables, const int32_t* seq_lens, float scale, int num_seqs,
                     int num_heads, int num_kv_heads, int head_size, int block_size, int partition_size,
                     int dtype, void* stream, int max_blocks_per_seq, int num_blocks, void* workspace,
                     size_t workspace_bytes);

/*
 * Multi-query decode over a 4-bit cache: the causal query rows of
 * pa_decode_v2_mq with the cache of pa_decode_v2_kv4.
 */
int pa_decode_v2_mq_kv4(void* out, float* lse, const void* query, const void* kv_cache,
                        const int32_t* block_tables, const int32_t* seq_lens, float scale, int num_seqs,
                        int q_len, int num_heads, int num_kv_heads, int head_size, int block_size,
                        int partition_size, int dtype, void* stream, int max_blocks_per_seq,
                        int num_blocks, void* workspace, size_t workspace_bytes);

/*
 * pa_decode_v2_mq_kv4 with the controls of pa_decode_v2_ex, for tests and
 * measurement: max_ctas bounds the persistent grid (0 = one CTA per SM),
 * timeout_ns every device-side wait (0 = 2^31 ns); a wait that runs out is
 * recorded as PA_ERR_TIMEOUT.  The units left over at the end are shared by as
 * many warps as the grid leaves to them, so outputs for two grids may differ by
 * the roundings of fp32 sums (for one grid they are bitwise the same).
 */
int pa_decode_v2_kv4_ex(void* out, float* lse, const void* query, const void* kv_cache,
                        const int32_t* block_tables, const int32_t* seq_lens, float scale, int num_seqs,
                        int q_len, int num_heads, int num_kv_heads, int head_size, int block_size,
                        int partition_size, int dtype, void* stream, int max_blocks_per_seq,
                        int num_blocks, void* workspace, size_t workspace_bytes, int max_ctas,
                        long long timeout_ns);

/*
 * Writes new tokens into a 4-bit cache.  Sequence s has the rows
 * cu_tokens[s] .. cu_tokens[s+1] - 1 of key and value, and they are its last
 * cached tokens: with n of them, row cu_tokens[s] + i goes to position
 * seq_lens[s] - n + i (seq_lens counts the new tokens, as for pa_decode_v2_mq).
 * Per token and kv head, for the key and the value x[0 .. head_size):
 *   zero  = min x (+0 for a zero of either sign)
 *   scale = (max x - min x) / 15, computed in fp32, rounded to the dtype
 *   code  = (x - zero) / scale in fp32, rounded to the nearest integer (ties
 *           to even), at most 15; 0 where the scale is 0
 * A vector with a NaN or an infinity, or whose spread is not finite in fp32,
 * gets NaN for scale and zero and reads back as NaN.
 *   kv_cache     as above, written: only the slots of the new tokens
 *   key, value   [num_tokens, num_kv_heads, head_size] dtype, rows
 *                key_stride / value_stride elements apart (multiples of 8, at
 *                least num_kv_heads * head_size), 16-byte aligned
 *   cu_tokens    DEVICE [num_seqs + 1] int32, ascending from 0; NULL: every
 *                sequence has num_tokens / num_seqs rows.  Rows at or behind
 *                cu_tokens[num_seqs] count for nothing.
 *   workspace    >= 256 bytes, 16-byte aligned, required; holds the status
 *                (pa_decode_v2_device_status), whatever it held before
 * The lengths have to count the new tokens already: after a pa_pages_resize that
 * was refused (PA_ERR_NO_BLOCKS) they do not, and the rows would go over cached
 * tokens.  A position of several sequences (a shared block) must not be written
 * by two of them.  A length below the sequence's row count or above the table's
 * capacity, offsets of a sequence that descend, start below 0 or pass
 * num_tokens, and block ids outside the pool are recorded as
 * PA_ERR_DEVICE_BOUNDS; all rows of such a sequence (of a bad block id: those
 * of its block) are skipped.  Where offsets descend, rows of other sequences may
 * be skipped too, and one that several claim goes to one of them.  One launch on
 * `stream`; it can be captured into a CUDA graph.
 */
int pa_kv4_append(void* kv_cache, const void* key, const void* value, const int32_t* block_tables,
                  const int32_t* seq_lens, const int32_t* cu_tokens, int num_seqs, int num_tokens,
                  int num_kv_heads, int head_size, int block_size, long long key_stride,
                  long long value_stride, int dtype, void* stream, int max_blocks_per_seq,
                  int num_blocks, void* workspace, size_t workspace_bytes);

/*
 * The reverse: the last cu_tokens[s+1] - cu_tokens[s] cached tokens of each
 * sequence as rows of the dtype, each value scale * code + zero rounded once
 * (for prefill attention over earlier context, or to leave the format).
 * Arguments as for pa_kv4_append; rows that belong to no sequence, or whose
 * length, offsets or block id are refused, keep what they held.
 */
int pa_kv4_gather(void* key_out, void* value_out, const void* kv_cache, const int32_t* block_tables,
                  const int32_t* seq_lens, const int32_t* cu_tokens, int num_seqs, int num_tokens,
                  int num_kv_heads, int head_size, int block_size, long long key_stride,
                  long long value_stride, int dtype, void* stream, int max_blocks_per_seq,
                  int num_blocks, void* workspace, size_t workspace_bytes);

/*
 * Pages of a pool.  For callers that keep block tables, lengths and the pool's
 * state on the device: sequences share, take and give back blocks without a
 * round trip to the host.  The state is
 *   refcounts [num_blocks] int32, read and written: the number of table rows
 *   that hold a block within their length; 0 (or less) is a free block
 * and the blocks of a row are its first ceil(seq_lens / block_size) entries.
 * Blocks are taken lowest free id first, in row order and within a row in table
 * order, so the result does not depend on timing.  Blocks given back by a call
 * are free for the calls after it.  After a fork or a resize a row's partly
 * filled last block is held by that row alone, so that appending to one
 * sequence never writes another's tokens.
 *
 * Arguments shared by the three calls:
 *   caches       HOST array of num_caches DEVICE pointers: every cache whose
 *                pages follow the tables (keys, values, of every layer; any
 *                layout whose first dimension is the block).  16-byte aligned.
 *   page_bytes   HOST array: bytes of one block in each cache, multiples of 16,
 *                at most 2^35
 *   block_size   tokens per block, any positive number
 *   workspace    >= pa_pages_workspace_bytes(rows, ...) bytes (rows:
 *                num_children or num_seqs, below 2^24), 16-byte aligned,
 *                required; holds the status (pa_decode_v2_device_status)
 * Calls enqueue two launches on `stream` (one more per further 128 caches),
 * never synchronise and can be captured into a CUDA graph.  The arrays caches
 * and page_bytes are read before the call returns.  No array that a call writes
 * may overlap another of its arrays (PA_ERR_INVALID_ARG; the new lengths of a
 * resize may be the lengths themselves).  Calls on one pool must be
 * ordered on one stream, also with those that read its tables and caches.
 *
 * Errors on the device: a call that needs more blocks than are free records
 * PA_ERR_NO_BLOCKS and changes nothing.  What is enqueued behind it runs all the
 * same: a pa_kv4_append finds the old lengths and writes its rows over each
 * sequence's last tokens.  So the status is to be read before it, unless the host
 * knows that enough blocks are free.  Rows with a parent, length or new
 * length out of range, or whose partly filled block has an id outside the
 * pool, are recorded as PA_ERR_DEVICE_BOUNDS and left as they were (a child
 * becomes an empty row); other ids outside the pool are recorded and counted
 * nowhere; a count that would fall below 0 is recorded and stays.
 * Returns 0 for invalid sizes.
 */
size_t pa_pages_workspace_bytes(int num_rows, int max_blocks_per_seq, int num_blocks);

/*
 * Forks: row i of the outputs becomes a copy of sequence parents[i] (parallel
 * samples, beams).  It shares the parent's full blocks (their counts go up) and
 * gets a copy of its partly filled last block in a block of its own; the
 * parents keep theirs.  Table entries past the child's blocks keep what they
 * held.
 *   block_tables_out [num_children, max_blocks_per_seq], seq_lens_out
 *                [num_children]: written
 *   block_tables [num_seqs, max_blocks_per_seq], seq_lens [num_seqs]
 *   parents      [num_children] int32 in [0, num_seqs), in any order, with
 *                repeats; -1 makes an empty row
 */
int pa_pages_fork(int32_t* block_tables_out, int32_t* seq_lens_out, const int32_t* block_tables,
                  const int32_t* seq_lens, const int32_t* parents, int32_t* refcounts,
                  void* const* caches, const size_t* page_bytes, int num_caches, int num_seqs,
                  int num_children, int max_blocks_per_seq, int block_size, int num_blocks,
                  void* stream, void* workspace, size_t workspace_bytes);

/*
 * Resizes: sequence s gets room for new_lens[s] tokens, and seq_lens[s] becomes
 * new_lens[s].  A longer sequence takes blocks, a shorter one gives back those
 * past its new end, 0 frees it.  Where the last token kept lies in a partly
 * filled block that other rows hold too (a sequence cut back into a part it
 * shares, or that ends there already, whatever its new length), the row gets a
 * copy of it.  So does every such row of a call: where they are all the holders,
 * the block that they shared becomes free, and the call has needed one block more
 * than they hold in the end.
 *   block_tables [num_seqs, max_blocks_per_seq], seq_lens [num_seqs]: updated
 *   new_lens     [num_seqs] int32 in [0, max_blocks_per_seq * block_size]
 */
int pa_pages_resize(int32_t* block_tables, int32_t* seq_lens, const int32_t* new_lens,
                    int32_t* refcounts, void* const* caches, const size_t* page_bytes, int num_caches,
                    int num_seqs, int max_blocks_per_seq, int block_size, int num_blocks, void* stream,
                    void* workspace, size_t workspace_bytes);

/*
 * Compacts: with U blocks in use, those with ids of U and up move, in ascending
 * order, into the free ids below U, ascending; pages, counts and table entries
 * follow, and the blocks U .. num_blocks - 1 are free afterwards (so the
 * caches' tails can be given up or used otherwise).  A pool without holes is
 * left as it is.
 *   block_tables [num_seqs, max_blocks_per_seq]: updated; every row that holds
 *                blocks has to be among them (or follow new_ids)
 *   new_ids      NULL, or DEVICE [num_blocks] int32, written: the block's id
 *                after the call, -1 for a block that was free
 */
int pa_pages_compact(int32_t* block_tables, const int32_t* seq_lens, int32_t* refcounts,
                     int32_t* new_ids, void* const* caches, const size_t* page_bytes, int num_caches,
                     int num_seqs, int max_blocks_per_seq, int block_size, int num_blocks, void* stream,
                     void* workspace, size_t workspace_bytes);

/*
 * Bytes of device workspace pa_decode_v2_host_io needs: the workspace of
 * pa_decode_v2 plus device staging for query, out (room for 4-byte elements,
 * whatever the dtype), block_tables and seq_lens.  Returns 0 for invalid sizes.
 */
size_t pa_decode_v2_host_io_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads,
                                            int head_size, int max_blocks_per_seq, int block_size,
                                            int partition_size);

/*
 * pa_decode_v2 for callers that hold the per-step inputs in HOST memory (a
 * serving loop): query_host, block_tables_host and seq_lens_host are copied
 * into device staging inside `workspace`, the decode runs on the device-
 * resident caches (key_cache, value_cache: DEVICE pointers), and the result is
 * copied back into out_host.  Everything is enqueued on `stream` with
 * cudaMemcpyAsync; the call returns without synchronising, so the host buffers
 * must stay alive and untouched until the stream has passed this call (use
 * page-locked host memory for the copies to be asynchronous).  `workspace`
 * (DEVICE, 16-byte aligned, >= pa_decode_v2_host_io_workspace_bytes()) is
 * required.  Sizes, layouts and status codes as for pa_decode_v2.
 */
int pa_decode_v2_host_io(void* out_host, const void* query_host, const void* key_cache,
                         const void* value_cache, const int32_t* block_tables_host,
                         const int32_t* seq_lens_host, float scale, int num_seqs, int num_heads,
                         int num_kv_heads, int head_size, int block_size, int partition_size,
                         int dtype, void* stream, int max_blocks_per_seq, int num_blocks,
                         void* workspace, size_t workspace_bytes);

/*
 * Size of the scratch array behind pa_decode_v2_static_scratch: 32 MiB of
 * device memory, reserved on every device that loads the library, for as long
 * as the process lives.
 */
#define PA_DECODE_V2_STATIC_SCRATCH_BYTES (32u * 1024u * 1024u)

/*
 * pa_decode_v2 for callers that must not allocate device memory at call time.
 * The pages have no counterpart: this is a deployment aid of this library.
 *
 * Who needs it: a process whose device memory is all reserved in advance by
 * another allocator (so a new cudaMalloc would fail), a latency-critical loop
 * that cannot risk an allocation call synchronising the device or stalling
 * other streams, or a deployment that fixes its memory footprint at start-up
 * and forbids allocation afterwards.  Such callers can use neither a
 * workspace of their own nor the library's stream-ordered allocation.
 *
 * What it does: the same computation as pa_decode_v2 (same arguments, minus
 * the workspace), with the scratch taken from a fixed array of
 * PA_DECODE_V2_STATIC_SCRATCH_BYTES inside the library's device memory.  It
 * calls no cudaMalloc, cudaFree or other allocating routine.  The caller
 * still provides all inputs and `out`.
 *   - Sizes whose workspace (pa_decode_v2_workspace_bytes) exceeds the array
 *     are rejected with PA_ERR_WORKSPACE before anything is enqueued.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current) and caches it with the
 *     id of the device's context; make that first call before any stream
 *     capture.  If the context is destroyed and recreated (cudaDeviceReset),
 *     the array is a new one: the next call sees the new context id and looks
 *     the address up again, so make that call before any capture too.  (The
 *     array's contents do not survive the reset; nothing relies on them.)
 *   - All calls on a device share the one array, which keeps the last call's
 *     contents; the counters that must start at zero are cleared by each call
 *     on its stream.  Calls whose execution overlaps on the GPU (different
 *     streams, or threads without ordering between them) race on the array
 *     and give undefined results: order them on one stream.
 * Status codes as for pa_decode_v2.
 */
int pa_decode_v2_static_scratch(void* out, const void* query, const void* key_cache,
                                const void* value_cache, const int32_t* block_tables,
                                const int32_t* seq_lens, float scale, int num_seqs, int num_heads,
                                int num_kv_heads, int head_size, int block_size, int partition_size,
                                int dtype, void* stream, int max_blocks_per_seq, int num_blocks);

/*
 * Device-side status of the last call that used `workspace`: synchronises
 * `stream`, copies the error word and stores it in *status (PA_OK if none).
 * (A decode call or pa_tree_accept with num_seqs 0 enqueues nothing and does not use
 * its workspace.)
 * Returns PA_OK, or PA_ERR_CUDA if the copy or the synchronisation failed.
 */
int pa_decode_v2_device_status(const void* workspace, void* stream, int* status);

/* Static description of a status code. */
const char* pa_decode_v2_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* PA_DECODE_H */
