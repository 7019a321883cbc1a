// pa_internal.h — host-side interface between the C ABI (pa_api.cpp) and the
// kernel translation units. Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace pa {

// Bit of the per-translation-unit status word a kernel sets when it meets an
// out-of-range block id, slot or context length (and skips the access).
constexpr unsigned kStatusBadIndex = 1u;
// Bit set when a bounded wait on a shared-memory pipeline barrier gave up.
constexpr unsigned kStatusTimeout = 2u;
// Bit set when a kernel found its dynamic shared memory not 1024-byte aligned
// (it then returns without running; the outputs are not written).
constexpr unsigned kStatusSmemAlign = 4u;

// Everything one decode launch needs. Offsets are in elements unless noted.
struct DecodeParams {
    void* out;                  // [S][H][D], cache dtype
    const void* q;              // [S][H][D]
    const void* k_cache;        // [NB][Hkv][BS][D]
    const void* v_cache;
    const int32_t* block_tables;
    const int32_t* context_lens;
    float* ws_o;                // [S][H][P][D] normalised partial outputs (P > 1)
    float* ws_ml;               // [S][H][P][2]  (running max in log2 units, running sum)
    int64_t table_stride;
    int32_t max_context_len;
    int32_t num_seqs;
    int32_t num_heads;
    int32_t num_kv_heads;
    int32_t num_blocks;
    int32_t block_size;
    int32_t log2_block_size;
    int32_t partition_size;     // tokens per partition (whole context when P == 1)
    int32_t num_partitions;     // P
    float scale_log2;           // softmax scale * log2(e)
    int32_t test_skip_position; // -1; >= 0 only under pa_test_skip_load (timeout test)
    // Multi-token queries (pa_decode_multi), else query_start == nullptr: q / out
    // rows of sequence s are query_start[s] .. query_start[s+1]-1 of num_rows;
    // grouped items take q_chunks chunks of <= gs query tokens per sequence.
    const int32_t* query_start;
    int32_t q_chunks;
    int32_t num_rows;           // rows of q / out: num_seqs, or the query tokens
    // Quantised caches (codes): per-kv-head scales, K_t = value(code) * k_scale[kh];
    // nullptr for bf16 / f32 caches.
    const float* k_scale;
    const float* v_scale;
    // head_dim of q / out / the workspace rows. The consumers over codes are
    // built for 128-code rows and take head_dim 64 pools as rows whose upper
    // half the TMA fills with zero codes (q zero there too, outputs not stored).
    int32_t head_dim;
    // Dynamic item schedule of the persistent kernels: a counter zeroed before
    // the launch, from which CTAs claim work items in order (nullptr: static
    // schedule, item u to CTA u mod grid).
    unsigned int* sched;
    // pa_decode_weights, else nullptr: scores [row of out][score_stride] (log2 units;
    // a token's at its position) and per (row, partition) the pair (running max,
    // sum of the unrounded weights).
    float* scores;
    int64_t score_stride;
    float* score_ml;
};

// One launch of the rotary append (pa_rope.cu). Strides are in elements.
struct RopeParams {
    const void* q;              // [T] rows of num_heads x head_dim, q_stride apart
    const void* k;
    const void* v;
    void* q_out;                // [T][num_heads][head_dim]
    void* k_cache;
    void* v_cache;
    const int32_t* positions;   // [axes][T]
    const int64_t* slot_mapping;
    const float* k_scale;       // codes: [num_kv_heads]
    const float* v_scale;
    int64_t q_stride, k_stride, v_stride;
    int64_t num_slots;
    int32_t num_tokens, num_heads, num_kv_heads, head_dim;
    int32_t block_size, log2_block_size;
    int32_t half;               // rotary_dim / 2: frequencies
    int32_t adjacent;           // pairs (2i, 2i + 1) instead of (i, i + half)
    int32_t tokens_per_cta;
    float mscale;
    uint8_t axis[64];
    uint64_t turns[64];         // inv_freq / (2 pi) mod 1, in units of 2^-64
};

// Eviction (pa_evict.cu).
struct EvictParams {
    uint4* k_cache;
    uint4* v_cache;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const float* weights;       // [S][Hkv][weights_stride]
    float* weights_out;
    int32_t* new_context_lens;
    int32_t* kept;              // [S][Hkv][budget]
    int64_t table_stride;
    int64_t weights_stride;
    int32_t max_context_len, num_seqs, num_kv_heads, num_blocks;
    int32_t block_size, log2_block_size, row_vecs;
    int32_t budget, recent;
};

// weights += the softmax weights of a decode step (pa_evict.cu).
struct AddWeightsParams {
    const float* scores;        // [S][H][score_stride], log2 units
    const float* ml;            // [S][H][P][2]
    const int32_t* context_lens;
    float* weights;             // [S][Hkv][weights_stride]
    int64_t score_stride, weights_stride;
    int32_t max_context_len, num_seqs, num_heads, num_kv_heads;
    int32_t partition_size, num_partitions;
};

// Attention over whole packed prompts and the weights their tokens received
// (pa_prefill.cu, pa_prefill_simt.cu). Strides in elements, between tokens.
struct PrefillParams {
    void* out;                  // [T][H][D]
    const void* q;
    const void* k;
    const void* v;
    const int32_t* cu_seqlens;  // [S + 1]
    float* lse;                 // [H][T], natural log (pa_prefill_weights: read)
    float* weights;             // [S][Hkv][weights_stride]
    int64_t q_stride, k_stride, v_stride;
    int64_t weights_stride;
    int32_t num_seqs, total_tokens, max_seq_len, num_heads, num_kv_heads, head_dim;
    int32_t last_queries;       // pa_prefill_weights: 0 = every query
    int32_t split_heads;        // pa_prefill_weights, set by its launcher
    int32_t test_skip_position; // -1; >= 0 only under pa_test_skip_load (timeout test)
    float scale_log2;           // softmax scale * log2(e)
};

struct CopyParams {
    int32_t num_blocks;
    int32_t num_kv_heads;
    int32_t block_size;
    int32_t log2_block_size;
    int32_t row_vecs;           // 16-byte chunks per K/V vector = head_dim * elem / 16
};

// Launchers: return cudaSuccess or the launch error. dtype: 0 = f32, 1 = bf16.
cudaError_t launch_kv_append(const void* k, const void* v, const int64_t* slot_mapping,
                             int32_t num_tokens, void* k_cache, void* v_cache,
                             const CopyParams& cp, cudaStream_t stream);
// Quantising append: bf16 k, v [T][Hkv][D] -> codes (fmt 2 = FP8 E4M3, 3 = int8)
// of x / scale[kv head].
cudaError_t launch_kv_append_quant(const void* k, const void* v, const int64_t* slot_mapping,
                                   int32_t num_tokens, void* k_cache, void* v_cache,
                                   const float* k_scale, const float* v_scale, int fmt,
                                   const CopyParams& cp, cudaStream_t stream);
cudaError_t launch_block_copy(const int64_t* pairs, int32_t num_pairs, void* k_cache,
                              void* v_cache, const CopyParams& cp, cudaStream_t stream);
// Blocks of one pool into another of the same block shape (either may be
// mapped pinned host memory); block ids checked against each pool's size.
cudaError_t launch_block_swap(const int64_t* pairs, int32_t num_pairs, const void* src_k,
                              const void* src_v, int32_t src_blocks, void* dst_k, void* dst_v,
                              int32_t dst_blocks, const CopyParams& cp, cudaStream_t stream);

// Which decode kernel a call uses: the tensor-core GQA consumer for bf16 with
// a query group of 2..8, the CUDA-core consumer otherwise.
bool mma_supported(int dtype, int head_dim, int group);
// CTA slots per SM the persistent tensor-core kernel is built for (its grid is
// at most this many CTAs per SM; the partition policy sizes items for it).
int mma_ctas_per_sm();

// Decode with K/V staged through shared memory by TMA (producer warp +
// consumer warps); `mma` selects the tensor-core GQA consumer. The tensor maps
// describe k_cache / v_cache as [num_blocks * num_kv_heads * block_size rows]
// x [head_dim], boxes of 16 rows x 128 bytes, 128-byte swizzle.
cudaError_t launch_decode_tma(const DecodeParams& p, int dtype, int head_dim, bool mma,
                              const CUtensorMap& kmap, const CUtensorMap& vmap,
                              cudaStream_t stream);
// Grouped decode: sequences [k gs, (k + 1) gs) form group k and run in one CTA,
// so blocks they share are read once; with p.query_start set, the members of an
// item are up to gs query tokens of one sequence instead. bf16, head_dim
// 64 / 128, 1 <= gs <= 8, gs * (H / Hkv) <= 64 query columns.
bool grouped_supported(int dtype, int head_dim, int group, int gs);
// Select the grouped consumer (PA_GROUPED_MMA_SYNC / PA_GROUPED_TCGEN05);
// returns the previous one.
int set_grouped_consumer(int consumer);
// Most query columns (tokens x heads per kv head) one multi-token item may hold.
int grouped_max_cols(int dtype, int head_dim, int group);
// Whether the grouped kernel for (dtype, head_dim, gs, H / Hkv) is the tcgen05 consumer.
bool grouped_is_tcgen05(int dtype, int head_dim, int gs, int group);
// CTA slots per SM of the grouped kernel chosen for (dtype, head_dim, gs, H / Hkv).
int grouped_ctas_per_sm(int dtype, int head_dim, int gs, int group);
cudaError_t launch_decode_grouped(const DecodeParams& p, int dtype, int head_dim, int gs,
                                  const CUtensorMap& kmap, const CUtensorMap& vmap,
                                  cudaStream_t stream);
// Log-sum-exp merge of the P partial results into out.
cudaError_t launch_partition_reduce(const DecodeParams& p, int dtype, int head_dim,
                                    cudaStream_t stream);

cudaError_t launch_rope_append(RopeParams p, int dtype, cudaStream_t stream);

// Longest context pa_evict takes (its selection keeps two words per 32 tokens in
// shared memory).
int evict_max_context();
cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream);
cudaError_t launch_add_weights(const AddWeightsParams& p, cudaStream_t stream);

// bf16, on the tensor cores. The maps describe q, k and v as [tokens][heads][head_dim],
// boxes of 128 tokens x 1 head x 128 bytes, 128-byte swizzle.
cudaError_t launch_prefill(const PrefillParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap,
                           const CUtensorMap& vmap, cudaStream_t stream);
cudaError_t launch_prefill_weights(const PrefillParams& p, const CUtensorMap& qmap,
                                   const CUtensorMap& kmap, cudaStream_t stream);
// fp32, on the CUDA cores.
cudaError_t launch_prefill_simt(const PrefillParams& p, cudaStream_t stream);
cudaError_t launch_prefill_weights_simt(const PrefillParams& p, cudaStream_t stream);

// Record `fmt` as this host thread's last error (read by pa_get_last_error)
// and return `code`.
int report_error(int code, const char* fmt, ...);

// Status words of the kernel translation units: OR of kStatus* bits since the
// last clear. Return cudaSuccess or the copy error.
cudaError_t read_status_copy(unsigned* bits, bool clear);
cudaError_t read_status_tma(unsigned* bits, bool clear);
cudaError_t read_status_rope(unsigned* bits, bool clear);
cudaError_t read_status_evict(unsigned* bits, bool clear);
cudaError_t read_status_prefill(unsigned* bits, bool clear);
cudaError_t read_status_prefill_simt(unsigned* bits, bool clear);

}  // namespace pa
