// Arguments and launchers of the quantised cache's kernels (quant_cache.cu,
// quant_decode.cu) and of prompt attention (prompt_attention.cu), between them
// and the entry points (quant_api.cu).
#pragma once

#include <cuda_bf16.h>

#include "step_internal.h"

// The validated handle behind kv_quant_pool.
struct kv_quant_pool {
    kv_quant_pool_desc d;
    int row_bytes;        // codes of one row: head_dim * bits / 8
    size_t layer_rows;    // rows of one layer of one tensor
};

namespace pkv {

// What the operators here leave zero for the next call on a workspace lies in its first bytes, and nothing else does, so
// that calls of all of them may share one.
constexpr size_t kWorkspaceZeros = 65536;

// A TMA descriptor (128-byte swizzle, no fill) of a tensor of `bytes`-byte
// elements; false where the driver has none.  strides: of dimensions 1 .. rank - 1.
bool encode_map(CUtensorMap* map, int elem_bytes, int rank, const void* base, const uint64_t* dims,
                const uint64_t* strides, const uint32_t* box);

// ------------------------------------------------------- append and read-back
struct QuantAppendArgs {
    const void *k, *v;                // rows of one token at t * stride elements
    int64_t k_stride, v_stride;
    const int64_t* slots;
    uint8_t *k_codes, *v_codes;       // of the layer
    uint32_t *k_params, *v_params;    // bfloat16 pairs (scale low, offset high)
    int num_tokens, num_kv_heads, block_shift;
    int64_t num_slots;
    int32_t* err;
};
cudaError_t launch_quant_append(int bits, pkv_dtype in, int head_dim, const QuantAppendArgs& a, cudaStream_t stream);

struct ReadArgs {
    const uint8_t *k, *v;                      // codes or elements of the layer
    const uint32_t *k_params, *v_params;       // quantised pools
    float k_scale, v_scale;                    // E4M3 pools
    const int32_t *tables, *offsets;
    void *k_out, *v_out;
    int num_seqs, num_rows, max_blocks, num_kv_heads, block_shift, num_blocks;
    int32_t* err;
};
// What a pool's rows hold.
enum ReadKind { kReadF32, kReadBf16, kReadE4m3, kReadQ8, kReadQ4 };
cudaError_t launch_read(ReadKind kind, int head_dim, const ReadArgs& a, cudaStream_t stream);

// ---------------------------------------------------------- decode attention
struct QuantDecodeArgs {
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    const uint8_t *k_codes, *v_codes;          // of the layer
    const uint32_t *k_params, *v_params;
    const int32_t *tables, *lens;
    int32_t* err;
    int num_seqs, num_q_heads, num_kv_heads, max_blocks, max_len, block_shift, num_blocks;
    float scale_log2;                          // scale * log2(e)
    // workspace
    int32_t* counters;
    float *part_o, *part_ml;
};
size_t quant_decode_workspace(int num_q_heads, int num_kv_heads, int head_dim, uint8_t* base, QuantDecodeArgs* a);
cudaError_t launch_quant_decode(int bits, int head_dim, const QuantDecodeArgs& a, cudaStream_t stream);

// ---------------------------------------------------------- prompt attention
struct PromptArgs {
    const void *q, *k, *v;
    void* out;
    int64_t q_stride, k_stride, v_stride;      // elements
    const int32_t *q_offsets, *k_offsets;
    int32_t* err;
    int num_seqs, q_rows, k_rows, num_q_heads, num_kv_heads;
    float scale_log2;
    int32_t test_wait_polls, test_wait_cta;    // as first_wait_limit gives them
    // tensor-core design: {units, CTAs} and row tiles that are cut, zero between calls, and the pieces' sums
    int32_t* counters;
    int4* tiles;
    float2* part_ml;
    float4* part_o;
};
size_t prompt_tc_workspace(int head_dim, uint8_t* base, PromptArgs* a);
constexpr int kPromptMaxSeqs = 2048;           // sequences that the tensor-core design plans in shared memory
bool prompt_tc_fits(pkv_dtype t, int num_seqs, int q_rows, int num_q_heads, int num_kv_heads);
cudaError_t launch_prompt_tc(int head_dim, const PromptArgs& a, cudaStream_t stream);
cudaError_t launch_prompt_simt(pkv_dtype t, int head_dim, const PromptArgs& a, cudaStream_t stream);

}  // namespace pkv
