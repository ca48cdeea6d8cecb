// Arguments and launchers of the serving-step kernels (prefix_attention.cu,
// norm_rope_append.cu, step_tables.cu), between them and the entry points.
#pragma once

#include "pkv_internal.h"

namespace pkv {

// Launch `kernel` to start as the kernel before it on the stream drains; the
// kernel waits for that one's results itself (griddepcontrol.wait).
template <typename... Params, typename... Args>
inline cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                                    Args... args) {
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ------------------------------------------------- decode over shared prefixes
constexpr int kPrefixMaxSeqs = 4096;   // sequences and groups that a CTA plans in its shared memory
constexpr int kPrefixMaxGroups = 512;
constexpr int kPrefixRows = 128;      // query rows of one tile

struct PrefixArgs {
    const void* q;
    void* out;
    const int32_t* tables;
    const int32_t* lens;
    const int32_t* group_offsets;  // [num_groups + 1]
    const int32_t* prefix_lens;    // [num_groups]
    int32_t* err;
    int layer, max_blocks, max_len, num_seqs, num_groups, num_q_heads, num_kv_heads, block_size, num_blocks;
    int gh;                        // query heads per KV head
    int seqs_per_tile;             // sequences whose rows fill a 128-row tile
    int ctas;                      // CTAs of the attention kernel
    int unit_cost;                 // cost of a unit beside its tiles, in tiles (set by the launch)
    float qk_scale_log2, v_scale;
    int test_polls, test_cta;      // test hook: polls of that CTA's (< 0: every CTA's) first wait for a tile; < 0: none
    // workspace: the plan ...
    int32_t* totals;               // cost of the whole list
    int2* seqs;                    // [B] {clamped length, tiles read with the group}
    int4* groups;                  // [G] {first sequence, sequences, shared tiles, table row}
    int4* pieces;                  // [B][2] {start of head 0's unit, shared tiles, rows before / gh, row / gh},
                                   //        {rows from head to head, start of head 0's own unit, own tiles, -}
    // ... and the pieces: fp32 rows of O / l and log2-sum-exp
    float *pre_o, *pre_lse;        // [B * Hq + ctas * 128]
    float *own_o, *own_lse;        // [B * Hq + ctas * gh]
};
cudaError_t launch_prefix_attention(pkv_dtype kv, const PrefixArgs& a, const void* tmap_k, const void* tmap_v,
                                    const void* tmap_q_group, const void* tmap_q_own, cudaStream_t stream);

// -------------------------------------------------- norm, rotation and append
struct NormRopeArgs {
    const void *q, *k, *v;                      // rows of one token at t * stride elements
    int64_t q_stride, k_stride, v_stride;
    void* q_out;                                // [T][Hq][D]
    uint8_t *k_layer, *v_layer;
    const int32_t* positions;                   // [num_axes][T]
    const int64_t* slots;                       // [T]
    const float* cos_sin;                       // [max_pos][rotary_dim]
    const void *q_weight, *k_weight;            // [D], both or neither
    int weight_dtype;
    float eps;
    int num_tokens, num_q_heads, num_kv_heads;
    int64_t num_slots;
    int block_shift;                            // log2(block_size)
    int max_pos, rotary_dim, interleaved, num_axes;
    int axis_end[2];                            // pairs of the first, and of the first two axes
    float k_inv_scale, v_inv_scale;
    int32_t* err;
};
cudaError_t launch_norm_rope_append(pkv_dtype pool, pkv_dtype in, int head_dim, const NormRopeArgs& a,
                                    cudaStream_t stream);

// ----------------------------------------------------- tables and slots of a step
struct GrowArgs {
    const int32_t* lens;
    const int32_t* new_tokens;
    int32_t* tables;                            // [B][max_blocks]
    const int32_t* ring;                        // free blocks: entries head .. head + count - 1, wrapping
    const int32_t* free_state;                  // {head, count}
    int ring_size, num_seqs, max_blocks, block_shift, num_blocks, max_tokens;  // block_shift: log2(block_size)
    int64_t* slots;                             // [max_tokens]
    int32_t *positions, *token_seqs;            // [max_tokens]
    int32_t* token_offsets;                     // [B + 1]
    int32_t *granted, *lens_out;                // [B]
    int32_t* free_out;
    int32_t* err;
};
cudaError_t launch_tables_grow(const GrowArgs& a, cudaStream_t stream);

struct ReleaseArgs {
    const int32_t* lens;
    const int32_t* finished;
    const int32_t* keep_blocks;                 // optional
    const int32_t* tables;
    int32_t* ring;
    const int32_t* free_state;
    int ring_size, num_seqs, max_blocks, block_shift, num_blocks;
    int32_t* lens_out;
    int32_t* free_out;
    int32_t* err;
};
cudaError_t launch_tables_release(const ReleaseArgs& a, cudaStream_t stream);

}  // namespace pkv
