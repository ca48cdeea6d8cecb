// C ABI of the quantised cache and of prompt attention: argument checks and
// launches, as in api.cu.
#include <cmath>
#include <new>

#include "quant_internal.h"

namespace pkv {
namespace {

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

pkv_status status_of(cudaError_t e) {
    if (e == cudaSuccess) return PKV_OK;
    if (e == cudaErrorNotSupported) return PKV_ERR_UNSUPPORTED;
    set_last_error(e);
    return PKV_ERR_CUDA;
}

int shift_of(int block_size) { return block_size == 16 ? 4 : (block_size == 32 ? 5 : 6); }

// A token stride in elements: whole 16-byte chunks, and no offset past 64 bits.
bool stride_ok(int64_t s, int64_t rows) { return s >= 0 && s % 8 == 0 && s <= INT64_MAX / 8 / (rows > 0 ? rows : 1); }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

pkv_status desc_ok(const kv_quant_pool_desc* d) {
    if (!d || d->num_layers < 1 || d->num_blocks < 1 || d->num_kv_heads < 1) return PKV_ERR_INVALID_ARG;
    if (d->block_size != 16 && d->block_size != 32 && d->block_size != 64) return PKV_ERR_UNSUPPORTED;
    if (d->head_dim != 64 && d->head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (d->bits != 4 && d->bits != 8) return PKV_ERR_UNSUPPORTED;
    // slots and element offsets are int64; keep one layer's slot count in int32
    if (static_cast<int64_t>(d->num_blocks) * d->block_size > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    if (d->num_kv_heads > (1 << 20)) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

size_t rows_of_layer(const kv_quant_pool_desc* d) {
    return static_cast<size_t>(d->num_blocks) * d->num_kv_heads * d->block_size;
}

// The checks and arguments that reading back any pool shares (row: bytes of a packed row).
pkv_status read_call(const int32_t* tables, int32_t max_blocks, const int32_t* offsets, int32_t num_seqs,
                     int32_t num_rows, size_t row, void* k_out, void* v_out, ReadArgs* a) {
    if (max_blocks < 1 || num_seqs < 0 || num_rows < 0) return PKV_ERR_INVALID_ARG;
    if (num_seqs == 0 || num_rows == 0) return PKV_OK;
    if (!tables || !offsets || !k_out || !v_out) return PKV_ERR_INVALID_ARG;
    if (!aligned(tables, 4) || !aligned(offsets, 4) || !aligned(k_out, 16) || !aligned(v_out, 16))
        return PKV_ERR_INVALID_ARG;
    if (overlap(k_out, num_rows * row, v_out, num_rows * row)) return PKV_ERR_INVALID_ARG;
    a->tables = tables;
    a->offsets = offsets;
    a->k_out = k_out;
    a->v_out = v_out;
    a->num_seqs = num_seqs;
    a->num_rows = num_rows;
    a->max_blocks = max_blocks;
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status kv_quant_pool_bytes(const kv_quant_pool_desc* d, size_t* codes, size_t* params) {
    const pkv_status st = desc_ok(d);
    if (st != PKV_OK) return st;
    const size_t rows = rows_of_layer(d) * d->num_layers;
    if (codes) *codes = rows * (d->head_dim * d->bits / 8);
    if (params) *params = rows * 4;
    return PKV_OK;
}

pkv_status kv_quant_pool_create(const kv_quant_pool_desc* d, kv_quant_pool** out) {
    if (!d || !out) return PKV_ERR_INVALID_ARG;
    *out = nullptr;
    const pkv_status st = desc_ok(d);
    if (st != PKV_OK) return st;
    for (const void* p : {d->k_codes, d->v_codes, d->k_params, d->v_params})
        if (!p || !aligned(p, 16)) return PKV_ERR_INVALID_ARG;
    if (d->error_word && !aligned(d->error_word, 4)) return PKV_ERR_INVALID_ARG;
    kv_quant_pool* p = new (std::nothrow) kv_quant_pool;
    if (!p) return PKV_ERR_INVALID_ARG;
    p->d = *d;
    p->row_bytes = d->head_dim * d->bits / 8;
    p->layer_rows = rows_of_layer(d);
    *out = p;
    return PKV_OK;
}

void kv_quant_pool_destroy(kv_quant_pool* p) { delete p; }

pkv_status kv_quant_append(const kv_quant_pool* p, int32_t layer, const void* k, const void* v, pkv_dtype in_dtype,
                           int64_t k_stride, int64_t v_stride, const int64_t* slot_mapping, int32_t num_tokens,
                           void* stream) {
    if (!p || layer < 0 || layer >= p->d.num_layers || num_tokens < 0) return PKV_ERR_INVALID_ARG;
    if (in_dtype != PKV_F32 && in_dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
    if (!stride_ok(k_stride, num_tokens) || !stride_ok(v_stride, num_tokens)) return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    if (!k || !v || !slot_mapping || !aligned(k, 16) || !aligned(v, 16) || !aligned(slot_mapping, 8))
        return PKV_ERR_INVALID_ARG;
    const size_t first = p->layer_rows * layer;
    QuantAppendArgs a{};
    a.k = k;
    a.v = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.slots = slot_mapping;
    a.k_codes = static_cast<uint8_t*>(p->d.k_codes) + first * p->row_bytes;
    a.v_codes = static_cast<uint8_t*>(p->d.v_codes) + first * p->row_bytes;
    a.k_params = static_cast<uint32_t*>(p->d.k_params) + first;
    a.v_params = static_cast<uint32_t*>(p->d.v_params) + first;
    a.num_tokens = num_tokens;
    a.num_kv_heads = p->d.num_kv_heads;
    a.block_shift = shift_of(p->d.block_size);
    a.num_slots = static_cast<int64_t>(p->d.num_blocks) * p->d.block_size;
    a.err = p->d.error_word;
    return status_of(launch_quant_append(p->d.bits, in_dtype, p->d.head_dim, a, static_cast<cudaStream_t>(stream)));
}

pkv_status kv_read(const pkv_pool* p, int32_t layer, const int32_t* tables, int32_t max_blocks, const int32_t* offsets,
                   int32_t num_seqs, int32_t num_rows, void* k_out, void* v_out, void* stream) {
    if (!p || layer < 0 || layer >= p->d.num_layers) return PKV_ERR_INVALID_ARG;
    ReadArgs a{};
    const size_t row = static_cast<size_t>(p->d.num_kv_heads) * p->d.head_dim * (p->d.kv_dtype == PKV_F32 ? 4 : 2);
    const pkv_status st = read_call(tables, max_blocks, offsets, num_seqs, num_rows, row, k_out, v_out, &a);
    if (st != PKV_OK || !a.tables) return st;
    a.k = static_cast<const uint8_t*>(p->d.k_base) + static_cast<size_t>(layer) * p->layer_bytes;
    a.v = static_cast<const uint8_t*>(p->d.v_base) + static_cast<size_t>(layer) * p->layer_bytes;
    a.k_scale = p->d.k_scale;
    a.v_scale = p->d.v_scale;
    a.num_kv_heads = p->d.num_kv_heads;
    a.block_shift = shift_of(p->d.block_size);
    a.num_blocks = p->d.num_blocks;
    a.err = p->d.error_word;
    const ReadKind kind = p->d.kv_dtype == PKV_F32 ? kReadF32 : (p->d.kv_dtype == PKV_BF16 ? kReadBf16 : kReadE4m3);
    return status_of(launch_read(kind, p->d.head_dim, a, static_cast<cudaStream_t>(stream)));
}

pkv_status kv_quant_read(const kv_quant_pool* p, int32_t layer, const int32_t* tables, int32_t max_blocks,
                         const int32_t* offsets, int32_t num_seqs, int32_t num_rows, void* k_out, void* v_out,
                         void* stream) {
    if (!p || layer < 0 || layer >= p->d.num_layers) return PKV_ERR_INVALID_ARG;
    ReadArgs a{};
    const size_t row = static_cast<size_t>(p->d.num_kv_heads) * p->d.head_dim * 2;
    const pkv_status st = read_call(tables, max_blocks, offsets, num_seqs, num_rows, row, k_out, v_out, &a);
    if (st != PKV_OK || !a.tables) return st;
    const size_t first = p->layer_rows * layer;
    a.k = static_cast<const uint8_t*>(p->d.k_codes) + first * p->row_bytes;
    a.v = static_cast<const uint8_t*>(p->d.v_codes) + first * p->row_bytes;
    a.k_params = static_cast<const uint32_t*>(p->d.k_params) + first;
    a.v_params = static_cast<const uint32_t*>(p->d.v_params) + first;
    a.num_kv_heads = p->d.num_kv_heads;
    a.block_shift = shift_of(p->d.block_size);
    a.num_blocks = p->d.num_blocks;
    a.err = p->d.error_word;
    return status_of(launch_read(p->d.bits == 8 ? kReadQ8 : kReadQ4, p->d.head_dim, a, static_cast<cudaStream_t>(stream)));
}

pkv_status paged_quant_decode_plan(const kv_quant_pool* p, int32_t num_seqs, int32_t num_q_heads, int32_t max_seq_len,
                                   size_t* ws_out) {
    if (!p || num_seqs < 0 || num_q_heads < 1 || max_seq_len < 0) return PKV_ERR_INVALID_ARG;
    if (num_q_heads % p->d.num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
    if (num_seqs > 65535 || num_q_heads > 65535 || max_seq_len > INT32_MAX - 63) return PKV_ERR_UNSUPPORTED;  // (tiles of 64)
    if (ws_out) *ws_out = quant_decode_workspace(num_q_heads, p->d.num_kv_heads, p->d.head_dim, nullptr, nullptr);
    return PKV_OK;
}

pkv_status paged_quant_decode_attention(const void* q, pkv_dtype q_dtype, const kv_quant_pool* p, int32_t layer,
                                        const int32_t* tables, int32_t max_blocks, const int32_t* seq_lens,
                                        int32_t num_seqs, int32_t num_q_heads, int32_t max_seq_len, float scale,
                                        void* workspace, size_t workspace_bytes, void* out, void* stream) {
    if (!p || layer < 0 || layer >= p->d.num_layers || max_blocks < 1) return PKV_ERR_INVALID_ARG;
    size_t need = 0;
    const pkv_status st = paged_quant_decode_plan(p, num_seqs, num_q_heads, max_seq_len, &need);
    if (st != PKV_OK) return st;
    if (static_cast<int64_t>(max_seq_len) > static_cast<int64_t>(max_blocks) * p->d.block_size) return PKV_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return PKV_ERR_INVALID_ARG;
    if (q_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!q || !out || !tables || !seq_lens) return PKV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(tables, 4) || !aligned(seq_lens, 4)) return PKV_ERR_INVALID_ARG;
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return PKV_ERR_WORKSPACE;
    const size_t first = p->layer_rows * layer;
    QuantDecodeArgs a{};
    quant_decode_workspace(num_q_heads, p->d.num_kv_heads, p->d.head_dim, static_cast<uint8_t*>(workspace), &a);
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.k_codes = static_cast<const uint8_t*>(p->d.k_codes) + first * p->row_bytes;
    a.v_codes = static_cast<const uint8_t*>(p->d.v_codes) + first * p->row_bytes;
    a.k_params = static_cast<const uint32_t*>(p->d.k_params) + first;
    a.v_params = static_cast<const uint32_t*>(p->d.v_params) + first;
    a.tables = tables;
    a.lens = seq_lens;
    a.err = p->d.error_word;
    a.num_seqs = num_seqs;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = p->d.num_kv_heads;
    a.max_blocks = max_blocks;
    a.max_len = max_seq_len;
    a.block_shift = shift_of(p->d.block_size);
    a.num_blocks = p->d.num_blocks;
    a.scale_log2 = scale * 1.4426950408889634f;
    return status_of(launch_quant_decode(p->d.bits, p->d.head_dim, a, static_cast<cudaStream_t>(stream)));
}

pkv_status prompt_attention_plan(int32_t num_seqs, int32_t q_rows, int32_t num_q_heads, int32_t num_kv_heads,
                                 int32_t head_dim, pkv_dtype dtype, size_t* ws_out) {
    if (num_seqs < 0 || q_rows < 0 || num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0)
        return PKV_ERR_INVALID_ARG;
    if (dtype != PKV_F32 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (num_q_heads > 65535) return PKV_ERR_UNSUPPORTED;
    if (ws_out)
        *ws_out = prompt_tc_fits(dtype, num_seqs, q_rows, num_q_heads, num_kv_heads) ? prompt_tc_workspace(head_dim, nullptr, nullptr) : 0;
    return PKV_OK;
}

pkv_status prompt_attention(const void* q, const void* k, const void* v, pkv_dtype dtype, int64_t q_stride,
                            int64_t k_stride, int64_t v_stride, const int32_t* q_offsets, const int32_t* k_offsets,
                            int32_t num_seqs, int32_t q_rows, int32_t k_rows, int32_t num_q_heads, int32_t num_kv_heads,
                            int32_t head_dim, float scale, void* workspace, size_t workspace_bytes, void* out,
                            int32_t* error_word, void* stream) {
    size_t need = 0;
    const pkv_status st = prompt_attention_plan(num_seqs, q_rows, num_q_heads, num_kv_heads, head_dim, dtype, &need);
    if (st != PKV_OK) return st;
    if (k_rows < 0 || !std::isfinite(scale)) return PKV_ERR_INVALID_ARG;
    const int64_t q_row = static_cast<int64_t>(num_q_heads) * head_dim, kv_row = static_cast<int64_t>(num_kv_heads) * head_dim;
    if (!stride_ok(q_stride, q_rows) || !stride_ok(k_stride, k_rows) || !stride_ok(v_stride, k_rows))
        return PKV_ERR_INVALID_ARG;
    if ((q_rows > 1 && q_stride < q_row) || (k_rows > 1 && (k_stride < kv_row || v_stride < kv_row))) return PKV_ERR_INVALID_ARG;
    if (error_word && !aligned(error_word, 4)) return PKV_ERR_INVALID_ARG;
    if (num_seqs == 0 || q_rows == 0) return PKV_OK;
    if (!q || !out || !q_offsets || !k_offsets || (k_rows > 0 && (!k || !v))) return PKV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(q_offsets, 4) ||
        !aligned(k_offsets, 4))
        return PKV_ERR_INVALID_ARG;
    const size_t e = dtype_bytes(dtype), out_bytes = static_cast<size_t>(q_rows) * q_row * e;
    if (overlap(out, out_bytes, q, (static_cast<size_t>(q_rows - 1) * q_stride + q_row) * e)) return PKV_ERR_INVALID_ARG;
    if (k_rows > 0 && (overlap(out, out_bytes, k, (static_cast<size_t>(k_rows - 1) * k_stride + kv_row) * e) ||
                       overlap(out, out_bytes, v, (static_cast<size_t>(k_rows - 1) * v_stride + kv_row) * e)))
        return PKV_ERR_INVALID_ARG;
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return PKV_ERR_WORKSPACE;
    PromptArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.out = out;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_offsets = q_offsets;
    a.k_offsets = k_offsets;
    a.err = error_word;
    a.num_seqs = num_seqs;
    a.q_rows = q_rows;
    a.k_rows = k_rows;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.scale_log2 = scale * 1.4426950408889634f;
    first_wait_limit(&a.test_wait_polls, &a.test_wait_cta);
    prompt_tc_workspace(head_dim, static_cast<uint8_t*>(workspace), &a);
    // without a key the other design writes the zero rows (a descriptor has no empty dimension)
    if (k_rows > 0 && prompt_tc_fits(dtype, num_seqs, q_rows, num_q_heads, num_kv_heads)) {
        const cudaError_t r = launch_prompt_tc(head_dim, a, static_cast<cudaStream_t>(stream));
        if (r != cudaErrorNotSupported) return status_of(r);  // (no descriptor of such rows: strides past 2^39, say)
    }
    return status_of(launch_prompt_simt(dtype, head_dim, a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
