// The quantised cache's rows: written with a scale and an offset of their own,
// and read back through block tables as the values that they stand for.
#include "device_common.cuh"
#include "quant_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 128;

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

// One thread per (token, head, K or V) row.
template <int kBits, typename T>
__global__ void __launch_bounds__(kThreads) quant_append_kernel(const QuantAppendArgs a, int dim) {
    const int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    const int64_t rows = static_cast<int64_t>(a.num_tokens) * a.num_kv_heads;
    if (i >= 2 * rows) return;
    const bool is_v = i >= rows;
    const int64_t row = is_v ? i - rows : i;
    const int t = static_cast<int>(row / a.num_kv_heads), h = static_cast<int>(row % a.num_kv_heads);
    const int64_t slot = a.slots[t];
    if (slot == -1) return;
    if (slot < 0 || slot >= a.num_slots) {
        if (a.err) atomicOr(a.err, PKV_ERRBIT_SLOT);
        return;
    }
    const T* x = static_cast<const T*>(is_v ? a.v : a.k) + t * (is_v ? a.v_stride : a.k_stride) + h * dim;
    float lo = INFINITY, hi = -INFINITY;
    bool nan = false;
    for (int j = 0; j < dim; ++j) {
        const float f = to_f32(x[j]);
        nan |= f != f;
        lo = fminf(lo, f);
        hi = fmaxf(hi, f);
    }
    constexpr float N = (1 << kBits) - 1;
    lo += 0.f;  // (no negative zero)
    uint32_t zb = __float_as_uint(lo) & 0xFFFF0000u;
    if (lo < 0.f && zb != __float_as_uint(lo)) zb += 0x10000u;
    const float z = __uint_as_float(zb), r = hi - z;
    const bool bad = nan || !(r <= 3.402823466e38f);
    const float s0 = fmaxf(fmaxf(__fdiv_rn(r, N), fabsf(z) * 0x1p-16f), 0x1p-100f);
    const uint32_t sb = (__float_as_uint(s0) + 0xFFFFu) & 0xFFFF0000u;
    const float inv = __fmul_rn(__frcp_rn(__uint_as_float(sb)), 1.f + 0x1p-21f);
    const int64_t bs = 1ll << a.block_shift;
    const int64_t at = ((slot >> a.block_shift) * a.num_kv_heads + h) * bs + (slot & (bs - 1));
    (is_v ? a.v_params : a.k_params)[at] = bad ? 0x7FC07FC0u : (sb >> 16 | zb);
    uint8_t* c = (is_v ? a.v_codes : a.k_codes) + at * (dim * kBits / 8);
    auto code = [&](int j) -> uint32_t {
        if (bad) return 0u;
        return static_cast<uint32_t>(floorf(__fadd_rn(__fmul_rn(__fsub_rn(to_f32(x[j]), z), inv), 0.5f)));
    };
    for (int j = 0; j < dim; j += 8 / kBits)
        c[j * kBits / 8] = static_cast<uint8_t>(kBits == 8 ? code(j) : code(j) | code(j + 1) << 4);
}

// One warp per packed row and KV head, both tensors.
template <int kKind>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadArgs a, int dim) {
    const int64_t w = (blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (w >= static_cast<int64_t>(a.num_rows) * a.num_kv_heads) return;
    const int row = static_cast<int>(w / a.num_kv_heads), h = static_cast<int>(w % a.num_kv_heads);
    for (int b = 0; b < a.num_seqs; ++b) {
        const int first = a.offsets[b], end = a.offsets[b + 1];
        if (first < 0 || end < first || end > a.num_rows) {
            if (a.err && w == 0 && lane == 0) atomicOr(a.err, PKV_ERRBIT_OFFSETS);
            continue;
        }
        if (row < first || row >= end) continue;
        const int pos = row - first, col = pos >> a.block_shift;
        int blk = -1;
        if (col >= a.max_blocks) {
            if (a.err && lane == 0) atomicOr(a.err, PKV_ERRBIT_SEQ_LEN);
        } else {
            blk = a.tables[static_cast<int64_t>(b) * a.max_blocks + col];
            if (static_cast<unsigned>(blk) >= static_cast<unsigned>(a.num_blocks)) {
                if (a.err && lane == 0) atomicOr(a.err, PKV_ERRBIT_BLOCK_ID);
                blk = -1;
            }
        }
        const int bs = 1 << a.block_shift;
        const int64_t at = ((static_cast<int64_t>(blk) * a.num_kv_heads + h) << a.block_shift) + (pos & (bs - 1));
        for (int v = 0; v < 2; ++v) {
            const uint8_t* src = v ? a.v : a.k;
            for (int j = lane; j < dim; j += 32) {
                float x = 0.f;
                if (blk >= 0) {
                    if constexpr (kKind == kReadF32) {
                        x = reinterpret_cast<const float*>(src)[at * dim + j];
                    } else if constexpr (kKind == kReadBf16) {
                        x = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(src)[at * dim + j]);
                    } else if constexpr (kKind == kReadE4m3) {
                        x = e4m3x2_to_float2(src[at * dim + j]).x * (v ? a.v_scale : a.k_scale);
                    } else {
                        const uint32_t p = (v ? a.v_params : a.k_params)[at];
                        const uint32_t c = kKind == kReadQ8 ? src[at * dim + j]
                                                            : (src[(at * dim + j) >> 1] >> (4 * (j & 1))) & 15u;
                        x = fmaf(bf16_lo(p), static_cast<float>(c), bf16_hi(p));
                    }
                }
                const int64_t o = (static_cast<int64_t>(row) * a.num_kv_heads + h) * dim + j;
                if constexpr (kKind == kReadF32) static_cast<float*>(v ? a.v_out : a.k_out)[o] = x;
                else static_cast<__nv_bfloat16*>(v ? a.v_out : a.k_out)[o] = __float2bfloat16_rn(x);
            }
        }
    }
}

}  // namespace

cudaError_t launch_quant_append(int bits, pkv_dtype in, int head_dim, const QuantAppendArgs& a, cudaStream_t stream) {
    const int64_t rows = 2ll * a.num_tokens * a.num_kv_heads;
    const int64_t blocks = (rows + kThreads - 1) / kThreads;
    if (blocks > INT32_MAX) return cudaErrorNotSupported;
    auto run = [&](auto kernel) {
        kernel<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a, head_dim);
        return cudaGetLastError();
    };
    if (bits == 4) return in == PKV_F32 ? run(quant_append_kernel<4, float>) : run(quant_append_kernel<4, __nv_bfloat16>);
    return in == PKV_F32 ? run(quant_append_kernel<8, float>) : run(quant_append_kernel<8, __nv_bfloat16>);
}

cudaError_t launch_read(ReadKind kind, int head_dim, const ReadArgs& a, cudaStream_t stream) {
    const int64_t blocks = (static_cast<int64_t>(a.num_rows) * a.num_kv_heads * 32 + kThreads - 1) / kThreads;
    if (blocks > INT32_MAX) return cudaErrorNotSupported;
    auto run = [&](auto kernel) {
        kernel<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a, head_dim);
        return cudaGetLastError();
    };
    switch (kind) {
        case kReadF32: return run(read_kernel<kReadF32>);
        case kReadBf16: return run(read_kernel<kReadBf16>);
        case kReadE4m3: return run(read_kernel<kReadE4m3>);
        case kReadQ8: return run(read_kernel<kReadQ8>);
        case kReadQ4: return run(read_kernel<kReadQ4>);
    }
    return cudaErrorNotSupported;
}

}  // namespace pkv
