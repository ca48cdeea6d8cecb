// Causal attention over packed prompts on the CUDA cores, in binary32.
//
// A unit is 64 consecutive query rows of one (sequence, KV head), rows being
// (query, head of the group) pairs, so that a K or V row serves the whole group.
// A CTA of 256 threads keeps their O in registers (4 rows x head_dim / 16 columns
// each) and walks over the keys, 64 at a time: S = Q K^T (4 x 4 each), softmax
// statistics by the 16 threads of a row, P through shared memory, O += P V.
//
// Bound by its reads of shared memory (a 4 x 4 square takes eight 16-byte reads, 32 cycles of
// the SM's port, for 64 FMAs a lane, 16 of its cycles): 4 prompts of 2000 tokens, 32 query
// heads on 8 of 128, FP32, take 3.8 ms, 34.6 TFLOP/s of what is seen; 47 of 400 tokens of 8 heads
// 0.69 ms, 22.4 TFLOP/s.  Eight rows a thread: 3.4 and 0.83 ms, so not taken.
//
// For F32 rows, and for BF16 ones that the tensor-core design does not take (more than
// 128 query heads per KV head, more sequences than it plans for, no key at all).
#include "device_common.cuh"
#include "quant_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 64, kKeys = 64;

// The rows of sequence b in packed tensors, empty where its offsets cannot be.
struct Span {
    int q0, n, k0, m;
};
__device__ __forceinline__ Span span_of(const PromptArgs& a, int b, bool report) {
    Span s{a.q_offsets[b], a.q_offsets[b + 1], a.k_offsets[b], a.k_offsets[b + 1]};
    const bool ok = s.q0 >= 0 && s.n >= s.q0 && s.n <= a.q_rows && s.k0 >= 0 && s.m >= s.k0 && s.m <= a.k_rows;
    if (!ok && report && a.err) atomicOr(a.err, PKV_ERRBIT_OFFSETS);
    s.n = ok ? s.n - s.q0 : 0;
    s.m = ok ? s.m - s.k0 : 0;
    return s;
}

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}

template <typename T, int kDim>
__global__ void __launch_bounds__(kThreads, 2) prompt_simt_kernel(const PromptArgs a) {
    constexpr int kPitch = kDim + 4, kCols = kDim / 16;
    extern __shared__ float smem[];
    float* sq = smem;                       // [kRows][kPitch]
    float* skv = sq + kRows * kPitch;       // [kKeys][kPitch] K, then V
    float* sp = skv + kKeys * kPitch;       // [kRows][kKeys + 4]
    const int tid = threadIdx.x, gh = a.num_q_heads / a.num_kv_heads, h = blockIdx.y;
    // unit blockIdx.x: the sequences' row tiles, one sequence after the other (256 sequences at a time)
    __shared__ long long sums[kThreads / 32];
    __shared__ Span mine_;
    __shared__ long long tile_;
    const bool reports = blockIdx.x == 0 && h == 0;
    long long before = 0;
    bool found = false;
    for (int b0 = 0; b0 < a.num_seqs && (reports || !found); b0 += kThreads) {
        const Span at = b0 + tid < a.num_seqs ? span_of(a, b0 + tid, reports) : Span{};
        const long long tiles = (static_cast<long long>(at.n) * gh + kRows - 1) / kRows;
        long long incl = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long x = __shfl_up_sync(0xFFFFFFFFu, incl, d);
            if (tid % 32 >= d) incl += x;
        }
        if (tid % 32 == 31) sums[tid / 32] = incl;
        __syncthreads();
        incl += before;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < tid / 32) incl += sums[w];
            before += sums[w];
        }
        const bool here = blockIdx.x >= incl - tiles && blockIdx.x < incl;
        if (here) mine_ = at, tile_ = incl - 1 - blockIdx.x;  // (the longest first)
        found |= __syncthreads_or(here) != 0;
    }
    if (!found) return;
    const Span s = mine_;
    const long long tile = tile_;
    const int64_t row0 = tile * kRows, rows = static_cast<int64_t>(s.n) * gh;
    const T* q = static_cast<const T*>(a.q);
    const T* k = static_cast<const T*>(a.k) + s.k0 * a.k_stride + static_cast<int64_t>(h) * kDim;
    const T* v = static_cast<const T*>(a.v) + s.k0 * a.v_stride + static_cast<int64_t>(h) * kDim;
    constexpr int kQuads = kDim / 4;  // four elements at a time
    for (int i = tid; i < kRows * kQuads; i += kThreads) {
        const int64_t r = row0 + i / kQuads;
        const int d = i % kQuads * 4;
        *reinterpret_cast<float4*>(sq + i / kQuads * kPitch + d) =
            r < rows ? load4(q + (s.q0 + r / gh) * a.q_stride + (h * gh + r % gh) * kDim + d) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int ty = tid / 16, tx = tid % 16;  // rows 4 ty .. + 3, keys tx + 16 j, columns tx * 4 + 64 j
    int seen[4];                             // keys that each row sees
    for (int i = 0; i < 4; ++i) {
        const int64_t r = row0 + 4 * ty + i;
        seen[i] = r < rows ? max(0, s.m - s.n + static_cast<int>(r / gh) + 1) : 0;
    }
    const int64_t last = min(rows, row0 + kRows) - 1;
    const int keys = max(0, s.m - s.n + static_cast<int>(last / gh) + 1);
    float o[4][kCols] = {}, mx[4], l[4] = {};
    for (int i = 0; i < 4; ++i) mx[i] = -INFINITY;
    for (int t0 = 0; t0 < keys; t0 += kKeys) {
        // V's rows are on their way, in registers, while K's are multiplied
        constexpr int kMine = kKeys * kQuads / kThreads;
        float4 vr[kMine];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int e = tid + i * kThreads, t = t0 + e / kQuads, d = e % kQuads * 4;
            *reinterpret_cast<float4*>(skv + e / kQuads * kPitch + d) =
                t < keys ? load4(k + t * a.k_stride + d) : make_float4(0.f, 0.f, 0.f, 0.f);
            vr[i] = t < keys ? load4(v + t * a.v_stride + d) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        __syncthreads();
        float x[4][4] = {};
#pragma unroll 4
        for (int d = 0; d < kDim; d += 4) {
            float4 qa[4], kb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) qa[i] = *reinterpret_cast<const float4*>(sq + (4 * ty + i) * kPitch + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) kb[j] = *reinterpret_cast<const float4*>(skv + (tx + 16 * j) * kPitch + d);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[i][j] = fmaf(qa[i].x, kb[j].x, fmaf(qa[i].y, kb[j].y, fmaf(qa[i].z, kb[j].z, fmaf(qa[i].w, kb[j].w, x[i][j]))));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][j] = t0 + tx + 16 * j < seen[i] ? x[i][j] * a.scale_log2 : -INFINITY;
                top = fmaxf(top, x[i][j]);
            }
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, w));
            const float m_new = fmaxf(mx[i], top), base = m_new == -INFINITY ? 0.f : m_new;
            const float alpha = exp2f(mx[i] - base);
            mx[i] = m_new;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = t0 + tx + 16 * j < seen[i] ? exp2f(x[i][j] - base) : 0.f;
                sp[(4 * ty + i) * (kKeys + 4) + tx + 16 * j] = p;
                sum += p;
            }
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, w);
            l[i] = l[i] * alpha + sum;
#pragma unroll
            for (int c = 0; c < kCols; ++c) o[i][c] *= alpha;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int e = tid + i * kThreads;
            *reinterpret_cast<float4*>(skv + e / kQuads * kPitch + e % kQuads * 4) = vr[i];
        }
        __syncthreads();
#pragma unroll 2
        for (int t = 0; t < kKeys; t += 4) {
            float4 p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(sp + (4 * ty + i) * (kKeys + 4) + t);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
#pragma unroll
                for (int c = 0; c < kCols; c += 4) {
                    const float4 w = *reinterpret_cast<const float4*>(skv + (t + u) * kPitch + 16 * c + 4 * tx);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float pu = u == 0 ? p[i].x : u == 1 ? p[i].y : u == 2 ? p[i].z : p[i].w;
                        o[i][c] = fmaf(pu, w.x, o[i][c]);
                        o[i][c + 1] = fmaf(pu, w.y, o[i][c + 1]);
                        o[i][c + 2] = fmaf(pu, w.z, o[i][c + 2]);
                        o[i][c + 3] = fmaf(pu, w.w, o[i][c + 3]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = row0 + 4 * ty + i;
        if (r >= rows) continue;
        T* dst = static_cast<T*>(a.out) + ((s.q0 + r / gh) * a.num_q_heads + h * gh + r % gh) * static_cast<int64_t>(kDim);
        const float inv = 1.f / l[i];
#pragma unroll
        for (int c = 0; c < kCols; ++c) dst[16 * (c & ~3) + 4 * tx + (c & 3)] = to_out<T>(seen[i] > 0 ? o[i][c] * inv : 0.f);
    }
}

template <typename T, int kDim>
cudaError_t launch_simt(const PromptArgs& a, cudaStream_t stream) {
    constexpr int smem = (kRows * (kDim + 4) + kKeys * (kDim + 4) + kRows * (kKeys + 4)) * 4;  // (two CTAs an SM)
    const int64_t tiles = static_cast<int64_t>(a.q_rows) * (a.num_q_heads / a.num_kv_heads) / kRows + a.num_seqs;
    if (tiles > INT32_MAX || a.num_kv_heads > 65535) return cudaErrorNotSupported;
    const cudaError_t e = cudaFuncSetAttribute(prompt_simt_kernel<T, kDim>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    prompt_simt_kernel<T, kDim><<<dim3(static_cast<unsigned>(tiles), a.num_kv_heads), kThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_simt(pkv_dtype t, int head_dim, const PromptArgs& a, cudaStream_t stream) {
    if (t == PKV_F32) return head_dim == 64 ? launch_simt<float, 64>(a, stream) : launch_simt<float, 128>(a, stream);
    return head_dim == 64 ? launch_simt<__nv_bfloat16, 64>(a, stream) : launch_simt<__nv_bfloat16, 128>(a, stream);
}

}  // namespace pkv
