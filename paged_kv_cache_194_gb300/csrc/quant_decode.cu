// Decode attention over a quantised cache: with codes n and pairs (s, z),
//     t_j = scale (s_j (q . n_j) + z_j sum(q)),   out = sum_j softmax(t)_j (s'_j n'_j + z'_j).
#include "device_common.cuh"
#include "quant_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 128;

// One CTA per (sequence, query head): a thread per token for the scores of 128
// tokens, then a thread per dimension.
template <int kBits, int kDim>
__global__ void __launch_bounds__(kThreads) quant_decode_kernel(const QuantDecodeArgs a) {
    __shared__ float q[kDim], p[kThreads], pz[kThreads], red[8];
    __shared__ int64_t at[kThreads];
    const int b = blockIdx.x, hq = blockIdx.y, h = hq / (a.num_q_heads / a.num_kv_heads), tid = threadIdx.x;
    int L = a.lens[b];
    if (L < 0 || L > a.max_len) {
        if (a.err && hq == 0 && tid == 0) atomicOr(a.err, PKV_ERRBIT_SEQ_LEN);
        L = L < 0 ? 0 : a.max_len;
    }
    const int64_t o = (static_cast<int64_t>(b) * a.num_q_heads + hq) * kDim;
    float sum_q = 0.f;
    if (tid < kDim) q[tid] = __bfloat162float(a.q[o + tid]);
    __syncthreads();
    for (int j = 0; j < kDim; ++j) sum_q += q[j];
    float m = -INFINITY, l = 0.f, acc = 0.f;
    constexpr int kRow = kDim * kBits / 8;
    auto code = [&](const uint8_t* row, int j) {
        return static_cast<float>(kBits == 8 ? row[j] : (row[j >> 1] >> (4 * (j & 1))) & 15);
    };
    for (int t0 = 0; t0 < L; t0 += kThreads) {
        const int t = t0 + tid, bs = 1 << a.block_shift;
        float x = -INFINITY;
        at[tid] = 0;
        if (t < L) {
            int blk = a.tables[static_cast<int64_t>(b) * a.max_blocks + (t >> a.block_shift)];
            if (static_cast<unsigned>(blk) >= static_cast<unsigned>(a.num_blocks)) {
                if (a.err) atomicOr(a.err, PKV_ERRBIT_BLOCK_ID);
                blk = 0;
            }
            at[tid] = ((static_cast<int64_t>(blk) * a.num_kv_heads + h) << a.block_shift) + (t & (bs - 1));
            const uint8_t* row = a.k_codes + at[tid] * kRow;
            float dot = 0.f;
            for (int j = 0; j < kDim; ++j) dot = fmaf(q[j], code(row, j), dot);
            const uint32_t kp = a.k_params[at[tid]];
            x = a.scale_log2 * (bf16_lo(kp) * dot + bf16_hi(kp) * sum_q);
        }
        // (a NaN score stays one: the maximum ignores it, its weight does not)
        const float wm = warp_max(x);
        if ((tid & 31) == 0) red[tid >> 5] = wm;
        __syncthreads();
        const float mt = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        const float base = mt == -INFINITY ? 0.f : mt, alpha = exp2f(m - base);
        const float w = t < L ? exp2f(x - base) : 0.f;
        const uint32_t vp = t < L ? a.v_params[at[tid]] : 0u;
        p[tid] = w * bf16_lo(vp);
        pz[tid] = w * bf16_hi(vp);
        const float ws = warp_sum(w);
        if ((tid & 31) == 0) red[4 + (tid >> 5)] = ws;
        __syncthreads();
        l = l * alpha + red[4] + red[5] + red[6] + red[7];
        m = mt;
        if (tid < kDim) {
            acc *= alpha;
            const int n = min(kThreads, L - t0);
            for (int i = 0; i < n; ++i) acc += fmaf(p[i], code(a.v_codes + at[i] * kRow, tid), pz[i]);
        }
        __syncthreads();
    }
    if (tid < kDim) a.out[o + tid] = __float2bfloat16_rn(L > 0 ? acc / l : 0.f);
}

}  // namespace

size_t quant_decode_workspace(int, int, int, int, uint8_t*, QuantDecodeArgs*) { return 0; }

cudaError_t launch_quant_decode(int bits, int head_dim, const QuantDecodeArgs& a, cudaStream_t stream) {
    const dim3 grid(a.num_seqs, a.num_q_heads);
    auto run = [&](auto kernel) {
        kernel<<<grid, kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    };
    if (bits == 4) return head_dim == 64 ? run(quant_decode_kernel<4, 64>) : run(quant_decode_kernel<4, 128>);
    return head_dim == 64 ? run(quant_decode_kernel<8, 64>) : run(quant_decode_kernel<8, 128>);
}

}  // namespace pkv
