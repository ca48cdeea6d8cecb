// From the QKV projection to the cache in one pass: RMS norm of every query
// and key head, rotary position embedding, and the append of the keys and
// values ("How does TensorRT-LLM work?", "Kernel fusion": steps that touch
// the same data are merged so that it is read once; "The paged KV cache":
// each new token's keys and values go into the request's blocks).
//
// One head's row x of D elements becomes
//     y_i = x_i * w_i / sqrt(mean(x^2) + eps)           (when weights are given)
//     (z_a, z_b) = (y_a c - y_b s, y_b c + y_a s)       for every rotated pair
// with the pair (a, b) = (j, j + r/2), or (2j, 2j + 1) interleaved, j < r/2,
// and c, s read from the table's row of the token's position on the axis that
// pair j belongs to (time, height, width for images and video; one axis for
// text).  Everything is binary32 from the loaded element to the one rounding
// of the stored one.
//
// It moves bytes and computes almost nothing (about 2 flops per byte), so the
// layout serves the loads: D / 8 lanes hold one head's row, 8 elements each,
// as one 16-byte load (two for fp32) and one store; the norm is a shuffle
// tree over those lanes, the half-split partner of a rotated pair another
// shuffle.  A CTA takes a token at a time and its lane groups the heads, so
// cosines, sines and weights stay in registers over a token's heads (short
// batches spread a token's heads over several CTAs instead: there latency
// counts, not L1 traffic).
#include "device_common.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;

template <int IDT>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&x)[8]) {
    if constexpr (IDT == PKV_F32) {
        const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
        const float4 a = s[0], b = s[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
        const uint4 c = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at);
        KvTraits<PKV_BF16>::to_float(c, x);
    }
}

// 8 elements in dtype ODT; FP8 as the append encodes it: e4m3(x * inv).
template <int ODT>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&x)[8], float inv) {
    if constexpr (ODT == PKV_F32) {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
        d[0] = make_float4(x[0], x[1], x[2], x[3]);
        d[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else if constexpr (ODT == PKV_BF16) {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + at) =
            make_uint4(pack_bf16x2_rn(x[0], x[1]), pack_bf16x2_rn(x[2], x[3]), pack_bf16x2_rn(x[4], x[5]),
                       pack_bf16x2_rn(x[6], x[7]));
    } else {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p) + at) =
            make_uint2(quant4(x[0], x[1], x[2], x[3], inv), quant4(x[4], x[5], x[6], x[7], inv));
    }
}

// Cosines and sines of this lane's 8 elements at one token.  Half-split: of
// pairs j0 .. j0 + 7.  Interleaved: of pairs j0 .. j0 + 3, in c[0..3], s[0..3].
template <bool kInter>
struct Angles {
    static constexpr int kN = kInter ? 4 : 8;
    float c[kN], s[kN];
};

// kWide: every section holds a multiple of kN pairs, so a lane's pairs share
// one axis and load as vectors.
template <bool kInter, bool kWide>
__device__ __forceinline__ void load_angles(const NormRopeArgs& a, const int* pos, int j0, Angles<kInter>& g) {
    constexpr int N = Angles<kInter>::kN;
    const int half = a.rotary_dim >> 1;
    auto axis = [&](int j) { return j < a.axis_end[0] ? 0 : (j < a.axis_end[1] ? 1 : 2); };
    if constexpr (kWide) {
        const int ax = axis(j0);
        const int p = ax == 0 ? pos[0] : (ax == 1 ? pos[1] : pos[2]);
        const float* row = a.cos_sin + static_cast<int64_t>(p) * a.rotary_dim + j0;
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 cv = __ldg(reinterpret_cast<const float4*>(row + i));
            const float4 sv = __ldg(reinterpret_cast<const float4*>(row + half + i));
            g.c[i] = cv.x, g.c[i + 1] = cv.y, g.c[i + 2] = cv.z, g.c[i + 3] = cv.w;
            g.s[i] = sv.x, g.s[i + 1] = sv.y, g.s[i + 2] = sv.z, g.s[i + 3] = sv.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int ax = axis(j0 + i);
            const int p = ax == 0 ? pos[0] : (ax == 1 ? pos[1] : pos[2]);
            const float* row = a.cos_sin + static_cast<int64_t>(p) * a.rotary_dim + j0 + i;
            g.c[i] = __ldg(row);
            g.s[i] = __ldg(row + half);
        }
    }
}

template <int PDT, int IDT, int D, bool kInter, bool kWide>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeArgs a) {
    // (no early trigger of dependents: whatever attends next waits for the whole grid anyway)
    constexpr int kLanes = D / 8, kGroups = kThreads / kLanes;
    constexpr int QDT = PDT == PKV_F32 ? PKV_F32 : PKV_BF16;
    const int sub = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const int heads = a.num_q_heads + 2 * a.num_kv_heads;
    const int half = a.rotary_dim >> 1, e0 = 8 * sub;
    const bool rotated = e0 < a.rotary_dim;
    const bool upper = !kInter && e0 >= half;
    const int j0 = kInter ? e0 / 2 : (upper ? e0 - half : e0);
    // the lane (of this head's kLanes) that holds the other half of the pairs
    const int partner = !rotated ? sub : (upper ? sub - half / 8 : sub + half / 8);
    const unsigned mask = kLanes == 16 ? (0xFFFFu << (threadIdx.x & 16)) : (0xFFu << (threadIdx.x & 24));

    float wq[8], wk[8];
    const bool normed = a.q_weight != nullptr;
    if (normed) {
        if (a.weight_dtype == PKV_F32) {
            load8<PKV_F32>(a.q_weight, e0, wq);
            load8<PKV_F32>(a.k_weight, e0, wk);
        } else {
            load8<PKV_BF16>(a.q_weight, e0, wq);
            load8<PKV_BF16>(a.k_weight, e0, wk);
        }
    }

    // blockIdx.x: a tile of tokens_per_cta tokens (more than one only when a
    // token has fewer heads than the CTA has groups); blockIdx.y: a share of the heads
    const int items = a.tokens_per_cta * heads;
    const int stride = kGroups * gridDim.y, first = blockIdx.y * kGroups + group;
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens_per_cta; t0 < a.num_tokens;
         t0 += static_cast<int64_t>(gridDim.x) * a.tokens_per_cta) {
        int64_t loaded = -1;  // token whose angles and slot are in registers
        Angles<kInter> g;
        int64_t slot = -1;
        bool bad = false;
        for (int i = first; i < items; i += stride) {
            const int dt = a.tokens_per_cta == 1 ? 0 : i / heads;
            const int h = i - dt * heads;
            const int64_t t = t0 + dt;
            if (t >= a.num_tokens) break;
            const bool is_q = h < a.num_q_heads, is_v = h >= a.num_q_heads + a.num_kv_heads;
            const int hk = h - a.num_q_heads - (is_v ? a.num_kv_heads : 0);
            float x[8];
            load8<IDT>(is_q ? a.q : (is_v ? a.v : a.k),
                       is_q ? t * a.q_stride + h * D + e0 : t * (is_v ? a.v_stride : a.k_stride) + hk * D + e0, x);
            if (t != loaded) {
                loaded = t;
                int pos[3] = {0, 0, 0};
                bad = false;
#pragma unroll
                for (int ax = 0; ax < 3; ++ax)
                    if (ax < a.num_axes) {
                        pos[ax] = __ldg(a.positions + static_cast<int64_t>(ax) * a.num_tokens + t);
                        if (static_cast<unsigned>(pos[ax]) >= static_cast<unsigned>(a.max_pos)) {
                            bad = true;
                            pos[ax] = 0;
                        }
                    }
                if (bad && sub == 0 && a.err) atomicOr(a.err, PKV_ERRBIT_POSITION);
                slot = __ldg(a.slots + t);
                if (slot != -1 && (slot < 0 || slot >= a.num_slots)) {
                    if (sub == 0 && a.err) atomicOr(a.err, PKV_ERRBIT_SLOT);
                    slot = -1;
                }
                if (rotated) load_angles<kInter, kWide>(a, pos, j0, g);
            }
            if (!is_q && (slot < 0 || bad)) continue;  // (the whole lane group)
            const int64_t row = is_q ? 0
                                     : ((slot >> a.block_shift) * a.num_kv_heads + hk) * (int64_t(1) << a.block_shift) +
                                           (slot & ((int64_t(1) << a.block_shift) - 1));
            if (is_v) {
                store8<PDT>(a.v_layer, row * D + e0, x, a.v_inv_scale);
                continue;
            }
            if (normed) {
                float ss = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) ss = fmaf(x[k], x[k], ss);
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
                const float r = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = x[k] * r * (is_q ? wq[k] : wk[k]);
            }
            if constexpr (kInter) {
                if (rotated) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float u = x[2 * k], w = x[2 * k + 1];
                        x[2 * k] = u * g.c[k] - w * g.s[k];
                        x[2 * k + 1] = w * g.c[k] + u * g.s[k];
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float y = __shfl_sync(mask, x[k], partner, kLanes);
                    if (rotated) x[k] = upper ? x[k] * g.c[k] + y * g.s[k] : x[k] * g.c[k] - y * g.s[k];
                }
            }
            if (is_q) {
                if (bad) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = 0.f;
                }
                store8<QDT>(a.q_out, (t * a.num_q_heads + h) * D + e0, x, 1.f);
            } else {
                store8<PDT>(a.k_layer, row * D + e0, x, a.k_inv_scale);
            }
        }
    }
}

template <int PDT, int IDT, int D>
cudaError_t launch(NormRopeArgs& a, cudaStream_t stream) {
    constexpr int kGroups = kThreads / (D / 8);
    const int heads = a.num_q_heads + 2 * a.num_kv_heads;
    a.tokens_per_cta = heads >= kGroups ? 1 : kGroups / heads;
    const int64_t tiles = (static_cast<int64_t>(a.num_tokens) + a.tokens_per_cta - 1) / a.tokens_per_cta;
    // Spread a token's heads over CTAs while that gives no more than about one
    // wave (8 CTAs of 256 threads per SM).
    const int sms = num_sms() > 0 ? num_sms() : 148;
    int split = (a.tokens_per_cta * heads + kGroups - 1) / kGroups;
    if (tiles * split > 8LL * sms) split = 1;
    const dim3 grid(static_cast<unsigned>(tiles < (1 << 30) ? tiles : (1 << 30)), split);
    bool wide = true;  // every axis' pairs in whole vectors
    for (int i = 0; i < 2; ++i) wide = wide && a.axis_end[i] % (a.interleaved ? 4 : 8) == 0;
    if (a.interleaved) {
        if (wide) norm_rope_kernel<PDT, IDT, D, true, true><<<grid, kThreads, 0, stream>>>(a);
        else norm_rope_kernel<PDT, IDT, D, true, false><<<grid, kThreads, 0, stream>>>(a);
    } else {
        if (wide) norm_rope_kernel<PDT, IDT, D, false, true><<<grid, kThreads, 0, stream>>>(a);
        else norm_rope_kernel<PDT, IDT, D, false, false><<<grid, kThreads, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

template <int PDT, int IDT>
cudaError_t launch_dim(NormRopeArgs& a, int dim, cudaStream_t stream) {
    return dim == 64 ? launch<PDT, IDT, 64>(a, stream) : launch<PDT, IDT, 128>(a, stream);
}

}  // namespace

cudaError_t launch_norm_rope_append(pkv_dtype pool, pkv_dtype in, int head_dim, NormRopeArgs a, cudaStream_t stream) {
    switch (pool) {
        case PKV_F32:
            if (in == PKV_F32) return launch_dim<PKV_F32, PKV_F32>(a, head_dim, stream);
            break;
        case PKV_BF16:
            if (in == PKV_BF16) return launch_dim<PKV_BF16, PKV_BF16>(a, head_dim, stream);
            if (in == PKV_F32) return launch_dim<PKV_BF16, PKV_F32>(a, head_dim, stream);
            break;
        case PKV_FP8_E4M3:
            if (in == PKV_BF16) return launch_dim<PKV_FP8_E4M3, PKV_BF16>(a, head_dim, stream);
            if (in == PKV_F32) return launch_dim<PKV_FP8_E4M3, PKV_F32>(a, head_dim, stream);
            break;
    }
    return cudaErrorNotSupported;
}

}  // namespace pkv
