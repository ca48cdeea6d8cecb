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
// It moves bytes, but at two flops a byte and 8 elements a lane the instructions
// count (to keep up with memory a warp may spend about 170 on 1 KB), and so does
// the chain position -> angles -> rows.  Hence:
//  * a warp takes a fixed run of query, key or value heads (blockIdx.y) and
//    walks over tokens; D / 8 lanes hold one head's row, so weights stay in
//    registers, and the slot and the angles are fetched, and weights and angles
//    multiplied, once for the kRows rows of a lane, which lie at constant offsets;
//  * a lane holds both halves of its four rotated pairs (two 8-byte loads in
//    the half-split layout, one 16-byte load interleaved): no shuffle, four
//    angles instead of eight.  Lanes past the rotated part hold 8 elements in a
//    row;
//  * a token's rows and angles are under way together (its position was fetched
//    a token ahead); 24 warps per SM overlap one another's waits.  Fetching the
//    rows a token ahead as well costs the registers of a third of the warps, and
//    was slower (170 us where this takes 130).
// 4096 tokens of 48 heads, BF16, 103 MB: 21.1 us, 4.9 TB/s (72 % of the measured
// copy rate), over buffers that rotate through six times that much; 17.5 us on
// the same ones again and again, which the L2 (129 MB) serves in part.  What
// bounds it is the walk, not memory: a warp takes about seven tokens, and asks
// for the rows of one only after it has stored those of the one before.  32771
// tokens, three position axes, interleaved, FP8 pool: 132 us, 5.6 TB/s (83 %).  64
// tokens: 3 us, an empty launch being 2.
#include "device_common.cuh"
#include "step_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;

template <int IDT>
struct Raw;  // 4 + 4 elements as loaded
template <>
struct Raw<PKV_BF16> {
    uint2 a, b;
    template <bool kTogether = false>  // o1 = o0 + 4: one access
    __device__ __forceinline__ void load(const void* p, int64_t at, int o0, int o1) {
        const __nv_bfloat16* s = static_cast<const __nv_bfloat16*>(p) + at;
        if constexpr (kTogether) {
            const uint4 v = *reinterpret_cast<const uint4*>(s + o0);
            a = make_uint2(v.x, v.y);
            b = make_uint2(v.z, v.w);
        } else {
            a = *reinterpret_cast<const uint2*>(s + o0);
            b = *reinterpret_cast<const uint2*>(s + o1);
        }
    }
    __device__ __forceinline__ void get(float (&x)[4], float (&y)[4]) const {
        x[0] = bf16_lo(a.x), x[1] = bf16_hi(a.x), x[2] = bf16_lo(a.y), x[3] = bf16_hi(a.y);
        y[0] = bf16_lo(b.x), y[1] = bf16_hi(b.x), y[2] = bf16_lo(b.y), y[3] = bf16_hi(b.y);
    }
};
template <>
struct Raw<PKV_F32> {
    float4 a, b;
    template <bool kTogether = false>
    __device__ __forceinline__ void load(const void* p, int64_t at, int o0, int o1) {
        const float* s = static_cast<const float*>(p) + at;
        a = *reinterpret_cast<const float4*>(s + o0);
        b = *reinterpret_cast<const float4*>(s + o1);
    }
    __device__ __forceinline__ void get(float (&x)[4], float (&y)[4]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        y[0] = b.x, y[1] = b.y, y[2] = b.z, y[3] = b.w;
    }
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {  // both rounded to nearest even
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// 4 + 4 elements in dtype ODT; FP8 as the append encodes it: e4m3(x * inv).
template <int ODT, bool kTogether>
__device__ __forceinline__ void store(void* p, int64_t at, int o0, int o1, const float (&x)[4], const float (&y)[4], float inv) {
    if constexpr (ODT == PKV_F32) {
        float* d = static_cast<float*>(p) + at;
        *reinterpret_cast<float4*>(d + o0) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(d + o1) = make_float4(y[0], y[1], y[2], y[3]);
    } else if constexpr (ODT == PKV_BF16) {
        __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p) + at;
        const uint2 a = make_uint2(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]));
        const uint2 b = make_uint2(bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]));
        if constexpr (kTogether) {
            *reinterpret_cast<uint4*>(d + o0) = make_uint4(a.x, a.y, b.x, b.y);
        } else {
            *reinterpret_cast<uint2*>(d + o0) = a;
            *reinterpret_cast<uint2*>(d + o1) = b;
        }
    } else {
        uint8_t* d = static_cast<uint8_t*>(p) + at;
        const uint32_t a = quant4(x[0], x[1], x[2], x[3], inv), b = quant4(y[0], y[1], y[2], y[3], inv);
        if constexpr (kTogether) {
            *reinterpret_cast<uint2*>(d + o0) = make_uint2(a, b);
        } else {
            *reinterpret_cast<uint32_t*>(d + o0) = a;
            *reinterpret_cast<uint32_t*>(d + o1) = b;
        }
    }
}

// 1 / sqrt on the special-function unit (relative error about 2^-22).
__device__ __forceinline__ float rsqrt_fast(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

// Rows of a lane: a run is kRows * 256 / D heads.  Two rows with more warps
// resident take 181 us on 32771 tokens of 48 heads (three position axes, FP8
// pool) where four take 130, eight 156: fewer do not pay for the lookups, more
// leave too few warps.
constexpr int kRows = 4;
constexpr int ctas_per_sm(int in_dtype) { return in_dtype == PKV_F32 ? 2 : 3; }  // what the registers allow

// kMulti: more than one position axis.
template <int PDT, int IDT, int D, bool kInter, bool kMulti>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(IDT)) norm_rope_kernel(const NormRopeArgs a) {
    constexpr int kLanes = D / 8, kSide = 32 / kLanes, kRun = kRows * kSide;  // rows side by side in a warp; heads of a run
    constexpr int QDT = PDT == PKV_F32 ? PKV_F32 : PKV_BF16;
    const int lane = threadIdx.x & 31, sub = lane % kLanes, side = lane / kLanes;
    const int Hq = a.num_q_heads, Hk = a.num_kv_heads;
    const int q_runs = (Hq + kRun - 1) / kRun, k_runs = (Hk + kRun - 1) / kRun, run = blockIdx.y;
    const bool is_q = run < q_runs, is_v = run >= q_runs + k_runs;
    const int heads = is_q ? Hq : Hk;
    const int h0 = (is_q ? run : (is_v ? run - q_runs - k_runs : run - q_runs)) * kRun + side;

    const int half = a.rotary_dim >> 1;
    const bool rotated = sub < half / 4;
    // this lane's elements: o0 .. o0 + 3 and o1 .. o1 + 3; its pairs j0 .. j0 + 3
    const int j0 = 4 * sub;
    const int o0 = kInter ? 8 * sub : (rotated ? j0 : a.rotary_dim + 8 * (sub - half / 4));
    const int o1 = !kInter && rotated ? half + j0 : o0 + 4;
    // (where the axis changes inside the lane's pairs, they are looked up one by one)
    const bool one_axis = (j0 < a.axis_end[0]) == (j0 + 3 < a.axis_end[0]) && (j0 < a.axis_end[1]) == (j0 + 3 < a.axis_end[1]);

    const int64_t step_t = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    int64_t t = blockIdx.x * static_cast<int64_t>(kThreads / 32) + (threadIdx.x >> 5);
    if (t >= a.num_tokens) return;

    constexpr int kAxes = kMulti ? 3 : 1;
    struct Token {  // of the warp
        int pos[kAxes];
        bool bad;
        int64_t slot;
    };
    auto look_up = [&](int64_t tt, Token& k) {
        k.bad = false;
        k.pos[0] = __ldg(a.positions + tt);
        if constexpr (kMulti) {
            k.pos[1] = __ldg(a.positions + a.num_tokens + tt);
            k.pos[2] = a.num_axes > 2 ? __ldg(a.positions + 2LL * a.num_tokens + tt) : 0;
        }
        k.slot = __ldg(a.slots + tt);
    };
    auto check = [&](Token& k) {  // (run 0 of every token reports)
#pragma unroll
        for (int ax = 0; ax < kAxes; ++ax) k.bad = k.bad || static_cast<unsigned>(k.pos[ax]) >= static_cast<unsigned>(a.max_pos);
        if (k.bad && run == 0 && lane == 0 && a.err) atomicOr(a.err, PKV_ERRBIT_POSITION);
        if (k.slot < -1 || k.slot >= a.num_slots) {
            if (run == 0 && lane == 0 && a.err) atomicOr(a.err, PKV_ERRBIT_SLOT);
            k.slot = -1;
        }
    };
    const void* src = is_q ? a.q : (is_v ? a.v : a.k);
    const int64_t src_stride = is_q ? a.q_stride : (is_v ? a.v_stride : a.k_stride);
    auto fetch = [&](int64_t tt, Raw<IDT> (&raw)[kRows]) {
        const int64_t from = tt * src_stride + static_cast<int64_t>(h0) * D;
#pragma unroll
        for (int u = 0; u < kRows; ++u)
            if (h0 + u * kSide < heads) raw[u].template load<kInter>(src, from + u * kSide * D, o0, o1);
    };
    // cosines and sines of this lane's pairs (a bad position reads nothing)
    auto on_axis = [&](const Token& k, int j) {
        if constexpr (!kMulti) return k.pos[0];
        else return j < a.axis_end[0] ? k.pos[0] : (j < a.axis_end[1] ? k.pos[1] : k.pos[2]);
    };
    auto turn = [&](const Token& k, float (&c)[4], float (&s)[4]) {
        if (!rotated || is_v || k.bad) return;
        if (!kMulti || one_axis) {
            const int p = on_axis(k, j0);
            const float* row = a.cos_sin + static_cast<int64_t>(p) * a.rotary_dim + j0;
            const float4 c4 = __ldg(reinterpret_cast<const float4*>(row));
            const float4 s4 = __ldg(reinterpret_cast<const float4*>(row + half));
            c[0] = c4.x, c[1] = c4.y, c[2] = c4.z, c[3] = c4.w;
            s[0] = s4.x, s[1] = s4.y, s[2] = s4.z, s[3] = s4.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int p = on_axis(k, j0 + i);
                const float* row = a.cos_sin + static_cast<int64_t>(p) * a.rotary_dim + j0 + i;
                c[i] = __ldg(row);
                s[i] = __ldg(row + half);
            }
        }
    };

    Token now, next;
    look_up(t, next);
    const bool normed = a.q_weight != nullptr;
    float w0[4] = {1.f, 1.f, 1.f, 1.f}, w1[4] = {1.f, 1.f, 1.f, 1.f};
    if (normed && !is_v) {
        const void* w = is_q ? a.q_weight : a.k_weight;
        if (a.weight_dtype == PKV_F32) {
            Raw<PKV_F32> r;
            r.load(w, 0, o0, o1);
            r.get(w0, w1);
        } else {
            Raw<PKV_BF16> r;
            r.load(w, 0, o0, o1);
            r.get(w0, w1);
        }
    }

    for (; t < a.num_tokens; t += step_t) {
        Raw<IDT> raw[kRows];
        fetch(t, raw);
        now = next;
        check(now);
        float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
        turn(now, c, s);
        if (t + step_t < a.num_tokens) look_up(t + step_t, next);
        const Token& cur = now;
        // where the rows go: consecutive heads of a token, or of a slot of the pool
        const int64_t block_rows = int64_t(1) << a.block_shift;
        const int64_t step = is_q ? kSide * D : kSide * D * block_rows;
        int64_t at = is_q ? (t * Hq + h0) * D
                          : (((cur.slot >> a.block_shift) * Hk + h0) * block_rows + (cur.slot & (block_rows - 1))) * D;
        if (is_v) {
            if (cur.slot >= 0 && !cur.bad) {
#pragma unroll
                for (int u = 0; u < kRows; ++u, at += step)
                    if (h0 + u * kSide < heads) {
                        float x[4], y[4];
                        raw[u].get(x, y);
                        store<PDT, kInter>(a.v_layer, at, o0, o1, x, y, a.v_inv_scale);
                    }
            }
        } else if (cur.bad) {
            if (is_q) {
                const float none[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int u = 0; u < kRows; ++u, at += step)
                    if (h0 + u * kSide < heads) {
                        store<QDT, kInter>(a.q_out, at, o0, o1, none, none, 1.f);
                    }
            }
        } else if (is_q || cur.slot >= 0) {
            // Weights and angles multiplied: the first element of pair k becomes
            // f c w_f - g s w_g, the second g c w_g + f s w_f.
            float fc[4], gs[4], gc[4], fs[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float wf = kInter ? (k < 2 ? w0[2 * k] : w1[2 * k - 4]) : w0[k];
                const float wg = kInter ? (k < 2 ? w0[2 * k + 1] : w1[2 * k - 3]) : w1[k];
                fc[k] = wf * c[k];
                gs[k] = wg * s[k];
                gc[k] = wg * c[k];
                fs[k] = wf * s[k];
            }
#pragma unroll
            for (int u = 0; u < kRows; ++u, at += step) {
                if (h0 + u * kSide - side >= heads) break;  // (the whole warp)
                float x[4], y[4];
                raw[u].get(x, y);
                if (normed) {
                    float p = 0.f, q = 0.f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        p = fmaf(x[k], x[k], p);
                        q = fmaf(y[k], y[k], q);
                    }
                    float ss = p + q;
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
                    const float r = rsqrt_fast(fmaf(ss, 1.f / D, a.eps));
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        x[k] *= r;
                        y[k] *= r;
                    }
                }
                if (rotated) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float& f = kInter ? (k < 2 ? x[2 * k] : y[2 * k - 4]) : x[k];
                        float& g = kInter ? (k < 2 ? x[2 * k + 1] : y[2 * k - 3]) : y[k];
                        const float f0 = f;
                        f = f0 * fc[k] - g * gs[k];
                        g = g * gc[k] + f0 * fs[k];
                    }
                } else if (normed) {  // (kept apart: one of the elements may be infinite)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        x[k] *= w0[k];
                        y[k] *= w1[k];
                    }
                }
                if (h0 + u * kSide < heads) {
                    if (is_q) store<QDT, kInter>(a.q_out, at, o0, o1, x, y, 1.f);
                    else store<PDT, kInter>(a.k_layer, at, o0, o1, x, y, a.k_inv_scale);
                }
            }
        }
    }
}

template <int PDT, int IDT, int D>
cudaError_t launch(const NormRopeArgs& a, cudaStream_t stream) {
    constexpr int kRun = kRows * 256 / D, kWarps = kThreads / 32;
    const int64_t runs = (a.num_q_heads + kRun - 1) / kRun + 2LL * ((a.num_kv_heads + kRun - 1) / kRun);
    if (runs > 65535) return cudaErrorNotSupported;
    // One wave in all; every warp walks over as many tokens.
    const int sms = num_sms() > 0 ? num_sms() : 148;
    const int64_t most = (a.num_tokens + kWarps - 1LL) / kWarps;
    int64_t x = (static_cast<int64_t>(ctas_per_sm(IDT)) * sms + runs - 1) / runs;
    if (x > most) x = most;
    const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(runs));
    const bool multi = a.num_axes > 1;
    auto kernel = a.interleaved
                      ? (multi ? norm_rope_kernel<PDT, IDT, D, true, true> : norm_rope_kernel<PDT, IDT, D, true, false>)
                      : (multi ? norm_rope_kernel<PDT, IDT, D, false, true> : norm_rope_kernel<PDT, IDT, D, false, false>);
    kernel<<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <int PDT, int IDT>
cudaError_t launch_dim(const NormRopeArgs& a, int dim, cudaStream_t stream) {
    return dim == 64 ? launch<PDT, IDT, 64>(a, stream) : launch<PDT, IDT, 128>(a, stream);
}

}  // namespace

cudaError_t launch_norm_rope_append(pkv_dtype pool, pkv_dtype in, int head_dim, const NormRopeArgs& a,
                                    cudaStream_t stream) {
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
