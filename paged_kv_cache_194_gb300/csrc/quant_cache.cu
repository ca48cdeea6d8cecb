// The quantised cache's rows: written with a scale and an offset of their own,
// and read back through block tables as the values that they stand for.
//
// Both are one pass over memory, and what bounds them is HBM; per 16 bytes of BF16 the
// copy rate leaves an SM about 14 instructions a lane, so the work per element counts.
#include "device_common.cuh"
#include "quant_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr unsigned kAll = 0xFFFFFFFFu;

__device__ __forceinline__ float min_nan(float a, float b) {  // NaN if one is
    float d;
    asm("min.NaN.f32 %0, %1, %2;\n" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
// (the bits of 2^23 + floor(x), 0 <= x < 2^23: the integer lies in the low bits)
__device__ __forceinline__ uint32_t floor_bits(float x) {
    float d;
    asm("add.rm.f32 %0, %1, 0f4B000000;\n" : "=f"(d) : "f"(x));
    return __float_as_uint(d);
}
__device__ __forceinline__ uint4 load16(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// ------------------------------------------------------------------- append
// Eight elements a lane, kDim / 8 lanes a row, kUnroll groups of rows under way in a
// warp.  A row's lanes share its minimum and maximum by shuffles: one of both together
// with BF16 rows, as the pair (min, -max).
template <int kBits, int kDim, typename T, int kUnroll>
__global__ void __launch_bounds__(kThreads) quant_append_kernel(const QuantAppendArgs a) {
    constexpr int kLanes = kDim / 8, kRows = 32 / kLanes;  // lanes of a row, rows of a warp
    constexpr bool kWide = sizeof(T) == 4;
    constexpr float N = (1 << kBits) - 1;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int lane = threadIdx.x & 31, part = lane % kLanes;
    const int per_token = 2 * a.num_kv_heads;  // rows: K heads, then V heads of each token
    const int64_t total = static_cast<int64_t>(a.num_tokens) * per_token;
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * (kRows * kUnroll) + lane / kLanes;
    uint4 raw[kUnroll][kWide ? 2 : 1];
    int64_t slot[kUnroll];
    int head[kUnroll];
    bool is_v[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const int64_t r = first + i * kRows;
        const bool there = r < total;
        // (a 32-bit division where it will do)
        const int t = !there ? 0 : static_cast<int>(total <= UINT32_MAX ? static_cast<uint32_t>(r) / per_token : r / per_token);
        const int j = there ? static_cast<int>(r - static_cast<int64_t>(t) * per_token) : 0;
        is_v[i] = j >= a.num_kv_heads;
        head[i] = is_v[i] ? j - a.num_kv_heads : j;
        slot[i] = there ? a.slots[t] : -1;
        const T* x = static_cast<const T*>(is_v[i] ? a.v : a.k) + t * (is_v[i] ? a.v_stride : a.k_stride) +
                     static_cast<int64_t>(head[i]) * kDim + 8 * part;
        raw[i][0] = load16(x);
        if constexpr (kWide) raw[i][1] = load16(x + 4);
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        float x[8], lo, hi;
        const uint32_t w[4] = {raw[i][0].x, raw[i][0].y, raw[i][0].z, raw[i][0].w};
        if constexpr (kWide) {
            const uint32_t u[4] = {raw[i][1].x, raw[i][1].y, raw[i][1].z, raw[i][1].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = __uint_as_float(w[k]), x[4 + k] = __uint_as_float(u[k]);
            lo = hi = x[0];
#pragma unroll
            for (int k = 1; k < 8; ++k) lo = min_nan(lo, x[k]), hi = max_nan(hi, x[k]);
#pragma unroll
            for (int d = kLanes / 2; d > 0; d >>= 1) {
                lo = min_nan(lo, __shfl_xor_sync(kAll, lo, d));
                hi = max_nan(hi, __shfl_xor_sync(kAll, hi, d));
            }
        } else {
            __nv_bfloat162 mn, mx;
            const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(w);
            mn = __hmin2_nan(__hmin2_nan(h[0], h[1]), __hmin2_nan(h[2], h[3]));
            mx = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
            __nv_bfloat162 both = __halves2bfloat162(__hmin_nan(__low2bfloat16(mn), __high2bfloat16(mn)),
                                                     __hneg(__hmax_nan(__low2bfloat16(mx), __high2bfloat16(mx))));
#pragma unroll
            for (int d = kLanes / 2; d > 0; d >>= 1) {
                const uint32_t o = __shfl_xor_sync(kAll, *reinterpret_cast<uint32_t*>(&both), d);
                both = __hmin2_nan(both, *reinterpret_cast<const __nv_bfloat162*>(&o));
            }
            lo = __low2float(both);
            hi = -__high2float(both);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[2 * k] = bf16_lo(w[k]), x[2 * k + 1] = bf16_hi(w[k]);
        }
        lo = __fadd_rn(lo, 0.f);  // (no negative zero)
        uint32_t zb = __float_as_uint(lo) & 0xFFFF0000u;
        if (kWide && lo < 0.f && zb != __float_as_uint(lo)) zb += 0x10000u;  // (BF16 rows have their minimum in BF16)
        const float z = __uint_as_float(zb), r = __fsub_rn(hi, z);
        const bool bad = !(r <= 3.402823466e38f);  // an infinity or a NaN in the row, or a range that is not finite
        const float s0 = fmaxf(fmaxf(__fdiv_rn(r, N), fabsf(z) * 0x1p-16f), 0x1p-100f);
        const uint32_t sb = (__float_as_uint(s0) + 0xFFFFu) & 0xFFFF0000u;
        const float inv = bad ? 0.f : __fmul_rn(__frcp_rn(__uint_as_float(sb)), 1.f + 0x1p-21f);
        if (slot[i] == -1) continue;
        if (slot[i] < 0 || slot[i] >= a.num_slots) {
            if (a.err && part == 0) atomicOr(a.err, PKV_ERRBIT_SLOT);
            continue;
        }
        uint32_t n[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            n[k] = floor_bits(__fadd_rn(__fmul_rn(bad ? 0.f : __fsub_rn(x[k], z), inv), 0.5f));
        const int64_t at = (((slot[i] >> a.block_shift) * a.num_kv_heads + head[i]) << a.block_shift) +
                           (slot[i] & ((1 << a.block_shift) - 1));
        uint8_t* codes = (is_v[i] ? a.v_codes : a.k_codes) + at * (kDim * kBits / 8) + part * kBits;
        if constexpr (kBits == 4) {
            const uint32_t even = __byte_perm(__byte_perm(n[0], n[2], 0x0040), __byte_perm(n[4], n[6], 0x0040), 0x5410);
            const uint32_t odd = __byte_perm(__byte_perm(n[1], n[3], 0x0040), __byte_perm(n[5], n[7], 0x0040), 0x5410);
            *reinterpret_cast<uint32_t*>(codes) = even | odd << 4;
        } else {
            uint2 c;
            c.x = __byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410);
            c.y = __byte_perm(__byte_perm(n[4], n[5], 0x0040), __byte_perm(n[6], n[7], 0x0040), 0x5410);
            *reinterpret_cast<uint2*>(codes) = c;
        }
        if (part == 0) (is_v[i] ? a.v_params : a.k_params)[at] = bad ? 0x7FC07FC0u : (sb >> 16 | zb);
    }
}

template <int kBits, int kDim, typename T>
cudaError_t launch_append(const QuantAppendArgs& a, cudaStream_t stream) {
    constexpr int kRows = 32 / (kDim / 8);
    const int64_t rows = 2ll * a.num_tokens * a.num_kv_heads;
    auto run = [&](auto kernel, int unroll) {
        const int64_t per = static_cast<int64_t>(kWarps) * kRows * unroll, blocks = (rows + per - 1) / per;
        if (blocks > INT32_MAX) return cudaErrorNotSupported;
        return launch_dependent(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, a);
    };
    // Several rows under way in a warp once there are enough for all SMs.
    if (rows >= 152 * kWarps * kRows * 4) return run(quant_append_kernel<kBits, kDim, T, 4>, 4);
    return run(quant_append_kernel<kBits, kDim, T, 1>, 1);
}

// ---------------------------------------------------------------- read back
// A warp takes a packed row, all of its heads, K and V: eight elements a lane, a few
// passes' loads at once.  Its sequence is found in the offsets, which each CTA keeps in
// shared memory.
constexpr int kMaxOffsets = 2048;

template <int kKind>
struct Source;  // bytes of eight elements in the pool
template <> struct Source<kReadF32> { static constexpr int kBytes = 32; };
template <> struct Source<kReadBf16> { static constexpr int kBytes = 16; };
template <> struct Source<kReadE4m3> { static constexpr int kBytes = 8; };
template <> struct Source<kReadQ8> { static constexpr int kBytes = 8; };
template <> struct Source<kReadQ4> { static constexpr int kBytes = 4; };

template <int kKind>
struct Eight {
    uint32_t w[Source<kKind>::kBytes / 4];
    uint32_t p;
    __device__ __forceinline__ void load(const uint8_t* base, const uint32_t* params, int64_t row, int part, int dim) {
        constexpr int n = Source<kKind>::kBytes;
        const uint8_t* src = base + (row * (dim / 8) + part) * n;
        if constexpr (n == 4) {
            asm volatile("ld.global.L1::no_allocate.b32 %0, [%1];\n" : "=r"(w[0]) : "l"(src));
        } else if constexpr (n == 8) {
            asm volatile("ld.global.L1::no_allocate.v2.b32 {%0,%1}, [%2];\n" : "=r"(w[0]), "=r"(w[1]) : "l"(src));
        } else {
#pragma unroll
            for (int i = 0; i < n / 16; ++i) {
                const uint4 v = load16(src + 16 * i);
                w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
            }
        }
        if constexpr (kKind == kReadQ8 || kKind == kReadQ4) p = params[row];
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < Source<kKind>::kBytes / 4; ++i) w[i] = 0u;
        p = 0u;
    }
    __device__ __forceinline__ void store(void* out, int64_t at, float scale) const {
        if constexpr (kKind == kReadF32) {
            uint4* o = reinterpret_cast<uint4*>(static_cast<float*>(out) + at);
            o[0] = make_uint4(w[0], w[1], w[2], w[3]);
            o[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
            uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + at);
            if constexpr (kKind == kReadBf16) {
                o[0] = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
                uint32_t y[4];
                if constexpr (kKind == kReadE4m3) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = e4m3x2_to_float2(static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1))));
                        y[i] = pack_bf16x2_rn(f.x * scale, f.y * scale);
                    }
                } else {
                    const float s = bf16_lo(p), z = bf16_hi(p);
                    uint32_t even, odd, lo, hi;  // bytes of codes 0, 2, 4, 6 and 1, 3, 5, 7
                    if constexpr (kKind == kReadQ4) {
                        even = w[0] & 0x0F0F0F0Fu, odd = (w[0] >> 4) & 0x0F0F0F0Fu;
                    } else {
                        even = __byte_perm(w[0], w[1], 0x6420), odd = __byte_perm(w[0], w[1], 0x7531);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {  // (2^23 + code as a float, and the 2^23 away again)
                        lo = __byte_perm(even, 0x4B000000u, 0x7540 + i);
                        hi = __byte_perm(odd, 0x4B000000u, 0x7540 + i);
                        y[i] = pack_bf16x2_rn(fmaf(s, __uint_as_float(lo) - 8388608.f, z), fmaf(s, __uint_as_float(hi) - 8388608.f, z));
                    }
                }
                o[0] = make_uint4(y[0], y[1], y[2], y[3]);
            }
        }
    }
};

template <int kKind, int kDim>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadArgs a) {
    constexpr int kLanes = kDim / 8, kHeads = 32 / kLanes;      // lanes of a head's row, heads of a pass
    constexpr int kPasses = Source<kKind>::kBytes <= 8 ? 4 : 2;  // passes under way
    __shared__ int32_t offs[kMaxOffsets + 1];
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, part = lane % kLanes;
    const bool kept = a.num_seqs <= kMaxOffsets;
    bool bad = false;  // offsets that do not ascend in [0, num_rows]
    for (int b = tid; b <= a.num_seqs; b += kThreads) {
        const int o = a.offsets[b];
        if (kept) offs[b] = o;
        if (b < a.num_seqs) {
            const int e = a.offsets[b + 1];
            bad |= o < 0 || e < o || e > a.num_rows;
        }
    }
    bad = __syncthreads_or(bad);
    if (bad && blockIdx.x == 0 && tid == 0 && a.err) atomicOr(a.err, PKV_ERRBIT_OFFSETS);
    const int32_t* off = kept ? offs : a.offsets;
    const int bs_mask = (1 << a.block_shift) - 1;

    auto copy = [&](int row, int b, int pos) {
        const int col = pos >> a.block_shift;
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
        for (int h0 = lane / kLanes; h0 < a.num_kv_heads; h0 += kHeads * kPasses) {
            Eight<kKind> k[kPasses], v[kPasses];
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int h = h0 + i * kHeads;
                k[i].clear();
                v[i].clear();
                if (h < a.num_kv_heads && blk >= 0) {
                    const int64_t src = ((static_cast<int64_t>(blk) * a.num_kv_heads + h) << a.block_shift) + (pos & bs_mask);
                    k[i].load(a.k, a.k_params, src, part, kDim);
                    v[i].load(a.v, a.v_params, src, part, kDim);
                }
            }
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int h = h0 + i * kHeads;
                if (h >= a.num_kv_heads) continue;
                const int64_t dst = (static_cast<int64_t>(row) * a.num_kv_heads + h) * kDim + 8 * part;
                k[i].store(a.k_out, dst, a.k_scale);
                v[i].store(a.v_out, dst, a.v_scale);
            }
        }
    };
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + (tid >> 5); r < a.num_rows;
         r += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int row = static_cast<int>(r);
        if (!bad) {
            if (row < off[0] || row >= off[a.num_seqs]) continue;
            int lo = 0, hi = a.num_seqs;  // the last sequence that starts at or before the row
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (off[mid] <= row) lo = mid;
                else hi = mid;
            }
            copy(row, lo, row - off[lo]);
        } else {
            for (int b = 0; b < a.num_seqs; ++b) {
                const int first = off[b], end = off[b + 1];
                if (first >= 0 && end >= first && end <= a.num_rows && row >= first && row < end) copy(row, b, row - first);
            }
        }
    }
}

template <int kKind>
cudaError_t launch_kind(int head_dim, const ReadArgs& a, cudaStream_t stream) {
    const int sms = num_sms() > 0 ? num_sms() : 148;
    const int64_t want = (static_cast<int64_t>(a.num_rows) + kWarps - 1) / kWarps;
    const int blocks = static_cast<int>(want < 8 * sms ? want : 8 * sms);
    if (head_dim == 64) return launch_dependent(read_kernel<kKind, 64>, dim3(blocks), dim3(kThreads), 0, stream, a);
    return launch_dependent(read_kernel<kKind, 128>, dim3(blocks), dim3(kThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_quant_append(int bits, pkv_dtype in, int head_dim, const QuantAppendArgs& a, cudaStream_t stream) {
    auto pick = [&](auto b4, auto b8) { return bits == 4 ? b4(a, stream) : b8(a, stream); };
    if (in == PKV_F32)
        return head_dim == 64 ? pick(launch_append<4, 64, float>, launch_append<8, 64, float>)
                              : pick(launch_append<4, 128, float>, launch_append<8, 128, float>);
    return head_dim == 64 ? pick(launch_append<4, 64, __nv_bfloat16>, launch_append<8, 64, __nv_bfloat16>)
                          : pick(launch_append<4, 128, __nv_bfloat16>, launch_append<8, 128, __nv_bfloat16>);
}

cudaError_t launch_read(ReadKind kind, int head_dim, const ReadArgs& a, cudaStream_t stream) {
    switch (kind) {
        case kReadF32: return launch_kind<kReadF32>(head_dim, a, stream);
        case kReadBf16: return launch_kind<kReadBf16>(head_dim, a, stream);
        case kReadE4m3: return launch_kind<kReadE4m3>(head_dim, a, stream);
        case kReadQ8: return launch_kind<kReadQ8>(head_dim, a, stream);
        case kReadQ4: return launch_kind<kReadQ4>(head_dim, a, stream);
    }
    return cudaErrorNotSupported;
}

}  // namespace pkv
