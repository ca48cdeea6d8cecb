// The quantised cache's rows: written with a scale and an offset of their own,
// and read back through block tables as the values that they stand for.
//
// Both are one pass over memory: HBM bounds them, and instructions come next (at the copy
// rate an SM has about 14 for each element of a lane).  On a GB300, whose copies run at 6.79
// TB/s, with 8 heads of 128: FP32 rows of 36 thousand tokens to 4 bits 51 us or 6.5 TB/s (72 us
// with eight elements a lane and one FP32 an instruction); the same rows from 4 bits to BF16 32
// us or 5.8 TB/s (33 with stores that stay in the L2); 41 thousand rows of E4M3 to BF16 41 us or
// 6.2 TB/s.  Calls of a few rows take 1.7 and 4.7 us: the launch, and four
// dependent reads (offsets, table, codes) for the read-back.
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
__device__ __forceinline__ uint4 load16(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// pairs of FP32 numbers, one instruction for both
__device__ __forceinline__ uint64_t pair(float a, float b) {
    return static_cast<uint64_t>(__float_as_uint(b)) << 32 | __float_as_uint(a);
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2_down(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rm.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// (a product of pairs would be fused with a sum that follows, which the format rounds by itself)
__device__ __forceinline__ uint64_t mul_each(uint64_t a, float b) {
    return pair(__fmul_rn(__uint_as_float(static_cast<uint32_t>(a)), b), __fmul_rn(__uint_as_float(static_cast<uint32_t>(a >> 32)), b));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// ------------------------------------------------------------------- append
// Sixteen elements a lane, eight from each half of the row, so that kDim / 16 lanes have
// a row; kUnroll groups of rows under way in a warp.  A row's lanes share its minimum and
// maximum by shuffles: one of both together with BF16 rows, as the pair (min, -max).
template <int kBits, int kDim, typename T, int kUnroll>
__global__ void __launch_bounds__(kThreads) quant_append_kernel(const QuantAppendArgs a) {
    constexpr int kLanes = kDim / 16, kRows = 32 / kLanes;  // lanes of a row, rows of a warp
    constexpr bool kWide = sizeof(T) == 4;
    constexpr int kHalf = kWide ? 2 : 1;  // loads for a half's eight elements
    constexpr float N = (1 << kBits) - 1;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int lane = threadIdx.x & 31, part = lane % kLanes;
    const int per_token = 2 * a.num_kv_heads;  // rows: K heads, then V heads of each token
    const int64_t total = static_cast<int64_t>(a.num_tokens) * per_token;
    int64_t r = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * (kRows * kUnroll) + lane / kLanes;
    // (a 32-bit division where it will do)
    int t = static_cast<int>(total <= INT32_MAX ? static_cast<uint32_t>(r) / static_cast<uint32_t>(per_token) : r / per_token);
    int j = static_cast<int>(r - static_cast<int64_t>(t) * per_token);
    uint4 raw[kUnroll][2 * kHalf];
    int64_t slot[kUnroll];
    int head[kUnroll];
    bool is_v[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const bool there = r < total;
        is_v[i] = j >= a.num_kv_heads;
        head[i] = is_v[i] ? j - a.num_kv_heads : j;
        slot[i] = -1;
        if (there) {
            slot[i] = a.slots[t];
            const T* x = static_cast<const T*>(is_v[i] ? a.v : a.k) + t * (is_v[i] ? a.v_stride : a.k_stride) +
                         head[i] * kDim + 8 * part;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int u = 0; u < kHalf; ++u) raw[i][h * kHalf + u] = load16(x + h * (kDim / 2) + 4 * u);
        } else {
#pragma unroll
            for (int u = 0; u < 2 * kHalf; ++u) raw[i][u] = make_uint4(0u, 0u, 0u, 0u);
        }
        r += kRows;
        for (j += kRows; j >= per_token; j -= per_token) ++t;
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        float lo, hi;
        uint64_t x[8];  // the sixteen elements
        if constexpr (kWide) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(raw[i]);
            lo = hi = __uint_as_float(w[0]);
#pragma unroll
            for (int k = 1; k < 16; ++k) lo = min_nan(lo, __uint_as_float(w[k])), hi = max_nan(hi, __uint_as_float(w[k]));
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = pair(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
#pragma unroll
            for (int d = kLanes / 2; d > 0; d >>= 1) {
                lo = min_nan(lo, __shfl_xor_sync(kAll, lo, d));
                hi = max_nan(hi, __shfl_xor_sync(kAll, hi, d));
            }
        } else {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(raw[i]);
            const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(raw[i]);
            __nv_bfloat162 mn = h[0], mx = h[0];
#pragma unroll
            for (int k = 1; k < 8; ++k) mn = __hmin2_nan(mn, h[k]), mx = __hmax2_nan(mx, h[k]);
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
            for (int k = 0; k < 8; ++k) x[k] = pair(bf16_lo(w[k]), bf16_hi(w[k]));
        }
        if (slot[i] == -1) continue;
        if (slot[i] < 0 || slot[i] >= a.num_slots) {
            if (a.err && part == 0) atomicOr(a.err, PKV_ERRBIT_SLOT);
            continue;
        }
        lo = __fadd_rn(lo, 0.f);  // (no negative zero)
        uint32_t zb = __float_as_uint(lo) & 0xFFFF0000u;
        if (kWide && lo < 0.f && zb != __float_as_uint(lo)) zb += 0x10000u;  // (BF16 rows have their minimum in BF16)
        const float z = __uint_as_float(zb), range = __fsub_rn(hi, z);
        const bool bad = !(range <= 3.402823466e38f);  // an infinity or a NaN in the row, or a range that is not finite
        const float s0 = fmaxf(fmaxf(__fdiv_rn(range, N), fabsf(z) * 0x1p-16f), 0x1p-100f);
        const uint32_t sb = (__float_as_uint(s0) + 0xFFFFu) & 0xFFFF0000u;
        const float inv = __fmul_rn(__frcp_rn(__uint_as_float(sb)), 1.f + 0x1p-21f);
        const uint64_t z2 = pair(-z, -z), half2 = pair(0.5f, 0.5f), int2 = pair(8388608.f, 8388608.f);
        // floor((x - z) inv + 1/2): in the low bits of 2^23 + it
        uint32_t n[16];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint64_t y = add2_down(add2(mul_each(add2(x[k], z2), inv), half2), int2);
            n[2 * k] = static_cast<uint32_t>(y), n[2 * k + 1] = static_cast<uint32_t>(y >> 32);
        }
        const int in = static_cast<int>(slot[i]) & ((1 << a.block_shift) - 1);
        const int64_t at = (((slot[i] >> a.block_shift) * a.num_kv_heads + head[i]) << a.block_shift) + in;
        uint8_t* codes = (is_v[i] ? a.v_codes : a.k_codes) + at * (kDim * kBits / 8) + part * kBits;
#pragma unroll
        for (int h = 0; h < 2; ++h, codes += kDim * kBits / 16) {
            const uint32_t* m = n + 8 * h;
            if constexpr (kBits == 4) {
                // (two codes of a byte's: the upper one's in place by a shift and an or)
                const uint32_t even = __byte_perm(__byte_perm(m[0], m[2], 0x0040), __byte_perm(m[4], m[6], 0x0040), 0x5410);
                const uint32_t odd = __byte_perm(__byte_perm(m[1], m[3], 0x0040), __byte_perm(m[5], m[7], 0x0040), 0x5410);
                *reinterpret_cast<uint32_t*>(codes) = bad ? 0u : even | odd << 4;
            } else {
                uint2 c;
                c.x = __byte_perm(__byte_perm(m[0], m[1], 0x0040), __byte_perm(m[2], m[3], 0x0040), 0x5410);
                c.y = __byte_perm(__byte_perm(m[4], m[5], 0x0040), __byte_perm(m[6], m[7], 0x0040), 0x5410);
                *reinterpret_cast<uint2*>(codes) = bad ? make_uint2(0u, 0u) : c;
            }
        }
        if (part == 0) (is_v[i] ? a.v_params : a.k_params)[at] = bad ? 0x7FC07FC0u : (sb >> 16 | zb);
    }
}

template <int kBits, int kDim, typename T>
cudaError_t launch_append(const QuantAppendArgs& a, cudaStream_t stream) {
    constexpr int kRows = 32 / (kDim / 16);
    const int64_t rows = 2ll * a.num_tokens * a.num_kv_heads;
    auto run = [&](auto kernel, int unroll) {
        const int64_t per = static_cast<int64_t>(kWarps) * kRows * unroll, blocks = (rows + per - 1) / per;
        if (blocks > INT32_MAX) return cudaErrorNotSupported;
        return launch_dependent(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, a);
    };
    // Several rows under way in a warp once there are enough for all SMs.
    const int64_t sms = num_sms() > 0 ? num_sms() : 148;
    if (rows >= sms * kWarps * kRows * 4) return run(quant_append_kernel<kBits, kDim, T, 2>, 2);
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
    __device__ __forceinline__ void load(const uint8_t* src, const uint32_t* params) {
        constexpr int n = Source<kKind>::kBytes;
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
        if constexpr (kKind == kReadQ8 || kKind == kReadQ4) p = *params;
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < Source<kKind>::kBytes / 4; ++i) w[i] = 0u;
        p = 0u;
    }
    __device__ __forceinline__ void store(uint8_t* out, float scale) const {
        if constexpr (kKind == kReadF32) {
            uint4* o = reinterpret_cast<uint4*>(out);
            __stcs(o + 0, make_uint4(w[0], w[1], w[2], w[3]));
            __stcs(o + 1, make_uint4(w[4], w[5], w[6], w[7]));
        } else {
            uint4* o = reinterpret_cast<uint4*>(out);
            if constexpr (kKind == kReadBf16) {
                __stcs(o + 0, make_uint4(w[0], w[1], w[2], w[3]));
            } else {
                uint32_t y[4];
                if constexpr (kKind == kReadE4m3) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = e4m3x2_to_float2(static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1))));
                        y[i] = pack_bf16x2_rn(f.x * scale, f.y * scale);
                    }
                } else {
                    const uint64_t s2 = pair(bf16_lo(p), bf16_lo(p)), z2 = pair(bf16_hi(p), bf16_hi(p));
                    uint32_t even, odd;  // bytes of codes 0, 2, 4, 6 and 1, 3, 5, 7
                    if constexpr (kKind == kReadQ4) {
                        even = w[0] & 0x0F0F0F0Fu, odd = (w[0] >> 4) & 0x0F0F0F0Fu;
                    } else {
                        even = __byte_perm(w[0], w[1], 0x6420), odd = __byte_perm(w[0], w[1], 0x7531);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {  // (2^23 + code as a float, and the 2^23 away again)
                        const uint64_t n = pair(__uint_as_float(__byte_perm(even, 0x4B000000u, 0x7540 + i)),
                                                __uint_as_float(__byte_perm(odd, 0x4B000000u, 0x7540 + i)));
                        const uint64_t f = fma2(s2, add2(n, pair(-8388608.f, -8388608.f)), z2);
                        y[i] = pack_bf16x2_rn(__uint_as_float(static_cast<uint32_t>(f)), __uint_as_float(static_cast<uint32_t>(f >> 32)));
                    }
                }
                __stcs(o + 0, make_uint4(y[0], y[1], y[2], y[3]));
            }
        }
    }
};

template <int kKind, int kDim>
__global__ void __launch_bounds__(kThreads, 4) read_kernel(const ReadArgs a) {
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

    // the row's block, or -1
    auto block_of = [&](int b, int pos) -> int {
        const int col = pos >> a.block_shift;
        if (col >= a.max_blocks) {
            if (a.err && lane == 0) atomicOr(a.err, PKV_ERRBIT_SEQ_LEN);
            return -1;
        }
        const int blk = a.tables[static_cast<int64_t>(b) * a.max_blocks + col];
        if (static_cast<unsigned>(blk) < static_cast<unsigned>(a.num_blocks)) return blk;
        if (a.err && lane == 0) atomicOr(a.err, PKV_ERRBIT_BLOCK_ID);
        return -1;
    };
    constexpr int kIn = Source<kKind>::kBytes, kOut = kKind == kReadF32 ? 32 : 16;  // bytes of eight elements
    const int h0 = lane / kLanes;
    const int64_t src_step = static_cast<int64_t>(kHeads << a.block_shift) * (kLanes * kIn);
    auto copy = [&](int row, int blk, int pos) {
        const int64_t src = ((static_cast<int64_t>(blk) * a.num_kv_heads + h0) << a.block_shift) + (pos & bs_mask);
        const int64_t from = (src * kLanes + part) * kIn;
        const uint8_t *kp = a.k + from, *vp = a.v + from;
        const uint32_t *ks = a.k_params + src, *vs = a.v_params + src;
        const int64_t to = ((static_cast<int64_t>(row) * a.num_kv_heads + h0) * kLanes + part) * kOut;
        uint8_t *ko = static_cast<uint8_t*>(a.k_out) + to, *vo = static_cast<uint8_t*>(a.v_out) + to;
        for (int h = h0; h < a.num_kv_heads; h += kHeads * kPasses) {
            Eight<kKind> k[kPasses], v[kPasses];
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                k[i].clear();
                v[i].clear();
                if (h + i * kHeads < a.num_kv_heads && blk >= 0) {
                    k[i].load(kp, ks);
                    v[i].load(vp, vs);
                }
                kp += src_step, vp += src_step;
                ks += kHeads << a.block_shift, vs += kHeads << a.block_shift;
            }
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                if (h + i * kHeads < a.num_kv_heads) {
                    k[i].store(ko, a.k_scale);
                    v[i].store(vo, a.v_scale);
                }
                ko += kHeads * kLanes * kOut, vo += kHeads * kLanes * kOut;
            }
        }
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
    int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + (tid >> 5);
    if (!bad) {
        // a row's block is looked up while the row before is under way
        const int64_t end = min(static_cast<int64_t>(a.num_rows), static_cast<int64_t>(off[a.num_seqs]));
        const int start = off[0];
        if (r < start) r += (start - r + step - 1) / step * step;
        int blk = 0, pos = 0;
        auto find = [&](int row) {
            int lo = 0, hi = a.num_seqs;  // the last sequence that starts at or before the row
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (off[mid] <= row) lo = mid;
                else hi = mid;
            }
            pos = row - off[lo];
            blk = block_of(lo, pos);
        };
        if (r < end) find(static_cast<int>(r));
        while (r < end) {
            const int row = static_cast<int>(r), at = pos, from = blk;
            r += step;
            if (r < end) find(static_cast<int>(r));
            copy(row, from, at);
        }
    } else {
        for (; r < a.num_rows; r += step) {
            const int row = static_cast<int>(r);
            for (int b = 0; b < a.num_seqs; ++b) {
                const int first = off[b], end = off[b + 1];
                if (first >= 0 && end >= first && end <= a.num_rows && row >= first && row < end)
                    copy(row, block_of(b, row - first), row - first);
            }
        }
    }
}

template <int kKind>
cudaError_t launch_kind(int head_dim, const ReadArgs& a, cudaStream_t stream) {
    const int sms = num_sms() > 0 ? num_sms() : 148;
    const int64_t want = (static_cast<int64_t>(a.num_rows) + kWarps - 1) / kWarps;
    // A warp's next row is looked up while one is under way, which pays for codes (us for 41 thousand rows, 8 CTAs an SM / 64:
    // 4 bits 37.3 / 38.3, with head_dim 64 25.3 / 27.8; 8 bits 43.4 / 41.8, 27.8 / 29.0); wider rows come faster from many
    // warps of few rows (E4M3 43.3 / 40.7, head_dim 64 26.5 / 27.5; BF16 54.8 / 51.6; 20 thousand of FP32 58.1 / 53.9).
    const int most = (kKind == kReadQ4 || kKind == kReadQ8 ? 8 : 64) * sms;
    const int blocks = static_cast<int>(want < most ? want : most);
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
