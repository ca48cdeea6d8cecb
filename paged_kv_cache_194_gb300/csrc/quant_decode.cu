// Decode attention over a quantised cache.  With codes n, pairs (s, z) of a K row
// and (s', z') of a V row,
//     t_j = scale log2(e) (s_j (q . n_j) + z_j sum(q)),
//     out = sum_j 2^t_j (s'_j n'_j + z'_j) / sum_j 2^t_j.
//
// Bound by HBM: a token costs 2 (head_dim bits / 8 + 4) bytes per KV head, and the
// work on its codes is what has to be kept small:
//
//  * Codes are matrix operands as they lie.  A 4- or 8-bit code at the bottom of a
//    16-bit word is a subnormal FP16 number, n 2^-24 exactly, and the tensor core
//    takes those at full rate: one AND makes two operand elements of K (or of V,
//    one byte permute before it), no conversion and no offset to take away again.
//    A nibble that stands four bits higher is 16 times that; for K the query's
//    element is 1/16 of its value there, for V the output row is divided at the end.
//  * S^T = K Q^T and O^T = V^T P^T with mma.m16n8k16: tokens (dimensions) fill the
//    16 rows, up to 8 query heads the 8 columns.  The order of the summed index is
//    free, so each lane takes one contiguous run of its rows' bytes, straight from
//    global memory to registers; P turns around by movmatrix.
//  * Queries enter in FP16 after a power of two that brings the row's largest to
//    [2^14, 2^15): exact for every element within 2^-29 of it.
//  * V's scale goes into the weight's exponent: w_j = 2^(t_j + log2 s'_j - m) with m
//    the running maximum of those exponents, so FP16 weights neither overflow nor
//    lose what matters whatever the scales.  The sum of 2^t_j and the offsets' part
//    sum 2^t_j z'_j have a running maximum of their own and stay in binary32.
//
// Schedule: the 64-token tiles of all (sequence, KV head, part of the group) units
// form one list, cut into equal ranges, one per resident CTA.  In a tile each of a
// CTA's four warps has 16 tokens of one block, and loads its next steps' rows while
// it multiplies; the warps meet at the end of a unit.  A unit cut by ranges leaves
// pieces in the workspace, and the CTA that leaves the last of them joins them, in
// order (the result does not depend on who that is).
#include "device_common.cuh"
#include "quant_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 128, kWarps = 4;
constexpr int kTile = 64, kStep = 16;
constexpr int kCtasPerSm = 4;
constexpr int kMaxCtas = 1024;
constexpr unsigned kAll = 0xFFFFFFFFu;

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2f(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t turn(uint32_t x) {  // 8x8 transpose of 16-bit elements
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <int kWords>
__device__ __forceinline__ void load_words(uint32_t* w, const uint8_t* p) {
    if constexpr (kWords == 1) {
        asm volatile("ld.global.L1::no_allocate.b32 %0, [%1];\n" : "=r"(w[0]) : "l"(p));
    } else if constexpr (kWords == 2) {
        asm volatile("ld.global.L1::no_allocate.v2.b32 {%0,%1}, [%2];\n" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    } else {
        asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];\n"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "l"(p));
    }
}
__device__ __forceinline__ int count_up(int* p) {
    int old;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;\n" : "=r"(old) : "l"(p) : "memory");
    return old;
}

// Shapes of one lane's share.  kBits, kDim: of the cache; kNT: 8-column tiles of query heads.
template <int kBits, int kDim>
struct Share {
    static constexpr int kRow = kDim * kBits / 8;     // bytes of a row
    static constexpr int kKW = kRow / 16;             // words of a K row (a quarter of it)
    static constexpr int kVW = kRow / 32;             // words of a V row (an eighth)
    static constexpr int kKSteps = kDim / 16;         // products of K, and 16-dimension tiles of V
    // dimension of the first element of word w of a K row's share
    __device__ static int k_dim(int t, int w) {
        constexpr int per = 32 / kBits;
        if constexpr (kKW == 8) return (w >> 2) * (kDim / 2) + t * 4 * per + (w & 3) * per;  // two runs of 16 bytes
        return t * kKW * per + w * per;
    }
};

template <int kBits, int kDim>
struct Loaded {  // one step's rows of a lane: K rows g, g + 8; V rows 2t, 2t + 1, 2t + 8, 2t + 9; pairs of g, g + 8
    uint32_t k[2][Share<kBits, kDim>::kKW];
    uint32_t v[4][Share<kBits, kDim>::kVW];
    uint32_t kp[2], vp[2];
};

template <int kBits, int kDim, int kNT>
__global__ void __launch_bounds__(kThreads, kNT == 1 ? kCtasPerSm : 3) quant_decode_kernel(const QuantDecodeArgs a) {
    using S = Share<kBits, kDim>;
    constexpr int kCols = 8 * kNT, kPitch = kDim + 4;
    __shared__ float so[kWarps][kCols][kPitch];
    __shared__ float sm[kWarps][kCols], sl[kWarps][kCols], sz[kWarps][kCols];
    __shared__ long long scan[kThreads];
    __shared__ int last_flag, found[2];
    __shared__ long long found_at;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int gh = a.num_q_heads / a.num_kv_heads, parts = (gh + kCols - 1) / kCols;
    const int per_seq = a.num_kv_heads * parts, bs_mask = (1 << a.block_shift) - 1;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");

    auto len_of = [&](int b) {
        const int L = a.lens[b];
        return L < 0 ? 0 : (L > a.max_len ? a.max_len : L);
    };
    auto tiles_of = [&](int b) { return static_cast<long long>((len_of(b) + kTile - 1) / kTile) * per_seq; };
    // empty sequences' rows, and lengths that cannot be
    for (int b = blockIdx.x; b < a.num_seqs; b += gridDim.x) {
        const int L = a.lens[b];
        if ((L < 0 || L > a.max_len) && tid == 0 && a.err) atomicOr(a.err, PKV_ERRBIT_SEQ_LEN);
        if (L > 0) continue;
        uint32_t* o = reinterpret_cast<uint32_t*>(a.out + static_cast<size_t>(b) * a.num_q_heads * kDim);
        for (int i = tid; i < a.num_q_heads * kDim / 2; i += kThreads) o[i] = 0u;
    }

    // this CTA's range [g0, g1) of the list, and the sequence that tile g0 lies in
    const int run = (a.num_seqs + kThreads - 1) / kThreads;  // sequences per thread
    long long mine = 0;
    for (int i = 0; i < run; ++i)
        if (tid * run + i < a.num_seqs) mine += tiles_of(tid * run + i);
    scan[tid] = mine;
    __syncthreads();
    for (int d = 1; d < kThreads; d <<= 1) {
        const long long x = tid >= d ? scan[tid - d] : 0;
        __syncthreads();
        scan[tid] += x;
        __syncthreads();
    }
    const long long total = scan[kThreads - 1];
    const long long P = total < static_cast<long long>(gridDim.x) ? total : static_cast<long long>(gridDim.x);
    const long long c = blockIdx.x;
    if (c >= P) return;
    const long long g0 = c * total / P, g1 = (c + 1) * total / P;
    if (g0 >= scan[tid] - mine && g0 < scan[tid]) {
        long long at = scan[tid] - mine;
        int b = tid * run;
        for (;; ++b) {
            const long long n = tiles_of(b);
            if (g0 < at + n) break;
            at += n;
        }
        found[0] = b;
        found_at = at;
    }
    __syncthreads();
    int b = found[0], L = len_of(b), nt = (L + kTile - 1) / kTile;
    long long seq_at = found_at;  // list place of the sequence's first tile

    for (long long at = g0; at < g1;) {
        // the segment: tiles [first, end) of unit `unit` of sequence b
        const int unit = static_cast<int>((at - seq_at) / nt), first = static_cast<int>((at - seq_at) % nt);
        const long long unit_at = seq_at + static_cast<long long>(unit) * nt;
        const int end = static_cast<int>(g1 - unit_at < nt ? g1 - unit_at : nt);
        const int h = unit / parts, q0 = (unit % parts) * kCols, rows = min(kCols, gh - q0);
        const int token0 = first * kTile, token1 = min(L, end * kTile);

        // ------------------------------------------------- queries -> operands
        uint32_t qf[kNT][S::kKSteps][2];
        float fs[kNT][2], fz[kNT][2];  // of columns 2t, 2t + 1: factors of s (q . n) and of z
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
            float x[S::kKW][32 / kBits];
            float top = 0.f, sum = 0.f;
            const bool real = 8 * n + g < rows;
            const __nv_bfloat16* qr =
                a.q + (static_cast<size_t>(b) * a.num_q_heads + h * gh + q0 + (real ? 8 * n + g : 0)) * kDim;
#pragma unroll
            for (int w = 0; w < S::kKW; ++w) {
                const uint32_t* src = reinterpret_cast<const uint32_t*>(qr + S::k_dim(t, w));
#pragma unroll
                for (int j = 0; j < 32 / kBits; j += 2) {
                    const uint32_t two = real ? src[j / 2] : 0u;
                    x[w][j] = bf16_lo(two);
                    x[w][j + 1] = bf16_hi(two);
                    top = fmaxf(top, fmaxf(fabsf(x[w][j]), fabsf(x[w][j + 1])));
                }
            }
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
            // 2^e: brings the largest to [2^14, 2^15) (rows of zeros and of what is not finite stay; e at
            // most 126: a smaller row stays smaller)
            const int ex = static_cast<int>(__float_as_uint(top) >> 23);
            const int e = ex == 0 || ex == 255 ? 0 : min(126, 127 + 14 - ex);
            const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
            for (int w = 0; w < S::kKW; ++w)
#pragma unroll
                for (int j = 0; j < 32 / kBits; ++j) {
                    x[w][j] *= up;
                    sum += x[w][j];
                }
            sum += __shfl_xor_sync(kAll, sum, 1);
            sum += __shfl_xor_sync(kAll, sum, 2);
#pragma unroll
            for (int ks = 0; ks < S::kKSteps; ++ks) {
                if constexpr (kBits == 4) {  // nibbles u and u + 4, then the ones above them
                    const int w = ks / 2, u = 2 * (ks & 1);
                    qf[n][ks][0] = half2_of(x[w][u], x[w][u + 4]);
                    qf[n][ks][1] = half2_of(x[w][u + 1] * 0.0625f, x[w][u + 5] * 0.0625f);
                } else {
                    qf[n][ks][0] = half2_of(x[ks][0], x[ks][2]);
                    qf[n][ks][1] = half2_of(x[ks][1], x[ks][3]);
                }
            }
            // (two factors: 2^-e alone may not be a normal number, and the codes' 2^24 comes back here)
            const float down = __uint_as_float(static_cast<uint32_t>(127 - e / 2) << 23);
            const float down2 = __uint_as_float(static_cast<uint32_t>(127 - (e - e / 2)) << 23);
            const float f = a.scale_log2 * down * down2;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float fj = __shfl_sync(kAll, f, (2 * t + j) * 4);
                fs[n][j] = fj * 16777216.f;
                fz[n][j] = fj * __shfl_sync(kAll, sum, (2 * t + j) * 4);
            }
        }

        // ---------------------------------------------------------- the tokens
        // step i of this warp: 16 tokens from token0 + 16 (warp + 4 i)
        const int steps = token0 + kStep * warp < token1 ? (token1 - token0 - kStep * warp + kTile - 1) / kTile : 0;
        const int32_t* table = a.tables + static_cast<size_t>(b) * a.max_blocks;
        // table entries of 32 steps, one a lane, and of the next 32
        auto entries = [&](int i0) {
            const int i = i0 + lane;
            int blk = 0;
            if (i < steps) {
                blk = table[(token0 + kStep * (warp + kWarps * i)) >> a.block_shift];
                if (static_cast<unsigned>(blk) >= static_cast<unsigned>(a.num_blocks)) {
                    if (a.err) atomicOr(a.err, PKV_ERRBIT_BLOCK_ID);
                    blk = 0;  // (the flag marks the output as wrong)
                }
            }
            return blk;
        };
        int win = entries(0), win_next = 0;
        auto load = [&](Loaded<kBits, kDim>& x, int i) {
            if (i >= steps) return;
            if ((i & 31) == 0 && i > 0) win = win_next;
            if ((i & 31) == 16) win_next = entries((i & ~31) + 32);
            const int blk = __shfl_sync(kAll, win, i & 31);
            const int tok = token0 + kStep * (warp + kWarps * i);
            const size_t row = ((static_cast<size_t>(blk) * a.num_kv_heads + h) << a.block_shift) + (tok & bs_mask);
            const uint8_t* k = a.k_codes + row * S::kRow;
            const uint8_t* v = a.v_codes + row * S::kRow;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint8_t* p = k + (g + 8 * r) * S::kRow;
                if constexpr (S::kKW == 8) {
                    load_words<4>(x.k[r], p + 16 * t);
                    load_words<4>(x.k[r] + 4, p + 64 + 16 * t);
                } else {
                    load_words<S::kKW>(x.k[r], p + 4 * S::kKW * t);
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
                load_words<S::kVW>(x.v[r], v + (2 * t + (r & 1) + 8 * (r >> 1)) * S::kRow + 4 * S::kVW * g);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                load_words<1>(&x.kp[r], reinterpret_cast<const uint8_t*>(a.k_params + row + g + 8 * r));
                load_words<1>(&x.vp[r], reinterpret_cast<const uint8_t*>(a.v_params + row + g + 8 * r));
            }
        };

        float o[kNT][S::kKSteps][4];
        float mw[kNT][2], m[kNT][2], l[kNT][2], zs[kNT][2];  // bases of O, and of l and zs
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
#pragma unroll
            for (int i = 0; i < S::kKSteps; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[n][i][j] = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) mw[n][j] = m[n][j] = -INFINITY, l[n][j] = zs[n][j] = 0.f;
        }

        auto use = [&](const Loaded<kBits, kDim>& x, int i) {
            const int left = token1 - (token0 + kStep * (warp + kWarps * i));  // tokens of the step that are there
            // S^T
            float sc[kNT][2][4] = {};
#pragma unroll
            for (int ks = 0; ks < S::kKSteps; ++ks) {
                uint32_t a0, a1, a2, a3;
                if constexpr (kBits == 4) {
                    const uint32_t w0 = x.k[0][ks / 2] >> (8 * (ks & 1)), w1 = x.k[1][ks / 2] >> (8 * (ks & 1));
                    a0 = w0 & 0x000F000Fu, a2 = w0 & 0x00F000F0u;
                    a1 = w1 & 0x000F000Fu, a3 = w1 & 0x00F000F0u;
                } else {
                    a0 = x.k[0][ks] & 0x00FF00FFu, a2 = (x.k[0][ks] >> 8) & 0x00FF00FFu;
                    a1 = x.k[1][ks] & 0x00FF00FFu, a3 = (x.k[1][ks] >> 8) & 0x00FF00FFu;
                }
#pragma unroll
                for (int n = 0; n < kNT; ++n) mma16(sc[n][ks & 1], a0, a1, a2, a3, qf[n][ks][0], qf[n][ks][1]);
            }
            // exponents of the weights: rows g (r = 0) and g + 8 (r = 1)
            float ks_[2], kz[2], lg[2], vz[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const bool there = g + 8 * r < left;
                ks_[r] = bf16_lo(x.kp[r]), kz[r] = bf16_hi(x.kp[r]);
                lg[r] = there ? lg2f(bf16_lo(x.vp[r])) : 0.f;
                vz[r] = there ? bf16_hi(x.vp[r]) : 0.f;
            }
            uint32_t pb[kNT][2];
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
                float y[2][2], e[2][2];
                bool grown = false;
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float dot = sc[n][0][2 * r + j] + sc[n][1][2 * r + j];
                        const float x_ = fmaf(ks_[r], dot * fs[n][j], kz[r] * fz[n][j]);
                        y[r][j] = g + 8 * r < left ? x_ : -INFINITY;
                        e[r][j] = y[r][j] + lg[r];
                        grown |= y[r][j] > m[n][j] + 8.f || e[r][j] > mw[n][j] + 8.f;
                    }
                // the maxima move only when an exponent passes one by 8 (weights stay below 2^8)
                if (__any_sync(kAll, grown)) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float top = fmaxf(y[0][j], y[1][j]), topw = fmaxf(e[0][j], e[1][j]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) {
                            top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
                            topw = fmaxf(topw, __shfl_xor_sync(kAll, topw, d));
                        }
                        top = fmaxf(top, m[n][j]);
                        topw = fmaxf(topw, mw[n][j]);
                        const float f = m[n][j] == -INFINITY ? 0.f : ex2f(m[n][j] - top);
                        const float fw = mw[n][j] == -INFINITY ? 0.f : ex2f(mw[n][j] - topw);
                        m[n][j] = top;
                        mw[n][j] = topw;
                        l[n][j] *= f;
                        zs[n][j] *= f;
#pragma unroll
                        for (int k = 0; k < S::kKSteps; ++k) {
                            o[n][k][j] *= fw;
                            o[n][k][2 + j] *= fw;
                        }
                    }
                }
                float w[2][2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float base = m[n][j] == -INFINITY ? 0.f : m[n][j], basew = mw[n][j] == -INFINITY ? 0.f : mw[n][j];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        w[r][j] = ex2f(e[r][j] - basew);
                        const float p = ex2f(y[r][j] - base);
                        l[n][j] += p;
                        zs[n][j] = fmaf(p, vz[r], zs[n][j]);
                    }
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) pb[n][r] = turn(half2_of(w[r][0], w[r][1]));
            }
            // O^T
#pragma unroll
            for (int wi = 0; wi < S::kVW; ++wi) {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const uint32_t sel = hf ? 0x7632u : 0x5410u;
                    const uint32_t x0 = __byte_perm(x.v[0][wi], x.v[1][wi], sel), x1 = __byte_perm(x.v[2][wi], x.v[3][wi], sel);
                    if constexpr (kBits == 4) {
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const uint32_t y0 = x0 >> (8 * u), y1 = x1 >> (8 * u);
#pragma unroll
                            for (int n = 0; n < kNT; ++n)
                                mma16(o[n][4 * wi + 2 * hf + u], y0 & 0x000F000Fu, y0 & 0x00F000F0u, y1 & 0x000F000Fu,
                                      y1 & 0x00F000F0u, pb[n][0], pb[n][1]);
                        }
                    } else {
#pragma unroll
                        for (int n = 0; n < kNT; ++n)
                            mma16(o[n][2 * wi + hf], x0 & 0x00FF00FFu, (x0 >> 8) & 0x00FF00FFu, x1 & 0x00FF00FFu,
                                  (x1 >> 8) & 0x00FF00FFu, pb[n][0], pb[n][1]);
                    }
                }
            }
        };

        if constexpr (kBits == 4) {  // two steps under way
            Loaded<kBits, kDim> s0, s1;
            load(s0, 0);
            load(s1, 1);
            for (int i = 0; i < steps; i += 2) {
                use(s0, i);
                load(s0, i + 2);
                if (i + 1 < steps) {
                    use(s1, i + 1);
                    load(s1, i + 3);
                }
            }
        } else {
            Loaded<kBits, kDim> s0, s1;
            load(s0, 0);
            for (int i = 0; i < steps; i += 2) {
                load(s1, i + 1);
                use(s0, i);
                if (i + 1 < steps) {
                    load(s0, i + 2);
                    use(s1, i + 1);
                }
            }
        }

        // ------------------------------------------------ the warps' sums meet
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    l[n][j] += __shfl_xor_sync(kAll, l[n][j], d);
                    zs[n][j] += __shfl_xor_sync(kAll, zs[n][j], d);
                }
                const int col = 8 * n + 2 * t + j;
                // O in the base of l, the codes' 2^24 (and the upper nibbles' 2^-4) taken out
                const float up = 16777216.f * (mw[n][j] == -INFINITY ? 0.f : ex2f(mw[n][j] - m[n][j]));
                if (g == 0) {
                    sm[warp][col] = m[n][j];
                    sl[warp][col] = l[n][j];
                    sz[warp][col] = zs[n][j];
                }
                // element (dimension g (kDim / 8) + x) of column col at [x][g]: all lanes in different banks
#pragma unroll
                for (int i = 0; i < S::kKSteps; ++i) {
                    so[warp][col][(2 * i) * 8 + g] = o[n][i][j] * up;
                    so[warp][col][(2 * i + 1) * 8 + g] = o[n][i][2 + j] * (kBits == 4 ? 0.0625f * up : up);
                }
            }
        __syncthreads();
        const bool whole = first == 0 && end == nt;
        const int slot = 2 * static_cast<int>(c) + (at == g0 ? 0 : 1);
        const size_t out0 = static_cast<size_t>(b) * a.num_q_heads + h * gh + q0;
        for (int i = tid; i < rows * kDim; i += kThreads) {
            const int r = i / kDim, d = i % kDim, at_ = (d % (kDim / 8)) * 8 + d / (kDim / 8);
            float M = sm[0][r];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sm[w][r]);
            float lw = 0.f, ow = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = sm[w][r] == -INFINITY && sl[w][r] == 0.f ? 0.f : ex2f(sm[w][r] - (M == -INFINITY ? 0.f : M));
                lw += f * sl[w][r];
                ow += f * (so[w][r][at_] + sz[w][r]);
            }
            if (whole) {
                a.out[(out0 + r) * kDim + d] = __float2bfloat16_rn(__fdiv_rn(ow, lw));
            } else {
                a.part_o[(static_cast<size_t>(slot) * kCols + r) * kDim + d] = ow;
                if (d == 0) {
                    a.part_ml[2 * (static_cast<size_t>(slot) * kCols + r)] = M;
                    a.part_ml[2 * (static_cast<size_t>(slot) * kCols + r) + 1] = lw;
                }
            }
        }
        if (!whole) {
            // the unit's pieces: CTAs c0 .. c1, each one piece
            const long long c0 = ((unit_at + 1) * P - 1) / total, c1 = ((unit_at + nt) * P - 1) / total;
            int* counter = a.counters + static_cast<size_t>(b) * per_seq + unit;
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const int pieces = static_cast<int>(c1 - c0 + 1);
                last_flag = count_up(counter) == pieces - 1;
                if (last_flag) *counter = 0;
            }
            __syncthreads();
            if (last_flag) {
                __threadfence();
                const int extra = unit_at > c0 * total / P ? 1 : 0;  // the first piece does not begin its CTA's range
                const int n = static_cast<int>(c1 - c0 + 1);
                auto slot_of = [&](int i) { return static_cast<size_t>(2 * (c0 + i) + (i == 0 ? extra : 0)); };
                for (int r = warp; r < rows; r += kWarps) {
                    float M = -INFINITY;
                    for (int i = lane; i < n; i += 32) M = fmaxf(M, __ldcg(a.part_ml + 2 * (slot_of(i) * kCols + r)));
                    M = warp_max(M);
                    const float base = M == -INFINITY ? 0.f : M;
                    constexpr int kPer = kDim / 32;
                    float acc[kPer] = {}, lw = 0.f;
                    for (int i0 = 0; i0 < n; i0 += 32) {
                        float f = 0.f, lf = 0.f;
                        if (i0 + lane < n) {
                            const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + slot_of(i0 + lane) * kCols + r);
                            f = ex2f(ml.x - base);
                            lf = f * ml.y;
                        }
                        lw += warp_sum(lf);
                        const int k1 = min(32, n - i0);
#pragma unroll 8
                        for (int k = 0; k < k1; ++k) {
                            const float fk = __shfl_sync(kAll, f, k);
                            const float* src = a.part_o + (slot_of(i0 + k) * kCols + r) * kDim + kPer * lane;
                            if constexpr (kPer == 4) {
                                const float4 y = __ldcg(reinterpret_cast<const float4*>(src));
                                acc[0] += fk * y.x, acc[1] += fk * y.y, acc[2] += fk * y.z, acc[3] += fk * y.w;
                            } else {
                                const float2 y = __ldcg(reinterpret_cast<const float2*>(src));
                                acc[0] += fk * y.x, acc[1] += fk * y.y;
                            }
                        }
                    }
                    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + (out0 + r) * kDim + kPer * lane);
#pragma unroll
                    for (int k = 0; k < kPer; k += 2)
                        dst[k / 2] = pack_bf16x2_rn(__fdiv_rn(acc[k], lw), __fdiv_rn(acc[k + 1], lw));
                }
            }
        }
        __syncthreads();  // (the shared sums are read)
        at = unit_at + end;
        if (at < g1 && unit == per_seq - 1) {  // the next sequence that has tokens
            seq_at += static_cast<long long>(nt) * per_seq;
            do {
                ++b;
                L = len_of(b);
            } while (L == 0);
            nt = (L + kTile - 1) / kTile;
        }
    }
}

int columns(int gh) { return gh <= 8 ? 8 : 16; }

}  // namespace

size_t quant_decode_workspace(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, uint8_t* base,
                              QuantDecodeArgs* a) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const int gh = num_q_heads / num_kv_heads, cols = columns(gh), parts = (gh + cols - 1) / cols;
    const size_t counters = up(static_cast<size_t>(num_seqs) * num_kv_heads * parts * sizeof(int32_t));
    const size_t ml = up(static_cast<size_t>(kMaxCtas) * 2 * cols * 2 * sizeof(float));
    if (a) {
        a->counters = reinterpret_cast<int32_t*>(base);
        a->part_ml = reinterpret_cast<float*>(base + counters);
        a->part_o = reinterpret_cast<float*>(base + counters + ml);
    }
    return counters + ml + static_cast<size_t>(kMaxCtas) * 2 * cols * head_dim * sizeof(float);
}

cudaError_t launch_quant_decode(int bits, int head_dim, const QuantDecodeArgs& a, cudaStream_t stream) {
    const int cols = columns(a.num_q_heads / a.num_kv_heads);
    const int sms = num_sms() > 0 ? num_sms() : 148;
    const int ctas = min(kMaxCtas, sms * (cols == 8 ? kCtasPerSm : 3));
    auto run = [&](auto kernel) {
        return launch_dependent(kernel, dim3(ctas), dim3(kThreads), 0, stream, a);
    };
    auto pick = [&](auto narrow, auto wide) { return cols == 8 ? run(narrow) : run(wide); };
    if (bits == 4)
        return head_dim == 64 ? pick(quant_decode_kernel<4, 64, 1>, quant_decode_kernel<4, 64, 2>)
                              : pick(quant_decode_kernel<4, 128, 1>, quant_decode_kernel<4, 128, 2>);
    return head_dim == 64 ? pick(quant_decode_kernel<8, 64, 1>, quant_decode_kernel<8, 64, 2>)
                          : pick(quant_decode_kernel<8, 128, 1>, quant_decode_kernel<8, 128, 2>);
}

}  // namespace pkv
