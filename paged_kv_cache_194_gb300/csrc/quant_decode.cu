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
//    free, so each lane takes one contiguous run of its rows' bytes; P turns around by
//    movmatrix.
//  * Queries enter in FP16 after a power of two that brings the row's largest to
//    [2^14, 2^15): exact for every element within 2^-31 of it (2^-27 for those that
//    meet upper nibbles, as 1/16 of themselves); what is less is rounded by 2^-25.
//  * V's scale goes into the weight's exponent: w_j = 2^((t_j - m) + log2 s'_j - lift)
//    with m the running maximum of the t_j, m + lift + 7 that of t_j + log2 s'_j: FP16
//    weights (the type that codes are multiplied with) of up to 2^7, 2^15 while the
//    maxima lag by 8, which are rounded by 2^-11 and, below 2^-21 of the largest, by
//    2^-32 of it.  The sum of 2^(t_j - m) and the offsets' part sum 2^(t_j - m) z'_j
//    stay in binary32.
//
// Schedule: the 64-token tiles of all (sequence, KV head, part of the group) units
// form one list, in which a unit weighs kUnitCost tiles beside its own; it is cut into
// equal ranges, one per resident CTA.  In a tile each of a CTA's four warps has 16
// tokens of one block; the rows of its next few steps, of the next unit's first ones at
// a unit's end, are on their way into a ring of its own in shared memory while it
// multiplies.  The warps meet at the end of a unit.
// A unit cut by ranges leaves pieces in the workspace, and the CTA that leaves the last
// of them joins them, in order (the result does not depend on who that is).  Few short
// units are a CTA's own each, many short ones a warp's.
//
// Measured with 32 query heads on 8 of 128, rows read from HBM at up to 6.79 TB/s: 55
// sequences of 8192 tokens of 8 bits 162 us (5.9 TB/s); two of 130 thousand of 4 bits 59 us
// (4.8 TB/s); 64 of 128 to 4096 of 4 bits 42 us (3.5 TB/s); four of up to 512 8.4 us.  Of 4-bit
// rows neither memory nor the issue slots are full: 250 instructions for 16 tokens of a warp are
// issued in 51 % of the cycles (two long ones; 47 % of the mixed batch's) by the three warps of a
// scheduler that registers leave room for, each of which waits for its own results, and at a
// unit's end for the next one's rows; a call's start, until rows flow, takes 3 to 4 us, and
// writing and joining pieces at its end 4 to 5.
#include <type_traits>

#include "device_common.cuh"
#include "quant_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 128, kWarps = 4;
constexpr int kTile = 64, kStep = 16;
// (us for 64 sequences of 128 to 4096 tokens with 4, 6, 10: 42.5, 41.6, 42.5; of 8 bits 61.4, 61.0, 61.3; head_dim 64 32.0,
// 32.1, 32.0; 16 heads per KV head 33.9, 32.6, 33.6; 256 of 256 to 512, cut: 45.2, 44.9, 44.4)
constexpr int kUnitCost = 6;
constexpr int kMaxCtas = 1024;
// CTAs per SM, and steps whose rows are under way in a warp (pair: taken two at a time).  HBM answers after 2.5 to 3 us
// under load, so an SM wants 130 to 150 KB on their way.
constexpr int ctas_per_sm(int bits, int dim, int nt) {
    if (dim == 64) return nt == 1 ? 4 : 3;
    return nt == 1 && bits == 4 ? 3 : 2;
}
constexpr int depth_of(int bits, int dim, int nt) {
    if (dim == 64) return bits == 4 ? 10 : 6;
    return nt == 2 && bits == 4 ? 12 : 6;
}
constexpr float kNone = -3.402823466e38f;  // a maximum of nothing: finite, so that nothing minus nothing is 0
constexpr float kHigh = 7.f;  // log2 of the largest weight: FP16's small numbers then reach far below it
constexpr float kLag = 8.f;   // that the maxima may be behind
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
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (kWords == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x, w[1] = v.y;
    } else {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
}
template <int kWords>
__device__ __forceinline__ void load_global(uint32_t* w, const void* p) {
    if constexpr (kWords == 2) {
        asm volatile("ld.global.v2.b32 {%0,%1}, [%2];\n" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    } else {
        asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];\n" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
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

// A warp's 16 rows in shared memory: K, V, then the pairs of both.  Rows and their 16-byte chunks are placed so that
// the lanes of a load below meet no bank twice (head_dim 128): K row r at place r, its chunks of an odd 128-byte
// row exchanged by halves; V's even rows first, chunks exchanged by row.
template <int kBits, int kDim>
struct Stage {
    static constexpr int kRow = kDim * kBits / 8, kChunks = kRow / 16;
    static constexpr int kV = 16 * kRow, kPairs = 32 * kRow, kBytes = kPairs + 128;
    __device__ static int k_at(int row, int chunk) { return row * kRow + ((kChunks == 8 ? chunk ^ ((row & 1) << 2) : chunk) << 4); }
    __device__ static int v_at(int row, int chunk) {
        if constexpr (kChunks == 8) return kV + row * kRow + ((chunk ^ (row & 6)) << 4);
        const int place = (row >> 1) | ((row & 1) << 3);
        if constexpr (kChunks == 4) return kV + place * kRow + ((chunk ^ (place & 2)) << 4);
        return kV + place * kRow + (chunk << 4);
    }
};

// A segment: tiles [first, end) of a unit, tokens [token0, token1) of its sequence.
struct Seg {
    int b, nt, unit, first, end, token0, token1;
    long long at;  // list place of the unit, whose tiles lie behind its own cost
};

template <int kBits, int kDim, int kNT, bool kPair>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(kBits, kDim, kNT)) quant_decode_kernel(const QuantDecodeArgs a) {
    using S = Share<kBits, kDim>;
    static_assert(!kPair || kNT == 1);
    constexpr int kCols = 8 * kNT, kSumCols = kPair ? 4 : kCols, kPitch = kDim + 4;
    constexpr int kDepth = depth_of(kBits, kDim, kNT), kNS = kPair ? 2 : 1;  // (steps at a time)
    using St = Stage<kBits, kDim>;
    extern __shared__ __align__(16) uint8_t dynamic[];
    constexpr int kRing = kDepth * St::kBytes;
    // a warp's sums for the others, over the last places of its ring: so(w)[column][kPitch]
    constexpr int kSumBytes = static_cast<int>(sizeof(float)) * kSumCols * kPitch;
    constexpr int kSumPlaces = (kSumBytes + St::kBytes - 1) / St::kBytes, kEarly = kDepth - kSumPlaces;
    static_assert(kEarly >= kNS);
    uint8_t* ring = dynamic + (threadIdx.x >> 5) * kRing;
    auto so = [&](int w) { return reinterpret_cast<float (*)[kPitch]>(dynamic + w * kRing + kEarly * St::kBytes); };
    __shared__ float sm[kWarps][kCols], sl[kWarps][kCols], sz[kWarps][kCols];
    __shared__ long long scan[kWarps];
    __shared__ int lengths[kWarps];
    __shared__ int last_flag[2], found[kWarps];
    __shared__ long long found_at[kWarps];
    __shared__ Seg split[2];  // this CTA's pieces of units that others share: at its range's start, and at its end
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int gh = a.num_q_heads / a.num_kv_heads, parts = (gh + kCols - 1) / kCols;
    const int per_seq = a.num_kv_heads * parts, bs_mask = (1 << a.block_shift) - 1;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");

    auto len_of = [&](int b) {
        const int L = a.lens[b];
        return L < 0 ? 0 : (L > a.max_len ? a.max_len : L);
    };
    // empty sequences' rows, and lengths that cannot be
    for (int b = blockIdx.x; b < a.num_seqs; b += gridDim.x) {
        const int L = a.lens[b];
        if ((L < 0 || L > a.max_len) && tid == 0 && a.err) atomicOr(a.err, PKV_ERRBIT_SEQ_LEN);
        if (L > 0) continue;
        uint32_t* o = reinterpret_cast<uint32_t*>(a.out + static_cast<size_t>(b) * a.num_q_heads * kDim);
        for (int i = tid; i < a.num_q_heads * kDim / 2; i += kThreads) o[i] = 0u;
    }

    // this CTA's range [g0, g1) of the list, and the sequence that it begins in
    const int run = (a.num_seqs + kThreads - 1) / kThreads;  // sequences per thread
    long long mine = 0;   // cost of this thread's
    int some = 0, most = 0;  // how many have tokens, and the most tiles of one
    for (int i = 0; i < run; ++i)
        if (tid * run + i < a.num_seqs) {
            const int nt = (len_of(tid * run + i) + kTile - 1) / kTile;
            if (nt > 0) mine += nt + kUnitCost, ++some;
            most = max(most, nt);
        }
    // With no more units than CTAs, and none long, every unit is a CTA's of its own: joining its pieces would take longer
    // than they save.  (us whole / cut, 32 heads: 8.2 / 10.2 for one sequence of 512 tokens, 11.6 / 10.5 for one of 1024;
    // 12.3 / 20.6 and 17.9 / 24.9 for fifty; thirty of 512 11.0 / 14.4, of 8 bits 10.8 / 19.2, head_dim 64 10.3 / 12.7; eight
    // of 900 15.1 / 12.4, 13.7 / 12.7, 13.4 / 11.0.  16 heads per KV head, four times the sequences: 14.0 / 33.3, and 18.4 /
    // 20.7 for 900, where the rule cuts.)
    most = __reduce_max_sync(kAll, most);
    long long incl = mine | static_cast<long long>(some) << 40;  // (both sums at once: costs stay below 2^40)
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long x = __shfl_up_sync(kAll, incl, d);
        if (lane >= d) incl += x;
    }
    if (lane == 31) scan[warp] = incl, lengths[warp] = most;
    __syncthreads();
    long long sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) incl += scan[w];
        sum += scan[w];
        most = max(most, lengths[w]);
    }
    const long long units = (sum >> 40) * per_seq;
    const bool apart = units <= gridDim.x && most <= (4 * units >= gridDim.x ? 16 : 8);
    // Many short units are a warp's own each: nothing to meet for.  The rule goes by tiles of one warp: the longest unit or
    // an equal share, and half of the other, against a share of a CTA's tiles and the ends of its units.  (us with warps'
    // own units / cut, 32 heads on 8, 4 bits: 256 sequences of 64 to 128 tokens 15.9 / 26.2, of 256 to 512 36.9 / 44.9,
    // 128 of 512 26.5 / 30.5; 100 of 300 to 600 27.2 / 25.0, 300 of up to 2000 93.8 / 83.7: cut.  The first, the second
    // and the fourth of them: 8 bits 18.4 / 32.9, 47.5 / 57.1, 26.0 / 31.8; head_dim 64 11.0 / 20.8, 25.1 / 32.9, and
    // 22.8 / 20.4: cut; 16 heads per KV head, four times the sequences, 24.4 / 61.2, 57.6 / 87.9, 33.0 / 47.0.)
    const long long mask = (1ll << 40) - 1, tiles = ((sum & mask) - kUnitCost * (sum >> 40)) * per_seq;
    bool alone = false;
    if (!apart && units >= gridDim.x && tiles + 2 * units <= 1 << 18) {
        const float ctas = gridDim.x, fair = __fdividef(tiles + 2 * units, kWarps * ctas);
        alone = fmaxf(most + 2, fair) + 0.5f * fminf(most + 2, fair) < __fdividef(0.3f * tiles + 3.5f * units, ctas);
    }
    const int own = alone ? 2 : kUnitCost;  // of a unit, beside its tiles
    auto cost = [&](int nt) { return apart ? 1 : nt + own; };
    auto pick = [&](long long x) { return (apart ? x >> 40 : (x & mask) - (kUnitCost - own) * (x >> 40)) * per_seq; };
    const long long total = pick(sum), before = pick(incl) - (apart ? some : mine - (kUnitCost - own) * some) * per_seq;
    const long long P = total < static_cast<long long>(gridDim.x) ? total : static_cast<long long>(gridDim.x);
    const long long c = blockIdx.x;
    if (c >= P) return;
    // (products in 32 bits where they will do: a 64-bit division is a call, around which the compiler keeps its registers
    // otherwise: 65.8 us instead of 59.5 for two sequences of 130 thousand tokens, with two barriers fewer before it)
    auto share = [&](long long i) {
        return total <= (1 << 21) ? static_cast<long long>(static_cast<uint32_t>(i * total) / static_cast<uint32_t>(P)) : i * total / P;
    };
    // place i of the list's kWarps gridDim.x ranges, one for each warp
    auto fine = [&](int i) { return static_cast<long long>(static_cast<uint32_t>(i) * static_cast<uint32_t>(total) / (kWarps * gridDim.x)); };
    const int nth = warp * gridDim.x + blockIdx.x;
    long long g0, g1;
    if (alone) g0 = fine(nth), g1 = fine(nth + 1);
    else g0 = share(c), g1 = share(c + 1);
    auto look = [&](long long from, int w) {
        if (from < before || from >= pick(incl)) return;
        long long at = before;
        int b = tid * run;
        for (;; ++b) {
            const int nt = (len_of(b) + kTile - 1) / kTile;
            const long long n = nt > 0 ? static_cast<long long>(cost(nt)) * per_seq : 0;
            if (from < at + n) break;
            at += n;
        }
        found[w] = b;
        found_at[w] = at;
    };
    if (!alone) {
        look(g0, 0);
    } else {
        for (int w = 0; w < kWarps; ++w) look(fine(w * gridDim.x + blockIdx.x), w);
    }
    __syncthreads();

    auto work = [&](auto alone_) {
        constexpr bool kAlone = decltype(alone_)::value;
        // step i of this warp: 16 tokens from token0 + 16 (first_step + kEvery i)
        const int first_step = kAlone ? 0 : warp;
        constexpr int kEvery = kAlone ? 1 : kWarps;
        // (whether [first, end) is a piece of the CTA's range, which ends at g1)
        auto clip = [&](Seg& s, int L) -> bool {
            const long long left = g1 - s.at - kUnitCost;
            s.end = kAlone || apart || left > s.nt ? s.nt : static_cast<int>(left);
            s.token0 = s.first * kTile;
            s.token1 = min(L, s.end * kTile);
            return s.end > s.first;
        };
        auto next = [&](Seg& s) -> bool {  // the unit behind s
            s.at += cost(s.nt);
            if (s.at + (kAlone || apart ? 0 : kUnitCost) >= g1) return false;
            int L = 0;
            if (++s.unit == per_seq) {
                s.unit = 0;
                do L = len_of(++s.b);
                while (L == 0);
                s.nt = (L + kTile - 1) / kTile;
            } else {
                L = len_of(s.b);
            }
            s.first = 0;
            return clip(s, L);
        };
        auto head_of = [&](const Seg& s) { return s.unit / parts; };
        auto q0_of = [&](const Seg& s) { return (s.unit % parts) * kCols; };
        auto steps_of = [&](const Seg& s) {
            const int from = s.token0 + kStep * first_step;
            return from < s.token1 ? (s.token1 - from + kStep * kEvery - 1) / (kStep * kEvery) : 0;
        };
        // table entries of the 32 steps from i0 on, one a lane
        auto entries = [&](const Seg& s, int i0) {
            const int i = i0 + lane;
            int blk = 0;
            if (i < steps_of(s)) {
                blk = a.tables[static_cast<size_t>(s.b) * a.max_blocks + ((s.token0 + kStep * (first_step + kEvery * i)) >> a.block_shift)];
                if (static_cast<unsigned>(blk) >= static_cast<unsigned>(a.num_blocks)) {
                    if (a.err) atomicOr(a.err, PKV_ERRBIT_BLOCK_ID);
                    blk = 0;  // (the flag marks the output as wrong)
                }
            }
            return blk;
        };
        int win = 0, win_next = 0;
        // asks for the rows of step i, into this place of the ring (one group of copies, an empty one behind the last step)
        const uint64_t block_rows = static_cast<uint64_t>(a.num_kv_heads) << a.block_shift;
        uint64_t head_row = 0;  // first row of the segment's head in a block
        auto ask = [&](const Seg& s, int steps, int i, uint8_t* dst) {
            if (i < steps) {
                if ((i & 31) == 0 && i > 0) win = win_next;
                if ((i & 31) == 16) win_next = entries(s, (i & ~31) + 32);
                const uint32_t blk = __shfl_sync(kAll, win, i & 31);
                const uint64_t row = blk * block_rows + head_row + ((s.token0 + kStep * (first_step + kEvery * i)) & bs_mask);
                const uint8_t* k = a.k_codes + row * S::kRow + 16 * lane;
                const uint8_t* v = a.v_codes + row * S::kRow + 16 * lane;
                constexpr int kAll16 = 16 * St::kChunks;  // 16-byte chunks of K
#pragma unroll
                for (int c0 = 0; c0 < kAll16; c0 += 32) {
                    const int c = c0 + lane;
                    cp_async16(dst + St::k_at(c / St::kChunks, c % St::kChunks), k + 16 * c0, 16);
                    cp_async16(dst + St::v_at(c / St::kChunks, c % St::kChunks), v + 16 * c0, 16);
                }
                if (lane < 8)
                    cp_async16(dst + St::kPairs + 16 * lane,
                               reinterpret_cast<const uint8_t*>(lane < 4 ? a.k_params + row : a.v_params + row) + 16 * (lane & 3), 16);
            }
            cp_async_commit();
        };
        // parts of a step's rows to this lane's registers
        auto take_k = [&](uint32_t (&k)[2][S::kKW], const uint8_t* src) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                if constexpr (S::kKW == 8) {
                    load_words<4>(k[r], src + St::k_at(g + 8 * r, t));
                    load_words<4>(k[r] + 4, src + St::k_at(g + 8 * r, 4 + t));
                } else {
                    load_words<S::kKW>(k[r], src + St::k_at(g + 8 * r, 4 * S::kKW * t / 16) + 4 * S::kKW * t % 16);
                }
            }
        };
        auto take_v = [&](uint32_t (&v)[4][S::kVW], const uint8_t* src) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                load_words<S::kVW>(v[r], src + St::v_at(2 * t + (r & 1) + 8 * (r >> 1), 4 * S::kVW * g / 16) + 4 * S::kVW * g % 16);
        };
        auto q_row = [&](const Seg& s, int n) {  // of column 8 n + g (the first one's where there is no such head)
            const int q0 = q0_of(s), r = 8 * n + g;
            return a.q + (static_cast<size_t>(s.b) * a.num_q_heads + head_of(s) * gh + q0 + (r < min(kCols, gh - q0) ? r : 0)) * kDim;
        };

        Seg seg;
        seg.b = found[kAlone ? warp : 0];
        {
            int L = len_of(seg.b);
            const long long at = found_at[kAlone ? warp : 0];
            seg.nt = (L + kTile - 1) / kTile;
            if constexpr (kAlone) {  // the first unit that begins in the range
                seg.unit = static_cast<int>((static_cast<uint32_t>(g0 - at) + cost(seg.nt) - 1) / cost(seg.nt));
                seg.at = at + static_cast<long long>(seg.unit) * cost(seg.nt);
                if (seg.at >= g1) return;
                if (seg.unit == per_seq) {
                    seg.unit = 0;
                    do L = len_of(++seg.b);
                    while (L == 0);
                    seg.nt = (L + kTile - 1) / kTile;
                }
                seg.first = 0;
            } else {
                seg.unit = static_cast<int>((g0 - at) / cost(seg.nt));
                seg.at = at + static_cast<long long>(seg.unit) * cost(seg.nt);
                seg.first = static_cast<int>(!apart && g0 - seg.at > kUnitCost ? g0 - seg.at - kUnitCost : 0);
            }
            if (!clip(seg, L)) return;  // (nothing but a unit's own cost)
        }
        // this lane's share of the unit's query rows, BF16 pairs: asked for before the cache's rows, behind whose flood they
        // would come 3 us later
        uint32_t qw[kNT][S::kKW][16 / kBits];
        auto load_q = [&]() {
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
                const __nv_bfloat16* qr = q_row(seg, n);
#pragma unroll
                for (int w = 0; w < S::kKW; ++w) load_global<16 / kBits>(qw[n][w], qr + S::k_dim(t, w));
            }
        };
        load_q();
        win = entries(seg, 0);
        head_row = static_cast<uint64_t>(head_of(seg)) << a.block_shift;
#pragma unroll
        for (int d = 0; d < kDepth; ++d) ask(seg, steps_of(seg), d, ring + d * St::kBytes);
        bool has[2] = {false, false};
        for (bool more = true; more;) {
            // ------------------------------------------------- queries -> operands
            uint32_t qf[kNT][S::kKSteps][2];
            float fs[kNT][2], fz[kNT][2];  // of this lane's columns in the softmax: factors of s (q . n) and of z
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
                float x[S::kKW][32 / kBits];
                float top = 0.f, sum = 0.f;
                const bool real = 8 * n + g < min(kCols, gh - q0_of(seg));
#pragma unroll
                for (int w = 0; w < S::kKW; ++w) {
#pragma unroll
                    for (int j = 0; j < 32 / kBits; j += 2) {
                        x[w][j] = real ? bf16_lo(qw[n][w][j / 2]) : 0.f;
                        x[w][j + 1] = real ? bf16_hi(qw[n][w][j / 2]) : 0.f;
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
                    const int col = 2 * (kPair ? t & 1 : t) + j;
                    const float fj = __shfl_sync(kAll, f, col * 4);
                    fs[n][j] = fj * 16777216.f;
                    fz[n][j] = fj * __shfl_sync(kAll, sum, col * 4);
                }
            }

            // ---------------------------------------------------------- the tokens
            const int steps = steps_of(seg);
            float o[kNT][S::kKSteps][4];
            float m[kNT][2], lift[kNT][2], l[kNT][2], zs[kNT][2];  // the base of l and zs, and how far O's lies above it
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
#pragma unroll
                for (int i = 0; i < S::kKSteps; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[n][i][j] = 0.f;
#pragma unroll
                for (int j = 0; j < 2; ++j) m[n][j] = kNone, lift[n][j] = l[n][j] = zs[n][j] = 0.f;
            }

            // Steps i .. i + kNS - 1.  With at most four heads two steps share the softmax: columns 4 to 7 of the products
            // are nobody's, so lanes with t >= 2 take the second step's scores of the first four.
            auto use = [&](int i, const uint8_t* at_ring, auto whole_steps) {
                constexpr bool kWhole = decltype(whole_steps)::value;  // every token is there
                float sc[kNS][kNT][2][4] = {};
#pragma unroll
                for (int e = 0; e < kNS; ++e) {
                    uint32_t xk[2][S::kKW];
                    take_k(xk, at_ring + e * St::kBytes);
#pragma unroll
                    for (int ks = 0; ks < S::kKSteps; ++ks) {
                        uint32_t a0, a1, a2, a3;
                        if constexpr (kBits == 4) {
                            const uint32_t w0 = xk[0][ks / 2] >> (8 * (ks & 1)), w1 = xk[1][ks / 2] >> (8 * (ks & 1));
                            a0 = w0 & 0x000F000Fu, a2 = w0 & 0x00F000F0u;
                            a1 = w1 & 0x000F000Fu, a3 = w1 & 0x00F000F0u;
                        } else {
                            a0 = xk[0][ks] & 0x00FF00FFu, a2 = (xk[0][ks] >> 8) & 0x00FF00FFu;
                            a1 = xk[1][ks] & 0x00FF00FFu, a3 = (xk[1][ks] >> 8) & 0x00FF00FFu;
                        }
#pragma unroll
                        for (int n = 0; n < kNT; ++n) mma16(sc[e][n][ks & 1], a0, a1, a2, a3, qf[n][ks][0], qf[n][ks][1]);
                    }
                }
                // exponents of the weights: rows g (r = 0) and g + 8 (r = 1) of this lane's step
                const int my = i + (kPair ? t >> 1 : 0);
                const int left = kWhole ? kStep : seg.token1 - (seg.token0 + kStep * (first_step + kEvery * my));  // tokens that are there
                const uint32_t* pairs = reinterpret_cast<const uint32_t*>(at_ring + (my - i) * St::kBytes + St::kPairs);
                float ks_[2], kz[2], lg[2], vz[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const bool there = g + 8 * r < left;
                    const uint32_t kp = pairs[g + 8 * r], vp = pairs[16 + g + 8 * r];
                    ks_[r] = bf16_lo(kp), kz[r] = bf16_hi(kp);
                    lg[r] = there ? lg2f(bf16_lo(vp)) : 0.f;
                    vz[r] = there ? bf16_hi(vp) : 0.f;
                }
                uint32_t pb[kNS][kNT][2];
#pragma unroll
                for (int n = 0; n < kNT; ++n) {
                    // Exponents of the weights: u of l's, e of O's, above l's base both.  (V's scale is added to the
                    // difference: the scores themselves may be too large to hold it.)
                    float y[2][2], u[2][2], e[2][2];
                    bool grown = false;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            float dot = sc[0][n][0][2 * r + j] + sc[0][n][1][2 * r + j];
                            if constexpr (kPair) {
                                const float other = __shfl_xor_sync(kAll, sc[1][n][0][2 * r + j] + sc[1][n][1][2 * r + j], 2);
                                dot = t < 2 ? dot : other;
                            }
                            const float x_ = fmaf(ks_[r], dot * fs[n][j], kz[r] * fz[n][j]);
                            y[r][j] = g + 8 * r < left ? x_ : -INFINITY;
                            u[r][j] = y[r][j] - m[n][j];
                            e[r][j] = u[r][j] + lg[r];
                        }
                        grown |= fmaxf(u[0][j], u[1][j]) > kLag || fmaxf(e[0][j], e[1][j]) > lift[n][j] + (kHigh + kLag);
                    }
                    // the maxima move only when an exponent passes one by 8 (weights stay below 2^8, FP16 ones below 2^15)
                    if (__any_sync(kAll, grown)) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float top = fmaxf(y[0][j], y[1][j]);
#pragma unroll
                            for (int x = kPair ? 2 : 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, x));
                            top = fmaxf(top, m[n][j]);
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                u[r][j] = y[r][j] - top;
                                e[r][j] = u[r][j] + lg[r];
                            }
                            float topw = fmaxf(e[0][j], e[1][j]);
#pragma unroll
                            for (int x = kPair ? 2 : 4; x < 32; x <<= 1) topw = fmaxf(topw, __shfl_xor_sync(kAll, topw, x));
                            const float down = m[n][j] - top;
                            topw = fmaxf(topw - kHigh, lift[n][j] + down);
                            const float f = ex2f(down), fw = ex2f(lift[n][j] - topw + down);
                            m[n][j] = top;
                            lift[n][j] = topw;
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
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            w[r][j] = ex2f(e[r][j] - lift[n][j]);
                            const float p = ex2f(u[r][j]);
                            l[n][j] += p;
                            zs[n][j] = fmaf(p, vz[r], zs[n][j]);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        pb[0][n][r] = turn(half2_of(w[r][0], w[r][1]));
                        if constexpr (kPair) pb[1][n][r] = __shfl_xor_sync(kAll, pb[0][n][r], 16);  // (rows 4 to 7 come to 0 to 3)
                    }
                }
                // O^T
#pragma unroll
                for (int e = 0; e < kNS; ++e) {
                    if (e > 0 && !kWhole && i + e >= steps) break;
                    uint32_t xv[4][S::kVW];
                    take_v(xv, at_ring + e * St::kBytes);
#pragma unroll
                    for (int wi = 0; wi < S::kVW; ++wi) {
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const uint32_t sel = hf ? 0x7632u : 0x5410u;
                            const uint32_t x0 = __byte_perm(xv[0][wi], xv[1][wi], sel), x1 = __byte_perm(xv[2][wi], xv[3][wi], sel);
                            if constexpr (kBits == 4) {
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    const uint32_t y0 = x0 >> (8 * u), y1 = x1 >> (8 * u);
#pragma unroll
                                    for (int n = 0; n < kNT; ++n)
                                        mma16(o[n][4 * wi + 2 * hf + u], y0 & 0x000F000Fu, y0 & 0x00F000F0u, y1 & 0x000F000Fu,
                                              y1 & 0x00F000F0u, pb[e][n][0], pb[e][n][1]);
                                }
                            } else {
#pragma unroll
                                for (int n = 0; n < kNT; ++n)
                                    mma16(o[n][2 * wi + hf], x0 & 0x00FF00FFu, (x0 >> 8) & 0x00FF00FFu, x1 & 0x00FF00FFu,
                                          (x1 >> 8) & 0x00FF00FFu, pb[e][n][0], pb[e][n][1]);
                            }
                        }
                    }
                }
            };

            static_assert(kDepth % kNS == 0);
            uint8_t* place = ring;  // of step i
            for (int i = 0; i < steps; i += kNS) {
                cp_async_wait<kDepth - kNS>();
                __syncwarp();
                // (only a sequence's last tokens lie in steps that are not whole, or have no second one)
                if (i + kNS < steps) use(i, place, std::true_type{});
                else use(i, place, std::false_type{});
                __syncwarp();  // (the rows may be written over)
#pragma unroll
                for (int e = 0; e < kNS; ++e) ask(seg, steps, i + e + kDepth, place + e * St::kBytes);
                place = place + kNS * St::kBytes == ring + kRing ? ring : place + kNS * St::kBytes;
            }
            // the next unit's first rows are under way from here on
            const Seg done = seg;
            more = next(seg);
            if (more) {
                load_q();
                win = entries(seg, 0);
                head_row = static_cast<uint64_t>(head_of(seg)) << a.block_shift;
            }

            if constexpr (kAlone) {
                if (more) {
#pragma unroll
                    for (int d = 0; d < kDepth; ++d) ask(seg, steps_of(seg), d, ring + d * St::kBytes);
                }
                const int rows = min(kCols, gh - q0_of(done));
                const size_t out0 = static_cast<size_t>(done.b) * a.num_q_heads + head_of(done) * gh + q0_of(done);
#pragma unroll
                for (int n = 0; n < kNT; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
#pragma unroll
                        for (int d = kPair ? 2 : 4; d < 32; d <<= 1) {
                            l[n][j] += __shfl_xor_sync(kAll, l[n][j], d);
                            zs[n][j] += __shfl_xor_sync(kAll, zs[n][j], d);
                        }
                        const int col = 8 * n + 2 * t + j;
                        if ((kPair && t >= 2) || col >= rows) continue;
                        // O in the base of l, the codes' 2^24 (and the upper nibbles' 2^-4) taken out.  The bases differ by V's
                        // scale, up to 2^132 with the maxima's lag: in two halves.
                        const float half = ex2f(0.5f * lift[n][j]), inv = 1.f / l[n][j];
                        const float up = 16777216.f * inv * half, up2 = kBits == 4 ? 0.0625f * up : up, z = zs[n][j] * inv;
                        // this lane's dimensions of the head: kDim / 8 from g (kDim / 8) on
                        uint32_t y[S::kKSteps];
#pragma unroll
                        for (int i = 0; i < S::kKSteps; ++i)
                            y[i] = pack_bf16x2_rn(fmaf(o[n][i][j] * up, half, z), fmaf(o[n][i][2 + j] * up2, half, z));
                        uint4* dst = reinterpret_cast<uint4*>(a.out + (out0 + col) * kDim + g * (kDim / 8));
#pragma unroll
                        for (int i = 0; i < S::kKSteps; i += 4) dst[i / 4] = make_uint4(y[i], y[i + 1], y[i + 2], y[i + 3]);
                    }
            } else {
                // ------------------------------------------------ the warps' sums meet
#pragma unroll
                for (int n = 0; n < kNT; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
#pragma unroll
                        for (int d = kPair ? 2 : 4; d < 32; d <<= 1) {
                            l[n][j] += __shfl_xor_sync(kAll, l[n][j], d);
                            zs[n][j] += __shfl_xor_sync(kAll, zs[n][j], d);
                        }
                        const int col = 8 * n + 2 * t + j;
                        if (kPair && t >= 2) continue;
                        const float half = ex2f(0.5f * lift[n][j]), up = 16777216.f * half;  // (as above)
                        const float up2 = kBits == 4 ? 0.0625f * up : up;
                        if (g == 0) {
                            sm[warp][col] = m[n][j];
                            sl[warp][col] = l[n][j];
                            sz[warp][col] = zs[n][j];
                        }
                        // element (dimension g (kDim / 8) + x) of column col at [x][g]: all lanes in different banks
#pragma unroll
                        for (int i = 0; i < S::kKSteps; ++i) {
                            so(warp)[col][(2 * i) * 8 + g] = o[n][i][j] * up * half;
                            so(warp)[col][(2 * i + 1) * 8 + g] = o[n][i][2 + j] * up2 * half;
                        }
                    }
                __syncthreads();
                if (more) {
#pragma unroll
                    for (int d = 0; d < kEarly; ++d) ask(seg, steps_of(seg), d, ring + d * St::kBytes);
                }
                const bool whole = done.first == 0 && done.end == done.nt;
                const int side = g0 >= done.at + kUnitCost ? 0 : 1, rows = min(kCols, gh - q0_of(done));
                const size_t slot = 2 * static_cast<size_t>(c) + side;
                const size_t out0 = static_cast<size_t>(done.b) * a.num_q_heads + head_of(done) * gh + q0_of(done);
                // lane (w, r): what the sums of warp w weigh in column r, by shuffles over the warps' lanes
                constexpr int kPerPass = kThreads / kDim;  // rows that the CTA's threads write at once
                const int d = tid % kDim, at_ = (d % (kDim / 8)) * 8 + d / (kDim / 8);
#pragma unroll
                for (int n = 0; n < kNT; ++n) {
                    const int w = lane >> 3, r8 = 8 * n + (lane & 7);
                    const float mr = sm[w][r8], lr = sl[w][r8];
                    float M = fmaxf(mr, __shfl_xor_sync(kAll, mr, 8));
                    M = fmaxf(M, __shfl_xor_sync(kAll, M, 16));
                    const float f = ex2f(mr - M);
                    float lw = f * lr, zw = f * sz[w][r8];
                    lw += __shfl_xor_sync(kAll, lw, 8);
                    lw += __shfl_xor_sync(kAll, lw, 16);
                    zw += __shfl_xor_sync(kAll, zw, 8);
                    zw += __shfl_xor_sync(kAll, zw, 16);
                    const float inv = 1.f / lw;
                    if (!whole && tid < 8 && r8 < rows)
                        reinterpret_cast<float2*>(a.part_ml)[slot * kCols + r8] = make_float2(M, lw);
#pragma unroll
                    for (int k = 0; k < (kPair ? 4 : 8); k += kPerPass) {
                        const int r = k + tid / kDim;  // (the same in a warp)
                        float y = __shfl_sync(kAll, zw, r);
#pragma unroll
                        for (int v = 0; v < kWarps; ++v) y = fmaf(__shfl_sync(kAll, f, 8 * v + r), so(v)[8 * n + r][at_], y);
                        const float i = __shfl_sync(kAll, inv, r);
                        if (8 * n + r < rows) {
                            if (whole) a.out[(out0 + 8 * n + r) * kDim + d] = __float2bfloat16_rn(y * i);
                            else a.part_o[(slot * kCols + 8 * n + r) * kDim + d] = y;
                        }
                    }
                }
                __syncthreads();  // (the shared sums are read, the piece is written)
                if (more) {
#pragma unroll
                    for (int d = kEarly; d < kDepth; ++d) ask(seg, steps_of(seg), d, ring + d * St::kBytes);
                }
                if (!whole) {
                    has[side] = true;
                    if (tid == 0) {  // count the piece; who counts the last one joins them, when its own range is done
                        split[side] = done;
                        __threadfence();
                        const long long c0 = ((done.at + kUnitCost + 1) * P - 1) / total, c1 = ((done.at + kUnitCost + done.nt) * P - 1) / total;
                        int* counter = a.counters + c0;  // (no other unit's first piece is this CTA's)
                        last_flag[side] = count_up(counter) == static_cast<int>(c1 - c0);
                        if (last_flag[side]) *counter = 0;
                    }
                }
            }
        }
        if constexpr (!kAlone) {
            if (!has[0] && !has[1]) return;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (!has[k] || !last_flag[k]) continue;
                __threadfence();
                const Seg u = split[k];
                // the unit's pieces: CTAs c0 .. c0 + n - 1, each one piece, the first one's at its range's start or end
                const long long c0 = ((u.at + kUnitCost + 1) * P - 1) / total, c1 = ((u.at + kUnitCost + u.nt) * P - 1) / total;
                const int n = static_cast<int>(c1 - c0 + 1), extra = c0 * total / P >= u.at + kUnitCost ? 0 : 1;
                const int rows = min(kCols, gh - q0_of(u));
                const size_t out0 = static_cast<size_t>(u.b) * a.num_q_heads + head_of(u) * gh + q0_of(u);
                auto slot_of = [&](int i) { return static_cast<size_t>(2 * (c0 + i) + (i == 0 ? extra : 0)); };
                for (int r = warp; r < rows; r += kWarps) {
                    float M = kNone;
                    for (int i = lane; i < n; i += 32) M = fmaxf(M, __ldcg(a.part_ml + 2 * (slot_of(i) * kCols + r)));
                    M = warp_max(M);
                    constexpr int kPer = kDim / 32;
                    float acc[kPer] = {}, lw = 0.f;
                    for (int i0 = 0; i0 < n; i0 += 32) {
                        float f = 0.f, lf = 0.f;
                        if (i0 + lane < n) {
                            const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + slot_of(i0 + lane) * kCols + r);
                            f = ex2f(ml.x - M);
                            lf = f * ml.y;
                        }
                        lw += warp_sum(lf);
                        const int k1 = min(32, n - i0);
                        for (int j0 = 0; j0 < k1; j0 += 16) {  // 16 pieces' rows in one round trip
                            float y[16][kPer];
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const float* src = a.part_o + (slot_of(i0 + min(j0 + j, k1 - 1)) * kCols + r) * kDim + kPer * lane;
                                if constexpr (kPer == 4) {
                                    const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
                                    y[j][0] = v.x, y[j][1] = v.y, y[j][2] = v.z, y[j][3] = v.w;
                                } else {
                                    const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
                                    y[j][0] = v.x, y[j][1] = v.y;
                                }
                            }
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const float fj = __shfl_sync(kAll, f, (j0 + j) & 31);
#pragma unroll
                                for (int k = 0; k < kPer; ++k)
                                    if (j0 + j < k1) acc[k] = fmaf(fj, y[j][k], acc[k]);
                            }
                        }
                    }
                    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + (out0 + r) * kDim + kPer * lane);
#pragma unroll
                    for (int j = 0; j < kPer; j += 2) dst[j / 2] = pack_bf16x2_rn(__fdiv_rn(acc[j], lw), __fdiv_rn(acc[j + 1], lw));
                }
            }
        }
    };
    if (!alone) work(std::false_type{});
    else work(std::true_type{});
}

int columns(int gh) { return gh <= 8 ? 8 : 16; }

}  // namespace

size_t quant_decode_workspace(int num_q_heads, int num_kv_heads, int head_dim, uint8_t* base, QuantDecodeArgs* a) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const int cols = columns(num_q_heads / num_kv_heads);
    // (counters at one place for calls of all sizes: they are what a call leaves for the next)
    constexpr size_t counters = kWorkspaceZeros;
    static_assert(kMaxCtas * sizeof(int32_t) <= counters);
    const size_t ml = up(static_cast<size_t>(kMaxCtas) * 2 * cols * 2 * sizeof(float));
    if (a) {
        a->counters = reinterpret_cast<int32_t*>(base);
        a->part_ml = reinterpret_cast<float*>(base + counters);
        a->part_o = reinterpret_cast<float*>(base + counters + ml);
    }
    return counters + ml + static_cast<size_t>(kMaxCtas) * 2 * cols * head_dim * sizeof(float);
}

template <int kBits, int kDim, int kNT, bool kPair>
static cudaError_t launch(const QuantDecodeArgs& a, cudaStream_t stream) {
    constexpr int smem = kWarps * depth_of(kBits, kDim, kNT) * Stage<kBits, kDim>::kBytes;
    static_assert(ctas_per_sm(kBits, kDim, kNT) * (smem + 3 * 1024) <= 228 * 1024, "shared memory per SM");
    const auto kernel = quant_decode_kernel<kBits, kDim, kNT, kPair>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)  // (all of an SM's CTAs have to fit)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    const int sms = num_sms() > 0 ? num_sms() : 148, ctas = sms * ctas_per_sm(kBits, kDim, kNT);
    return launch_dependent(kernel, dim3(ctas < kMaxCtas ? ctas : kMaxCtas), dim3(kThreads), smem, stream, a);
}

cudaError_t launch_quant_decode(int bits, int head_dim, const QuantDecodeArgs& a, cudaStream_t stream) {
    const int gh = a.num_q_heads / a.num_kv_heads;
    auto pick = [&](auto four, auto eight, auto sixteen) {
        return gh <= 4 ? four(a, stream) : columns(gh) == 8 ? eight(a, stream) : sixteen(a, stream);
    };
    if (bits == 4)
        return head_dim == 64 ? pick(launch<4, 64, 1, true>, launch<4, 64, 1, false>, launch<4, 64, 2, false>)
                              : pick(launch<4, 128, 1, true>, launch<4, 128, 1, false>, launch<4, 128, 2, false>);
    return head_dim == 64 ? pick(launch<8, 64, 1, true>, launch<8, 64, 1, false>, launch<8, 64, 2, false>)
                          : pick(launch<8, 128, 1, true>, launch<8, 128, 1, false>, launch<8, 128, 2, false>);
}

}  // namespace pkv
