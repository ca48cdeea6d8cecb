// Causal attention over packed prompts on the 5th-generation tensor cores
// (tcgen05 with accumulators in tensor memory): BF16, head_dim 64 or 128.
//
// A row tile is 128 rows (query, head of the group) of one (sequence, KV head), so
// a K or V row serves the whole group and a tile's causal edge spans few positions.
// A unit is two row tiles, A and B, that walk over the same 128-key tiles together:
// while the softmax of one runs, the tensor core multiplies for the other.  One
// persistent CTA per SM takes units from a common counter, long sequences' first and
// within a sequence the ones with the most keys first, so that what is left for the
// end is short.  Of the units behind the last round that fills all SMs (all, where they are
// fewer than SMs) the keys are cut into pieces, whose sums a second kernel joins (us, 32
// query heads on 8: 300 queries behind 8000 keys 158 -> 58, 512 behind 32256 596 -> 235, 20
// behind 1980 24 -> 20, 4 x 300 behind 7700, 160 units, 216 -> 143), unless that would not
// shorten a unit by three tiles (3 x 100 queries on 600 keys: 18.6, cut 23.9; units are then
// single row tiles if they are fewer than SMs), or those units fill more than half of the
// SMs (2048 queries behind 8192, 256 units: 247, as they are).  The second kernel's launch costs 2 to 3 us (8 prompts of 130: 15.3, with it
// 17.8), so calls whose rows alone make a unit for every SM, or have few keys a sequence,
// take an instance without it.
//
// What bounds it: the chain of a row tile, 3300 cycles for each key tile (clock stamps): S seen
// and loaded 320, weights 850, written and signalled 400, taken by the issuer 330, P V and the
// next S 1030, S seen 350.  The other row tile fills it, so the tensor core works 2060 of 3300
// cycles.  Scores in two places would break the chain, but two row tiles' scores and outputs
// take all of tensor memory; halves of 64 keys in turn made the score products slower (48.5
// cycles for 64 keys, 64 for 128: their operands' way out of shared memory) and the whole too
// (1.66 ms for the case below).  A unit costs about two more key tiles than it has.
// Measured over rotating inputs, 32 query heads on 8 of 128: one prompt of 16384 tokens 1.54 ms,
// 1.43 PFLOP/s of what is seen (1.49 ms back to back on the same ones); 16 prompts of 128 to 4096
// 591 to 668 us; 8 chunks of 256 to 512 behind up to 8192 185 to 204 us; 33 prompts of 1 to 127
// 21.3 us, of which a call of one row takes 7.6.
//
// 20 warps (the last one idle; a row's scores live in registers, 96 for each of 640 threads):
//  * warp 16, producer: takes units, loads Q tiles, and K and V tiles into one ring
//    (K 0, V 0, K 1, ...) by TMA;
//  * warps 17 and 18, one thread each issues the MMAs of A and of B: S = Q K^T into the
//    row tile's 128 score columns, then O += P V with P (BF16) read from tensor memory
//    over those columns (each thread's 64 keys in the first half of its own 64 columns),
//    then S of the next key tile.  One thread's MMAs complete in
//    order, so "S j + 1 done" says that P V j is done too.  (One issuer for both spent
//    4200 of 4500 cycles per pair of tiles on its own instructions);
//  * warps 0-7 and 8-15, softmax of A and of B: two threads own a row, one its first 64
//    keys of a tile and half of its output columns, the other the rest.  The base of a
//    row's weights is a past maximum, agreed on while the tile's products run: it moves
//    only when a score passes it by 8 (log2 units), which rescales O in tensor memory
//    before the next tile's products, or by 16 at once, before this tile's.  Statistics
//    and sums are FP32; a weight is rounded to BF16 for its product with V, the type that
//    the tensor core takes beside V's.
// Tensor memory: 2 x 128 score columns, 2 x head_dim output columns.
// Shared memory: Q 2 x 32 KB, four ring stages of 32 KB, the units' plan.
// Every wait is bounded: an expired one sets PKV_ERRBIT_TIMEOUT and ends the CTA, whose
// copies and products have landed by then; the rows of the units that it had are NaN.
#include <cuda.h>

#include <climits>
#include <type_traits>

#include "quant_internal.h"
#include "tc_common.cuh"

namespace pkv {
namespace {

constexpr int kSoftmaxWarps = 16;     // eight for each row tile, two threads a row
constexpr int kProducer = 16, kIssuer = 17;  // warps (two issuers)
constexpr int kThreads = 640;
constexpr int kRows = 128, kKeys = 128;
constexpr int kHalf = 128 * 128;     // 64 columns of 128 rows
constexpr int kStages = 4;
constexpr int kSlots = 2;            // units in the queue
constexpr float kFar = 16.f;         // weights stay below 2^16, and sums of 2^96 times the values' 2^16 keys in 32 bits
constexpr float kLarge = 0x1p29f;    // from here on kFar does not show beside a base, whose steps are wider than 2 kFar
constexpr int kSortSeqs = 256;       // up to so many sequences are taken longest first
constexpr int kLeastPiece = 4;       // key tiles of a unit's piece, at least
constexpr int kWorth = 3;            // what cutting costs, in key tiles
constexpr int kPieces = 2;           // pieces for each SM, at most
constexpr int kJoinThreads = 1024;

// Words of the plan and, for a CTA that gives up, of what it had in hand.
enum Misc {
    kPerUnit = 0,       // row tiles of a unit
    kPart = 1,          // key tiles of a piece (0: nothing is cut)
    kWhole = 2,         // places of the list whose units are whole
    kAhead = 3,         // whole units of the next place
    kUntaken = 4,       // the first unit that no CTA took (for the last CTA to finish)
    kTaken = 5,         // units that this CTA took
    kHeld = 6,          // the last eight of them
    kStopped = kHeld + 8,  // for each softmax warp, which of the CTA's units it gave up at
    kMiscWords = kStopped + kSoftmaxWarps
};

enum Bar {
    kQFull = 0, kQFree = 2, kFull = 4, kFree = kFull + kStages, kSFull = kFree + kStages, kPFull = kSFull + 2,
    kOFull = kPFull + 2, kOFree = kOFull + 2, kUFull = kOFree + 2, kUFree = kUFull + kSlots, kDone = kUFree + kSlots,
    kBars = kDone + 2
};

struct Unit {
    int q0;        // first query row (packed)
    int n;         // queries from there to the end of the sequence
    int k0, m;     // first key row, keys of the sequence
    int head;      // KV head
    int seen;      // keys that query q0 sees (may be negative)
    int more;      // 0: no unit, the list is at its end
    // Of a unit whose keys are cut into pieces (k0, m and seen count from the piece's first key):
    int first;     // key tiles before the piece
    int len;       // key tiles of a piece; INT_MAX: not cut
    int slot;      // place of the unit's first piece in the workspace
};

template <int kDim>
struct Layout {
    static constexpr int kHalves = kDim / 64;
    static constexpr int kTile = kHalves * kHalf;  // bytes of a Q, K or V tile
    static constexpr int kQ = 0, kRing = 2 * kTile, kBar = kRing + kStages * kTile;
    static constexpr int kQueue = kBar + 8 * kBars + 16, kMisc = kQueue + kSlots * static_cast<int>(sizeof(Unit));
    static constexpr int kSay = (kMisc + 4 * kMiscWords + 127) / 128 * 128;  // what a row's two threads tell each other
    static constexpr int kPlan = kSay + 3 * 4 * kRows * 8;
    static constexpr int kSmem = kPlan + (kPromptMaxSeqs + 1) * 4 + kPromptMaxSeqs * 2 + 1024;
    static_assert(kSmem <= 232448, "shared memory per CTA");
};

struct Span {
    int q0, n, k0, m;
};
__device__ __forceinline__ Span span_of(const PromptArgs& a, int b, bool report, bool* bad = nullptr) {
    Span s{a.q_offsets[b], a.q_offsets[b + 1], a.k_offsets[b], a.k_offsets[b + 1]};
    const bool ok = s.q0 >= 0 && s.n >= s.q0 && s.n <= a.q_rows && s.k0 >= 0 && s.m >= s.k0 && s.m <= a.k_rows;
    if (!ok && report && a.err) atomicOr(a.err, PKV_ERRBIT_OFFSETS);
    if (bad) *bad |= !ok;
    s.n = ok ? s.n - s.q0 : 0;
    s.m = ok ? s.m - s.k0 : 0;
    return s;
}

// Pieces that a sequence's units are cut into (part: tiles of a piece, 0: not cut).
__device__ __forceinline__ int pieces_of(int m, int part) {
    return part > 0 && m > 0 ? ((m - 1) / kKeys + part) / part : 1;
}

// Keys that a sequence's units behind its first `whole` see at most (units of `queries`, the ones that see the most first).
__device__ __forceinline__ int keys_behind(const Span& s, int queries, int whole) {
    const int units = (s.n + queries - 1) / queries;
    return max(0, min(s.m, s.m - s.n + (units - whole) * queries));
}

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int half, int head, int row, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(half), "r"(head), "r"(row), "r"(bar)
        : "memory");
}

// Eight columns of this thread's lane times f.  (Few registers: a row's scores are live around it.)
__device__ __forceinline__ void tmem_scale8(uint32_t at, float f) {
    uint32_t v[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * f);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(at), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// The same for BF16 pairs.
__device__ __forceinline__ void tmem_scale8_bf16(uint32_t at, float f) {
    uint32_t v[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = bf16x2(bf16_lo(v[k]) * f, bf16_hi(v[k]) * f);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(at), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// 16 columns of this thread's lane.
__device__ __forceinline__ void tmem_st16_nowait(uint32_t at, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(at),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// The next base: whole steps above the last one, so that a change of base is exact.  (Far enough above, nothing is left of
// the weights before, and the sum might miss `top` by more than weights may be above the base.)
__device__ __forceinline__ float above(float base, float top) {
    return top - base > 4096.f ? top : base + ceilf(top - base);
}

// What the roles agree on about a unit.
template <bool kCut>
struct Shape {
    int tiles[2];  // key tiles of row tile A and of B
    int nt;        // of the unit
    __device__ Shape(const Unit& u, int qpt, int per_unit) {
        for (int x = 0; x < 2; ++x) {
            const int first = x * qpt;  // first query of the row tile
            const int last = min(u.n, first + qpt) - 1;
            const bool there = x < per_unit && first < u.n;
            tiles[x] = there ? max(0, (u.seen + last + kKeys - 1) / kKeys) : 0;
            if (kCut) tiles[x] = min(tiles[x], u.len);
        }
        nt = max(tiles[0], tiles[1]);
    }
};

// The plan in shared memory.
struct Plan {
    const int *misc, *cum;
    const uint16_t* order;
};
// Unit `id` of the list.
template <bool kCut>
__device__ __forceinline__ Unit unit_at(const PromptArgs& a, const Plan& p, int id, int per_unit) {
    const int *misc = p.misc, *cum = p.cum, qpt = kRows / (a.num_q_heads / a.num_kv_heads);
    const uint16_t* order = p.order;
    int lo = 0, hi = a.num_seqs;  // the last place whose first unit is at or before id
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (static_cast<int64_t>(cum[mid]) * a.num_kv_heads <= id) lo = mid;
        else hi = mid;
    }
    const Span s = span_of(a, order[lo], false);
    const int j = id - cum[lo] * a.num_kv_heads, head = j % a.num_kv_heads;
    int unit = j / a.num_kv_heads, pieces = 1, piece = 0, part = 0, slot = 0;
    if constexpr (kCut) {
        part = misc[kPart];
        const int ahead = lo < misc[kWhole] ? INT_MAX : lo == misc[kWhole] ? misc[kAhead] : 0;  // whole units
        if (unit >= ahead) {
            pieces = pieces_of(keys_behind(s, per_unit * qpt, ahead), part);
            piece = (unit - ahead) % pieces;
            unit = ahead + (unit - ahead) / pieces;
            slot = id - (piece + cum[misc[kWhole]] + misc[kAhead]) * a.num_kv_heads;  // (counted from the first that is cut)
        }
    }
    const int skip = piece * part * kKeys;
    const int first = ((s.n + per_unit * qpt - 1) / (per_unit * qpt) - 1 - unit) * per_unit * qpt;
    return Unit{s.q0 + first, s.n - first, s.k0 + skip, s.m - skip, head, s.m - s.n + first + 1 - skip, 1,
                piece * part, pieces > 1 ? part : INT_MAX, slot};
}

// NaN for what unit `id` was to write: its rows, or a piece's statistics, with the joining kernel told of its row tile.
// (A call of its own: inlined, it cost the kernel's loops 1 %.)
template <int kDim, bool kCut>
__device__ __noinline__ void lose_unit(const PromptArgs& a, const Plan plan, int id, int per_unit) {
    const Unit u = unit_at<kCut>(a, plan, id, per_unit);
    const int gh = a.num_q_heads / a.num_kv_heads, qpt = kRows / gh, tid = threadIdx.x;
    const Shape<kCut> sh(u, qpt, per_unit);
    const float nan = __uint_as_float(0x7FC00000u);
    for (int x = 0; x < per_unit; ++x) {
        const int n = min(u.n - x * qpt, qpt), sees = u.seen + u.first * kKeys + x * qpt;
        if (n <= 0) continue;
        const int pieces = u.len == INT_MAX ? 1 : (max(0, (sees + n - 1 + kKeys - 1) / kKeys) + u.len - 1) / u.len;
        if (pieces > 1) {
            if (sh.tiles[x] == 0) continue;  // (no query sees this piece)
            const int64_t part_ = (static_cast<int64_t>(u.slot) + u.first / u.len * a.num_kv_heads) * kSoftmaxWarps + 8 * x;
            if (tid < 8 * 32) a.part_ml[part_ * 32 + tid] = make_float2(nan, nan);
            if (tid == 0) a.tiles[2 * u.slot + x] = make_int4(pieces, u.q0 + x * qpt, n | u.head << 8, sees);
        } else if (u.first == 0) {
            uint4* out = reinterpret_cast<uint4*>(a.out);
            for (int e = tid; e < n * gh * (kDim / 8); e += kThreads) {
                const int r = e / (kDim / 8), h = u.head * gh + r % gh;
                out[(static_cast<int64_t>(u.q0 + x * qpt + r / gh) * a.num_q_heads + h) * (kDim / 8) + e % (kDim / 8)] =
                    make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
            }
        }
    }
}

// kCut: the keys of units may be cut into pieces.
template <int kDim, bool kCut>
__global__ void __launch_bounds__(kThreads, 1)
prompt_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                 const __grid_constant__ CUtensorMap mv, const __grid_constant__ PromptArgs a) {
    using Lt = Layout<kDim>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = su32(smem);
    auto B = [&](int i) { return sbase + Lt::kBar + 8u * i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lt::kBar + 8 * kBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lt::kBar + 8 * kBars + 4);
    int* turn = reinterpret_cast<int*>(smem + Lt::kBar + 8 * kBars + 8);  // 1 while an issuer has the tensor core
    volatile Unit* queue = reinterpret_cast<volatile Unit*>(smem + Lt::kQueue);
    int* misc = reinterpret_cast<int*>(smem + Lt::kMisc);
    int* cum = reinterpret_cast<int*>(smem + Lt::kPlan);   // [B + 1] units (pieces) of one KV head before each sequence in order
    uint16_t* order = reinterpret_cast<uint16_t*>(smem + Lt::kPlan + (kPromptMaxSeqs + 1) * 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gh = a.num_q_heads / a.num_kv_heads, qpt = kRows / gh;  // queries of a row tile

    if (tid == 0) {
        for (int i = 0; i < kBars; ++i)
            bar_init(B(i), (i >= kPFull && i < kPFull + 2) || (i >= kOFree && i < kOFree + 2) ? 8u
                           : i >= kUFree && i < kDone ? kSoftmaxWarps + 2u
                           : i >= kFree && i < kFree + kStages ? 2u : 1u);
        *abort_flag = 0;
        *turn = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == kProducer && lane < 3)
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(lane == 0 ? &mq : lane == 1 ? &mk : &mv)) : "memory");
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(su32(tmem_slot)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    }
    if (qpt * gh < kRows) {  // rows of Q tiles that no query has
        const int gone = kRows - qpt * gh;
        for (int e = tid; e < 2 * Lt::kHalves * gone * 8; e += kThreads)
            *reinterpret_cast<uint4*>(smem + Lt::kQ + e / (gone * 8) * kHalf + (qpt * gh + e % (gone * 8) / 8) * 128 + e % 8 * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        fence_async_smem();
    }
    for (int i = tid; i < 3 * 4 * kRows; i += kThreads)  // (tellings are numbered from 1)
        reinterpret_cast<uint2*>(smem + Lt::kSay)[i] = make_uint2(0u, 0u);
    // (nothing before reads or writes what the kernel before this one may)
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    // the plan: sequences in order, and the row tiles before each
    int* keys = cum + 1;  // (first the keys, for the order)
    bool bad = false;
    for (int b = tid; b < a.num_seqs; b += kThreads) keys[b] = span_of(a, b, blockIdx.x == 0, &bad).m;
    bad = __syncthreads_or(bad);
    for (int b = tid; b < a.num_seqs; b += kThreads) {
        int rank = b;
        if (a.num_seqs <= kSortSeqs) {
            rank = 0;
            for (int o = 0; o < a.num_seqs; ++o) rank += keys[o] > keys[b] || (keys[o] == keys[b] && o < b);
        }
        order[rank] = static_cast<uint16_t>(b);
    }
    __syncthreads();
    if (warp == 0) {
        // Two row tiles a unit.  The units behind the last round that fills all SMs have their keys cut into pieces of
        // equal length, if they are few enough; with fewer units than SMs and none cut, a unit is one row tile.
        int per = 2, part = 0, whole = a.num_seqs, ahead = 0;  // places whose units are whole, whole ones of the next
        bool sound = true;  // no more queries than there are rows: units are counted in 32 bits
        auto count = [&](int n) { return (n + per * qpt - 1) / (per * qpt); };
        auto items = [&](const Span& s, int r) {  // of place r
            const int n = sound ? count(s.n) : 0, first = r < whole ? n : r == whole ? min(ahead, n) : 0;
            return n == first ? n : first + (n - first) * pieces_of(keys_behind(s, per * qpt, first), part);
        };
        auto fill = [&]() {
            int at = 0;
            for (int r0 = 0; r0 < a.num_seqs; r0 += 32) {
                const int n = r0 + lane < a.num_seqs ? items(span_of(a, order[r0 + lane], false), r0 + lane) : 0;
                int incl = n;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int x = __shfl_up_sync(0xFFFFFFFFu, incl, d);
                    if (lane >= d) incl += x;
                }
                if (r0 + lane < a.num_seqs) cum[r0 + lane + 1] = at + incl;
                at += __shfl_sync(0xFFFFFFFFu, incl, 31);
            }
            if (lane == 0) cum[0] = 0;
            __syncwarp();
            return at;
        };
        // Sequences of offsets that descend may overlap, so that their queries are more than the rows: none is taken then.
        if (bad) {
            int64_t queries = 0;
            for (int r = lane; r < a.num_seqs; r += 32) queries += span_of(a, r, false).n;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) queries += __shfl_xor_sync(0xFFFFFFFFu, queries, d);
            sound = queries <= a.q_rows;
        }
        const int64_t units = static_cast<int64_t>(fill()) * a.num_kv_heads;
        const int grid = gridDim.x;
        if constexpr (kCut) {
            const int64_t rounds = units / grid;
            const int in_full = static_cast<int>(rounds * grid / a.num_kv_heads);  // units of a head in full rounds
            const int64_t room = rounds == 0 ? grid : kPieces * grid;              // pieces that fit
            if (2 * (units - rounds * grid) <= grid || rounds == 0) {
                int lo = 0, hi = a.num_seqs;  // the place of unit in_full
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (cum[mid] <= in_full) lo = mid;
                    else hi = mid;
                }
                whole = lo, ahead = in_full - cum[lo];
                int most = 0;  // key tiles of the longest unit behind
                int64_t tiles = 0;
                for (int r = whole + lane; r < a.num_seqs; r += 32) {
                    const Span s = span_of(a, order[r], false);
                    const int first = r == whole ? ahead : 0, n = count(s.n) - first;
                    const int nt = (keys_behind(s, per * qpt, first) + kKeys - 1) / kKeys;
                    if (n > 0) most = max(most, nt), tiles += static_cast<int64_t>(n) * nt;
                }
                most = __reduce_max_sync(0xFFFFFFFFu, most);
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) tiles += __shfl_xor_sync(0xFFFFFFFFu, tiles, d);
                part = static_cast<int>(max(static_cast<int64_t>(kLeastPiece), tiles * a.num_kv_heads / room));
                for (; part < most; part += 1 + part / 16) {
                    int64_t all = 0;
                    for (int r = whole + lane; r < a.num_seqs; r += 32) {
                        const Span s = span_of(a, order[r], false);
                        all += items(s, r) - (r == whole ? ahead : 0);
                    }
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, d);
                    if (all * a.num_kv_heads <= room) break;
                }
                if (part + kWorth > most) part = 0;
                if (part == 0) whole = a.num_seqs, ahead = 0;
                else fill();
            }
        }
        if (part == 0 && units < grid) {
            per = 1;
            fill();
        }
        if (lane == 0) misc[kPerUnit] = per, misc[kPart] = part, misc[kWhole] = whole, misc[kAhead] = ahead, misc[kUntaken] = INT_MAX;
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;
    const int per_unit = misc[kPerUnit];
    auto fail = [&]() {
        *abort_flag = 1;
        if (a.err) atomicOr(a.err, PKV_ERRBIT_TIMEOUT);
    };
    // a bounded wait that ends early when another role has given up
    auto wait = [&](int i, int parity, uint32_t polls = kSpin) -> bool {
        for (uint32_t k = 0; k < polls; ++k) {
            uint32_t ok;
            asm volatile(
                "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
                : "=r"(ok)
                : "r"(B(i)), "r"(parity)
                : "memory");
            if (ok) return true;
            if ((k & 255) == 255 && *abort_flag) return false;
        }
        return false;
    };
    auto take = [&](int i) -> Unit {  // the i-th unit of this CTA, once it is in the queue
        const volatile Unit& s = queue[i % kSlots];
        return Unit{s.q0, s.n, s.k0, s.m, s.head, s.seen, s.more, 0, kCut ? s.len : 0, 0};
    };
    const Plan plan{misc, cum, order};
    auto unit_of = [&](int id) -> Unit { return unit_at<kCut>(a, plan, id, per_unit); };

    if (warp == kProducer) {
        // ------------------------------------------------------------ producer
        bool ok = true;
        int stage = 0, q_count[2] = {0, 0};  // tiles put into the ring, Q tiles loaded
        const int total = cum[a.num_seqs] * a.num_kv_heads;
        // (the first unit is the CTA's own number's; the others come from the counter)
        int next = blockIdx.x, taken = 0;
        for (int i = 0; ok; ++i) {
            const int id = __shfl_sync(0xFFFFFFFFu, next, 0);
            if (lane == 0 && id < total) next = gridDim.x + atomicAdd(a.counters, 1);  // the one after, while this one runs
            taken = i + 1;
            if (lane == 0) misc[kHeld + i % 8] = id;
            Unit u{};
            if (id < total) {
                u = unit_of(id);
                if (kCut && u.first > 0 && Shape<kCut>(u, qpt, per_unit).nt == 0) {  // (no query sees this piece)
                    --i;
                    continue;
                }
            }
            if (i >= kSlots) ok = wait(kUFree + i % kSlots, (i / kSlots - 1) & 1);
            if (!ok) break;
            if (lane == 0) {
                volatile Unit& s = queue[i % kSlots];
                s.q0 = u.q0, s.n = u.n, s.k0 = u.k0, s.m = u.m, s.head = u.head, s.seen = u.seen, s.more = u.more;
                if constexpr (kCut) s.first = u.first, s.len = u.len, s.slot = u.slot;
                bar_arrive(B(kUFull + i % kSlots));
            }
            __syncwarp();
            if (!u.more) break;
            const Shape<kCut> sh(u, qpt, per_unit);
            auto load_q = [&](int x) {
                if (sh.tiles[x] == 0) return;
                if (q_count[x] > 0 && !wait(kQFree + x, (q_count[x] - 1) & 1)) {
                    ok = false;
                    return;
                }
                if (lane == 0) bar_expect_tx(B(kQFull + x), Lt::kHalves * qpt * gh * 128);
                __syncwarp();
                if (lane < Lt::kHalves)
                    tma_4d(sbase + Lt::kQ + x * Lt::kTile + lane * kHalf, &mq, lane, u.head * gh, u.q0 + x * qpt, B(kQFull + x));
                ++q_count[x];
            };
            auto load_kv = [&](const CUtensorMap* map, int j) {
                const int s = stage % kStages;
                if (stage >= kStages && !wait(kFree + s, (stage / kStages - 1) & 1)) {
                    ok = false;
                    return;
                }
                if (lane == 0) bar_expect_tx(B(kFull + s), Lt::kTile);
                __syncwarp();
                if (lane < Lt::kHalves)
                    tma_4d(sbase + Lt::kRing + s * Lt::kTile + lane * kHalf, map, lane, u.head, u.k0 + j * kKeys, B(kFull + s));
                ++stage;
            };
            if (sh.nt > 0) load_q(0);
            for (int j = 0; j < sh.nt && ok; ++j) {
                load_kv(&mk, j);
                if (j == 0 && ok) load_q(1);
                if (ok) load_kv(&mv, j);
            }
        }
        if (!ok && lane == 0) fail();
        if (lane == 0) {  // (the one after is this CTA's, too)
            misc[kHeld + taken % 8] = next;
            misc[kTaken] = taken + 1;
        }
        // the copies under way land before the CTA ends
        for (int k = stage - 1; k >= 0 && k >= stage - kStages; --k) bar_wait(B(kFull + k % kStages), (k / kStages) & 1);
        for (int x = 0; x < 2; ++x)
            if (q_count[x] > 0) bar_wait(B(kQFull + x), (q_count[x] - 1) & 1);
        // the last CTA to finish leaves the counters at zero
        if (lane == 0) {
            __threadfence();
            if (atomicAdd(a.counters + 1, 1) == static_cast<int>(gridDim.x) - 1) {
                if (ok) a.counters[0] = 0;  // (this CTA saw the list's end)
                else misc[kUntaken] = gridDim.x + atomicExch(a.counters, 0);
                a.counters[1] = 0;
            }
        }
    } else if (warp == kIssuer || warp == kIssuer + 1) {
        // ------------------------------------------- MMA issuers: A's and B's
        // The whole warp walks through the list, so that descriptors and addresses are uniform values;
        // one lane issues.  (A single lane's walk issued an MMA every 85 cycles, of the 64 that one takes.)
        const int x = __shfl_sync(0xFFFFFFFFu, warp - kIssuer, 0);
        uint32_t leader_;
        asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(leader_));
        const bool leader = leader_ != 0;
        const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
        const uint32_t ts = tm + x * kKeys, to = tm + 2 * kKeys + x * kDim;
        const uint64_t dq = sdesc(sbase + Lt::kQ + x * Lt::kTile, 16), dk = sdesc(sbase + Lt::kRing, 16);
        const uint64_t dv = sdesc(sbase + Lt::kRing + Lt::kTile, kHalf);
        constexpr uint64_t kPair = (2 * Lt::kTile) >> 4;  // from a K (V) stage to the next
        int units = 0, q_count = 0, p_count = 0, o_count = 0;
        int c = -1, j = -1, tiles = 0, nt = 0;  // key tile of all, of the unit; the row tile's, the unit's
        auto await = [&](int i, int parity) -> bool { return __all_sync(0xFFFFFFFFu, wait(i, parity)); };
        auto arrive = [&](int i) {
            if (leader) bar_arrive(B(i));
        };
        // the next key tile of this row tile, in another unit: 1, 0 at the list's end, -1 on failure
        auto next_unit = [&]() -> int {
            for (;;) {
                for (++j; j < nt; ++j) {  // tiles that only the other row tile multiplies
                    ++c;
                    const int st = 2 * (c & 1), ph = (c >> 1) & 1;
                    for (int v = 0; v < 2; ++v) {
                        if (!await(kFull + st + v, ph)) return -1;
                        arrive(kFree + st + v);
                    }
                }
                if (!await(kUFull + units % kSlots, (units / kSlots) & 1)) return -1;
                const Unit u = take(units);
                __syncwarp();
                arrive(kUFree + units % kSlots);
                ++units;
                const Shape<kCut> sh(u, qpt, per_unit);
                const int more = __shfl_sync(0xFFFFFFFFu, u.more, 0);
                if (!more) return 0;
                tiles = __shfl_sync(0xFFFFFFFFu, sh.tiles[x], 0), nt = __shfl_sync(0xFFFFFFFFu, sh.nt, 0), j = -1;
                if (tiles > 0) {
                    j = 0;
                    ++c;
                    return 1;
                }
            }
        };
        // One issuer's products at a time, so that a row tile's come as fast as they can while the other
        // tile's softmax runs (side by side both tiles would wait for both, and the tensor core for them)
        auto begin = [&]() -> bool {
            for (uint32_t k = 0; k < kSpin; ++k) {
                int got = 0;
                if (leader) got = atomicCAS(turn, 0, 1) == 0;
                if (__any_sync(0xFFFFFFFFu, got)) return true;
                if ((k & 255) == 255 && __any_sync(0xFFFFFFFFu, *abort_flag)) return false;
            }
            return false;
        };
        auto end = [&]() {
            if (leader) atomicExch(turn, 0);
        };
        auto scores = [&](int t) {  // S of key tile t
            const uint64_t k = dk + (t & 1) * kPair;
            if (leader) {
#pragma unroll
                for (int ks = 0; ks < kDim / 16; ++ks) {
                    const uint32_t off = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
                    mma_bf16(ts, dq + off, k + off, idesc(kKeys, 0), ks > 0 ? 1u : 0u);
                }
            }
        };
        bool ok = true;
        int more = next_unit();
        if (x == 0 && more > 0 && a.test_wait_polls >= 0 && (a.test_wait_cta < 0 || a.test_wait_cta == static_cast<int>(blockIdx.x)) &&
            !__all_sync(0xFFFFFFFFu, wait(kFull + 2 * (c & 1), (c >> 1) & 1, a.test_wait_polls)))
            more = -1;  // (under test: the first wait for a key tile)
        bool fresh = true;  // S of the current tile is not issued yet
        while (more > 0) {
            if (fresh) {
                ok = await(kQFull + x, q_count++ & 1) && await(kFull + 2 * (c & 1), (c >> 1) & 1) && begin();
                if (!ok) break;
                fence_after();
                scores(c);
                end();
                if (leader) {
                    mma_commit(B(kSFull + x));
                    mma_commit(B(kFree + 2 * (c & 1)));
                    if (tiles == 1) mma_commit(B(kQFree + x));
                }
                __syncwarp();
                fresh = false;
            }
            // P V of this tile, then S of the unit's next
            const int st = 2 * (c & 1) + 1;
            const uint64_t v = dv + (c & 1) * kPair;
            const bool last = j == tiles - 1;
            ok = await(kFull + st, (c >> 1) & 1) && (j > 0 || o_count == 0 || await(kOFree + x, (o_count - 1) & 1)) &&
                 (last || await(kFull + 2 * ((c + 1) & 1), ((c + 1) >> 1) & 1)) && await(kPFull + x, p_count & 1) && begin();
            if (!ok) break;
            ++p_count;
            fence_after();
            if (leader) {
#pragma unroll
                for (int ks = 0; ks < kKeys / 16; ++ks)
                    mma_bf16_ta(to, ts + (ks & 4) * (kKeys / 8) + (ks & 3) * 8, v + ((ks * 16 * 128) >> 4), idesc(kDim, 1), (j > 0 || ks > 0) ? 1u : 0u);
            }
            if (!last) scores(c + 1);
            end();
            if (leader) {
                if (last) {
                    mma_commit(B(kOFull + x));
                } else {
                    mma_commit(B(kSFull + x));
                    mma_commit(B(kFree + 2 * ((c + 1) & 1)));
                    if (j == tiles - 2) mma_commit(B(kQFree + x));
                }
                mma_commit(B(kFree + st));
            }
            __syncwarp();
            if (last) {
                ++o_count;
                more = next_unit();
                fresh = true;
            } else {
                ++c;
                ++j;
            }
        }
        if (lane == 0 && (!ok || more < 0)) fail();
        if (leader) {
            mma_commit(B(kDone + x));  // every product, and every signal of one, has landed before the CTA ends
            if (!bar_wait(B(kDone + x), 0)) fail();
        }
        __syncwarp();
    } else if (warp < kSoftmaxWarps) {
        // -------------------------------------------------- softmax and output
        const int x = warp >> 3, hf = (warp >> 2) & 1, m = 32 * (warp & 3) + lane;  // row tile, half of the keys, row
        constexpr int kMine = kKeys / 2, kCols = kDim / 2;                          // this thread's keys, and columns of O
        const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lane_off + x * kKeys, to = tmem + lane_off + 2 * kKeys + x * kDim + hf * kCols;
        const float qk = a.scale_log2;
        const int qi = m / gh, hi = m % gh;  // query of the tile, head of the group
        int s_count = 0, o_count = 0, base = 0;
        bool ok = true;
        // A row's two threads tell each other a value: {value, number of the telling}.  (No named barrier: a
        // wait for it would have no end if the other warp had given up.)
        const uint32_t say = sbase + Lt::kSay + ((x * 2 + hf) * kRows + m) * 8;
        const uint32_t its_say = sbase + Lt::kSay + ((x * 2 + 1 - hf) * kRows + m) * 8;
        // Tiles' maxima take two places in turn: a thread may be a tile ahead of the other, but not two, as products wait
        // for both.
        auto tell = [&](int slot, float mine, int number) {
            asm volatile("st.volatile.shared.v2.b32 [%0], {%1, %2};\n" ::"r"(say + slot * 4 * kRows * 8),
                         "r"(__float_as_uint(mine)), "r"(number)
                         : "memory");
        };
        auto hear = [&](int slot, int number, float& other) -> bool {
            for (uint32_t k = 0; k < kSpin; ++k) {
                uint32_t bits, n;
                asm volatile("ld.volatile.shared.v2.b32 {%0, %1}, [%2];\n" : "=r"(bits), "=r"(n) : "r"(its_say + slot * 4 * kRows * 8) : "memory");
                if (__all_sync(0xFFFFFFFFu, n == static_cast<uint32_t>(number))) {
                    other = __uint_as_float(bits);
                    return true;
                }
                if ((k & 255) == 255 && __any_sync(0xFFFFFFFFu, *abort_flag)) return false;
            }
            return false;
        };
        int i = 0;
        for (; ok; ++i) {
            if (!__all_sync(0xFFFFFFFFu, wait(kUFull + i % kSlots, (i / kSlots) & 1))) {
                ok = false;
                break;
            }
            // (a unit's place in the queue is kept while it is worked on: what is needed once is read when it is)
            const volatile Unit& slot = queue[i % kSlots];
            if (!slot.more) break;
            int lim, tiles, place0, m_keys;  // keys that the row sees, key tiles of the row tile and of the units before, keys
            bool busy, valid;
            {
                const Unit u = take(i);
                const Shape<kCut> sh(u, qpt, per_unit);
                place0 = base;
                m_keys = u.m;
                base += sh.nt;
                const int query = x * qpt + qi;
                valid = x < per_unit && qi < qpt && query < u.n;
                busy = __any_sync(0xFFFFFFFFu, valid);
                lim = u.seen + min(query, u.n - 1);  // (no row: as another)
                tiles = sh.tiles[x];
            }
            float m_used = -INFINITY, m_next = -INFINITY, l = 0.f;  // base of this tile's weights, of the next one's
            for (int j = 0; j < tiles; ++j) {
                if (!__all_sync(0xFFFFFFFFu, wait(kSFull + x, s_count & 1))) {
                    ok = false;
                    break;
                }
                ++s_count;
                fence_after();
                const int key0 = j * kKeys + hf * kMine;  // this thread's first key
                float mx = -INFINITY, its = -INFINITY, m_own = 0.f, l0 = 0.f;
                if (busy) {
                    // a row sees its first `mine` keys; all rows of the warp see the first `all`, none one from `any` on
                    const int mine = min(max(lim - key0, 0), kMine);
                    const int all = __reduce_min_sync(0xFFFFFFFFu, mine), any = __reduce_max_sync(0xFFFFFFFFu, mine);
                    const bool full = all == kMine;
                    // The base of this tile's weights 2^(score - base) was agreed on after the tile before, so that no
                    // thread waits here for its row's maximum: they tell each other theirs when the weights are made.
                    if (j > 0 && __any_sync(0xFFFFFFFFu, m_next != m_used)) {  // ("S j done": P V j - 1 is, too)
                        const float alpha = m_used == -INFINITY ? 0.f : ex2(m_used - m_next);
#pragma unroll 1
                        for (int c = 0; c < kCols; c += 8) tmem_scale8(to + c, alpha);
                        asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
                        l *= alpha;
                        m_used = m_next;
                    }
                    float l1 = 0.f;
                    bool made = false;
                    if (j > 0 && full && qk > 0.f) {
                        // one pass: the maximum beside the weights, which are written unless one was far above the base
                        uint32_t v[kMine];
#pragma unroll
                        for (int c = 0; c < kMine / 32; ++c) tmem_ld32_nowait(ts + hf * kMine + 32 * c, v + 32 * c);
                        asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
                        const float base2 = m_used == -INFINITY ? 0.f : m_used;
                        float m2[2] = {-INFINITY, -INFINITY};
#pragma unroll
                        for (int k = 0; k < kMine / 2; ++k) {
                            const float y0 = __uint_as_float(v[2 * k]), y1 = __uint_as_float(v[2 * k + 1]);
                            m2[k & 1] = max3(m2[k & 1], y0, y1);
                            float x0, x1;
                            fma2(x0, x1, y0, y1, qk, qk, -base2, -base2);
                            const float p0 = ex2(x0), p1 = ex2(x1);
                            add2(l0, l1, l0, l1, p0, p1);
                            v[k] = bf16x2(p0, p1);
                        }
                        mx = fmaxf(m2[0], m2[1]) * qk;
                        // (equal: a base from kLarge on; scores below such a one are so by a step, and weigh nothing)
                        made = !__any_sync(0xFFFFFFFFu, mx >= m_used + kFar);
                        if (made) {
                            m_own = m_used;
                            tmem_st16_nowait(ts + hf * kMine, v);
                            tmem_st16_nowait(ts + hf * kMine + 16, v + 16);
                        } else {
                            mx = -INFINITY, l0 = l1 = 0.f;
                        }
                    }
                    if (!made) {
                        {  // the maximum first, from a load of its own: the weights' loop then keeps few registers
                            uint32_t v[kMine];
#pragma unroll
                            for (int c = 0; c < kMine / 32; ++c) tmem_ld32_nowait(ts + hf * kMine + 32 * c, v + 32 * c);
                            asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
                            if (full && qk > 0.f) {
                                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                                for (int k = 0; k < kMine; k += 2)
                                    m4[(k >> 1) & 3] = max3(m4[(k >> 1) & 3], __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
                                mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * qk;
                            } else {
#pragma unroll
                                for (int c = 0; c < kMine; c += 16) {
                                    if (c >= any) continue;
                                    float m2[2] = {-INFINITY, -INFINITY};
#pragma unroll
                                    for (int k = c; k < c + 16; ++k)
                                        m2[k & 1] = fmaxf(m2[k & 1], k < mine ? __uint_as_float(v[k]) * qk : -INFINITY);
                                    mx = max3(mx, m2[0], m2[1]);
                                }
                            }
                        }
                        if (j == 0) {  // (the unit's first tile has no tile before)
                            tell(2 * (s_count & 1), mx, s_count);
                            if (!hear(2 * (s_count & 1), s_count, its)) {
                                ok = false;
                                break;
                            }
                            m_used = fmaxf(mx, its);
                        }
                        // far above the base: a base of this thread's own, until both know better
                        m_own = mx > m_used + kFar ? above(m_used, mx) : m_used;
                        const float base2 = m_own == -INFINITY ? 0.f : m_own;
                        // P as BF16 pairs, 16 columns at a time over this thread's own scores, which it has read by then
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t v[32];
                            if (32 * c >= any) {  // nobody's keys
#pragma unroll
                                for (int k = 0; k < 16; ++k) v[k] = 0u;
                            } else {
                                tmem_ld32_nowait(ts + hf * kMine + 32 * c, v);
                                asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
                                float q_ = qk;
                                if (__any_sync(0xFFFFFFFFu, fabsf(base2) >= kLarge)) {
                                    // as the largest score was rounded, before the base is taken away
                                    q_ = 1.f;
#pragma unroll
                                    for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__fmul_rn(__uint_as_float(v[k]), qk));
                                }
                                auto weights = [&](auto hide) {
#pragma unroll
                                    for (int k = 0; k < 16; ++k) {
                                        float x0, x1;
                                        fma2(x0, x1, __uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]), q_, q_, -base2, -base2);
                                        if (hide()) {  // a weight of 0 for what the row does not see
                                            x0 = 32 * c + 2 * k < mine ? x0 : -INFINITY;
                                            x1 = 32 * c + 2 * k + 1 < mine ? x1 : -INFINITY;
                                        }
                                        const float p0 = ex2(x0), p1 = ex2(x1);
                                        add2(l0, l1, l0, l1, p0, p1);
                                        v[k] = bf16x2(p0, p1);
                                    }
                                };
                                if (32 * c + 32 <= all) weights(std::false_type());
                                else weights(std::true_type());
                            }
                            tmem_st16_nowait(ts + hf * kMine + 16 * c, v);
                        }
                    }
                    l0 += l1;
                    const bool far = j > 0 && !made && __any_sync(0xFFFFFFFFu, mx > m_used + kFar);
                    asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
                    if (j > 0) {
                        fence_before();
                        tell(2 * (s_count & 1), mx, s_count);  // (told: its weights are written)
                        if (far) {
                            // One warp of the two brings the rows' weights, and O, to a common base; the first if it
                            // has such a row
                            if (!hear(2 * (s_count & 1), s_count, its)) {
                                ok = false;
                                break;
                            }
                            fence_after();
                            const float top = fmaxf(mx, its);
                            if (hf == 0 || !__any_sync(0xFFFFFFFFu, its > m_used + kFar)) {
                                const float m_new = top > m_used + kFar ? above(m_used, top) : m_used;
                                const float m_its = its > m_used + kFar ? above(m_used, its) : m_used;
                                auto f = [&](float from) { return from == m_new ? 1.f : from == -INFINITY ? 0.f : ex2(from - m_new); };
#pragma unroll 1
                                for (int c = 0; c < kMine / 2; c += 8) {
                                    tmem_scale8_bf16(ts + hf * kMine + c, f(m_own));
                                    tmem_scale8_bf16(ts + (1 - hf) * kMine + c, f(m_its));
                                }
#pragma unroll 1
                                for (int c = 0; c < kDim; c += 8) tmem_scale8(to - hf * kCols + c, f(m_used));
                                asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
                            }
                        }
                    }
                }
                // V rows behind the sequence: zero (they are another's, or unwritten, and may hold NaN), before
                // P is ready; A and B both see to it
                const int there = m_keys - j * kKeys;
                if (there < kKeys) {
                    const int c = place0 + j, s = 2 * (c & 1) + 1;
                    if (!__all_sync(0xFFFFFFFFu, wait(kFull + s, (c >> 1) & 1))) {
                        ok = false;
                        break;
                    }
                    uint8_t* vs = smem + Lt::kRing + s * Lt::kTile;
                    const int gone = kKeys - there;  // whole 128-byte rows: the swizzle does not matter
                    for (int e = (tid & 255); e < Lt::kHalves * gone * 8; e += 256) {
                        const int h = e / (gone * 8), r = there + e % (gone * 8) / 8;
                        *reinterpret_cast<uint4*>(vs + h * kHalf + r * 128 + e % 8 * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_async_smem();
                }
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(B(kPFull + x));
                if (busy) {  // the next tile's base, while the products run
                    if (j > 0 && !hear(2 * (s_count & 1), s_count, its)) {
                        ok = false;
                        break;
                    }
                    const float top = fmaxf(mx, its);
                    if (__any_sync(0xFFFFFFFFu, top > m_used + kFar)) {
                        const float m_new = top > m_used + kFar ? above(m_used, top) : m_used;
                        // (from no base: l is 0, or NaN where the row has seen a key that is)
                        l = m_used == m_new || m_used == -INFINITY ? l : l * ex2(m_used - m_new);
                        l0 = m_own == m_new ? l0 : l0 * ex2(m_own - m_new);
                        m_used = m_new;
                    }
                    m_next = top > m_used + 8.f ? above(m_used, top) : m_used;
                    l += l0;
                }
            }
            if (!ok) break;
            // the row's place in the output, counted in heads; -1: no row
            const int64_t row = valid ? static_cast<int64_t>(slot.q0 + x * qpt + qi) * a.num_q_heads + slot.head * gh + hi : -1;
            // the row tile's pieces, and this one's place among them
            int pieces = 1, before = 0, len = INT_MAX, slot0 = 0;
            if constexpr (kCut) before = slot.first, len = slot.len, slot0 = slot.slot;
            if (len != INT_MAX) {
                const int n = min(slot.n - x * qpt, qpt), sees = slot.seen + x * qpt;
                if (n > 0) pieces = (max(0, (sees + n - 1 + kKeys - 1) / kKeys) + before + len - 1) / len;
                if (tid % 256 == 0 && before == 0 && pieces > 1)
                    a.tiles[2 * slot0 + x] = make_int4(pieces, slot.q0 + x * qpt, n | slot.head << 8, sees);
            }
            // Chunks of 16 bytes are stored with kChunks lanes on a row: lane g kChunks + c has chunk c of the
            // rows of the group's lanes.  (A row to a lane took 4000 cycles of a unit: a line for each lane of a store.)
            constexpr int kChunks = kCols / 8;
            auto store = [&](const uint4* w) {
                const int own = lane % kChunks;
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + hf * kCols + own * 8;
#pragma unroll
                for (int k = 0; k < kChunks; ++k) {
                    const int64_t r = __shfl_sync(0xFFFFFFFFu, row, lane - own + k);
                    if (r >= 0) *reinterpret_cast<uint4*>(out + r * kDim) = w[k];
                }
            };
            __syncwarp();
            if (lane == 0) bar_arrive(B(kUFree + i % kSlots));
            if (tiles == 0) {  // no key is seen
                uint4 w[kChunks] = {};
                if (before == 0) store(w);
                continue;
            }
            // (a base that was to change stays: both threads' l and O are in this one)
            float l_other = 0.f;
            if (busy) tell(1, l, s_count);
            if ((busy && !hear(1, s_count, l_other)) || !__all_sync(0xFFFFFFFFu, wait(kOFull + x, o_count & 1))) {
                ok = false;
                break;
            }
            ++o_count;
            fence_after();
            uint32_t o[kCols];
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c) tmem_ld32_nowait(to + 32 * c, o + 32 * c);
            asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(B(kOFree + x));  // the next unit's first P V may overwrite it
            l += l_other;
            if (pieces > 1) {  // a part of each row's sums: the pieces are joined by the next kernel
                const int64_t part_ = (static_cast<int64_t>(slot0) + before / len * a.num_kv_heads) * kSoftmaxWarps + warp;
                float4* po = a.part_o + part_ * (kCols / 4) * 32 + lane;
#pragma unroll
                for (int k = 0; k < kCols / 4; ++k)
                    po[32 * k] = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]), __uint_as_float(o[4 * k + 2]),
                                             __uint_as_float(o[4 * k + 3]));
                a.part_ml[part_ * 32 + lane] = make_float2(m_used, l);
                continue;
            }
            const float inv = 1.f / l;
            uint4 w[kChunks];
#pragma unroll
            for (int k = 0; k < kChunks; ++k) {
                uint32_t y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[e] = lim > 0 ? bf16x2(__uint_as_float(o[8 * k + 2 * e]) * inv, __uint_as_float(o[8 * k + 2 * e + 1]) * inv) : 0u;
                w[k] = make_uint4(y[0], y[1], y[2], y[3]);
            }
            // chunk c of lane r to lane c, place r, of the group: a transposition by halves
#pragma unroll
            for (int d = kChunks / 2; d > 0; d >>= 1) {
                const bool up = lane & d;
#pragma unroll
                for (int k = 0; k < kChunks; ++k) {
                    if (k & d) continue;
                    auto swap = [&](uint32_t& lo, uint32_t& hi2) {
                        const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? lo : hi2, d);
                        if (up) lo = got;
                        else hi2 = got;
                    };
                    swap(w[k].x, w[k + d].x);
                    swap(w[k].y, w[k + d].y);
                    swap(w[k].z, w[k + d].z);
                    swap(w[k].w, w[k + d].w);
                }
            }
            store(w);
        }
        if (lane == 0) misc[kStopped + warp] = ok ? INT_MAX : i;
        if (!ok && lane == 0) fail();
    }
    fence_before();  // every role has left its waits
    __syncthreads();
    fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512) : "memory");

    // Rows that are lost become NaN: of the units that this CTA had in hand when it gave up, and, where every CTA did, of
    // those that none took.
    if (*abort_flag == 0 && misc[kUntaken] == INT_MAX) return;
    const int total = cum[a.num_seqs] * a.num_kv_heads;
    int first = INT_MAX;
    for (int w = 0; w < kSoftmaxWarps; ++w) first = min(first, misc[kStopped + w]);
    for (int i = first; i < misc[kTaken]; ++i)
        if (misc[kHeld + i % 8] < total) lose_unit<kDim, kCut>(a, plan, misc[kHeld + i % 8], per_unit);
    for (int id = misc[kUntaken]; id < total; ++id) lose_unit<kDim, kCut>(a, plan, id, per_unit);
}

// The pieces of row tiles, joined in their order.  A CTA has one row tile (or none: the place's units were not cut), a
// thread one row and a quarter of half of its columns: as the pieces lie, so that a warp's loads are whole lines.
template <int kDim>
__global__ void __launch_bounds__(kJoinThreads) prompt_join_kernel(const PromptArgs a) {
    constexpr int kQuads = kDim / 8, kMine = kQuads / 4, kAtOnce = 8 / kMine;  // of a half row, of a thread; pieces under way
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int place = blockIdx.x;
    const int4 tile = a.tiles[place];
    const int pieces = tile.x;
    if (pieces == 0) return;
    __syncthreads();
    if (threadIdx.x == 0) a.tiles[place] = make_int4(0, 0, 0, 0);  // (for the next call, of either operator)
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 7, quarter = threadIdx.x >> 8;
    const int gh = a.num_q_heads / a.num_kv_heads, row = 32 * (w & 3) + lane, qi = row / gh;
    if (qi >= (tile.z & 255)) return;
    const int64_t part = static_cast<int64_t>(place / 2) * kSoftmaxWarps + place % 2 * 8 + w;
    const int64_t step = static_cast<int64_t>(a.num_kv_heads) * kSoftmaxWarps;  // from a piece to the next
    const float2* ml = a.part_ml + part * 32 + lane;
    const float4* po = a.part_o + (part * kQuads + quarter * kMine) * 32 + lane;
    float top = -INFINITY;
#pragma unroll 8
    for (int p = 0; p < pieces; ++p) top = fmaxf(top, ml[p * step * 32].x);
    if (top == -INFINITY) top = 0.f;
    float l = 0.f, o[kMine][4] = {};
    for (int p0 = 0; p0 < pieces; p0 += kAtOnce) {
        float2 s[kAtOnce];
        float4 y[kAtOnce][kMine];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int64_t p = min(p0 + i, pieces - 1);
            s[i] = ml[p * step * 32];
            if (p0 + i >= pieces) s[i].x = -INFINITY;
#pragma unroll
            for (int k = 0; k < kMine; ++k) y[i][k] = po[(p * step * kQuads + k) * 32];
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const float f = ex2(s[i].x - top);
            // (a piece that weighs nothing, or of which the row sees nothing; a sum of NaN tells of a key that is)
            if (f == 0.f && s[i].y == s[i].y) continue;
            l = fmaf(f, s[i].y, l);
#pragma unroll
            for (int k = 0; k < kMine; ++k) {
                o[k][0] = fmaf(f, y[i][k].x, o[k][0]);
                o[k][1] = fmaf(f, y[i][k].y, o[k][1]);
                o[k][2] = fmaf(f, y[i][k].z, o[k][2]);
                o[k][3] = fmaf(f, y[i][k].w, o[k][3]);
            }
        }
    }
    const float inv = 1.f / l;
    const bool sees = tile.w + qi > 0;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                         ((static_cast<int64_t>(tile.y) + qi) * a.num_q_heads + (tile.z >> 8) * gh + row % gh) * kDim +
                         (w >> 2) * (kDim / 2) + quarter * kMine * 4;
#pragma unroll
    for (int k = 0; k < kMine; ++k)
        reinterpret_cast<uint2*>(out)[k] =
            sees ? make_uint2(bf16x2(o[k][0] * inv, o[k][1] * inv), bf16x2(o[k][2] * inv, o[k][3] * inv)) : make_uint2(0u, 0u);
}

// Descriptor of packed rows [rows][heads][kDim] as {64 columns, column halves, heads, rows}.
bool encode_rows(CUtensorMap* map, const void* base, int dim, int64_t rows, int heads, int64_t stride, int box_heads,
                 int box_rows) {
    const uint64_t dims[4] = {64, static_cast<uint64_t>(dim / 64), static_cast<uint64_t>(heads), static_cast<uint64_t>(rows)};
    const uint64_t row = rows > 1 ? static_cast<uint64_t>(stride) : static_cast<uint64_t>(heads) * dim;
    const uint64_t strides[3] = {128, static_cast<uint64_t>(dim) * 2, row * 2};
    const uint32_t box[4] = {64, 1, static_cast<uint32_t>(box_heads), static_cast<uint32_t>(box_rows)};
    return encode_map(map, 2, 4, base, dims, strides, box);
}

constexpr int kMostSms = 1000;  // whose row tiles' list has room among the workspace's zeros
static_assert(256 + kPieces * kMostSms * 2 * sizeof(int4) <= kWorkspaceZeros);
int grid_size() {
    const int n = num_sms();
    return n < 1 ? 148 : n < kMostSms ? n : kMostSms;
}

template <int kDim>
cudaError_t launch(const PromptArgs& a, cudaStream_t stream) {
    const int gh = a.num_q_heads / a.num_kv_heads, qpt = kRows / gh;
    CUtensorMap mq, mk, mv;
    if (!encode_rows(&mq, a.q, kDim, a.q_rows, a.num_q_heads, a.q_stride, gh, qpt) ||
        !encode_rows(&mk, a.k, kDim, a.k_rows, a.num_kv_heads, a.k_stride, 1, kKeys) ||
        !encode_rows(&mv, a.v, kDim, a.k_rows, a.num_kv_heads, a.v_stride, 1, kKeys))
        return cudaErrorNotSupported;
    const int sms = grid_size();
    // Keys may be cut where sequences are long enough on the whole, and the units of all rows are fewer than SMs, or a few
    // more than fill them a few times, with prefixes long enough for units to be of like length.
    const int64_t units = static_cast<int64_t>(a.q_rows) / (2 * qpt) * a.num_kv_heads;
    const bool cut = a.k_rows >= (kLeastPiece + kWorth) * kKeys && a.k_rows / a.num_seqs >= (kLeastPiece + kWorth) * kKeys / 2 &&
                     (units < sms || (units < 4 * sms && 2 * (units % sms) <= sms && a.k_rows / 3 >= a.q_rows));
    const auto kernel = cut ? prompt_tc_kernel<kDim, true> : prompt_tc_kernel<kDim, false>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<kDim>::kSmem);
    if (e != cudaSuccess) return e;
    // row tiles, times the key tiles that one may have
    const int64_t most = (static_cast<int64_t>(a.q_rows) / qpt + a.num_seqs) * a.num_kv_heads * (a.k_rows / kKeys + 1);
    const cudaError_t r = launch_dependent(kernel, dim3(static_cast<unsigned>(most < sms ? most : sms)), dim3(kThreads),
                                           Layout<kDim>::kSmem, stream, mq, mk, mv, a);
    if (r != cudaSuccess || !cut) return r;
    return launch_dependent(prompt_join_kernel<kDim>, dim3(2 * kPieces * sms), dim3(kJoinThreads), 0, stream, a);
}

}  // namespace

bool prompt_tc_fits(pkv_dtype t, int num_seqs, int q_rows, int num_q_heads, int num_kv_heads) {
    const int gh = num_q_heads / num_kv_heads;
    // (units are counted in 32 bits)
    return t == PKV_BF16 && gh <= kRows && num_seqs <= kPromptMaxSeqs &&
           (static_cast<int64_t>(q_rows) + num_seqs) * num_kv_heads <= INT32_MAX / 2;
}

// {counter of units, of CTAs}, for each row tile that is cut what the joining kernel needs, and its pieces' (maximum, sum)
// and O.
// (The counters and what the joining kernel needs, 64 bytes an SM, are the part that calls leave zero.)
size_t prompt_tc_workspace(int head_dim, uint8_t* base, PromptArgs* a) {
    const size_t pieces = static_cast<size_t>(kPieces * grid_size()), parts = pieces * kSoftmaxWarps;
    const size_t tiles = 256, ml = kWorkspaceZeros, o = ml + parts * 32 * sizeof(float2);
    if (a) {
        a->counters = reinterpret_cast<int32_t*>(base);
        a->tiles = reinterpret_cast<int4*>(base + tiles);
        a->part_ml = reinterpret_cast<float2*>(base + ml);
        a->part_o = reinterpret_cast<float4*>(base + o);
    }
    return o + parts * 32 * (head_dim / 2) * sizeof(float);
}

cudaError_t launch_prompt_tc(int head_dim, const PromptArgs& a, cudaStream_t stream) {
    return head_dim == 64 ? launch<64>(a, stream) : launch<128>(a, stream);
}

}  // namespace pkv
