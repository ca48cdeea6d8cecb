// Decode attention of a batch whose sequences share prefixes, each prefix
// read and multiplied once for its whole group ("How does TensorRT-LLM
// work?", "The paged KV cache": requests that begin with the same text point
// at the same blocks; "TensorRT-LLM, in depth", "The paged KV cache and block
// reuse").  BF16 and FP8 pools, head_dim 128.
//
// For sequence b of a group with P shared tokens the softmax splits at P:
//     out = (2^(s1 - M) o1 + 2^(s2 - M) o2) / (2^(s1 - M) + 2^(s2 - M)),
// (o1, s1) the normalised output and log2-sum-exp over tokens [0, P), (o2,
// s2) those over its own tokens [P, L), M = max(s1, s2).  The first part has
// the same keys for the whole group: its queries stack to rows of one matrix
// (n sequences x gh query heads per KV head), so the group's prefix is two
// matrix products instead of n x gh vector-matrix ones, and its bytes are
// read once instead of n times.  With 64 sequences over a 32768-token prefix
// that is 0.27 GB instead of 8.7 GB, and 35 GFLOP that the tensor cores take.
//
// Two launches.
//  * prefix_tc_kernel, 2 persistent CTAs per SM.  Its units are the 128-row
//    query tiles of a (group, KV head), over the group's shared tiles (64
//    tokens; a remainder of the prefix counts as own tokens), then the
//    (sequence, KV head) pairs, over the sequence's own tiles.  Every CTA plans
//    the call and takes an equal share of that list; each unit's piece leaves
//    O / l and its log2-sum-exp in the workspace.
//  * prefix_merge_kernel, one warp per output row, merges the pieces.
// The tile pipeline has 12 warps:
//  * two TMA producers, for K and for V: one box {64 columns, bs rows, 1 half}
//    per KV block and half, 128-byte swizzled: the K-major operand layout for K
//    and the MN-major one for V;
//  * two MMA threads: S = Q K^T (M 128, N 64 tokens, K 128), a tile ahead of the
//    softmax (and the copies of Q), and O += P V (N 128, K 64).
//    Their twelve instructions a tile set the pace of shared tiles; one thread
//    for both spent as long between them, on barriers, as issuing them;
//  * eight softmax warps, two threads per row (= TMEM lane): base 2, P back to
//    tensor memory as BF16 pairs (at most 2^-8 of each weight; the sum l is
//    taken in fp32 before that rounding), the running maximum moved only when
//    it grows by more than 8, so that O is seldom rescaled.
// FP8 pools: the tensor cores multiply K as stored (kind f8f6f4, E4M3
// operands); Q enters as the sum of two E4M3 terms, so S is two passes over K's
// 128 columns, 32 a step: as many instructions as for BF16.  The weights need
// more range than E4M3 has: below 2^-15 of a row's largest a sum of two E4M3
// terms is zero, and with one key 11 nats above 8192 others nine tenths of the
// output were lost.  Hence P is FP16, and the softmax warps write each V tile as
// FP16 (exactly) to shared memory for PV.  (That takes 4 us more than two E4M3
// terms on prefixes or own tokens alone, 6 to 7 %, and 4 us less where both are
// mixed.)
// Every wait at an mbarrier is bounded; a CTA whose wait expires sets
// PKV_ERRBIT_TIMEOUT, makes its pieces NaN, waits for its copies and products in
// flight, frees its TMEM and leaves.  (Only the pairs' named barriers have no
// bound of their own: see pair_any.)
//
// Measured (calls back to back in a graph; 32 query over 8 KV heads; "floor" is
// bytes at the measured copy rate):
//   64 sequences, 32768 shared tokens, up to 1024 own   64 us, floor 40 us
//   the same prefix alone                               46 us, floor 20 (products at the measured rate: 18)
//   64 sequences, 2048 shared, 128 to 2048 own          61 us, floor 43.5
//   64 sequences, 2048 own tokens, nothing shared       88 us, floor 79.5 (6.1 TB/s)
//   55 in 8 groups, FP8, 1024 to 8192 shared            49 us, floor 20
//   4 sequences, 512 shared, up to 64 own               12 us
// (paged_decode_attention: 622, 597, 79, 86, 104 and 21.6 us.)  What bounds a
// shared tile of a BF16 pool is the chain S issued (900 cycles of the S thread,
// two CTAs side by side) - done (500) - taken to registers (270) - told
// (100): 1870 cycles a tile and CTA, tensor pipe active 42 %; of an FP8 pool the
// softmax (250 to load, 850 maxima and exponentials, then the weights and the V
// tile).
// A call adds 2.5 us of plan, 2 until the first tiles land, and the merge's 3.
#include <cuda.h>

#include <atomic>
#include <climits>

#include "step_internal.h"
#include "tc_common.cuh"

namespace pkv {
namespace {

constexpr int kSoftmaxWarps = 8;
constexpr int kSoftmax = 32 * kSoftmaxWarps;
// softmax warps, then:
constexpr int kWarpK = kSoftmaxWarps, kWarpS = kWarpK + 1, kWarpV = kWarpK + 2, kWarpPv = kWarpK + 3;
constexpr int kThreads = kSoftmax + 128;
constexpr int kRows = kPrefixRows;
constexpr int kTok = 64;
constexpr int kDim = 128;
constexpr int kNS = 2;                        // P buffers, stages of the K ring and of the V ring
constexpr int kQHalf = kRows * 128;           // one 64-column half of the Q tile
constexpr int kHalfBytes = kTok * 128;        // one 64-column half of a K or V tile
constexpr int kKVOff = 2 * kQHalf;
constexpr int kStageBytes = 4 * kHalfBytes;   // K + V
constexpr int kRawBytes = kTok * kDim;        // FP8 pools: a K or V tile, [64 rows][128 bytes]
constexpr int kWideOff = kKVOff + kNS * 2 * kRawBytes;  // and behind their rings V tiles in FP16, as BF16 ones lie
static_assert(kNS * (2 * kRawBytes + 2 * kHalfBytes) == kNS * kStageBytes, "64 KB either way");
constexpr int kAlignSlack = 1024;
static_assert(12 * kPrefixMaxSeqs + 24 * kPrefixMaxGroups <= kNS * kStageBytes, "the plan fits into the ring");
// Tensor memory: the scores of one tile, two P buffers, O.  The softmax takes the
// scores to registers at once, so S k + 1 waits for that and for nothing behind
// it (P written over its scores in one of two score buffers made it wait for PV
// k - 1).
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kPCol = kTok, kPCols = kTok / 2;
constexpr uint32_t kOCol = kPCol + kNS * kPCols;
static_assert(kOCol + kDim == kTmemCols, "tensor memory");

enum Bar { kQReady, kQFree, kOFree, kDone, kSRead, kSFull, kPFull = kSFull + kNS, kPvDone = kPFull + kNS, kKFull = kPvDone + kNS,
           kVFull = kKFull + kNS,
           // (kSRead: the scores are in registers, S may be written again)
           // FP8 pools: Q split into E4M3 terms, V stages that the softmax warps have read
           kQOp = kVFull + kNS, kVEmpty, kNumBars = kVEmpty + kNS };
constexpr int kBarOff = kKVOff + kNS * kStageBytes;
constexpr int kExOff = kBarOff + (8 * kNumBars + 8 + 63) / 64 * 64;  // the two threads of a row meet here: maxima
constexpr int kSumOff = kExOff + 2 * kRows * 4;                        // and sums, [2][kRows] floats each
// The units of this CTA's range, as far as they fit (else the workspace's copy).
constexpr int kSeqCache = 1024, kGroupCache = 128;
constexpr int kQMaxOff = kSumOff + 2 * kRows * 4;  // and, FP8 pools, the largest |q|, [2][kRows] ints
constexpr int kGroupOff = kQMaxOff + 2 * kRows * 4;
constexpr int kSeqOff = kGroupOff + 16 * kGroupCache;
constexpr int kSmem = kSeqOff + 8 * kSeqCache + kAlignSlack;
static_assert(kSmem <= 115712, "two CTAs per SM");

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t b) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(b)
        : "memory");
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t b) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(b)
        : "memory");
}
// 16 consecutive TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(a),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}
// 64 TMEM columns of 16 lanes: thread 4 r + c gets columns 8 j + 2 c, + 1 of
// lane r in v[4 j], v[4 j + 1] and of lane r + 8 in v[4 j + 2], v[4 j + 3].
__device__ __forceinline__ void tmem_ld_16x64(uint32_t a, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(a));
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}
// Instruction descriptor with operand formats 0, otherwise as idesc(): E4M3 x
// E4M3 -> F32 for kind f8f6f4, F16 x F16 -> F32 for kind f16.
constexpr uint32_t idesc0(int n, int b_mn) { return idesc(n, b_mn) & ~((1u << 7) | (1u << 10)); }
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}
// Four values up to 448 as the sum of two E4M3 terms: hi = rn(x), lo = rn(x -
// hi), x rounded to FP16 first.  Exact for 8-bit significands whose last bit is
// at least 2^-9; else off by at most 2^-8 of x (two halved steps of 2^-4, and
// 2^-11 for FP16), or 2^-10 where lo is subnormal.
__device__ __forceinline__ void split4(float x0, float x1, float x2, float x3, uint32_t& hi, uint32_t& lo) {
    asm("{\n .reg .b16 a, b, c, d;\n .reg .b32 p, q, r, s;\n"
        " cvt.rn.satfinite.e4m3x2.f32 a, %3, %2;\n cvt.rn.satfinite.e4m3x2.f32 b, %5, %4;\n"
        " cvt.rn.f16x2.e4m3x2 p, a;\n cvt.rn.f16x2.e4m3x2 q, b;\n"
        " cvt.rn.f16x2.f32 r, %3, %2;\n cvt.rn.f16x2.f32 s, %5, %4;\n"
        " sub.rn.f16x2 r, r, p;\n sub.rn.f16x2 s, s, q;\n"
        " cvt.rn.satfinite.e4m3x2.f16x2 c, r;\n cvt.rn.satfinite.e4m3x2.f16x2 d, s;\n"
        " mov.b32 %0, {a, b};\n mov.b32 %1, {c, d};\n}\n"
        : "=r"(hi), "=r"(lo)
        : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
}
// Slack of the running maximum (log2), and the power of two that FP16 weights
// are scaled by: 2^(7 + 8) stays below 65504, and weights are normal numbers
// (half a step: 2^-11 of them) down to 2^-21 of the base, and not zero down to
// 2^-32.  BF16 has FP32's range.
constexpr float kSlack = 8.f;
template <bool kFp8>
constexpr float weight_shift_of() { return kFp8 ? 7.f : 0.f; }
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
// 16 E4M3 values as FP16, exactly: 0-7 to a, 8-15 to b.
__device__ __forceinline__ void widen16(const uint4& x, uint4& a, uint4& b) {
    auto four = [](uint32_t u, uint32_t& lo, uint32_t& hi) {
        asm("{\n .reg .b16 c, d;\n mov.b32 {c, d}, %2;\n cvt.rn.f16x2.e4m3x2 %0, c;\n cvt.rn.f16x2.e4m3x2 %1, d;\n}\n"
            : "=r"(lo), "=r"(hi)
            : "r"(u));
    };
    four(x.x, a.x, a.y);
    four(x.y, a.z, a.w);
    four(x.z, b.x, b.y);
    four(x.w, b.z, b.w);
}

// Rendezvous of the two warps that share 32 rows (named barrier 1 + id), and
// with it: does any of their threads say yes?  Both warps come to the same ones
// in the same order, in a CTA that gave up as well: which ones there are follows
// from the segments, the pair's common votes and nothing else, and every wait in
// between is bounded.
__device__ __forceinline__ bool pair_any(int id, bool yes) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 64, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"(yes ? 1u : 0u), "r"(1 + id)
        : "memory");
    return r != 0;
}
// A wait that also ends when another role of the CTA has given up (a poll lasts
// about 1.5 us, so within 0.1 ms).
__device__ __forceinline__ bool bar_wait_or(uint32_t b, uint32_t parity, const volatile int* abort_flag, uint32_t polls = kSpin) {
    for (uint32_t i = 0; i < polls; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(b), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((i & 63u) == 63u && *abort_flag) break;
    }
    return false;
}
__device__ __forceinline__ void pair_sync(int id) { asm volatile("barrier.cta.sync %0, 64;\n" ::"r"(1 + id) : "memory"); }

// ------------------------------------------------------------------- plan
// A unit costs more than its tiles: its Q rows to fetch (and, FP8 pools, to
// split), its piece to write out, the pipeline to refill.  The list is cut by
// cost, every unit being nt + unit_cost long; the last unit_cost places of it
// hold no tile.  Two tiles' worth for BF16 (64 sequences over 32768 shared
// tokens: 69, 64, 65 us with 1, 2, 3), five for FP8 (eight groups over
// 1024 to 8192 tokens: 52, 52, 50, 51 us with 3 to 6; prefixes alone and own
// tokens alone differ by less than 1 %).
int unit_cost_of(pkv_dtype kv) { return kv == PKV_FP8_E4M3 ? 5 : 2; }

// A list of cost T is cut into n = min(T, ctas) ranges, none of them empty, the
// first T % n one longer than the others.
struct Cut {
    int n, len, longer;
    __device__ __forceinline__ Cut(int T, int ctas) : n(T < ctas ? T : ctas), len(0), longer(0) {
        if (n > 0) {
            len = T / n;
            longer = T - len * n;
        }
    }
    __device__ __forceinline__ int start(int r) const { return r * len + min(r, longer); }
    __device__ __forceinline__ int of(int x) const {  // the range that x is in
        const int y = x - longer * (len + 1);
        return y < 0 ? x / (len + 1) : longer + y / len;
    }
};
// The range of this CTA.  The list begins with the shared tiles, which the
// tensor cores and the softmax bound, and ends with the own ones, which memory
// does: the two CTAs of an SM (c and c + ctas / 2, as blocks are handed out)
// get one of each, as far as there are.
__device__ __forceinline__ int my_range(int ctas) {
    const int c = static_cast<int>(blockIdx.x), half = ctas / 2;
    return c < half ? c : ctas - 1 - (c - half);
}

// The plan runs once per CTA, so its time is that of fetching its instructions
// (7 thousand cycles where the loops were unrolled): short code, rolled loops,
// and sequences and groups side by side, each by warps of their own.
constexpr int kSeqThreads = 256, kGroupThreads = kThreads - kSeqThreads;

// Exclusive sum of v over this thread's kind, sequences or groups; the totals of both.
__device__ __forceinline__ int plan_scan(int v, int* sums, int* seqs, int* groups) {
    constexpr int kWarps = kThreads / 32, kSeqWarps = kSeqThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    const int all = lane < kWarps ? sums[lane] : 0;
    const bool of_seq = lane < kSeqWarps;
    *seqs = __reduce_add_sync(0xFFFFFFFFu, of_seq ? all : 0);
    *groups = __reduce_add_sync(0xFFFFFFFFu, of_seq ? 0 : all);
    return x - v + __reduce_add_sync(0xFFFFFFFFu, lane < warp && of_seq == (warp < kSeqWarps) ? all : 0);
}

struct Start {
    int own, i, u, t, left;  // of this CTA's range: list half, group or sequence, unit, place in the unit, cost
    int seq0;                // the sequence cache's first entry
    int groups_cached;       // the group cache holds them all (else the workspace does)
    int pos, T;              // start of the range in the list, cost of the list
};

__device__ __forceinline__ int row_tiles(const PrefixArgs& a, int seqs) {
    return (seqs + a.seqs_per_tile - 1) / a.seqs_per_tile;
}

// What a thread fetches of the call's lengths or groups before anything else.
struct Early {
    int x, y, z;  // a length; or a group's first and last + 1 sequence and its prefix
};
__device__ __forceinline__ Early fetch_early(const PrefixArgs& a) {
    const int b = threadIdx.x, g = b - kSeqThreads;
    Early e{0, 0, 0};
    if (b < kSeqThreads) {
        if (b < a.num_seqs) e.x = a.lens[b];
    } else if (g < a.num_groups) {
        e.x = a.group_offsets[g];
        e.y = a.group_offsets[g + 1];
        e.z = a.prefix_lens[g];
    }
    return e;
}

// Every CTA plans the whole call in its own shared memory (the ring's, before
// the first copy): a launch less, and the latency is one round of loads plus
// the sums.  It keeps the units it will walk over (those that its caches cannot
// hold in the workspace); what the merge needs the CTAs write together.
__device__ void make_plan(const PrefixArgs& a, const Early& early, uint8_t* scratch, int2* seq_cache,
                          int4* group_cache, Start* start) {
    __shared__ int sums[2][kThreads / 32];
    __shared__ Start found_smem;
    Start* found = &found_smem;
    const int B = a.num_seqs, Hkv = a.num_kv_heads, tid = threadIdx.x, lane = tid & 31;
    const bool of_seq = tid < kSeqThreads;
    const int id = of_seq ? tid : tid - kSeqThreads;
    const bool report = blockIdx.x == 0;
    int4* group = reinterpret_cast<int4*>(scratch);             // [G] {first sequence, sequences, members, table row}
    int* cum_p = reinterpret_cast<int*>(group + a.num_groups);  // [G] cost of the shared units before
    int* pre = cum_p + a.num_groups;                            // [G] prefix lengths
    int* len = pre + a.num_groups;                              // [B]
    int* mine = len + B;                                        // [B] the group it reads with, or -1
    int* cum_s = mine + B;                                      // [B] cost of the own units before, from the first own one
    bool bad = false;
    if (of_seq) {
#pragma unroll 1
        for (int b = id; b < B; b += kSeqThreads) {
            int L = b == id ? early.x : a.lens[b];
            if (L < 0 || L > a.max_len) {
                if (report && a.err) atomicOr(a.err, PKV_ERRBIT_SEQ_LEN);
                L = L < 0 ? 0 : a.max_len;
            }
            len[b] = L;
        }
    } else {
#pragma unroll 1
        for (int g = id; g < a.num_groups; g += kGroupThreads) {
            Early e = early;
            if (g != id) e = Early{a.group_offsets[g], a.group_offsets[g + 1], a.prefix_lens[g]};
            if (e.x < 0 || e.y < e.x || e.y > B) bad = true;
            if (e.z < 0 && report && a.err) atomicOr(a.err, PKV_ERRBIT_GROUP);
            group[g] = make_int4(e.x, e.y - e.x, 0, INT_MAX);
            pre[g] = e.z < 0 || e.z > a.max_len ? 0 : e.z - e.z % kTok;  // (no sequence is longer than max_len)
        }
    }
    bad = __syncthreads_or(bad);
    const int G = bad ? 0 : a.num_groups;  // no sharing at all when the groups make no sense
    if (bad && tid == 0 && report && a.err) atomicOr(a.err, PKV_ERRBIT_GROUP);
    // A group's members are the sequences that hold all of its shared tiles;
    // below two there is nothing to share.
#pragma unroll 1
    for (int base = 0; of_seq && base < B; base += kSeqThreads) {
        const int b = base + id;
        int lo = 0, hi = G;  // the last group that starts at or before b (the empty ones before it start there too)
        bool member = false;
        if (b < B && G > 0) {
#pragma unroll 1
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (group[mid].x <= b) lo = mid;
                else hi = mid;
            }
            const int first = group[lo].x, n = group[lo].y;
            member = b >= first && b < first + n && pre[lo] > 0 && len[b] >= pre[lo];
        }
        if (b < B) mine[b] = member ? lo : -1;
        const unsigned m = __ballot_sync(0xFFFFFFFFu, member);
        if (m != 0) {  // counted once per warp where they are of one group
            const int lead = __ffs(m) - 1, g = __shfl_sync(0xFFFFFFFFu, lo, lead);
            const bool one = __all_sync(0xFFFFFFFFu, !member || lo == g);
            if (member && (!one || lane == lead)) {
                atomicAdd(&group[lo].z, one ? __popc(m) : 1);
                atomicMin(&group[lo].w, b);
            }
        }
    }
    __syncthreads();
    auto shared_of = [&](int g) { return g >= 0 && group[g].z >= 2 ? pre[g] / kTok : 0; };  // tiles
    auto own_of = [&](int b) { return (len[b] + kTok - 1) / kTok - shared_of(mine[b]); };
    int T1 = 0, T2 = 0;  // cost of the shared tiles, and of the own ones
#pragma unroll 1
    for (int round = 0; round * kSeqThreads < B || round * kGroupThreads < G; ++round) {
        const int x = round * (of_seq ? kSeqThreads : kGroupThreads) + id;
        int v = 0, seqs, groups;
        if (of_seq) {
            const int nt = x < B ? own_of(x) : 0;
            v = nt > 0 ? (nt + a.unit_cost) * Hkv : 0;
        } else if (x < G) {
            const int tiles = shared_of(x);
            v = tiles > 0 ? row_tiles(a, group[x].y) * Hkv * (tiles + a.unit_cost) : 0;
        }
        v = plan_scan(v, sums[round & 1], &seqs, &groups);
        if (x < (of_seq ? B : G)) (of_seq ? cum_s : cum_p)[x] = (of_seq ? T2 : T1) + v;
        T1 += groups;
        T2 += seqs;
    }
    __syncthreads();
    const int T = T1 + T2;
    const Cut cut(T, a.ctas);
    const int r = my_range(a.ctas);
    Start st{0, 0, 0, 0, 0, 0, 0, 0, T};
    int x0 = 0, x1 = 0;  // this CTA's range, counted from the first own unit
    if (r < cut.n) {
        st.pos = cut.start(r);
        st.left = cut.start(r + 1) - st.pos;
        st.own = st.pos >= T1;
        x0 = st.pos - T1;
        x1 = x0 + st.left;
    }
    // The thread whose sequence or group the range begins in says where (a
    // search would be a chain of ten loads).  Of batches that the cache cannot
    // hold it keeps the part from there on.
    auto begin = [&](int i, int x, int tiles) {
        const int vt = tiles + a.unit_cost;
        found->i = i;
        found->u = x / vt;
        found->t = x - found->u * vt;
    };
    auto own_end = [&](int b) { return b + 1 < B ? cum_s[b + 1] : T2; };
    if (of_seq) {
#pragma unroll 1
        for (int b = id; b < B; b += kSeqThreads) {
            const int lo = cum_s[b], hi = own_end(b);
            if (lo <= x0 && x0 < hi) begin(b, x0 - lo, own_of(b));
            if (lo < x1 && hi > x0 && B <= kSeqCache) seq_cache[b] = make_int2(len[b], shared_of(mine[b]));
        }
    } else {
#pragma unroll 1
        for (int g = id; g < G; g += kGroupThreads) {
            const int lo = cum_p[g] - T1, hi = (g + 1 < G ? cum_p[g + 1] : T1) - T1;
            if (lo <= x0 && x0 < hi) begin(g, x0 - lo, shared_of(g));
            if (lo < x1 && hi > x0) {
                const int tiles = shared_of(g);
                (G <= kGroupCache ? group_cache : a.groups)[g] =
                    make_int4(group[g].x, group[g].y, tiles, tiles > 0 ? group[g].w : 0);
            }
        }
        // where the merge finds the pieces of a sequence's rows: a few by every CTA
#pragma unroll 1
        for (int b = static_cast<int>(blockIdx.x + gridDim.x * id); b < B; b += static_cast<int>(gridDim.x * kGroupThreads)) {
            const int g = mine[b], shared = shared_of(g);
            int4 p = make_int4(0, 0, 0, 0);
            int stride = 0;
            if (shared > 0) {
                const int r = (b - group[g].x) / a.seqs_per_tile, seq0 = group[g].x + r * a.seqs_per_tile;
                stride = min(a.seqs_per_tile, group[g].y - r * a.seqs_per_tile) * a.gh;
                p = make_int4(cum_p[g] + r * Hkv * (shared + a.unit_cost), shared, Hkv * seq0, b - seq0);
            }
            a.pieces[2 * b] = p;
            a.pieces[2 * b + 1] = make_int4(stride, T1 + cum_s[b], own_of(b), 0);
        }
        if (report && id == 0) *a.totals = T;
    }
    st.groups_cached = G <= kGroupCache;
    if (B > kSeqCache) {
        __syncthreads();
        st.seq0 = st.own ? found->i : 0;
#pragma unroll 1
        for (int b = st.seq0 + tid; b < B; b += kThreads)
            if (cum_s[b] < x1 && own_end(b) > x0) {
                const int2 q = make_int2(len[b], shared_of(mine[b]));
                if (b - st.seq0 < kSeqCache) seq_cache[b - st.seq0] = q;
                else a.seqs[b] = q;
            }
    }
    // the units' data, for every thread of this CTA; and no generic access to
    // the ring behind the copies that follow
    fence_async_smem();
    __syncthreads();
    st.i = found->i;
    st.u = found->u;
    st.t = found->t;
    *start = st;
}

// ------------------------------------------------------------------- walk
// A run of one unit's tiles.
struct Seg {
    int own;             // 0: shared tiles of a group, 1: own tiles of a sequence
    int tile, n;         // first tile's index in the sequence, tiles
    int row;             // table row
    int end;             // tokens visible to the unit's rows
    int seq0, nseq;      // the sequences whose queries are the rows
    int head;
    int range;           // of the list (see piece_row)
    int turn;            // shared tiles are taken from this one on, then the ones before it

    __device__ int rows(const PrefixArgs& a) const { return nseq * a.gh; }
    // First row of this piece in the list's partials.  Consecutive pieces
    // differ by a range, a unit or both, so (rows of the units before) + (range)
    // x (rows of a full unit) never collides.
    __device__ size_t piece_row(const PrefixArgs& a) const {
        const size_t before = static_cast<size_t>(a.gh) * (static_cast<size_t>(a.num_kv_heads) * seq0 +
                                                           static_cast<size_t>(head) * nseq);
        return before + static_cast<size_t>(range) * (own ? a.gh : kRows);
    }
};

// The segments of this CTA's range, in order.
struct Walk {
    Start at;
    int range;
    const int2* seq_cache;
    const int4* group_cache;

    __device__ bool next(const PrefixArgs& a, Seg& s) {
        while (at.left > 0) {
            const int nt = unit(a, s);
            const int t0 = at.t, cost = min(at.left, nt + a.unit_cost - t0);
            at.left -= cost;
            at.t = 0;
            if (++at.u == units) {
                at.u = 0;
                ++at.i;
            }
            s.n = min(cost, nt - t0);
            s.tile += t0;
            s.range = range;
            s.turn = 0;
            if (ahead > 0 && s.n > 0) {
                const Cut cut(at.T, a.ctas);
                const int x = at.pos - ahead, next = cut.start(cut.of(x) + 1) - x;
                if (next < s.n) s.turn = next;
            }
            at.pos += cost;
            if (s.n > 0) return true;  // (else only the end of a unit's cost fell into the range)
        }
        return false;
    }

  private:
    int units = 0;
    // How far before this unit's tiles in the list the same tiles stand for the
    // group's first queries.  All of a group's row tiles read the same keys, at
    // the same time if they take them in step: the range that reads a tile
    // for the first queries begins with the tile after its border, so another
    // row tile's range begins there, too, and ends with those before it.  Each
    // byte then comes from memory once (out of step, 64 sequences over a
    // prefix as large as the L2, 134 MB, took 50 us instead of 46).
    int ahead = 0;
    // The unit at (i, u), or of the next i with tiles: everything but the range of tiles.  Returns its tiles.
    __device__ int unit(const PrefixArgs& a, Seg& s) {
        while (!at.own) {
            if (at.i == a.num_groups) {  // on to the own tiles
                at.own = 1;
                at.i = 0;
                break;
            }
            const int4 g = at.groups_cached ? group_cache[at.i] : a.groups[at.i];
            if (g.z > 0) {
                const int r = at.u / a.num_kv_heads;
                units = row_tiles(a, g.y) * a.num_kv_heads;
                s.own = 0;
                s.row = g.w;
                s.head = at.u - r * a.num_kv_heads;
                s.seq0 = g.x + r * a.seqs_per_tile;
                s.nseq = min(a.seqs_per_tile, g.y - r * a.seqs_per_tile);
                s.tile = 0;
                s.end = g.z * kTok;
                ahead = r * a.num_kv_heads * (g.z + a.unit_cost);
                return g.z;
            }
            ++at.i;
        }
        for (;; ++at.i) {
            const int2 q = at.i - at.seq0 < kSeqCache ? seq_cache[at.i - at.seq0] : a.seqs[at.i];
            const int nt = (q.x + kTok - 1) / kTok - q.y;
            if (nt <= 0) continue;
            units = a.num_kv_heads;
            ahead = 0;
            s.own = 1;
            s.row = s.seq0 = at.i;
            s.nseq = 1;
            s.head = at.u;
            s.tile = q.y;
            s.end = q.x;
            return nt;
        }
    }
};

template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 2)
prefix_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                 const __grid_constant__ CUtensorMap tmq_group, const __grid_constant__ CUtensorMap tmq_own,
                 const PrefixArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = su32(smem), bars = sbase + kBarOff;
    auto B = [&](int i) { return bars + 8u * i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kBarOff + 8 * kNumBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kBarOff + 8 * kNumBars + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const Early early = fetch_early(a);  // (under way while the CTA sets itself up)
    // Setting up is shared out to warps that the plan's first part hardly needs
    // (kWarpK and behind); its barriers cover what they write.
    if (warp == kWarpS) {
        for (int i = lane; i < kNumBars; i += 32)
            bar_init(B(i), (i >= kPFull && i < kPFull + kNS) || i == kOFree || i == kSRead || i == kQOp || i >= kVEmpty
                               ? kSoftmaxWarps
                               : (i == kDone ? 2u : 1u));
        if (lane == 0) *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp >= kWarpK && lane == 0) {  // (the descriptors are fetched while the plan is made)
        const CUtensorMap* map = warp == kWarpK ? &tmk : (warp == kWarpV ? &tmv : (warp == kWarpS ? &tmq_own : &tmq_group));
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
    }
    if (warp == kWarpPv) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(su32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
        fence_before();
    }
    Walk w;
    w.range = my_range(a.ctas);
    w.seq_cache = reinterpret_cast<const int2*>(smem + kSeqOff);
    w.group_cache = reinterpret_cast<const int4*>(smem + kGroupOff);
    make_plan(a, early, smem + kKVOff, reinterpret_cast<int2*>(smem + kSeqOff), reinterpret_cast<int4*>(smem + kGroupOff), &w.at);
    fence_after();
    const uint32_t tmem = *tmem_slot;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    auto fail = [&]() {
        *abort_flag = 1;
        if (a.err) atomicOr(a.err, PKV_ERRBIT_TIMEOUT);
    };

    if (warp == kWarpK || warp == kWarpV) {
        // ------------------------------------------------ producers: K, V
        // A stage is freed by the completion of the products that read it (no
        // commit of its own for the MMA threads, who set the pace): S done for K, PV
        // done for V; an FP8 V tile by the softmax warps that have read it.
        const bool is_v = warp == kWarpV;
        const CUtensorMap* map = is_v ? &tmv : &tmk;
        const int full0 = is_v ? kVFull : kKFull;
        const int empty0 = is_v ? (kFp8 ? kVEmpty : kPvDone) : kSFull;
        const int bs = a.block_size;
        const int64_t layer_blk0 = static_cast<int64_t>(a.layer) * a.num_blocks;
        int k = 0;
        bool ok = true;
        Seg sg, nx;
        bool has = w.next(a, sg);
        while (has && ok) {
            const bool has_next = w.next(a, nx);  // (early: its loads overlap this segment)
            int cache = 0, cache_base = INT_MIN / 2;  // 32 table entries, one per lane
            for (int t = 0; t < sg.n && ok; ++t, ++k) {
                const int s = k % kNS;
                const int tt = t + sg.turn < sg.n ? t + sg.turn : t + sg.turn - sg.n;
                const int tok0 = (sg.tile + tt) * kTok, n = min(kTok, sg.end - tok0), nblk = (n + bs - 1) / bs;
                const int idx0 = tok0 / bs;
                if (idx0 < cache_base || idx0 + nblk > cache_base + 32) {
                    cache_base = idx0;
                    const int idx = idx0 + lane;
                    cache = idx < a.max_blocks ? __ldg(a.tables + static_cast<size_t>(sg.row) * a.max_blocks + idx) : 0;
                }
                if (__any_sync(0xFFFFFFFFu, *abort_flag != 0) ||
                    (k >= kNS && !__all_sync(0xFFFFFFFFu, bar_wait_or(B(empty0 + s), ((k / kNS) - 1) & 1, abort_flag)))) {
                    ok = false;
                    break;
                }
                const uint32_t dst0 = kFp8 ? sbase + kKVOff + (2 * s + (is_v ? 1 : 0)) * kRawBytes
                                           : sbase + kKVOff + s * kStageBytes + (is_v ? 2 * kHalfBytes : 0);
                if (lane == 0) bar_expect_tx(B(full0 + s), static_cast<uint32_t>(nblk * bs * kDim * (kFp8 ? 1 : 2)));
                __syncwarp();
                // one copy instruction: lane 2 kb + hf, half hf of block kb (FP8: lane kb, block kb)
                const int kb = kFp8 ? lane : lane >> 1, hf = kFp8 ? 0 : lane & 1;
                int blk = __shfl_sync(0xFFFFFFFFu, cache, (idx0 + kb - cache_base) & 31);
                if (kb < nblk) {
                    if (static_cast<unsigned>(blk) >= static_cast<unsigned>(a.num_blocks)) {
                        if (a.err) atomicOr(a.err, PKV_ERRBIT_BLOCK_ID);
                        blk = 0;  // an in-bounds block; the flag marks the output invalid
                    }
                    const int y = static_cast<int>(((layer_blk0 + blk) * a.num_kv_heads + sg.head) * bs);
                    if constexpr (kFp8) tma_2d(dst0 + kb * bs * 128, map, 0, y, B(full0 + s));
                    else tma_3d(dst0 + hf * kHalfBytes + kb * bs * 128, map, 0, y, hf, B(full0 + s));
                }
            }
            sg = nx;
            has = has_next;
        }
        if (!ok && lane == 0) fail();
        // drain: the copies in flight land before the CTA frees anything
        if (lane == 0)
            for (int j = k - 1; j >= 0 && j >= k - kNS; --j)
                if (!bar_wait(B(full0 + j % kNS), (j / kNS) & 1)) fail();
    } else if (warp == kWarpS) {
        // ----------------------------------------------------- S = Q K^T
        // (The softmax warps tell at an mbarrier that they have read a tile's
        // scores.  A named barrier in its place, which has no bound, took 1 to 2 %
        // longer on every batch timed.)
        if (lane == 0) {
            bool ok = true;
            const uint64_t dq = sdesc(sbase, 16);
            const uint64_t dk0 = sdesc(sbase + kKVOff, 16);
            // (test hook: this CTA's first wait for a tile may be cut short)
            const uint32_t first_polls =
                a.test_polls >= 0 && (a.test_cta < 0 || a.test_cta == static_cast<int>(blockIdx.x)) ? a.test_polls : kSpin;
            Seg sg;
            int k = 0, copies = 0;
            for (int seg = 0; ok && w.next(a, sg); ++seg) {
                // This segment's Q rows, once the last S of the one before has read its own.
                if (seg > 0 && !bar_wait_or(B(kQFree), (seg - 1) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                bar_expect_tx(B(kQReady), static_cast<uint32_t>((sg.own ? 1 : a.seqs_per_tile) * a.gh * kDim * 2));
                for (int h2 = 0; h2 < 2; ++h2)
                    tma_4d(sbase + h2 * kQHalf, sg.own ? &tmq_own : &tmq_group, 0, sg.head * a.gh, sg.seq0, h2, B(kQReady));
                ++copies;
                for (int t = 0; t < sg.n; ++t, ++k) {
                    const int s = k % kNS;
                    // Q (FP8: split), K k, and S k - 1 taken to registers
                    if (*abort_flag || (t == 0 && !bar_wait_or(B(kFp8 ? kQOp : kQReady), seg & 1, abort_flag)) ||
                        !bar_wait_or(B(kKFull + s), (k / kNS) & 1, abort_flag, k == 0 ? first_polls : kSpin) ||
                        (k > 0 && !bar_wait_or(B(kSRead), (k - 1) & 1, abort_flag))) {
                        ok = false;
                        break;
                    }
                    fence_after();
                    const uint64_t dk = dk0 + static_cast<uint64_t>((s * (kFp8 ? 2 * kRawBytes : kStageBytes)) >> 4);
                    const uint32_t sb = tmem;
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {  // 16 columns a step; FP8: 32, first of Q's high terms, then of the low ones
                        const uint32_t kin = (ks & 3) * 32;
                        if constexpr (kFp8)
                            mma_f8(sb, dq + (((ks >> 2) * kQHalf + kin) >> 4), dk + (kin >> 4), idesc0(kTok, 0), ks > 0 ? 1u : 0u);
                        else mma_bf16(sb, dq + (((ks >> 2) * kQHalf + kin) >> 4), dk + (((ks >> 2) * kHalfBytes + kin) >> 4),
                                 idesc(kTok, 0), ks > 0 ? 1u : 0u);
                    }
                    mma_commit(B(kSFull + s));
                    if (t == sg.n - 1) mma_commit(B(kQFree));
                }
            }
            if (!ok) fail();
            // (no copy of Q may land after the CTA has gone)
            if (copies > 0 && !bar_wait(B(kQReady), (copies - 1) & 1)) fail();
            mma_commit(B(kDone));  // completes once every MMA this thread issued has finished
            if (!bar_wait(B(kDone), 0)) fail();
        }
        __syncwarp();
    } else if (warp == kWarpPv) {
        // ------------------------------------------------------- O += P V
        if (lane == 0) {
            bool ok = true;
            const uint64_t dv0 = sdesc(sbase + (kFp8 ? kWideOff : kKVOff + 2 * kHalfBytes), kHalfBytes);
            Seg sg;
            int k = 0;
            for (int seg = 0; ok && w.next(a, sg); ++seg) {
                for (int t = 0; t < sg.n; ++t, ++k) {
                    const int s = k % kNS;
                    // V k (FP8: with P k), P k, and for a new segment an O that has been read out
                    if (*abort_flag || (!kFp8 && !bar_wait_or(B(kVFull + s), (k / kNS) & 1, abort_flag)) ||
                        !bar_wait_or(B(kPFull + s), (k / kNS) & 1, abort_flag) ||
                        (t == 0 && seg > 0 && !bar_wait_or(B(kOFree), (seg - 1) & 1, abort_flag))) {
                        ok = false;
                        break;
                    }
                    fence_after();
                    const uint64_t dv = dv0 + static_cast<uint64_t>((s * (kFp8 ? 2 * kHalfBytes : kStageBytes)) >> 4);
                    const uint32_t pb = tmem + kPCol + static_cast<uint32_t>(s) * kPCols;
#pragma unroll
                    for (int ks = 0; ks < kTok / 16; ++ks)  // 16 tokens a step
                        mma_bf16_ta(tmem + kOCol, pb + 8 * ks, dv + ((ks * 16 * 128) >> 4), kFp8 ? idesc0(kDim, 1) : idesc(kDim, 1),
                                  t > 0 || ks > 0 ? 1u : 0u);
                    mma_commit(B(kPvDone + s));
                }
            }
            if (!ok) fail();
            mma_commit(B(kDone));
            if (!bar_wait(B(kDone), 0)) fail();
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ softmax and epilogue
        // Warps w and w + 4 share TMEM lanes 32 (w % 4) .. + 31: row m has one
        // thread for tokens 0-31 of a tile and output columns 0-63, another
        // for the rest.
        const int pair = warp & 3, hf = warp >> 2;
        const int m = 32 * pair + lane;
        const uint32_t lane_off = static_cast<uint32_t>(32 * pair) << 16;
        // (written once more only after a later rendezvous of the pair)
        float* ex = reinterpret_cast<float*>(smem + kExOff);
        float* sums = reinterpret_cast<float*>(smem + kSumOff);
        float qk = a.qk_scale_log2;  // FP8 pools: of this row, see convert_q
        // A wait that expires makes the warp `dead`: it goes on through the
        // loop, without waiting or working, only to meet its partner.
        bool dead = false;
        auto wait = [&](int b, int phase) {
            // (one look first: passing a barrier that is complete takes a third of
            // the time that way, and with FP8 pools S mostly is)
            if (!dead && !__all_sync(0xFFFFFFFFu, bar_test(B(b), phase & 1)) &&
                !__all_sync(0xFFFFFFFFu, bar_wait_or(B(b), phase & 1, abort_flag))) {
                dead = true;
                if (lane == 0) fail();
                __syncwarp();
            }
        };

        // FP8 pools: the tensor cores take K and V as stored, and one type for
        // both operands.  A query row is scaled by the power of two that brings
        // its largest element to [2^7, 2^8) and split into two E4M3 terms: a BF16
        // significand has 8 bits, hi takes 4 and lo the rest, so the sum is exact
        // for elements down to 2^-10 of the largest (below, off by 2^-18 of it).
        // The scale goes back into the row's score scale.
        int* qmax = reinterpret_cast<int*>(smem + kQMaxOff);
        auto convert_q = [&](int seg, const Seg& s) {
            wait(kQReady, seg);
            if (32 * pair < s.rows(a)) {
                uint4 v[8];
                int top = 0;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    v[c] = *reinterpret_cast<const uint4*>(smem + tile_off(m, 8 * hf + c, kQHalf));
                    const uint32_t u[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        top = max(top, max(static_cast<int>(u[i] & 0x7FFFu), static_cast<int>((u[i] >> 16) & 0x7FFFu)));
                }
                qmax[hf * kRows + m] = top;
                pair_sync(pair);  // (and both threads of the row have read it)
                const int ex = max(top, qmax[(hf ^ 1) * kRows + m]) >> 7;  // exponent field: 0 zero or subnormal, 255 inf, NaN
                const int shift = ex == 0 || ex == 255 ? 0 : min(134 - ex, 126);
                const float up = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
                // (an infinite or NaN query, which E4M3 would clamp, makes the whole row NaN)
                qk = ex == 255 ? __uint_as_float(0x7FC00000u)
                               : a.qk_scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
                // columns 64 hf .. 64 hf + 63: four 16-byte chunks of the high tile, four of the low one
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t u[8] = {v[2 * c].x,     v[2 * c].y,     v[2 * c].z,     v[2 * c].w,
                                           v[2 * c + 1].x, v[2 * c + 1].y, v[2 * c + 1].z, v[2 * c + 1].w};
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        split4(bf16_lo(u[2 * i]) * up, bf16_hi(u[2 * i]) * up, bf16_lo(u[2 * i + 1]) * up,
                               bf16_hi(u[2 * i + 1]) * up, hi[i], lo[i]);
                    const uint32_t at = tile_off(m, 4 * hf + c, 0);
                    *reinterpret_cast<uint4*>(smem + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(smem + kQHalf + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) bar_arrive(B(kQOp));
        };

        // FP8 pools: V k as FP16, the rows behind the last token as zeros, by the
        // pairs that have no rows (else by all, behind their weights; 64 sequences
        // with 2048 own tokens took 85 us with one FP16 tile, which waits for PV
        // k - 1, and 74 with two, prefixes alone 60 and 56).  Eight threads read a
        // row's 128 bytes and write its two 64-column halves, those of the second
        // half their odd chunks first, so that the eight stores fall into different
        // banks.  The FP16 tile is free: the warp has waited for PV k - 2.
        auto widen_v = [&](int k, int visible, int rows) {
            constexpr int kPairs = kSoftmaxWarps / 2;
            const int s = k % kNS, with_rows = (rows + 31) / 32, skip = with_rows < kPairs ? with_rows : 0;
            if (pair >= skip) {
                wait(kVFull + s, k / kNS);
                const uint8_t* raw = smem + kKVOff + (2 * s + 1) * kRawBytes;
                const int c = lane & 7, half = c >> 2, ch = 2 * (c & 3) + half;
                uint8_t* wide = smem + kWideOff + (2 * s + half) * kHalfBytes;
                auto row = [&](int t) {
                    uint4 x = *reinterpret_cast<const uint4*>(raw + tile_off(t, c, 0)), lo, hi;
                    if (t >= visible) x = make_uint4(0u, 0u, 0u, 0u);
                    widen16(x, lo, hi);
                    *reinterpret_cast<uint4*>(wide + tile_off(t, ch, 0)) = half ? hi : lo;
                    *reinterpret_cast<uint4*>(wide + tile_off(t, ch ^ 1, 0)) = half ? lo : hi;
                };
                if (skip == 0) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) row(4 * warp + (lane >> 3) + i * (kTok / 2));
                } else {
                    const int pairs = kPairs - skip;
                    for (int t = 4 * (hf * pairs + pair - skip) + (lane >> 3); t < kTok; t += 8 * pairs) row(t);
                }
                fence_async_smem();
                __syncwarp();
            }
            if (lane == 0) bar_arrive(B(kVEmpty + s));
        };

        Seg sg, nx;
        bool has = w.next(a, sg);
        if (kFp8 && has) convert_q(0, sg);
        int seg = 0;
        for (int k0 = 0; has; ++seg) {
            const bool has_next = w.next(a, nx);  // (early: its loads overlap the first S)
            const int nv = sg.rows(a);
            const bool busy = 32 * pair < nv;
            float m_used = -INFINITY, l = 0.f;
            for (int t = 0; t < sg.n; ++t) {
                const int k = k0 + t, s = k % kNS;
                const int visible = sg.end - (sg.tile + t) * kTok;  // of this tile, the same for every row
                // S k, and (odd lanes) the P buffer that PV k - 2 has read
                const bool odd = (lane & 1) != 0 && k >= kNS;
                wait(odd ? kPvDone + s : kSFull + s, odd ? k / kNS - 1 : k / kNS);
                fence_after();
                const uint32_t sa = tmem + lane_off, pa = sa + kPCol + static_cast<uint32_t>(s) * kPCols;
                bool rescale = false;
                float alpha = 1.f;
                if (busy) {
                    uint32_t v[32];
                    tmem_ld32(sa + 32 * hf, v);
                    fence_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive(B(kSRead));
                    const int seen = visible - 32 * hf;  // of this thread's 32 tokens
                    float mx = -INFINITY;
                    if (qk > 0.f) {
                        if (seen < 32) {  // what lies behind the last token: no weight, on the path below
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (i >= seen) v[i] = 0xFF800000u;
                        }
                        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            m4[(i >> 1) & 3] = max3(m4[(i >> 1) & 3], __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                        mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * qk;
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i < seen) mx = fmaxf(mx, __uint_as_float(v[i]) * qk);
                    }
                    // Lazy base: it moves (and O and l are rescaled) only when
                    // a row's maximum grew by more than the slack; only then do the two
                    // threads of a row exchange theirs.
                    if (pair_any(pair, m < nv && (mx > m_used + kSlack || m_used == -INFINITY))) {
                        ex[hf * kRows + m] = mx;
                        pair_sync(pair);
                        const float m_new = fmaxf(m_used, fmaxf(mx, ex[(hf ^ 1) * kRows + m]));
                        rescale = m < nv && m_used != -INFINITY && m_new > m_used + kSlack;
                        alpha = rescale ? ex2(m_used - m_new) : 1.f;
                        if (rescale || m_used == -INFINITY) m_used = m_new;
                    }
                    const float base = m_used == -INFINITY ? 0.f : m_used - weight_shift_of<kFp8>();
                    uint32_t pk[16];
                    float lt = 0.f;
                    if (seen >= 32 || qk > 0.f) {
                        float l0 = 0.f, l1 = 0.f;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float x0, x1;
                            fma2(x0, x1, __uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]), qk, qk, -base, -base);
                            const float p0 = ex2(x0), p1 = ex2(x1);
                            add2(l0, l1, l0, l1, p0, p1);
                            pk[i] = kFp8 ? f16x2(p0, p1) : bf16x2(p0, p1);
                        }
                        lt = l0 + l1;
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float p0 = 2 * i < seen ? ex2(fmaf(__uint_as_float(v[2 * i]), qk, -base)) : 0.f;
                            const float p1 = 2 * i + 1 < seen ? ex2(fmaf(__uint_as_float(v[2 * i + 1]), qk, -base)) : 0.f;
                            lt += p0 + p1;
                            pk[i] = kFp8 ? f16x2(p0, p1) : bf16x2(p0, p1);
                        }
                    }
                    l = l * alpha + lt;
                    tmem_st16(pa + 16 * hf, pk);
                    // This warp has waited for PV k - 2 and k - 3, and PV k + 1 cannot
                    // finish before P k + 1 is signalled, so a parity wait for PV
                    // k - 1, or for PV k at the end, is unambiguous.
                    if (__any_sync(0xFFFFFFFFu, rescale)) {
                        wait(kPvDone + (k + kNS - 1) % kNS, (k - 1) / kNS);
                        fence_after();
#pragma unroll 1
                        for (int c = 0; c < 2; ++c) {
                            uint32_t o[32];
                            const uint32_t oa = tmem + lane_off + kOCol + 64 * hf + 32 * c;
                            tmem_ld32(oa, o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                            tmem_st32(oa, o);
                        }
                    }
                } else if (lane == 0) {
                    bar_arrive(B(kSRead));
                }
                // V rows past the last token: zero (stale or unwritten rows could hold NaN)
                if constexpr (kFp8) {
                    widen_v(k, visible, nv);
                } else if (visible < kTok) {
                    wait(kVFull + s, k / kNS);
                    uint8_t* vs = smem + kKVOff + s * kStageBytes + 2 * kHalfBytes;
                    const int nz = kTok - visible;
                    for (int e = threadIdx.x; e < 2 * nz * 8; e += kSoftmax) {  // whole 128-byte rows: any swizzle
                        const int h2 = e / (nz * 8), rem = e % (nz * 8);
                        *reinterpret_cast<uint4*>(vs + h2 * kHalfBytes + (visible + rem / 8) * 128 + (rem % 8) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_async_smem();
                }
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(B(kPFull + s));
            }
            // ---- the piece ends
            const int kl = k0 + sg.n - 1;
            if (kFp8 && has_next) convert_q(seg + 1, nx);  // (sets qk, which this piece is done with)
            if (busy) {
                sums[hf * kRows + m] = l;
                pair_sync(pair);
                l += sums[(hf ^ 1) * kRows + m];
            }
            wait(kPvDone + kl % kNS, kl / kNS);
            fence_after();
            if (busy) {
                const float inv = l > 0.f ? 1.f / l : 0.f;
                const size_t row0 = sg.piece_row(a) + 32 * pair;
                float* po = (sg.own ? a.own_o : a.pre_o) + row0 * kDim + 64 * hf + 2 * (lane & 3);
                // Rows in quarters of the warp: eight rows by 32 bytes a store,
                // whole sectors (a row per thread wrote half ones, 32 lines a store).
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t v[32];
                    if (32 * pair + 16 * c < nv)
                        tmem_ld_16x64(tmem + lane_off + (static_cast<uint32_t>(16 * c) << 16) + kOCol + 64 * hf, v);
                    if (c == 1) {  // O is read: the next segment's first PV may overwrite it
                        fence_before();
                        __syncwarp();
                        if (lane == 0) bar_arrive(B(kOFree));
                    }
#pragma unroll
                    for (int up = 0; up < 2; ++up) {
                        if (32 * pair + 16 * c + 8 * up >= nv) break;  // (own units have a few rows only)
                        const int r = 16 * c + 8 * up + (lane >> 2);
                        const float f = __shfl_sync(0xFFFFFFFFu, inv, r);
                        if (32 * pair + r < nv) {
                            float* dst = po + r * kDim;
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                *reinterpret_cast<float2*>(dst + 8 * q) =
                                    make_float2(__uint_as_float(v[4 * q + 2 * up]) * f, __uint_as_float(v[4 * q + 2 * up + 1]) * f);
                        }
                    }
                }
                // (NaN from a CTA that gave up: its rows must not look like results)
                if (m < nv && hf == 0)
                    (sg.own ? a.own_lse : a.pre_lse)[row0 + lane] =
                        dead || *abort_flag != 0 ? __uint_as_float(0x7FC00000u)
                                                 : (l > 0.f ? m_used - weight_shift_of<kFp8>() + log2f(l) : -INFINITY);
            } else if (lane == 0) {
                bar_arrive(B(kOFree));
            }
            k0 += sg.n;
            sg = nx;
            has = has_next;
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// ------------------------------------------------------------------ merge
constexpr int kMergeThreads = 256;

constexpr int kMergeAhead = 8;  // pieces whose rows are loaded before their weights are known

// One warp per output row; lane d holds columns 4 d .. 4 d + 3.  A row has one
// piece per range that its two units touch.  Three dependent rounds of loads:
// the plan, the log-sum-exps beside the first rows, the other rows.
__global__ void __launch_bounds__(kMergeThreads) prefix_merge_kernel(const PrefixArgs a) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int lane = threadIdx.x & 31;
    const unsigned out_row = blockIdx.x * (kMergeThreads / 32u) + (threadIdx.x >> 5);  // (fits: checked on the host)
    if (out_row >= static_cast<unsigned>(a.num_seqs) * static_cast<unsigned>(a.num_q_heads)) return;
    const int b = static_cast<int>(out_row / a.num_q_heads), hq = static_cast<int>(out_row - static_cast<unsigned>(b) * a.num_q_heads);
    const int h = hq / a.gh;
    const int4 p = a.pieces[2 * b], q = a.pieces[2 * b + 1];
    const Cut cut(*a.totals, a.ctas);
    // pieces 0 .. n0 - 1: rows pre0 + j * kRows; then n1 more: rows own0 + j * gh
    int n0 = 0, n1 = 0;
    size_t pre0 = 0, own0 = 0;
    if (p.y > 0) {
        const int ps = p.x + h * (p.y + a.unit_cost), c0 = cut.of(ps);
        n0 = cut.of(ps + p.y - 1) - c0 + 1;
        pre0 = static_cast<size_t>(a.gh) * (p.z + p.w) + static_cast<size_t>(h) * q.x + hq % a.gh +
               static_cast<size_t>(c0) * kRows;
    }
    if (q.z > 0) {
        const int ps = q.y + h * (q.z + a.unit_cost), c0 = cut.of(ps);
        n1 = cut.of(ps + q.z - 1) - c0 + 1;
        own0 = static_cast<size_t>(out_row) + static_cast<size_t>(c0) * a.gh;
    }
    const int pieces = n0 + n1;
    auto row_of = [&](int j) {
        return j < n0 ? pre0 + static_cast<size_t>(j) * kRows : own0 + static_cast<size_t>(j - n0) * a.gh;
    };
    auto lse_of = [&](int j) { return (j < n0 ? a.pre_lse : a.own_lse)[row_of(j)]; };
    auto o_of = [&](int j) {
        return reinterpret_cast<const float4*>((j < n0 ? a.pre_o : a.own_o) + row_of(j) * kDim)[lane];
    };
    float4 v[kMergeAhead];
#pragma unroll
    for (int j = 0; j < kMergeAhead; ++j) v[j] = j < pieces ? o_of(j) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float first = lane < pieces ? lse_of(lane) : -INFINITY;
    float M = first;
    for (int j = 32 + lane; j < pieces; j += 32) M = fmaxf(M, lse_of(j));
    M = warp_max(M);
    float z = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float w, const float4& o) {
        acc.x = fmaf(w, o.x, acc.x);
        acc.y = fmaf(w, o.y, acc.y);
        acc.z = fmaf(w, o.z, acc.z);
        acc.w = fmaf(w, o.w, acc.w);
    };
    for (int j0 = 0; j0 < pieces; j0 += 32) {
        const float s = j0 == 0 ? first : (j0 + lane < pieces ? lse_of(j0 + lane) : -INFINITY);
        const float wt = s == -INFINITY ? 0.f : exp2f(s - M);
        z += warp_sum(wt);
        int j = 0;
        if (j0 == 0) {
#pragma unroll
            for (; j < kMergeAhead; ++j) add(__shfl_sync(0xFFFFFFFFu, wt, j), v[j]);
        }
        const int last = min(32, pieces - j0);
        for (; j < last; j += kMergeAhead) {
#pragma unroll
            for (int e = 0; e < kMergeAhead; ++e) v[e] = j + e < last ? o_of(j0 + j + e) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int e = 0; e < kMergeAhead; ++e) add(__shfl_sync(0xFFFFFFFFu, wt, (j + e) & 31), v[e]);
        }
    }
    const float inv = z > 0.f ? a.v_scale / z : 0.f;  // no token: a zero row
    uint2 pk;
    pk.x = bf16x2(acc.x * inv, acc.y * inv);
    pk.y = bf16x2(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + static_cast<size_t>(out_row) * kDim + 4 * lane) = pk;
}

}  // namespace

namespace {
template <bool kFp8>
cudaError_t launch_tc(const PrefixArgs& a, const void* tmap_k, const void* tmap_v, const void* tmap_q_group,
                      const void* tmap_q_own, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> configured{0};  // a bit per device; setting the attributes twice does no harm
    if (dev < 0 || dev >= 64) return cudaErrorNotSupported;
    if (!(configured.load() >> dev & 1)) {
        e = cudaFuncSetAttribute(prefix_tc_kernel<kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(prefix_tc_kernel<kFp8>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
        configured.fetch_or(1ull << dev);
    }
    prefix_tc_kernel<kFp8><<<a.ctas, kThreads, kSmem, stream>>>(
        *static_cast<const CUtensorMap*>(tmap_k), *static_cast<const CUtensorMap*>(tmap_v),
        *static_cast<const CUtensorMap*>(tmap_q_group), *static_cast<const CUtensorMap*>(tmap_q_own), a);
    return cudaGetLastError();
}
}  // namespace

cudaError_t launch_prefix_attention(pkv_dtype kv, const PrefixArgs& args, const void* tmap_k, const void* tmap_v,
                                    const void* tmap_q_group, const void* tmap_q_own, cudaStream_t stream) {
    PrefixArgs a = args;
    a.unit_cost = unit_cost_of(kv);
    const cudaError_t e = kv == PKV_FP8_E4M3 ? launch_tc<true>(a, tmap_k, tmap_v, tmap_q_group, tmap_q_own, stream)
                                             : launch_tc<false>(a, tmap_k, tmap_v, tmap_q_group, tmap_q_own, stream);
    if (e != cudaSuccess) return e;
    const int64_t rows = static_cast<int64_t>(a.num_seqs) * a.num_q_heads;
    constexpr int per = kMergeThreads / 32;
    return launch_dependent(prefix_merge_kernel, dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(kMergeThreads),
                            0, stream, a);
}

}  // namespace pkv
