// Decode attention of a batch whose sequences share prefixes, each prefix
// read and multiplied once for its whole group ("How does TensorRT-LLM
// work?", "The paged KV cache": requests that begin with the same text point
// at the same blocks; "TensorRT-LLM, in depth", "The paged KV cache and block
// reuse").  BF16 pools, head_dim 128.
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
// Three launches.
//  * prefix_plan_kernel, one CTA: per group the shared tiles (64 tokens; a
//    remainder of the prefix counts as own tokens), prefix sums of the tiles
//    over groups and over sequences, and for every CTA of the next kernel its
//    range of each list.
//  * prefix_tc_kernel, 2 persistent CTAs per SM.  The units are the 128-row
//    query tiles of a (group, KV head), over the group's shared tiles, and
//    the (sequence, KV head) pairs, over the sequence's own tiles.  Every CTA
//    takes an equal share of both lists, odd CTAs the own tiles first: shared
//    tiles are bound by the tensor cores and the softmax (128 rows), own
//    tiles by memory (gh rows), and the two CTAs of an SM overlap them.  Each
//    unit's piece leaves O / l and its log2-sum-exp in the workspace.
//  * prefix_merge_kernel, one warp per output row, merges the pieces.
// The tile pipeline has 7 warps:
//  * warps 4 and 6, TMA producers for K and for V: one box {64 columns, bs
//    rows, 1 half} per KV block and half, 128-byte swizzled: the K-major
//    operand layout for K and the MN-major one for V;
//  * warp 5, one thread: S = Q K^T (M 128, N 64 tokens, K 128) into one of two
//    TMEM buffers, a tile ahead of the softmax; then O += P V (N 128, K 64);
//  * warps 0-3: softmax of row m = TMEM lane m in base 2, P back to tensor
//    memory as BF16 pairs (half a step of 2^-9 relative each: the sum l is
//    taken before that rounding, in fp32), the running maximum moved only
//    when it grows by more than 8, so that O is seldom rescaled.
// Every wait is bounded; a CTA whose wait expires sets PKV_ERRBIT_TIMEOUT,
// waits for its copies and products in flight, frees its TMEM and leaves.
#include <cuda.h>

#include <climits>

#include "tc_common.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 224;  // warps 0-3 softmax, 4 K producer, 5 MMA, 6 V producer
constexpr int kRows = kPrefixRows;
constexpr int kTok = 64;
constexpr int kDim = 128;
constexpr int kNS = 2;                        // stages of each ring, and score buffers
constexpr int kQHalf = kRows * 128;           // one 64-column half of the Q tile
constexpr int kHalfBytes = kTok * 128;        // one 64-column half of a K or V tile
constexpr int kKVOff = 2 * kQHalf;
constexpr int kStageBytes = 4 * kHalfBytes;   // K + V
constexpr int kAlignSlack = 1024;
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kOCol = kNS * kTok;

enum Bar { kQReady, kOFree, kDone, kSFull, kPFull = kSFull + kNS, kPvDone = kPFull + kNS, kKFull = kPvDone + kNS,
           kVFull = kKFull + kNS, kNumBars = kVFull + kNS };
constexpr int kBarOff = kKVOff + kNS * kStageBytes;
constexpr int kSmem = kBarOff + (8 * kNumBars + 8 + 63) / 64 * 64 + kAlignSlack;
static_assert(kSmem <= 115712, "two CTAs per SM");

constexpr int kPlanThreads = 1024;

// ------------------------------------------------------------------- plan
__device__ __forceinline__ int plan_scan(int v, int* warp_sums, int* total) {  // inclusive, over the CTA
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += x;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    const int mine = warp_sums[lane];
    int s = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += x;
    }
    *total = __shfl_sync(0xFFFFFFFFu, s, 31);
    const int before = __shfl_sync(0xFFFFFFFFu, s - mine, warp);
    __syncthreads();
    return v + before;
}

// A list of T tiles is cut into min(T, ctas) ranges, none of them empty: range
// c is [c T / n, (c + 1) T / n).
__device__ __forceinline__ int num_ranges(int T, int ctas) { return T < ctas ? T : ctas; }
__device__ __forceinline__ int range_of(int x, int T, int ctas) {  // the range that tile x is in
    return static_cast<int>(((x + 1LL) * num_ranges(T, ctas) - 1) / T);
}
// Start of range c: unit group i (cum[i] <= tile < cum[i + 1]), tile x within
// it, tiles in the range (0 from range n on).
__device__ __forceinline__ void range_start(const int* cum, int n, int total, int ctas, int c, int* i, int* x, int* left) {
    const long long T = total, ranges = num_ranges(total, ctas);
    *i = *x = *left = 0;
    if (c >= ranges) return;
    const int g0 = static_cast<int>(c * T / ranges), g1 = static_cast<int>((c + 1) * T / ranges);
    *left = g1 - g0;
    int lo = 0, hi = n;
    while (hi - lo > 1) {  // the last i with cum[i] <= g0 (the empty ones before it share its start)
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= g0) lo = mid;
        else hi = mid;
    }
    *i = lo;
    *x = g0 - cum[lo];
}

__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const PrefixArgs a) {
    __shared__ int cum_s[kPrefixMaxSeqs + 1], cum_p[kPrefixMaxSeqs + 1];
    __shared__ int sums[32];
    __shared__ int bad;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int B = a.num_seqs, Hkv = a.num_kv_heads, tid = threadIdx.x;
    const int lane = tid & 31, warp = tid >> 5;
    if (tid == 0) bad = 0;
    __syncthreads();
    for (int g = tid; g < a.num_groups; g += kPlanThreads) {
        const int o0 = a.group_offsets[g], o1 = a.group_offsets[g + 1];
        if (o0 < 0 || o1 < o0 || o1 > B) bad = 1;
    }
    for (int b = tid; b < B; b += kPlanThreads) {
        int L = a.lens[b];
        if (L < 0 || L > a.max_len) {
            if (a.err) atomicOr(a.err, PKV_ERRBIT_SEQ_LEN);
            L = L < 0 ? 0 : a.max_len;
        }
        a.seq_len[b] = L;
        a.seq_pre[b] = 0;
        a.seq_group[b] = -1;
    }
    __syncthreads();
    const int G = bad ? 0 : a.num_groups;  // no sharing at all when the groups make no sense
    if (bad && tid == 0 && a.err) atomicOr(a.err, PKV_ERRBIT_GROUP);
    // per group: its members are the sequences that hold all of its shared tiles
    for (int g = warp; g < G; g += kPlanThreads / 32) {
        const int o0 = a.group_offsets[g], o1 = a.group_offsets[g + 1];
        int P = a.prefix_lens[g];
        if (P < 0 && lane == 0 && a.err) atomicOr(a.err, PKV_ERRBIT_GROUP);
        if (P < 0 || P > a.max_len) P = 0;  // (no sequence is that long)
        P -= P % kTok;
        int members = 0, leader = INT_MAX;
        for (int b = o0 + lane; b < o1 && P > 0; b += 32)
            if (a.seq_len[b] >= P) {
                ++members;
                leader = min(leader, b);
            }
        members = __reduce_add_sync(0xFFFFFFFFu, members);
        leader = __reduce_min_sync(0xFFFFFFFFu, leader);
        if (members < 2) P = 0;
        for (int b = o0 + lane; b < o1 && P > 0; b += 32)
            if (a.seq_len[b] >= P) {
                a.seq_pre[b] = P;
                a.seq_group[b] = g;
            }
        if (lane == 0) a.groups[g] = make_int4(o0, o1 - o0, P / kTok, P > 0 ? leader : 0);
    }
    __syncthreads();
    int before = 0, total;
    for (int base = 0; base < G; base += kPlanThreads) {
        const int g = base + tid;
        int v = 0;
        if (g < G) {
            const int4 u = a.groups[g];
            v = (u.y + a.seqs_per_tile - 1) / a.seqs_per_tile * Hkv * u.z;
        }
        const int incl = before + plan_scan(v, sums, &total);
        if (g < G) {
            cum_p[g] = incl - v;
            a.cum_p[g] = incl - v;
        }
        before += total;
    }
    const int T1 = before;
    before = 0;
    for (int base = 0; base < B; base += kPlanThreads) {
        const int b = base + tid;
        const int v = b < B ? ((a.seq_len[b] + kTok - 1) / kTok - a.seq_pre[b] / kTok) * Hkv : 0;
        const int incl = before + plan_scan(v, sums, &total);
        if (b < B) {
            cum_s[b] = incl - v;
            a.cum_s[b] = incl - v;
        }
        before += total;
    }
    const int T2 = before;
    if (tid == 0) {
        a.totals[0] = T1;
        a.totals[1] = T2;
    }
    __syncthreads();
    for (int c = tid; c < a.ctas; c += kPlanThreads) {
        int i, x, left;
        range_start(cum_p, G, T1, a.ctas, c, &i, &x, &left);
        const int nt = left > 0 ? a.groups[i].z : 1;
        a.starts[c] = make_int4(i, x / nt, x % nt, left);
        range_start(cum_s, B, T2, a.ctas, c, &i, &x, &left);
        const int ns = left > 0 ? (a.seq_len[i] + kTok - 1) / kTok - a.seq_pre[i] / kTok : 1;
        a.starts[a.ctas + c] = make_int4(i, x / ns, x % ns, left);
    }
}

// ------------------------------------------------------------------- walk
// The tiles of this CTA, in order: its range of one list, then of the other.
// CTA c has range c of the shared tiles and the c-th range from the end of the
// own tiles, so that short lists fall to different CTAs.
struct Walk {
    int own = 0;             // 0: shared tiles of a group, 1: own tiles of a sequence
    int phase = 0, left = 0;
    int i = 0, u = 0;        // group or sequence; KV head, or row tile * KV heads + KV head
    int t = 0, nt = 0;       // tile of the unit, its tiles
    int row = 0, tile0 = 0;  // table row; first tile's index in the sequence
    int end = 0;             // tokens visible to the unit's rows
    int seq0 = 0, nseq = 0;  // sequences of the unit's row tile
    bool first = true;       // at the first tile of a segment

    __device__ bool more() const { return left > 0; }
    __device__ bool last() const { return left == 1 || t == nt - 1; }
    __device__ int head(const PrefixArgs& a) const { return u % a.num_kv_heads; }
    __device__ int rows(const PrefixArgs& a) const { return nseq * a.gh; }
    __device__ int range(const PrefixArgs& a) const { return own ? a.ctas - 1 - static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x); }
    // first row of this piece in the list's partials.  Consecutive pieces
    // differ by a range, a unit or both, so (rows of the units before) + (range)
    // x (rows of a full unit) never collides.
    __device__ size_t piece_row(const PrefixArgs& a) const {
        const size_t before = static_cast<size_t>(a.gh) * (static_cast<size_t>(a.num_kv_heads) * seq0 +
                                                           static_cast<size_t>(head(a)) * nseq);
        return before + static_cast<size_t>(range(a)) * (own ? a.gh : kRows);
    }

    __device__ void load(const PrefixArgs& a) {
        if (own) {
            const int L = a.seq_len[i], P = a.seq_pre[i];
            row = seq0 = i;
            nseq = 1;
            tile0 = P / kTok;
            nt = (L + kTok - 1) / kTok - tile0;
            end = L;
        } else {
            const int4 g = a.groups[i];
            const int r = u / a.num_kv_heads;
            row = g.w;
            nt = g.z;
            tile0 = 0;
            end = nt * kTok;
            seq0 = g.x + r * a.seqs_per_tile;
            nseq = min(a.seqs_per_tile, g.y - r * a.seqs_per_tile);
        }
    }
    __device__ void start(const PrefixArgs& a) {
        own = phase ^ static_cast<int>(blockIdx.x & 1);
        const int4 s = a.starts[own * a.ctas + range(a)];
        i = s.x, u = s.y, t = s.z, left = s.w;
        first = true;
        if (left > 0) load(a);
    }
    __device__ void init(const PrefixArgs& a) {
        start(a);
        if (left == 0) {
            phase = 1;
            start(a);
        }
    }
    __device__ void next(const PrefixArgs& a) {
        --left;
        ++t;
        first = false;
        if (left == 0) {
            if (phase == 0) {
                phase = 1;
                start(a);
            }
            return;
        }
        if (t < nt) return;
        t = 0;
        first = true;
        ++u;
        if (own) {
            if (u < a.num_kv_heads) return;
            u = 0;
            do {
                ++i;
                load(a);
            } while (nt <= 0);
        } else {
            const int4 g = a.groups[i];
            const int units = (g.y + a.seqs_per_tile - 1) / a.seqs_per_tile * a.num_kv_heads;
            if (u < units) {
                load(a);
                return;
            }
            u = 0;
            do {
                ++i;
                load(a);
            } while (nt <= 0 || nseq <= 0);
        }
    }
};

__global__ void __launch_bounds__(kThreads, 2)
prefix_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const PrefixArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = su32(smem), bars = sbase + kBarOff;
    auto B = [&](int i) { return bars + 8u * i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kBarOff + 8 * kNumBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kBarOff + 8 * kNumBars + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kNumBars; ++i)
            bar_init(B(i), ((i >= kPFull && i < kPFull + kNS) || i == kQReady || i == kOFree) ? 4u : 1u);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(su32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the plan, and everything before it
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    auto fail = [&]() {
        *abort_flag = 1;
        if (a.err) atomicOr(a.err, PKV_ERRBIT_TIMEOUT);
    };
    Walk w;
    w.init(a);

    if (warp == 4 || warp == 6) {
        // ------------------------------------------- producers: K (warp 4), V (warp 6)
        // Stage s is freed by the completion that signals score buffer s: S
        // done for K, PV done for V.
        const bool is_v = warp == 6;
        const CUtensorMap* map = is_v ? &tmv : &tmk;
        const int full0 = is_v ? kVFull : kKFull, empty0 = is_v ? kPvDone : kSFull;
        const int bs = a.block_size;
        const int64_t layer_blk0 = static_cast<int64_t>(a.layer) * a.num_blocks;
        int cache = 0, cache_base = 0, cache_row = -1;  // 32 table entries, one per lane
        int k = 0;
        for (; w.more() && !*abort_flag; w.next(a), ++k) {
            const int s = k % kNS;
            const int tok0 = (w.tile0 + w.t) * kTok, n = min(kTok, w.end - tok0), nblk = (n + bs - 1) / bs;
            const int idx0 = tok0 / bs;
            if (w.row != cache_row || idx0 < cache_base || idx0 + nblk > cache_base + 32) {
                cache_row = w.row;
                cache_base = idx0;
                const int idx = idx0 + lane;
                cache = idx < a.max_blocks ? __ldg(a.tables + static_cast<size_t>(w.row) * a.max_blocks + idx) : 0;
            }
            if (k >= kNS && !bar_wait(B(empty0 + s), ((k / kNS) - 1) & 1)) {
                if (lane == 0) fail();
                break;
            }
            const uint32_t dst0 = sbase + kKVOff + s * kStageBytes + (is_v ? 2 * kHalfBytes : 0);
            if (lane == 0) bar_expect_tx(B(full0 + s), static_cast<uint32_t>(nblk * bs * 128 * 2));
            __syncwarp();
            const int kb = lane >> 1, hf = lane & 1;  // one copy instruction: lane 2 kb + hf, half hf of block kb
            int blk = __shfl_sync(0xFFFFFFFFu, cache, (idx0 + kb - cache_base) & 31);
            if (kb < nblk) {
                if (static_cast<unsigned>(blk) >= static_cast<unsigned>(a.num_blocks)) {
                    if (a.err) atomicOr(a.err, PKV_ERRBIT_BLOCK_ID);
                    blk = 0;  // an in-bounds block; the flag marks the output invalid
                }
                const int y = static_cast<int>(((layer_blk0 + blk) * a.num_kv_heads + w.head(a)) * bs);
                tma_3d(dst0 + hf * kHalfBytes + kb * bs * 128, map, 0, y, hf, B(full0 + s));
            }
        }
        // drain: the copies in flight land before the CTA frees anything
        if (lane == 0)
            for (int j = k - 1; j >= 0 && j >= k - kNS; --j)
                if (!bar_wait(B(full0 + j % kNS), (j / kNS) & 1)) fail();
    } else if (warp == 5) {
        // ------------------------------------------------------- MMA issuer
        if (lane == 0) {
            bool ok = true;
            const uint64_t dq = sdesc(sbase, 16);
            const uint64_t dk0 = sdesc(sbase + kKVOff, 16);
            const uint64_t dv0 = sdesc(sbase + kKVOff + 2 * kHalfBytes, kHalfBytes);
            Walk ws = w;
            int ns = 0, seg_s = 0, seg = 0;  // S issued; segments begun by the S and by the PV cursor
            for (int k = 0; w.more() && ok && !*abort_flag; w.next(a), ++k) {
                // S of tile k, and of k + 1 (whose scores' buffer PV k - 1, issued
                // already, has read).  Both may block: the softmax of tile k
                // needs nothing further to signal P k or to store the next Q.
                while (ws.more() && ns < k + kNS) {
                    const int st = ns % kNS;
                    if (ws.first && !bar_wait(B(kQReady), seg_s & 1)) {
                        ok = false;
                        break;
                    }
                    if (!bar_wait(B(kKFull + st), (ns / kNS) & 1)) {
                        ok = false;
                        break;
                    }
                    if (ws.first) ++seg_s;
                    fence_after();
                    const uint64_t dk = dk0 + static_cast<uint64_t>((st * kStageBytes) >> 4);
                    const uint32_t sb = tmem + static_cast<uint32_t>(st * kTok);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        const uint32_t kin = (ks & 3) * 32;
                        mma_bf16(sb, dq + (((ks >> 2) * kQHalf + kin) >> 4), dk + (((ks >> 2) * kHalfBytes + kin) >> 4),
                                 idesc(kTok, 0), ks > 0 ? 1u : 0u);
                    }
                    mma_commit(B(kSFull + st));
                    ws.next(a);
                    ++ns;
                }
                if (!ok) break;
                const int s = k % kNS;
                if (!bar_wait(B(kPFull + s), (k / kNS) & 1) || !bar_wait(B(kVFull + s), (k / kNS) & 1)) {
                    ok = false;
                    break;
                }
                if (w.first && seg > 0 && !bar_wait(B(kOFree), (seg - 1) & 1)) {  // O has been read out
                    ok = false;
                    break;
                }
                if (w.first) ++seg;
                fence_after();
                const uint64_t dv = dv0 + static_cast<uint64_t>((s * kStageBytes) >> 4);
                const uint32_t pb = tmem + static_cast<uint32_t>(s * kTok);
#pragma unroll
                for (int ks = 0; ks < kTok / 16; ++ks)
                    mma_bf16_ta(tmem + kOCol, pb + 8 * ks, dv + ((ks * 16 * 128) >> 4), idesc(kDim, 1),
                                (!w.first || ks > 0) ? 1u : 0u);
                mma_commit(B(kPvDone + s));
            }
            if (!ok) fail();
            mma_commit(B(kDone));  // completes once every MMA issued above has finished
            if (!bar_wait(B(kDone), 0)) fail();
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ softmax and epilogue
        const int m = threadIdx.x;  // row of the tile = TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>(32 * warp) << 16;
        const int gh = a.gh;
        const int dseq = m / gh, dhead = m % gh;
        const float qk = a.qk_scale_log2;
        // Q rows of a unit -> shared memory; the rows of warps without one
        // keep what they held (their scores are never read)
        auto load_q = [&](const Walk& wq) {
            const int nv = wq.rows(a);
            if (32 * warp < nv) {
                const bool valid = m < nv;
                const uint4* src = reinterpret_cast<const uint4*>(
                    static_cast<const __nv_bfloat16*>(a.q) +
                    (static_cast<size_t>(wq.seq0 + (valid ? dseq : 0)) * a.num_q_heads +
                     static_cast<size_t>(wq.head(a)) * gh + dhead) *
                        kDim);
#pragma unroll 4
                for (int ch = 0; ch < 16; ++ch) {
                    const uint4 v = valid ? __ldg(src + ch) : make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4*>(smem + tile_off(m, ch, kQHalf)) = v;
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) bar_arrive(B(kQReady));
        };
        if (w.more()) load_q(w);

        float m_used = -INFINITY, l = 0.f;
        bool ok = true;
        for (int k = 0; w.more(); w.next(a), ++k) {
            const int s = k % kNS, tok0 = (w.tile0 + w.t) * kTok;
            const bool busy = 32 * warp < w.rows(a);
            const int visible = w.end - tok0;  // of this tile, the same for every row
            if (w.first) {
                m_used = -INFINITY;
                l = 0.f;
            }
            if (!bar_wait_warp(B(kSFull + s), (k / kNS) & 1)) {
                ok = false;
                break;
            }
            fence_after();
            const uint32_t sa = tmem + lane_off + static_cast<uint32_t>(s * kTok);
            bool rescale = false;
            float alpha = 1.f;
            if (busy) {
                uint32_t v[kTok];
#pragma unroll
                for (int c4 = 0; c4 < kTok / 32; ++c4) tmem_ld32_nowait(sa + 32 * c4, v + 32 * c4);
                asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
                const bool full = visible >= kTok;
                float mx = -INFINITY;
                if (full && qk > 0.f) {
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < kTok; i += 2)
                        m4[(i >> 1) & 3] = max3(m4[(i >> 1) & 3], __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                    mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * qk;
                } else {
#pragma unroll
                    for (int i = 0; i < kTok; ++i)
                        if (i < visible) mx = fmaxf(mx, __uint_as_float(v[i]) * qk);
                }
                const float m_new = fmaxf(m_used, mx);
                rescale = m_used != -INFINITY && m_new > m_used + 8.f;
                const float base_new = m_used == -INFINITY || rescale ? m_new : m_used;
                alpha = rescale ? ex2(m_used - m_new) : 1.f;
                m_used = base_new;
                const float base = m_used == -INFINITY ? 0.f : m_used;
                uint32_t pk[kTok / 2];
                float lt = 0.f;
                if (full) {
                    float l0 = 0.f, l1 = 0.f;
#pragma unroll
                    for (int i = 0; i < kTok / 2; ++i) {
                        float x0, x1;
                        fma2(x0, x1, __uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]), qk, qk, -base, -base);
                        const float p0 = ex2(x0), p1 = ex2(x1);
                        add2(l0, l1, l0, l1, p0, p1);
                        pk[i] = bf16x2(p0, p1);
                    }
                    lt = l0 + l1;
                } else {
#pragma unroll
                    for (int i = 0; i < kTok / 2; ++i) {
                        const float p0 = 2 * i < visible ? ex2(fmaf(__uint_as_float(v[2 * i]), qk, -base)) : 0.f;
                        const float p1 = 2 * i + 1 < visible ? ex2(fmaf(__uint_as_float(v[2 * i + 1]), qk, -base)) : 0.f;
                        lt += p0 + p1;
                        pk[i] = bf16x2(p0, p1);
                    }
                }
                l = l * alpha + lt;
                tmem_st32(sa, pk);
            }
            // Every PV before S k has finished (MMAs complete in order) and PV
            // k + 1 cannot finish before P k + 1 is signalled, so a parity wait
            // for PV k - 1 or PV k is unambiguous.
            if (busy && __any_sync(0xFFFFFFFFu, rescale)) {
                if (!bar_wait_warp(B(kPvDone + (k - 1) % kNS), ((k - 1) / kNS) & 1)) {
                    ok = false;
                    break;
                }
                fence_after();
#pragma unroll 1
                for (int c4 = 0; c4 < 4; ++c4) {
                    uint32_t o[32];
                    const uint32_t oa = tmem + lane_off + kOCol + 32 * c4;
                    tmem_ld32(oa, o);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                    tmem_st32(oa, o);
                }
            }
            // V rows past the last token: zero (stale or unwritten rows could hold NaN)
            if (visible < kTok) {
                if (!bar_wait_warp(B(kVFull + s), (k / kNS) & 1)) {
                    ok = false;
                    break;
                }
                uint8_t* vs = smem + kKVOff + s * kStageBytes + 2 * kHalfBytes;
                const int nz = kTok - visible;
                for (int e = m; e < 2 * nz * 8; e += 128) {  // whole 128-byte rows: the swizzle does not matter
                    const int hf = e / (nz * 8), rem = e % (nz * 8);
                    *reinterpret_cast<uint4*>(vs + hf * kHalfBytes + (visible + rem / 8) * 128 + (rem % 8) * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
                }
                fence_async_smem();
            }
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(B(kPFull + s));
            if (!w.last()) continue;

            // ---- the unit's piece ends: its last S is done, so the next Q may be stored
            {
                Walk wn = w;
                wn.next(a);
                if (wn.more()) load_q(wn);
            }
            if (!bar_wait_warp(B(kPvDone + s), (k / kNS) & 1)) {
                ok = false;
                break;
            }
            fence_after();
            if (busy) {
                const bool valid = m < w.rows(a);
                const float inv = l > 0.f ? 1.f / l : 0.f;
                const size_t prow = w.piece_row(a) + (valid ? m : 0);
                float* po = (w.own ? a.own_o : a.pre_o) + prow * kDim;
#pragma unroll 1
                for (int c4 = 0; c4 < 4; ++c4) {
                    uint32_t v[32];
                    tmem_ld32(tmem + lane_off + kOCol + 32 * c4, v);
                    if (!valid) continue;
                    float4* dst = reinterpret_cast<float4*>(po + 32 * c4);
#pragma unroll
                    for (int q4 = 0; q4 < 8; ++q4)
                        dst[q4] = make_float4(__uint_as_float(v[4 * q4 + 0]) * inv, __uint_as_float(v[4 * q4 + 1]) * inv,
                                              __uint_as_float(v[4 * q4 + 2]) * inv, __uint_as_float(v[4 * q4 + 3]) * inv);
                }
                if (valid) (w.own ? a.own_lse : a.pre_lse)[prow] = l > 0.f ? m_used + log2f(l) : -INFINITY;
            }
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(B(kOFree));
        }
        if (!ok && lane == 0) fail();
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// ------------------------------------------------------------------ merge
constexpr int kMergeThreads = 256;

// One warp per output row; lane d holds columns 4 d .. 4 d + 3.
__global__ void __launch_bounds__(kMergeThreads) prefix_merge_kernel(const PrefixArgs a) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int64_t out_row = blockIdx.x * static_cast<int64_t>(kMergeThreads / 32) + (threadIdx.x >> 5);
    if (out_row >= static_cast<int64_t>(a.num_seqs) * a.num_q_heads) return;
    const int b = static_cast<int>(out_row / a.num_q_heads), hq = static_cast<int>(out_row % a.num_q_heads);
    const int h = hq / a.gh, Hkv = a.num_kv_heads;
    const int L = a.seq_len[b], P = a.seq_pre[b], g = a.seq_group[b];

    // the two lists' pieces of this row: ranges c0 .. c0 + n - 1, rows base + c * step
    int c0[2] = {0, 0}, n[2] = {0, 0};
    size_t base[2] = {0, 0};
    if (g >= 0) {
        const int4 u = a.groups[g];
        const int r = (b - u.x) / a.seqs_per_tile, seq0 = u.x + r * a.seqs_per_tile;
        const int nseq = min(a.seqs_per_tile, u.y - r * a.seqs_per_tile);
        const int T = a.totals[0], ps = a.cum_p[g] + (r * Hkv + h) * u.z;
        c0[0] = range_of(ps, T, a.ctas);
        n[0] = range_of(ps + u.z - 1, T, a.ctas) - c0[0] + 1;
        base[0] = static_cast<size_t>(a.gh) * (static_cast<size_t>(Hkv) * seq0 + static_cast<size_t>(h) * nseq) +
                  (b - seq0) * a.gh + hq % a.gh;
    }
    const int nt = (L + kTok - 1) / kTok - P / kTok;
    if (nt > 0) {
        const int T = a.totals[1], ps = a.cum_s[b] + h * nt;
        c0[1] = range_of(ps, T, a.ctas);
        n[1] = range_of(ps + nt - 1, T, a.ctas) - c0[1] + 1;
        base[1] = static_cast<size_t>(out_row);
    }
    const int pieces = n[0] + n[1];
    auto row_of = [&](int j) {
        return j < n[0] ? base[0] + static_cast<size_t>(c0[0] + j) * kRows
                        : base[1] + static_cast<size_t>(c0[1] + j - n[0]) * a.gh;
    };
    auto lse_of = [&](int j) { return j < n[0] ? a.pre_lse[row_of(j)] : a.own_lse[row_of(j)]; };
    float M = -INFINITY;
    for (int j = lane; j < pieces; j += 32) M = fmaxf(M, lse_of(j));
    M = warp_max(M);
    float z = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j0 = 0; j0 < pieces; j0 += 32) {
        float wt = 0.f;
        if (j0 + lane < pieces) {
            const float s = lse_of(j0 + lane);
            wt = s == -INFINITY ? 0.f : exp2f(s - M);
        }
        z += warp_sum(wt);
        const int last = min(32, pieces - j0);
#pragma unroll 4
        for (int j = 0; j < last; ++j) {
            const float wj = __shfl_sync(0xFFFFFFFFu, wt, j);
            const float* o = (j0 + j < n[0] ? a.pre_o : a.own_o) + row_of(j0 + j) * kDim;
            const float4 v = reinterpret_cast<const float4*>(o)[lane];
            acc.x = fmaf(wj, v.x, acc.x);
            acc.y = fmaf(wj, v.y, acc.y);
            acc.z = fmaf(wj, v.z, acc.z);
            acc.w = fmaf(wj, v.w, acc.w);
        }
    }
    const float inv = z > 0.f ? a.v_scale / z : 0.f;  // no token: a zero row
    uint2 pk;
    pk.x = bf16x2(acc.x * inv, acc.y * inv);
    pk.y = bf16x2(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + out_row * kDim + 4 * lane) = pk;
}

}  // namespace

cudaError_t launch_prefix_attention(const PrefixArgs& a, const void* tmap_k, const void* tmap_v, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static uint64_t configured = 0;
    if (dev < 0 || dev >= 64) return cudaErrorNotSupported;
    if (!(configured >> dev & 1)) {
        e = cudaFuncSetAttribute(prefix_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(prefix_tc_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
        configured |= 1ull << dev;
    }
    prefix_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_dependent(prefix_tc_kernel, dim3(a.ctas), dim3(kThreads), kSmem, stream,
                         *static_cast<const CUtensorMap*>(tmap_k), *static_cast<const CUtensorMap*>(tmap_v), a);
    if (e != cudaSuccess) return e;
    const int64_t rows = static_cast<int64_t>(a.num_seqs) * a.num_q_heads;
    constexpr int per = kMergeThreads / 32;
    return launch_dependent(prefix_merge_kernel, dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(kMergeThreads),
                            0, stream, a);
}

}  // namespace pkv
