// Block tables, slot maps and the free list of a decode step, built on the
// GPU from request lengths, so that a step (or a captured loop of steps)
// needs no host block manager in between ("How does TensorRT-LLM work?", "The
// paged KV cache": blocks are handed out one at a time when a request needs
// more room and go back the moment it finishes; "TensorRT-LLM, in depth",
// "In-flight batching and the scheduler": a request that cannot get a block
// waits).
//
// Growing.  With L_b tokens cached and n_b new ones, request b holds
// h_b = ceil(L_b / bs) blocks and needs d_b = ceil((L_b + n_b) / bs) - h_b
// more.  Handing blocks out in request order is a prefix sum: request b takes
// entries D_b .. D_b + d_b - 1 of the free list, D_b = d_0 + .. + d_{b-1}, if
// D_b + d_b does not exceed the number of free blocks; a later request never
// overtakes one that had to wait, except for those that need no block.
// Releasing is the same sum over the blocks given back, behind the list's
// tail.
//
// A batch is at most some thousand lengths, so nothing here is bound by bytes:
// a call costs its launch, a few dependent rounds to L2, and the instructions
// that one SM issues.  Hence one CTA that scans 1024 requests a round (both
// sums at once, in 32 bits that saturate, one barrier), writes tables and, where
// they are few, the slots too; a second kernel, launched to start as the first
// ends, fills longer slot maps, one thread per token row.
// (Block sizes are powers of two; with runtime divisions instead of shifts the
// scan took four times as long.)  256 requests of one token each: 3.3 us, of
// which an empty launch is 2; 1024 requests, 128 of them prompts of up to 2048
// tokens, 8 thousand blocks and 131 thousand rows: 11.5 us, six of them in the
// one CTA.  Releases of a quarter of 256 requests: 4.6 us; of 4096 requests'
// two hundred thousand blocks: 6.6 us.
#include "device_common.cuh"
#include "step_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kDirect = 2;           // rows or blocks of a request that its own thread writes
constexpr int kAhead = 8;            // blocks that a thread fetches at once
constexpr int kFillThreads = 256;

// Sums end at kMost, which stands for "too many" (limits are at most 2^30): half
// the instructions of 64-bit sums, and one SM issues them all.
constexpr int kMost = INT32_MAX;
__device__ __forceinline__ int sat(long long x) { return static_cast<int>(x < kMost ? x : kMost); }
__device__ __forceinline__ int sat_add(int a, int b) {  // of values 0 .. kMost
    return static_cast<int>(min(static_cast<unsigned>(a) + static_cast<unsigned>(b), static_cast<unsigned>(kMost)));
}
// Exclusive sums of N values over the CTA's threads; total[] gets the sums of
// all of them.  (The caller has a barrier before `sums` is written again.)
template <int N>
__device__ __forceinline__ void block_scan(int (&v)[N], int (*sums)[kWarps], int (&total)[N]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int x = __shfl_up_sync(0xFFFFFFFFu, v[e], o);
            if (lane >= o) v[e] = sat_add(v[e], x);
        }
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if (lane == 31) sums[e][warp] = v[e];
        v[e] = __shfl_up_sync(0xFFFFFFFFu, v[e], 1);
        if (lane == 0) v[e] = 0;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < N; ++e) {
        int s = lane < nw ? sums[e][lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xFFFFFFFFu, s, o);
            if (lane >= o) s = sat_add(s, x);
        }
        total[e] = __shfl_sync(0xFFFFFFFFu, s, nw - 1);
        const int before = __shfl_sync(0xFFFFFFFFu, s, max(warp - 1, 0));
        if (warp > 0) v[e] = sat_add(v[e], before);
    }
}

// Block sizes are powers of two: blocks that `a` tokens occupy.
__device__ __forceinline__ long long blocks_of(long long a, int shift) { return (a + (1LL << shift) - 1) >> shift; }
__device__ __forceinline__ int sat_pos(long long p) { return p > INT32_MAX ? INT32_MAX : static_cast<int>(p); }

struct FreeRing {
    const int32_t* ring;
    int cap, head;
    __device__ __forceinline__ unsigned index(int i) const {  // i <= cap, head < cap
        const unsigned x = static_cast<unsigned>(head) + static_cast<unsigned>(i), c = static_cast<unsigned>(cap);
        return x >= c ? x - c : x;
    }
};

// A request of a round of the scan.
struct Job {
    int b, L;
    int first;   // its first entry of the free list, counted from the head
    int served;
};
// The last of n ascending starts that is <= x (starts[0] is): with starts that
// are exclusive sums of counts, the item that holds place x.  (Sixty
// instructions; all threads of one SM share its issue slots, so that those who
// take consecutive places search only where one has left its item.)
__device__ __forceinline__ int holder(const int* starts, int n, int x) {
    int lo = 0;
#pragma unroll
    for (int step = kThreads / 2; step > 0; step >>= 1)
        if (lo + step < n && starts[lo + step] <= x) lo += step;
    return lo;
}

// Block id read from a table or the free list: -1 (flagged) outside the pool.
__device__ __forceinline__ int checked_block(int blk, int num_blocks, int32_t* err) {
    if (static_cast<unsigned>(blk) < static_cast<unsigned>(num_blocks)) return blk;
    if (err) atomicOr(err, PKV_ERRBIT_BLOCK_ID);
    return -1;
}

// Entry `i` of the free list, counted from the head, to place `at` of the tables.
__device__ __forceinline__ void grow_entry(const GrowArgs& a, const FreeRing& f, long long at, int i) {
    a.tables[at] = checked_block(__ldg(f.ring + f.index(i)), a.num_blocks, a.err);
}

__device__ __forceinline__ void grow_row(const GrowArgs& a, const FreeRing& f, const Job& j, int row, int i) {
    const long long p = static_cast<long long>(j.L > 0 ? j.L : 0) + i;
    long long slot = -1;
    if (j.served) {
        const int held = static_cast<int>(blocks_of(j.L, a.block_shift)), col = static_cast<int>(p >> a.block_shift);
        // the last block held may have room; the others come from the free list
        const int blk = col < held ? a.tables[static_cast<size_t>(j.b) * a.max_blocks + col]
                                   : f.ring[f.index(j.first + (col - held))];
        if (checked_block(blk, a.num_blocks, a.err) >= 0)
            slot = (static_cast<long long>(blk) << a.block_shift) + (p & ((1LL << a.block_shift) - 1));
    }
    a.slots[row] = slot;
    a.positions[row] = sat_pos(p);
    a.token_seqs[row] = j.b;
}

// lens_out may be lens and free_out may be free_state: every request's values
// are read by the thread that writes them, and the free list's state by every
// thread before the first barrier.
__global__ void __launch_bounds__(kThreads, 1) grow_kernel(const GrowArgs a, const int fill_rows) {
    __shared__ int sums[2][kWarps];
    __shared__ Job jobs[kThreads];
    // of the round's requests: first block and first row of each, counted from
    // the round's first; place of its blocks in the tables, less the former
    __shared__ int entry_start[kThreads], row_start[kThreads];
    __shared__ long long entry_at[kThreads];
    __shared__ int taken;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    FreeRing f{a.ring, a.ring_size, a.free_state[0]};
    int count = a.free_state[1];
    const bool bad_state = f.head < 0 || f.head >= f.cap || count < 0 || count > f.cap;
    if (threadIdx.x == 0) {
        taken = 0;
        if (bad_state && a.err) atomicOr(a.err, PKV_ERRBIT_STEP);
    }
    if (bad_state) count = 0;
    const int head0 = f.head, count0 = a.free_state[1];
    if (bad_state) f.head = 0;
    const long long room = static_cast<long long>(a.max_blocks) << a.block_shift;
    const int lane = threadIdx.x & 31;

    int rows_before = 0, need_before = 0;
    for (int base = 0; base < a.num_seqs; base += blockDim.x) {
        const int b = base + threadIdx.x, round = min(a.num_seqs - base, static_cast<int>(blockDim.x));
        const bool in = b < a.num_seqs;
        const int L = in ? a.lens[b] : 0, n = in ? a.new_tokens[b] : 0;
        const int rows = n > 0 ? n : 0;
        const bool len_ok = L >= 0 && L <= room;
        // Requests past max_tokens still count in the sum of needs: all
        // later ones with new tokens are past it too, so it changes nothing.
        const bool fits = in && len_ok && n >= 0 && static_cast<long long>(L) + n <= room;
        const int held = static_cast<int>(blocks_of(len_ok ? L : 0, a.block_shift));
        const int need = fits ? static_cast<int>(blocks_of(static_cast<long long>(L) + n, a.block_shift)) - held : 0;
        int before[2] = {rows, need}, total[2];
        block_scan(before, sums, total);
        const int off = sat_add(rows_before, before[0]), first = sat_add(need_before, before[1]);
        const bool rows_ok = n >= 0 && (n == 0 || sat_add(off, n) <= a.max_tokens);
        if (in && a.err && (!len_ok || !rows_ok)) atomicOr(a.err, (len_ok ? 0 : PKV_ERRBIT_SEQ_LEN) | (rows_ok ? 0 : PKV_ERRBIT_STEP));
        // (served requests that need blocks come before all others that do)
        const bool served = fits && rows_ok && (need == 0 || sat_add(first, need) <= count);
        const int off_in = min(off, a.max_tokens), off0 = min(rows_before, a.max_tokens);
        const Job j{b, L, served ? first : 0, served ? 1 : 0};
        const long long at = static_cast<long long>(b) * a.max_blocks + held;
        jobs[threadIdx.x] = j;
        entry_start[threadIdx.x] = before[1];
        entry_at[threadIdx.x] = at - before[1];
        row_start[threadIdx.x] = off_in - off0;
        if (in) {
            a.token_offsets[b] = off_in;
            a.granted[b] = served ? n : 0;
            a.lens_out[b] = served ? L + n : L;
            if (served && need > 0) atomicMax(&taken, first + need);
        }
        // A few blocks and rows each, by the request's own thread; else shared
        // out over all threads, each finding the request that its entry is of.
        if (!__syncthreads_or((served && need > kDirect) || (fill_rows && rows > kDirect))) {
            if (served)
                for (int i = 0; i < need; ++i) grow_entry(a, f, at + i, first + i);
            if (in && fill_rows)
                for (int i = 0; i < rows && off_in + i < a.max_tokens; ++i) grow_row(a, f, j, off_in + i, i);
        } else {
            const int entries = taken - min(need_before, taken);
            const int stride = (entries + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x) * 32;  // of a warp
            const int e0 = (threadIdx.x >> 5) * stride + lane, last = min(entries, e0 - lane + stride);
            int i = -1;
            for (int e = e0; e < last; e += 32 * kAhead) {  // kAhead loads under way at once
                int blk[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) blk[u] = e + 32 * u < last ? __ldg(f.ring + f.index(need_before + e + 32 * u)) : 0;
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int x = e + 32 * u;
                    if (x >= last) break;
                    if (i < 0 || (i + 1 < round && entry_start[i + 1] <= x)) i = holder(entry_start, round, x);
                    a.tables[entry_at[i] + x] = checked_block(blk[u], a.num_blocks, a.err);
                }
            }
            if (fill_rows) {
                const int num_rows = min(sat_add(rows_before, total[0]), a.max_tokens) - off0;
                const int stride = (num_rows + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x) * 32;
                for (int r = (threadIdx.x >> 5) * stride + lane, last = min(num_rows, r - lane + stride), i = -1; r < last; r += 32) {
                    if (i < 0 || (i + 1 < round && row_start[i + 1] <= r)) i = holder(row_start, round, r);
                    grow_row(a, f, jobs[i], off0 + r, r - row_start[i]);
                }
            }
        }
        rows_before = sat_add(rows_before, total[0]);
        need_before = sat_add(need_before, total[1]);
        __syncthreads();
    }
    const int end = min(rows_before, a.max_tokens);
    if (threadIdx.x == 0) {
        a.token_offsets[a.num_seqs] = end;
        a.free_out[0] = bad_state ? head0 : f.index(taken);
        a.free_out[1] = bad_state ? count0 : count - taken;
    }
    if (fill_rows)
        for (int r = end + threadIdx.x; r < a.max_tokens; r += blockDim.x) {
            a.slots[r] = -1;
            a.positions[r] = 0;
            a.token_seqs[r] = -1;
        }
}

// Slots of long steps, one thread per token row.  A warp's 32 rows mostly
// belong to one request: the warp finds the first row's by a 32-way search over
// the row offsets (two rounds of loads for a thousand requests), and only rows
// behind that request's last search on.
__global__ void __launch_bounds__(kFillThreads) fill_kernel(const GrowArgs a) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int lane = threadIdx.x & 31;
    const long long row = blockIdx.x * static_cast<long long>(kFillThreads) + threadIdx.x, row0 = row - lane;
    if (row0 >= a.max_tokens) return;  // (the whole warp)
    const int end = a.token_offsets[a.num_seqs];
    long long slot = -1;
    int pos = 0, seq = -1;
    int lo = 0, hi = a.num_seqs;  // the last request whose first row is <= row0 (the loads do not wait for `end`)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5, at = lo + lane * step;
        const unsigned below = __ballot_sync(0xFFFFFFFFu, at < hi && a.token_offsets[at] <= row0);
        lo += (31 - __clz(below)) * step;  // (lane 0 always is)
        hi = min(hi, lo + step);
    }
    if (row < end) {
        // (what a row needs of its request, in one round: mostly it is the first row's)
        int n = a.granted[lo], len = a.lens_out[lo], first = a.token_offsets[lo];
        if (a.token_offsets[lo + 1] <= row) {
            for (hi = a.num_seqs; hi - lo > 1;) {
                const int mid = (lo + hi) >> 1;
                if (a.token_offsets[mid] <= row) lo = mid;
                else hi = mid;
            }
            n = a.granted[lo], len = a.lens_out[lo], first = a.token_offsets[lo];
        }
        seq = lo;
        const int L = len - n;  // the length before the step
        const long long p = static_cast<long long>(L > 0 ? L : 0) + (row - first);
        pos = sat_pos(p);
        if (n > 0) {
            const int blk = checked_block(
                a.tables[static_cast<size_t>(seq) * a.max_blocks + (p >> a.block_shift)], a.num_blocks, a.err);
            if (blk >= 0) slot = (static_cast<long long>(blk) << a.block_shift) + (p & ((1LL << a.block_shift) - 1));
        }
    }
    if (row >= a.max_tokens) return;
    a.slots[row] = slot;
    a.positions[row] = pos;
    a.token_seqs[row] = seq;
}

// ---------------------------------------------------------------- release
constexpr int kReleasePerCta = kWarps;  // requests of one CTA of the large form: one per warp
// Requests up to which one CTA does it all (us, half of them finished, one CTA /
// many: 16 requests 2.8 / 3.3, or 15.6 / 16.1 with 64 thousand table entries;
// 128: 3.1 / 3.2 and 10.9 / 9.2; 256: 3.7 / 3.2 and 14.5 / 9.0 with 256
// thousand; 1024: 5.9 / 3.5 and 37 / 9.7 with a million).
constexpr int kSmallRelease = 128;
static_assert(kSmallRelease <= kThreads, "a thread each");

// Blocks request b gives back: entries [*first, *first + *count) of its row.
// *len: its length; *gone: whether it is released (if the ring has room).
struct Given {
    int len, first, count;
    bool gone;
};
__device__ __forceinline__ Given given(const ReleaseArgs& a, int b, bool report) {
    // (unconditional loads: one round to L2)
    const int done = a.finished[b], L = a.lens[b], keep0 = a.keep_blocks ? a.keep_blocks[b] : 0;
    Given g{L, 0, 0, false};
    if (done == 0) return g;
    if (L < 0 || L > static_cast<long long>(a.max_blocks) << a.block_shift) {
        if (report && a.err) atomicOr(a.err, PKV_ERRBIT_SEQ_LEN);
        return g;
    }
    const int held = static_cast<int>(blocks_of(L, a.block_shift));
    g.first = keep0 < 0 ? 0 : (keep0 > held ? held : keep0);
    g.count = held - g.first;
    g.gone = true;
    return g;
}

// Entries k0, k0 + step, .. of what request b gives back, behind the ring's
// `tail` entries.
__device__ __forceinline__ void release_copy(const ReleaseArgs& a, int head, int tail, int b, int first, int count,
                                             int k0, int step) {
    const int32_t* src = a.tables + static_cast<size_t>(b) * a.max_blocks + first;
#pragma unroll 4
    for (int k = k0; k < count; k += step) {
        unsigned at = static_cast<unsigned>(head) + static_cast<unsigned>(tail + k);  // < 2 * ring_size
        if (at >= static_cast<unsigned>(a.ring_size)) at -= static_cast<unsigned>(a.ring_size);
        a.ring[at] = checked_block(src[k], a.num_blocks, a.err);
    }
}

__device__ __forceinline__ bool ring_ok(const ReleaseArgs& a, int head, int count, int total) {
    return head >= 0 && head < a.ring_size && count >= 0 && static_cast<long long>(count) + total <= a.ring_size;
}
__device__ __forceinline__ void put_state(const ReleaseArgs& a, int head, int count, int total, bool ok) {
    a.free_out[0] = head;
    a.free_out[1] = ok ? count + total : count;
    if (!ok && a.err) atomicOr(a.err, PKV_ERRBIT_STEP);
}

// Up to kSmallRelease requests in one CTA: a thread each, then the blocks of
// those that have any by a warp each.  The outputs may be the inputs.
__global__ void __launch_bounds__(kThreads, 1) release_small_kernel(const ReleaseArgs a) {
    __shared__ int sums[1][kWarps];
    struct Run {
        int b, first, count, tail;
    };
    __shared__ Run runs[kSmallRelease];
    __shared__ int num_runs;
    const int head = a.free_state[0], count = a.free_state[1], b = threadIdx.x;
    Given g{0, 0, 0, false};
    if (b < a.num_seqs) g = given(a, b, true);
    if (b == 0) num_runs = 0;
    int before[1] = {g.count}, total[1];
    block_scan(before, sums, total);
    const bool ok = ring_ok(a, head, count, total[0]);
    if (ok && g.count > 0) runs[atomicAdd(&num_runs, 1)] = Run{b, g.first, g.count, count + before[0]};
    if (b < a.num_seqs) a.lens_out[b] = ok && g.gone ? 0 : g.len;
    if (b == 0) put_state(a, head, count, total[0], ok);
    __syncthreads();
    for (int i = b >> 5; i < num_runs; i += static_cast<int>(blockDim.x >> 5))
        release_copy(a, head, runs[i].tail, runs[i].b, runs[i].first, runs[i].count, b & 31, 32);
}

// One pass over the batch: the blocks given back by requests before `upto`
// (*before) and by all of them (*total), for every thread of the CTA.
__device__ __forceinline__ void release_sums(const ReleaseArgs& a, int upto, int (*sums)[kWarps], int* before,
                                             int* total) {
    long long s[2] = {0, 0};
#pragma unroll 4
    for (int b = threadIdx.x; b < a.num_seqs; b += blockDim.x) {
        const int n = given(a, b, false).count;
        s[1] += n;
        if (b < upto) s[0] += n;
    }
    int part[2] = {sat(s[0]), sat(s[1])}, all[2];
    block_scan(part, sums, all);
    *before = all[0];
    *total = all[1];
}

// Larger batches: every CTA sums the whole batch (some tens of KB from L2) and
// moves the blocks of its own 32 requests, a warp each.  Outputs apart from the
// inputs are written here (commit); others by a second kernel, once every CTA
// has read them.
__global__ void __launch_bounds__(kThreads, 1) release_copy_kernel(const ReleaseArgs a, const int commit) {
    __shared__ int sums[2][kWarps];
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int head = a.free_state[0], count = a.free_state[1];
    const int b0 = blockIdx.x * kReleasePerCta, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Given g{0, 0, 0, false};
    if (b0 + lane < a.num_seqs) g = given(a, b0 + lane, warp == 0);
    int before, total;
    release_sums(a, b0, sums, &before, &total);
    const bool ok = ring_ok(a, head, count, total);
    if (commit) {
        if (warp == 0 && b0 + lane < a.num_seqs) a.lens_out[b0 + lane] = ok && g.gone ? 0 : g.len;
        if (b0 == 0 && threadIdx.x == 0) put_state(a, head, count, total, ok);
    }
    if (!ok) return;
    int incl = g.count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += x;
    }
    const int tail = count + before + __shfl_sync(0xFFFFFFFFu, incl - g.count, warp);
    const int first = __shfl_sync(0xFFFFFFFFu, g.first, warp), n = __shfl_sync(0xFFFFFFFFu, g.count, warp);
    if (b0 + warp < a.num_seqs) release_copy(a, head, tail, b0 + warp, first, n, lane, 32);
}

__global__ void __launch_bounds__(kThreads, 1) release_commit_kernel(const ReleaseArgs a) {
    __shared__ int sums[2][kWarps];
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int head = a.free_state[0], count = a.free_state[1];
    int zero, total;
    release_sums(a, 0, sums, &zero, &total);
    const bool ok = ring_ok(a, head, count, total);
    for (int b = threadIdx.x; b < a.num_seqs; b += blockDim.x) {
        const Given g = given(a, b, false);
        a.lens_out[b] = ok && g.gone ? 0 : g.len;
    }
    if (threadIdx.x == 0) put_state(a, head, count, total, ok);
}

}  // namespace

// The scanning CTA fills the token rows itself where they are few, or no more
// than its threads write for their own requests (kDirect each); else the second
// kernel does.  Us, scanning CTA / second kernel, requests x rows in all: 1 x
// 256 3.9 / 4.0, 1 x 1024 4.9 / 4.5; 64 x 256 4.1 / 4.6, 64 x 512 5.2 / 4.6; 256
// x 512 3.5 / 5.0, 256 x 1024 7.0 / 4.8; 1024 x 2048 5.2 / 6.8, 1024 x 4096 9.1 /
// 6.6; 4096 x 4096 12.3 / 12.9, 4096 x 8192 16.6 / 13.3.  256 threads start sooner
// than 1024 (64 requests: 4.6 / 5.2 us), which scan more at once (512: 6.4 / 6.1).
cudaError_t launch_tables_grow(const GrowArgs& a, cudaStream_t stream) {
    const int64_t direct = static_cast<int64_t>(kDirect) * a.num_seqs;
    const bool inline_rows = a.max_tokens <= 256 || a.max_tokens <= (direct < 4096 ? direct : 4096);
    const int threads = a.num_seqs <= 256 ? 256 : kThreads;
    grow_kernel<<<1, threads, 0, stream>>>(a, inline_rows ? 1 : 0);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || inline_rows) return e;
    return launch_dependent(fill_kernel, dim3((a.max_tokens + kFillThreads - 1) / kFillThreads), dim3(kFillThreads), 0,
                            stream, a);
}

cudaError_t launch_tables_release(const ReleaseArgs& a, cudaStream_t stream) {
    if (a.num_seqs <= kSmallRelease) {
        release_small_kernel<<<1, kThreads, 0, stream>>>(a);  // (all 32 warps: they share out the blocks)
        return cudaGetLastError();
    }
    // (arrays that overlap otherwise than by being the same are not for this call)
    const bool apart = a.lens_out != a.lens && a.free_out != a.free_state && a.lens_out != a.finished &&
                       a.lens_out != a.keep_blocks;
    release_copy_kernel<<<(a.num_seqs + kReleasePerCta - 1) / kReleasePerCta, kThreads, 0, stream>>>(a, apart ? 1 : 0);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || apart) return e;
    return launch_dependent(release_commit_kernel, dim3(1), dim3(kThreads), 0, stream, a);
}

}  // namespace pkv
