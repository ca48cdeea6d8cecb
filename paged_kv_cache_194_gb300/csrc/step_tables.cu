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
// a call costs its launch and a few dependent rounds to L2.  Hence one CTA
// that scans 1024 requests a round (registers and shuffles, two barriers per
// sum), writes tables and, for up to kInlineTokens token rows, the slots too;
// a second kernel, launched to start as the first ends, fills longer slot
// maps, one thread per token row.  (Block sizes are powers of two; with runtime
// divisions instead of shifts the scan took four times as long.)
#include "device_common.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kInlineTokens = 8192;  // token rows the scanning CTA fills itself
constexpr int kDirect = 2;           // rows or blocks of a request that its own thread writes
constexpr int kFillThreads = 256;

// Inclusive sum over the CTA's threads; *total gets the sum of all of them.
__device__ __forceinline__ long long block_scan(long long v, long long* warp_sums, long long* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += x;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    const int nw = blockDim.x >> 5;
    const long long mine = lane < nw ? warp_sums[lane] : 0;
    long long s = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += x;
    }
    *total = __shfl_sync(0xFFFFFFFFu, s, nw - 1);
    const long long before = __shfl_sync(0xFFFFFFFFu, s - mine, warp);
    __syncthreads();  // warp_sums may be written again
    return v + before;
}

// Block sizes are powers of two: blocks that `a` tokens occupy.
__device__ __forceinline__ long long blocks_of(long long a, int shift) { return (a + (1LL << shift) - 1) >> shift; }
__device__ __forceinline__ int sat_pos(long long p) { return p > INT32_MAX ? INT32_MAX : static_cast<int>(p); }

struct FreeRing {
    const int32_t* ring;
    int cap, head;
    __device__ __forceinline__ int index(long long i) const {  // i <= cap, head < cap
        const long long x = head + i;
        return static_cast<int>(x >= cap ? x - cap : x);
    }
};

// A request whose rows or blocks are too many for its own thread.
struct Job {
    int b, L, n, off;
    int first;   // its first entry of the free list, counted from the head
    int need;    // blocks it is given
    int served;
};

// Block id read from a table or the free list: -1 (flagged) outside the pool.
__device__ __forceinline__ int checked_block(int blk, int num_blocks, int32_t* err) {
    if (static_cast<unsigned>(blk) < static_cast<unsigned>(num_blocks)) return blk;
    if (err) atomicOr(err, PKV_ERRBIT_BLOCK_ID);
    return -1;
}

__device__ __forceinline__ void grow_entry(const GrowArgs& a, const FreeRing& f, const Job& j, int i) {
    const int blk = checked_block(f.ring[f.index(j.first + static_cast<long long>(i))], a.num_blocks, a.err);
    a.tables[static_cast<size_t>(j.b) * a.max_blocks + blocks_of(j.L, a.block_shift) + i] = blk;
}

__device__ __forceinline__ void grow_row(const GrowArgs& a, const FreeRing& f, const Job& j, int i) {
    const long long row = static_cast<long long>(j.off) + i;
    if (row >= a.max_tokens) return;
    const long long p = static_cast<long long>(j.L > 0 ? j.L : 0) + i;
    long long slot = -1;
    if (j.served) {
        const int held = static_cast<int>(blocks_of(j.L, a.block_shift)), col = static_cast<int>(p >> a.block_shift);
        // the last block held may have room; the others come from the free list
        const int blk = col < held ? a.tables[static_cast<size_t>(j.b) * a.max_blocks + col]
                                   : f.ring[f.index(j.first + static_cast<long long>(col - held))];
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
    __shared__ long long sums[kWarps];
    __shared__ Job jobs[kThreads];
    __shared__ int num_jobs, num_wide, taken;
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
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;

    long long rows_before = 0, need_before = 0;
    for (int base = 0; base < a.num_seqs; base += blockDim.x) {
        if (threadIdx.x == 0) num_jobs = num_wide = 0;
        const int b = base + threadIdx.x;
        const bool in = b < a.num_seqs;
        const int L = in ? a.lens[b] : 0, n = in ? a.new_tokens[b] : 0;
        const long long rows = n > 0 ? n : 0;
        long long total;
        const long long off = rows_before + block_scan(rows, sums, &total) - rows;
        rows_before += total;
        const bool len_ok = L >= 0 && L <= room;
        const bool rows_ok = n >= 0 && (n == 0 || off + n <= a.max_tokens);
        // Requests past max_tokens still count in the sum of needs: all
        // later ones with new tokens are past it too, so it changes nothing.
        const bool fits = in && len_ok && n >= 0 && static_cast<long long>(L) + n <= room;
        const long long need =
            fits ? blocks_of(static_cast<long long>(L) + n, a.block_shift) - blocks_of(L, a.block_shift) : 0;
        const long long incl = need_before + block_scan(need, sums, &total);
        need_before += total;
        if (in && a.err && (!len_ok || !rows_ok)) atomicOr(a.err, (len_ok ? 0 : PKV_ERRBIT_SEQ_LEN) | (rows_ok ? 0 : PKV_ERRBIT_STEP));
        const bool served = fits && rows_ok && (need == 0 || incl <= count);
        if (in) {
            a.token_offsets[b] = static_cast<int>(off < a.max_tokens ? off : a.max_tokens);
            a.granted[b] = served ? n : 0;
            a.lens_out[b] = served ? L + n : L;
            if (served && need > 0) atomicMax(&taken, static_cast<int>(incl));
            Job j{b, L, static_cast<int>(rows), static_cast<int>(off < a.max_tokens ? off : a.max_tokens),
                  served ? static_cast<int>(incl - need) : 0, served ? static_cast<int>(need) : 0, served ? 1 : 0};
            if (j.need <= kDirect && (!fill_rows || j.n <= kDirect)) {
                for (int i = 0; i < j.need; ++i) grow_entry(a, f, j, i);
                if (fill_rows)
                    for (int i = 0; i < j.n; ++i) grow_row(a, f, j, i);
            } else {
                // narrow ones from the front of the list, wide ones from its end
                const bool wide = j.need > kThreads || (fill_rows && j.n > kThreads);
                jobs[wide ? kThreads - 1 - atomicAdd(&num_wide, 1) : atomicAdd(&num_jobs, 1)] = j;
            }
        }
        __syncthreads();
        // one warp per remaining request; very long ones by the whole CTA
        auto serve = [&](const Job& j, int k0, int step) {
#pragma unroll 4
            for (int k = k0; k < j.need; k += step) grow_entry(a, f, j, k);
            if (fill_rows) {
                const int last = j.n < a.max_tokens - j.off ? j.n : a.max_tokens - j.off;
#pragma unroll 4
                for (int k = k0; k < last; k += step) grow_row(a, f, j, k);
            }
        };
        for (int i = warp; i < num_jobs; i += warps) serve(jobs[i], lane, 32);
        for (int i = 0; i < num_wide; ++i) serve(jobs[kThreads - 1 - i], threadIdx.x, blockDim.x);
        __syncthreads();
    }
    const int end = static_cast<int>(rows_before < a.max_tokens ? rows_before : a.max_tokens);
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
    if (row0 < end) {
        int lo = 0, hi = a.num_seqs;  // the last request whose first row is <= row0
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) >> 5, at = lo + lane * step;
            const unsigned below = __ballot_sync(0xFFFFFFFFu, at < hi && a.token_offsets[at] <= row0);
            lo += (31 - __clz(below)) * step;  // (lane 0 always is)
            hi = min(hi, lo + step);
        }
        if (row < end) {
            if (a.token_offsets[lo + 1] <= row)
                for (hi = a.num_seqs; hi - lo > 1;) {
                    const int mid = (lo + hi) >> 1;
                    if (a.token_offsets[mid] <= row) lo = mid;
                    else hi = mid;
                }
            seq = lo;
            const int n = a.granted[seq];
            const int L = a.lens_out[seq] - n;  // the length before the step
            const long long p = static_cast<long long>(L > 0 ? L : 0) + (row - a.token_offsets[seq]);
            pos = sat_pos(p);
            if (n > 0) {
                const int blk = checked_block(
                    a.tables[static_cast<size_t>(seq) * a.max_blocks + (p >> a.block_shift)], a.num_blocks, a.err);
                if (blk >= 0) slot = (static_cast<long long>(blk) << a.block_shift) + (p & ((1LL << a.block_shift) - 1));
            }
        }
    }
    if (row >= a.max_tokens) return;
    a.slots[row] = slot;
    a.positions[row] = pos;
    a.token_seqs[row] = seq;
}

// ---------------------------------------------------------------- release
constexpr int kReleasePerCta = kWarps;        // requests of one CTA of the large form: one per warp
constexpr long long kSmallEntries = 1 << 18;  // table entries up to which one CTA does it all

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
__device__ __forceinline__ void release_copy(const ReleaseArgs& a, int head, long long tail, int b, int first, int count,
                                             int k0, int step) {
    const int32_t* src = a.tables + static_cast<size_t>(b) * a.max_blocks + first;
#pragma unroll 4
    for (int k = k0; k < count; k += step) {
        long long at = head + tail + k;  // < 2 * ring_size
        if (at >= a.ring_size) at -= a.ring_size;
        a.ring[at] = checked_block(src[k], a.num_blocks, a.err);
    }
}

__device__ __forceinline__ bool ring_ok(const ReleaseArgs& a, int head, int count, long long total) {
    return head >= 0 && head < a.ring_size && count >= 0 && count + total <= a.ring_size;
}
__device__ __forceinline__ void put_state(const ReleaseArgs& a, int head, int count, long long total, bool ok) {
    a.free_out[0] = head;
    a.free_out[1] = ok ? static_cast<int>(count + total) : count;
    if (!ok && a.err) atomicOr(a.err, PKV_ERRBIT_STEP);
}

// Up to kThreads requests in one CTA: a thread each, then the blocks of those
// that have any by a warp each.  The outputs may be the inputs.
__global__ void __launch_bounds__(kThreads, 1) release_small_kernel(const ReleaseArgs a) {
    __shared__ long long sums[kWarps];
    struct Run {
        int b, first, count, tail;
    };
    __shared__ Run runs[kThreads];
    __shared__ int num_runs;
    const int head = a.free_state[0], count = a.free_state[1], b = threadIdx.x;
    Given g{0, 0, 0, false};
    if (b < a.num_seqs) g = given(a, b, true);
    if (b == 0) num_runs = 0;
    long long total;
    const long long incl = block_scan(g.count, sums, &total);
    const bool ok = ring_ok(a, head, count, total);
    if (ok && g.count > 0) runs[atomicAdd(&num_runs, 1)] = Run{b, g.first, g.count, static_cast<int>(count + incl - g.count)};
    if (b < a.num_seqs) a.lens_out[b] = ok && g.gone ? 0 : g.len;
    if (b == 0) put_state(a, head, count, total, ok);
    __syncthreads();
    for (int i = b >> 5; i < num_runs; i += static_cast<int>(blockDim.x >> 5))
        release_copy(a, head, runs[i].tail, runs[i].b, runs[i].first, runs[i].count, b & 31, 32);
}

// One pass over the batch: the blocks given back by requests before `upto`
// (*before) and by all of them (*total), for every thread of the CTA.
__device__ __forceinline__ void release_sums(const ReleaseArgs& a, int upto, long long* sums, long long* before,
                                             long long* total) {
    long long s0 = 0, s1 = 0;
#pragma unroll 4
    for (int b = threadIdx.x; b < a.num_seqs; b += blockDim.x) {
        const int n = given(a, b, false).count;
        s1 += n;
        if (b < upto) s0 += n;
    }
    block_scan(s0, sums, before);
    block_scan(s1, sums, total);
}

// Larger batches: every CTA sums the whole batch (some tens of KB from L2) and
// moves the blocks of its own 32 requests, a warp each.  Outputs apart from the
// inputs are written here (commit); others by a second kernel, once every CTA
// has read them.
__global__ void __launch_bounds__(kThreads, 1) release_copy_kernel(const ReleaseArgs a, const int commit) {
    __shared__ long long sums[kWarps];
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int head = a.free_state[0], count = a.free_state[1];
    const int b0 = blockIdx.x * kReleasePerCta, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Given g{0, 0, 0, false};
    if (b0 + lane < a.num_seqs) g = given(a, b0 + lane, warp == 0);
    long long before, total;
    release_sums(a, b0, sums, &before, &total);
    const bool ok = ring_ok(a, head, count, total);
    if (commit) {
        if (warp == 0 && b0 + lane < a.num_seqs) a.lens_out[b0 + lane] = ok && g.gone ? 0 : g.len;
        if (b0 == 0 && threadIdx.x == 0) put_state(a, head, count, total, ok);
    }
    if (!ok) return;
    long long incl = g.count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += x;
    }
    const long long tail = count + before + __shfl_sync(0xFFFFFFFFu, incl - g.count, warp);
    const int first = __shfl_sync(0xFFFFFFFFu, g.first, warp), n = __shfl_sync(0xFFFFFFFFu, g.count, warp);
    if (b0 + warp < a.num_seqs) release_copy(a, head, tail, b0 + warp, first, n, lane, 32);
}

__global__ void __launch_bounds__(kThreads, 1) release_commit_kernel(const ReleaseArgs a) {
    __shared__ long long sums[kWarps];
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int head = a.free_state[0], count = a.free_state[1];
    long long zero, total;
    release_sums(a, 0, sums, &zero, &total);
    const bool ok = ring_ok(a, head, count, total);
    for (int b = threadIdx.x; b < a.num_seqs; b += blockDim.x) {
        const Given g = given(a, b, false);
        a.lens_out[b] = ok && g.gone ? 0 : g.len;
    }
    if (threadIdx.x == 0) put_state(a, head, count, total, ok);
}

}  // namespace

cudaError_t launch_tables_grow(const GrowArgs& a, cudaStream_t stream) {
    const bool inline_rows = a.max_tokens <= kInlineTokens;
    const int threads = a.num_seqs <= 256 && a.max_tokens <= 1024 ? 256 : kThreads;
    grow_kernel<<<1, threads, 0, stream>>>(a, inline_rows ? 1 : 0);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || inline_rows) return e;
    return launch_dependent(fill_kernel, dim3((a.max_tokens + kFillThreads - 1) / kFillThreads), dim3(kFillThreads), 0,
                            stream, a);
}

cudaError_t launch_tables_release(const ReleaseArgs& a, cudaStream_t stream) {
    if (a.num_seqs <= kThreads && static_cast<long long>(a.num_seqs) * a.max_blocks <= kSmallEntries) {
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
