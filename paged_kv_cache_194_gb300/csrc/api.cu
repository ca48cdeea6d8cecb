// C ABI of libpkv.so: argument validation, split planning and launches.
// Everything here runs on the host; it allocates no device memory and never
// synchronises a stream.
#include <atomic>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "pkv_internal.h"
#include "step_internal.h"

namespace pkv {

namespace {
thread_local char g_last_cuda_error[256] = "";
// pkv_set_first_wait_limit_for_testing: polls (< 0: off) and the CTA it targets
thread_local int32_t g_test_wait_polls = -1;
thread_local int32_t g_test_wait_cta = -1;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
bool valid_dtype(pkv_dtype t) { return t == PKV_F32 || t == PKV_BF16 || t == PKV_FP8_E4M3; }

pkv_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return PKV_OK;
    if (e == cudaErrorNotSupported) return PKV_ERR_UNSUPPORTED;
    set_last_error(e);
    return PKV_ERR_CUDA;
}

std::atomic<int> g_sms[64];

// Balanced persistent schedule: at most this many sequences (each CTA scans
// the lengths once), at most kBalCtasPerSm CTAs per SM.
constexpr int kMaxBalancedSeqs = 4096;
constexpr int kBalCtasPerSm = 2;

size_t counters_bytes(int B, int Hkv) { return round_up(static_cast<size_t>(B) * Hkv * sizeof(int32_t), 256); }
size_t fixed_bytes(int B, int Hq, int D, int64_t ns) {
    if (ns <= 1) return 0;
    const size_t rows = static_cast<size_t>(B) * Hq * ns;
    return round_up(rows * D * sizeof(float), 256) + round_up(rows * sizeof(float), 256);
}
int bal_ctas() { return (num_sms() > 0 ? num_sms() : 148) * kBalCtasPerSm; }
size_t bal_o_bytes(int ctas, int G, int D) { return round_up(static_cast<size_t>(ctas) * 2 * G * D * sizeof(float), 256); }
size_t bal_bytes(int ctas, int G, int D) {
    return bal_o_bytes(ctas, G, D) + round_up(static_cast<size_t>(ctas) * 2 * G * sizeof(float), 256);
}

// Queries per launch.  A launch serves rows = queries x gh query rows per KV
// head: at most kMmaMaxRows for the tensor-core design; for the SIMT design
// a power of two up to kSimtMaxRows.  Longer query lists run as several
// launches over consecutive query chunks.
int mma_chunk(int gh, int C) {
    const int cap = gh <= kMmaMaxRows ? kMmaMaxRows / gh : 1;
    return C < cap ? C : cap;
}
int simt_chunk(const pkv_pool* p, int gh, int C) {
    int cap = gh <= kSimtMaxRows ? kSimtMaxRows / gh : 1;
    if (C < cap) cap = C;
    int c = 1;
    while (c * 2 <= cap) c *= 2;
    while (c > 1 && !decode_simt_supported(p->d.kv_dtype, p->d.head_dim, c * gh)) c /= 2;
    return c;
}
// Template row bound of the tensor-core kernel for `rows` rows.
int row_bound(int rows) {
    int p = 1;
    while (p < rows) p *= 2;
    return p;
}
constexpr int kMaxQueries = 1 << 20;
constexpr int kTcMinRows = 8;  // query rows per KV head from which AUTO takes the tcgen05 design
// Up to this many query rows per KV head (one 128-row tile) the tcgen05
// design can run the balanced persistent schedule.
constexpr int kTcBalMaxRows = 128;
// The tcgen05 design takes the balanced schedule when one CTA per (sequence,
// KV head) would leave CTA slots idle (a few long sequences).  With enough
// units the grid keeps every SM busy, and whole units need no Q reload or
// merge at segment ends, so the grid is as fast or faster.
bool tc_balanced(int num_seqs, int num_kv_heads, int64_t rows) {
    return rows <= kTcBalMaxRows && num_seqs <= kMaxBalancedSeqs &&
           static_cast<int64_t>(num_seqs) * num_kv_heads < bal_ctas();
}
// Rows of one balanced-schedule partial slot: the template row bound of the
// largest launch (a KV-head pair's 2 * gh rows for decode).
int bal_rows(int gh, int C) {
    const int r = row_bound(mma_chunk(gh, C) * gh);
    const int pair = (C == 1 && 2 * gh <= 8) ? row_bound(2 * gh) : 0;
    return r > pair ? r : pair;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = []() -> EncodeTiledFn {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        const bool found =
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess;
        return found ? reinterpret_cast<EncodeTiledFn>(p) : nullptr;
    }();
    return fn;
}

// cuTensorMapEncodeTiled, which wants a current context: a host thread has none
// before its first call that binds its device's (a launch or a copy would).
template <typename... Args>
bool encode_tiled(EncodeTiledFn fn, Args... args) {
    if (fn(args...) == CUDA_SUCCESS) return true;
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && fn(args...) == CUDA_SUCCESS;
}

// TMA descriptors over the whole K and V pools, viewed as 2D tensors
// [rows = layers*blocks*kv_heads*block_size][head_dim]; one box is one
// (block, kv head) chunk of 64 BF16 or 128 E4M3 columns, 128-byte swizzled.
bool encode_tmaps(pkv_pool* p) {
    const pkv_pool_desc& d = p->d;
    if (d.kv_dtype != PKV_BF16 && d.kv_dtype != PKV_FP8_E4M3) return false;
    const uint64_t rows = static_cast<uint64_t>(d.num_layers) * d.num_blocks * d.num_kv_heads * d.block_size;
    if (rows > static_cast<uint64_t>(INT32_MAX)) return false;
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const bool bf16 = d.kv_dtype == PKV_BF16;
    if (bf16 && d.head_dim == 128) {
        // One box per (block, kv head): dims {64 columns, rows, 2 halves} with
        // the half stride (128 B) inside the row stride (256 B), so the box
        // lands as [half][bs rows][128 B].
        const cuuint64_t dims3[3] = {64, rows, 2};
        const cuuint64_t strides3[2] = {256, 128};
        const cuuint32_t box3[3] = {64, static_cast<cuuint32_t>(d.block_size), 2};
        const cuuint32_t estr3[3] = {1, 1, 1};
        bool ok3 = true;
        for (int i = 0; i < 2 && ok3; ++i) {
            const bool r = encode_tiled(enc, i == 0 ? &p->tmap_k : &p->tmap_v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                                        i == 0 ? d.k_base : d.v_base, dims3, strides3, box3, estr3,
                                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
            ok3 = r;
        }
        if (ok3) {
            p->tmap_3d = 1;
            // Boxes of one 64-column half of a block (the tcgen05 kernel keeps
            // the two halves of a tile apart).
            const cuuint32_t boxh[3] = {64, static_cast<cuuint32_t>(d.block_size), 1};
            bool okh = true;
            for (int i = 0; i < 2 && okh; ++i) {
                const bool r = encode_tiled(enc, i == 0 ? &p->tmap_kh : &p->tmap_vh,
                                            CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, i == 0 ? d.k_base : d.v_base, dims3,
                                            strides3, boxh, estr3, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
                okh = r;
            }
            p->tmap_half = okh ? 1 : 0;
            // Boxes of two adjacent KV heads of a block (the rows of head h+1
            // follow those of head h): 8 KB per box at 16-token blocks.
            p->tmap_pair = 0;
            if (d.block_size == 16 && d.num_kv_heads % 2 == 0) {
                const cuuint32_t box2[3] = {64, static_cast<cuuint32_t>(2 * d.block_size), 2};
                bool ok2 = true;
                for (int i = 0; i < 2 && ok2; ++i) {
                    const bool r = encode_tiled(enc, i == 0 ? &p->tmap_k2 : &p->tmap_v2,
                                                CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, i == 0 ? d.k_base : d.v_base,
                                                dims3, strides3, box2, estr3, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
                    ok2 = r;
                }
                p->tmap_pair = ok2 ? 1 : 0;
            }
            return true;
        }
    }
    p->tmap_3d = 0;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d.head_dim), rows};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(d.head_dim) * p->elem_bytes};
    const cuuint32_t box[2] = {bf16 ? 64u : 128u, static_cast<cuuint32_t>(d.block_size)};
    const cuuint32_t estr[2] = {1, 1};
    const CUtensorMapDataType dt = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    for (int i = 0; i < 2; ++i) {
        const bool r = encode_tiled(enc, i == 0 ? &p->tmap_k : &p->tmap_v, dt, 2, i == 0 ? d.k_base : d.v_base, dims,
                                    strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (!r) return false;
    }
    return true;
}

// Encodes them with the pool's first call that wants them.  First calls may come
// from several threads at once: none looks at a pool that another is encoding.
bool ensure_tmaps(pkv_pool* p) {
    int state = __atomic_load_n(&p->tmap_state, __ATOMIC_ACQUIRE);
    if (state == 0) {
        static std::mutex encoding;
        const std::lock_guard<std::mutex> lock(encoding);
        state = p->tmap_state;
        if (state == 0) {
            state = encode_tmaps(p) ? 1 : -1;
            __atomic_store_n(&p->tmap_state, state, __ATOMIC_RELEASE);
        }
    }
    return state == 1;
}
}  // namespace

void set_last_error(cudaError_t e) {
    std::snprintf(g_last_cuda_error, sizeof(g_last_cuda_error), "%s: %s", cudaGetErrorName(e),
                  cudaGetErrorString(e));
}

int dtype_bytes(pkv_dtype t) {
    switch (t) {
        case PKV_F32: return 4;
        case PKV_BF16: return 2;
        case PKV_FP8_E4M3: return 1;
    }
    return 0;
}

size_t workspace_counter_bytes(int num_seqs, int num_kv_heads) { return counters_bytes(num_seqs, num_kv_heads); }

int num_sms() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
    if (dev < 64 && g_sms[dev] > 0) return g_sms[dev];
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 64) g_sms[dev] = n;
    return n;
}

}  // namespace pkv

using namespace pkv;

extern "C" {

const char* pkv_status_string(pkv_status s) {
    switch (s) {
        case PKV_OK: return "ok";
        case PKV_ERR_INVALID_ARG: return "invalid argument";
        case PKV_ERR_UNSUPPORTED: return "unsupported geometry or dtype";
        case PKV_ERR_WORKSPACE: return "workspace missing or too small";
        case PKV_ERR_CUDA: return "CUDA error";
        case PKV_ERR_DEVICE_BOUNDS: return "device-side index out of bounds";
        case PKV_ERR_OUT_OF_BLOCKS: return "out of KV blocks";
        case PKV_ERR_INCONSISTENT: return "block manager invariant violated";
    }
    return "unknown status";
}

const char* pkv_last_cuda_error(void) { return g_last_cuda_error; }

void pkv_set_first_wait_limit_for_testing(int32_t polls, int32_t cta) {
    g_test_wait_polls = polls < 0 ? -1 : polls;
    g_test_wait_cta = cta < 0 ? -1 : cta;
}

int64_t kv_bytes_per_token(int32_t num_layers, int32_t num_kv_heads, int32_t head_dim, pkv_dtype dtype) {
    return 2LL * num_layers * num_kv_heads * head_dim * dtype_bytes(dtype);
}

size_t kv_pool_tensor_bytes(const pkv_pool_desc* d) {
    if (!d || !valid_dtype(d->kv_dtype)) return 0;
    return static_cast<size_t>(d->num_layers) * d->num_blocks * d->num_kv_heads * d->block_size *
           d->head_dim * dtype_bytes(d->kv_dtype);
}

pkv_status kv_pool_create(const pkv_pool_desc* d, pkv_pool** out) {
    if (!d || !out) return PKV_ERR_INVALID_ARG;
    *out = nullptr;
    if (!valid_dtype(d->kv_dtype)) return PKV_ERR_INVALID_ARG;
    if (d->num_layers < 1 || d->num_blocks < 1 || d->num_kv_heads < 1) return PKV_ERR_INVALID_ARG;
    if (d->block_size != 16 && d->block_size != 32 && d->block_size != 64) return PKV_ERR_UNSUPPORTED;
    if (d->head_dim != 64 && d->head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (!d->k_base || !d->v_base || !aligned(d->k_base, 16) || !aligned(d->v_base, 16))
        return PKV_ERR_INVALID_ARG;
    if (d->error_word && !aligned(d->error_word, 4)) return PKV_ERR_INVALID_ARG;
    // slots and element offsets are int64; keep one layer's slot count in int32
    if (static_cast<int64_t>(d->num_blocks) * d->block_size > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    float ks = 1.f, vs = 1.f;
    if (d->kv_dtype == PKV_FP8_E4M3) {
        if (!(std::isfinite(d->k_scale) && d->k_scale > 0.f && std::isfinite(d->v_scale) && d->v_scale > 0.f))
            return PKV_ERR_INVALID_ARG;
        ks = d->k_scale;
        vs = d->v_scale;
    }
    // CUtensorMap needs 64-byte alignment
    pkv_pool* p = static_cast<pkv_pool*>(std::aligned_alloc(64, round_up(sizeof(pkv_pool), 64)));
    if (!p) return PKV_ERR_INVALID_ARG;
    std::memset(p, 0, sizeof(pkv_pool));
    p->d = *d;
    p->d.k_scale = ks;
    p->d.v_scale = vs;
    p->elem_bytes = dtype_bytes(d->kv_dtype);
    p->layer_bytes = static_cast<size_t>(d->num_blocks) * d->num_kv_heads * d->block_size * d->head_dim *
                     p->elem_bytes;
    volatile float one = 1.f;  // one binary32 division each, on the host
    p->k_inv_scale = one / ks;
    p->v_inv_scale = one / vs;
    *out = p;
    return PKV_OK;
}

void kv_pool_destroy(pkv_pool* p) { std::free(p); }

pkv_status kv_append(const pkv_pool* p, int32_t layer, const void* k, const void* v, pkv_dtype in_dtype,
                     const int64_t* slot_mapping, int32_t num_tokens, void* stream) {
    if (!p || layer < 0 || layer >= p->d.num_layers || num_tokens < 0) return PKV_ERR_INVALID_ARG;
    if (in_dtype != PKV_F32 && in_dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
    if (p->d.kv_dtype == PKV_F32 && in_dtype != PKV_F32) return PKV_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PKV_OK;
    if (!k || !v || !slot_mapping || !aligned(k, 16) || !aligned(v, 16) || !aligned(slot_mapping, 8))
        return PKV_ERR_INVALID_ARG;
    return cuda_status(launch_kv_append(p, layer, k, v, in_dtype, slot_mapping, num_tokens,
                                        static_cast<cudaStream_t>(stream)));
}

pkv_status paged_multi_query_plan(const pkv_pool* p, int32_t num_seqs, int32_t num_queries, int32_t num_q_heads,
                                  int32_t max_seq_len, int32_t split_tokens, int32_t* split_out,
                                  int32_t* nsplit_out, size_t* ws_out) {
    if (!p || num_seqs < 0 || num_q_heads < 1 || max_seq_len < 0 || split_tokens < 0) return PKV_ERR_INVALID_ARG;
    if (num_queries < 1 || num_queries > kMaxQueries) return PKV_ERR_INVALID_ARG;
    if (num_q_heads % p->d.num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
    int S = split_tokens;
    if (S > 0) {
        if (S % kTileTokens != 0 || S % p->d.block_size != 0) return PKV_ERR_INVALID_ARG;
    } else {
        // Auto: 1024-token splits, halved (down to one tile) while the batch
        // would give fewer than two CTAs per SM.
        const int sms = num_sms() > 0 ? num_sms() : 148;
        const int64_t pairs = static_cast<int64_t>(num_seqs) * p->d.num_kv_heads;
        S = 1024;
        while (S > kTileTokens && pairs * ((max_seq_len + S - 1) / S) < 2LL * sms) S /= 2;
        if (S % p->d.block_size != 0) S = p->d.block_size > kTileTokens ? p->d.block_size : kTileTokens;
    }
    int64_t ns = max_seq_len > 0 ? (static_cast<int64_t>(max_seq_len) + S - 1) / S : 1;
    if (ns < 1) ns = 1;
    if (ns > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    // layout: [counters][partials of whichever schedule the call runs], sized
    // for the largest query chunk of either design (the tensor-core one's)
    const int gh = num_q_heads / p->d.num_kv_heads;
    const int cq = mma_chunk(gh, num_queries);
    size_t body = fixed_bytes(num_seqs, cq * num_q_heads, p->d.head_dim, ns);
    if (split_tokens == 0 && num_seqs <= kMaxBalancedSeqs) {
        size_t bb = bal_bytes(bal_ctas(), bal_rows(gh, num_queries), p->d.head_dim);
        // the tcgen05 design's balanced schedule: one slot row per query row
        if (static_cast<int64_t>(num_queries) * gh <= kTcBalMaxRows) {
            const size_t bt = bal_bytes(bal_ctas(), num_queries * gh, p->d.head_dim);
            if (bt > bb) bb = bt;
        }
        if (bb > body) body = bb;
    }
    size_t ws = body > 0 ? counters_bytes(num_seqs, p->d.num_kv_heads) + body : 0;
    if (split_out) *split_out = S;
    if (nsplit_out) *nsplit_out = static_cast<int32_t>(ns);
    if (ws_out) *ws_out = ws;
    return PKV_OK;
}

pkv_status paged_decode_plan(const pkv_pool* p, int32_t num_seqs, int32_t num_q_heads, int32_t max_seq_len,
                             int32_t split_tokens, int32_t* split_out, int32_t* nsplit_out, size_t* ws_out) {
    return paged_multi_query_plan(p, num_seqs, 1, num_q_heads, max_seq_len, split_tokens, split_out, nsplit_out,
                                  ws_out);
}

int32_t paged_decode_algo(const pkv_pool* p, int32_t G, pkv_algo algo) {
    if (!p || G < 1) return -1;
    pkv_pool* mp = const_cast<pkv_pool*>(p);
    const bool mma_ok = decode_mma_supported(p->d.kv_dtype, p->d.head_dim, G, p->d.block_size);
    if (algo == PKV_ALGO_MMA) return (mma_ok && ensure_tmaps(mp)) ? PKV_ALGO_MMA : -1;
    if (algo == PKV_ALGO_SIMT) return PKV_ALGO_SIMT;  // (any number of heads, in parts if need be)
    if (algo != PKV_ALGO_AUTO) return -1;
    return mma_ok && ensure_tmaps(mp) ? PKV_ALGO_MMA : PKV_ALGO_SIMT;
}

}  // extern "C"

namespace pkv {
namespace {
// The kernel design a call runs: PKV_ALGO_TC (tcgen05, whole query list in
// one launch; the default from kTcMinRows query rows per KV head), MMA or
// SIMT, or -1 when the request cannot be served.  fused: the decode step's
// append runs inside the launch (tensor-core design only).
int design_for(const pkv_pool* p, int C, int gh, int split_tokens, pkv_algo algo, bool fused) {
    pkv_pool* mp = const_cast<pkv_pool*>(p);  // the handle caches its TMA descriptors
    const bool tc_fits = attention_tc_supported(p->d.kv_dtype, p->d.head_dim, p->d.block_size) && !fused &&
                         split_tokens == 0 && static_cast<int64_t>(C) * gh <= (1 << 24);
    const bool mma_fits = decode_mma_supported(p->d.kv_dtype, p->d.head_dim, mma_chunk(gh, C) * gh, p->d.block_size);
    const int cs = simt_chunk(p, gh, C);
    // (a single query's heads may run in parts, so that any number of them fits)
    const bool simt_fits = cs == 1 || decode_simt_supported(p->d.kv_dtype, p->d.head_dim, cs * gh);
    int d = -1;
    if (algo == PKV_ALGO_TC) {
        d = tc_fits && ensure_tmaps(mp) && p->tmap_half == 1 ? PKV_ALGO_TC : -1;
    } else if (algo == PKV_ALGO_MMA) {
        d = mma_fits && ensure_tmaps(mp) ? PKV_ALGO_MMA : -1;
    } else if (algo == PKV_ALGO_SIMT) {
        d = simt_fits ? PKV_ALGO_SIMT : -1;
    } else if (algo == PKV_ALGO_AUTO) {
        if (tc_fits && C > 1 && C * gh >= kTcMinRows && ensure_tmaps(mp) && p->tmap_half == 1)
            d = PKV_ALGO_TC;
        else if (mma_fits && ensure_tmaps(mp))
            d = PKV_ALGO_MMA;
        else if (simt_fits)
            d = PKV_ALGO_SIMT;
    }
    if (fused && (d != PKV_ALGO_MMA || C != 1 || gh > 8)) return -1;
    return d;
}

// Attention for C queries per sequence; with new_k != nullptr (decode only)
// the kernel also appends each sequence's newest token.
pkv_status attention_call(const void* q, pkv_dtype q_dtype, const pkv_pool* p, int32_t layer,
                          const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                          int32_t num_seqs, int32_t num_queries, int32_t num_q_heads, int32_t max_seq_len,
                          float scale, int32_t split_tokens, pkv_algo algo, void* workspace, size_t workspace_bytes,
                          void* out, void* stream, const void* new_k, const void* new_v, pkv_dtype new_dtype,
                          bool dry_run = false) {
    if (!p || layer < 0 || layer >= p->d.num_layers) return PKV_ERR_INVALID_ARG;
    if (num_queries < 1 || num_queries > kMaxQueries) return PKV_ERR_INVALID_ARG;
    if (num_seqs < 0 || num_q_heads < 1 || max_blocks_per_seq < 1 || max_seq_len < 0) return PKV_ERR_INVALID_ARG;
    if (num_q_heads % p->d.num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
    if (static_cast<int64_t>(max_seq_len) > static_cast<int64_t>(max_blocks_per_seq) * p->d.block_size)
        return PKV_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return PKV_ERR_INVALID_ARG;
    const pkv_dtype want_q = p->d.kv_dtype == PKV_F32 ? PKV_F32 : PKV_BF16;
    if (q_dtype != want_q) return PKV_ERR_UNSUPPORTED;
    if (algo != PKV_ALGO_AUTO && algo != PKV_ALGO_SIMT && algo != PKV_ALGO_MMA && algo != PKV_ALGO_TC)
        return PKV_ERR_INVALID_ARG;
    if (num_seqs == 0) return PKV_OK;
    if (num_seqs > 65535) return PKV_ERR_UNSUPPORTED;
    if (!q || !out || !block_tables || !seq_lens) return PKV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(block_tables, 4) || !aligned(seq_lens, 4))
        return PKV_ERR_INVALID_ARG;
    const int gh = num_q_heads / p->d.num_kv_heads;  // query heads per KV head
    const int cq_mma = mma_chunk(gh, num_queries);  // the largest chunk: sizes the fixed-split partials
    const int design = design_for(p, num_queries, gh, split_tokens, algo, new_k != nullptr);
    if (design < 0) return PKV_ERR_UNSUPPORTED;
    const bool use_tc = design == PKV_ALGO_TC, use_mma = design == PKV_ALGO_MMA;

    int32_t S = 0, NS = 0;
    size_t need = 0;
    pkv_status st =
        paged_multi_query_plan(p, num_seqs, num_queries, num_q_heads, max_seq_len, split_tokens, &S, &NS, &need);
    if (st != PKV_OK) return st;
    const bool tc_bal = use_tc && split_tokens == 0 && tc_balanced(num_seqs, p->d.num_kv_heads, static_cast<int64_t>(num_queries) * gh);
    if ((!use_tc || tc_bal) && need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return PKV_ERR_WORKSPACE;
    if (dry_run) return PKV_OK;  // every host-side check passed; nothing enqueued

    DecodeArgs a{};
    a.q = q;
    a.out = out;
    a.k_layer = static_cast<const uint8_t*>(p->d.k_base) + static_cast<size_t>(layer) * p->layer_bytes;
    a.v_layer = static_cast<const uint8_t*>(p->d.v_base) + static_cast<size_t>(layer) * p->layer_bytes;
    a.tables = block_tables;
    a.lens = seq_lens;
    a.err = p->d.error_word;
    a.layer = layer;
    a.tma_3d = p->tmap_3d;
    a.max_blocks = max_blocks_per_seq;
    a.max_len = max_seq_len;
    a.num_seqs = num_seqs;
    a.q_total = num_queries;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = p->d.num_kv_heads;
    a.head_dim = p->d.head_dim;
    a.block_size = p->d.block_size;
    a.num_blocks = p->d.num_blocks;
    a.split_tokens = S;
    a.num_splits = NS;
    const bool balanced = use_mma && split_tokens == 0 && num_seqs <= kMaxBalancedSeqs;
    const float log2e = 1.4426950408889634f;
    a.qk_scale_log2 = scale * p->d.k_scale * log2e;
    a.v_scale = p->d.v_scale;
    if (g_test_wait_polls >= 0) {
        a.test_wait_on = 1;
        a.test_wait_polls = static_cast<uint32_t>(g_test_wait_polls);
        a.test_wait_cta = g_test_wait_cta;
    }
    if (new_k) {
        a.new_k = static_cast<const uint8_t*>(new_k);
        a.new_v = static_cast<const uint8_t*>(new_v);
        a.new_dtype = new_dtype;
        a.k_inv_scale = p->k_inv_scale;
        a.v_inv_scale = p->v_inv_scale;
        a.k_layer_w = static_cast<uint8_t*>(p->d.k_base) + static_cast<size_t>(layer) * p->layer_bytes;
        a.v_layer_w = static_cast<uint8_t*>(p->d.v_base) + static_cast<size_t>(layer) * p->layer_bytes;
    }
    if (need > 0) {
        uint8_t* w = static_cast<uint8_t*>(workspace);
        a.counters = reinterpret_cast<int32_t*>(w);
        uint8_t* body = w + counters_bytes(num_seqs, p->d.num_kv_heads);
        if (balanced || tc_bal) {
            a.bal_max_ctas = bal_ctas();
            a.bal_o = reinterpret_cast<float*>(body);
            const int rows = tc_bal ? num_queries * gh : bal_rows(gh, num_queries);
            a.bal_lse = reinterpret_cast<float*>(body + bal_o_bytes(a.bal_max_ctas, rows, p->d.head_dim));
        } else if (NS > 1) {
            const size_t rows = static_cast<size_t>(num_seqs) * cq_mma * num_q_heads * NS;
            a.o_part = reinterpret_cast<float*>(body);
            a.lse_part = reinterpret_cast<float*>(body + round_up(rows * p->d.head_dim * sizeof(float), 256));
        }
    }
    // Decode on BF16 pools of 16-token blocks: one CTA serves two adjacent KV
    // heads, so each block arrives as one 8 KB box instead of two 4 KB ones
    // (per-box cost dominates at 4 KB).
    const bool pair = use_mma && num_queries == 1 && p->tmap_pair == 1 && p->tmap_3d == 1 && 2 * gh <= 8;
    a.heads_per_cta = pair ? 2 : 1;
    const void* tk = pair ? &p->tmap_k2 : &p->tmap_k;
    const void* tv = pair ? &p->tmap_v2 : &p->tmap_v;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (use_tc) {  // the balanced schedule (bal_max_ctas > 0) or one CTA per row tile
        a.heads_per_cta = 1;
        a.q_first = 0;
        a.num_queries = num_queries;
        a.len_trim = 0;
        if (!tc_bal) a.bal_max_ctas = 0;
        return cuda_status(launch_attention_tc(a, &p->tmap_kh, &p->tmap_vh, s));
    }
    // one launch (plus combine) per query chunk; a chunk reads only the tokens
    // its last query can see
    for (int c0 = 0; c0 < num_queries;) {
        int cq = use_mma ? mma_chunk(gh, num_queries - c0) : simt_chunk(p, gh, num_queries - c0);
        a.q_first = c0;
        a.num_queries = cq;
        a.len_trim = num_queries - c0 - cq;
        cudaError_t e = use_mma ? launch_decode_mma(p->d.kv_dtype, a, tk, tv, s) : launch_decode_simt(p->d.kv_dtype, a, s);
        if (e != cudaSuccess) return cuda_status(e);
        if (!balanced && NS > 1) {
            e = launch_combine(q_dtype, a, s);
            if (e != cudaSuccess) return cuda_status(e);
        }
        c0 += cq;
    }
    return PKV_OK;
}
}  // namespace

pkv_status decode_attention_check(const void* q, pkv_dtype q_dtype, const pkv_pool* p, int32_t layer,
                                  const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                  int32_t num_seqs, int32_t num_q_heads, int32_t max_seq_len, float scale,
                                  int32_t split_tokens, pkv_algo algo, void* workspace, size_t workspace_bytes,
                                  void* out) {
    return attention_call(q, q_dtype, p, layer, block_tables, max_blocks_per_seq, seq_lens, num_seqs, 1, num_q_heads,
                          max_seq_len, scale, split_tokens, algo, workspace, workspace_bytes, out, nullptr, nullptr,
                          nullptr, PKV_BF16, true);
}
}  // namespace pkv

extern "C" {

pkv_status paged_multi_query_attention(const void* q, pkv_dtype q_dtype, const pkv_pool* p, int32_t layer,
                                       const int32_t* block_tables, int32_t max_blocks_per_seq,
                                       const int32_t* seq_lens, int32_t num_seqs, int32_t num_queries,
                                       int32_t num_q_heads, int32_t max_seq_len, float scale, int32_t split_tokens,
                                       pkv_algo algo, void* workspace, size_t workspace_bytes, void* out,
                                       void* stream) {
    return pkv::attention_call(q, q_dtype, p, layer, block_tables, max_blocks_per_seq, seq_lens, num_seqs,
                               num_queries, num_q_heads, max_seq_len, scale, split_tokens, algo, workspace,
                               workspace_bytes, out, stream, nullptr, nullptr, PKV_BF16);
}

int32_t paged_multi_query_algo(const pkv_pool* p, int32_t num_queries, int32_t num_q_heads, int32_t split_tokens,
                               pkv_algo algo) {
    if (!p || num_queries < 1 || num_queries > pkv::kMaxQueries || num_q_heads < 1 ||
        num_q_heads % p->d.num_kv_heads != 0 || split_tokens < 0)
        return -1;
    return pkv::design_for(p, num_queries, num_q_heads / p->d.num_kv_heads, split_tokens, algo, false);
}

pkv_status paged_decode_append_attention(const void* q, pkv_dtype q_dtype, const void* k_new, const void* v_new,
                                         pkv_dtype in_dtype, const pkv_pool* p, int32_t layer,
                                         const int32_t* block_tables, int32_t max_blocks_per_seq,
                                         const int32_t* seq_lens, int32_t num_seqs, int32_t num_q_heads,
                                         int32_t max_seq_len, float scale, int32_t split_tokens, pkv_algo algo,
                                         void* workspace, size_t workspace_bytes, void* out, void* stream) {
    if (!p) return PKV_ERR_INVALID_ARG;
    if (in_dtype != PKV_BF16 && in_dtype != PKV_F32) return PKV_ERR_UNSUPPORTED;
    if (num_seqs > 0 && (!k_new || !v_new || !aligned(k_new, 16) || !aligned(v_new, 16))) return PKV_ERR_INVALID_ARG;
    return pkv::attention_call(q, q_dtype, p, layer, block_tables, max_blocks_per_seq, seq_lens, num_seqs, 1,
                               num_q_heads, max_seq_len, scale, split_tokens, algo, workspace, workspace_bytes, out,
                               stream, num_seqs > 0 ? k_new : nullptr, v_new, in_dtype);
}

pkv_status paged_decode_attention(const void* q, pkv_dtype q_dtype, const pkv_pool* p, int32_t layer,
                                  const int32_t* block_tables, int32_t max_blocks_per_seq,
                                  const int32_t* seq_lens, int32_t num_seqs, int32_t num_q_heads,
                                  int32_t max_seq_len, float scale, int32_t split_tokens, pkv_algo algo,
                                  void* workspace, size_t workspace_bytes, void* out, void* stream) {
    return paged_multi_query_attention(q, q_dtype, p, layer, block_tables, max_blocks_per_seq, seq_lens, num_seqs, 1,
                                       num_q_heads, max_seq_len, scale, split_tokens, algo, workspace,
                                       workspace_bytes, out, stream);
}

}  // extern "C"

// ------------------------------------------- shared prefixes, norm + rotation, tables
namespace pkv {
namespace {

bool prefix_tc_fits(const pkv_pool* p, int num_seqs, int num_groups, int gh, int max_seq_len) {
    if ((p->d.kv_dtype != PKV_BF16 && p->d.kv_dtype != PKV_FP8_E4M3) || p->d.head_dim != 128) return false;
    if (num_seqs > kPrefixMaxSeqs || num_groups > kPrefixMaxGroups || gh > kPrefixRows) return false;
    if (static_cast<int64_t>(num_seqs) * p->d.num_kv_heads * gh > INT32_MAX / 2) return false;  // rows are int32
    // tile counts are int32
    const int64_t tiles = (static_cast<int64_t>(max_seq_len) + kTileTokens - 1) / kTileTokens;
    return (tiles + 8) * num_seqs * p->d.num_kv_heads <= INT32_MAX / 4;
}

// Workspace of the sharing design behind the decode counters (which it leaves
// alone, so that both kinds of calls may use one workspace).
size_t prefix_layout(const pkv_pool* p, int num_seqs, int num_groups, int num_q_heads, uint8_t* base, PrefixArgs* a) {
    size_t at = counters_bytes(num_seqs, p->d.num_kv_heads);
    auto take = [&](size_t bytes) {
        uint8_t* r = base + at;
        at += round_up(bytes, 256);
        return r;
    };
    const int ctas = bal_ctas();
    const size_t B = num_seqs, G = num_groups, gh = num_q_heads / p->d.num_kv_heads;
    const size_t pre = B * num_q_heads + static_cast<size_t>(ctas) * kPrefixRows, own = B * num_q_heads + ctas * gh;
    const size_t row = static_cast<size_t>(p->d.head_dim) * sizeof(float);
    PrefixArgs x{};
    x.ctas = ctas;
    x.totals = reinterpret_cast<int32_t*>(take(sizeof(int32_t)));
    x.seqs = reinterpret_cast<int2*>(take(B * sizeof(int2)));
    x.pieces = reinterpret_cast<int4*>(take(2 * B * sizeof(int4)));
    x.groups = reinterpret_cast<int4*>(take(G * sizeof(int4)));
    x.pre_o = reinterpret_cast<float*>(take(pre * row));
    x.pre_lse = reinterpret_cast<float*>(take(pre * sizeof(float)));
    x.own_o = reinterpret_cast<float*>(take(own * row));
    x.own_lse = reinterpret_cast<float*>(take(own * sizeof(float)));
    if (a) *a = x;
    return at;
}

// Descriptor of the queries [B][Hq][128] BF16 as {64 columns, Hq, B, 2 column
// halves}; one box is the heads of one KV head of `seqs` sequences, so it lands
// as rows (sequence, head) of 128 bytes.
bool encode_q_map(CUtensorMap* map, const void* q, int num_seqs, int num_q_heads, int gh, int seqs) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(num_q_heads), static_cast<cuuint64_t>(num_seqs), 2};
    const cuuint64_t strides[3] = {256, 256ull * num_q_heads, 128};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(gh), static_cast<cuuint32_t>(seqs), 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return encode_tiled(enc, map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// PKV_ALGO_TC when the sharing design runs, else what decode attention runs.
// Without groups there is nothing to share, and over FP8 pools AUTO leaves calls
// of less than 8 query heads per KV head to decode attention (us here / there, 32
// query over 8 KV heads: 72 / 59 for 64 x 2048 tokens, 70 / 59 for 8 x 16384, 40 /
// 28 for 256 x 64, 36 / 31 for 64 of up to 1024; only few long sequences lose, 23
// / 34 for 1 x 16384).  From 8 heads on the sharing design, whose time hardly
// depends on them, is as fast or faster (8: 74 / 64, 68 / 65 and 20 / 23 for 8 x
// 2048; 16: 28 / 44, 28 / 70, 15 / 47), and over BF16 pools for any number (89 /
// 88, 87 / 92, 27 / 23, 33 / 36, 20 / 67).
int prefix_design(const pkv_pool* p, int num_seqs, int num_groups, int num_q_heads, int max_seq_len, pkv_algo algo) {
    const int gh = num_q_heads / p->d.num_kv_heads;
    const bool left = num_groups == 0 && p->d.kv_dtype == PKV_FP8_E4M3 && gh < 8;
    if ((algo == PKV_ALGO_AUTO && !left) || algo == PKV_ALGO_TC) {
        pkv_pool* mp = const_cast<pkv_pool*>(p);
        if (prefix_tc_fits(p, num_seqs, num_groups, gh, max_seq_len) && ensure_tmaps(mp) &&
            (p->d.kv_dtype == PKV_FP8_E4M3 || p->tmap_half == 1))
            return PKV_ALGO_TC;
        if (algo == PKV_ALGO_TC) return -1;
    }
    return design_for(p, 1, gh, 0, algo, false);
}

constexpr int32_t kMaxListed = 1 << 30;  // token rows and free blocks: their sums and places are int32

int block_shift(const pkv_pool* p) { return p->d.block_size == 16 ? 4 : (p->d.block_size == 32 ? 5 : 6); }

bool ranges_overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

}  // namespace
}  // namespace pkv

extern "C" {

pkv_status paged_prefix_decode_plan(const pkv_pool* p, int32_t num_seqs, int32_t num_groups, int32_t num_q_heads,
                                    int32_t max_seq_len, size_t* ws_out) {
    if (num_groups < 0) return PKV_ERR_INVALID_ARG;
    size_t need = 0;
    const pkv_status st = paged_decode_plan(p, num_seqs, num_q_heads, max_seq_len, 0, nullptr, nullptr, &need);
    if (st != PKV_OK) return st;
    if (prefix_tc_fits(p, num_seqs, num_groups, num_q_heads / p->d.num_kv_heads, max_seq_len)) {
        const size_t shared = prefix_layout(p, num_seqs, num_groups, num_q_heads, nullptr, nullptr);
        if (shared > need) need = shared;
    }
    if (ws_out) *ws_out = need;
    return PKV_OK;
}

int32_t paged_prefix_decode_algo(const pkv_pool* p, int32_t num_seqs, int32_t num_groups, int32_t num_q_heads,
                                 int32_t max_seq_len, pkv_algo algo) {
    if (!p || num_seqs < 0 || num_groups < 0 || num_q_heads < 1 || num_q_heads % p->d.num_kv_heads != 0 ||
        max_seq_len < 0)
        return -1;
    return prefix_design(p, num_seqs, num_groups, num_q_heads, max_seq_len, algo);
}

pkv_status paged_prefix_decode_attention(const void* q, pkv_dtype q_dtype, const pkv_pool* p, int32_t layer,
                                         const int32_t* block_tables, int32_t max_blocks_per_seq,
                                         const int32_t* seq_lens, int32_t num_seqs, int32_t num_q_heads,
                                         int32_t max_seq_len, const int32_t* group_offsets,
                                         const int32_t* prefix_lens, int32_t num_groups, float scale, pkv_algo algo,
                                         void* workspace, size_t workspace_bytes, void* out, void* stream) {
    size_t need = 0;
    if (!p) return PKV_ERR_INVALID_ARG;
    pkv_status st = paged_prefix_decode_plan(p, num_seqs, num_groups, num_q_heads, max_seq_len, &need);
    if (st != PKV_OK) return st;
    if (num_groups > 0 && (!group_offsets || !prefix_lens || !aligned(group_offsets, 4) || !aligned(prefix_lens, 4)))
        return PKV_ERR_INVALID_ARG;
    const int design = prefix_design(p, num_seqs, num_groups, num_q_heads, max_seq_len, algo);
    // every other check is decode attention's (TC there means another kernel)
    const pkv_algo decode_algo = algo == PKV_ALGO_TC ? PKV_ALGO_AUTO : algo;
    st = attention_call(q, q_dtype, p, layer, block_tables, max_blocks_per_seq, seq_lens, num_seqs, 1, num_q_heads,
                        max_seq_len, scale, 0, decode_algo, workspace, workspace_bytes, out, stream, nullptr, nullptr,
                        PKV_BF16, true);
    if (st != PKV_OK) return st;
    if (design < 0) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return PKV_ERR_WORKSPACE;
    if (design != PKV_ALGO_TC)
        return attention_call(q, q_dtype, p, layer, block_tables, max_blocks_per_seq, seq_lens, num_seqs, 1,
                              num_q_heads, max_seq_len, scale, 0, algo, workspace, workspace_bytes, out, stream,
                              nullptr, nullptr, PKV_BF16);
    PrefixArgs a{};
    prefix_layout(p, num_seqs, num_groups, num_q_heads, static_cast<uint8_t*>(workspace), &a);
    a.q = q;
    a.out = out;
    a.tables = block_tables;
    a.lens = seq_lens;
    a.group_offsets = group_offsets;
    a.prefix_lens = prefix_lens;
    a.err = p->d.error_word;
    a.layer = layer;
    a.max_blocks = max_blocks_per_seq;
    a.max_len = max_seq_len;
    a.num_seqs = num_seqs;
    a.num_groups = num_groups;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = p->d.num_kv_heads;
    a.block_size = p->d.block_size;
    a.num_blocks = p->d.num_blocks;
    a.test_polls = g_test_wait_polls;
    a.test_cta = g_test_wait_cta;
    a.gh = num_q_heads / p->d.num_kv_heads;
    a.seqs_per_tile = kPrefixRows / a.gh;
    a.qk_scale_log2 = scale * p->d.k_scale * 1.4426950408889634f;
    a.v_scale = p->d.v_scale;
    CUtensorMap q_group, q_own;
    if (!encode_q_map(&q_group, q, num_seqs, num_q_heads, a.gh, a.seqs_per_tile) ||
        !encode_q_map(&q_own, q, num_seqs, num_q_heads, a.gh, 1))
        return PKV_ERR_UNSUPPORTED;
    const bool fp8 = p->d.kv_dtype == PKV_FP8_E4M3;
    return cuda_status(launch_prefix_attention(p->d.kv_dtype, a, fp8 ? &p->tmap_k : &p->tmap_kh,
                                               fp8 ? &p->tmap_v : &p->tmap_vh, &q_group, &q_own,
                                               static_cast<cudaStream_t>(stream)));
}

pkv_status kv_append_norm_rope(const pkv_pool* p, int32_t layer, const void* q, const void* k, const void* v,
                               pkv_dtype in_dtype, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                               const int32_t* positions, const int64_t* slot_mapping, int32_t num_tokens,
                               int32_t num_q_heads, const pkv_norm_rope* r, void* q_out, void* stream) {
    if (!p || !r || layer < 0 || layer >= p->d.num_layers || num_tokens < 0 || num_q_heads < 1)
        return PKV_ERR_INVALID_ARG;
    if (in_dtype != PKV_F32 && in_dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
    if (p->d.kv_dtype == PKV_F32 && in_dtype != PKV_F32) return PKV_ERR_UNSUPPORTED;
    const int D = p->d.head_dim;
    if (static_cast<int64_t>(num_q_heads) + 2LL * p->d.num_kv_heads > (1 << 20)) return PKV_ERR_UNSUPPORTED;
    if (r->rotary_dim < 16 || r->rotary_dim > D || r->rotary_dim % 16 != 0 || r->max_pos < 1)
        return PKV_ERR_INVALID_ARG;
    if ((r->interleaved != 0 && r->interleaved != 1) || r->num_axes < 1 || r->num_axes > 3) return PKV_ERR_INVALID_ARG;
    int64_t pairs = 0;
    for (int i = 0; i < r->num_axes; ++i) {
        if (r->sections[i] < 0) return PKV_ERR_INVALID_ARG;
        pairs += r->sections[i];
    }
    if (pairs != r->rotary_dim / 2) return PKV_ERR_INVALID_ARG;
    if ((r->q_weight == nullptr) != (r->k_weight == nullptr)) return PKV_ERR_INVALID_ARG;
    if (r->q_weight) {
        if (r->weight_dtype != PKV_F32 && r->weight_dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
        if (!aligned(r->q_weight, 16) || !aligned(r->k_weight, 16)) return PKV_ERR_INVALID_ARG;
        // (a subnormal eps would count as zero, and a row of zeros become NaN)
        if (!(std::isnormal(r->eps) && r->eps > 0.f)) return PKV_ERR_INVALID_ARG;
    }
    for (int64_t s : {q_stride, k_stride, v_stride})
        if (s < 0 || s % 8 != 0 || s > INT64_MAX / 8 / (num_tokens > 0 ? num_tokens : 1)) return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    if (!q || !k || !v || !q_out || !positions || !slot_mapping || !r->cos_sin) return PKV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(r->cos_sin, 16) ||
        !aligned(positions, 4) || !aligned(slot_mapping, 8))
        return PKV_ERR_INVALID_ARG;
    const pkv_dtype q_dtype = p->d.kv_dtype == PKV_F32 ? PKV_F32 : PKV_BF16;
    const size_t in_bytes = dtype_bytes(in_dtype), T1 = num_tokens - 1;
    const size_t q_row = static_cast<size_t>(num_q_heads) * D, kv_row = static_cast<size_t>(p->d.num_kv_heads) * D;
    const size_t out_bytes = q_row * num_tokens * dtype_bytes(q_dtype);
    const bool in_place = q_out == q && q_dtype == in_dtype && (num_tokens == 1 || q_stride == static_cast<int64_t>(q_row));
    if (!in_place && ranges_overlap(q_out, out_bytes, q, (T1 * q_stride + q_row) * in_bytes)) return PKV_ERR_INVALID_ARG;
    if (ranges_overlap(q_out, out_bytes, k, (T1 * k_stride + kv_row) * in_bytes) ||
        ranges_overlap(q_out, out_bytes, v, (T1 * v_stride + kv_row) * in_bytes))
        return PKV_ERR_INVALID_ARG;
    NormRopeArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out = q_out;
    a.k_layer = static_cast<uint8_t*>(p->d.k_base) + static_cast<size_t>(layer) * p->layer_bytes;
    a.v_layer = static_cast<uint8_t*>(p->d.v_base) + static_cast<size_t>(layer) * p->layer_bytes;
    a.positions = positions;
    a.slots = slot_mapping;
    a.cos_sin = r->cos_sin;
    a.q_weight = r->q_weight;
    a.k_weight = r->k_weight;
    a.weight_dtype = r->weight_dtype;
    a.eps = r->eps;
    a.num_tokens = num_tokens;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = p->d.num_kv_heads;
    a.num_slots = static_cast<int64_t>(p->d.num_blocks) * p->d.block_size;
    a.block_shift = block_shift(p);
    a.max_pos = r->max_pos;
    a.rotary_dim = r->rotary_dim;
    a.interleaved = r->interleaved;
    a.num_axes = r->num_axes;
    a.axis_end[0] = r->sections[0];
    a.axis_end[1] = r->num_axes > 1 ? r->sections[0] + r->sections[1] : r->sections[0];
    a.k_inv_scale = p->k_inv_scale;
    a.v_inv_scale = p->v_inv_scale;
    a.err = p->d.error_word;
    return cuda_status(launch_norm_rope_append(p->d.kv_dtype, in_dtype, D, a, static_cast<cudaStream_t>(stream)));
}

pkv_status kv_tables_grow(const pkv_pool* p, int32_t* block_tables, int32_t max_blocks_per_seq,
                          const int32_t* seq_lens, const int32_t* new_tokens, int32_t num_seqs,
                          const int32_t* free_ring, int32_t ring_size, const int32_t* free_state, int32_t max_tokens,
                          int64_t* slot_mapping, int32_t* positions, int32_t* token_seqs, int32_t* token_offsets,
                          int32_t* granted, int32_t* seq_lens_out, int32_t* free_state_out, void* stream) {
    if (!p || num_seqs < 0 || max_blocks_per_seq < 1 || ring_size < 1 || max_tokens < 0) return PKV_ERR_INVALID_ARG;
    if (static_cast<int64_t>(max_blocks_per_seq) * p->d.block_size > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    if (ring_size > pkv::kMaxListed || max_tokens > pkv::kMaxListed) return PKV_ERR_UNSUPPORTED;
    if (num_seqs > 0 && (!block_tables || !seq_lens || !new_tokens || !granted || !seq_lens_out))
        return PKV_ERR_INVALID_ARG;
    if (max_tokens > 0 && (!slot_mapping || !positions || !token_seqs)) return PKV_ERR_INVALID_ARG;
    if (!free_ring || !free_state || !free_state_out || !token_offsets) return PKV_ERR_INVALID_ARG;
    for (const void* x : {static_cast<const void*>(block_tables), static_cast<const void*>(seq_lens),
                          static_cast<const void*>(new_tokens), static_cast<const void*>(free_ring),
                          static_cast<const void*>(free_state), static_cast<const void*>(positions),
                          static_cast<const void*>(token_seqs), static_cast<const void*>(token_offsets),
                          static_cast<const void*>(granted), static_cast<const void*>(seq_lens_out),
                          static_cast<const void*>(free_state_out)})
        if (!aligned(x, 4)) return PKV_ERR_INVALID_ARG;
    if (!aligned(slot_mapping, 8)) return PKV_ERR_INVALID_ARG;
    GrowArgs a{};
    a.lens = seq_lens;
    a.new_tokens = new_tokens;
    a.tables = block_tables;
    a.ring = free_ring;
    a.free_state = free_state;
    a.ring_size = ring_size;
    a.num_seqs = num_seqs;
    a.max_blocks = max_blocks_per_seq;
    a.block_shift = block_shift(p);
    a.num_blocks = p->d.num_blocks;
    a.max_tokens = max_tokens;
    a.slots = slot_mapping;
    a.positions = positions;
    a.token_seqs = token_seqs;
    a.token_offsets = token_offsets;
    a.granted = granted;
    a.lens_out = seq_lens_out;
    a.free_out = free_state_out;
    a.err = p->d.error_word;
    return cuda_status(launch_tables_grow(a, static_cast<cudaStream_t>(stream)));
}

pkv_status kv_tables_release(const pkv_pool* p, const int32_t* block_tables, int32_t max_blocks_per_seq,
                             const int32_t* seq_lens, const int32_t* finished, const int32_t* keep_blocks,
                             int32_t num_seqs, int32_t* free_ring, int32_t ring_size, const int32_t* free_state,
                             int32_t* seq_lens_out, int32_t* free_state_out, void* stream) {
    if (!p || num_seqs < 0 || max_blocks_per_seq < 1 || ring_size < 1) return PKV_ERR_INVALID_ARG;
    if (static_cast<int64_t>(max_blocks_per_seq) * p->d.block_size > INT32_MAX || ring_size > pkv::kMaxListed)
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs > 0 && (!block_tables || !seq_lens || !finished || !seq_lens_out)) return PKV_ERR_INVALID_ARG;
    if (!free_ring || !free_state || !free_state_out) return PKV_ERR_INVALID_ARG;
    for (const void* x : {static_cast<const void*>(block_tables), static_cast<const void*>(seq_lens),
                          static_cast<const void*>(finished), static_cast<const void*>(keep_blocks),
                          static_cast<const void*>(free_ring), static_cast<const void*>(free_state),
                          static_cast<const void*>(seq_lens_out), static_cast<const void*>(free_state_out)})
        if (!aligned(x, 4)) return PKV_ERR_INVALID_ARG;
    ReleaseArgs a{};
    a.lens = seq_lens;
    a.finished = finished;
    a.keep_blocks = keep_blocks;
    a.tables = block_tables;
    a.ring = free_ring;
    a.free_state = free_state;
    a.ring_size = ring_size;
    a.num_seqs = num_seqs;
    a.max_blocks = max_blocks_per_seq;
    a.block_shift = block_shift(p);
    a.num_blocks = p->d.num_blocks;
    a.lens_out = seq_lens_out;
    a.free_out = free_state_out;
    a.err = p->d.error_word;
    return cuda_status(launch_tables_release(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
