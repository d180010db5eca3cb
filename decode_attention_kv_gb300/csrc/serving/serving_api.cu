// serving_api.cu -- the C ABI of the serving step's operators: argument checks,
// plans and launches.  Allocates nothing, never synchronises; every launch goes to
// the caller's stream.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../kvd_internal.h"
#include "serving_common.cuh"

using namespace kvd;

namespace {

kvd_status fail(kvd_status s, const char* fmt, ...) {
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    set_last_error(msg);
    return s;
}

kvd_status ok() {
    set_last_error("");
    return KVD_OK;
}

kvd_status launched(const char* fn, cudaError_t e) {
    return e == cudaSuccess ? ok() : fail(KVD_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
}

template <typename... Ptr>
bool aligned(size_t a, Ptr... p) {
    return ((reinterpret_cast<uintptr_t>(p) % a == 0) && ...);
}
bool dtype_ok(kvd_dtype dt) { return dt == KVD_BF16 || dt == KVD_F32; }
size_t elem_size(kvd_dtype dt) { return dt == KVD_BF16 ? 2 : 4; }
size_t round256(size_t x) { return (x + 255) / 256 * 256; }

kvd_status check_rotation(const char* fn, int N, int D, int Dr, kvd_dtype dt) {
    if (N < 0) return fail(KVD_ERR_INVALID_ARG, "%s: N >= 0 required", fn);
    if (!dtype_ok(dt)) return fail(KVD_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (D != 64 && D != 128)
        return fail(KVD_ERR_UNSUPPORTED, "%s: head_dim %d (supported: 64, 128)", fn, D);
    if (Dr < 0 || Dr > D || Dr % 16)
        return fail(KVD_ERR_UNSUPPORTED, "%s: Dr = %d (supported: multiples of 16 up to D)", fn, Dr);
    return KVD_OK;
}

// How kvd_attend_paged_prefix divides a call (a function of the sizes only).
struct PrefixPlan {
    int rows, keys, lead, workers;
    PagedPartial own;
    size_t off_meta, off_plse, off_po, off_wlse, off_wo, bytes;
};

kvd_status prefix_plan(const char* fn, int Q, int G, int Hq, int Hkv, int BS, int pcols, int cols,
                       int D, kvd_dtype dt, PrefixPlan* pl) {
    if (Q < 0 || G < 0 || Hq < 1 || Hkv < 1 || BS < 1 || pcols < 1 || cols < 1)
        return fail(KVD_ERR_INVALID_ARG,
                    "%s: Q, G >= 0 and Hq, Hkv, BS, pcols, cols >= 1 required", fn);
    if (Hq % Hkv)
        return fail(KVD_ERR_INVALID_ARG, "%s: Hq (%d) must be a multiple of Hkv (%d)", fn, Hq, Hkv);
    if (!dtype_ok(dt)) return fail(KVD_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (D != 64 && D != 128)
        return fail(KVD_ERR_UNSUPPORTED, "%s: head_dim %d (supported: 64, 128)", fn, D);
    if (G > kMaxGroups) return fail(KVD_ERR_UNSUPPORTED, "%s: G > %d", fn, kMaxGroups);
    if ((long long)cols * BS >= (1ll << 31))
        return fail(KVD_ERR_UNSUPPORTED, "%s: cols*BS >= 2^31", fn);
    // (a prefix's length is rounded up to whole tiles of at most 128 keys in 32 bits)
    if ((long long)pcols * BS > (1ll << 31) - 128)
        return fail(KVD_ERR_UNSUPPORTED, "%s: pcols*BS > 2^31 - 128", fn);
    if ((long long)Q * Hq > (1ll << 28)) return fail(KVD_ERR_UNSUPPORTED, "%s: Q*Hq > 2^28", fn);
    const int g = Hq / Hkv, n = Q < 1 ? 1 : Q;
    const bool mma = dt == KVD_BF16;
    const int piece = prefix_piece_rows(BS);
    // bf16: two tiles of 128 rows a CTA, one where all sequences together have no more
    pl->rows = mma ? ((long long)n * g > 128 ? 256 : 128) : 16;
    pl->keys = mma ? 128 / piece * piece : 32;
    pl->lead = mma ? 4 : 2;  // (one place: 256 sequences behind 8192 tokens 76 us, four: 73)
    pl->workers = mma ? kServingSMs : 2 * kServingSMs;
    // the longest line that the groups can make
    const long long tiles = (long long)n * g / pl->rows + G + 1,
                    span = (long long)pcols * BS / pl->keys + 1 + pl->lead;
    if ((double)tiles * Hkv * span >= (double)(1 << 30))
        return fail(KVD_ERR_UNSUPPORTED, "%s: too many tiles of queries and prefix keys", fn);
    pl->own = paged_partial_plan(n, Hq, Hkv, BS, cols, D, dt);
    if (pl->own.units >= (1ll << 31))
        return fail(KVD_ERR_UNSUPPORTED, "%s: too many (row, split) units", fn);
    const size_t slots = 2 * (size_t)pl->workers * pl->rows, R = (size_t)n * Hq;
    pl->off_meta = round256(pl->own.bytes);
    pl->off_plse = pl->off_meta + round256((size_t)(n + 1) * sizeof(int4));
    pl->off_po = pl->off_plse + round256(slots * 4);
    pl->off_wlse = pl->off_po + round256(slots * D * 4);
    pl->off_wo = pl->off_wlse + round256(R * 4);
    pl->bytes = pl->off_wo + R * D * 4;
    return KVD_OK;
}

}  // namespace

extern "C" {

kvd_status kvd_plan_pages(int32_t* block_tables, int32_t* pages_held, int32_t* free_pages,
                          int32_t* free_count, const int32_t* kept_lens, const int32_t* new_lens,
                          const int32_t* pos_base, int32_t* seq_lens, int32_t* slots,
                          int32_t* positions, int Q, int N, int BS, int cols, int F,
                          int32_t* dev_status, kvd_stream_t stream) {
    const char* fn = "kvd_plan_pages";
    if (Q < 0 || N < 0 || F < 0 || BS < 1 || cols < 1)
        return fail(KVD_ERR_INVALID_ARG, "%s: Q, N, F >= 0 and BS, cols >= 1 required", fn);
    if (Q > (1 << 20) || N > (1 << 30))
        return fail(KVD_ERR_UNSUPPORTED, "%s: Q > 2^20 or N > 2^30", fn);
    if (!new_lens || !seq_lens || (Q > 0 && (!block_tables || !pages_held || !kept_lens)) ||
        (F > 0 && !free_pages) || !free_count || (N > 0 && (!slots || !positions)))
        return fail(KVD_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(4, block_tables, pages_held, free_pages, free_count, kept_lens, new_lens, pos_base,
                 seq_lens, slots, positions, dev_status))
        return fail(KVD_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    PlanArgs a{block_tables, pages_held, free_pages, free_count, kept_lens, new_lens, pos_base,
               seq_lens,     slots,      positions,  dev_status, Q,         N,        BS,
               cols,         F};
    return launched(fn, launch_plan_pages(a, (cudaStream_t)stream));
}

kvd_status kvd_rotary_freqs(double* freqs, int Dr, double base, kvd_rope_scaling scaling,
                            double factor, double trained, double fast, double slow) {
    const char* fn = "kvd_rotary_freqs";
    if (!freqs || Dr < 2 || Dr % 2 || !(base > 1.0) || !std::isfinite(base))
        return fail(KVD_ERR_INVALID_ARG, "%s: freqs, an even Dr >= 2 and base > 1 required", fn);
    if (scaling < KVD_ROPE_PLAIN || scaling > KVD_ROPE_PARTS)
        return fail(KVD_ERR_INVALID_ARG, "%s: unknown scaling", fn);
    if (scaling != KVD_ROPE_PLAIN && !(factor > 0.0 && std::isfinite(factor)))
        return fail(KVD_ERR_INVALID_ARG, "%s: factor > 0 required", fn);
    if (scaling == KVD_ROPE_BASE && Dr == 2)
        return fail(KVD_ERR_INVALID_ARG, "%s: a scaled base needs Dr > 2", fn);
    if (scaling == KVD_ROPE_PARTS && !(trained > 0.0 && fast > slow && slow > 0.0 &&
                                       std::isfinite(trained) && std::isfinite(fast)))
        return fail(KVD_ERR_INVALID_ARG, "%s: trained > 0 and fast > slow > 0 required", fn);
    const double kTurn = 6.283185307179586476925;
    if (scaling == KVD_ROPE_BASE) base *= std::pow(factor, (double)Dr / (Dr - 2));
    for (int i = 0; i < Dr / 2; ++i) {
        double f = std::pow(base, -2.0 * i / Dr);
        if (scaling == KVD_ROPE_LINEAR) f /= factor;
        if (scaling == KVD_ROPE_PARTS) {
            const double turns = trained * f / kTurn;
            const double x = (turns - slow) / (fast - slow);
            const double keep = x < 0.0 ? 0.0 : x > 1.0 ? 1.0 : x;
            f = f * keep + f / factor * (1.0 - keep);
        }
        freqs[i] = f;
    }
    return ok();
}

kvd_status kvd_rotate(const void* x, const void* weight, const double* freqs,
                      const int32_t* positions, void* out, int N, int H, int D, int Dr,
                      int interleaved, float rotary_scale, float eps, kvd_dtype dtype,
                      int32_t* dev_status, kvd_stream_t stream) {
    const char* fn = "kvd_rotate";
    const kvd_status st = check_rotation(fn, N, D, Dr, dtype);
    if (st != KVD_OK) return st;
    if (H < 1) return fail(KVD_ERR_INVALID_ARG, "%s: H >= 1 required", fn);
    if (H > 65535) return fail(KVD_ERR_UNSUPPORTED, "%s: H > 65535", fn);
    if (N == 0) return ok();
    if (!x || !positions || !out || (Dr > 0 && !freqs))
        return fail(KVD_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(16, x, weight, out) || !aligned(8, freqs) || !aligned(4, positions, dev_status))
        return fail(KVD_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    RotateArgs a{};
    a.x = x;
    a.q_weight = weight;
    a.freqs = freqs;
    a.positions = positions;
    a.q_out = out;
    a.dev_status = dev_status;
    a.N = N;
    a.Hq = H;
    a.D = D;
    a.Dr = Dr;
    a.stretch = rotary_scale;
    a.eps = eps;
    return launched(fn, launch_rotate(a, interleaved != 0, dtype, (cudaStream_t)stream));
}

kvd_status kvd_rotate_append_paged(const void* qkv, const void* q_weight, const void* k_weight,
                                   const double* freqs, const int32_t* positions,
                                   const int32_t* slots, void* q_out, void* key_cache,
                                   void* value_cache, int N, int Hq, int Hkv, int NB, int BS,
                                   int D, int Dr, int interleaved, float rotary_scale, float eps,
                                   kvd_dtype dtype, int32_t* dev_status, kvd_stream_t stream) {
    const char* fn = "kvd_rotate_append_paged";
    const kvd_status st = check_rotation(fn, N, D, Dr, dtype);
    if (st != KVD_OK) return st;
    if (Hq < 1 || Hkv < 1 || NB < 1 || BS < 1)
        return fail(KVD_ERR_INVALID_ARG, "%s: Hq, Hkv, NB, BS >= 1 required", fn);
    if (Hq > 65535 || Hkv > 65535) return fail(KVD_ERR_UNSUPPORTED, "%s: Hq or Hkv > 65535", fn);
    if ((long long)NB * BS >= (1ll << 31))
        return fail(KVD_ERR_UNSUPPORTED, "%s: NB*BS >= 2^31", fn);
    if (N == 0) return ok();
    if (!qkv || !positions || !slots || !q_out || !key_cache || !value_cache || (Dr > 0 && !freqs))
        return fail(KVD_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(16, qkv, q_weight, k_weight, q_out, key_cache, value_cache) || !aligned(8, freqs) ||
        !aligned(4, positions, slots, dev_status))
        return fail(KVD_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    RotateArgs a{};
    a.x = qkv;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.freqs = freqs;
    a.positions = positions;
    a.slots = slots;
    a.q_out = q_out;
    a.key_cache = key_cache;
    a.value_cache = value_cache;
    a.dev_status = dev_status;
    a.N = N;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = D;
    a.Dr = Dr;
    a.rows = (long long)NB * BS;
    a.stretch = rotary_scale;
    a.eps = eps;
    return launched(fn, launch_rotate(a, interleaved != 0, dtype, (cudaStream_t)stream));
}

size_t kvd_attend_paged_prefix_workspace_bytes(int Q, int G, int Hq, int Hkv, int BS, int pcols,
                                               int cols, int D, kvd_dtype dtype) {
    PrefixPlan pl;
    const kvd_status st = prefix_plan("kvd_attend_paged_prefix_workspace_bytes", Q, G, Hq, Hkv, BS,
                                      pcols, cols, D, dtype, &pl);
    return st == KVD_OK ? pl.bytes : 0;
}

kvd_status kvd_attend_paged_prefix(const void* q, const void* key_cache, const void* value_cache,
                                   const int32_t* prefix_tables, const int32_t* prefix_lens,
                                   const int32_t* group_lens, const int32_t* block_tables,
                                   const int32_t* seq_lens, const int32_t* seq_offset, void* out,
                                   float* lse_out, int Q, int G, int Hq, int Hkv, int NB, int BS,
                                   int pcols, int cols, int D, float scale, kvd_dtype dtype,
                                   void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                   kvd_stream_t stream) {
    const char* fn = "kvd_attend_paged_prefix";
    PrefixPlan pl;
    kvd_status st = prefix_plan(fn, Q, G, Hq, Hkv, BS, pcols, cols, D, dtype, &pl);
    if (st != KVD_OK) return st;
    if (NB < 1) return fail(KVD_ERR_INVALID_ARG, "%s: NB >= 1 required", fn);
    if ((long long)NB * BS >= (1ll << 31))
        return fail(KVD_ERR_UNSUPPORTED, "%s: NB*BS >= 2^31", fn);
    if (Q == 0) return ok();
    if (!q || !key_cache || !value_cache || !block_tables || !seq_lens || !out ||
        (G > 0 && (!prefix_tables || !prefix_lens || !group_lens)))
        return fail(KVD_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(16, q, key_cache, value_cache, out) ||
        !aligned(4, prefix_tables, prefix_lens, group_lens, block_tables, seq_lens, seq_offset,
                 lse_out, dev_status))
        return fail(KVD_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    if (!workspace || workspace_bytes < pl.bytes)
        return fail(KVD_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, pl.bytes,
                    workspace ? workspace_bytes : (size_t)0);
    if (!aligned(256, workspace))
        return fail(KVD_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", fn);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    PrefixArgs a{};
    a.q = q;
    a.k = key_cache;
    a.v = value_cache;
    a.prefix_tables = prefix_tables;
    a.prefix_lens = prefix_lens;
    a.group_lens = group_lens;
    a.out = out;
    a.lse_out = lse_out;
    a.dev_status = dev_status;
    a.Q = Q;
    a.G = G;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.g = Hq / Hkv;
    a.NB = NB;
    a.BS = BS;
    a.pcols = pcols;
    a.D = D;
    a.qscale = scale * kLog2e;
    a.rows = pl.rows;
    a.keys = pl.keys;
    a.lead = pl.lead;
    a.workers = pl.workers;
    if (dtype == KVD_BF16) {
        // A place costs 2.5 (1.75 alone, up to 4 while the sequences' own keys fill the queues
        // to memory): 64 sequences behind 16384 tokens with 64 to 1024 own ones 61, 58.4,
        // 57.7 and 59.8 us with 2, 2.5, 3 and 4; 256 behind 8192 with 16 to 256 70, 73, 77 and
        // 77.  An SM's share of the memory's rate is 45000 bytes a microsecond.  (All at D = 128
        // with two row tiles; D = 64 and one tile go by the same numbers.  own_units counts
        // splits of the tables' width, empty ones among them: the first case with tables
        // four times as wide as needed 69 us instead of 61.)
        a.place_cost = 2.5f;
        a.token_cost = (float)Hkv * D * 4 / 45000.f;
        a.own_units = (int)pl.own.units;
    }
    a.seq_lens = seq_lens;
    a.meta = reinterpret_cast<int4*>(ws + pl.off_meta);
    a.part_lse = reinterpret_cast<float*>(ws + pl.off_plse);
    a.part_o = reinterpret_cast<float*>(ws + pl.off_po);
    a.whole_lse = reinterpret_cast<float*>(ws + pl.off_wlse);
    a.whole_o = reinterpret_cast<float*>(ws + pl.off_wo);
    a.own_lse = reinterpret_cast<const float*>(ws + pl.own.off_lse);
    a.own_o = reinterpret_cast<const float*>(ws + pl.own.off_o);
    a.S = pl.own.S;
    a.counters = reinterpret_cast<uint32_t*>(ws);
    cudaError_t e = dtype == KVD_BF16 ? launch_prefix_mma(a, (cudaStream_t)stream)
                                      : launch_prefix_simt(a, (cudaStream_t)stream);
    if (e != cudaSuccess) return launched(fn, e);
    st = launch_paged_partial(fn, pl.own, q, key_cache, value_cache, block_tables, seq_lens,
                              seq_offset, Q, Hq, Hkv, NB, BS, cols, D, scale, dtype, ws, dev_status,
                              (cudaStream_t)stream);
    if (st != KVD_OK) return st;
    return launched(fn, launch_prefix_combine(a, dtype, (cudaStream_t)stream));
}

static kvd_status run_sampling(const char* fn, const void* logits, const float* temperature,
                               const int32_t* top_k, const float* top_p, const float* min_p,
                               const float* u, int32_t* tokens, void* probs, int R, int V,
                               kvd_dtype dtype, kvd_dtype probs_dtype, int32_t* dev_status,
                               kvd_stream_t stream) {
    if (R < 0 || V < 1) return fail(KVD_ERR_INVALID_ARG, "%s: R >= 0 and V >= 1 required", fn);
    if (!dtype_ok(dtype) || !dtype_ok(probs_dtype))
        return fail(KVD_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (R > (1 << 24) || V > (1 << 20))
        return fail(KVD_ERR_UNSUPPORTED, "%s: R > 2^24 or V > 2^20", fn);
    if (R == 0) return ok();
    if (!logits || (!probs && (!u || !tokens))) return fail(KVD_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(elem_size(dtype), logits) || !aligned(elem_size(probs_dtype), probs) ||
        !aligned(4, temperature, top_k, top_p, min_p, u, tokens, dev_status))
        return fail(KVD_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    SampleArgs a{logits, temperature, top_k, top_p, min_p, u, tokens, probs, dev_status,
                 R,      V,           probs_dtype == KVD_BF16};
    return launched(fn, launch_sample(a, dtype, (cudaStream_t)stream));
}

kvd_status kvd_sample(const void* logits, const float* temperature, const int32_t* top_k,
                      const float* top_p, const float* min_p, const float* u, int32_t* tokens,
                      int R, int V, kvd_dtype dtype, int32_t* dev_status, kvd_stream_t stream) {
    return run_sampling("kvd_sample", logits, temperature, top_k, top_p, min_p, u, tokens, nullptr,
                        R, V, dtype, KVD_F32, dev_status, stream);
}

kvd_status kvd_filter_probs(const void* logits, const float* temperature, const int32_t* top_k,
                            const float* top_p, const float* min_p, void* probs, int R, int V,
                            kvd_dtype dtype, kvd_dtype probs_dtype, int32_t* dev_status,
                            kvd_stream_t stream) {
    if (R > 0 && !probs) return fail(KVD_ERR_INVALID_ARG, "kvd_filter_probs: null pointer");
    return run_sampling("kvd_filter_probs", logits, temperature, top_k, top_p, min_p, nullptr,
                        nullptr, probs, R, V, dtype, probs_dtype, dev_status, stream);
}

}  // extern "C"
