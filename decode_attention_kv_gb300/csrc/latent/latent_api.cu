// latent_api.cu -- the C ABI of the latent-cache operators: argument checks,
// plans and launches.  Allocates nothing, never synchronises; every launch
// goes to the caller's stream.
#include <cudaTypedefs.h>

#include <cstdarg>
#include <cstdio>
#include <mutex>

#include "../kvd_internal.h"
#include "latent_common.cuh"

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

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t elem_size(kvd_dtype dt) { return dt == KVD_BF16 ? 2 : 4; }
bool dtype_ok(kvd_dtype dt) { return dt == KVD_BF16 || dt == KVD_F32; }
size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// How kvd_attend_latent divides a call (a function of the sizes only).
struct LatentPlan {
    int groups, rpg, workers, min_shift, lead;
    size_t off_lse, off_o, bytes;
};

kvd_status latent_plan(const char* fn, int Q, int T, int H, int BS, int cols, int R, int P,
                       kvd_dtype dt, LatentPlan* pl) {
    if (Q < 0 || T < 1 || H < 1 || BS < 1 || cols < 1)
        return fail(KVD_ERR_INVALID_ARG, "%s: Q >= 0 and T, H, BS, cols >= 1 required", fn);
    if (!dtype_ok(dt)) return fail(KVD_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (R != 128 && R != 256 && R != 384 && R != 512)
        return fail(KVD_ERR_UNSUPPORTED, "%s: R = %d (supported: 128, 256, 384, 512)", fn, R);
    if (P != 64) return fail(KVD_ERR_UNSUPPORTED, "%s: P = %d (supported: 64)", fn, P);
    if (Q > 65535) return fail(KVD_ERR_UNSUPPORTED, "%s: Q > 65535", fn);
    if ((long long)Q * T * H >= (1ll << 31)) return fail(KVD_ERR_UNSUPPORTED, "%s: Q*T*H >= 2^31", fn);
    if ((long long)T * H > 65535) return fail(KVD_ERR_UNSUPPORTED, "%s: T*H > 65535", fn);
    if ((long long)cols * BS >= (1ll << 31)) return fail(KVD_ERR_UNSUPPORTED, "%s: cols*BS >= 2^31", fn);
    const bool mma = dt == KVD_BF16;
    // fp32: two CTAs an SM, above R = 256 one (shared memory)
    const int rows = T * H, most = mma ? 64 : 16,
              ctas = mma || R > 256 ? kLatentSMs : 2 * kLatentSMs;
    pl->groups = (rows + most - 1) / most;
    pl->rpg = (rows + pl->groups - 1) / pl->groups;
    pl->workers = pl->groups < ctas ? ctas / pl->groups : 1;
    pl->min_shift = mma ? 1 : 0;
    pl->lead = mma ? 2 : 1;
    // a single worker shares no sequence: no partial rows
    const size_t slots = pl->workers > 1 ? (size_t)pl->workers * pl->groups * 2 : 0;
    pl->off_lse = round256((size_t)(Q < 1 ? 1 : Q) * sizeof(int4));
    pl->off_o = pl->off_lse + round256(slots * pl->rpg * 4);
    pl->bytes = pl->off_o + slots * pl->rpg * R * 4;
    return KVD_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;
cudaError_t g_encode_err = cudaSuccess;

}  // namespace

namespace kvd {

cudaError_t encode_rows(CUtensorMap* map, const void* base, long long width, long long stride,
                        long long rows, int box_rows, int box_chunks) {
    std::call_once(g_encode_once, [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q{};
        g_encode_err = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                        cudaEnableDefault, &q);
        if (g_encode_err == cudaSuccess && q != cudaDriverEntryPointSuccess)
            g_encode_err = cudaErrorNotSupported;
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    if (g_encode_err != cudaSuccess) return g_encode_err;
    const cuuint64_t dims[3] = {64u, (cuuint64_t)rows, (cuuint64_t)(width / 64)};
    const cuuint64_t strides[2] = {(cuuint64_t)stride * 2, 128u};
    const cuuint32_t box[3] = {64u, (cuuint32_t)box_rows, (cuuint32_t)box_chunks};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    const CUresult r =
        g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
                 box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace kvd

extern "C" {

kvd_status kvd_append_latent(void* latent_cache, void* rope_cache, const void* latent_new,
                             const void* rope_new, const int32_t* block_tables,
                             const int32_t* seq_offset, const int32_t* new_lens,
                             const int32_t* pos, int Q, int N, int NB, int BS, int cols, int R,
                             int P, kvd_dtype dtype, int32_t* dev_status, kvd_stream_t stream) {
    const char* fn = "kvd_append_latent";
    if (Q < 0 || N < 0 || NB < 1 || BS < 1 || cols < 1 || R < 1 || P < 1)
        return fail(KVD_ERR_INVALID_ARG, "%s: Q, N >= 0 and NB, BS, cols, R, P >= 1 required", fn);
    if (!dtype_ok(dtype)) return fail(KVD_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (Q == 0 || N == 0) return ok();
    if (!latent_cache || !rope_cache || !latent_new || !rope_new || !block_tables || !new_lens ||
        !pos)
        return fail(KVD_ERR_INVALID_ARG, "%s: null pointer", fn);
    const long long lb = (long long)R * elem_size(dtype), rb = (long long)P * elem_size(dtype);
    if (lb % 16 || rb % 16)
        return fail(KVD_ERR_INVALID_ARG, "%s: rows must be whole 16-byte vectors", fn);
    if (lb >= (1ll << 31) || rb >= (1ll << 31))
        return fail(KVD_ERR_UNSUPPORTED, "%s: row too large", fn);
    if (!aligned(latent_cache, 16) || !aligned(rope_cache, 16) || !aligned(latent_new, 16) ||
        !aligned(rope_new, 16) || !aligned(block_tables, 4) || !aligned(seq_offset, 4) ||
        !aligned(new_lens, 4) || !aligned(pos, 4) || !aligned(dev_status, 4))
        return fail(KVD_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    return launched(fn, launch_append_latent(latent_cache, rope_cache, latent_new, rope_new,
                                             block_tables, seq_offset, new_lens, pos, Q, N, NB, BS,
                                             cols, (int)lb, (int)rb, dev_status,
                                             (cudaStream_t)stream));
}

size_t kvd_attend_latent_workspace_bytes(int Q, int T, int H, int BS, int cols, int R, int P,
                                         kvd_dtype dtype) {
    LatentPlan pl;
    const kvd_status st = latent_plan("kvd_attend_latent_workspace_bytes", Q, T, H, BS, cols, R, P,
                                      dtype, &pl);
    return st == KVD_OK ? pl.bytes : 0;
}

kvd_status kvd_attend_latent(const void* q_latent, const void* q_rope, const void* latent_cache,
                             const void* rope_cache, const int32_t* block_tables,
                             const int32_t* seq_lens, const int32_t* seq_offset, void* out,
                             float* lse_out, int Q, int T, int H, int NB, int BS, int cols, int R,
                             int P, float scale, kvd_dtype dtype, void* workspace,
                             size_t workspace_bytes, int32_t* dev_status, kvd_stream_t stream) {
    const char* fn = "kvd_attend_latent";
    LatentPlan pl;
    const kvd_status st = latent_plan(fn, Q, T, H, BS, cols, R, P, dtype, &pl);
    if (st != KVD_OK) return st;
    if (NB < 1) return fail(KVD_ERR_INVALID_ARG, "%s: NB >= 1 required", fn);
    if ((long long)NB * BS >= (1ll << 31)) return fail(KVD_ERR_UNSUPPORTED, "%s: NB*BS >= 2^31", fn);
    if (Q == 0) return ok();
    if (!q_latent || !q_rope || !latent_cache || !rope_cache || !block_tables || !seq_lens || !out)
        return fail(KVD_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(q_latent, 16) || !aligned(q_rope, 16) || !aligned(latent_cache, 16) ||
        !aligned(rope_cache, 16) || !aligned(out, 16) || !aligned(lse_out, 4) ||
        !aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(seq_offset, 4) ||
        !aligned(dev_status, 4))
        return fail(KVD_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    if (!workspace || workspace_bytes < pl.bytes)
        return fail(KVD_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, pl.bytes,
                    workspace ? workspace_bytes : (size_t)0);
    if (!aligned(workspace, 256))
        return fail(KVD_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", fn);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    LatentArgs a{};
    a.q_latent = q_latent;
    a.q_rope = q_rope;
    a.latent = latent_cache;
    a.rope = rope_cache;
    a.block_tables = block_tables;
    a.seq_lens = seq_lens;
    a.seq_offset = seq_offset;
    a.out = out;
    a.lse_out = lse_out;
    a.dev_status = dev_status;
    a.Q = Q;
    a.T = T;
    a.H = H;
    a.NB = NB;
    a.BS = BS;
    a.cols = cols;
    a.R = R;
    a.P = P;
    a.qscale = scale * kLog2e;
    a.rows = T * H;
    a.groups = pl.groups;
    a.rpg = pl.rpg;
    a.workers = pl.workers;
    a.min_shift = pl.min_shift;
    a.by_page = FastDiv(BS);
    a.by_head = FastDiv(H);
    a.lead = pl.lead;
    a.meta = reinterpret_cast<int4*>(ws);
    a.part_lse = reinterpret_cast<float*>(ws + pl.off_lse);
    a.part_o = reinterpret_cast<float*>(ws + pl.off_o);
    cudaError_t e = dtype == KVD_BF16 ? launch_latent_mma(a, (cudaStream_t)stream)
                                      : launch_latent_simt(a, (cudaStream_t)stream);
    if (e == cudaSuccess) e = launch_latent_combine(a, dtype, (cudaStream_t)stream);
    return launched(fn, e);
}

kvd_status kvd_attend_expanded(const void* q, const void* kv, const void* k_rope,
                               const int32_t* q_lens, const int32_t* k_lens, void* out,
                               float* lse_out, int Q, int Nq, int Nk, int H, int Dn, int Dv, int P,
                               float scale, int causal, kvd_dtype dtype, int32_t* dev_status,
                               kvd_stream_t stream) {
    const char* fn = "kvd_attend_expanded";
    if (Q < 0 || Nq < 0 || Nk < 0 || H < 1)
        return fail(KVD_ERR_INVALID_ARG, "%s: Q, Nq, Nk >= 0 and H >= 1 required", fn);
    if (!dtype_ok(dtype)) return fail(KVD_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if ((Dn != 64 && Dn != 128) || (Dv != 64 && Dv != 128) || P != 64)
        return fail(KVD_ERR_UNSUPPORTED, "%s: Dn = %d, Dv = %d, P = %d (supported: 64 or 128, 64 or 128, 64)",
                    fn, Dn, Dv, P);
    if (H > 65535) return fail(KVD_ERR_UNSUPPORTED, "%s: H > 65535", fn);
    if (Nq > (1 << 23) || Nk > (1 << 30) || Q > (1 << 14))
        return fail(KVD_ERR_UNSUPPORTED, "%s: Q > 2^14, Nq > 2^23 or Nk > 2^30", fn);
    if (Q == 0 || Nq == 0) return ok();
    if (!q || !q_lens || !k_lens || !out || (Nk > 0 && (!kv || !k_rope)))
        return fail(KVD_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(k_rope, 16) || !aligned(out, 16) ||
        !aligned(lse_out, 4) || !aligned(q_lens, 4) || !aligned(k_lens, 4) ||
        !aligned(dev_status, 4))
        return fail(KVD_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    ExpandedArgs a{};
    a.q = q;
    a.kv = kv;
    a.k_rope = k_rope;
    a.q_lens = q_lens;
    a.k_lens = k_lens;
    a.out = out;
    a.lse_out = lse_out;
    a.dev_status = dev_status;
    a.Q = Q;
    a.Nq = Nq;
    a.Nk = Nk;
    a.H = H;
    a.Dn = Dn;
    a.Dv = Dv;
    a.P = P;
    a.qscale = scale * kLog2e;
    a.causal = causal != 0;
    return launched(fn, dtype == KVD_BF16 ? launch_expanded_mma(a, (cudaStream_t)stream)
                                          : launch_expanded_simt(a, (cudaStream_t)stream));
}

kvd_status kvd_verify_drafts(const void* target_probs, const void* draft_probs,
                             const int32_t* draft_tokens, const float* u_accept,
                             const float* u_sample, const int32_t* num_drafts, int32_t* tokens,
                             int32_t* accepted, int Q, int T, int V, kvd_dtype dtype,
                             int32_t* dev_status, kvd_stream_t stream) {
    const char* fn = "kvd_verify_drafts";
    if (Q < 0 || T < 0 || V < 1)
        return fail(KVD_ERR_INVALID_ARG, "%s: Q, T >= 0 and V >= 1 required", fn);
    if (!dtype_ok(dtype)) return fail(KVD_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (Q > (1 << 24) || T > (1 << 24) || V > (1 << 30))
        return fail(KVD_ERR_UNSUPPORTED, "%s: Q or T > 2^24, or V > 2^30", fn);
    if (Q == 0) return ok();
    if (!target_probs || !u_sample || !tokens || !accepted ||
        (T > 0 && (!draft_probs || !draft_tokens || !u_accept)))
        return fail(KVD_ERR_INVALID_ARG, "%s: null pointer", fn);
    const size_t es = elem_size(dtype);
    if (!aligned(target_probs, es) || !aligned(draft_probs, es) || !aligned(draft_tokens, 4) ||
        !aligned(u_accept, 4) || !aligned(u_sample, 4) || !aligned(num_drafts, 4) ||
        !aligned(tokens, 4) || !aligned(accepted, 4) || !aligned(dev_status, 4))
        return fail(KVD_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    return launched(fn, launch_verify_drafts(target_probs, draft_probs, draft_tokens, u_accept,
                                             u_sample, num_drafts, tokens, accepted, Q, T, V,
                                             dtype, dev_status, (cudaStream_t)stream));
}

}  // extern "C"
