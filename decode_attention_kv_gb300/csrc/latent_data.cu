// latent_data.cu -- the latent cache's append and the verification of drafted
// tokens: the two latent-decode operators that are bound by memory alone.
#include <cooperative_groups.h>

#include "kvd_internal.h"
#include "latent_common.cuh"

namespace kvd {
namespace {

namespace cg = cooperative_groups;

// ------------------------------------------------------------ append_latent
// One warp a row: 16-byte vectors of the latent row, then of the rotary row.
// The sequence of a packed row comes from a binary search in new_lens.  The
// row's own loads do not depend on the search, so they are issued first.
constexpr int kAppendWarps = 8;
constexpr int kAppendVecs = 4;  // vectors a lane holds across the search

__global__ void __launch_bounds__(kAppendWarps * 32)
append_latent_kernel(unsigned char* __restrict__ latent, unsigned char* __restrict__ rope,
                     const unsigned char* __restrict__ latent_new,
                     const unsigned char* __restrict__ rope_new,
                     const int32_t* __restrict__ block_tables,
                     const int32_t* __restrict__ seq_offset, const int32_t* __restrict__ new_lens,
                     const int32_t* __restrict__ pos, int Q, int N, int NB, int BS, int cols,
                     int lv, int rv, int32_t* dev_status) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    if (blockIdx.x == 0) {  // the whole of new_lens is checked once
        bool bad = false;
        for (int b = threadIdx.x; b < Q; b += blockDim.x) {
            const int s0 = new_lens[b], s1 = new_lens[b + 1];
            bad |= (b == 0 && s0 != 0) || s1 < s0 || s1 > N;
        }
        if (bad) report(dev_status, KVD_DEV_SEQLENS);
    }
    if (row >= N) return;
    const int nv = lv + rv;
    const uint4* ls = reinterpret_cast<const uint4*>(latent_new) + (size_t)row * lv;
    const uint4* rs = reinterpret_cast<const uint4*>(rope_new) + (size_t)row * rv;
    uint4 x[kAppendVecs];
#pragma unroll
    for (int i = 0; i < kAppendVecs; ++i) {
        const int v = lane + 32 * i;
        if (v < nv) x[i] = v < lv ? __ldcs(ls + v) : __ldcs(rs + (v - lv));
    }
    int lo = 0, hi = Q;  // the first b with new_lens[b + 1] > row
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (new_lens[mid + 1] > row)
            hi = mid;
        else
            lo = mid + 1;
    }
    if (lo >= Q) return;
    const int s0 = new_lens[lo], s1 = new_lens[lo + 1];
    if (new_lens[0] != 0 || s0 < 0 || row < s0 || s1 > N) return;  // reported above
    const long long p0 = pos[lo];
    if (p0 < 0) {
        if (lane == 0) report(dev_status, KVD_DEV_POS_RANGE);
        return;
    }
    const long long t = p0 + (row - s0);
    const int off = seq_offset ? seq_offset[lo] : 0;
    if (off < 0 || off % BS) {
        if (lane == 0) report(dev_status, KVD_DEV_SEQ_OFFSET);
        return;
    }
    const long long col = off / BS + t / BS;
    if (col >= cols) {
        if (lane == 0) report(dev_status, KVD_DEV_TABLE_COLS);
        return;
    }
    const int phys = block_tables[(size_t)lo * cols + col];
    if (phys < 0 || phys >= NB) {
        if (lane == 0) report(dev_status, KVD_DEV_BLOCK_RANGE);
        return;
    }
    const size_t dst = (size_t)phys * BS + (size_t)(t % BS);
    uint4* ld = reinterpret_cast<uint4*>(latent) + dst * lv;
    uint4* rd = reinterpret_cast<uint4*>(rope) + dst * rv;
#pragma unroll
    for (int i = 0; i < kAppendVecs; ++i) {
        const int v = lane + 32 * i;
        if (v < nv) (v < lv ? ld + v : rd + (v - lv))[0] = x[i];
    }
    for (int v = lane + 32 * kAppendVecs; v < nv; v += 32)
        (v < lv ? ld + v : rd + (v - lv))[0] = v < lv ? ls[v] : rs[v - lv];
}

// ------------------------------------------------------------ verify_drafts
// A cluster of kVerifyCtas CTAs a sequence, a contiguous share of the row each,
// a contiguous share of that per warp.  Pass 1 sums the weights of every warp's
// share; the cluster exchanges the sums through distributed shared memory, so
// every CTA knows where the target sum falls; the one warp whose share holds it
// reads that share again (from L2) in order.
//
// A sum must decide the same token as one in 64 bits, and 64-bit additions run
// at a small fraction of the fp32 rate here: the difference p - q is taken
// exactly as two fp32 words and the running sum is held in two (Knuth's
// two-sum), about 2^-48 relative, and only the sums of the threads are added in
// 64 bits.
constexpr int kVerifyCtas = 8;
constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyBatch = 8;  // loads in flight a lane and array

__device__ __forceinline__ float prob(const float* p, size_t i) { return p[i]; }
__device__ __forceinline__ float prob(const __nv_bfloat16* p, size_t i) {
    return __uint_as_float((uint32_t)reinterpret_cast<const unsigned short*>(p)[i] << 16);
}

// a + b = s + e exactly
__device__ __forceinline__ float two_sum(float a, float b, float& e) {
    const float s = __fadd_rn(a, b);
    const float bb = __fsub_rn(s, a);
    e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
    return s;
}

// The weight max(p - q, 0) as two words; NaN counts as zero.
__device__ __forceinline__ float2 weight(float p, float q) {
    float e;
    const float d = two_sum(p, -q, e);
    if (!(d > 0.f)) return make_float2(0.f, 0.f);  // d = 0 only where p = q
    return make_float2(d, isinf(d) ? 0.f : e);
}

struct VerifyShared {
    double warp_sum[kVerifyWarps];
    double cta_sum;
    int n, m, bad;
    int last;          // largest index of this CTA with a positive weight, or -1
    int warp_last[kVerifyWarps];
};

// Sum and largest positive index of this warp's share [lo, hi) of the row.
template <typename Elem, bool kRest>
__device__ __forceinline__ double share_sum(const Elem* p, const Elem* q, int lo, int hi,
                                            int& last) {
    const int lane = threadIdx.x & 31;
    float s = 0.f, c = 0.f;
    last = -1;
    for (int i0 = lo; i0 < hi; i0 += 32 * kVerifyBatch) {
        float a[kVerifyBatch], b[kVerifyBatch];
#pragma unroll
        for (int k = 0; k < kVerifyBatch; ++k) {
            const int i = i0 + 32 * k + lane;
            a[k] = i < hi ? prob(p, i) : 0.f;
            b[k] = kRest && i < hi ? prob(q, i) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kVerifyBatch; ++k) {
            const float2 w = weight(a[k], b[k]);
            float e;
            s = two_sum(s, w.x, e);
            c += e + w.y;
            if (w.x > 0.f) last = i0 + 32 * k + lane;
        }
    }
    double sum = (double)s + (isinf(s) ? 0.0 : (double)c);
#pragma unroll
    for (int k = 16; k; k >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, k);
        last = max(last, __shfl_xor_sync(0xffffffffu, last, k));
    }
    return sum;
}

// The first index of [lo, hi) whose running sum, from `border`, is above
// `want`; -1 if there is none.  Steps of 32 elements; the sums of a batch of
// steps are independent of one another, only the step that holds `want` is
// summed in order.
template <typename Elem, bool kRest>
__device__ __forceinline__ int find(const Elem* p, const Elem* q, int lo, int hi, double border,
                                    double want) {
    const int lane = threadIdx.x & 31;
    for (int i0 = lo; i0 < hi; i0 += 32 * kVerifyBatch) {
        double w[kVerifyBatch], s[kVerifyBatch];
#pragma unroll
        for (int k = 0; k < kVerifyBatch; ++k) {
            const int i = i0 + 32 * k + lane;
            const float2 x = weight(i < hi ? prob(p, i) : 0.f, kRest && i < hi ? prob(q, i) : 0.f);
            s[k] = w[k] = (double)x.x + (double)x.y;
        }
#pragma unroll
        for (int d = 16; d; d >>= 1)
#pragma unroll
            for (int k = 0; k < kVerifyBatch; ++k) s[k] += __shfl_xor_sync(0xffffffffu, s[k], d);
#pragma unroll
        for (int k = 0; k < kVerifyBatch; ++k) {
            if (border + s[k] > want) {
                double cum = w[k];
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const double o = __shfl_up_sync(0xffffffffu, cum, d);
                    if (lane >= d) cum += o;
                }
                const uint32_t above =
                    __ballot_sync(0xffffffffu, w[k] > 0.0 && border + cum > want);
                if (above) return i0 + 32 * k + __ffs(above) - 1;
            }
            border += s[k];
        }
    }
    return -1;
}

template <typename Elem>
__global__ void __cluster_dims__(kVerifyCtas, 1, 1) __launch_bounds__(kVerifyThreads)
verify_drafts_kernel(const Elem* __restrict__ target, const Elem* __restrict__ draft,
                     const int32_t* __restrict__ drafts, const float* __restrict__ u_accept,
                     const float* __restrict__ u_sample, const int32_t* __restrict__ num_drafts,
                     int32_t* __restrict__ tokens, int32_t* __restrict__ accepted, int T, int V,
                     int32_t* dev_status) {
    __shared__ VerifyShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster.block_rank();
    const int b = blockIdx.x / kVerifyCtas;
    const bool lead = rank == 0;
    if (warp == 0) {
        int m = num_drafts ? num_drafts[b] : T;
        const bool bad = m < 0 || m > T;
        if (bad) m = 0;
        int n = m;
        bool range = false;
        for (int i0 = 0; i0 < m && n == m; i0 += 32) {
            const int i = i0 + lane;
            bool ok = true, in = true;
            if (i < m) {
                const int x = drafts[(size_t)b * T + i];
                in = x >= 0 && x < V;
                ok = in && (double)u_accept[(size_t)b * T + i] *
                                   (double)prob(draft, ((size_t)b * T + i) * V + x) <
                               (double)prob(target, ((size_t)b * (T + 1) + i) * V + x);
            }
            const uint32_t no = __ballot_sync(0xffffffffu, !ok);
            const uint32_t out = __ballot_sync(0xffffffffu, !in);
            if (no) {
                const int first = __ffs(no) - 1;
                n = i0 + first;
                range = (out >> first) & 1u;
            }
        }
        if (lane == 0) {
            sh.n = n;
            sh.m = m;
            sh.bad = bad;
            if (lead && bad) report(dev_status, KVD_DEV_POS_RANGE);
            if (lead && range) report(dev_status, KVD_DEV_TOKEN_RANGE);
        }
    }
    __syncthreads();
    const int n = sh.n;
    if (lead) {
        for (int i = tid; i <= T; i += kVerifyThreads)
            if (i != n || sh.bad)
                tokens[(size_t)b * (T + 1) + i] = i < n ? drafts[(size_t)b * T + i] : -1;
        if (tid == 0) accepted[b] = n;
    }
    if (sh.bad) return;  // the same in all CTAs of the cluster
    const Elem* p = target + ((size_t)b * (T + 1) + n) * V;
    const Elem* q = draft + ((size_t)b * T + n) * V;
    const int share = (V + kVerifyCtas - 1) / kVerifyCtas;
    const int lo = min(rank * share, V), hi = min(lo + share, V);
    const int part = (hi - lo + kVerifyWarps - 1) / kVerifyWarps;
    const int wlo = min(lo + warp * part, hi), whi = min(wlo + part, hi);
    bool rest = n < sh.m;
    double total = 0.0, before = 0.0, behind = 0.0;
    int newest = -1;
    while (true) {
        int last;
        const double sum = rest ? share_sum<Elem, true>(p, q, wlo, whi, last)
                                : share_sum<Elem, false>(p, q, wlo, whi, last);
        if (lane == 0) {
            sh.warp_sum[warp] = sum;
            sh.warp_last[warp] = last;
        }
        __syncthreads();
        if (tid == 0) {
            double s = 0.0;
            int z = -1;
            for (int k = 0; k < kVerifyWarps; ++k) {
                s += sh.warp_sum[k];
                z = max(z, sh.warp_last[k]);
            }
            sh.cta_sum = s;
            sh.last = z;
        }
        cluster.sync();
        total = before = 0.0;
        newest = -1;
        for (int k = 0; k < kVerifyCtas; ++k) {
            const double s = *cluster.map_shared_rank(&sh.cta_sum, k);
            if (k == rank) before = total;
            total += s;
            if (k == rank) behind = total;
            newest = max(newest, *cluster.map_shared_rank(&sh.last, k));
        }
        cluster.sync();  // no CTA leaves or writes its sums again before all have read them
        if (!rest || newest >= 0) break;
        rest = false;    // nothing left of the target: the target itself
    }
    int32_t* token = tokens + (size_t)b * (T + 1) + n;
    if (newest < 0 || !isfinite(total)) {
        if (lead && tid == 0) {
            *token = -1;
            report(dev_status, KVD_DEV_PROBS);
        }
        return;
    }
    const double want = (double)u_sample[b] * total;
    if (!(want < total)) {
        if (lead && tid == 0) *token = newest;
        return;
    }
    // The CTAs' borders are the same sums in every CTA, so exactly one of them
    // has before <= want < behind; in it, one warp has the last border that is
    // not above `want`.
    if (!(before <= want && want < behind)) return;
    double border = before;
    for (int k = 0; k < warp; ++k) border += sh.warp_sum[k];
    if (!(border <= want) || (warp + 1 < kVerifyWarps && border + sh.warp_sum[warp] <= want))
        return;
    const int found = rest ? find<Elem, true>(p, q, wlo, whi, border, want)
                           : find<Elem, false>(p, q, wlo, whi, border, want);
    if (lane == 0) {
        // rounding between the two passes may leave none in the share: then its
        // largest positive index, or the nearest larger set's
        int v = found;
        if (v < 0) v = sh.warp_last[warp];
        if (v < 0) v = sh.last;
        *token = v < 0 ? newest : v;
    }
}

}  // namespace

cudaError_t launch_append_latent(void* latent, void* rope, const void* latent_new,
                                 const void* rope_new, const int32_t* block_tables,
                                 const int32_t* seq_offset, const int32_t* new_lens,
                                 const int32_t* pos, int Q, int N, int NB, int BS, int cols,
                                 int latent_bytes, int rope_bytes, int32_t* dev_status,
                                 cudaStream_t stream) {
    const dim3 grid((N + kAppendWarps - 1) / kAppendWarps);
    return launch_pdl(append_latent_kernel, grid, dim3(kAppendWarps * 32), 0, stream,
                      static_cast<unsigned char*>(latent), static_cast<unsigned char*>(rope),
                      static_cast<const unsigned char*>(latent_new),
                      static_cast<const unsigned char*>(rope_new), block_tables, seq_offset,
                      new_lens, pos, Q, N, NB, BS, cols, latent_bytes / 16, rope_bytes / 16,
                      dev_status);
}

cudaError_t launch_verify_drafts(const void* target, const void* draft, const int32_t* drafts,
                                 const float* u_accept, const float* u_sample,
                                 const int32_t* num_drafts, int32_t* tokens, int32_t* accepted,
                                 int Q, int T, int V, kvd_dtype dt, int32_t* dev_status,
                                 cudaStream_t stream) {
    const dim3 grid(Q * kVerifyCtas);
    if (dt == KVD_BF16)
        return launch_pdl(verify_drafts_kernel<__nv_bfloat16>, grid, dim3(kVerifyThreads), 0,
                          stream, static_cast<const __nv_bfloat16*>(target),
                          static_cast<const __nv_bfloat16*>(draft), drafts, u_accept, u_sample,
                          num_drafts, tokens, accepted, T, V, dev_status);
    return launch_pdl(verify_drafts_kernel<float>, grid, dim3(kVerifyThreads), 0, stream,
                      static_cast<const float*>(target), static_cast<const float*>(draft), drafts,
                      u_accept, u_sample, num_drafts, tokens, accepted, T, V, dev_status);
}

}  // namespace kvd
