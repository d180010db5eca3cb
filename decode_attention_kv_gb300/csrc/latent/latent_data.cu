// latent_data.cu -- the latent cache's append and the verification of drafted
// tokens: the two latent-decode operators that are bound by memory alone.
#include <cooperative_groups.h>

#include "../kvd_internal.h"
#include "latent_common.cuh"

namespace kvd {
namespace {

namespace cg = cooperative_groups;

// ------------------------------------------------------------ append_latent
// One warp a row: 16-byte vectors of the latent row, then of the rotary row.
// The sequence of a packed row comes from a binary search in new_lens.  The
// row's own loads do not depend on the search, so they are issued first.  (2, 4
// and 8 rows a warp copied 21000 rows of 1152 bytes no faster: 11.2, 11.9 and
// 13.3 against 11.1 us.)  21000 rows: 11.3 us in a graph, 10.6 as called over inputs in
// turn, 4.4 to 4.7 TB/s read and written; 64 rows: 2.8 and 3.3 us.
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
// A cluster of 1 to 8 CTAs a sequence (as many as keep the GPU full), a
// contiguous share of the row per CTA and of that per warp.  The row is read
// once: every warp sums its share, the CTAs push their sums to one another
// through distributed shared memory, and the CTA whose share the wanted sum
// falls into reads that one warp's share again (from L2), first a sixteenth of
// it per warp, then in order by the warp that holds the place.
//
// A sum must decide the same token as one in 64 bits, and 64-bit additions run
// at a small fraction of the fp32 rate here: the difference p - q is taken
// exactly as two fp32 words and the sums of 64 elements a lane are held in two
// (Knuth's two-sum; the second word's own rounding leaves about 2^-47 relative, at
// worst 2^-36); these are added in 64 bits, those of a CTA's warps by one warp (a
// 64-bit addition holds an SM's unit for 16 cycles a warp: with all warps at it
// every few elements they took longer than the row).
// 64 rows of 128000 fp32: 18.2 us, 3.6 TB/s, 21 instructions an element; one row of
// 32000: 7.0 us, a chain of five memory latencies and two barriers.
constexpr int kVerifyMaxCtas = 8;
constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyBatch = 16;  // elements a lane loads at once
// Elements of a warp between two additions in 64 bits: 64 a lane, so that the second
// word, which is a plain fp32 sum, stays right to about 2^-47 of the sum; over the 1024
// that a lane takes of a row of 2^22 it was right to 2^-37 (ones with thirds of 2^-25
// behind them).  Rows of 200000 take as long either way (96 of them 36.0 us).
constexpr int kVerifyFold = 4 * 32 * kVerifyBatch;

__device__ __forceinline__ float as_prob(float x) { return x; }
__device__ __forceinline__ float as_prob(__nv_bfloat16 x) { return __bfloat162float(x); }

// kVerifyBatch elements a lane of [i0, hi): element 32 * VEC * k + VEC * lane + e
// in x[VEC * k + e]; zeros behind hi.  VEC elements are one 16-byte load.
// (Rows of an odd length in bf16, 128 x 7 drafts over 50257: 18.4 us; cut out of two
// aligned vectors instead of 2-byte loads they took 21.6 where these took 19.2.)
template <typename Elem, int VEC>
__device__ __forceinline__ void load_batch(const Elem* p, int i0, int hi, float (&x)[kVerifyBatch]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < kVerifyBatch / VEC; ++k) {
        const int i = i0 + 32 * VEC * k + VEC * lane;
        if constexpr (VEC == 1) {
            x[k] = i < hi ? as_prob(p[i]) : 0.f;
        } else {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (i < hi) w = *reinterpret_cast<const uint4*>(p + i);
            const Elem* e = reinterpret_cast<const Elem*>(&w);
#pragma unroll
            for (int z = 0; z < VEC; ++z) x[VEC * k + z] = as_prob(e[z]);
        }
    }
}

// a + b = s + e exactly
__device__ __forceinline__ float two_sum(float a, float b, float& e) {
    const float s = __fadd_rn(a, b);
    const float bb = __fsub_rn(s, a);
    e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
    return s;
}

// The weight max(p - q, 0) as two words; NaN counts as zero.
template <bool kRest>
__device__ __forceinline__ float2 weight(float p, float q) {
    if (!kRest) return make_float2(p > 0.f ? p : 0.f, 0.f);
    float e;
    const float d = two_sum(p, -q, e);
    const bool some = d > 0.f;  // d = 0 only where p = q
    return make_float2(some ? d : 0.f, some ? e : 0.f);
}

// This warp's sum over [lo, hi) in every lane, as two words; infinite where fp32 does
// not reach.
template <typename Elem, int VEC, bool kRest>
__device__ __forceinline__ float2 fold_sum(const Elem* p, const Elem* q, int lo, int hi) {
    float s = 0.f, c = 0.f;
    for (int i0 = lo; i0 < hi; i0 += 32 * kVerifyBatch) {
        float a[kVerifyBatch], b[kVerifyBatch] = {};
        load_batch<Elem, VEC>(p, i0, hi, a);
        if (kRest) load_batch<Elem, VEC>(q, i0, hi, b);
#pragma unroll
        for (int k = 0; k < kVerifyBatch; ++k) {
            const float2 w = weight<kRest>(a[k], b[k]);
            float e;
            s = two_sum(s, w.x, e);
            c += e + w.y;
        }
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) {
        float e;
        const float so = __shfl_xor_sync(0xffffffffu, s, k), co = __shfl_xor_sync(0xffffffffu, c, k);
        s = two_sum(s, so, e);
        c += e + co;
    }
    return make_float2(s, c);
}

// The weight max(p - q, 0) in 64 bits; NaN counts as zero.
template <bool kRest>
__device__ __forceinline__ double weight64(float p, float q) {
    const double d = kRest ? (double)p - (double)q : (double)p;
    return d > 0.0 ? d : 0.0;
}

// This warp's sum over [lo, hi) in every lane, in 64 bits: for weights near the largest
// fp32 number, or above it, or infinite.  (Not inlined: registers.)
template <typename Elem, bool kRest>
__device__ __noinline__ double wide_sum(const Elem* p, const Elem* q, int lo, int hi) {
    double s = 0.0;
    for (int i = lo + (int)(threadIdx.x & 31); i < hi; i += 32)
        s += weight64<kRest>(as_prob(p[i]), kRest ? as_prob(q[i]) : 0.f);
    for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    return s;
}

// This warp's sum over [lo, hi) in every lane.
template <typename Elem, int VEC, bool kRest>
__device__ __forceinline__ double share_sum(const Elem* p, const Elem* q, int lo, int hi) {
    auto fold = [&](int i0) {
        const int end = min(i0 + kVerifyFold, hi);
        const float2 x = fold_sum<Elem, VEC, kRest>(p, q, i0, end);
        return x.x < INFINITY ? (double)x.x + (double)x.y : wide_sum<Elem, kRest>(p, q, i0, end);
    };
    double sum = fold(lo);
    for (int i0 = lo + kVerifyFold; i0 < hi; i0 += kVerifyFold) sum += fold(i0);
    return sum;
}

// Running sums of the first n (at most 32) values, lane by lane.
__device__ __forceinline__ double lane_sums(double x, int n) {
    const int lane = threadIdx.x & 31;
    for (int d = 1; d < n; d <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += o;
    }
    return x;
}

// By one warp: the first of n shares whose running sum, from `border`, is above
// `want` (the last one where rounding leaves none); `border` becomes its start.
__device__ __forceinline__ int pick(const double* sums, int n, double want, double& border) {
    const int lane = threadIdx.x & 31;
    const double run = border + lane_sums(lane < n ? sums[lane] : 0.0, n);
    const uint32_t above = __ballot_sync(0xffffffffu, lane < n && run > want);
    const int w = above ? __ffs(above) - 1 : n - 1;
    const double prev = __shfl_sync(0xffffffffu, run, w > 0 ? w - 1 : 0);
    if (w > 0) border = prev;
    return w;
}

// The first index of [lo, hi) whose running sum, from `border`, is above
// `want`, or -1: 32 elements at a time, in order, by one warp.
template <typename Elem, bool kRest>
__device__ __forceinline__ int find(const Elem* p, const Elem* q, int lo, int hi, double border,
                                    double want) {
    const int lane = threadIdx.x & 31;
    for (int i0 = lo; i0 < hi; i0 += 32) {
        const int i = i0 + lane;
        const double w = weight64<kRest>(i < hi ? as_prob(p[i]) : 0.f,
                                         kRest && i < hi ? as_prob(q[i]) : 0.f);
        double cum = w;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const double o = __shfl_up_sync(0xffffffffu, cum, d);
            if (lane >= d) cum += o;
        }
        const uint32_t above = __ballot_sync(0xffffffffu, w > 0.0 && border + cum > want);
        if (above) return i0 + __ffs(above) - 1;
        border += __shfl_sync(0xffffffffu, cum, 31);
    }
    return -1;
}

// The largest index below `hi` with a weight above zero, or -1, by one warp.
template <typename Elem, bool kRest>
__device__ __forceinline__ int newest(const Elem* p, const Elem* q, int hi) {
    const int lane = threadIdx.x & 31;
    for (int i0 = hi; i0 > 0; i0 -= 32) {
        const int i = i0 - 32 + lane;
        const bool some = i >= 0 && weight<kRest>(as_prob(p[i]), kRest ? as_prob(q[i]) : 0.f).x > 0.f;
        const uint32_t any = __ballot_sync(0xffffffffu, some);
        if (any) return i0 - 32 + 31 - __clz(any);
    }
    return -1;
}

struct VerifyShared {
    double cta_sum[2][kVerifyMaxCtas];  // of every CTA of the cluster; of p - q, of p
    double warp_sum[kVerifyWarps];
    double part_sum[kVerifyWarps];
    double border, want;
    int what, share;
    int n, m, bad;
};

// Where the wanted sum falls: no sum above zero, a sum that is not finite, not
// below the total, into this CTA's share, into another's.
enum : int { kNothing, kRefused, kNewest, kHere, kElsewhere };

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The replacement (or the token behind the last draft) from the weights of one
// row; returns false where they have no sum above zero.
template <typename Elem, int VEC, bool kRest>
__device__ __forceinline__ bool sample(VerifyShared& sh, cg::cluster_group& cluster, const Elem* p,
                                       const Elem* q, int V, float u, int32_t* token,
                                       int32_t* dev_status) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    // whole vectors to a share
    const int share = ((V + ctas - 1) / ctas + VEC - 1) / VEC * VEC;
    const int lo = min(rank * share, V), hi = min(lo + share, V);
    const int part = ((hi - lo + kVerifyWarps - 1) / kVerifyWarps + VEC - 1) / VEC * VEC;
    const int wlo = min(lo + warp * part, hi), whi = min(wlo + part, hi);
    const double sum = share_sum<Elem, VEC, kRest>(p, q, wlo, whi);
    if (lane == 0) sh.warp_sum[warp] = sum;
    __syncthreads();
    double* sums = sh.cta_sum[kRest];
    if (warp == 0) {
        const double s = __shfl_sync(
            0xffffffffu, lane_sums(lane < kVerifyWarps ? sh.warp_sum[lane] : 0.0, kVerifyWarps),
            kVerifyWarps - 1);
        if (lane < ctas) *cluster.map_shared_rank(&sums[rank], lane) = s;
    }
    cluster_arrive();
    cluster_wait();
    if (warp == 0) {
        // the same sums, and so the same choice, in every CTA
        const double total =
            __shfl_sync(0xffffffffu, lane_sums(lane < ctas ? sums[lane] : 0.0, ctas), ctas - 1);
        const double want = (double)u * total;
        int what = kElsewhere, w = 0;
        double border = 0.0;
        if (!(total > 0.0)) {
            what = kNothing;
        } else if (!(total < (double)INFINITY)) {
            what = kRefused;
        } else if (!(want < total)) {  // u = 1, or rounding
            what = kNewest;
        } else if (pick(sums, ctas, want, border) == rank) {
            what = kHere;
            w = pick(sh.warp_sum, kVerifyWarps, want, border);
        }
        if (lane == 0) {
            sh.what = what;
            sh.share = w;
            sh.border = border;
            sh.want = want;
        }
    }
    __syncthreads();
    const int what = sh.what;
    if (what == kNothing) return false;
    if (what == kRefused && rank == 0 && tid == 0) {
        *token = -1;
        report(dev_status, KVD_DEV_PROBS);
    }
    if (what == kNewest && rank == 0 && warp == 0) {
        const int v = newest<Elem, kRest>(p, q, V);
        if (lane == 0) *token = v;
    }
    if (what != kHere) return true;
    const int slo = min(lo + sh.share * part, hi), shi = min(slo + part, hi);
    const int sub = ((shi - slo + kVerifyWarps - 1) / kVerifyWarps + VEC - 1) / VEC * VEC;
    const double ps = share_sum<Elem, VEC, kRest>(p, q, min(slo + warp * sub, shi),
                                                  min(slo + (warp + 1) * sub, shi));
    if (lane == 0) sh.part_sum[warp] = ps;
    __syncthreads();
    if (warp == 0) {
        double border = sh.border;
        const double want = sh.want;
        const int z = pick(sh.part_sum, kVerifyWarps, want, border);
        const int plo = min(slo + z * sub, shi), phi = min(plo + sub, shi);
        int v = find<Elem, kRest>(p, q, plo, phi, border, want);
        // rounding between the passes may leave none there
        if (v < 0) v = newest<Elem, kRest>(p, q, phi);
        if (v < 0) v = newest<Elem, kRest>(p, q, V);
        if (lane == 0) *token = v;
    }
    return true;
}

template <typename Elem, int VEC>
__global__ void __launch_bounds__(kVerifyThreads, 2)
verify_drafts_kernel(const Elem* __restrict__ target, const Elem* __restrict__ draft,
                     const int32_t* __restrict__ drafts, const float* __restrict__ u_accept,
                     const float* __restrict__ u_sample, const int32_t* __restrict__ num_drafts,
                     int32_t* __restrict__ tokens, int32_t* __restrict__ accepted, int T, int V,
                     int32_t* dev_status) {
    __shared__ VerifyShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    cluster_arrive();  // waited for before the first write into another CTA
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / (int)cluster.num_blocks();
    const bool lead = cluster.block_rank() == 0;
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
                const float u = u_accept[(size_t)b * T + i];
                in = x >= 0 && x < V;
                ok = in && (double)u * (double)as_prob(draft[((size_t)b * T + i) * V + x]) <
                               (double)as_prob(target[((size_t)b * (T + 1) + i) * V + x]);
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
    cluster_wait();
    const int n = sh.n;
    if (lead) {
        for (int i = tid; i <= T; i += kVerifyThreads)
            if (i != n || sh.bad)
                tokens[(size_t)b * (T + 1) + i] = i < n ? drafts[(size_t)b * T + i] : -1;
        if (tid == 0) accepted[b] = n;
    }
    if (!sh.bad) {
        const Elem* p = target + ((size_t)b * (T + 1) + n) * V;
        const Elem* q = draft + ((size_t)b * T + n) * V;
        const float u = u_sample[b];
        int32_t* token = tokens + (size_t)b * (T + 1) + n;
        bool done = false;
        if (n < sh.m) done = sample<Elem, VEC, true>(sh, cluster, p, q, V, u, token, dev_status);
        // behind the last draft, or nothing of the target left: the target itself
        if (!done) done = sample<Elem, VEC, false>(sh, cluster, p, q, V, u, token, dev_status);
        if (!done && lead && tid == 0) {
            *token = -1;
            report(dev_status, KVD_DEV_PROBS);
        }
    }
}

template <typename Elem, int VEC>
cudaError_t go_verify(const Elem* target, const Elem* draft, const int32_t* drafts,
                      const float* u_accept, const float* u_sample, const int32_t* num_drafts,
                      int32_t* tokens, int32_t* accepted, int Q, int T, int V, int32_t* dev_status,
                      cudaStream_t stream) {
    // CTAs a sequence: while two CTAs an SM are not passed; shares of at least
    // half a batch a warp
    int ctas = 1;
    while (ctas < kVerifyMaxCtas && 2 * ctas * Q <= 2 * kLatentSMs &&
           V / (2 * ctas) >= 8 * 32 * kVerifyWarps)
        ctas *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(Q * ctas);
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify_drafts_kernel<Elem, VEC>, target, draft, drafts, u_accept,
                              u_sample, num_drafts, tokens, accepted, T, V, dev_status);
}

template <typename Elem>
cudaError_t go_verify(const void* target, const void* draft, const int32_t* drafts,
                      const float* u_accept, const float* u_sample, const int32_t* num_drafts,
                      int32_t* tokens, int32_t* accepted, int Q, int T, int V, int32_t* dev_status,
                      cudaStream_t stream) {
    constexpr int kVec = 16 / (int)sizeof(Elem);
    const Elem* p = static_cast<const Elem*>(target);
    const Elem* q = static_cast<const Elem*>(draft);
    // 16-byte loads where every row starts on a 16-byte boundary
    const bool vec = V % kVec == 0 && reinterpret_cast<uintptr_t>(target) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(draft) % 16 == 0;
    return vec ? go_verify<Elem, kVec>(p, q, drafts, u_accept, u_sample, num_drafts, tokens,
                                       accepted, Q, T, V, dev_status, stream)
               : go_verify<Elem, 1>(p, q, drafts, u_accept, u_sample, num_drafts, tokens, accepted,
                                    Q, T, V, dev_status, stream);
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
    return dt == KVD_BF16
               ? go_verify<__nv_bfloat16>(target, draft, drafts, u_accept, u_sample, num_drafts,
                                          tokens, accepted, Q, T, V, dev_status, stream)
               : go_verify<float>(target, draft, drafts, u_accept, u_sample, num_drafts, tokens,
                                  accepted, Q, T, V, dev_status, stream);
}

}  // namespace kvd
