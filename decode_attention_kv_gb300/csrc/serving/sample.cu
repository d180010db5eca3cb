// sample.cu -- kvd_sample and kvd_filter_probs.
//
// w_v = exp((l_v - max) / T).  In falling order of l (ties by index) temperature,
// top-k, top-p and min-p each keep a beginning of the row, so what is kept is a
// smallest logit and, where equal logits are cut, a last index.
#include "../kvd_internal.h"
#include "serving_common.cuh"

namespace kvd {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;

__device__ __forceinline__ float as_logit(float x) { return x; }
__device__ __forceinline__ float as_logit(__nv_bfloat16 x) { return __bfloat162float(x); }

// A number that rises with the logit; NaN counts as the lowest.
__device__ __forceinline__ uint32_t order_of(float x) {
    if (!(x == x)) return 0x007fffffu;  // that of -inf
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ double weight_of(float x, float top, double inv_t) {
    if (x == top) return 1.0;
    return exp(((double)x - (double)top) * inv_t);
}
constexpr double kOne = 8796093022208.0;  // 2^43: weights as whole numbers, summed in any order
__device__ __forceinline__ unsigned long long fixed_of(double w) {
    return (unsigned long long)(w * kOne + 0.5);
}

struct SampleShared {
    unsigned long long mass[256];
    unsigned int count[256];
    unsigned long long warp_sum[kWarps];
    uint32_t warp_max[kWarps];
    unsigned long long carry;
    uint32_t prefix;
    unsigned int left;
    int found;
};

__device__ __forceinline__ unsigned long long block_sum(SampleShared& sh, unsigned long long x) {
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.warp_sum[threadIdx.x >> 5] = x;
    __syncthreads();
    x = sh.warp_sum[threadIdx.x & 31];
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// Exclusive sums in thread order.
__device__ __forceinline__ unsigned long long block_before(SampleShared& sh, unsigned long long x,
                                                           unsigned long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long inc = x;
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
    }
    __syncthreads();
    if (lane == 31) sh.warp_sum[warp] = inc;
    __syncthreads();
    unsigned long long s = sh.warp_sum[lane];
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long o = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += o;
    }
    total = __shfl_sync(0xffffffffu, s, 31);
    const unsigned long long before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
    return inc - x + (warp > 0 ? before : 0);
}

template <typename Elem>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
    __shared__ SampleShared sh;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, row = blockIdx.x, V = a.V;
    const Elem* l = static_cast<const Elem*>(a.logits) + (size_t)row * V;
    auto put = [&](int i, float p) {
        if (a.probs_bf16)
            static_cast<__nv_bfloat16*>(a.probs)[(size_t)row * V + i] = __float2bfloat16_rn(p);
        else
            static_cast<float*>(a.probs)[(size_t)row * V + i] = p;
    };
    uint32_t top = 0;
    for (int i = tid; i < V; i += kThreads) top = max(top, order_of(as_logit(l[i])));
    top = __reduce_max_sync(0xffffffffu, top);
    if ((tid & 31) == 0) sh.warp_max[tid >> 5] = top;
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, sh.warp_max[tid & 31]);
    const float best = logit_of(top);
    const float T = a.temperature ? a.temperature[row] : 1.f;
    const float p = a.top_p ? a.top_p[row] : 1.f, mp = a.min_p ? fminf(a.min_p[row], 1.f) : 0.f;
    const float u = a.u ? a.u[row] : 0.f;
    const bool params = T >= 0.f && T < INFINITY && p == p &&
                        !(a.min_p && a.min_p[row] != a.min_p[row]) && u >= 0.f && u < 1.f;
    if (!params || best == -INFINITY) {
        if (tid == 0) report(a.dev_status, params ? KVD_DEV_PROBS : KVD_DEV_PARAM);
        if (a.tokens) {
            if (tid == 0) a.tokens[row] = -1;
        } else {
            for (int i = tid; i < V; i += kThreads) put(i, 0.f);
        }
        return;
    }
    const double inv_t = 1.0 / (double)T;
    const bool greedy = T == 0.f;
    uint32_t cut = 0;              // smallest order that is kept
    unsigned int ties = 0xffffffffu;  // how many of that order
    auto counts = [&](uint32_t k) { return k >= cut; };
    // top-k: the k-th largest, eight bits at a time
    const int k = greedy ? 1 : a.top_k ? a.top_k[row] : 0;
    if (k > 0 && k < V) {
        uint32_t prefix = 0;
        unsigned int left = k;
        for (int shift = 24; shift >= 0; shift -= 8) {
            __syncthreads();
            if (tid < 256) sh.count[tid] = 0;
            __syncthreads();
            for (int i = tid; i < V; i += kThreads) {
                const uint32_t o = order_of(as_logit(l[i]));
                if (shift == 24 || (o >> (shift + 8)) == prefix)
                    atomicAdd(&sh.count[(o >> shift) & 255u], 1u);
            }
            __syncthreads();
            if (tid == 0) {
                int b = 255;
                while (sh.count[b] < left) left -= sh.count[b--];
                sh.prefix = prefix << 8 | (uint32_t)b;
                sh.left = left;
            }
            __syncthreads();
            prefix = sh.prefix;
            left = sh.left;
        }
        cut = prefix;
        ties = left;
    }
    if (!greedy && p < 1.f) {
        // the sum of the first k; equal logits at the cut count as often as they are kept
        unsigned long long sum = 0;
        for (int i = tid; i < V; i += kThreads) {
            const float x = as_logit(l[i]);
            if (order_of(x) > cut) sum += fixed_of(weight_of(x, best, inv_t));
        }
        const unsigned long long at_cut =
            cut ? ties * fixed_of(weight_of(logit_of(cut), best, inv_t)) : 0;
        const unsigned long long total = block_sum(sh, sum) + at_cut;
        double want = ceil((double)p * (double)total);
        unsigned long long left = want < 1.0 ? 1ull : (unsigned long long)want;
        uint32_t prefix = 0;
        const uint32_t kcut = cut;
        for (int shift = 24; shift >= 0; shift -= 8) {
            __syncthreads();
            if (tid < 256) sh.mass[tid] = 0;
            __syncthreads();
            for (int i = tid; i < V; i += kThreads) {
                const float x = as_logit(l[i]);
                const uint32_t o = order_of(x);
                if (o > kcut && (shift == 24 || (o >> (shift + 8)) == prefix))
                    atomicAdd(&sh.mass[(o >> shift) & 255u], fixed_of(weight_of(x, best, inv_t)));
            }
            if (tid == 0 && kcut && (shift == 24 || (kcut >> (shift + 8)) == prefix))
                atomicAdd(&sh.mass[(kcut >> shift) & 255u], at_cut);
            __syncthreads();
            if (tid == 0) {
                int b = 255;
                while (b > 0 && sh.mass[b] < left) left -= sh.mass[b--];
                sh.prefix = prefix << 8 | (uint32_t)b;
                sh.carry = left;
            }
            __syncthreads();
            prefix = sh.prefix;
            left = sh.carry;
        }
        const unsigned long long each = fixed_of(weight_of(logit_of(prefix), best, inv_t));
        const unsigned long long some = each ? (left + each - 1) / each : 0xffffffffull;
        if (prefix > kcut)
            ties = (unsigned int)min(some, 0xffffffffull);
        else
            ties = (unsigned int)min(some, (unsigned long long)ties);
        cut = prefix;
    }
    // the last index of the cut's ties, if not all are kept
    int last = V;
    if (ties != 0xffffffffu) {
        unsigned long long before = 0;
        if (tid == 0) sh.found = V;
        for (int i0 = 0; i0 < V; i0 += kThreads) {
            const int i = i0 + tid;
            const unsigned long long is = i < V && order_of(as_logit(l[i])) == cut;
            unsigned long long t;
            const unsigned long long at = block_before(sh, is, t) + before;
            if (is && at + 1 == ties) sh.found = i;
            before += t;
        }
        __syncthreads();
        last = sh.found;
    }
    auto weight = [&](int i) {
        const float x = as_logit(l[i]);
        const uint32_t o = order_of(x);
        if (o < cut || (o == cut && i > last) || (x != x)) return 0.0;
        const double w = weight_of(x, best, inv_t);
        return w >= (double)mp ? w : 0.0;
    };
    unsigned long long sum = 0;
    for (int i = tid; i < V; i += kThreads) sum += fixed_of(weight(i));
    sum = block_sum(sh, sum);
    if (!a.tokens) {
        const double inv = kOne / (double)sum;
        for (int i = tid; i < V; i += kThreads) put(i, (float)(weight(i) * inv));
        return;
    }
    const unsigned long long want = (unsigned long long)((double)u * (double)sum);
    unsigned long long before = 0;
    __syncthreads();
    if (tid == 0) sh.found = -1;
    for (int i0 = 0; i0 < V; i0 += kThreads) {
        const int i = i0 + tid;
        const unsigned long long w = i < V ? fixed_of(weight(i)) : 0;
        unsigned long long t;
        const unsigned long long at = block_before(sh, w, t) + before;
        if (w > 0 && at <= want && at + w > want) sh.found = i;
        before += t;
        if (before > want) break;
    }
    __syncthreads();
    if (tid == 0) a.tokens[row] = sh.found;
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, kvd_dtype dt, cudaStream_t stream) {
    return dt == KVD_BF16
               ? launch_pdl(sample_kernel<__nv_bfloat16>, dim3(a.R), dim3(kThreads), 0, stream, a)
               : launch_pdl(sample_kernel<float>, dim3(a.R), dim3(kThreads), 0, stream, a);
}

}  // namespace kvd
