// plan_pages.cu -- kvd_plan_pages: pages, slots and positions of a step's new tokens
// from the requests' lengths.
//
// One cluster does the whole call, because three things have to follow one another
// over all sequences: pages given back enter the free list, pages are taken from its
// end, and tokens look up the tables that result.  A cluster barrier orders these in
// a microsecond; every CTA scans all sequences by itself (1024 at a time) instead of
// exchanging sums, and the CTAs share the pages and the tokens out by index, so that
// one sequence of many pages takes no longer than many of one page.
//
// Up to 1024 sequences take a kernel of their own: a thread a sequence, whose lengths are
// loaded once, two scans, pages straight from the list into the tables, and tokens from
// what shared memory holds; many tokens are looked up in a second launch by the whole GPU.
//
// It is latency alone: launch, lengths, scans, list, tables, tokens, a memory access each.
// With the call that gives the pages back, 64 sequences of one new token take 7.7 us (16.6 in
// the general kernel), 1024 of up to 127 16.0 (33).
#include <cooperative_groups.h>

#include "../kvd_internal.h"
#include "../latent/latent_common.cuh"  // FastDiv
#include "serving_common.cuh"

namespace kvd {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;
constexpr int kTokensApart = 16384;
constexpr int kPlanBatch = 4;  // tokens that a thread looks up at once

struct PlanShared {
    long long warp_sum[kWarps];
    int end[kThreads];    // of this chunk: pages up to and with a sequence's own
    int held[kThreads];
};

// Inclusive sums over the CTA; `total` is the last one.
__device__ __forceinline__ long long block_sums(PlanShared& sh, long long x, long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += o;
    }
    __syncthreads();
    if (lane == 31) sh.warp_sum[warp] = x;
    __syncthreads();
    long long s = sh.warp_sum[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += o;
    }
    total = __shfl_sync(0xffffffffu, s, 31);
    const long long before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
    return x + (warp > 0 ? before : 0);
}

// The sequence of the chunk that page i belongs to.
__device__ __forceinline__ int chunk_find(const PlanShared& sh, long long i) {
    int lo = 0, hi = kThreads - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sh.end[mid] > i)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// What a sequence has and wants.
struct PlanSeq {
    int kept, n, held, need;  // tokens, tokens, pages, pages
    bool good;
};

// (`lens`: new_lens is in order.)
__device__ __forceinline__ PlanSeq plan_seq(const PlanArgs& a, int q, bool lens, uint32_t& bits) {
    PlanSeq s{0, 0, 0, 0, false};
    if (q >= a.Q) return s;
    const int s0 = lens ? a.new_lens[q] : 0, s1 = lens ? a.new_lens[q + 1] : 0;
    const int kept = a.kept_lens[q], held = a.pages_held[q];
    const long long total = (long long)kept + (s1 - s0);
    if (kept < 0 || held < 0 || held > a.cols || kept > (long long)held * a.BS ||
        total > 0x7fffffffll) {
        bits |= KVD_DEV_POS_RANGE;
        return s;
    }
    s.kept = kept;
    s.n = s1 - s0;
    s.held = held;
    s.need = (int)((total + a.BS - 1) / a.BS);
    s.good = true;
    return s;
}

__global__ void __launch_bounds__(kThreads) plan_pages_kernel(const PlanArgs a) {
    __shared__ PlanShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, rank = (int)cluster.block_rank(),
              ctas = (int)cluster.num_blocks();
    const int all = ctas * kThreads, me = rank * kThreads + tid;
    const bool lead = rank == 0;
    uint32_t bits = 0;
    int count = a.free_count[0];
    bool lens_ok = true;
    for (int q = tid; q < a.Q; q += kThreads) {
        const int s0 = a.new_lens[q], s1 = a.new_lens[q + 1];
        lens_ok &= (q > 0 || s0 == 0) && s1 >= s0 && s1 <= a.N;
    }
    lens_ok = __syncthreads_and(lens_ok);
    // what refuses every sequence
    const bool usable = lens_ok && count >= 0 && count <= a.F;
    if (!lens_ok) bits |= KVD_DEV_SEQLENS;
    if (count < 0 || count > a.F) bits |= KVD_DEV_POS_RANGE;

    // pages given back: all, or none where the list has no room for all
    long long given = 0;
    for (int q0 = 0; usable && q0 < a.Q; q0 += kThreads) {
        const PlanSeq s = plan_seq(a, q0 + tid, true, bits);
        long long t;
        block_sums(sh, s.good && s.held > s.need ? s.held - s.need : 0, t);
        given += t;
    }
    const bool give_back = usable && given <= a.F - count;
    if (usable && !give_back) bits |= KVD_DEV_NO_PAGES;
    if (given > 0 && give_back) {
        long long before = 0;  // by the sequences before this chunk
        for (int q0 = 0; q0 < a.Q; q0 += kThreads) {
            const PlanSeq s = plan_seq(a, q0 + tid, true, bits);
            long long t;
            const long long end = block_sums(sh, s.good && s.held > s.need ? s.held - s.need : 0, t);
            sh.end[tid] = (int)end;
            sh.held[tid] = s.held;
            __syncthreads();
            // the last sequence's last page goes first: page i of the chunk (columns
            // rising) lies behind all pages after it
            const long long base = count + (given - before - t);
            for (long long i = me; i < t; i += all) {
                const int k = chunk_find(sh, i);
                a.free_pages[base + t - 1 - i] =
                    a.block_tables[(size_t)(q0 + k) * a.cols + sh.held[k] - (int)(sh.end[k] - i)];
            }
            before += t;
            __syncthreads();
        }
    }
    cluster.sync();  // the list is whole

    const long long avail = usable ? count + (give_back ? given : 0) : 0;
    // by the sequences before this chunk; asked: tokens of refused ones among them
    long long wanted = 0, taken = 0, asked = 0, tokens = 0;
    for (int q0 = 0; q0 < a.Q; q0 += kThreads) {
        const int q = q0 + tid;
        const PlanSeq s = plan_seq(a, q, lens_ok, bits);
        int grow = usable && s.good && s.need > s.held ? s.need - s.held : 0;
        bool served = s.good && usable;
        if (grow > 0 && s.need > a.cols) {
            bits |= KVD_DEV_TABLE_COLS;
            grow = 0;
            served = false;
        }
        long long t, lens;
        const long long run = block_sums(sh, grow, t) + wanted;
        wanted += t;
        if (grow > 0 && run > avail) {
            bits |= KVD_DEV_NO_PAGES;
            grow = 0;
            served = false;
        }
        int len = s.kept + (served ? s.n : 0);
        const long long at = block_sums(sh, len, lens) + asked;
        long long end = at;
        asked += lens;
        if (__syncthreads_or(at > 0x7fffffffll)) {  // lengths that 32 bits do not hold
            if (at > 0x7fffffffll && len > 0) {
                bits |= KVD_DEV_SEQLENS;
                len = grow = 0;
            }
            end = block_sums(sh, len, lens) + tokens;
        }
        if (lead && q < a.Q) a.seq_lens[q + 1] = (int)end;
        long long takes;
        const long long mine = block_sums(sh, grow, takes);
        sh.end[tid] = (int)mine;
        sh.held[tid] = s.held;
        __syncthreads();
        for (long long i = me; i < takes; i += all) {
            const int k = chunk_find(sh, i), before = k > 0 ? sh.end[k - 1] : 0;
            a.block_tables[(size_t)(q0 + k) * a.cols + sh.held[k] + (int)(i - before)] =
                a.free_pages[avail - 1 - taken - i];
        }
        taken += takes;
        tokens += lens;
        __syncthreads();
    }
    if (lead && tid == 0) a.seq_lens[0] = 0;
    cluster.sync();  // tables and lengths are whole; nobody reads held pages or the count again

    if (lead && tid == 0 && usable) a.free_count[0] = (int)(avail - taken);
    // pages held, by the thread that reads them
    for (int q = me; usable && q < a.Q; q += all) {
        uint32_t none = 0;
        const PlanSeq s = plan_seq(a, q, true, none);
        const int len = a.seq_lens[q + 1] - a.seq_lens[q];
        if (!s.good) continue;
        // what went onto the list is no longer held, whether or not the tokens have a place
        if (s.need < s.held ? give_back : s.need > s.held && len == s.kept + s.n)
            a.pages_held[q] = s.need;
    }
    for (int i = me; i < a.N; i += all) {
        int lo = usable ? 0 : a.Q, hi = a.Q;  // the first sequence that ends behind i
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (a.new_lens[mid + 1] > i)
                hi = mid;
            else
                lo = mid + 1;
        }
        int slot = -1, pos = -1;
        if (lo < a.Q) {
            const int s0 = a.new_lens[lo], n = a.new_lens[lo + 1] - s0, kept = a.kept_lens[lo];
            const int len = a.seq_lens[lo + 1] - a.seq_lens[lo];
            // refused ones are shorter than that
            if (kept >= 0 && len == (long long)kept + n) {
                const int t = kept + (i - s0);
                const long long p = (long long)t + (a.pos_base ? a.pos_base[lo] : 0);
                const int page = a.block_tables[(size_t)lo * a.cols + t / a.BS];
                const long long at = (long long)page * a.BS + t % a.BS;
                if (page < 0 || at > 0x7fffffffll) {
                    bits |= KVD_DEV_BLOCK_RANGE;
                } else if (p < 0 || p > 0x7fffffffll) {
                    bits |= KVD_DEV_POS_RANGE;
                } else {
                    slot = (int)at;
                    pos = (int)p;
                }
            }
        }
        a.slots[i] = slot;
        a.positions[i] = pos;
    }
    if (bits) report(a.dev_status, bits);
}

// ------------------------------------------------------------ up to 1024 sequences

template <int THREADS>
struct OneShared {
    longlong2 warp_sum[2][THREADS / 32];
    int start[THREADS + 1];  // first new token
    int kept[THREADS];       // -1: no place for the new tokens
    int base[THREADS];
    int held[THREADS];
    int end[THREADS];        // pages taken (given back) up to and with a sequence's own
};

// Inclusive sums of two numbers over the CTA; one barrier (`turn`: alternating).
template <int THREADS>
__device__ __forceinline__ longlong2 two_sums(OneShared<THREADS>& sh, int turn, long long x, long long y,
                                              longlong2& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, x, d), b = __shfl_up_sync(0xffffffffu, y, d);
        if (lane >= d) {
            x += a;
            y += b;
        }
    }
    if (lane == 31) sh.warp_sum[turn][warp] = make_longlong2(x, y);
    __syncthreads();
    constexpr int W = THREADS / 32;
    longlong2 s = lane < W ? sh.warp_sum[turn][lane] : make_longlong2(0, 0);
#pragma unroll
    for (int d = 1; d < W; d <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, s.x, d), b = __shfl_up_sync(0xffffffffu, s.y, d);
        if (lane >= d) {
            s.x += a;
            s.y += b;
        }
    }
    total = make_longlong2(__shfl_sync(0xffffffffu, s.x, W - 1), __shfl_sync(0xffffffffu, s.y, W - 1));
    const int from = warp > 0 ? warp - 1 : 0;
    const long long bx = __shfl_sync(0xffffffffu, s.x, from), by = __shfl_sync(0xffffffffu, s.y, from);
    return make_longlong2(x + (warp > 0 ? bx : 0), y + (warp > 0 ? by : 0));
}

// The first of n ascending numbers that is above i.
__device__ __forceinline__ int first_above(const int* x, int n, int i) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (x[mid] > i)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1) plan_one_kernel(const PlanArgs a, const FastDiv by_page,
                                                              const bool tokens) {
    __shared__ OneShared<THREADS> sh;
    cg::cluster_group cluster = cg::this_cluster();
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, rank = (int)cluster.block_rank(),
              ctas = (int)cluster.num_blocks();
    const int all = ctas * THREADS, me = rank * THREADS + tid;
    const bool lead = rank == 0;
    uint32_t bits = 0;
    const int count = a.free_count[0];
    const bool list_ok = count >= 0 && count <= a.F;
    bool lens_ok = true;
    if (tid < a.Q) {
        const int s0 = a.new_lens[tid], s1 = a.new_lens[tid + 1];
        lens_ok = (tid > 0 || s0 == 0) && s1 >= s0 && s1 <= a.N;
        sh.start[tid + 1] = s1;
        sh.base[tid] = a.pos_base ? a.pos_base[tid] : 0;
    }
    if (tid == 0) sh.start[0] = 0;
    PlanSeq s = plan_seq(a, tid, true, bits);
    lens_ok = __syncthreads_and(lens_ok);
    const bool usable = lens_ok && list_ok;
    if (!lens_ok) {
        bits = KVD_DEV_SEQLENS;
        s = plan_seq(a, tid, false, bits);
    }
    if (!list_ok) bits |= KVD_DEV_POS_RANGE;
    const int give = usable && s.good && s.held > s.need ? s.held - s.need : 0;
    int grow = usable && s.good && s.need > s.held ? s.need - s.held : 0;
    bool served = s.good && usable;
    if (grow > 0 && s.need > a.cols) {
        bits |= KVD_DEV_TABLE_COLS;
        grow = 0;
        served = false;
    }
    sh.held[tid] = s.held;
    longlong2 total;
    const longlong2 run = two_sums(sh, 0, give, grow, total);
    const long long given = total.x;
    const bool give_back = usable && given <= a.F - count;
    if (usable && !give_back) bits |= KVD_DEV_NO_PAGES;
    if (given > 0 && give_back) {
        sh.end[tid] = (int)run.x;
        __syncthreads();
        for (int i = me; i < (int)given; i += all) {
            const int k = first_above(sh.end, THREADS - 1, i);
            a.free_pages[count + given - 1 - i] =
                a.block_tables[(size_t)k * a.cols + sh.held[k] - (sh.end[k] - i)];
        }
        cluster.sync();  // the list is whole
    }
    const long long avail = usable ? count + (give_back ? given : 0) : 0;
    if (grow > 0 && run.y > avail) {
        bits |= KVD_DEV_NO_PAGES;
        grow = 0;
        served = false;
    }
    int len = s.kept + (served ? s.n : 0);
    longlong2 end = two_sums(sh, 1, len, grow, total);
    if (__syncthreads_or(end.x > 0x7fffffffll)) {  // lengths that 32 bits do not hold
        if (end.x > 0x7fffffffll && len > 0) {
            bits |= KVD_DEV_SEQLENS;
            len = grow = 0;
            served = false;
        }
        end = two_sums(sh, 0, len, grow, total);
    }
    // everything that this call changes in place has been read, but for the tables
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (lead && tid < a.Q) a.seq_lens[tid + 1] = (int)end.x;
    if (lead && tid == 0) a.seq_lens[0] = 0;
    const int taken = (int)total.y;
    sh.end[tid] = (int)end.y;
    sh.kept[tid] = served ? s.kept : -1;
    __syncthreads();
    const int32_t* list = a.free_pages + avail - 1;  // page i taken: list[-i]
    for (int i = me; i < taken; i += all) {
        const int k = first_above(sh.end, THREADS - 1, i), before = k > 0 ? sh.end[k - 1] : 0;
        a.block_tables[(size_t)k * a.cols + sh.held[k] + i - before] = list[-i];
    }
    for (int i0 = me; i0 < (tokens ? a.N : 0); i0 += kPlanBatch * all) {
        int seq[kPlanBatch], t[kPlanBatch], page[kPlanBatch];
#pragma unroll
        for (int k = 0; k < kPlanBatch; ++k) {
            const int i = i0 + k * all;
            const int q = i < a.N && usable ? first_above(sh.start + 1, a.Q, i) : a.Q;
            const int kept = q < a.Q ? sh.kept[q] : -1;
            seq[k] = q;
            t[k] = kept < 0 ? -1 : kept + i - sh.start[q];
            page[k] = -1;
            if (t[k] >= 0) {
                const int col = by_page(t[k]), own = col - sh.held[q];
                page[k] = own < 0 ? a.block_tables[(size_t)q * a.cols + col]
                                  : list[-((q > 0 ? sh.end[q - 1] : 0) + own)];
            }
        }
#pragma unroll
        for (int k = 0; k < kPlanBatch; ++k) {
            const int i = i0 + k * all;
            if (i >= a.N) continue;
            int slot = -1, pos = -1;
            if (t[k] >= 0) {
                const long long p = (long long)t[k] + sh.base[seq[k]];
                const long long at = (long long)page[k] * a.BS + t[k] - by_page(t[k]) * a.BS;
                if (page[k] < 0 || at > 0x7fffffffll) {
                    bits |= KVD_DEV_BLOCK_RANGE;
                } else if (p < 0 || p > 0x7fffffffll) {
                    bits |= KVD_DEV_POS_RANGE;
                } else {
                    slot = (int)at;
                    pos = (int)p;
                }
            }
            a.slots[i] = slot;
            a.positions[i] = pos;
        }
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (lead && usable) {
        if (tid == 0) a.free_count[0] = (int)(avail - taken);
        // what went onto the list is no longer held, whether or not the tokens have a place
        if (tid < a.Q && s.good && (s.need < s.held ? give_back : s.need > s.held && served))
            a.pages_held[tid] = s.need;
    }
    if (bits) report(a.dev_status, bits);
}

// Slots and positions of many tokens, behind the kernel that made tables and lengths.
__global__ void __launch_bounds__(256) plan_tokens_kernel(const PlanArgs a, const FastDiv by_page) {
    pdl_launch_dependents();
    pdl_wait();
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= a.N) return;
    int slot = -1, pos = -1;
    const int q = first_above(a.new_lens + 1, a.Q, i);
    if (q < a.Q) {
        // (lengths out of order leave no sequence longer than it was)
        const int s0 = a.new_lens[q], n = a.new_lens[q + 1] - s0, kept = a.kept_lens[q];
        const int len = a.seq_lens[q + 1] - a.seq_lens[q];
        if (s0 >= 0 && i >= s0 && n > 0 && kept >= 0 && len == (long long)kept + n) {
            const int t = kept + (i - s0), col = by_page(t);
            const long long p = (long long)t + (a.pos_base ? a.pos_base[q] : 0);
            const int page = col < a.cols ? a.block_tables[(size_t)q * a.cols + col] : -1;
            const long long at = (long long)page * a.BS + t - col * a.BS;
            if (page < 0 || at > 0x7fffffffll) {
                report(a.dev_status, KVD_DEV_BLOCK_RANGE);
            } else if (p < 0 || p > 0x7fffffffll) {
                report(a.dev_status, KVD_DEV_POS_RANGE);
            } else {
                slot = (int)at;
                pos = (int)p;
            }
        }
    }
    a.slots[i] = slot;
    a.positions[i] = pos;
}

}  // namespace

cudaError_t launch_plan_pages(const PlanArgs& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    // few sequences and tokens: one small CTA (64 x 1, taken and given back: 11.7 -> 7.7 us);
    // one CTA while a thread has at most one sequence and two tokens
    const bool small = a.Q <= 256 && a.N <= 512;
    const int ctas = small || (a.Q <= kThreads && a.N <= 2 * kThreads) ? 1 : kMaxCtas;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(small ? 256 : kThreads);
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
    if (a.Q > kThreads) return cudaLaunchKernelEx(&cfg, plan_pages_kernel, a);
    // many tokens: by the whole GPU, in a launch of their own (with the call that gives the
    // pages back: 1024 x 64 tokens 20.6 -> 16.3 us, 1024 x 32 15.7 -> 14.7)
    const bool apart = a.N > kTokensApart;
    const cudaError_t e = cudaLaunchKernelEx(
        &cfg, small ? plan_one_kernel<256> : plan_one_kernel<kThreads>, a, FastDiv(a.BS), !apart);
    if (e != cudaSuccess || !apart) return e;
    return launch_pdl(plan_tokens_kernel, dim3((a.N + 255) / 256), dim3(256), 0, stream, a,
                      FastDiv(a.BS));
}

}  // namespace kvd
