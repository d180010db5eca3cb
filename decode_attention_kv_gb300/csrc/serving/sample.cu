// sample.cu -- kvd_sample and kvd_filter_probs.
//
// w_v = exp((l_v - max) / T).  In falling order of l (ties by index) temperature,
// top-k, top-p and min-p each keep a beginning of the row, so what is kept is a cut: a
// smallest logit and, among those equal to it, a last index.
//
// A cluster of 1 to 8 CTAs takes a row, a contiguous share a CTA and of that a warp; the
// row comes from memory once and is read again from L2.
//   First pass: the largest logit, and with top-k a histogram of the logits' orders.  The
//   bins that hold the first k go to the first CTA, which sorts them, takes both cuts and
//   draws.
//   Without top-k, second pass (top-p): counts by distance from the largest logit, which
//   bracket the border (to a hundred elements or so) and tell whether min-p cuts well
//   before it.  Third pass: exact sums, of what min-p keeps where that decides alone, else
//   of the row and of what lies above the bracket; the bracket's elements go to the first
//   CTA, which sorts them and takes the cut.  The draw then reads again only the part of
//   one warp.
//   Where a list does not hold what it should (flat rows, ties, large k), the row is
//   divided into 512 bins of exact counts or weights, the bin of the border again, and so
//   on by the orders' bits, until a list takes it or one value is left, whose ties are
//   counted through in index order.
//
// Whole numbers decide, so sums must not depend on an order and have to agree with sums
// in 64 bits: a weight is a table's sixteenth of a factor of two times a polynomial, right
// to about 2^-28 of itself without a trend, and is counted in whole multiples of 2^-42 (sums of
// 2^20 of them fit 64 bits).  A flat tail is off by up to half a multiple a token, all to one
// side: 2^-23 of the largest weight for 2^20 tokens; below half a multiple nothing of it counts.
//
// Measured: a row of 32000 with all filters 10.3 us, 64 rows of 128000 46.2 (their bytes 4.8).
// In cycles of a row there, four CTAs to a row and two an SM: first pass 10000 (the bytes), with
// top-k's counts 16000; top-k then 5000 to 8000 for the list, 7000 for its way and sort,
// 10000 for both cuts and the draw: 48000 to 55000 in all.  Without top-k a count pass of 15000,
// the bracket 8000, the exact sums 23000 (38 instructions an element) where min-p does not
// decide (7000 where it does), 10000 for the border: 80000, which is what the call waits
// for.  No unit is full (issue slots 42 %): barriers of the cluster, sorts and code that is
// run once take the rest.  Not kept: bins only above a weight of (1 - p) / V with the rest
// added up as numbers (16000 for the count pass: the branch costs what the atomic does),
// exact sums on pairs of fp32 (spills: 21000 to 36000).
#include <cooperative_groups.h>

#include <cmath>
#include <cstring>

#include "../kvd_internal.h"
#include "serving_common.cuh"

namespace kvd {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;
constexpr int kBins = kThreads;  // a thread a bin when they are added up
// Bits of an order that its bin of the first pass leaves out: eight bins a factor of two
// (finer ones take longer to clear and to add up, and a list holds 2048 elements).
constexpr int kOrderShift = 20, kOrders = 1 << (32 - kOrderShift);
constexpr int kFine = 2048;      // bins of the second pass
constexpr int kList = 2048;      // elements that one CTA sorts
constexpr int kBatch = 16;       // elements that a lane loads at once
constexpr unsigned long long kOne = 1ull << 42;  // the weight 1
constexpr float kMagic = 12582912.f;             // 1.5 * 2^23: adding it rounds to whole numbers

__device__ __forceinline__ float as_logit(float x) { return x; }
__device__ __forceinline__ float as_logit(__nv_bfloat16 x) { return __bfloat162float(x); }

// A number that rises with the logit; NaN counts as -inf.
constexpr uint32_t kLowest = 0x007fffffu;
__device__ __forceinline__ uint32_t order_of(float x) {
    if (!(x == x)) return kLowest;
    const uint32_t b = __float_as_uint(x + 0.f);  // -0 as 0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// 2^(j / 16), j = 0 .. 15: in units of 2^-31, and in two fp32 words.
struct Table {
    uint2 fixed[16];  // the number, and fp32 of it
    float low[16];    // what fp32 of 2^(j / 16) leaves
};

// What the weights of a row go by.
struct Scale {
    float top;       // the largest logit
    float c, c_low;  // 16 log2(e) / T in two words
    // top c = whole + rest: whole a multiple of 1/64, so that sums with whole numbers are
    // exact; fast: |top c| is below 2^16, where that holds
    float whole, rest;
    int fast;
};

constexpr double kLn = 0.69314718055994530942 / 16.0;  // 2^(f / 16) - 1 = k1 f + k2 f^2 + ...
constexpr float kK1 = (float)kLn, kK2 = (float)(kLn * kLn / 2), kK3 = (float)(kLn * kLn * kLn / 6),
                kK4 = (float)(kLn * kLn * kLn * kLn / 24);

constexpr float kLeast = -2000.f;                  // 2^-125: smaller weights are zero
constexpr float kUnit = 4.656612873077393e-10f;    // 2^-31

// exp((x - top) / T) = 2^((n + f) / 16), n whole and |f| <= 1/2: n is a multiple of 1/16 of a
// factor of two, f comes from one rounding of x c - (whole + n), which is exact before it.
struct Split {
    int n;
    float q;  // 2^(f / 16) - 1
};
// 2^(f / 16) - 1
__device__ __forceinline__ float power_of(float f) {
    return __fmul_rn(f, __fmaf_rn(f, __fmaf_rn(f, __fmaf_rn(f, kK4, kK3), kK2), kK1));
}
__device__ __forceinline__ Split split_fast(const Scale& s, float x) {
    const float y = __fmaf_rn(x, s.c, -s.whole);
    const float r = __fadd_rn(y, kMagic), n = __fsub_rn(r, kMagic);
    const float f = __fadd_rn(__fmaf_rn(x, s.c, -__fadd_rn(n, s.whole)), __fmaf_rn(x, s.c_low, -s.rest));
    // (NaN and -inf fail the comparison)
    return Split{y > kLeast ? __float_as_int(r) - __float_as_int(kMagic) : (int)kLeast, power_of(f)};
}

// The same where top / T is too large for that: the difference from the largest logit
// first, in two words.  (Far off the way: logits above 2800 T.)
__device__ __noinline__ int2 split_slow(const Scale& s, float x) {
    const float d = __fsub_rn(x, s.top), b = __fsub_rn(d, x);
    const float dl = __fsub_rn(__fsub_rn(x, __fsub_rn(d, b)), __fadd_rn(s.top, b));
    const float y = __fmul_rn(d, s.c);
    if (!(y > kLeast)) return make_int2((int)kLeast, 0);
    const float yl = __fmaf_rn(dl, s.c, __fmaf_rn(d, s.c_low, __fmaf_rn(d, s.c, -y)));
    const float r = __fadd_rn(y, kMagic);
    const float f = __fadd_rn(__fsub_rn(y, __fsub_rn(r, kMagic)), yl);
    return make_int2(__float_as_int(r) - __float_as_int(kMagic), __float_as_int(power_of(f)));
}
__device__ __forceinline__ Split split_of(const Scale& s, float x) {
    if (s.fast) return split_fast(s, x);
    const int2 w = split_slow(s, x);
    return Split{w.x, __int_as_float(w.y)};
}

// A weight in multiples of 2^-42.  (Every operation rounds as written: all passes must get
// the same.)
__device__ __forceinline__ unsigned long long fixed_fast(const Table& t, const Scale& s, float x) {
    // (far below, -inf and NaN: shifted out whatever the polynomial gives)
    const float y = fmaxf(__fmaf_rn(x, s.c, -s.whole), -704.f);
    const float r = __fadd_rn(y, kMagic), n = __fsub_rn(r, kMagic);
    const float f = __fadd_rn(__fmaf_rn(x, s.c, -__fadd_rn(n, s.whole)), __fmaf_rn(x, s.c_low, -s.rest));
    const uint2 e = t.fixed[__float_as_int(r) & 15];
    const uint32_t v =
        e.x + (uint32_t)__float2int_rn(__fmul_rn(__uint_as_float(e.y), power_of(f)));
    // units of 2^-31 of a factor of two down to those of 2^-42 of one, rounded
    const int down = (__float_as_int(kMagic) + 15 - __float_as_int(r)) >> 4;
    if (down >= 12) return (__funnelshift_rc(v, 0u, down - 12) + 1u) >> 1;
    return (unsigned long long)v << (11 - down);
}
__device__ __noinline__ unsigned long long fixed_slow(const Table& t, const Scale& s, float x) {
    if (x == s.top) return kOne;
    const int2 w = split_slow(s, x);
    if (w.x <= -688) return 0;  // half a unit
    const uint2 e = t.fixed[w.x & 15];
    const uint32_t v =
        e.x + (uint32_t)__float2int_rn(__fmul_rn(__uint_as_float(e.y), __int_as_float(w.y)));
    return ((((unsigned long long)v << 32) >> (20 - (w.x >> 4))) + 1) >> 1;
}
__device__ __forceinline__ unsigned long long fixed_of(const Table& t, const Scale& s, float x) {
    return s.fast ? fixed_fast(t, s, x) : fixed_slow(t, s, x);
}

// The same as a number; and whether it is at least m, without that number's rounding.
__device__ __forceinline__ float weight_of(const Table& t, const Scale& s, float x) {
    if (x == s.top) return 1.f;
    const Split p = split_of(s, x);
    if (p.n <= (int)kLeast) return 0.f;
    const float hi = __fmul_rn(__uint_as_float(t.fixed[p.n & 15].y), kUnit);
    const float w = __fadd_rn(hi, __fmaf_rn(hi, p.q, t.low[p.n & 15]));
    return __fmul_rn(w, __int_as_float(((p.n >> 4) + 127) << 23));
}
__device__ __forceinline__ bool at_least(const Table& t, const Scale& s, float x, float m) {
    if (x == s.top) return true;
    const Split p = split_of(s, x);
    if (p.n <= (int)kLeast) return false;
    const float hi = __fmul_rn(__uint_as_float(t.fixed[p.n & 15].y), kUnit);
    const float scaled = m * __int_as_float((127 - (p.n >> 4)) << 23);
    return __fadd_rn(__fsub_rn(hi, scaled), __fmaf_rn(hi, p.q, t.low[p.n & 15])) >= 0.f;
}

// A beginning of the row: order above `key`, or equal to it and an index up to `last`.
struct Cut {
    uint32_t key;
    int last;
    __device__ __forceinline__ bool keeps(uint32_t o, int i) const {
        return o > key || (o == key && i <= last);
    }
};

struct Shared {
    Table table;
    union {
        uint32_t hist[4][kBins];  // counts; weights in three words of 14 bits
        uint32_t orders[kOrders]; // first pass: counts by the upper bits of the orders;
                                  // second pass: by the distance from the largest logit
    };
    unsigned long long list[kList];   // of this CTA; then sorted by the first
    unsigned long long merged[kList]; // of all CTAs, at the first
    unsigned long long warp_sum[kWarps], part_sum[kWarps];
    unsigned long long cta_sum[kMaxCtas], cta_above[kMaxCtas];
    unsigned long long kept;      // the sum of what is kept, from the first CTA
    float least;                  // the smallest logit that min-p keeps
    int good;                     // the bracket of the top-p border held it; min-p decides alone
    unsigned long long cta_top[kMaxCtas];
    uint32_t cta_low[kMaxCtas];
    uint32_t cta_lo[kMaxCtas], cta_hi[kMaxCtas];
    unsigned int cta_ties[kMaxCtas];
    Scale scale;
    Cut cut;
    unsigned long long before_mass, want[3];
    unsigned int n_list, n_merged, base;
    unsigned int bin, in_bin, before_count;
    int found;
};

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}

// Inclusive sums in thread order.
__device__ __forceinline__ unsigned long long block_sums(Shared& sh, unsigned long long x,
                                                         unsigned long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long o = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += o;
    }
    __syncthreads();
    if (lane == 31) sh.warp_sum[warp] = x;
    __syncthreads();
    unsigned long long s = lane < kWarps ? sh.warp_sum[lane] : 0;
#pragma unroll
    for (int d = 1; d < kWarps; d <<= 1) {
        const unsigned long long o = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += o;
    }
    total = __shfl_sync(0xffffffffu, s, kWarps - 1);
    const unsigned long long before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
    return x + (warp > 0 ? before : 0);
}
__device__ __forceinline__ unsigned long long warp_total(unsigned long long x) {
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// What a share p of a sum asks for, rounded up, one at least; and where u of it ends.  64-bit
// floating point is a small unit's work here: one thread does it and shares the result.
__device__ __forceinline__ unsigned long long share_of(float p, unsigned long long total) {
    const double x = ceil((double)p * (double)total);
    return x < 1.0 ? 1ull : (unsigned long long)x;
}
__device__ __forceinline__ unsigned long long part_of(float u, unsigned long long total) {
    return (unsigned long long)((double)u * (double)total);
}

// A row's elements as 16-byte vectors from the boundary at or before its start: vector v
// holds the elements v * VEC - shift and so on; the outer ones are loaded one by one.
template <typename Elem>
struct Row {
    static constexpr int VEC = 16 / (int)sizeof(Elem);
    const Elem* p;
    int V, shift, vectors;

    __device__ __forceinline__ Row(const Elem* base, int V_) : p(base), V(V_) {
        shift = (int)(reinterpret_cast<uintptr_t>(base) / sizeof(Elem) % VEC);
        vectors = (shift + V + VEC - 1) / VEC;
    }
    __device__ __forceinline__ bool has(int i) const { return (unsigned)i < (unsigned)V; }
    __device__ __forceinline__ static float most(const float (&x)[VEC]) {
        float y = x[0];
#pragma unroll
        for (int z = 1; z < VEC; ++z) y = fmaxf(y, x[z]);
        return y;  // (NaN only where all are)
    }
    // (-inf where the row has no element)
    __device__ __forceinline__ uint4 load(int v, int end) const {
        const int i = v * VEC - shift;
        constexpr uint32_t kNone = sizeof(Elem) == 4 ? 0xff800000u : 0xff80ff80u;
        uint4 w = make_uint4(kNone, kNone, kNone, kNone);
        if (v < end) {
            if (i >= 0 && i + VEC <= V) {
                w = *reinterpret_cast<const uint4*>(p + i);
            } else {
                Elem* e = reinterpret_cast<Elem*>(&w);
#pragma unroll
                for (int z = 0; z < VEC; ++z)
                    if (has(i + z)) e[z] = p[i + z];
            }
        }
        return w;
    }
    // f(vector, logits) for the vectors [lo, hi), by one warp, BATCH elements a lane at once.
    template <int BATCH = kBatch, typename F>
    __device__ __forceinline__ void vectors_of(int lo, int hi, F f) const {
        constexpr int N = BATCH / VEC;
        for (int v0 = lo + (int)(threadIdx.x & 31); v0 < hi; v0 += 32 * N) {
            uint4 w[N];
#pragma unroll
            for (int k = 0; k < N; ++k) w[k] = load(v0 + 32 * k, hi);
#pragma unroll
            for (int k = 0; k < N; ++k) {
                if (v0 + 32 * k >= hi) break;
                const Elem* e = reinterpret_cast<const Elem*>(&w[k]);
                float x[VEC];
#pragma unroll
                for (int z = 0; z < VEC; ++z) x[z] = as_logit(e[z]);
                f(v0 + 32 * k, x);
            }
        }
    }
    // f(index, logit) for the row's elements in the vectors [lo, hi), by one warp.
    template <typename F>
    __device__ __forceinline__ void each(int lo, int hi, F f) const {
        constexpr int N = kBatch / VEC;
        for (int v0 = lo + (int)(threadIdx.x & 31); v0 < hi; v0 += 32 * N) {
            uint4 w[N];
#pragma unroll
            for (int k = 0; k < N; ++k) w[k] = load(v0 + 32 * k, hi);
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const Elem* e = reinterpret_cast<const Elem*>(&w[k]);
                const int i = (v0 + 32 * k) * VEC - shift;
                if (v0 + 32 * k < hi) {
#pragma unroll
                    for (int z = 0; z < VEC; ++z)
                        if (has(i + z)) f(i + z, as_logit(e[z]));
                }
            }
        }
    }
};

// n <= kList numbers of sh.merged in falling order; all threads.
__device__ __forceinline__ void sort_falling(Shared& sh, int n) {
    const int tid = threadIdx.x;
    int size = 32;
    while (size < n) size <<= 1;
    if (size <= kThreads) {  // a number a thread: most steps stay within a warp
        unsigned long long v = tid < n ? sh.merged[tid] : 0;
#pragma unroll 1
        for (int k = 2; k <= size; k <<= 1)
#pragma unroll 1
            for (int j = k >> 1; j; j >>= 1) {
                unsigned long long o;
                if (j >= 32) {
                    __syncthreads();
                    sh.merged[tid] = v;
                    __syncthreads();
                    o = sh.merged[tid ^ j];
                } else {
                    o = __shfl_xor_sync(0xffffffffu, v, j);
                }
                if ((o > v) == (((tid & j) == 0) == ((tid & k) == 0))) v = o;
            }
        __syncthreads();
        sh.merged[tid] = v;
        __syncthreads();
        return;
    }
    for (int i = n + tid; i < size; i += kThreads) sh.merged[i] = 0;
    __syncthreads();
    for (int k = 2; k <= size; k <<= 1)
        for (int j = k >> 1; j; j >>= 1) {
            for (int t = tid; t < size / 2; t += kThreads) {
                const int a = 2 * t - (t & (j - 1)), b = a + j;
                const unsigned long long x = sh.merged[a], y = sh.merged[b];
                if ((x < y) == ((a & k) == 0)) {
                    sh.merged[a] = y;
                    sh.merged[b] = x;
                }
            }
            __syncthreads();
        }
}

template <typename Elem>
struct Picker {
    Shared& sh;
    const Row<Elem>& row;
    cg::cluster_group& cluster;
    int rank, ctas, wlo, whi;  // of this warp's vectors
    uint32_t low;              // the smallest order above kLowest (inf's where there is none)

    // Elements on their way to the first CTA: into this CTA's list, then all at once.
    __device__ __forceinline__ void note(int i, float x) {
        const unsigned int at = atomicAdd(&sh.n_list, 1u);
        if (at < kList)
            sh.list[at] = (unsigned long long)order_of(x) << 32 | (0xffffffffu - (uint32_t)i);
    }
    // (With what must be visible there as well; ends with a barrier of the cluster.)
    __device__ __forceinline__ void send() {
        const int tid = threadIdx.x;
        __syncthreads();
        const unsigned int n = sh.n_list;
        if (tid == 0 && n > 0) sh.base = atomicAdd(cluster.map_shared_rank(&sh.n_merged, 0), n);
        __syncthreads();
        unsigned long long* to = cluster.map_shared_rank(&sh.merged[0], 0);
        for (unsigned int i = tid; i < min(n, (unsigned int)kList); i += kThreads)
            if (sh.base + i < kList) to[sh.base + i] = sh.list[i];
        cluster_sync();
    }

    // The first `count` elements, and of these the share p, from the first pass's counts:
    // sorted at the first CTA (see find's `whole`).  False where no list holds them.
    __device__ __forceinline__ bool find_first(unsigned int count, float p, uint32_t top_key,
                                               float& from) {
        const int tid = threadIdx.x;
        const int bin = (int)(top_key >> kOrderShift) - tid;
        unsigned int n = 0;
        if (bin >= 0)
            for (int r = 0; r < ctas; ++r) n += cluster.map_shared_rank(&sh.orders[0], r)[bin];
        if (tid == 0) sh.bin = kBins;
        unsigned long long total;
        const unsigned long long end = block_sums(sh, n, total);
        if (end >= count && end - n < count) {
            sh.bin = tid;
            sh.in_bin = (unsigned int)end;
        }
        if (tid == 0) sh.n_list = 0;
        __syncthreads();
        if (sh.bin == kBins || sh.in_bin > kList) {
            cluster_sync();  // the counts are no longer read
            return false;
        }
        const uint32_t key = ((top_key >> kOrderShift) - sh.bin) << kOrderShift;
        from = key > kLowest ? logit_of(key) : -INFINITY;
        row.template vectors_of<2 * kBatch>(wlo, whi, [&](int v, const float (&x)[Row<Elem>::VEC]) {
            if (row.most(x) >= from)
#pragma unroll
            for (int z = 0; z < Row<Elem>::VEC; ++z)
                if (x[z] >= from && row.has(v * Row<Elem>::VEC - row.shift + z))
                    note(v * Row<Elem>::VEC - row.shift + z, x[z]);
        });
        send();
        if (rank == 0) {
            const int m = (int)min(sh.n_merged, (unsigned int)kList);
            sort_falling(sh, m);
            finish_whole((int)count, m, p, sh.scale);
        }
        return true;
    }

    // Gathers the elements that `take` accepts at the first CTA; n of them in all.
    template <typename F>
    __device__ __forceinline__ void gather(F take) {
        const int tid = threadIdx.x;
        if (tid == 0) sh.n_list = 0;
        if (rank == 0 && tid == 0) sh.n_merged = 0;
        __syncthreads();
        cluster_sync();
        row.each(wlo, whi, [&](int i, float x) {
            if (take(i, x, order_of(x))) note(i, x);
        });
        send();
    }

    // The first `count` elements of `set` (count > 0) or as many as reach the share p of
    // its sum (count = 0).  Where the list that decides holds everything that is kept
    // (`whole`: count and then p, both) it stays sorted at the first CTA, with the
    // number kept in sh.found; returns whether it does.
    __device__ __forceinline__ bool find(unsigned int count, float p, const Cut set, bool all,
                                         Cut& out) {
        const int tid = threadIdx.x, lane = tid & 31;
        const bool mass = count == 0;
        const Scale s = sh.scale;
        // the first bins: over the logits above 2^-24 of the largest
        const float span = fminf(24.f * 16.f / s.c, s.top - logit_of(low));
        const float per = span > 0.f && s.top < INFINITY ? fminf((kBins - 1) / span, 1e30f) : 1.f;
        auto first_bin = [&](float x) {
            if (x == s.top) return 0;
            return (int)fminf((s.top - x) * per, (float)(kBins - 1));  // NaN: the last
        };
        unsigned long long above = 0, want = 0;  // of the summed kind
        unsigned int above_count = 0;
        uint32_t klo = 0, khi = 0xffffffffu;
        int shift = 32;
        for (int round = 0;; ++round) {
            for (int i = tid; i < 4 * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0;
            __syncthreads();
            unsigned int last_n = 0;
            unsigned long long last_w = 0;
            row.each(wlo, whi, [&](int i, float x) {
                const uint32_t o = order_of(x);
                if (!all && !set.keeps(o, i)) return;
                int b;
                if (round == 0) {
                    b = first_bin(x);
                } else {
                    if (o < klo || o > khi) return;
                    b = (int)((khi - o) >> shift);
                }
                const unsigned long long u = mass ? fixed_of(sh.table, s, x) : 0;
                if (round == 0 && b == kBins - 1) {  // most of a steep row
                    ++last_n;
                    last_w += u;
                    return;
                }
                atomicAdd(&sh.hist[0][b], 1u);
                if (mass) {
                    atomicAdd(&sh.hist[1][b], (uint32_t)(u >> 28));
                    atomicAdd(&sh.hist[2][b], (uint32_t)(u >> 14) & 0x3fffu);
                    atomicAdd(&sh.hist[3][b], (uint32_t)u & 0x3fffu);
                }
            });
            if (round == 0) {
                const unsigned int n = __reduce_add_sync(0xffffffffu, last_n);
                if (lane == 0 && n) atomicAdd(&sh.hist[0][kBins - 1], n);
                if (mass) {
                    const unsigned long long u = warp_total(last_w);
                    if (lane == 0 && u) {
                        atomicAdd(&sh.hist[1][kBins - 1], (uint32_t)(u >> 28));
                        atomicAdd(&sh.hist[2][kBins - 1], (uint32_t)(u >> 14) & 0x3fffu);
                        atomicAdd(&sh.hist[3][kBins - 1], (uint32_t)u & 0x3fffu);
                    }
                }
            }
            cluster_sync();
            unsigned int n = 0;
            unsigned long long w = 0;
            for (int r = 0; r < ctas; ++r) {
                const uint32_t* h = cluster.map_shared_rank(&sh.hist[0][0], r);
                n += h[tid];
                if (mass)
                    w += ((unsigned long long)h[kBins + tid] << 28) +
                         ((unsigned long long)h[2 * kBins + tid] << 14) + h[3 * kBins + tid];
            }
            if (tid == 0) sh.bin = kBins;
            unsigned long long total;
            const unsigned long long mine = mass ? w : n, end = block_sums(sh, mine, total);
            if (round == 0) {
                if (mass) {
                    if (tid == 0) sh.want[0] = share_of(p, total);
                    __syncthreads();
                    want = sh.want[0];
                } else {
                    want = count;
                }
            }
            const unsigned long long left = want - above;
            if (end >= left && end - mine < left) {
                sh.bin = tid;
                sh.in_bin = n;
                sh.before_mass = end - mine;
            }
            unsigned long long skip;
            const unsigned long long counts = mass ? block_sums(sh, n, skip) : end;
            __syncthreads();
            const unsigned int bin = sh.bin, in_bin = sh.in_bin;
            if (bin == kBins) {  // the sums are exact, so that one bin is reached
                cluster_sync();
                out = set;
                return false;
            }
            if (tid == (int)bin) sh.before_count = (unsigned int)(counts - n);
            above += sh.before_mass;
            __syncthreads();
            above_count += sh.before_count;
            auto in_round = [&](int i, float x, uint32_t o, bool up) {
                if (!all && !set.keeps(o, i)) return false;
                if (round == 0) return up ? first_bin(x) <= (int)bin : first_bin(x) == (int)bin;
                return o >= klo && o <= khi && ((khi - o) >> shift) == bin;
            };
            const bool whole = !mass && round == 0 && above_count + in_bin <= kList;
            if (in_bin <= kList) {
                gather([&](int i, float x, uint32_t o) { return in_round(i, x, o, whole); });
                if (rank == 0) {
                    const int m = (int)min(sh.n_merged, (unsigned int)kList);
                    sort_falling(sh, m);
                    if (whole)
                        finish_whole((int)count, m, p, s);
                    else
                        finish(want - above, m, mass, s);
                    if (tid > 0 && tid < ctas) *cluster.map_shared_rank(&sh.cut, tid) = sh.cut;
                }
                cluster_sync();
                out = sh.cut;
                return whole;
            }
            // too many: their range of orders, divided again by its upper bits
            uint32_t lo = 0xffffffffu, hi = 0;
            row.each(wlo, whi, [&](int i, float x) {
                const uint32_t o = order_of(x);
                if (in_round(i, x, o, false)) {
                    lo = min(lo, o);
                    hi = max(hi, o);
                }
            });
            lo = __reduce_min_sync(0xffffffffu, lo);
            hi = __reduce_max_sync(0xffffffffu, hi);
            if (tid == 0) {
                sh.base = 0xffffffffu;  // smallest and largest of the CTA
                sh.n_list = 0;
            }
            __syncthreads();
            if (lane == 0) {
                atomicMin(&sh.base, lo);
                atomicMax(&sh.n_list, hi);
            }
            __syncthreads();
            if (tid < ctas) {
                cluster.map_shared_rank(&sh.cta_lo[0], tid)[rank] = sh.base;
                cluster.map_shared_rank(&sh.cta_hi[0], tid)[rank] = sh.n_list;
            }
            cluster_sync();
            klo = 0xffffffffu;
            khi = 0;
            for (int r = 0; r < ctas; ++r) {
                klo = min(klo, sh.cta_lo[r]);
                khi = max(khi, sh.cta_hi[r]);
            }
            if (klo == khi) {
                // ties: as many as are needed, in index order
                unsigned long long need = want - above;
                if (mass) {
                    const unsigned long long each = fixed_of(sh.table, s, logit_of(klo));
                    need = each ? (need + each - 1) / each : in_bin;
                }
                out.key = klo;
                out.last = nth_tie(klo, (unsigned int)min(need, (unsigned long long)in_bin), set, all);
                return false;
            }
            shift = max(0, 32 - __clz(khi - klo) - 9);
            cluster_sync();  // all have read the ranges and the bins
        }
    }

    // The first `need` numbers of a sorted list, by count or by weight; whether it has as many.
    __device__ __forceinline__ bool finish(unsigned long long need, int m, bool mass,
                                           const Scale& s) {
        const int tid = threadIdx.x;
        unsigned long long before = 0;
        if (!mass) {
            if (tid == 0) set_cut(sh.merged[min(need, (unsigned long long)m) - 1]);
            before = m;
        } else {
            if (tid == 0) set_cut(sh.merged[m - 1]);
            __syncthreads();
            for (int i0 = 0; i0 < m && before < need; i0 += kThreads) {
                const int i = i0 + tid;
                const unsigned long long u =
                    i < m ? fixed_of(sh.table, s, logit_of((uint32_t)(sh.merged[i] >> 32))) : 0;
                unsigned long long total;
                const unsigned long long end = block_sums(sh, u, total) + before;
                if (i < m && end >= need && end - u < need) set_cut(sh.merged[i]);
                before += total;
            }
        }
        __syncthreads();
        return before >= need;
    }

    // A sorted list that begins the row: the first `count`, and of these the share p.
    __device__ __forceinline__ void finish_whole(int count, int m, float p, const Scale& s) {
        const int tid = threadIdx.x;
        m = min(m, count);
        unsigned long long u[kList / kThreads], total = 0;
        // each thread a run of the list
        const int per = (m + kThreads - 1) / kThreads, lo = tid * per;
        unsigned long long mine = 0;
#pragma unroll
        for (int k = 0; k < kList / kThreads; ++k) {
            u[k] = k < per && lo + k < m
                       ? fixed_of(sh.table, s, logit_of((uint32_t)(sh.merged[lo + k] >> 32)))
                       : 0;
            mine += u[k];
        }
        unsigned long long at = block_sums(sh, mine, total) - mine;
        if (tid == 0) {
            sh.found = m;
            set_cut(sh.merged[m - 1]);
            if (p < 1.f) sh.want[0] = share_of(p, total);
        }
        __syncthreads();
        if (p < 1.f) {
            const unsigned long long want = sh.want[0];
#pragma unroll
            for (int k = 0; k < kList / kThreads; ++k) {
                if (u[k] > 0 && at < want && at + u[k] >= want) {
                    sh.found = lo + k + 1;
                    set_cut(sh.merged[lo + k]);
                }
                at += u[k];
            }
            __syncthreads();
        }
    }

    __device__ __forceinline__ void set_cut(unsigned long long e) {
        sh.cut.key = (uint32_t)(e >> 32);
        sh.cut.last = (int)(0xffffffffu - (uint32_t)e);
    }

    // The index of the need-th element of this order (need >= 1).
    __device__ __forceinline__ int nth_tie(uint32_t key, unsigned int need, const Cut set, bool all) {
        const int tid = threadIdx.x, lane = tid & 31;
        unsigned int n = 0;
        auto is = [&](int i, float x) {
            const uint32_t o = order_of(x);
            return o == key && (all || set.keeps(o, i));
        };
        row.each(wlo, whi, [&](int i, float x) { n += is(i, x); });
        n = __reduce_add_sync(0xffffffffu, n);
        unsigned long long total;
        const unsigned long long end = block_sums(sh, lane == 0 ? n : 0, total);  // lane 0's: with its warp
        if (tid < ctas) cluster.map_shared_rank(&sh.cta_ties[0], tid)[rank] = (unsigned int)total;
        cluster_sync();
        unsigned int before = 0;
        for (int r = 0; r < rank; ++r) before += sh.cta_ties[r];
        const unsigned int wend = before + (unsigned int)__shfl_sync(0xffffffffu, end, 0);
        if (need > wend - n && need <= wend) {
            // this warp's: 32 vectors at a time, in order
            unsigned int at = wend - n;
            for (int v0 = wlo; v0 < whi; v0 += 32) {
                const uint4 w = row.load(v0 + lane, whi);
                const Elem* e = reinterpret_cast<const Elem*>(&w);
                const int i = (v0 + lane) * Row<Elem>::VEC - row.shift;
                unsigned int c = 0;
                for (int z = 0; z < Row<Elem>::VEC; ++z)
                    c += v0 + lane < whi && row.has(i + z) && is(i + z, as_logit(e[z]));
                unsigned int inc = c;
                for (int d = 1; d < 32; d <<= 1) {
                    const unsigned int o = __shfl_up_sync(0xffffffffu, inc, d);
                    if (lane >= d) inc += o;
                }
                unsigned int run = at + inc - c;
                for (int z = 0; z < Row<Elem>::VEC; ++z)
                    if (v0 + lane < whi && row.has(i + z) && is(i + z, as_logit(e[z])) &&
                        ++run == need) {
                        for (int r = 0; r < ctas; ++r)
                            *cluster.map_shared_rank(&sh.cut.last, r) = i + z;
                    }
                at += __shfl_sync(0xffffffffu, inc, 31);
            }
        }
        cluster_sync();
        return sh.cut.last;
    }
};

template <typename Elem, bool kProbs>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a, const Table table) {
    extern __shared__ __align__(16) unsigned char raw[];
    Shared& sh = *reinterpret_cast<Shared*>(raw);
    cg::cluster_group cluster = cg::this_cluster();
    cluster_arrive();  // waited for before the first write into another CTA
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int r = blockIdx.x / ctas, V = a.V;
    const float T = a.temperature ? a.temperature[r] : 1.f;
    const float p = a.top_p ? a.top_p[r] : 1.f, m = a.min_p ? a.min_p[r] : 0.f;
    const float u = !kProbs ? a.u[r] : 0.f;
    const int k = a.top_k ? a.top_k[r] : 0;
    if (tid < 16) {
        sh.table.fixed[tid] = table.fixed[tid];
        sh.table.low[tid] = table.low[tid];
    }
    const Row<Elem> row(static_cast<const Elem*>(a.logits) + (size_t)r * V, V);
    const int share = (row.vectors + ctas - 1) / ctas, lo = min(rank * share, row.vectors),
              hi = min(lo + share, row.vectors);
    const int part = (hi - lo + kWarps - 1) / kWarps, wlo = min(lo + warp * part, hi),
              whi = min(wlo + part, hi);

    constexpr int VEC = Row<Elem>::VEC;
    const bool first_k = k > 0 && k < V;
    if (first_k) {
        for (int i = tid; i < kOrders; i += kThreads) sh.orders[i] = 0;
        __syncthreads();
    }
    // the largest logit and the first vector that holds it; the smallest above -inf (which the
    // bins of the passes below span; what lies beside the row is -inf too)
    float best = -INFINITY, least = INFINITY;
    int where = 0;
    row.vectors_of(wlo, whi, [&](int v, const float (&x)[VEC]) {
        float most = x[0], fewest = x[0];
#pragma unroll
        for (int z = 1; z < VEC; ++z) {
            most = fmaxf(most, x[z]);
            fewest = fminf(fewest, x[z]);
        }
        if (fewest == -INFINITY) {
            fewest = INFINITY;
#pragma unroll
            for (int z = 0; z < VEC; ++z)
                if (x[z] > -INFINITY) fewest = fminf(fewest, x[z]);
        }
        least = fminf(least, fewest);
        if (most > best) {
            best = most;
            where = v;
        }
        if (first_k) {
#pragma unroll
            for (int z = 0; z < VEC; ++z) {
                const int b = __float_as_int(x[z] + 0.f);  // -0 as 0
                if (x[z] == x[z])
                    atomicAdd(&sh.orders[(uint32_t)(b ^ ((b >> 31) | (int)0x80000000)) >> kOrderShift], 1u);
            }
        }
    });
    unsigned long long top = (unsigned long long)order_of(best) << 32 | (0xffffffffu - (uint32_t)where);
    uint32_t low = order_of(least);
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const unsigned long long o = __shfl_xor_sync(0xffffffffu, top, d);
        top = o > top ? o : top;
    }
    low = __reduce_min_sync(0xffffffffu, low);
    if (lane == 0) {
        sh.warp_sum[warp] = top;
        sh.part_sum[warp] = low;
    }
    if (tid == 0) {
        sh.n_merged = 0;
        sh.n_list = 0;
    }
    cluster_wait();
    __syncthreads();
    if (warp == 0) {
        top = lane < kWarps ? sh.warp_sum[lane] : 0;
        low = lane < kWarps ? (uint32_t)sh.part_sum[lane] : 0xffffffffu;
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const unsigned long long o = __shfl_xor_sync(0xffffffffu, top, d);
            top = o > top ? o : top;
        }
        low = __reduce_min_sync(0xffffffffu, low);
        if (lane < ctas) {
            cluster.map_shared_rank(&sh.cta_top[0], lane)[rank] = top;
            cluster.map_shared_rank(&sh.cta_low[0], lane)[rank] = low;
        }
    }
    cluster_sync();
    top = 0;
    low = 0xffffffffu;
    for (int c = 0; c < ctas; ++c) {
        top = sh.cta_top[c] > top ? sh.cta_top[c] : top;
        low = min(low, sh.cta_low[c]);
    }
    const uint32_t top_key = (uint32_t)(top >> 32);

    // outputs of a vector, whole where the rows of both start alike
    const size_t out_row = (size_t)r * V;
    const bool whole_out =
        a.probs_bf16 == (sizeof(Elem) == 2) &&
        ((reinterpret_cast<uintptr_t>(a.probs) - reinterpret_cast<uintptr_t>(a.logits)) & 15u) == 0;
    auto put = [&](int v, const float (&y)[VEC]) {
        const int i = v * VEC - row.shift;
        if (whole_out && i >= 0 && i + VEC <= V) {
            uint4 w;
            if constexpr (sizeof(Elem) == 4) {
                w = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]),
                               __float_as_uint(y[3]));
            } else {
                uint32_t h[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const __nv_bfloat162 q = __floats2bfloat162_rn(y[2 * z], y[2 * z + 1]);
                    h[z] = *reinterpret_cast<const uint32_t*>(&q);
                }
                w = make_uint4(h[0], h[1], h[2], h[3]);
            }
            *reinterpret_cast<uint4*>(static_cast<Elem*>(a.probs) + out_row + i) = w;
            return;
        }
#pragma unroll
        for (int z = 0; z < VEC; ++z) {
            if (!row.has(i + z)) continue;
            if (a.probs_bf16)
                static_cast<__nv_bfloat16*>(a.probs)[out_row + i + z] = __float2bfloat16_rn(y[z]);
            else
                static_cast<float*>(a.probs)[out_row + i + z] = y[z];
        }
    };
    const bool params = T >= 0.f && T <= 1e30f && p == p && m == m && u >= 0.f && u < 1.f;
    const bool some = top_key > kLowest;
    if (!params || !some || T == 0.f) {
        const bool good = params && some;
        if (!good && rank == 0 && tid == 0)
            report(a.dev_status, params ? KVD_DEV_PROBS : KVD_DEV_PARAM);
        int at = -1;
        if (good) {  // the first of the largest logits
            const int v = (int)(0xffffffffu - (uint32_t)top);
            const uint4 w = row.load(v, row.vectors);
            const Elem* e = reinterpret_cast<const Elem*>(&w);
            for (int z = VEC - 1; z >= 0; --z)
                if (order_of(as_logit(e[z])) == top_key && row.has(v * VEC - row.shift + z))
                    at = v * VEC - row.shift + z;
        }
        if (kProbs) {
            row.vectors_of(wlo, whi, [&](int v, const float (&)[VEC]) {
                float y[VEC];
#pragma unroll
                for (int z = 0; z < VEC; ++z) y[z] = v * VEC - row.shift + z == at ? 1.f : 0.f;
                put(v, y);
            });
        } else if (rank == 0 && tid == 0) {
            a.tokens[r] = at;
        }
        return;
    }
    // In pairs of fp32 words (about 2^-47 of themselves): in 64 bits one thread's division and
    // what follows it took 1500 cycles (a row of 32000 10.9 us, now 10.3; 4 rows with top-p
    // 17.9, 16.6).
    if (tid == 0) {
        constexpr double kPer = 23.083120654223414;  // 16 log2(e)
        constexpr float kHigh = (float)kPer, kLow = (float)(kPer - (double)kHigh);
        const float q = __fdiv_rn(kHigh, T);
        const float more =
            q < INFINITY ? __fdividef(__fadd_rn(__fmaf_rn(-q, T, kHigh), kLow), T) : 0.f;
        const float x = logit_of(top_key), c = __fadd_rn(q, more), c_low = __fsub_rn(more, __fsub_rn(c, q));
        const float y = __fmul_rn(x, c), whole = rintf(y * 64.f) * 0.015625f;
        sh.scale = Scale{x, c, c_low, whole,
                         __fadd_rn(__fsub_rn(y, whole), __fmaf_rn(x, c_low, __fmaf_rn(x, c, -y))),
                         fabsf(y) < 65536.f};
    }
    __syncthreads();
    const Scale s = sh.scale;
    if (warp == kWarps - 1) {
        // the smallest logit that min-p keeps: 32 orders a round (while the others go on; the
        // barriers before its first use are the passes')
        uint32_t lo_key = kLowest, hi_key = top_key;  // hi_key is kept, lo_key not (or below all)
        const float least_w = fminf(m, 1.f);
        while (m > 0.f && hi_key - lo_key > 1) {
            const uint32_t step = (hi_key - lo_key + 31) / 32;
            const uint32_t key = lo_key + min(step * (lane + 1), hi_key - lo_key);
            const uint32_t yes = __ballot_sync(0xffffffffu, at_least(sh.table, s, logit_of(key), least_w));
            const int first = __ffs(yes) - 1;  // the last lane's is kept
            hi_key = lo_key + min(step * (first + 1), hi_key - lo_key);
            lo_key = first > 0 ? lo_key + step * first : lo_key;
        }
        if (lane == 0) sh.least = m > 0.f ? logit_of(hi_key) : -INFINITY;
    }

    Picker<Elem> pick{sh, row, cluster, rank, ctas, wlo, whi, low};
    Cut cut{0u, 0x7fffffff};
    // whole: all that is kept is sorted in the first CTA's list; summed: part_sum holds
    // the sums of what is kept, a warp
    bool whole = false, summed = false;
    float from = -INFINITY;  // nothing below is kept
    if (first_k) {
        whole = pick.find_first((unsigned int)k, p, top_key, from);
        if (!whole) whole = pick.find((unsigned int)k, p, cut, true, cut);
    }
    if (!whole && !first_k) {
        float hi = -INFINITY, lo_x = -INFINITY;
        bool border = p < 1.f;  // top-p's has to be found
        if (border) {
            for (int i = tid; i < kFine; i += kThreads) sh.orders[i] = 0;
            __syncthreads();
            // bins of a 64th of a factor of two, as far as 2^-32 (or the smallest logit)
            const float span = fminf(32.f * 16.f / s.c, s.top - logit_of(low));
            const float per = span > 0.f && s.top < INFINITY ? fminf((kFine - 2) / span, 1e30f) : 1.f;
            unsigned int behind = 0;
            row.vectors_of(wlo, whi, [&](int, const float (&x)[VEC]) {
#pragma unroll
                for (int z = 0; z < VEC; ++z) {
                    const float d = fminf((s.top - x[z]) * per, (float)(kFine - 1));  // NaN: the last
                    const int b = __float_as_int(d + kMagic) & (kFine - 1);
                    if (b < kFine - 1)
                        atomicAdd(&sh.orders[b], 1u);
                    else
                        ++behind;
                }
            });
            behind = __reduce_add_sync(0xffffffffu, behind);
            if (lane == 0 && behind) atomicAdd(&sh.orders[kFine - 1], behind);
            cluster_sync();
            // approximate weights in whole units of 2^-32: every CTA gets the same bracket
            constexpr int kPer = kFine / kThreads;
            const float least_x = sh.least;
            unsigned int n[kPer] = {};
            for (int c = 0; c < ctas; ++c) {
                const uint4* h = reinterpret_cast<const uint4*>(cluster.map_shared_rank(&sh.orders[0], c)) +
                                 tid * (kPer / 4);
#pragma unroll
                for (int z = 0; z < kPer / 4; ++z) {
                    const uint4 q = h[z];
                    n[4 * z] += q.x;
                    n[4 * z + 1] += q.y;
                    n[4 * z + 2] += q.z;
                    n[4 * z + 3] += q.w;
                }
            }
            unsigned long long w[kPer], mine = 0, total;
#pragma unroll
            for (int z = 0; z < kPer; ++z) {
                // (the last bin weighs nothing: far elements, and, whatever the bins' width,
                // -inf and NaN)
                const int b = tid * kPer + z;
                const float e = b < kFine - 1 ? 32.f - (float)b * (s.c * 0.0625f) / per : -1.f;
                w[z] = (unsigned long long)n[z] * (unsigned long long)exp2f(fmaxf(e, -1.f));
                mine += w[z];
            }
            if (tid == 0) {
                sh.bin = sh.base = kFine - 1;
                sh.good = 0;
            }
            unsigned long long at = block_sums(sh, mine, total) - mine;
            if (tid == 0) {
                // (the second term: what fp32 rounds)
                const float sum = (float)total, want = p * sum,
                            off = (1e-3f * fminf(p, 1.f - p) + 2.4e-7f) * sum;
                sh.want[0] = (unsigned long long)fmaxf(want - off, 0.f);
                sh.want[1] = (unsigned long long)fmaxf(want + off, 0.f);
                sh.want[2] = (unsigned long long)fmaxf(want * 0.98f, 0.f);
            }
            __syncthreads();
            const unsigned long long from_w = sh.want[0], to_w = sh.want[1], surely = sh.want[2];
            // where min-p cuts: a bin's weights are within 0.6 % of its middle's
            const int bin_m = (int)fminf((s.top - least_x) * per + 0.5f, (float)(kFine - 1));
#pragma unroll
            for (int z = 0; z < kPer; ++z) {
                const int b = tid * kPer + z;
                const unsigned long long end = at + w[z];
                if (end > from_w && at <= from_w) sh.bin = b;
                if (end > to_w && at <= to_w) sh.base = b;
                if (b == bin_m + 1 && at < surely) sh.good = 1;
                at = end;
            }
            __syncthreads();
            // a bin's border lies half a bin before it; one bin more on either side
            const int b0 = (int)sh.bin - 1, b1 = (int)sh.base + 1;
            hi = b0 > 0 ? s.top - ((float)b0 - 0.5f) / per : INFINITY;
            lo_x = b1 < kFine - 1 ? s.top - ((float)b1 + 0.5f) / per : logit_of(low);
            if (sh.good) border = false;
            __syncthreads();
        }
        if (!(p < 1.f)) __syncthreads();
        const float least_x = sh.least;
        summed = true;
        unsigned long long all = 0, above = 0, kept = 0;
        if (!border && least_x > -INFINITY) {
            // min-p's alone: the sum of the few that it keeps
            row.template vectors_of<2 * kBatch>(wlo, whi, [&](int, const float (&x)[VEC]) {
                if (row.most(x) >= least_x)
#pragma unroll 1
                    for (int z = 0; z < VEC; ++z) {
                        float y = x[0];
#pragma unroll
                        for (int k2 = 1; k2 < VEC; ++k2) y = z == k2 ? x[k2] : y;
                        if (y >= least_x) kept += fixed_of(sh.table, s, y);
                    }
            });
        } else {
            // exact sums: of the row, above the bracket (without one: all), and of what is
            // kept there
            // (above its own: least_x only matters where it lies above the bracket)
            const bool few = least_x > hi;
            auto add = [&](auto weight) {
                row.vectors_of(wlo, whi, [&](int v, const float (&x)[VEC]) {
#pragma unroll
                    for (int z = 0; z < VEC; ++z) {
                        const unsigned long long q = weight(x[z]);
                        if (x[z] > hi)
                            above += q;
                        else
                            all += q;
                        if (few && x[z] >= least_x) kept += q;
                        if (border && x[z] <= hi && x[z] >= lo_x &&
                            row.has(v * VEC - row.shift + z))
                            pick.note(v * VEC - row.shift + z, x[z]);
                    }
                });
            };
            if (s.fast)
                add([&](float x) { return fixed_fast(sh.table, s, x); });
            else
                add([&](float x) { return fixed_slow(sh.table, s, x); });
            all += above;
            if (!few) kept = above;
        }
        kept = warp_total(kept);
        all = warp_total(all);
        above = warp_total(above);
        __syncthreads();
        if (lane == 0) {
            sh.part_sum[warp] = kept;
            sh.warp_sum[warp] = all;
            sh.merged[warp] = above;  // before any CTA sends
        }
        __syncthreads();
        if (!border) {
            cut.key = order_of(least_x);
        } else {
            if (warp == 0) {
                const unsigned long long t = warp_total(lane < kWarps ? sh.warp_sum[lane] : 0);
                const unsigned long long b = warp_total(lane < kWarps ? sh.merged[lane] : 0);
                if (lane == 0) {
                    cluster.map_shared_rank(&sh.cta_sum[0], 0)[rank] = t;
                    cluster.map_shared_rank(&sh.cta_above[0], 0)[rank] = b;
                }
            }
            cluster_sync();  // everybody's use of `merged` is over
            pick.send();
            if (rank == 0) {
                unsigned long long total = 0, over = 0;
                for (int c = 0; c < ctas; ++c) {
                    total += sh.cta_sum[c];
                    over += sh.cta_above[c];
                }
                if (tid == 0) sh.want[0] = share_of(p, total);
                __syncthreads();
                const unsigned long long want = sh.want[0];
                const int n = (int)min(sh.n_merged, (unsigned int)kList);
                bool good = sh.n_merged <= kList && n > 0 && want > over;
                if (good) {
                    sort_falling(sh, n);
                    good = pick.finish(want - over, n, true, s);
                }
                if (tid < ctas) {
                    *cluster.map_shared_rank(&sh.good, tid) = good;
                    *cluster.map_shared_rank(&sh.cut, tid) = sh.cut;
                }
            }
            cluster_sync();
            summed = sh.good;
            if (summed) {
                // what the cut keeps of this CTA's part of the bracket
                cut = sh.cut;
                for (unsigned int i = tid; i < sh.n_list; i += kThreads) {
                    const uint32_t o = (uint32_t)(sh.list[i] >> 32);
                    const int at = (int)(0xffffffffu - (uint32_t)sh.list[i]);
                    if (cut.keeps(o, at) && logit_of(o) >= least_x)
                        atomicAdd(&sh.part_sum[((at + row.shift) / VEC - lo) / part],
                                  fixed_of(sh.table, s, logit_of(o)));
                }
            } else {
                pick.find(0u, p, cut, true, cut);
            }
            __syncthreads();
        }
    } else if (!whole && p < 1.f) {
        const Cut set = cut;
        cluster_sync();
        pick.find(0u, p, set, false, cut);
    }
    const float least_x = sh.least;
    if (whole && rank == 0) {
        // the first CTA draws, or adds up, in index order
        const int n = sh.found;
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) sh.list[i] = sh.merged[i];
        __syncthreads();
        for (int i = tid; i < n; i += kThreads)
            sh.merged[i] = sh.list[i] << 32 | (sh.list[i] >> 32);  // falling: indices rise
        __syncthreads();
        if (!kProbs) sort_falling(sh, n);
        unsigned long long w[kList / kThreads], mine = 0, total;
        const int per = (n + kThreads - 1) / kThreads, at0 = tid * per;
#pragma unroll
        for (int z = 0; z < kList / kThreads; ++z) {
            w[z] = 0;
            if (z < per && at0 + z < n) {
                const float x = logit_of((uint32_t)sh.merged[at0 + z]);
                w[z] = x >= least_x ? fixed_of(sh.table, s, x) : 0;
            }
            mine += w[z];
        }
        unsigned long long at = block_sums(sh, mine, total) - mine;
        if constexpr (kProbs) {
            if (tid < ctas) {
                *cluster.map_shared_rank(&sh.cut, tid) = sh.cut;
                *cluster.map_shared_rank(&sh.kept, tid) = total;
            }
        } else {
            if (tid == 0) sh.want[0] = part_of(u, total);
            __syncthreads();
            const unsigned long long want = sh.want[0];
#pragma unroll
            for (int z = 0; z < kList / kThreads; ++z) {
                if (at <= want && at + w[z] > want)
                    a.tokens[r] = (int)(0xffffffffu - (uint32_t)(sh.merged[at0 + z] >> 32));
                at += w[z];
            }
        }
    }
    if (!kProbs && whole) return;

    auto counted = [&](int i, float x) -> unsigned long long {
        return x >= least_x && cut.keeps(order_of(x), i) ? fixed_of(sh.table, s, x) : 0;
    };
    unsigned long long total = 0, before = 0;
    if (!whole) {
        // sums of what is kept, a warp and a CTA
        if (!summed) {
            unsigned long long sum = 0;
            row.each(wlo, whi, [&](int i, float x) { sum += counted(i, x); });
            sum = warp_total(sum);
            __syncthreads();
            if (lane == 0) sh.part_sum[warp] = sum;
            __syncthreads();
        }
        if (warp == 0) {
            const unsigned long long t = warp_total(lane < kWarps ? sh.part_sum[lane] : 0);
            if (lane < ctas) cluster.map_shared_rank(&sh.cta_sum[0], lane)[rank] = t;
        }
        cluster_sync();
        for (int c = 0; c < ctas; ++c) {
            if (c < rank) before += sh.cta_sum[c];
            total += sh.cta_sum[c];
        }
    } else {
        cluster_sync();
        cut = sh.cut;
        total = sh.kept;
    }
    if constexpr (kProbs) {
        // one over the sum, corrected by what the quotient and fp32 of the sum leave
        const float sum = (float)total, left = (float)(long long)(total - (unsigned long long)sum);
        const float near = __fdiv_rn((float)kOne, sum);
        const float inv = __fmaf_rn(
            __fmaf_rn(-near, left, __fmaf_rn(-near, sum, (float)kOne)), __fdividef(1.f, sum), near);
        const float from_x = fmaxf(least_x, logit_of(max(cut.key, kLowest)));
        row.vectors_of(wlo, whi, [&](int v, const float (&x)[VEC]) {
            float y[VEC];
#pragma unroll
            for (int z = 0; z < VEC; ++z) {
                y[z] = 0.f;
                if (x[z] >= from_x && cut.keeps(order_of(x[z]), v * VEC - row.shift + z))
                    y[z] = weight_of(sh.table, s, x[z]) * inv;
            }
            put(v, y);
        });
        return;
    }
    if (tid == 0) sh.want[0] = part_of(u, total);
    __syncthreads();
    const unsigned long long want = sh.want[0];
    if (want < before || want >= before + sh.cta_sum[rank]) return;
    // in this CTA: the warp's part, a sixteenth of it a warp, then in order
    unsigned long long at = before;
    int w = 0;
    while (w < kWarps - 1 && at + sh.part_sum[w] <= want) at += sh.part_sum[w++];
    const int plo = min(lo + w * part, hi), phi = min(plo + part, hi);
    const int sub = (phi - plo + kWarps - 1) / kWarps;
    unsigned long long sum2 = 0;
    row.each(min(plo + warp * sub, phi), min(plo + (warp + 1) * sub, phi),
             [&](int i, float x) { sum2 += counted(i, x); });
    sum2 = warp_total(sum2);
    if (lane == 0) sh.warp_sum[warp] = sum2;
    __syncthreads();
    if (warp != 0) return;
    w = 0;
    while (w < kWarps - 1 && at + sh.warp_sum[w] <= want) at += sh.warp_sum[w++];
    const int slo = min(plo + w * sub, phi), shi = min(slo + sub, phi);
    for (int v0 = slo; v0 < shi; v0 += 32) {
        const uint4 x = row.load(v0 + lane, shi);
        const Elem* e = reinterpret_cast<const Elem*>(&x);
        const int i = (v0 + lane) * VEC - row.shift;
        unsigned long long c[VEC], mine = 0;
#pragma unroll
        for (int z = 0; z < VEC; ++z) {
            c[z] = v0 + lane < shi && row.has(i + z) ? counted(i + z, as_logit(e[z])) : 0;
            mine += c[z];
        }
        unsigned long long inc = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const unsigned long long o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        unsigned long long run = at + inc - mine;
#pragma unroll
        for (int z = 0; z < VEC; ++z) {
            if (run <= want && run + c[z] > want) a.tokens[r] = i + z;
            run += c[z];
        }
        at += __shfl_sync(0xffffffffu, inc, 31);
    }
}

template <typename Elem>
cudaError_t go_sample(const SampleArgs& a, cudaStream_t stream) {
    Table t;
    for (int j = 0; j < 16; ++j) {
        const double x = exp2(j / 16.0);
        const float y = (float)(x * 2147483648.0);
        t.fixed[j].x = (uint32_t)(unsigned long long)(x * 2147483648.0 + 0.5);
        memcpy(&t.fixed[j].y, &y, 4);
        t.low[j] = (float)(x - (double)(float)x);
    }
    // CTAs a row: while two an SM are not passed, with 2048 elements a CTA at least; a
    // share of 2^17 at most, so that a bin's words of 14 bits hold its sums
    int ctas = 1;
    while (ctas < kMaxCtas && ((2 * ctas * (long long)a.R <= 2 * kServingSMs &&
                                a.V / (2 * ctas) >= 4 * kThreads) ||
                               a.V / ctas > (1 << 17) - 64))
        ctas *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.R * ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = stream;
    auto kernel = a.tokens ? sample_kernel<Elem, false> : sample_kernel<Elem, true>;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared));
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a, t);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, kvd_dtype dt, cudaStream_t stream) {
    return dt == KVD_BF16 ? go_sample<__nv_bfloat16>(a, stream) : go_sample<float>(a, stream);
}

}  // namespace kvd
