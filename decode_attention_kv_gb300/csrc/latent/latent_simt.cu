// latent_simt.cu -- attention over latent caches and expanded rows in fp32, on
// CUDA cores, and the merge of partial rows.
//
// One tile is 16 query rows x 32 keys in shared memory; the next tile's keys
// arrive by cp.async meanwhile (two buffers).  Scores: 4 slices of the inner
// dimension x 64 threads, each 4 rows x 2 keys, so six 16-byte shared loads feed
// 16 packed multiply-adds (32 products).  Softmax: 16 threads a row keep the
// running max and sum.  Values: a thread owns 4 dims x RPT rows.
#include "../kvd_internal.h"
#include "latent_common.cuh"
#include "tcgen05_ptx.cuh"  // bar_sync

namespace kvd {
namespace {

constexpr int kThreads = 256;  // of a group: one tile of keys at a time
constexpr int kGroups = 2;     // groups of a CTA of the expanded form, every other tile each
constexpr int kRowsLog = 4, kRows = 1 << kRowsLog;  // query rows per tile
constexpr int kKeys = 32;   // keys per tile

// Row strides of the scores [slice, row, key] and of the weights [key, row]: no
// bank conflicts where 16 threads read a row's scores, two-way where they write
// its weights (8-way both at strides of 32 and 16).
constexpr int kSs = kKeys + 1, kPs = kRows + 4;

// Shared memory of one CTA, in floats.
struct SimtLayout {
    int qs, q, k, v, s, p, total;  // qs: padded row stride of q and k
    int ks, vs;                    // floats of a key buffer, row stride of v
    int vb;                        // floats of a value buffer (0: the keys are the values)
    int group;                     // floats of a group (k, v, s, p; group 0's are given)
    __host__ __device__ SimtLayout(int D, int Dv, bool own_v, int groups) {
        qs = D + 4;
        ks = kKeys * qs;
        vs = own_v ? Dv : qs;
        vb = own_v ? kKeys * Dv : 0;
        q = 0;
        k = q + kRows * qs;
        v = k + 2 * ks;
        s = v + 2 * vb;
        p = s + 4 * kRows * kSs;
        group = p + kKeys * kPs + kRows - k;
        total = k + groups * group;
    }
};

// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy16(float* dst, const float* src, bool some) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
                 "r"(some ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the newest N groups
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A row of `n` floats (a multiple of 4), by one warp.
__device__ __forceinline__ void copy_row(float* dst, const float* src, int n, bool some) {
    for (int c = 4 * (threadIdx.x & 31); c < n; c += 128) copy16(dst + c, src + c, some);
}

// Running state of one tile of rows, advanced one tile of keys at a time.
template <int RPT>
struct RowState {
    float2 acc[RPT][2];
    float m, l;  // of softmax row tid / 16

    __device__ void clear() {
#pragma unroll
        for (int i = 0; i < RPT; ++i) acc[i][0] = acc[i][1] = make_float2(0.f, 0.f);
        m = -INFINITY;
        l = 0.f;
    }

    // kt, vt: the tile's keys and values.  last: the newest key (index in the
    // tile) that softmax row tid / 16 sees.  valid: one bit per key of the tile.
    // sm: the group's shared memory; q: the queries; tid: the thread of the group;
    // bar: its barrier.
    __device__ void step(float* sm, const SimtLayout& L, const float* queries, const float* keys,
                         const float* vals, int tid, int bar, int D, int Dv, float qscale, int last,
                         uint32_t valid) {
        {
            const int slice = tid >> 6, u = tid & 63, rt = u >> 4, kt = u & 15;
            const int per = D / 4;  // D is a multiple of 64
            const float* q = queries + 4 * rt * L.qs + slice * per;
            const float* k = keys + kt * L.qs + slice * per;
            float2 s[4][2] = {};
#pragma unroll 2
            for (int j = 0; j < per; j += 4) {
                float4 kx[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    kx[i] = *reinterpret_cast<const float4*>(k + 16 * i * L.qs + j);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float4 qx = *reinterpret_cast<const float4*>(q + r * L.qs + j);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        s[r][i] = ffma2(make_float2(qx.x, qx.y), make_float2(kx[i].x, kx[i].y),
                                        ffma2(make_float2(qx.z, qx.w),
                                              make_float2(kx[i].z, kx[i].w), s[r][i]));
                }
            }
            float* to = sm + L.s + (slice * kRows + 4 * rt) * kSs + kt;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i) to[r * kSs + 16 * i] = s[r][i].x + s[r][i].y;
        }
        bar_sync(bar, kThreads);
        {
            const int row = tid >> 4, c = tid & 15;
            float x[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int key = c + 16 * i;
                float s = 0.f;
#pragma unroll
                for (int z = 0; z < 4; ++z) s += sm[L.s + (z * kRows + row) * kSs + key];
                x[i] = (key <= last && ((valid >> key) & 1u)) ? s * qscale : -INFINITY;
            }
            float mx = fmaxf(x[0], x[1]);
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float mn = fmaxf(m, mx);
            const float base = mn == -INFINITY ? 0.f : mn;
            const float corr = exp2f(m - base);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float p = exp2f(x[i] - base);
                sum += p;
                sm[L.p + (c + 16 * i) * kPs + row] = p;
            }
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            l = l * corr + sum;
            m = mn;
            if (c == 0) sm[L.p + kKeys * kPs + row] = corr;
        }
        bar_sync(bar, kThreads);
        {
            const int dgs = Dv / 4, dg = tid % dgs, rg = tid / dgs;
            if (rg < kRows / RPT) {
                const float* corr = sm + L.p + kKeys * kPs + rg * RPT;
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const float2 c = make_float2(corr[i], corr[i]);
                    acc[i][0] = fmul2(acc[i][0], c);
                    acc[i][1] = fmul2(acc[i][1], c);
                }
                const float* v = vals + 4 * dg;
                const float* p = sm + L.p + rg * RPT;
#pragma unroll 4
                for (int k = 0; k < kKeys; ++k) {
                    const float4 x = *reinterpret_cast<const float4*>(v + k * L.vs);
                    float w[RPT];
                    if constexpr (RPT % 4 == 0) {
#pragma unroll
                        for (int i = 0; i < RPT; i += 4)
                            *reinterpret_cast<float4*>(w + i) =
                                *reinterpret_cast<const float4*>(p + k * kPs + i);
                    } else {
#pragma unroll
                        for (int i = 0; i < RPT; ++i) w[i] = p[k * kPs + i];
                    }
#pragma unroll
                    for (int i = 0; i < RPT; ++i) {
                        const float2 ww = make_float2(w[i], w[i]);
                        acc[i][0] = ffma2(ww, make_float2(x.x, x.y), acc[i][0]);
                        acc[i][1] = ffma2(ww, make_float2(x.z, x.w), acc[i][1]);
                    }
                }
            }
        }
        bar_sync(bar, kThreads);
    }

    // Leaves every row's sum and max in the group's shared memory: sm[s + row],
    // sm[s + 16 + row].  Called by the whole CTA.
    __device__ void publish(float* sm, const SimtLayout& L, int tid) {
        if ((tid & 15) == 0) {
            sm[L.s + (tid >> 4)] = l;
            sm[L.s + kRows + (tid >> 4)] = m;
        }
        __syncthreads();
    }

    // This thread's 4 dims of its row i, divided by the row's sum.
    __device__ float4 result(const float* sm, const SimtLayout& L, int r, int i) const {
        const float sum = sm[L.s + r];
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        return make_float4(acc[i][0].x * inv, acc[i][0].y * inv, acc[i][1].x * inv,
                           acc[i][1].y * inv);
    }
};

__device__ __forceinline__ float lse2_of(float m, float l) {
    return l > 0.f ? m + log2f(l) : (l == 0.f ? -INFINITY : NAN);
}

template <int RPT>
__global__ void __launch_bounds__(kThreads) latent_simt_kernel(const LatentArgs a) {
    extern __shared__ __align__(16) float sm[];
    __shared__ int scratch[kFindWords];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = blockIdx.x, w = blockIdx.y;
    const int D = a.R + a.P;
    const SimtLayout L(D, a.R, false, 1);
    const float* latent = static_cast<const float*>(a.latent);
    const float* rope = static_cast<const float*>(a.rope);
    Runs runs;
    uint32_t refused = 0;
    const Found f = block_find_strided<kThreads>(
        a.Q, scratch,
        [&](int tot) {
            runs = Runs(tot, used_workers(a, tot));
            return w < runs.W ? runs.start(w) : tot;
        },
        [&](int b) {
            const SeqInfo s = latent_seq(a, b);
            refused |= s.bad;
            return a.lead + max(1, (s.n + kKeys - 1) / kKeys);
        });
    if (refused && g == 0 && w == 0) report(a.dev_status, refused);
    if (f.item >= a.Q) return;
    const int t0 = runs.start(w), t1 = runs.start(w + 1);
    const int row0 = g * a.rpg, nrows = min(a.rpg, a.rows - row0);
    int b = f.item, before = f.before;
    RowState<RPT> st;
    for (int t = t0; t < t1; ++b) {
        const SeqInfo seq = latent_seq(a, b);
        const int nt = max(1, (seq.n + kKeys - 1) / kKeys);
        // the run's part of the sequence's places: `lead` of them, then its tiles
        const int first = max(0, t - before - a.lead), end = min(nt, t1 - before - a.lead);
        if (end <= first) break;  // the run ends before the first tile
        // Starts the copies of tile k into buffer `buf` and returns its valid keys
        // (lane: the key); a warp brings every eighth of them.
        auto fetch = [&](int k, int buf) {
            const int key = k * kKeys + lane;
            long long row = -1;
            if (key < seq.n) {
                const int page = a.by_page(key);
                const int phys = a.block_tables[(size_t)b * a.cols + seq.col0 + page];
                if (phys >= 0 && phys < a.NB)
                    row = (long long)phys * a.BS + key - page * a.BS;
                else if (warp == 0)
                    report(a.dev_status, KVD_DEV_BLOCK_RANGE);
            }
#pragma unroll
            for (int i = 0; i < kKeys / 8; ++i) {
                const int r = warp + 8 * i;
                const long long from = __shfl_sync(0xffffffffu, row, r);
                float* to = sm + L.k + buf * L.ks + r * L.qs;
                const size_t at = from < 0 ? 0 : (size_t)from;
                copy_row(to, latent + at * a.R, a.R, from >= 0);
                copy_row(to + a.R, rope + at * a.P, a.P, from >= 0);
            }
            return __ballot_sync(0xffffffffu, row >= 0);
        };
        // the group's queries, with the first tile
#pragma unroll
        for (int i = 0; i < kRows / 8; ++i) {
            const int r = warp + 8 * i;
            const size_t row = (size_t)b * a.rows + row0 + min(r, nrows - 1);
            copy_row(sm + L.q + r * L.qs, static_cast<const float*>(a.q_latent) + row * a.R, a.R,
                     r < nrows);
            copy_row(sm + L.q + r * L.qs + a.R, static_cast<const float*>(a.q_rope) + row * a.P,
                     a.P, r < nrows);
        }
        uint32_t valid = fetch(first, 0);
        copies_commit();
        st.clear();
        const int srow = tid >> 4;
        // newest key the softmax row sees
        const int last = srow < nrows ? seq.n - a.T + a.by_head(row0 + srow) : -1;
        for (int k = first; k < end; ++k) {
            const int buf = (k - first) & 1;
            uint32_t next = 0;
            if (k + 1 < end) next = fetch(k + 1, buf ^ 1);
            copies_commit();
            copies_wait<1>();
            __syncthreads();
            const float* keys = sm + L.k + buf * L.ks;
            st.step(sm, L, sm + L.q, keys, keys, tid, 1, D, a.R, a.qscale, last - k * kKeys, valid);
            valid = next;
        }
        st.publish(sm, L, tid);
        const bool whole = first == 0 && end == nt;
        const size_t slot = ((size_t)w * a.groups + g) * 2 + (t == t0 ? 0 : 1);
        const int dgs = a.R / 4, dg = tid % dgs, rg = tid / dgs;
        if (rg < kRows / RPT) {
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const int r = rg * RPT + i;
                if (r < nrows) {
                    const size_t row = (size_t)b * a.rows + row0 + r;
                    float* to = whole ? static_cast<float*>(a.out) + row * a.R
                                      : a.part_o + (slot * a.rpg + r) * a.R;
                    *reinterpret_cast<float4*>(to + 4 * dg) = st.result(sm, L, r, i);
                }
            }
        }
        if (tid < nrows) {
            const float z = lse2_of(sm[L.s + kRows + tid], sm[L.s + tid]);
            if (!whole)
                a.part_lse[slot * a.rpg + tid] = z;
            else if (a.lse_out)
                a.lse_out[(size_t)b * a.rows + row0 + tid] = z * kLn2;
        }
        if (g == 0 && tid == 0 && first == 0)
            a.meta[b] = make_int4(w, runs.worker_of(before + a.lead + nt - 1),
                                  t == t0 ? 0 : 1, 0);
        __syncthreads();
        before += a.lead + nt;
        t = before;
    }
}

template <int RPT>
__global__ void __launch_bounds__(kGroups * kThreads) expanded_simt_kernel(const ExpandedArgs a) {
    extern __shared__ __align__(16) float smem[];
    __shared__ int scratch[kFindWords];
    pdl_launch_dependents();
    pdl_wait();
    // tid, warp: of the group
    const int group = threadIdx.x / kThreads, tid = threadIdx.x % kThreads, warp = tid >> 5;
    const int h = blockIdx.y, unit = blockIdx.x;
    const int D = a.Dn + a.P;
    const SimtLayout L(D, a.Dv, true, kGroups);
    float* sm = smem + group * L.group;
    const Found f = packed_find<kGroups * kThreads>(a, scratch, unit, kRowsLog, h == 0 && unit == 0);
    if (f.item >= a.Q) return;
    const PackedSeq seq = packed_seq(a, f.item);
    if (seq.nq == 0) return;
    // the last rows of a sequence first: under the causal mask they see most keys
    const int units = (seq.nq + kRows - 1) / kRows;
    const int row0 = (units - 1 - (unit - f.before)) * kRows, nrows = min(kRows, seq.nq - row0);
    const float* kv = static_cast<const float*>(a.kv);
    const float* rope = static_cast<const float*>(a.k_rope);
    const int shift = a.causal ? seq.nk - seq.nq : seq.nk - 1;
    const int srow = tid >> 4;
    const int last = srow < nrows ? (a.causal ? row0 + srow + shift : shift) : -1;
    const int nkeys = a.causal ? min(seq.nk, row0 + nrows + shift) : seq.nk;
    // Starts the copies of the keys from k0 on into buffer `buf`: a warp every
    // eighth key, a lane 16 bytes of each part of it (parts are at most 128 floats).
    const int lane = tid & 31, c4 = 4 * lane;
    const size_t stride = (size_t)a.H * (a.Dn + a.Dv);
    const float* kv_lane = kv + ((size_t)seq.k0 * a.H + h) * (a.Dn + a.Dv) + c4;
    const float* rope_lane = rope + (size_t)seq.k0 * a.P + c4;
    auto fetch = [&](int k0, int buf) {
        float* kd = sm + L.k + buf * L.ks + warp * L.qs + c4;
        float* vd = sm + L.v + buf * L.vb + warp * L.vs + c4;
#pragma unroll
        for (int i = 0; i < kKeys / 8; ++i) {
            const int r = k0 + warp + 8 * i;
            const bool some = r < nkeys;
            const float* row = kv_lane + (some ? r : 0) * stride;
            if (c4 < a.Dn) copy16(kd + 8 * i * L.qs, row, some);
            if (c4 < a.P)
                copy16(kd + 8 * i * L.qs + a.Dn, rope_lane + (size_t)(some ? r : 0) * a.P, some);
            if (c4 < a.Dv) copy16(vd + 8 * i * L.vs, row + a.Dn, some);
        }
    };
    for (int r = threadIdx.x >> 5; r < kRows; r += kGroups * kThreads / 32)
        copy_row(smem + L.q + r * L.qs,
                 static_cast<const float*>(a.q) +
                     ((size_t)(seq.q0 + row0 + min(r, nrows - 1)) * a.H + h) * D,
                 D, r < nrows);
    constexpr int kStride = kGroups * kKeys;
    const int first = group * kKeys;
    if (first < nkeys) fetch(first, 0);
    copies_commit();
    copies_wait<0>();
    __syncthreads();
    RowState<RPT> st;
    st.clear();
    for (int k0 = first; k0 < nkeys; k0 += kStride) {
        const int buf = (k0 / kStride) & 1, n = min(kKeys, nkeys - k0);
        if (k0 + kStride < nkeys) fetch(k0 + kStride, buf ^ 1);
        copies_commit();
        copies_wait<1>();
        bar_sync(1 + group, kThreads);
        st.step(sm, L, smem + L.q, sm + L.k + buf * L.ks, sm + L.v + buf * L.vb, tid, 1 + group, D,
                a.Dv, a.qscale, last - k0, n == 32 ? ~0u : (1u << n) - 1u);
    }
    copies_wait<0>();
    __syncthreads();
    // the groups' rows by their maxima: the second leaves its own where its keys were
    const int dgs = a.Dv / 4, dg = tid % dgs, rg = tid / dgs;
    float4* other = reinterpret_cast<float4*>(smem + L.group + L.k);
    st.publish(sm, L, tid);
    if (group == 1 && rg < kRows / RPT) {
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            other[(rg * RPT + i) * dgs + dg] = make_float4(st.acc[i][0].x, st.acc[i][0].y,
                                                           st.acc[i][1].x, st.acc[i][1].y);
    }
    __syncthreads();
    if (group == 1) return;
    const float* sum0 = smem + L.s;
    const float* sum1 = smem + L.group + L.s;
    auto merged = [&](int r, float& c0, float& c1, float& m) {
        const float m0 = sum0[kRows + r], m1 = sum1[kRows + r];
        m = fmaxf(m0, m1);
        const float base = m == -INFINITY ? 0.f : m;
        c0 = exp2f(m0 - base);
        c1 = exp2f(m1 - base);
        return sum0[r] * c0 + sum1[r] * c1;
    };
    float c0, c1, m;
    if (rg < kRows / RPT) {
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int r = rg * RPT + i;
            if (r < nrows) {
                const float l = merged(r, c0, c1, m), inv = l == 0.f ? 0.f : 1.f / l;
                const float4 o = other[r * dgs + dg];
                *reinterpret_cast<float4*>(static_cast<float*>(a.out) +
                                           ((size_t)(seq.q0 + row0 + r) * a.H + h) * a.Dv + 4 * dg) =
                    make_float4((st.acc[i][0].x * c0 + o.x * c1) * inv,
                                (st.acc[i][0].y * c0 + o.y * c1) * inv,
                                (st.acc[i][1].x * c0 + o.z * c1) * inv,
                                (st.acc[i][1].y * c0 + o.w * c1) * inv);
            }
        }
    }
    if (tid < nrows && a.lse_out) {
        const float l = merged(tid, c0, c1, m);
        a.lse_out[(size_t)(seq.q0 + row0 + tid) * a.H + h] = lse2_of(m, l) * kLn2;
    }
}

// A CTA a row: the workers' partial rows by log-sum-exp.  R / 128 warps share the
// dims, and as many sets of them as fit share the workers (every other one, every
// fourth ..): with one warp for 65 partial rows of 128 dims the merge of a short
// fp32 call took longer than its attention.  Few rows take 8 warps each (kWide);
// many take one set of warps, no shared memory and few registers, so that CTAs fit
// beside the attention and wait there for its end (2048 rows of 512: 92 us with the
// attention, 99 at 8 warps; 48 rows of 256: 23 us and 16).
template <typename Out, bool kWide>
__global__ void __launch_bounds__(kWide ? 256 : 128) latent_combine_kernel(const LatentArgs a) {
    constexpr int kMergeWarps = kWide ? 8 : 4, kBatch = kWide ? 8 : 4;
    pdl_launch_dependents();
    pdl_wait();
    const int b = blockIdx.y;
    const int4 meta = a.meta[b];
    const int w0 = meta.x, w1 = meta.y;
    if (w0 == w1) return;
    // a launch that gave up on a wait may have left no division behind
    if (w0 < 0 || w1 < w0 || w1 >= a.workers || (meta.z & ~1)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cols = a.R / 128, sets = kWide ? kMergeWarps / cols : 1, set = warp / cols;
    if (!kWide && set > 0) return;
    const int row = blockIdx.x, g = row / a.rpg, r = row % a.rpg;
    const int d = 128 * (warp % cols) + 4 * lane;
    const float* base_o = a.part_o + d;
    float M = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    // a lane a worker: its log-sum-exp, then its weight; up to 32 workers of the set
    // at a time against a running maximum
    for (int wb = w0 + set; set < sets && wb <= w1; wb += 32 * sets) {
        const int w = wb + lane * sets, n = min(32, (w1 - wb) / sets + 1);
        const int slot = (w * a.groups + g) * 2 + (w == w0 ? meta.z : 0);
        const float z = w <= w1 ? a.part_lse[(size_t)slot * a.rpg + r] : -INFINITY;
        // the first rows are on their way before the weights are known
        float4 x[kBatch];
        auto load = [&](int i0) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int sl = __shfl_sync(0xffffffffu, slot, min(i0 + i, n - 1));
                x[i] = i0 + i < n ? *reinterpret_cast<const float4*>(
                                        base_o + ((size_t)sl * a.rpg + r) * a.R)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        };
        load(0);
        float top = z;
#pragma unroll
        for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        top = fmaxf(top, M);
        const float base = top == -INFINITY ? 0.f : top;
        const float corr = exp2f(M - base), e = exp2f(z - base);
        M = top;
        l *= corr;
        acc.x *= corr;
        acc.y *= corr;
        acc.z *= corr;
        acc.w *= corr;
        for (int i0 = 0; i0 < n; i0 += kBatch) {
            float f[kBatch];
            if (i0 > 0) load(i0);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                f[i] = __shfl_sync(0xffffffffu, e, min(i0 + i, n - 1));
                if (i0 + i >= n) f[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                l += f[i];
                acc.x = fmaf(f[i], x[i].x, acc.x);
                acc.y = fmaf(f[i], x[i].y, acc.y);
                acc.z = fmaf(f[i], x[i].z, acc.z);
                acc.w = fmaf(f[i], x[i].w, acc.w);
            }
        }
    }
    if constexpr (kWide) {
        __shared__ float4 part[kMergeWarps][32];
        __shared__ float part_m[kMergeWarps], part_l[kMergeWarps];
        part[warp][lane] = acc;
        if (lane == 0) {
            part_m[warp] = M;
            part_l[warp] = l;
        }
        __syncthreads();
        if (set != 0) return;
        for (int k = 1; k < sets; ++k) M = fmaxf(M, part_m[warp + k * cols]);
        const float top = M == -INFINITY ? 0.f : M;
        l = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < sets; ++k) {
            const float c = exp2f(part_m[warp + k * cols] - top);
            const float4 x = part[warp + k * cols][lane];
            l = fmaf(c, part_l[warp + k * cols], l);
            acc.x = fmaf(c, x.x, acc.x);
            acc.y = fmaf(c, x.y, acc.y);
            acc.z = fmaf(c, x.z, acc.z);
            acc.w = fmaf(c, x.w, acc.w);
        }
    }
    const float base = M == -INFINITY ? 0.f : M;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const size_t at = (size_t)b * a.rows + row;
    ElemTraits<Out>::store4(a.out, at * a.R + d,
                            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    if (d == 0 && a.lse_out) a.lse_out[at] = lse2_of(base, l) * kLn2;
}

template <int RPT>
cudaError_t go_latent(const LatentArgs& a, cudaStream_t stream) {
    const SimtLayout L(a.R + a.P, a.R, false, 1);
    const int smem = L.total * 4;
    const cudaError_t e = cudaFuncSetAttribute(
        latent_simt_kernel<RPT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(latent_simt_kernel<RPT>, dim3(a.groups, a.workers), dim3(kThreads), smem,
                      stream, a);
}

template <int RPT>
cudaError_t go_expanded(const ExpandedArgs& a, cudaStream_t stream) {
    const SimtLayout L(a.Dn + a.P, a.Dv, true, kGroups);
    const int smem = L.total * 4;
    const cudaError_t e = cudaFuncSetAttribute(
        expanded_simt_kernel<RPT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int units = (a.Nq + kRows - 1) / kRows + a.Q;
    return launch_pdl(expanded_simt_kernel<RPT>, dim3(units, a.H), dim3(kGroups * kThreads), smem,
                      stream, a);
}

}  // namespace

cudaError_t launch_latent_simt(const LatentArgs& a, cudaStream_t stream) {
    if (a.R > 256) return go_latent<8>(a, stream);
    if (a.R > 128) return go_latent<4>(a, stream);
    return go_latent<2>(a, stream);
}

cudaError_t launch_expanded_simt(const ExpandedArgs& a, cudaStream_t stream) {
    return a.Dv == 128 ? go_expanded<2>(a, stream) : go_expanded<1>(a, stream);
}

template <typename Out>
static cudaError_t go_combine(const LatentArgs& a, cudaStream_t stream) {
    const dim3 grid(a.rows, a.Q);
    if ((long long)a.rows * a.Q <= 2 * kLatentSMs)
        return launch_pdl(latent_combine_kernel<Out, true>, grid, dim3(256), 0, stream, a);
    return launch_pdl(latent_combine_kernel<Out, false>, grid, dim3(128), 0, stream, a);
}

cudaError_t launch_latent_combine(const LatentArgs& a, kvd_dtype dt, cudaStream_t stream) {
    return dt == KVD_BF16 ? go_combine<__nv_bfloat16>(a, stream) : go_combine<float>(a, stream);
}

}  // namespace kvd
