// latent_simt.cu -- attention over latent caches on CUDA cores.
//
// One tile is 16 query rows x 32 keys, both in fp32 shared memory.  Scores:
// 4 slices of the inner dimension x 64 threads, each 4 rows x 2 keys, so six
// 16-byte shared loads feed 32 fused multiply-adds.  Softmax: 16 threads a row
// keep the running max and sum.  Values: a thread owns 4 dims x RPT rows.
#include "kvd_internal.h"
#include "latent_common.cuh"

namespace kvd {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 16;   // query rows per tile
constexpr int kKeys = 32;   // keys per tile

// Shared memory of one CTA, in floats.
struct SimtLayout {
    int qs, q, k, v, s, p, total;  // qs: padded row stride of q and k
    int vs;                        // row stride of v
    __host__ __device__ SimtLayout(int D, int Dv, bool own_v) {
        qs = D + 4;
        q = 0;
        k = q + kRows * qs;
        vs = own_v ? Dv : qs;
        v = own_v ? k + kKeys * qs : k;
        s = k + kKeys * qs + (own_v ? kKeys * Dv : 0);
        p = s + 4 * kKeys * kRows;
        total = p + kKeys * kRows + 2 * kRows;
    }
};

template <typename Elem>
__device__ __forceinline__ float4 load4(const Elem* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
    return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    const float2 a = bf16x2_to_float2(w.x), b = bf16x2_to_float2(w.y);
    return make_float4(a.x, a.y, b.x, b.y);
}

// Running state of one tile of rows, advanced one tile of keys at a time.
template <int RPT>
struct RowState {
    float4 acc[RPT];
    float m, l;  // of softmax row tid / 16

    __device__ void clear() {
#pragma unroll
        for (int i = 0; i < RPT; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        m = -INFINITY;
        l = 0.f;
    }

    // last: the newest key (index in the tile) that softmax row tid / 16 sees.
    // valid: one bit per key of the tile.
    __device__ void step(float* sm, const SimtLayout& L, int D, int Dv, float qscale, int last,
                         uint32_t valid) {
        const int tid = threadIdx.x;
        {
            const int slice = tid >> 6, u = tid & 63, rt = u >> 4, kt = u & 15;
            const int per = D / 4;  // D is a multiple of 64
            const float* q = sm + L.q + 4 * rt * L.qs + slice * per;
            const float* k = sm + L.k + kt * L.qs + slice * per;
            float s[4][2] = {};
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
                        s[r][i] = fmaf(qx.x, kx[i].x,
                                       fmaf(qx.y, kx[i].y,
                                            fmaf(qx.z, kx[i].z, fmaf(qx.w, kx[i].w, s[r][i]))));
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<float4*>(sm + L.s + (slice * kKeys + kt + 16 * i) * kRows + 4 * rt) =
                    make_float4(s[0][i], s[1][i], s[2][i], s[3][i]);
        }
        __syncthreads();
        {
            const int row = tid >> 4, c = tid & 15;
            float x[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int key = c + 16 * i;
                float s = 0.f;
#pragma unroll
                for (int z = 0; z < 4; ++z) s += sm[L.s + (z * kKeys + key) * kRows + row];
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
                sm[L.p + (c + 16 * i) * kRows + row] = p;
            }
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            l = l * corr + sum;
            m = mn;
            if (c == 0) sm[L.p + kKeys * kRows + row] = corr;
        }
        __syncthreads();
        {
            const int dgs = Dv / 4, dg = tid % dgs, rg = tid / dgs;
            if (rg < kRows / RPT) {
                const float* corr = sm + L.p + kKeys * kRows + rg * RPT;
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    acc[i].x *= corr[i];
                    acc[i].y *= corr[i];
                    acc[i].z *= corr[i];
                    acc[i].w *= corr[i];
                }
                const float* v = sm + L.v + 4 * dg;
                const float* p = sm + L.p + rg * RPT;
                for (int k = 0; k < kKeys; ++k) {
                    const float4 x = *reinterpret_cast<const float4*>(v + k * L.vs);
#pragma unroll
                    for (int i = 0; i < RPT; ++i) {
                        const float w = p[k * kRows + i];
                        acc[i].x = fmaf(w, x.x, acc[i].x);
                        acc[i].y = fmaf(w, x.y, acc[i].y);
                        acc[i].z = fmaf(w, x.z, acc[i].z);
                        acc[i].w = fmaf(w, x.w, acc[i].w);
                    }
                }
            }
        }
        __syncthreads();
    }

    // Leaves every row's sum and max in shared memory: sm[s + row], sm[s + 16 + row].
    __device__ void publish(float* sm, const SimtLayout& L) {
        const int tid = threadIdx.x;
        if ((tid & 15) == 0) {
            sm[L.s + (tid >> 4)] = l;
            sm[L.s + kRows + (tid >> 4)] = m;
        }
        __syncthreads();
    }
};

__device__ __forceinline__ float lse2_of(float m, float l) {
    return l > 0.f ? m + log2f(l) : (l == 0.f ? -INFINITY : NAN);
}

template <typename Elem, int RPT>
__global__ void __launch_bounds__(kThreads) latent_simt_kernel(const LatentArgs a) {
    extern __shared__ __align__(16) float sm[];
    __shared__ int scratch[kFindWords];
    __shared__ long long rows_of[kKeys];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, g = blockIdx.x, w = blockIdx.y;
    const int D = a.R + a.P;
    const SimtLayout L(D, a.R, false);
    int W = 1;
    Found f = block_find<kThreads>(
        a.Q, scratch,
        [&](int tot) {
            W = used_workers(a, tot);
            return w < W ? run_start(w, tot, W) : tot;
        },
        [&](int b) {
            const SeqInfo s = latent_seq(a, b);
            if (s.bad && g == 0 && w == 0) report(a.dev_status, s.bad);
            return a.lead + max(1, (s.n + kKeys - 1) / kKeys);
        });
    if (f.item >= a.Q) return;
    const int t0 = run_start(w, f.total, W), t1 = run_start(w + 1, f.total, W);
    const int row0 = g * a.rpg, nrows = min(a.rpg, a.rows - row0);
    int b = f.item, before = f.before;
    RowState<RPT> st;
    for (int t = t0; t < t1; ++b) {
        const SeqInfo seq = latent_seq(a, b);
        const int nt = max(1, (seq.n + kKeys - 1) / kKeys);
        // the run's part of the sequence's places: `lead` of them, then its tiles
        const int first = max(0, t - before - a.lead), end = min(nt, t1 - before - a.lead);
        if (end <= first) break;  // the run ends before the first tile
        // the group's queries
        for (int i = tid; i < kRows * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = 4 * (i % (D / 4));
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < nrows) {
                const size_t row = (size_t)b * a.rows + row0 + r;
                x = c < a.R ? load4(static_cast<const Elem*>(a.q_latent) + row * a.R + c)
                            : load4(static_cast<const Elem*>(a.q_rope) + row * a.P + (c - a.R));
            }
            *reinterpret_cast<float4*>(sm + L.q + r * L.qs + c) = x;
        }
        st.clear();
        const int srow = tid >> 4;
        // newest key the softmax row sees
        const int last = srow < nrows ? seq.n - a.T + (row0 + srow) / a.H : -1;
        for (int k = first; k < end; ++k) {
            if (tid < kKeys) {
                const int key = k * kKeys + tid;
                long long row = -1;
                if (key < seq.n) {
                    const long long phys =
                        a.block_tables[(size_t)b * a.cols + seq.col0 + key / a.BS];
                    if (phys < 0 || phys >= a.NB) {
                        report(a.dev_status, KVD_DEV_BLOCK_RANGE);
                    } else {
                        row = phys * a.BS + key % a.BS;
                    }
                }
                rows_of[tid] = row;
                const uint32_t valid = __ballot_sync(0xffffffffu, row >= 0);
                if (tid == 0) scratch[34] = (int)valid;
            }
            __syncthreads();
            for (int i = tid; i < kKeys * (D / 4); i += kThreads) {
                const int r = i / (D / 4), c = 4 * (i % (D / 4));
                const long long row = rows_of[r];
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (row >= 0)
                    x = c < a.R ? load4(static_cast<const Elem*>(a.latent) + row * a.R + c)
                                : load4(static_cast<const Elem*>(a.rope) + row * a.P + (c - a.R));
                *reinterpret_cast<float4*>(sm + L.k + r * L.qs + c) = x;
            }
            __syncthreads();
            st.step(sm, L, D, a.R, a.qscale, last - k * kKeys, (uint32_t)scratch[34]);
        }
        st.publish(sm, L);
        const bool whole = first == 0 && end == nt;
        const size_t slot = ((size_t)w * a.groups + g) * 2 + (t == t0 ? 0 : 1);
        const int dgs = a.R / 4, dg = tid % dgs, rg = tid / dgs;
        if (rg < kRows / RPT) {
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const int r = rg * RPT + i;
                if (r >= nrows) break;
                const float sum = sm[L.s + r];
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                const float4 x = make_float4(st.acc[i].x * inv, st.acc[i].y * inv,
                                             st.acc[i].z * inv, st.acc[i].w * inv);
                if (whole) {
                    const size_t row = (size_t)b * a.rows + row0 + r;
                    ElemTraits<Elem>::store4(a.out, row * a.R + 4 * dg, x);
                } else {
                    *reinterpret_cast<float4*>(a.part_o + (slot * a.rpg + r) * a.R + 4 * dg) = x;
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
            a.meta[b] = make_int4(w, worker_of(before + a.lead + nt - 1, f.total, W),
                                  t == t0 ? 0 : 1, 0);
        __syncthreads();
        before += a.lead + nt;
        t = before;
    }
}

template <typename Elem, int RPT>
__global__ void __launch_bounds__(kThreads) expanded_simt_kernel(const ExpandedArgs a) {
    extern __shared__ __align__(16) float sm[];
    __shared__ int scratch[kFindWords];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, h = blockIdx.y, unit = blockIdx.x;
    const int D = a.Dn + a.P;
    const SimtLayout L(D, a.Dv, true);
    const Found f = block_find<kThreads>(
        a.Q, scratch, [&](int) { return unit; },
        [&](int b) {
            const PackedSeq s = packed_seq(a, b);
            if (s.bad && h == 0 && unit == 0) report(a.dev_status, s.bad);
            return (s.nq + kRows - 1) / kRows;
        });
    if (f.item >= a.Q) return;
    const PackedSeq seq = packed_seq(a, f.item);
    const int row0 = (unit - f.before) * kRows, nrows = min(kRows, seq.nq - row0);
    const Elem* kv = static_cast<const Elem*>(a.kv);
    for (int i = tid; i < kRows * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = 4 * (i % (D / 4));
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < nrows)
            x = load4(static_cast<const Elem*>(a.q) +
                      ((size_t)(seq.q0 + row0 + r) * a.H + h) * D + c);
        *reinterpret_cast<float4*>(sm + L.q + r * L.qs + c) = x;
    }
    RowState<RPT> st;
    st.clear();
    const int shift = a.causal ? seq.nk - seq.nq : seq.nk - 1;
    const int srow = tid >> 4;
    const int last = srow < nrows ? (a.causal ? row0 + srow + shift : shift) : -1;
    const int nkeys = a.causal ? min(seq.nk, row0 + nrows + shift) : seq.nk;
    for (int k0 = 0; k0 < nkeys; k0 += kKeys) {
        const int n = min(kKeys, nkeys - k0);
        __syncthreads();
        for (int i = tid; i < kKeys * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = 4 * (i % (D / 4));
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < n) {
                const size_t key = (size_t)seq.k0 + k0 + r;
                x = c < a.Dn ? load4(kv + (key * a.H + h) * (a.Dn + a.Dv) + c)
                             : load4(static_cast<const Elem*>(a.k_rope) + key * a.P + (c - a.Dn));
            }
            *reinterpret_cast<float4*>(sm + L.k + r * L.qs + c) = x;
        }
        for (int i = tid; i < kKeys * (a.Dv / 4); i += kThreads) {
            const int r = i / (a.Dv / 4), c = 4 * (i % (a.Dv / 4));
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < n)
                x = load4(kv + (((size_t)seq.k0 + k0 + r) * a.H + h) * (a.Dn + a.Dv) + a.Dn + c);
            *reinterpret_cast<float4*>(sm + L.v + r * L.vs + c) = x;
        }
        __syncthreads();
        st.step(sm, L, D, a.Dv, a.qscale, last - k0, n == 32 ? ~0u : (1u << n) - 1u);
    }
    __syncthreads();
    st.publish(sm, L);
    const int dgs = a.Dv / 4, dg = tid % dgs, rg = tid / dgs;
    if (rg < kRows / RPT) {
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int r = rg * RPT + i;
            if (r >= nrows) break;
            const float sum = sm[L.s + r];
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            ElemTraits<Elem>::store4(
                a.out, ((size_t)(seq.q0 + row0 + r) * a.H + h) * a.Dv + 4 * dg,
                make_float4(st.acc[i].x * inv, st.acc[i].y * inv, st.acc[i].z * inv,
                            st.acc[i].w * inv));
        }
    }
    if (tid < nrows && a.lse_out)
        a.lse_out[(size_t)(seq.q0 + row0 + tid) * a.H + h] =
            lse2_of(sm[L.s + kRows + tid], sm[L.s + tid]) * kLn2;
}

// One warp per (row, 128 dims): the workers' partial rows by log-sum-exp.
template <typename Out>
__global__ void __launch_bounds__(128) latent_combine_kernel(const LatentArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int b = blockIdx.y;
    const int4 meta = a.meta[b];
    const int w0 = meta.x, w1 = meta.y;
    if (w0 == w1) return;
    // a launch that gave up on a wait may have left no division behind
    if (w0 < 0 || w1 < w0 || w1 >= a.workers || (meta.z & ~1)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x, g = row / a.rpg, r = row % a.rpg;
    const int d = 128 * warp + 4 * lane;
    if (128 * warp >= a.R) return;
    // a lane a worker: its log-sum-exp, then its weight; 32 workers at a time
    // against a running maximum
    const float* base_o = a.part_o + d;
    float M = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int wb = w0; wb <= w1; wb += 32) {
        const int w = wb + lane, n = min(32, w1 - wb + 1);
        const int slot = (w * a.groups + g) * 2 + (w == w0 ? meta.z : 0);
        const float z = w <= w1 ? a.part_lse[(size_t)slot * a.rpg + r] : -INFINITY;
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
        for (int i0 = 0; i0 < n; i0 += 8) {
            float4 x[8];
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int from = min(i0 + i, n - 1);
                const int sl = __shfl_sync(0xffffffffu, slot, from);
                f[i] = __shfl_sync(0xffffffffu, e, from);
                if (i0 + i >= n) f[i] = 0.f;
                x[i] = i0 + i < n ? *reinterpret_cast<const float4*>(
                                        base_o + ((size_t)sl * a.rpg + r) * a.R)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                l += f[i];
                acc.x = fmaf(f[i], x[i].x, acc.x);
                acc.y = fmaf(f[i], x[i].y, acc.y);
                acc.z = fmaf(f[i], x[i].z, acc.z);
                acc.w = fmaf(f[i], x[i].w, acc.w);
            }
        }
    }
    const float base = M == -INFINITY ? 0.f : M;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const size_t at = (size_t)b * a.rows + row;
    ElemTraits<Out>::store4(a.out, at * a.R + d,
                            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    if (d == 0 && a.lse_out) a.lse_out[at] = lse2_of(base, l) * kLn2;
}

template <typename Elem, int RPT>
cudaError_t go_latent(const LatentArgs& a, cudaStream_t stream) {
    const SimtLayout L(a.R + a.P, a.R, false);
    const int smem = L.total * 4;
    cudaError_t e = cudaFuncSetAttribute(latent_simt_kernel<Elem, RPT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(latent_simt_kernel<Elem, RPT>, dim3(a.groups, a.workers), dim3(kThreads),
                      smem, stream, a);
}

template <typename Elem, int RPT>
cudaError_t go_expanded(const ExpandedArgs& a, cudaStream_t stream) {
    const SimtLayout L(a.Dn + a.P, a.Dv, true);
    const int smem = L.total * 4;
    cudaError_t e = cudaFuncSetAttribute(expanded_simt_kernel<Elem, RPT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int units = (a.Nq + kRows - 1) / kRows + a.Q;
    return launch_pdl(expanded_simt_kernel<Elem, RPT>, dim3(units, a.H), dim3(kThreads), smem,
                      stream, a);
}

template <typename Elem>
cudaError_t go(const LatentArgs& a, cudaStream_t stream) {
    if (a.R > 256) return go_latent<Elem, 8>(a, stream);
    if (a.R > 128) return go_latent<Elem, 4>(a, stream);
    return go_latent<Elem, 2>(a, stream);
}

template <typename Elem>
cudaError_t go(const ExpandedArgs& a, cudaStream_t stream) {
    return a.Dv == 128 ? go_expanded<Elem, 2>(a, stream) : go_expanded<Elem, 1>(a, stream);
}

}  // namespace

cudaError_t launch_latent_simt(const LatentArgs& a, kvd_dtype dt, cudaStream_t stream) {
    return dt == KVD_BF16 ? go<__nv_bfloat16>(a, stream) : go<float>(a, stream);
}

cudaError_t launch_expanded_simt(const ExpandedArgs& a, kvd_dtype dt, cudaStream_t stream) {
    return dt == KVD_BF16 ? go<__nv_bfloat16>(a, stream) : go<float>(a, stream);
}

cudaError_t launch_latent_combine(const LatentArgs& a, kvd_dtype dt, cudaStream_t stream) {
    const dim3 grid(a.rows, a.Q);
    return dt == KVD_BF16
               ? launch_pdl(latent_combine_kernel<__nv_bfloat16>, grid, dim3(128), 0, stream, a)
               : launch_pdl(latent_combine_kernel<float>, grid, dim3(128), 0, stream, a);
}

}  // namespace kvd
