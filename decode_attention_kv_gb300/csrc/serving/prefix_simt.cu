// prefix_simt.cu -- kvd_attend_paged_prefix: the shared prefixes in fp32, on CUDA cores,
// and the merge of all partial rows.
//
// A tile is 16 query rows (sequences x query heads of one kv head of a group) x 32
// keys in shared memory: every prefix row is read once a row tile.  Scores: a thread
// a row and two keys; softmax: 16 threads a row keep the running max and sum; values:
// a thread owns four dims (D = 64) or eight of one row.
//
// What bounds it at the sizes it is for (checks of small models): latency.  9 sequences behind
// two prompts of 515 tokens, 8 / 2 heads of 64: 12.9 us a call, 6 of them this kernel's
// chain lengths -> page -> tile -> softmax -> rows, the rest the attention over own tokens
// beside it and the merge (3 us: meta row, log-sum-exps, up to eight rows at a time).
#include "../kvd_internal.h"
#include "serving_common.cuh"

namespace kvd {
namespace {

constexpr int kThreads = 256, kRows = 16, kKeys = 32;

template <int D>
__global__ void __launch_bounds__(kThreads) prefix_simt_kernel(const PrefixArgs a) {
    using Elem = float;
    constexpr int kStride = D + 4, kVec = 4;
    __shared__ PrefixGroups groups;
    extern __shared__ __align__(16) float sm[];
    float* qs = sm;                       // [kRows, kStride]
    float* ks = qs + kRows * kStride;     // [kKeys, kStride]
    float* vs = ks + kKeys * kStride;     // [kKeys, D]
    float* ps = vs + kKeys * D;           // [kRows, kKeys + 1]
    __shared__ uint32_t valid_bits;
    pdl_wait();
    const int tid = threadIdx.x, row = tid >> 4, sub = tid & 15;
    const PrefixRuns runs = prefix_setup<kThreads>(a, groups);
    prefix_meta(a, groups, runs, tid, kThreads);
    const int w = blockIdx.x;
    if (runs.tot == 0 || w >= runs.W) return;
    const int lo = runs.start(w), hi = runs.start(w + 1);
    const Elem* qg = static_cast<const Elem*>(a.q);
    const Elem* kg = static_cast<const Elem*>(a.k);
    const Elem* vg = static_cast<const Elem*>(a.v);
    for (int p = lo; p < hi;) {
        const PrefixPiece s = prefix_piece(a, groups, w, lo, hi, p);
        p = s.next;
        if (s.k0 >= s.k1) continue;
        const int s0 = groups.start[s.group], rows = groups.sequences(s.group) * a.g;
        const int n = groups.keys[s.group];
        const int r = s.tile * kRows + row;  // this thread's row of the group
        const bool live = r < rows;
        const size_t at = live ? (size_t)(s0 + r / a.g) * a.Hq + s.head * a.g + r % a.g : 0;
        __syncthreads();  // the last piece's shared memory is free
        for (int c = sub * kVec; c < D; c += 16 * kVec)
            if (live) {
                float2 x[kVec / 2];
                ElemTraits<Elem>::unpack(*reinterpret_cast<const uint4*>(qg + at * D + c), x);
#pragma unroll
                for (int e = 0; e < kVec / 2; ++e)
                    *reinterpret_cast<float2*>(qs + row * kStride + c + 2 * e) = x[e];
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e) qs[row * kStride + c + e] = 0.f;
            }
        float m = -INFINITY, l = 0.f;
        float4 acc[D / 64];
#pragma unroll
        for (int j = 0; j < D / 64; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = s.k0; k < s.k1; ++k) {
            if (tid == 0) valid_bits = 0;
            __syncthreads();
            {  // eight threads a key
                const int key = k * kKeys + (tid >> 3), c0 = (tid & 7) * kVec;
                int phys = -1;
                if (key < n) {
                    phys = __ldg(a.prefix_tables + (size_t)s.group * a.pcols + key / a.BS);
                    if (phys < 0 || phys >= a.NB) {
                        if (c0 == 0) report(a.dev_status, KVD_DEV_BLOCK_RANGE);
                        phys = -1;
                    }
                }
                const size_t src =
                    phys < 0 ? 0
                             : (((size_t)phys * a.BS + key % a.BS) * a.Hkv + s.head) * D;
                if (phys >= 0 && c0 == 0) atomicOr(&valid_bits, 1u << (tid >> 3));
                for (int c = c0; c < D; c += 8 * kVec) {
                    float2 x[kVec / 2], y[kVec / 2];
                    uint4 kx = make_uint4(0, 0, 0, 0), vx = kx;
                    if (phys >= 0) {
                        kx = *reinterpret_cast<const uint4*>(kg + src + c);
                        vx = *reinterpret_cast<const uint4*>(vg + src + c);
                    }
                    ElemTraits<Elem>::unpack(kx, x);
                    ElemTraits<Elem>::unpack(vx, y);
#pragma unroll
                    for (int e = 0; e < kVec / 2; ++e) {
                        *reinterpret_cast<float2*>(ks + (tid >> 3) * kStride + c + 2 * e) = x[e];
                        *reinterpret_cast<float2*>(vs + (tid >> 3) * D + c + 2 * e) = y[e];
                    }
                }
            }
            __syncthreads();
            const uint32_t valid = valid_bits;
            float2 d0 = make_float2(0.f, 0.f), d1 = d0;
#pragma unroll 8
            for (int c = 0; c < D; c += 4) {
                const float4 x = *reinterpret_cast<const float4*>(qs + row * kStride + c);
                const float4 y = *reinterpret_cast<const float4*>(ks + sub * kStride + c);
                const float4 z = *reinterpret_cast<const float4*>(ks + (sub + 16) * kStride + c);
                d0 = ffma2(make_float2(x.x, x.y), make_float2(y.x, y.y), d0);
                d1 = ffma2(make_float2(x.x, x.y), make_float2(z.x, z.y), d1);
                d0 = ffma2(make_float2(x.z, x.w), make_float2(y.z, y.w), d0);
                d1 = ffma2(make_float2(x.z, x.w), make_float2(z.z, z.w), d1);
            }
            const float sc0 = (valid >> sub) & 1u ? (d0.x + d0.y) * a.qscale : -INFINITY;
            const float sc1 = (valid >> (sub + 16)) & 1u ? (d1.x + d1.y) * a.qscale : -INFINITY;
            float top = fmaxf(sc0, sc1);
#pragma unroll
            for (int d = 8; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float mn = fmaxf(m, top);
            const float base = mn == -INFINITY ? 0.f : mn;
            const float corr = exp2f(m - base);
            const float e0 = exp2f(sc0 - base), e1 = exp2f(sc1 - base);
            m = mn;
            float sum = e0 + e1;
#pragma unroll
            for (int d = 8; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            l = l * corr + sum;
            ps[row * (kKeys + 1) + sub] = e0;
            ps[row * (kKeys + 1) + sub + 16] = e1;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                acc[j].x *= corr;
                acc[j].y *= corr;
                acc[j].z *= corr;
                acc[j].w *= corr;
            }
            __syncwarp();  // a row's weights are its own half warp's
#pragma unroll 8
            for (int e = 0; e < kKeys; ++e) {
                const float f = ps[row * (kKeys + 1) + e];
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    const float4 x = *reinterpret_cast<const float4*>(vs + e * D + 64 * j + 4 * sub);
                    acc[j].x = fmaf(f, x.x, acc[j].x);
                    acc[j].y = fmaf(f, x.y, acc[j].y);
                    acc[j].z = fmaf(f, x.z, acc[j].z);
                    acc[j].w = fmaf(f, x.w, acc[j].w);
                }
            }
            __syncthreads();
        }
        if (live) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const size_t to = s.slot < 0 ? at : (size_t)s.slot * a.rows + row;
            float* o = (s.slot < 0 ? a.whole_o : a.part_o) + to * D;
            if (sub == 0)
                (s.slot < 0 ? a.whole_lse : a.part_lse)[to] =
                    l > 0.f ? m + log2f(l) : (l == 0.f ? -INFINITY : NAN);
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
                *reinterpret_cast<float4*>(o + 64 * j + 4 * sub) = make_float4(
                    acc[j].x * inv, acc[j].y * inv, acc[j].z * inv, acc[j].w * inv);
        }
    }
}

template <int D>
cudaError_t go_simt(const PrefixArgs& a, cudaStream_t stream) {
    const int bytes = ((kRows + kKeys) * (D + 4) + kKeys * D + kRows * (kKeys + 1)) * 4;
    const cudaError_t e = cudaFuncSetAttribute(
        prefix_simt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(prefix_simt_kernel<D>, dim3(a.workers), dim3(kThreads), bytes, stream, a);
}

// ------------------------------------------------------------ merge
// One warp an output row: the pieces of its prefix and the splits of its own keys, by
// log-sum-exp; 32 partial rows at a time against a running maximum, a lane each for the
// weights, then D / 32 dims a lane.
// (Eight partial rows at a time: 8 sequences behind 4096 tokens 23.3 -> 22.4 us against four.  A
// warp a CTA: 256 sequences 90 -> 77 us against four, 4 sequences 15.7 -> 15.4.)
constexpr int kMergeWarps = 1, kMergeRows = 8;

template <typename Out, int D>
__global__ void __launch_bounds__(32 * kMergeWarps) prefix_combine_kernel(const PrefixArgs a) {
    constexpr int kDims = D / 32;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
    if (row >= a.Q * a.Hq) return;
    const int q = row / a.Hq, hq = row - q * a.Hq, h = hq / a.g;
    const int4 meta = a.meta[q];
    const int4 line = a.meta[a.Q];
    int w0 = 0, pieces = 0, in_tile = 0;  // pieces of the prefix
    // (a launch that gave up on a wait may have left no division behind)
    if (meta.z > 0 && line.x > 0 && line.y > 0 && line.y <= a.workers) {
        const PrefixRuns runs(line.x, line.y);
        const int r = meta.w * a.g + hq - h * a.g, tile = r / a.rows;
        in_tile = r - tile * a.rows;
        const int first = meta.x + (h * meta.y + tile) * (meta.z + a.lead) + a.lead;
        w0 = runs.worker_of(first);
        pieces = runs.worker_of(first + meta.z - 1) - w0 + 1;
        if (w0 < 0 || pieces < 1 || w0 + pieces > a.workers) pieces = 0;
    }
    const int n = pieces + a.S;
    float M = -INFINITY, l = 0.f, acc[kDims];
#pragma unroll
    for (int e = 0; e < kDims; ++e) acc[e] = 0.f;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        const float* src = nullptr;
        float z = -INFINITY;
        if (i < pieces) {
            if (pieces == 1) {
                z = a.whole_lse[row];
                src = a.whole_o + (size_t)row * D;
            } else {
                const size_t at = (size_t)(2 * (w0 + i) + (i == 0)) * a.rows + in_tile;
                z = a.part_lse[at];
                src = a.part_o + at * D;
            }
        } else if (i < n) {
            const size_t at = (size_t)row * a.S + i - pieces;
            z = a.own_lse[at] * kLog2e;
            src = a.own_o + at * D;
        }
        float top = z;
#pragma unroll
        for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        top = fmaxf(top, M);
        const float base = top == -INFINITY ? 0.f : top;
        const float corr = exp2f(M - base), wt = exp2f(z - base);
        M = top;
        l *= corr;
#pragma unroll
        for (int e = 0; e < kDims; ++e) acc[e] *= corr;
        const int many = min(32, n - i0);
        for (int j0 = 0; j0 < many; j0 += kMergeRows) {
            float f[kMergeRows], x[kMergeRows][kDims];
#pragma unroll
            for (int j = 0; j < kMergeRows; ++j) {
                f[j] = __shfl_sync(0xffffffffu, wt, min(j0 + j, 31));
                const float* o = reinterpret_cast<const float*>(__shfl_sync(
                    0xffffffffu, reinterpret_cast<unsigned long long>(src), min(j0 + j, 31)));
                if (j0 + j >= many) f[j] = 0.f;
                // an empty range's row was not written
#pragma unroll
                for (int e = 0; e < kDims; ++e) x[j][e] = 0.f;
                if (f[j] != 0.f) {
                    if constexpr (kDims == 4)
                        *reinterpret_cast<float4*>(x[j]) = *reinterpret_cast<const float4*>(o + 4 * lane);
                    else
                        *reinterpret_cast<float2*>(x[j]) = *reinterpret_cast<const float2*>(o + 2 * lane);
                }
            }
#pragma unroll
            for (int j = 0; j < kMergeRows; ++j) {
                l += f[j];
#pragma unroll
                for (int e = 0; e < kDims; ++e) acc[e] = fmaf(f[j], x[j][e], acc[e]);
            }
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    Out* out = static_cast<Out*>(a.out) + (size_t)row * D + kDims * lane;
#pragma unroll
    for (int e = 0; e < kDims; ++e) ElemTraits<Out>::store(out, e, acc[e] * inv);
    if (lane == 0 && a.lse_out)
        a.lse_out[row] = (l > 0.f ? M + log2f(l) : (l == 0.f ? -INFINITY : NAN)) * kLn2;
}

template <typename Out, int D>
cudaError_t go_combine(const PrefixArgs& a, cudaStream_t stream) {
    const int rows = a.Q * a.Hq;
    return launch_pdl(prefix_combine_kernel<Out, D>, dim3((rows + kMergeWarps - 1) / kMergeWarps),
                      dim3(32 * kMergeWarps), 0, stream, a);
}

}  // namespace

cudaError_t launch_prefix_simt(const PrefixArgs& a, cudaStream_t stream) {
    return a.D == 64 ? go_simt<64>(a, stream) : go_simt<128>(a, stream);
}

cudaError_t launch_prefix_combine(const PrefixArgs& a, kvd_dtype dt, cudaStream_t stream) {
    if (dt == KVD_BF16)
        return a.D == 64 ? go_combine<__nv_bfloat16, 64>(a, stream)
                         : go_combine<__nv_bfloat16, 128>(a, stream);
    return a.D == 64 ? go_combine<float, 64>(a, stream) : go_combine<float, 128>(a, stream);
}

}  // namespace kvd
