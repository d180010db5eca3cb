// rotate.cu -- kvd_rotate and kvd_rotate_append_paged: the norm of every head, the
// rotation by position and the way into the cache in one pass over the projection.
//
// y = x w / sqrt(mean x^2 + eps); the pair (a, b) of frequency i at position p turns
// to (a c - b s, a s + b c), c = m cos(p f_i), s = m sin(p f_i).
//
// The angle: at a position of 10^6 a product in fp32 is off by 0.03 rad, so
// f_i is taken as a fraction of a turn in 64 bits of fixed point (by whole numbers:
// 64-bit floating point is a small unit's work here), and the product with the position
// wraps to the angle within its turn by itself; what is left, reduced to an eighth of a
// turn, goes to sincospif.  A CTA does that once a token and frequency for all heads.
//
// A head is held by 16 lanes (8 of D = 64 in bf16, 32 of D = 128 in fp32), two pieces of 8
// bytes each: in the half layout a piece of the lower half and the one that it is paired
// with, so that no lane needs another's elements but for the norm's sum.
//
// Measured, 8192 tokens x 48 heads of 128 with norms: 40.9 us, 201 MB, 4.9 TB/s of the
// copy's 6.8.  Issue slots (70 to 78 % taken) bound it: without the norm 36 us, without
// the rotation 39, without both and the angles 34.4.  A step of 64 tokens takes 3.1 us,
// a launch and one chain of latencies.  Not kept: arithmetic on pairs of fp32 (45 us, spills or
// moves), loads into a head's registers as soon as it is through (55), 5 to 14 tokens a
// CTA (41.0 to 42.4).
#include "../kvd_internal.h"
#include "serving_common.cuh"

namespace kvd {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 128; // of a CTA at most: as many as it has groups, four times over
constexpr int kRows = 3;    // heads that a group of lanes loads at once

// cos and sin of p * f, f in radians, |error| of the angle about 2^-25.
__device__ __forceinline__ float2 turn_of(double f, int p) {
    const unsigned long long bits = (unsigned long long)__double_as_longlong(f);
    const int e = (int)(bits >> 52) & 0x7ff;
    if (e == 0x7ff) return make_float2(NAN, NAN);
    // f = m 2^(e - 1086); 2^66 / (2 pi) in whole numbers; then turns a position in 2^-64
    const unsigned long long m = e ? bits << 11 | 1ull << 63 : 0;
    const unsigned long long t = __umul64hi(m, 11743562013128004906ull);
    const int shift = e - 1024;
    unsigned long long turns = shift >= 64 || shift <= -64 ? 0 : shift >= 0 ? t << shift : t >> -shift;
    if (bits >> 63) turns = 0 - turns;
    const uint32_t turn = (uint32_t)((turns * (unsigned long long)(uint32_t)p) >> 32);
    // quarter turns, and an angle of an eighth of a turn at most behind them
    const uint32_t quarter = (turn + 0x20000000u) >> 30;
    const int rest = (int)(turn - (quarter << 30));
    float s, c;
    sincospif((float)rest * 4.656612873077393e-10f, &s, &c);  // 2^-31 half turns
    const bool swap = quarter & 1u;
    const float x = swap ? s : c, y = swap ? c : s;
    return make_float2((quarter + 1u) & 2u ? -x : x, quarter & 2u ? -y : y);
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&x);
}

// 8 bytes of a head as fp32, and back.
template <typename Elem>
struct Piece;
template <>
struct Piece<__nv_bfloat16> {
    static constexpr int kNum = 4;
    __device__ __forceinline__ static void unpack(uint2 v, float* x) {
        const float2 a = bf16x2_to_float2(v.x), b = bf16x2_to_float2(v.y);
        x[0] = a.x;
        x[1] = a.y;
        x[2] = b.x;
        x[3] = b.y;
    }
    __device__ __forceinline__ static uint2 pack(const float* x) {
        return make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
    }
};
template <>
struct Piece<float> {
    static constexpr int kNum = 2;
    __device__ __forceinline__ static void unpack(uint2 v, float* x) {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
    }
    __device__ __forceinline__ static uint2 pack(const float* x) {
        return make_uint2(__float_as_uint(x[0]), __float_as_uint(x[1]));
    }
};

// `tokens` tokens a CTA, their heads in parts over the grid's y; 2^side groups of lanes take
// a token's heads, the CTA's other groups other tokens.  A group takes up to kRows heads
// at once and loads the next ones before it turns to them; the first loads are issued
// before the angles are there.
// (kWhole: all groups take one token's heads.  With the token known to be the CTA's the
// loop needs 64 registers instead of 116 and 8192 tokens x 48 heads 42 us instead of 49;
// 1001 tokens x 12 heads take 3.2 us with four tokens at once and 5.5 with one.)
template <typename Elem, int D, bool kPairs, bool kWhole>
__global__ void __launch_bounds__(kThreads, kWhole ? 4 : 3)
rotate_kernel(const RotateArgs a, const int tokens, const int side) {
    using P = Piece<Elem>;
    constexpr int kNum = P::kNum, kLanes = D / (2 * kNum), kGroups = kThreads / kLanes;
    extern __shared__ float2 turns[];  // [tokens, D / 2]
    __shared__ int at[kTokens], slots[kTokens];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid % kLanes;
    const int wide = kWhole ? kGroups : 1 << side,
              group = kWhole ? tid / kLanes : (tid / kLanes) & (wide - 1),
              t0 = kWhole ? 0 : (tid / kLanes) >> side, step = kWhole ? 1 : kGroups >> side,
              batch = kRows * wide;
    const uint32_t mask = kLanes == 32 || kWhole ? 0xffffffffu
                                       : ((1u << (kLanes & 31)) - 1u) << ((tid & 31) / kLanes * kLanes);
    const int n0 = blockIdx.x * tokens, half = a.Dr / 2, live = min(tokens, a.N - n0);
    const int heads = a.Hq + 2 * a.Hkv, share = (heads + gridDim.y - 1) / gridDim.y,
              first = blockIdx.y * share, end = min(heads, first + share);
    // this lane's pieces, and the frequencies of the first one's elements
    const bool turned = 2 * kNum * lane < a.Dr;
    const int e0 = !kPairs && turned ? kNum * lane : 2 * kNum * lane,
              e1 = e0 + (!kPairs && turned ? half : kNum), f0 = kNum * lane;
    const Elem* x = static_cast<const Elem*>(a.x) + (size_t)n0 * heads * D;
    uint2 raw[2][kRows], next[2][kRows];
    auto load = [&](uint2 (&v)[2][kRows], int t, int h0) {
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int h = h0 + group + k * wide;
            if (h < end) {
                const Elem* r = x + ((size_t)t * heads + h) * D;
                v[0][k] = __ldcs(reinterpret_cast<const uint2*>(r + e0));
                v[1][k] = __ldcs(reinterpret_cast<const uint2*>(r + e1));
            }
        }
    };
    if (t0 < live) load(raw, t0, first);
    if (tid < live) {
        const int p = a.positions[n0 + tid];
        if (p < -1) report(a.dev_status, KVD_DEV_POS_RANGE);
        at[tid] = p;
        if (a.Hkv > 0) {
            const int slot = a.slots[n0 + tid];
            const bool bad = slot < -1 || slot >= a.rows;
            if (bad && p >= 0) report(a.dev_status, KVD_DEV_BLOCK_RANGE);
            slots[tid] = bad ? -1 : slot;
        }
    }
    for (int i = tid; i < live * half; i += kThreads) {
        const int t = i / half, p = a.positions[n0 + t];
        if (p >= 0) {
            const float2 cs = turn_of(a.freqs[i - t * half], p);
            turns[t * (D / 2) + i - t * half] = make_float2(cs.x * a.stretch, cs.y * a.stretch);
        }
    }
    uint2 qw[2] = {}, kw[2] = {};
    if (a.q_weight) {
        qw[0] = *reinterpret_cast<const uint2*>(static_cast<const Elem*>(a.q_weight) + e0);
        qw[1] = *reinterpret_cast<const uint2*>(static_cast<const Elem*>(a.q_weight) + e1);
    }
    if (a.k_weight) {
        kw[0] = *reinterpret_cast<const uint2*>(static_cast<const Elem*>(a.k_weight) + e0);
        kw[1] = *reinterpret_cast<const uint2*>(static_cast<const Elem*>(a.k_weight) + e1);
    }
    __syncthreads();
    for (int t = t0; t < live; t += step) {
        const int p = at[t], slot = a.Hkv > 0 ? slots[t] : -1;
        float2 cs[kNum];  // pair layout: the first kNum frequencies of the lane's kNum pairs
#pragma unroll
        for (int e = 0; e < kNum; ++e)
            cs[e] = turned ? turns[t * (D / 2) + f0 + e] : make_float2(1.f, 0.f);
        for (int h0 = first; h0 < end; h0 += batch) {
            if (h0 + batch < end)
                load(next, t, h0 + batch);
            else if (t + step < live)
                load(next, t + step, first);
            if (p >= 0)
#pragma unroll
                for (int k = 0; k < kRows; ++k) {
                    if (h0 + k * wide >= end) break;
                    const int h = h0 + group + k * wide;
                    const bool some = h < end, value = h >= a.Hq + a.Hkv;
                    float y[2 * kNum];  // the first piece, the second one
                    P::unpack(raw[0][k], y);
                    P::unpack(raw[1][k], y + kNum);
                    const bool norm = h < a.Hq ? a.q_weight != nullptr : a.k_weight != nullptr;
                    // a warp that holds values alone is spared the rest (8192 tokens x 48
                    // heads, 8 of them values: 41.7 us, now 40.9)
                    const bool work = !kWhole || __any_sync(0xffffffffu, !value);
                    if ((a.q_weight || a.k_weight) && work) {
                        float sum = 0.f;
#pragma unroll
                        for (int e = 0; e < 2 * kNum; ++e) sum = fmaf(y[e], y[e], sum);
#pragma unroll
                        for (int d = kLanes / 2; d; d >>= 1) sum += __shfl_xor_sync(mask, sum, d);
                        if (norm) {
                            const float r = rsqrtf(sum * (1.f / D) + a.eps);
                            float wt[2 * kNum];
                            P::unpack(h < a.Hq ? qw[0] : kw[0], wt);
                            P::unpack(h < a.Hq ? qw[1] : kw[1], wt + kNum);
#pragma unroll
                            for (int e = 0; e < 2 * kNum; ++e) y[e] = y[e] * r * wt[e];
                        }
                    }
                    if (turned && work) {
#pragma unroll
                        for (int e = 0; e < kNum; ++e) {
                            float& u = y[kPairs ? 2 * e : e];
                            float& v = y[kPairs ? 2 * e + 1 : e + kNum];
                            const float z = u * cs[e].x - v * cs[e].y;
                            v = u * cs[e].y + v * cs[e].x;
                            u = z;
                        }
                    }
                    if (!some || (h >= a.Hq && slot < 0)) continue;
                    Elem* to = h < a.Hq ? static_cast<Elem*>(a.q_out) + ((size_t)(n0 + t) * a.Hq + h) * D
                               : !value ? static_cast<Elem*>(a.key_cache) +
                                              ((size_t)slot * a.Hkv + h - a.Hq) * D
                                        : static_cast<Elem*>(a.value_cache) +
                                              ((size_t)slot * a.Hkv + h - a.Hq - a.Hkv) * D;
                    *reinterpret_cast<uint2*>(to + e0) = value ? raw[0][k] : P::pack(y);
                    *reinterpret_cast<uint2*>(to + e1) = value ? raw[1][k] : P::pack(y + kNum);
                }
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                raw[0][k] = next[0][k];
                raw[1][k] = next[1][k];
            }
        }
    }
}

template <typename Elem, int D>
cudaError_t go_rotate(const RotateArgs& a, bool pairs, cudaStream_t stream) {
    constexpr int kGroups = kThreads / (D / (2 * Piece<Elem>::kNum));
    const int heads = a.Hq + 2 * a.Hkv;
    // many tokens: kRows heads a group, four tokens one after the other (rounds of them while
    // four CTAs an SM are left); few: a head a group, and a token's heads over several CTAs
    int side = 0;
    while ((1 << side) < kGroups &&
           (kRows << side < heads || (long long)a.N * heads < (long long)kGroups * kServingSMs << side))
        ++side;
    const int at_once = kGroups >> side;
    int tokens = at_once;
    while (tokens < 4 * at_once && a.N / (2 * tokens) >= 4 * kServingSMs) tokens *= 2;
    const int ctas = (a.N + tokens - 1) / tokens;
    int parts = 1;
    while (ctas * parts * 2 <= 3 * kServingSMs && heads > parts << side) parts *= 2;
    const dim3 grid(ctas, parts);
    const size_t bytes = (size_t)tokens * (D / 2) * sizeof(float2);
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, grid, dim3(kThreads), bytes, stream, a, tokens, side);
    };
    const bool whole = at_once == 1;
    return pairs ? (whole ? go(rotate_kernel<Elem, D, true, true>) : go(rotate_kernel<Elem, D, true, false>))
                 : (whole ? go(rotate_kernel<Elem, D, false, true>) : go(rotate_kernel<Elem, D, false, false>));
}

}  // namespace

cudaError_t launch_rotate(const RotateArgs& a, bool pairs, kvd_dtype dt, cudaStream_t stream) {
    if (dt == KVD_BF16)
        return a.D == 64 ? go_rotate<__nv_bfloat16, 64>(a, pairs, stream)
                         : go_rotate<__nv_bfloat16, 128>(a, pairs, stream);
    return a.D == 64 ? go_rotate<float, 64>(a, pairs, stream)
                     : go_rotate<float, 128>(a, pairs, stream);
}

}  // namespace kvd
