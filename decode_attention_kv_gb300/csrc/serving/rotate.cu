// rotate.cu -- kvd_rotate and kvd_rotate_append_paged: the norm of every head, the
// rotation by position and the way into the cache in one pass over the projection.
//
// y = x w / sqrt(mean x^2 + eps); the pair (a, b) of frequency i at position p turns
// to (a c - b s, a s + b c), c = m cos(p f_i), s = m sin(p f_i).
//
// The angle: at a position of 10^6 a product in fp32 is off by 0.03 rad, so
// f_i is taken as a fraction of a turn in 64 bits of fixed point, and the product
// with the position wraps to the angle within its turn by itself; what is left,
// reduced to an eighth of a turn, goes to sincospif.  A CTA does that once a token and
// frequency for all heads.
//
// A head is held by D * bytes / 16 lanes, 16 bytes each.  In the half layout the
// partner of an element is on the lane Dr / 2 elements further.
#include "../kvd_internal.h"
#include "serving_common.cuh"

namespace kvd {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 4;  // of a CTA

// cos and sin of p * f, f in radians, |error| of the angle about 2^-25.
__device__ __forceinline__ float2 turn_of(double f, int p) {
    const double t = f * 0.15915494309189533577;  // turns per position
    if (!(fabs(t) < 4503599627370496.0)) return make_float2(NAN, NAN);
    const double frac = t - floor(t);
    const unsigned long long fixed =
        (unsigned long long)(frac * 4294967296.0) << 32 |
        (unsigned long long)((frac * 4294967296.0 - floor(frac * 4294967296.0)) * 4294967296.0);
    const uint32_t turn = (uint32_t)((fixed * (unsigned long long)(uint32_t)p) >> 32);
    // quarter turns, and an angle of an eighth of a turn at most behind them
    const uint32_t quarter = (turn + 0x20000000u) >> 30;
    const int rest = (int)(turn - (quarter << 30));
    float s, c;
    sincospif((float)rest * 4.656612873077393e-10f, &s, &c);  // 2^-31 half turns
    switch (quarter & 3u) {
        case 0: return make_float2(c, s);
        case 1: return make_float2(-s, c);
        case 2: return make_float2(-c, -s);
        default: return make_float2(s, -c);
    }
}

template <typename Elem>
__device__ __forceinline__ void unpack_vec(const uint4& v, float (&x)[ElemTraits<Elem>::kPerVec]) {
    float2 f[ElemTraits<Elem>::kPerVec / 2];
    ElemTraits<Elem>::unpack(v, f);
#pragma unroll
    for (int e = 0; e < ElemTraits<Elem>::kPerVec; e += 2) {
        x[e] = f[e / 2].x;
        x[e + 1] = f[e / 2].y;
    }
}

template <typename Elem, int D, bool kPairs>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const RotateArgs a) {
    constexpr int kVec = ElemTraits<Elem>::kPerVec, kLanes = D / kVec, kGroups = kThreads / kLanes;
    __shared__ float2 turns[kTokens][D / 2];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid % kLanes, group = tid / kLanes;
    const int n0 = blockIdx.x * kTokens, half = a.Dr / 2;
    for (int i = tid; i < kTokens * half; i += kThreads) {
        const int t = i / half, n = n0 + t;
        const int p = n < a.N ? a.positions[n] : -1;
        if (p >= 0) {
            const float2 cs = turn_of(a.freqs[i - t * half], p);
            turns[t][i - t * half] = make_float2(cs.x * a.stretch, cs.y * a.stretch);
        }
    }
    __syncthreads();
    const int heads = a.Hq + 2 * a.Hkv, e0 = lane * kVec;
    const Elem* x = static_cast<const Elem*>(a.x);
    const bool turned = e0 < a.Dr;
    // half layout: the partner's lane, the first frequency, the sign of the sine
    const bool upper = !kPairs && turned && e0 >= half;
    const int away = kPairs || !turned ? 0 : (upper ? -half : half) / kVec;
    const int f0 = kPairs ? e0 / 2 : upper ? e0 - half : e0;
    for (int t = 0; t < kTokens; ++t) {
        const int n = n0 + t;
        if (n >= a.N) return;
        const int p = a.positions[n];
        if (p < 0) {
            if (p < -1 && tid == 0) report(a.dev_status, KVD_DEV_POS_RANGE);
            continue;
        }
        long long slot = -1;
        if (a.Hkv > 0) {
            slot = a.slots[n];
            if (slot < -1 || slot >= a.rows) {
                if (tid == 0) report(a.dev_status, KVD_DEV_BLOCK_RANGE);
                slot = -1;
            }
        }
        float c[kVec], s[kVec];
        if (turned) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float2 cs = turns[t][f0 + (kPairs ? e / 2 : e)];
                c[e] = cs.x;
                s[e] = (kPairs ? e % 2 == 0 : !upper) ? -cs.y : cs.y;
            }
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                c[e] = 1.f;
                s[e] = 0.f;
            }
        }
        // all lanes of a warp take the same number of rounds
        for (int h0 = 0; h0 < heads; h0 += kGroups) {
            const int h = h0 + group;
            const bool some = h < heads;
            uint4 raw = make_uint4(0, 0, 0, 0);
            if (some)
                raw = *reinterpret_cast<const uint4*>(x + ((size_t)n * heads + h) * D + e0);
            const bool value = h >= a.Hq + a.Hkv;
            float y[kVec];
            unpack_vec<Elem>(raw, y);
            const Elem* w = static_cast<const Elem*>(h < a.Hq ? a.q_weight : a.k_weight);
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < kVec; ++e) sum = fmaf(y[e], y[e], sum);
#pragma unroll
            for (int d = kLanes / 2; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            if (some && !value && w) {
                const float r = 1.f / sqrtf(sum * (1.f / D) + a.eps);
                float wt[kVec];
                unpack_vec<Elem>(*reinterpret_cast<const uint4*>(w + e0), wt);
#pragma unroll
                for (int e = 0; e < kVec; ++e) y[e] = y[e] * r * wt[e];
            }
            float z[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float o = kPairs ? y[e ^ 1]
                                       : __shfl_sync(0xffffffffu, y[e], (tid & 31) + away);
                z[e] = turned ? y[e] * c[e] + o * s[e] : y[e];
            }
            if (!some || (h >= a.Hq && slot < 0)) continue;
            Elem* to = h < a.Hq ? static_cast<Elem*>(a.q_out) + ((size_t)n * a.Hq + h) * D
                       : !value ? static_cast<Elem*>(a.key_cache) +
                                      ((size_t)slot * a.Hkv + h - a.Hq) * D
                                : static_cast<Elem*>(a.value_cache) +
                                      ((size_t)slot * a.Hkv + h - a.Hq - a.Hkv) * D;
            if (value) {
                *reinterpret_cast<uint4*>(to + e0) = raw;
            } else {
#pragma unroll
                for (int e = 0; e < kVec; e += 4)
                    ElemTraits<Elem>::store4(to, e0 + e,
                                             make_float4(z[e], z[e + 1], z[e + 2], z[e + 3]));
            }
        }
    }
}

template <typename Elem, int D>
cudaError_t go_rotate(const RotateArgs& a, bool pairs, cudaStream_t stream) {
    const dim3 grid((a.N + kTokens - 1) / kTokens);
    return pairs ? launch_pdl(rotate_kernel<Elem, D, true>, grid, dim3(kThreads), 0, stream, a)
                 : launch_pdl(rotate_kernel<Elem, D, false>, grid, dim3(kThreads), 0, stream, a);
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
