// expanded_mma.cu -- kvd_attend_expanded in bf16 on the tensor cores.
//
// A CTA holds two tiles of 128 queries of one head and walks the keys 128 at a
// time: S_s = Q_s . K^T and O_s += P_s . V for s = 0, 1 in turn, so that one
// tile's softmax runs while the tensor cores work on the other.  Tensor memory
// is full: two score tiles and two outputs of 128 columns; the weights replace
// the scores they came from and are the A operand from there.  MMAs of one
// thread run in order, so the next scores may overwrite weights whose product
// was issued before, and a score tile that is complete tells that the product
// before it is too: the softmax may rescale its output without another wait.
//
// Keys and values arrive in blocks of 128 tokens x 64 elements through one ring,
// in the order K(0) V(0) K(1) V(1) ..; eight blocks are a tile of keys, one of
// values and the next of keys at 192 + 128 elements a token, and every block is
// asked for at least one product of 1280 cycles before it is needed.
//
// Warps 0-3 and 4-7: softmax of tile 0 and 1, a row a thread.  Warp 8 issues the
// MMAs, warp 9 the copies.
#include "kvd_internal.h"
#include "latent_common.cuh"
#include "tcgen05_ptx.cuh"

namespace kvd {
namespace {

constexpr int kRows = 128;               // queries of a tile, keys of a step
constexpr int kBlock = kRows * 128;      // bytes of 128 rows x 64 bf16
constexpr int kRing = 8;                 // blocks in flight
constexpr int kSteps = 4;                // steps with barriers of their own (the ring holds fewer)
constexpr int kMmaWarp = 8, kCopyWarp = 9;
constexpr int kThreads = 320;
constexpr float kSkip = 8.f;             // log2 units
constexpr uint32_t kTmemCols = 512;

struct ExpandedShared {
    uint64_t q_full[2], k_full[kSteps], v_full[kSteps], empty[kRing];
    uint64_t s_full[2], p_full[2], o_full[2], drain;
    uint32_t tmem;
    int abort;
    int scratch[kFindWords];
};

struct ExpandedLayout {
    int q_blocks;  // of one query tile
    int ring, shared, total;
    __host__ __device__ explicit ExpandedLayout(int Dn) {
        q_blocks = Dn / 64 + 1;
        ring = 2 * q_blocks * kBlock;
        shared = ring + kRing * kBlock;
        total = shared + (int)sizeof(ExpandedShared) + 1024;  // 1024: alignment of the base
    }
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    unsigned long long since = 0;
    while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
        const unsigned long long now = global_timer_ns();
        if (since == 0) since = now;
        if (__any_sync(0xffffffffu, *abort_flag || now - since > kWaitLimitNs)) return false;
    }
    return true;
}

__global__ void __launch_bounds__(kThreads, 1)
expanded_mma_kernel(const ExpandedArgs a, const __grid_constant__ CUtensorMap qmap,
                    const __grid_constant__ CUtensorMap kvmap,
                    const __grid_constant__ CUtensorMap ropemap) {
    extern __shared__ __align__(1024) unsigned char raw[];
    unsigned char* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const ExpandedLayout L(a.Dn);
    ExpandedShared& sh = *reinterpret_cast<ExpandedShared*>(sm + L.shared);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x, unit = blockIdx.y;
    const int KC = L.q_blocks, VC = a.Dv / 64, per = KC + VC;  // blocks of a step

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.q_full[s], 1);
            mbar_init(&sh.s_full[s], 1);
            mbar_init(&sh.p_full[s], kRows);
            mbar_init(&sh.o_full[s], 1);
        }
        for (int i = 0; i < kSteps; ++i) {
            mbar_init(&sh.k_full[i], 1);
            mbar_init(&sh.v_full[i], 1);
        }
        for (int i = 0; i < kRing; ++i) mbar_init(&sh.empty[i], 1);
        mbar_init(&sh.drain, 1);
        sh.abort = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) tmem_alloc(&sh.tmem, kTmemCols);
    if (warp == kCopyWarp && lane == 0) {
        prefetch_tensormap(&qmap);
        prefetch_tensormap(&kvmap);
        prefetch_tensormap(&ropemap);
    }
    pdl_launch_dependents();
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    volatile int* abort_flag = &sh.abort;

    const Found f = block_find<kThreads>(
        a.Q, sh.scratch, [&](int) { return unit; },
        [&](int b) {
            const PackedSeq s = packed_seq(a, b);
            if (s.bad && h == 0 && unit == 0) report(a.dev_status, s.bad);
            return (s.nq + 2 * kRows - 1) / (2 * kRows);
        });
    const bool some = f.item < a.Q;
    const PackedSeq seq = some ? packed_seq(a, f.item) : PackedSeq{0, 0, 0, 0, 0u};
    // the last unit of a sequence first: under the causal mask it sees most keys
    const int units = (seq.nq + 2 * kRows - 1) / (2 * kRows);
    const int row0 = some ? (units - 1 - (unit - f.before)) * 2 * kRows : 0;
    const int shift = seq.nk - seq.nq;  // query i sees the keys 0 .. i + shift
    int steps[2];                       // key tiles that each query tile sees
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int first = row0 + s * kRows, rows = min(kRows, seq.nq - first);
        const int keys = rows <= 0 ? 0
                         : a.causal ? max(0, min(seq.nk, first + rows + shift))
                                    : seq.nk;
        steps[s] = (keys + kRows - 1) / kRows;
    }
    const int nsteps = max(steps[0], steps[1]);
    bool bad = false;

    if (warp == kCopyWarp) {
        // ------------------------------------------------------------ copies
        // the keys and values are read again by the sequence's other query tiles
        const uint64_t policy = policy_evict_normal();
        if (nsteps > 0) {
            const int qchunk = h * KC, kchunk = h * per - h;  // (Dn + Dv) / 64 = per - 1
            const int n = uniform(nsteps);
            int slot = 0, lap = 0;
            auto block = [&](const CUtensorMap* map, int row, int chunk, uint64_t* full) {
                if (lap > 0 && !warp_wait(&sh.empty[slot], (lap - 1) & 1, abort_flag)) return false;
                if (elect_one())
                    tma_g2s_3d(sm + L.ring + slot * kBlock, map, 0, row, chunk, full, policy);
                __syncwarp();
                if (++slot == kRing) {
                    slot = 0;
                    ++lap;
                }
                return true;
            };
            for (int i = 0; i < n && !bad; ++i) {
                const int row = uniform(seq.k0 + i * kRows);
                uint64_t* kf = &sh.k_full[i % kSteps];
                uint64_t* vf = &sh.v_full[i % kSteps];
                if (elect_one()) {
                    if (i == 0) {
                        for (int s = 0; s < 2; ++s) {
                            if (steps[s] == 0) continue;
                            mbar_arrive_expect_tx(&sh.q_full[s], KC * kBlock);
                            for (int c = 0; c < KC; ++c)
                                tma_g2s_3d(sm + (s * KC + c) * kBlock, &qmap, 0,
                                           seq.q0 + row0 + s * kRows, qchunk + c, &sh.q_full[s],
                                           policy);
                        }
                    }
                    mbar_arrive_expect_tx(kf, KC * kBlock);
                    mbar_arrive_expect_tx(vf, VC * kBlock);
                }
                __syncwarp();
                for (int c = 0; c + 1 < KC && !bad; ++c) bad = !block(&kvmap, row, kchunk + c, kf);
                if (!bad) bad = !block(&ropemap, row, 0, kf);
                for (int c = 0; c < VC && !bad; ++c)
                    bad = !block(&kvmap, row, kchunk + KC - 1 + c, vf);
            }
            if (bad) {
                if (lane == 0) sh.abort = 1;
                // blocks still in flight land within the limit; nothing reads them
                const unsigned long long since = global_timer_ns();
                while (global_timer_ns() - since < 1000000ull) {
                }
            }
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMA issue
        const uint32_t sdesc = mma_desc(kRows, kRows), odesc = mma_desc(kRows, 64, kBMn);
        const uint32_t base = uniform(smem_u32(sm)), tm = uniform(tmem);
        const int n0 = uniform(steps[0]), n1 = uniform(steps[1]), n = uniform(nsteps);
        // Scores of query tile s over key tile i; the last of the two tiles that
        // uses the keys frees their blocks.
        auto scores = [&](int s, int i) {
            const uint32_t q_low = uniform(desc_low(base + s * KC * kBlock, 16));
            const bool last = s == 1 || i >= n1;
            const int b0 = uniform(i * per % kRing);
            if (elect_one()) {
#pragma unroll 1
                for (int c = 0; c < KC; ++c) {
                    const int slot = (b0 + c) % kRing;
                    const uint32_t k_low = desc_low(base + L.ring + slot * kBlock, 16);
                    const uint32_t qc = q_low + ((c * kBlock) >> 4);
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        mma_ss(tm + s * kRows, desc_of(qc + 2 * z), desc_of(k_low + 2 * z), sdesc,
                               c > 0 || z > 0);
                    if (last) mma_commit(&sh.empty[slot]);
                }
                mma_commit(&sh.s_full[s]);
            }
            __syncwarp();
        };
        auto values = [&](int s, int i, bool final) {
            const bool last = s == 1 || i >= n1;
            const int b0 = uniform((i * per + KC) % kRing);
            if (elect_one()) {
#pragma unroll 1
                for (int c = 0; c < VC; ++c) {
                    const int slot = (b0 + c) % kRing;
                    const uint32_t v_low = desc_low(base + L.ring + slot * kBlock, 16);
#pragma unroll
                    for (int z = 0; z < 8; ++z)
                        mma_ts(tm + 256 + s * kRows + 64 * c, tm + s * kRows + 8 * z,
                               desc_of(v_low + ((z * 2048) >> 4)), odesc, i > 0 || z > 0);
                    if (last) mma_commit(&sh.empty[slot]);
                }
                if (final) mma_commit(&sh.o_full[s]);
            }
            __syncwarp();
        };
        if (n > 0) {
            bad = !warp_wait(&sh.k_full[0], 0, abort_flag);
            if (!bad && n0 > 0) {
                bad = !warp_wait(&sh.q_full[0], 0, abort_flag);
                tc_fence_after();
                if (!bad) scores(0, 0);
            }
            if (!bad && n1 > 0) {
                bad = !warp_wait(&sh.q_full[1], 0, abort_flag);
                tc_fence_after();
                if (!bad) scores(1, 0);
            }
            for (int i = 0; i < n && !bad; ++i) {
#pragma unroll 1
                for (int s = 0; s < 2 && !bad; ++s) {
                    const int ns = s == 0 ? n0 : n1;
                    if (i >= ns) continue;
                    if (!warp_wait(&sh.p_full[s], i & 1, abort_flag) ||
                        !warp_wait(&sh.v_full[i % kSteps], (i / kSteps) & 1, abort_flag)) {
                        bad = true;
                        break;
                    }
                    tc_fence_after();
                    values(s, i, i + 1 == ns);
                    if (i + 1 < ns) {
                        if (!warp_wait(&sh.k_full[(i + 1) % kSteps], ((i + 1) / kSteps) & 1,
                                       abort_flag)) {
                            bad = true;
                            break;
                        }
                        tc_fence_after();
                        scores(s, i + 1);
                    }
                }
            }
            if (bad) {
                if (lane == 0) sh.abort = 1;
                __syncwarp();
                if (elect_one()) mma_commit(&sh.drain);
                __syncwarp();
                const unsigned long long since = global_timer_ns();
                while (!mbar_try_wait(&sh.drain, 0) && global_timer_ns() - since < kWaitLimitNs) {
                }
            }
        }
    } else {
        // ------------------------------------------------------------ softmax
        const int s = warp >> 2;
        const int row = row0 + s * kRows + 32 * (warp & 3) + lane;  // in the sequence
        const bool live = some && row < seq.nq;
        const uint32_t quarter = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + s * kRows + quarter, to = tmem + 256 + s * kRows + quarter;
        const int last = !live ? -1 : a.causal ? min(seq.nk - 1, row + shift) : seq.nk - 1;
        // newest key that every row of the warp sees
        const int all_see = __reduce_min_sync(0xffffffffu, live ? last : 0x3fffffff);
        const bool flip = a.qscale < 0.f;
        const float qs = fmaxf(fabsf(a.qscale), 1e-30f);
        const int ns = steps[s];
        float m = -INFINITY, l = 0.f;
        for (int i = 0; i < ns; ++i) {
            if (!mbar_wait(&sh.s_full[s], i & 1, abort_flag)) bad = true;
            if (__any_sync(0xffffffffu, bad)) {
                bad = true;
                break;
            }
            tc_fence_after();
            const bool masked = all_see < (i + 1) * kRows - 1;
            const int lim = last - i * kRows;  // keys 0 .. lim of the tile
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float x[32];
                tmem_ld32(ts + 32 * c, reinterpret_cast<uint32_t*>(x));
                tmem_wait_ld();
                if (flip) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = -x[e];
                }
                if (masked) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (32 * c + e > lim) x[e] = -INFINITY;
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], x[e]);
            }
            const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * qs);
            if (i == 0) m = mn;
            const bool need = mn > m + kSkip;
            if (__any_sync(0xffffffffu, need)) {
                const float fac = need ? exp2f(m - mn) : 1.f;
                if (need) m = mn;
                l *= fac;
                for (int c = 0; c < a.Dv; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(to + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = __float_as_uint(__uint_as_float(o[e]) * fac);
                    tmem_st32(to + c, o);
                }
            }
            const float base = m == -INFINITY ? 0.f : m;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float x[32];
                tmem_ld32(ts + 32 * c, reinterpret_cast<uint32_t*>(x));
                tmem_wait_ld();
                if (flip) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = -x[e];
                }
                if (masked) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (32 * c + e > lim) x[e] = -INFINITY;
                }
                float p[16];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float e0 = fast_exp2(fmaf(x[e], qs, -base));
                    const float e1 = fast_exp2(fmaf(x[e + 1], qs, -base));
                    sum[(e >> 1) & 3] += e0 + e1;
                    p[e >> 1] = __uint_as_float(pack_bf16(e0, e1));
                }
                // over scores that have been read: 16 columns hold 32 weights
                tmem_st16(ts + 16 * c, p);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            const int valid = seq.nk - i * kRows;
            if (valid < kRows) {
                // rows behind the sequence's keys: a weight of zero does not keep
                // what they contain (NaN) out of the sum
                if (!mbar_wait(&sh.v_full[i % kSteps], (i / kSteps) & 1, abort_flag)) bad = true;
                for (int c = 0; c < VC; ++c) {
                    unsigned char* v = sm + L.ring + (i * per + KC + c) % kRing * kBlock;
                    for (int e = valid * 8 + (tid & 127); e < kRows * 8; e += 128)
                        *reinterpret_cast<uint4*>(v + e * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&sh.p_full[s]);
        }
        if (ns > 0 && !bad && !mbar_wait(&sh.o_full[s], 0, abort_flag)) bad = true;
        if (__any_sync(0xffffffffu, bad)) {
            bad = true;
            sh.abort = 1;
        }
        __syncwarp();
        if (!bad) {
            tc_fence_after();
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const size_t at = (size_t)(seq.q0 + (live ? row : 0)) * a.H + h;
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + at * a.Dv;
            for (int c = 0; c < a.Dv; c += 32) {
                float o[32];
                if (ns > 0) {
                    tmem_ld32(to + c, reinterpret_cast<uint32_t*>(o));
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                }
                if (live) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        *reinterpret_cast<uint4*>(out + c + e) = make_uint4(
                            pack_bf16(o[e] * inv, o[e + 1] * inv),
                            pack_bf16(o[e + 2] * inv, o[e + 3] * inv),
                            pack_bf16(o[e + 4] * inv, o[e + 5] * inv),
                            pack_bf16(o[e + 6] * inv, o[e + 7] * inv));
                }
            }
            if (live && a.lse_out)
                a.lse_out[at] =
                    (l > 0.f ? m + log2f(l) : (l == 0.f ? -INFINITY : NAN)) * kLn2;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && sh.abort) report(a.dev_status, KVD_DEV_TIMEOUT);
    if (warp == kMmaWarp) tmem_free(tmem, kTmemCols);
}

}  // namespace

cudaError_t launch_expanded_mma(const ExpandedArgs& a, cudaStream_t stream) {
    CUtensorMap qmap, kvmap, ropemap;
    const long long qw = (long long)a.H * (a.Dn + a.P), kw = (long long)a.H * (a.Dn + a.Dv);
    cudaError_t e = encode_rows(&qmap, a.q, qw, qw, a.Nq, kRows, 1);
    // no keys at all: nothing is copied, but a map needs a row
    const void* kv = a.Nk > 0 ? a.kv : a.q;
    const void* rope = a.Nk > 0 ? a.k_rope : a.q;
    const long long nk = a.Nk > 0 ? a.Nk : 1;
    if (e == cudaSuccess)
        e = a.Nk > 0 ? encode_rows(&kvmap, kv, kw, kw, nk, kRows, 1)
                     : encode_rows(&kvmap, kv, 64, 64, nk, kRows, 1);
    if (e == cudaSuccess) e = encode_rows(&ropemap, rope, a.P, a.P, nk, kRows, 1);
    const ExpandedLayout L(a.Dn);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(expanded_mma_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 L.total);
    if (e != cudaSuccess) return e;
    const int units = (a.Nq + 2 * kRows - 1) / (2 * kRows) + a.Q;
    return launch_pdl(expanded_mma_kernel, dim3(a.H, units), dim3(kThreads), L.total, stream, a,
                      qmap, kvmap, ropemap);
}

}  // namespace kvd
