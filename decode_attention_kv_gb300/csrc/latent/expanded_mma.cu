// expanded_mma.cu -- kvd_attend_expanded in bf16 on the tensor cores.
//
// A CTA holds two tiles of 128 queries of one head (one where there are few) and
// walks the keys 128 at a time: S_s = Q_s . K^T and O_s += P_s . V for s = 0, 1 in turn, so that one
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
// What bounds it: the chain of a step (softmax 1160 cycles, hand-overs, products
// 1500) is 3300 cycles against 2616 of MMA time for both tiles: 218 us in a graph, 220
// as called (1560 TFLOP/s) at one sequence of 8192 x 16 heads; 330 us in a graph over
// the same inputs, 350 as called over inputs in turn (1220 TFLOP/s) at four of 1024 to
// 4096 x 32 heads, where starting and ending a unit counts.
//
// Warps 0-3 and 4-7: softmax of tile 0 and 1, a row a thread.  Warps 8 and 9
// issue the MMAs of tile 0 and 1: what one spends on waiting and setting up (450
// cycles a step) the other's products fill.  Warp 10 issues the copies.
#include "../kvd_internal.h"
#include "latent_common.cuh"
#include "tcgen05_ptx.cuh"

namespace kvd {
namespace {

constexpr int kRows = 128;               // queries of a tile, keys of a step
constexpr int kBlock = kRows * 128;      // bytes of 128 rows x 64 bf16
constexpr int kRing = 8;                 // blocks in flight
constexpr int kSteps = 4;                // steps with barriers of their own (the ring holds fewer)
constexpr int kMmaWarp = 8, kCopyWarp = 10;
constexpr int kThreads = 384;  // warp 11 completes the third warpgroup
// Registers a thread: the softmax holds a row of 128 scores.  2 x 208 + 80 is
// within the 3 x 168 that three warpgroups start with.
constexpr int kSoftmaxRegs = 208, kIssueRegs = 80;
constexpr float kSkip = 8.f;             // log2 units
constexpr uint32_t kTmemCols = 512;

struct ExpandedShared {
    uint64_t q_full[2], k_full[kSteps], v_full[kSteps], empty[kRing];
    uint64_t s_full[2], p_full[2], o_full[2], turn, drain[2];
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

template <int KC, int VC>  // blocks of a step: keys (Dn / 64 + 1), values (Dv / 64)
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
    constexpr int per = KC + VC;

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.q_full[s], 1);
            mbar_init(&sh.s_full[s], 1);
            mbar_init(&sh.p_full[s], kRows / 32);
            mbar_init(&sh.o_full[s], 1);
        }
        for (int i = 0; i < kSteps; ++i) {
            mbar_init(&sh.k_full[i], 1);
            mbar_init(&sh.v_full[i], 1);
        }
        for (int i = 0; i < kRing; ++i) mbar_init(&sh.empty[i], 2);  // both tiles are done with it
        mbar_init(&sh.turn, 1);
        mbar_init(&sh.drain[0], 1);
        mbar_init(&sh.drain[1], 1);
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

    const Found f =
        packed_find<kThreads>(a, sh.scratch, unit, a.span_log, h == 0 && unit == 0);
    const PackedSeq seq = f.item < a.Q ? packed_seq(a, f.item) : PackedSeq{0, 0, 0, 0, 0u, false};
    const bool some = seq.nq > 0;
    // the last unit of a sequence first: under the causal mask it sees most keys
    const int units = (seq.nq + (1 << a.span_log) - 1) >> a.span_log;
    const int row0 = some ? (units - 1 - (unit - f.before)) << a.span_log : 0;
    const int behind = min(seq.nq, row0 + (1 << a.span_log));  // the first row that is not its
    const int shift = seq.nk - seq.nq;  // query i sees the keys 0 .. i + shift
    int steps[2];                       // key tiles that each query tile sees
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int first = row0 + s * kRows, rows = min(kRows, behind - first);
        const int keys = rows <= 0 ? 0
                         : a.causal ? max(0, min(seq.nk, first + rows + shift))
                                    : seq.nk;
        steps[s] = (keys + kRows - 1) / kRows;
    }
    const int nsteps = max(steps[0], steps[1]);
    bool bad = false;

    if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
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
            auto queries = [&](int s) {
                if (elect_one()) {
                    mbar_arrive_expect_tx(&sh.q_full[s], KC * kBlock);
#pragma unroll
                    for (int c = 0; c < KC; ++c)
                        tma_g2s_3d(sm + (s * KC + c) * kBlock, &qmap, 0,
                                   seq.q0 + row0 + s * kRows, qchunk + c, &sh.q_full[s], policy);
                }
                __syncwarp();
            };
            for (int i = 0; i < n && !bad; ++i) {
                const int row = uniform(seq.k0 + i * kRows);
                uint64_t* kf = &sh.k_full[i % kSteps];
                uint64_t* vf = &sh.v_full[i % kSteps];
                if (i == 0 && steps[0] > 0) queries(0);
                if (elect_one()) {
                    mbar_arrive_expect_tx(kf, KC * kBlock);
                    mbar_arrive_expect_tx(vf, VC * kBlock);
                }
                __syncwarp();
                for (int c = 0; c + 1 < KC && !bad; ++c) bad = !block(&kvmap, row, kchunk + c, kf);
                if (!bad) bad = !block(&ropemap, row, 0, kf);
                // behind the first keys: tile 1 starts half a step later
                if (i == 0 && steps[1] > 0) queries(1);
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
    } else if (warp < kCopyWarp) {
        // ------------------------------------------------------------ MMA issue
        // (What an MMA is issued with goes through uniform(), see latent_mma.cu.)
        const int s = uniform(warp - kMmaWarp);
        const uint32_t sdesc = mma_desc(kRows, kRows), odesc = mma_desc(kRows, 64, kBMn);
        const uint32_t base = uniform(smem_u32(sm)), tm = uniform(tmem);
        const uint32_t q_low = uniform(desc_low(base + s * KC * kBlock, 16));
        const uint32_t td = uniform(tm + s * kRows), to = uniform(tm + 256 + s * kRows);
        const int n = uniform(nsteps), ns = uniform(steps[s]);
        uint32_t k_low[KC];  // the key blocks of the next scores
        auto keys_of = [&](int i) {
#pragma unroll
            for (int c = 0; c < KC; ++c)
                k_low[c] = uniform(desc_low(base + L.ring + (i * per + c) % kRing * kBlock, 16));
        };
        // scores of step i; then its blocks are free as far as this tile goes
        auto scores = [&](int i) {
            if (elect_one()) {
#pragma unroll
                for (int c = 0; c < KC; ++c)
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        mma_ss(td, desc_of(q_low + ((c * kBlock) >> 4) + 2 * z),
                               desc_of(k_low[c] + 2 * z), sdesc, c > 0 || z > 0);
                mma_commit(&sh.s_full[s]);
#pragma unroll
                for (int c = 0; c < KC; ++c) mma_commit(&sh.empty[(i * per + c) % kRing]);
            }
            __syncwarp();
        };
        if (ns > 0) {
            // tile 1 starts half a step behind tile 0, so that one's products and the
            // other's softmax take turns from the first step on
            if (s == 1 && n > 0 && steps[0] > 0) bad = !warp_wait(&sh.turn, 0, abort_flag);
            bad = bad || !warp_wait(&sh.q_full[s], 0, abort_flag) ||
                  !warp_wait(&sh.k_full[0], 0, abort_flag);
            tc_fence_after();
            keys_of(0);
            if (!bad) scores(0);
        }
        for (int i = 0; i < ns && !bad; ++i) {
            const uint32_t keep = uniform((int)(i > 0));
            const int b0 = i * per + KC;
            uint32_t v_low[VC];
#pragma unroll
            for (int c = 0; c < VC; ++c)
                v_low[c] = uniform(desc_low(base + L.ring + (b0 + c) % kRing * kBlock, 16));
            keys_of(i + 1);
            // looked at while the softmax still runs; not waited for before the values,
            // whose blocks the keys' copies may need
            uint64_t* kf = &sh.k_full[(i + 1) % kSteps];
            const uint32_t kpar = ((i + 1) / kSteps) & 1;
            if (!warp_wait(&sh.v_full[i % kSteps], (i / kSteps) & 1, abort_flag)) {
                bad = true;
                break;
            }
            const bool keys = i + 1 < ns && __all_sync(0xffffffffu, mbar_test(kf, kpar));
            if (!warp_wait(&sh.p_full[s], i & 1, abort_flag)) {
                bad = true;
                break;
            }
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int c = 0; c < VC; ++c)
#pragma unroll
                    for (int z = 0; z < 8; ++z)
                        mma_ts(to + 64 * c, td + 8 * z, desc_of(v_low[c] + ((z * 2048) >> 4)),
                               odesc, z > 0 || keep);
#pragma unroll
                for (int c = 0; c < VC; ++c) mma_commit(&sh.empty[(b0 + c) % kRing]);
                if (i + 1 == ns) mma_commit(&sh.o_full[s]);
                if (s == 0 && i == 0) mbar_arrive(&sh.turn);
            }
            __syncwarp();
            if (i + 1 < ns) {
                if (!keys && !warp_wait(kf, kpar, abort_flag)) {
                    bad = true;
                    break;
                }
                tc_fence_after();
                scores(i + 1);
            }
        }
        // steps that only the other tile takes
        for (int i = ns; i < n && !bad; ++i) {
            if (!warp_wait(&sh.v_full[i % kSteps], (i / kSteps) & 1, abort_flag)) {
                bad = true;
                break;
            }
            if (elect_one())
                for (int c = 0; c < per; ++c) mbar_arrive(&sh.empty[(i * per + c) % kRing]);
            __syncwarp();
        }
        if (bad) {
            if (lane == 0) sh.abort = 1;
            __syncwarp();
            if (elect_one()) mma_commit(&sh.drain[s]);
            __syncwarp();
            const unsigned long long since = global_timer_ns();
            while (!mbar_try_wait(&sh.drain[s], 0) && global_timer_ns() - since < kWaitLimitNs) {
            }
        }
    }
    } else {
        // ------------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int s = warp >> 2;
        const int row = row0 + s * kRows + 32 * (warp & 3) + lane;  // in the sequence
        const bool live = some && row < behind;
        const uint32_t quarter = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + s * kRows + quarter, to = tmem + 256 + s * kRows + quarter;
        const int last = !live ? -1 : a.causal ? min(seq.nk - 1, row + shift) : seq.nk - 1;
        // newest key that every row of the warp sees
        const int all_see = __reduce_min_sync(0xffffffffu, live ? last : 0x3fffffff);
        const bool flip = a.qscale < 0.f;
        const float qs = fmaxf(fabsf(a.qscale), kTinyScale);
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
            float x[kRows];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                tmem_ld32(ts + 32 * c, reinterpret_cast<uint32_t*>(x + 32 * c));
            tmem_wait_ld();
            if (flip) {
#pragma unroll
                for (int e = 0; e < kRows; ++e) x[e] = -x[e];
            }
            if (masked) {
#pragma unroll
                for (int e = 0; e < kRows; ++e)
                    if (e > lim) x[e] = -INFINITY;
            }
            float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int e = 4; e < kRows; e += 8) {
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    mx[z] = e + 4 + z < kRows ? fmaxf(mx[z], fmaxf(x[e + z], x[e + 4 + z]))
                                              : fmaxf(mx[z], x[e + z]);
            }
            const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * qs);
            if (i == 0) m = mn;
            const bool need = mn > m + kSkip;
            if (__any_sync(0xffffffffu, need)) {
                const float fac = need ? exp2f(m - mn) : 1.f;
                if (need) m = mn;
                l *= fac;
                for (int c = 0; c < a.Dv; c += 16) {
                    float o[16];
                    tmem_ld16(to + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] *= fac;
                    tmem_st16(to + c, o);
                }
            }
            const float base = m == -INFINITY ? 0.f : m;
            const float2 q2 = make_float2(qs, qs), b2 = make_float2(-base, -base);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                // over scores that have been read: 16 columns hold 32 weights, rounded to
                // bf16 as the matrix unit takes them (2^-8 of each); their sum keeps fp32
                float p[16];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float2 y =
                        ffma2(make_float2(x[32 * c + e], x[32 * c + e + 1]), q2, b2);
                    const float2 z = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                    sum[(e >> 1) & 1] = fadd2(sum[(e >> 1) & 1], z);
                    p[e >> 1] = __uint_as_float(pack_bf16(z.x, z.y));
                }
                tmem_st16(ts + 16 * c, p);
            }
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
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
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[s]);  // one arrival a warp
        }
        if (ns > 0 && !bad && !mbar_wait(&sh.o_full[s], 0, abort_flag)) bad = true;
        if (__any_sync(0xffffffffu, bad)) {
            bad = true;
            sh.abort = 1;
        }
        __syncwarp();
        if (!bad) {
            tc_fence_after();
            // a scale of NaN (the weights above do without it): every query that sees a key
            if (a.qscale != a.qscale && l != 0.f) l = a.qscale;
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

template <int KC, int VC>
cudaError_t go_expanded(const ExpandedArgs& a, const CUtensorMap& qmap, const CUtensorMap& kvmap,
                        const CUtensorMap& ropemap, cudaStream_t stream) {
    const ExpandedLayout L(a.Dn);
    const cudaError_t e = cudaFuncSetAttribute(
        expanded_mma_kernel<KC, VC>, cudaFuncAttributeMaxDynamicSharedMemorySize, L.total);
    if (e != cudaSuccess) return e;
    const int units = ((a.Nq - 1) >> a.span_log) + 1 + a.Q;
    return launch_pdl(expanded_mma_kernel<KC, VC>, dim3(a.H, units), dim3(kThreads), L.total,
                      stream, a, qmap, kvmap, ropemap);
}

}  // namespace

cudaError_t launch_expanded_mma(const ExpandedArgs& args, cudaStream_t stream) {
    ExpandedArgs a = args;
    // One query tile a CTA where all CTAs still run at once: the tensor cores wait, but
    // a step is over sooner (in a graph: 300 x 8 heads 10.8 -> 9.4 us, 1024 x 16 20.1 ->
    // 17.0, 2048 x 8 32.3 -> 28.5; but 4 x 512 x 16, 256 CTAs of work, 16.4 -> 21.5).
    a.span_log = (long long)a.H * ((a.Nq - 1) / kRows + 1 + a.Q) <= kLatentSMs ? 7 : 8;
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
    if (e != cudaSuccess) return e;
    auto go = a.Dn == 128 ? (a.Dv == 128 ? go_expanded<3, 2> : go_expanded<3, 1>)
                          : (a.Dv == 128 ? go_expanded<2, 2> : go_expanded<2, 1>);
    return go(a, qmap, kvmap, ropemap, stream);
}

}  // namespace kvd
