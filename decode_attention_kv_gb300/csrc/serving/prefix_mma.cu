// prefix_mma.cu -- the shared prefixes of kvd_attend_paged_prefix in bf16 on the tensor
// cores.
//
// The query heads of a kv head over all sequences of a group are the rows of a matrix:
// S = Q . K^T and O += P . V, so that a prefix row is read once for 256 of them.  A CTA
// takes an equal run of the line of key tiles (serving_common.cuh) with two tiles of 128
// rows (one where a group has no more) and 128 keys at a time; the two tiles go through
// the tensor cores in turn, so that one's softmax runs under the other's products.
// Tensor memory: two score tiles, whose weights replace them and are the A operand from
// there, and two outputs.  MMAs of one thread run in order, so the next scores may
// overwrite weights whose product was issued before, and a complete score tile tells
// that the product before it is complete too: the softmax may rescale its output
// without another wait.
//
// Keys and values arrive page by page (boxes of the page size's largest divisor not
// above 128 rows) in a ring of eight blocks of 128 tokens x 64 elements.
//
// Warps 0-3 and 4-7: softmax of tile 0 and 1, a row a thread; they also lay out the
// queries.  Warps 8 and 9 issue the MMAs of tile 0 and 1.  Warp 10 looks up pages and
// issues the copies.
#include "../kvd_internal.h"
#include "../latent/latent_common.cuh"  // encode_rows, FastDiv, kTinyScale
#include "../latent/tcgen05_ptx.cuh"
#include "serving_common.cuh"

namespace kvd {
namespace {

constexpr int kRows = 128;           // queries of a tile, keys of a step
constexpr int kBlock = kRows * 128;  // bytes of 128 rows x 64 bf16
constexpr int kRing = 8;             // blocks in flight
constexpr int kSteps = 4;            // steps with barriers of their own (the ring holds no more)
// Steps whose valid words are kept: those of step i are written when the scores of step
// i - 4 at the latest are complete, so that step i - 5 has been through the softmax.
constexpr int kValid = 8;
constexpr int kMmaWarp = 8, kCopyWarp = 10;
constexpr int kThreads = 384;  // warp 11 completes the third warpgroup
// Registers a thread: the softmax holds a row of 128 scores.  2 x 208 + 80 is
// within the 3 x 168 that three warpgroups start with.
constexpr int kSoftmaxRegs = 208, kIssueRegs = 80;
constexpr float kSkip = 8.f;  // log2 units by which a maximum may rise before the output is rescaled
constexpr uint32_t kTmemCols = 512;

struct MmaShared {
    alignas(16) uint32_t valid[kValid][4];  // keys of a step that count
    uint64_t q_full[2], k_full[kSteps], v_full[kSteps], empty[kRing];
    uint64_t s_full[2], p_full[2], o_full[2], turn, drain[2];
    uint32_t tmem;
    int abort;
    PrefixGroups groups;
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

// 32 bytes of a row of partial results.
__device__ __forceinline__ void store8(float* p, const float* x) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]),
                 "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
}

// Bits [b0, b1) of four words.
__device__ __forceinline__ uint32_t range_word(int b0, int b1, int w) {
    const int lo = max(b0 - 32 * w, 0), hi = min(b1 - 32 * w, 32);
    return lo >= hi ? 0u : (hi - lo == 32 ? 0xffffffffu : ((1u << (hi - lo)) - 1u) << lo);
}

template <int KC>  // blocks of 64 dims
__global__ void __launch_bounds__(kThreads, 1)
prefix_mma_kernel(const PrefixArgs a, const int piece, const FastDiv by_page, const FastDiv by_head,
                  const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    constexpr int per = 2 * KC, D = 64 * KC;
    extern __shared__ __align__(1024) unsigned char raw[];
    unsigned char* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    unsigned char* ring = sm + 2 * KC * kBlock;
    MmaShared& sh = *reinterpret_cast<MmaShared*>(ring + kRing * kBlock);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.q_full[s], kRows / 32);
            mbar_init(&sh.s_full[s], 2);  // the scores; the valid words
            mbar_init(&sh.p_full[s], kRows / 32);
            mbar_init(&sh.o_full[s], 1);
            mbar_init(&sh.drain[s], 1);
        }
        for (int i = 0; i < kSteps; ++i) {
            mbar_init(&sh.k_full[i], 1);
            mbar_init(&sh.v_full[i], 1);
        }
        for (int i = 0; i < kRing; ++i) mbar_init(&sh.empty[i], 2);  // both tiles are done with it
        mbar_init(&sh.turn, 1);
        sh.abort = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) tmem_alloc(&sh.tmem, kTmemCols);
    if (warp == kCopyWarp && lane == 0) {
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    if (a.keys < kRows) {  // rows of a block that no page reaches stay zero
        for (int i = tid; i < kRing * kBlock / 16; i += kThreads)
            reinterpret_cast<uint4*>(ring)[i] = make_uint4(0, 0, 0, 0);
        fence_async_smem();
    }
    pdl_launch_dependents();
    pdl_wait();
    tc_fence_before();
    const int tot = prefix_setup<kThreads>(a, sh.groups);  // ends with a barrier
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    volatile int* abort_flag = &sh.abort;
    const PrefixRuns runs(tot, a.workers);
    const int w = blockIdx.x;
    const bool works = tot > 0 && w < runs.W;
    const int lo = works ? runs.start(w) : 0, hi = works ? runs.start(w + 1) : 0;
    bool bad = false;

    // query rows of a piece in its tile
    auto rows_of = [&](const PrefixPiece& s) {
        return min(a.rows, sh.groups.sequences(s.group) * a.g - s.tile * a.rows);
    };

    if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == kCopyWarp) {
        // ------------------------------------------------------------ copies
        const uint64_t policy = policy_evict_normal();  // other heads' tiles read the same lines
        const int pieces = kRows / piece;
        const uint32_t bytes = (uint32_t)piece * 128u;
        int it = 0, slot = 0;
        uint32_t lap = 0;
        for (int p = lo; p < hi && !bad;) {
            const PrefixPiece s = prefix_piece(a, sh.groups, w, lo, hi, p);
            p = s.next;
            const int n = sh.groups.keys[s.group], chunk = s.head * KC;
            const int32_t* table = a.prefix_tables + (size_t)s.group * a.pcols;
            for (int k = s.k0; k < s.k1 && !bad; ++k, ++it) {
                int src[4];  // first row of this lane's pieces in the cache, or -1
                uint32_t valid[4] = {0u, 0u, 0u, 0u};
                int loads = 0;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    src[u] = -1;
                    if (32 * u >= pieces) continue;
                    const int b0 = (lane + 32 * u) * piece, key = k * a.keys + b0;
                    if (lane + 32 * u < pieces && key < n) {
                        const int page = by_page(key), phys = __ldg(table + page);
                        if (phys < 0 || phys >= a.NB) {
                            report(a.dev_status, KVD_DEV_BLOCK_RANGE);
                        } else {
                            src[u] = phys * a.BS + key - page * a.BS;
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                valid[x] |= range_word(b0, b0 + min(piece, n - key), x);
                        }
                    }
                    loads += __popc(__ballot_sync(0xffffffffu, src[u] >= 0));
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) valid[x] = __reduce_or_sync(0xffffffffu, valid[x]);
                uint64_t* kf = &sh.k_full[it % kSteps];
                uint64_t* vf = &sh.v_full[it % kSteps];
                auto blocks = [&](const CUtensorMap* map, uint64_t* full) {
                    for (int c = 0; c < KC; ++c)
                        if (lap > 0 && !warp_wait(&sh.empty[slot + c], (lap - 1) & 1, abort_flag))
                            return false;
                    if (lane == 0) mbar_arrive_expect_tx(full, loads * bytes * KC);
                    __syncwarp();
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        if (src[u] < 0) continue;
#pragma unroll
                        for (int c = 0; c < KC; ++c)
                            tma_g2s_3d(ring + (slot + c) * kBlock + (lane + 32 * u) * bytes, map, 0,
                                       src[u], chunk + c, full, policy);
                    }
                    __syncwarp();
                    slot += KC;
                    if (slot == kRing) {
                        slot = 0;
                        ++lap;
                    }
                    return true;
                };
                // before the words of the step: its blocks are free
                const bool free = lap == 0 || warp_wait(&sh.empty[slot], (lap - 1) & 1, abort_flag);
                if (lane == 0)
                    *reinterpret_cast<uint4*>(sh.valid[it % kValid]) =
                        make_uint4(valid[0], valid[1], valid[2], valid[3]);
                __syncwarp();
                bad = !free || !blocks(&kmap, kf) || !blocks(&vmap, vf);
            }
        }
        if (bad) {
            if (lane == 0) sh.abort = 1;
            // blocks still in flight land within the limit; nothing reads them
            const unsigned long long since = global_timer_ns();
            while (global_timer_ns() - since < 1000000ull) {
            }
        }
    } else if (warp < kCopyWarp) {
        // ------------------------------------------------------------ MMA issue
        const int s = uniform(warp - kMmaWarp);
        const uint32_t sdesc = mma_desc(kRows, kRows), odesc = mma_desc(kRows, 64, kBMn);
        const uint32_t tm = uniform(tmem);
        const uint32_t q_low = uniform(desc_low(smem_u32(sm) + s * KC * kBlock, 16));
        const uint32_t td = uniform(tm + s * kRows), to = uniform(tm + 256 + s * kRows);
        const uint32_t base = uniform(smem_u32(ring));
        int it = 0, cnt = 0, seg = 0;
        uint32_t k_low[KC];
        auto keys_of = [&](int i) {
#pragma unroll
            for (int c = 0; c < KC; ++c)
                k_low[c] = uniform(desc_low(base + (i * per + c) % kRing * kBlock, 16));
        };
        auto scores = [&](int i) {
            if (elect_one()) {
#pragma unroll
                for (int c = 0; c < KC; ++c)
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        mma_ss(td, desc_of(q_low + ((c * kBlock) >> 4) + 2 * z),
                               desc_of(k_low[c] + 2 * z), sdesc, c > 0 || z > 0);
                // the copying warp's valid words (this warp has waited for the keys) are
                // ordered before the softmax's reads by an arrival of its own
                mbar_arrive(&sh.s_full[s]);
                mma_commit(&sh.s_full[s]);
#pragma unroll
                for (int c = 0; c < KC; ++c) mma_commit(&sh.empty[(i * per + c) % kRing]);
            }
            __syncwarp();
        };
        for (int p = lo; p < hi && !bad;) {
            const PrefixPiece pc = prefix_piece(a, sh.groups, w, lo, hi, p);
            p = uniform(pc.next);
            const int n = uniform(max(pc.k1 - pc.k0, 0)), rows = uniform(rows_of(pc));
            if (n == 0) continue;
            const int end = it + n;
            if (s * kRows >= rows) {  // only the other tile has rows
                for (; it < end && !bad; ++it) {
                    if (!warp_wait(&sh.v_full[it % kSteps], (it / kSteps) & 1, abort_flag)) {
                        bad = true;
                        break;
                    }
                    if (elect_one())
                        for (int c = 0; c < per; ++c) mbar_arrive(&sh.empty[(it * per + c) % kRing]);
                    __syncwarp();
                }
                continue;
            }
            // tile 1 starts half a step behind tile 0, so that one's products and the
            // other's softmax take turns from the first step on
            if (s == 1 && it == 0) bad = !warp_wait(&sh.turn, 0, abort_flag);
            bad = bad || !warp_wait(&sh.q_full[s], seg & 1, abort_flag) ||
                  !warp_wait(&sh.k_full[it % kSteps], (it / kSteps) & 1, abort_flag);
            ++seg;
            tc_fence_after();
            keys_of(it);
            if (!bad) scores(it);
            for (int i0 = it; it < end && !bad; ++it, ++cnt) {
                const uint32_t keep = uniform((int)(it > i0));
                const int b0 = it * per + KC;
                uint32_t v_low[KC];
#pragma unroll
                for (int c = 0; c < KC; ++c)
                    v_low[c] = uniform(desc_low(base + (b0 + c) % kRing * kBlock, 16));
                keys_of(it + 1);
                uint64_t* kf = &sh.k_full[(it + 1) % kSteps];
                const uint32_t kpar = ((it + 1) / kSteps) & 1;
                if (!warp_wait(&sh.v_full[it % kSteps], (it / kSteps) & 1, abort_flag)) {
                    bad = true;
                    break;
                }
                // looked at while the softmax still runs; not waited for before the values,
                // whose blocks the keys' copies may need
                const bool keys = it + 1 < end && __all_sync(0xffffffffu, mbar_test(kf, kpar));
                if (!warp_wait(&sh.p_full[s], cnt & 1, abort_flag)) {
                    bad = true;
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int c = 0; c < KC; ++c)
#pragma unroll
                        for (int z = 0; z < 8; ++z)
                            mma_ts(to + 64 * c, td + 8 * z, desc_of(v_low[c] + ((z * 2048) >> 4)),
                                   odesc, z > 0 || keep);
#pragma unroll
                    for (int c = 0; c < KC; ++c) mma_commit(&sh.empty[(b0 + c) % kRing]);
                    if (it + 1 == end) mma_commit(&sh.o_full[s]);
                    if (s == 0 && it == 0) mbar_arrive(&sh.turn);
                }
                __syncwarp();
                if (it + 1 < end) {
                    if (!keys && !warp_wait(kf, kpar, abort_flag)) {
                        bad = true;
                        break;
                    }
                    tc_fence_after();
                    scores(it + 1);
                }
            }
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
        const int s = warp >> 2, in_tile = s * kRows + 32 * (warp & 3) + lane;
        const uint32_t quarter = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + s * kRows + quarter, to = tmem + 256 + s * kRows + quarter;
        const bool flip = a.qscale < 0.f;
        const float qs = fmaxf(fabsf(a.qscale), kTinyScale);
        int it = 0, cnt = 0, seg = 0;
        for (int p = lo; p < hi && !bad;) {
            const PrefixPiece pc = prefix_piece(a, sh.groups, w, lo, hi, p);
            p = pc.next;
            const int n = max(pc.k1 - pc.k0, 0), rows = rows_of(pc);
            if (n == 0) continue;
            if (s * kRows >= rows) {
                it += n;
                continue;
            }
            const bool live = in_tile < rows;
            size_t at = 0;  // output row
            {
                // the queries, under the 128-byte swizzle: 16-byte piece j of a row at j ^ (row % 8)
                const int r = pc.tile * a.rows + in_tile, seq = by_head(live ? r : 0);
                if (live)
                    at = (size_t)(sh.groups.start[pc.group] + seq) * a.Hq + pc.head * a.g + r - seq * a.g;
                const uint4* q = reinterpret_cast<const uint4*>(
                    static_cast<const __nv_bfloat16*>(a.q) + at * D);
                const int row = in_tile & (kRows - 1);
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    uint4 x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = live ? q[8 * c + j] : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        *reinterpret_cast<uint4*>(sm + (s * KC + c) * kBlock + row * 128 +
                                                  ((j ^ (row & 7)) << 4)) = x[j];
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.q_full[s]);
            }
            float m = -INFINITY, l = 0.f;
            for (int i = 0; i < n; ++i, ++it, ++cnt) {
                if (!mbar_wait(&sh.s_full[s], cnt & 1, abort_flag)) bad = true;
                if (__any_sync(0xffffffffu, bad)) {
                    bad = true;
                    break;
                }
                tc_fence_after();
                const uint4 valid = *reinterpret_cast<const uint4*>(sh.valid[it % kValid]);
                const bool whole = (valid.x & valid.y & valid.z & valid.w) == 0xffffffffu;
                float x[kRows];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_ld32(ts + 32 * c, reinterpret_cast<uint32_t*>(x + 32 * c));
                tmem_wait_ld();
                if (flip) {
#pragma unroll
                    for (int e = 0; e < kRows; ++e) x[e] = -x[e];
                }
                if (!whole) {
                    const uint32_t v[4] = {valid.x, valid.y, valid.z, valid.w};
#pragma unroll
                    for (int e = 0; e < kRows; ++e)
                        if (!((v[e >> 5] >> (e & 31)) & 1u)) x[e] = -INFINITY;
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
                    for (int c = 0; i > 0 && c < D; c += 16) {
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
                    float pk[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 y =
                            ffma2(make_float2(x[32 * c + e], x[32 * c + e + 1]), q2, b2);
                        const float2 z = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                        sum[(e >> 1) & 1] = fadd2(sum[(e >> 1) & 1], z);
                        pk[e >> 1] = __uint_as_float(pack_bf16(z.x, z.y));
                    }
                    tmem_st16(ts + 16 * c, pk);
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                if (!whole) {
                    // rows of other tokens: a weight of zero does not keep what they contain
                    // (NaN) out of the sum
                    if (!mbar_wait(&sh.v_full[it % kSteps], (it / kSteps) & 1, abort_flag)) bad = true;
                    const int row = tid & 127;
                    const uint32_t word = row < 64 ? (row < 32 ? valid.x : valid.y)
                                                   : (row < 96 ? valid.z : valid.w);
                    if (!((word >> (row & 31)) & 1u))
                        for (int c = 0; c < KC; ++c) {
                            unsigned char* v = ring + (it * per + KC + c) % kRing * kBlock + row * 128;
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                *reinterpret_cast<uint4*>(v + 16 * j) = make_uint4(0, 0, 0, 0);
                        }
                    fence_async_smem();
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_full[s]);  // one arrival a warp
            }
            if (!bad && !mbar_wait(&sh.o_full[s], seg & 1, abort_flag)) bad = true;
            ++seg;
            if (__any_sync(0xffffffffu, bad)) {
                bad = true;
                break;
            }
            tc_fence_after();
            // a scale of NaN (the weights above do without it): every query that sees a key
            if (a.qscale != a.qscale && l != 0.f) l = a.qscale;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const size_t row = pc.slot < 0 ? at : (size_t)pc.slot * a.rows + in_tile;
            float* out = (pc.slot < 0 ? a.whole_o : a.part_o) + row * D;
            for (int c = 0; c < D; c += 32) {
                float o[32];
                tmem_ld32(to + c, reinterpret_cast<uint32_t*>(o));
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= inv;
                if (live) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) store8(out + c + e, o + e);
                }
            }
            if (live)
                (pc.slot < 0 ? a.whole_lse : a.part_lse)[row] =
                    l > 0.f ? m + log2f(l) : (l == 0.f ? -INFINITY : NAN);
            tc_fence_before();
        }
        if (bad) sh.abort = 1;
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && sh.abort) report(a.dev_status, KVD_DEV_TIMEOUT);
    if (warp == kMmaWarp) tmem_free(tmem, kTmemCols);
}

template <int KC>
cudaError_t go_mma(const PrefixArgs& a, cudaStream_t stream) {
    const int piece = prefix_piece_rows(a.BS);
    const long long width = (long long)a.Hkv * a.D, rows = (long long)a.NB * a.BS;
    CUtensorMap kmap, vmap;
    cudaError_t e = encode_rows(&kmap, a.k, width, width, rows, piece, 1);
    if (e == cudaSuccess) e = encode_rows(&vmap, a.v, width, width, rows, piece, 1);
    if (e != cudaSuccess) return e;
    const int bytes = (2 * KC + kRing) * kBlock + (int)sizeof(MmaShared) + 1024;
    e = cudaFuncSetAttribute(prefix_mma_kernel<KC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             bytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(prefix_mma_kernel<KC>, dim3(a.workers), dim3(kThreads), bytes, stream, a,
                      piece, FastDiv(a.BS), FastDiv(a.g), kmap, vmap);
}

}  // namespace

cudaError_t launch_prefix_mma(const PrefixArgs& a, cudaStream_t stream) {
    return a.D == 64 ? go_mma<1>(a, stream) : go_mma<2>(a, stream);
}

}  // namespace kvd
