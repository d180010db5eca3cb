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
// queries.  Warp 8 issues the MMAs.  Warp 9 looks up pages and issues the copies.  Warp 10
// writes what the merge has to know.
//
// Measured, 64 sequences x 32 / 8 heads of 128 behind 16384 tokens: a step of 256 rows x 128
// keys takes 1.7 us, 1.17 of them the tensor cores' at the rate of a large matrix product;
// the kernel alone 25 us, of which 4 go before the first copy (lengths, division, table),
// 5 on the first copy and the first softmax, 12 on seven steps and 3 on the rows.  With
// the attention over own tokens (154 MB) and the merge the call takes 58 us; HBM needs 33.
// Not kept: an idle warp that asks L2 for the tiles two to eight steps ahead (+1 to +5 us: the
// ring's two steps are not what waits), scores taken 32 or 64 at a time in a loop
// (2 us less there, but 2 more for 4 sequences behind 1000 tokens).
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
constexpr int kMmaWarp = 8, kCopyWarp = 9;
constexpr int kMetaWarp = 10;
constexpr int kThreads = 384;  // warp 11 completes the third warpgroup
// Registers a thread: the softmax holds a row of 128 scores.  2 x 208 + 80 is
// within the 3 x 168 that three warpgroups start with.
constexpr int kSoftmaxRegs = 208, kIssueRegs = 80;
constexpr float kSkip = 8.f;  // log2 units by which a maximum may rise before the output is rescaled
constexpr uint32_t kTmemCols = 512;

struct MmaShared {
    alignas(16) uint32_t valid[kValid][4];  // keys of a step that count
    uint64_t q_full[2], k_full[kSteps], v_full[kSteps], empty[kRing];
    uint64_t s_full[2], p_full[2], o_full[2], drain;
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
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    if (a.keys < kRows) {  // rows of a block that no page reaches stay zero
        for (int i = tid; i < kRing * kBlock / 16; i += kThreads)
            reinterpret_cast<uint4*>(ring)[i] = make_uint4(0, 0, 0, 0);
        fence_async_smem();
    }
    pdl_wait();
    tc_fence_before();
    const PrefixRuns runs = prefix_setup<kThreads>(a, sh.groups);  // with barriers
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    volatile int* abort_flag = &sh.abort;
    const int w = blockIdx.x;
    const bool works = runs.tot > 0 && w < runs.W;
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
            // first row in the cache of piece p of key tile k, or -1
            auto source = [&](int k, int p) {
                const int key = k * a.keys + p * piece;
                if (p >= pieces || key >= n) return -1;
                const int page = by_page(key), phys = __ldg(table + page);
                return phys < 0 || phys >= a.NB ? -2 : phys * a.BS + key - page * a.BS;
            };
            for (int k = s.k0; k < s.k1 && !bad; ++k, ++it) {
                int src[4];  // first row of this lane's pieces in the cache
                uint32_t valid[4] = {0u, 0u, 0u, 0u};
                int loads = 0;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    src[u] = -1;
                    if (32 * u >= pieces) continue;
                    src[u] = source(k, lane + 32 * u);
                    const int b0 = (lane + 32 * u) * piece;
                    if (src[u] == -2) report(a.dev_status, KVD_DEV_BLOCK_RANGE);
                    if (src[u] >= 0)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            valid[x] |= range_word(b0, b0 + min(piece, n - k * a.keys - b0), x);
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
    } else if (warp == kMetaWarp) {
        prefix_meta(a, sh.groups, runs, lane, 32);
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMA issue
        // One warp in a fixed order, S0(0) S1(0) PV0(0) S0(1) PV1(0) S1(1) PV0(1) ..: a warp
        // per tile leaves the tiles in step (the products of both, then the softmax of
        // both: 4400 cycles a step).
        constexpr int kN = 64 * KC;
        const uint32_t sdesc = mma_desc(kRows, kRows), odesc = mma_desc(kRows, kN, kBMn);
        const uint32_t tm = uniform(tmem), base = uniform(smem_u32(ring));
        const uint32_t q_base = uniform(smem_u32(sm));
        int it = 0, cnt[2] = {0, 0}, seg[2] = {0, 0};
        // scores of tile s, step i; the keys are free behind the last tile's
        auto scores = [&](int s, int i, bool last) {
            const uint32_t q_low = uniform(desc_low(q_base + s * KC * kBlock, 16));
            const uint32_t k_low = uniform(desc_low(base + (i * per) % kRing * kBlock, 16));
            if (elect_one()) {
#pragma unroll
                for (int c = 0; c < KC; ++c)
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        mma_ss(tm + s * kRows, desc_of(q_low + ((c * kBlock) >> 4) + 2 * z),
                               desc_of(k_low + ((c * kBlock) >> 4) + 2 * z), sdesc, c > 0 || z > 0);
                // the copying warp's valid words (this warp has waited for the keys) are
                // ordered before the softmax's reads by an arrival of its own
                mbar_arrive(&sh.s_full[s]);
                mma_commit(&sh.s_full[s]);
                if (last)
#pragma unroll
                    for (int c = 0; c < KC; ++c) mma_commit(&sh.empty[(i * per + c) % kRing]);
            }
            __syncwarp();
        };
        auto values = [&](int s, int i, bool keep, bool end, bool last) {
            const uint32_t v_low =
                uniform(desc_low(base + (i * per + KC) % kRing * kBlock, KC > 1 ? kBlock : 16));
            if (elect_one()) {
#pragma unroll
                for (int z = 0; z < 8; ++z)
                    mma_ts(tm + 256 + s * kRows, tm + s * kRows + 8 * z,
                           desc_of(v_low + ((z * 2048) >> 4)), odesc, z > 0 || keep);
                if (end) mma_commit(&sh.o_full[s]);
                if (last)
#pragma unroll
                    for (int c = 0; c < KC; ++c) mma_commit(&sh.empty[(i * per + KC + c) % kRing]);
            }
            __syncwarp();
        };
        auto await = [&](uint64_t* bar, uint32_t parity) {
            if (!bad && !warp_wait(bar, parity, abort_flag)) bad = true;
            return !bad;
        };
        for (int p = lo; p < hi && !bad;) {
            const PrefixPiece pc = prefix_piece(a, sh.groups, w, lo, hi, p);
            p = uniform(pc.next);
            const int n = uniform(max(pc.k1 - pc.k0, 0)), tiles = uniform(rows_of(pc)) > kRows ? 2 : 1;
            if (n == 0) continue;
            const int first = it, end = it + n;
            await(&sh.k_full[it % kSteps], (it / kSteps) & 1);
            for (int s = 0; s < tiles; ++s) {
                if (!await(&sh.q_full[s], seg[s]++ & 1)) break;
                tc_fence_after();
                scores(s, it, s + 1 == tiles);
            }
            for (; it < end && !bad; ++it) {
                await(&sh.v_full[it % kSteps], (it / kSteps) & 1);
                for (int s = 0; s < tiles && !bad; ++s) {
                    if (!await(&sh.p_full[s], cnt[s]++ & 1)) break;
                    tc_fence_after();
                    values(s, it, it > first, it + 1 == end, s + 1 == tiles);
                    if (it + 1 < end) {
                        if (!await(&sh.k_full[(it + 1) % kSteps], ((it + 1) / kSteps) & 1)) break;
                        tc_fence_after();
                        scores(s, it + 1, s + 1 == tiles);
                    }
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
                // whole rows at a time: D / 8 lanes a row
                constexpr int kLanes = D / 8, kAt = 32 / kLanes;
                const uint4* q = static_cast<const uint4*>(a.q);
                const int j = lane % kLanes;
                unsigned char* to = sm + (s * KC + j / 8) * kBlock;
                const uint32_t rows_live = __ballot_sync(0xffffffffu, live);
#pragma unroll
                for (int i0 = 0; i0 < kLanes; i0 += kLanes) {
                    uint4 x[kLanes];
#pragma unroll
                    for (int i = 0; i < kLanes; ++i) {
                        const int r = (i0 + i) * kAt + lane / kLanes;
                        const unsigned long long from = __shfl_sync(0xffffffffu, (unsigned long long)at, r);
                        x[i] = (rows_live >> r) & 1u ? q[from * kLanes + j] : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < kLanes; ++i) {
                        const int row = 32 * (warp & 3) + (i0 + i) * kAt + lane / kLanes;
                        *reinterpret_cast<uint4*>(to + row * 128 + (((j & 7) ^ (row & 7)) << 4)) = x[i];
                    }
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
                    // bf16 as the matrix unit takes them beside bf16 values (2^-8 of each); their
                    // sum keeps fp32.  (Two bf16 words a weight, the second one's product added:
                    // bf16 outputs 1.7e-3 from 64 bits instead of 2.3e-3, but 64 sequences behind
                    // 16384 tokens 65 us instead of 55.5, 8 37.1 instead of 30.3.)
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
            // through shared memory, so that a store covers whole rows; kDims dims of the warp's
            // 32 rows at a time, in the place of the queries of the same rows: their products
            // are complete, and no other warp puts its next queries there
            constexpr int kDims = 32 * KC, kVecs = kDims / 4;
            float* out = pc.slot < 0 ? a.whole_o : a.part_o;
            unsigned char* stage = sm + s * KC * kBlock + (warp & 3) * 32 * 128;
            auto staged = [&](int r, int j) {  // 16-byte piece j of the warp's row r
                return reinterpret_cast<uint4*>(stage + (j >> 3) * kBlock + r * 128 +
                                                (((j ^ r) & 7) << 4));
            };
            const uint32_t rows_live = __ballot_sync(0xffffffffu, live);
#pragma unroll 1
            for (int c = 0; c < D; c += kDims) {
                for (int half = 0; half < (rows_live ? KC : 0); ++half) {
                    float o[32];
                    tmem_ld32(to + c + 32 * half, reinterpret_cast<uint32_t*>(o));
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        *staged(lane, 8 * half + e / 4) =
                            make_uint4(__float_as_uint(o[e] * inv), __float_as_uint(o[e + 1] * inv),
                                       __float_as_uint(o[e + 2] * inv), __float_as_uint(o[e + 3] * inv));
                    }
                }
                __syncwarp();
                const int count = __popc(rows_live);  // the warp's first rows
#pragma unroll 8
                for (int i = 0; i < kVecs; ++i) {
                    if ((32 / kVecs) * i >= count) break;
                    const int r = (32 / kVecs) * i + lane / kVecs, j = lane % kVecs;
                    const unsigned long long to_row =
                        __shfl_sync(0xffffffffu, (unsigned long long)row, r);
                    if ((rows_live >> r) & 1u)
                        *reinterpret_cast<uint4*>(out + to_row * D + c + 4 * j) =
                            *staged(r, j);
                }
                __syncwarp();
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
    // In clusters of two, for their place alone: the two SMs of a cluster share their way to
    // memory, and a CTA beside one of the attention over own tokens took half as long again.
    // So pairs go to the one or the other as a whole (64 sequences behind 16384 tokens: 63.2
    // -> 59.8 us).
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.workers);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, prefix_mma_kernel<KC>, a, piece, FastDiv(a.BS), FastDiv(a.g),
                              kmap, vmap);
}

}  // namespace

cudaError_t launch_prefix_mma(const PrefixArgs& a, cudaStream_t stream) {
    return a.D == 64 ? go_mma<1>(a, stream) : go_mma<2>(a, stream);
}

}  // namespace kvd
