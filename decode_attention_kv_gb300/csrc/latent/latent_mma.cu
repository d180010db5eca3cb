// latent_mma.cu -- kvd_attend_latent in bf16 on the tensor cores.
//
// Per 64-key tile and up to 64 query rows (heads x drafted tokens):
//   S [64 rows, 64 keys]  = Q [64, R + P] . K^T    K-major operands, 36 MMAs at R = 512
//   O^T [R dims, N rows] += V^T [R, 64] . P^T      V^T is the K tile read MN-major,
//                                                  so a token is in shared memory once
// The output is kept transposed (dims on the lanes of tensor memory, rows on
// its columns): M is then always full, N is the number of rows, and 64 rows of
// R = 512 take 256 of the 512 columns.  Untransposed, 64 rows would leave half
// the lanes of a 512-column accumulator empty.
//
// Warps 0-3: softmax (four threads a row), rescaling, epilogue.  Warps 4 and 5
// issue the MMAs of the scores and of the values; the scores run up to two tiles
// ahead of the softmax.  Warps 6-9: tensor copies of the pages, a warp per pair of
// 64-wide chunks.  Warp 10: of the queries.
// The running output is rescaled only when some row's maximum rose by more
// than 8 (log2 units), as in the decode kernel: weights stay below 2^8.
//
// What bounds it: at 16 rows HBM (64 sequences of 512 to 8192 tokens, R = 512:
// 64.4 us with the merge in a graph, 65.5 as called from Python, 5.0 TB/s; 6.2 TB/s
// where 8 sequences of 100000 stream), at 64 rows the round of a stage (copy, scores,
// softmax, values: two tiles in 5900 cycles, 1920 of MMA time each; 16 sequences of
// 1001 to 16384, 128 rows: 90.8 us, as called 91.5, 744 TFLOP/s).  Two stages of 72 KB
// are what 72 KB of queries leave.
#include "../kvd_internal.h"
#include "latent_common.cuh"
#include "tcgen05_ptx.cuh"

namespace kvd {
namespace {

constexpr int kSoftmax = 128;            // threads of warps 0-3
constexpr int kCopyWarp = 6;              // the first of the copying warps, one per pair
constexpr int kQueryWarp = kCopyWarp + 4;  // copies the queries
constexpr int kThreads = 32 * (kQueryWarp + 1);
constexpr int kTile = 64;                // keys of an MMA tile, rows of the query tile
constexpr int kChunk = kTile * 128;      // bytes of 64 rows x 64 bf16
constexpr int kMaxStages = 4;
constexpr int kValid = 2 * kMaxStages;
constexpr int kMaxPairs = 4;             // R / 128
constexpr uint32_t kTmemCols = 512;
constexpr float kSkip = 8.f;             // log2 units

struct MmaShared {
    uint64_t full[kMaxStages][kMaxPairs];
    uint64_t empty[kMaxStages][kMaxPairs];
    uint64_t s_full[2], s_free[2];
    uint64_t p_full, pv_done, q_full, q_free, drain[2];
    unsigned long long valid[kValid];  // tile it's at it % kValid
    alignas(16) float factor[kTile];
    uint32_t tmem;
    int abort;
    int scratch[kFindWords];
};

// Dynamic shared memory: query tile | key stages | P tile | MmaShared.
struct MmaLayout {
    int chunks, stages;
    int q, kv, p, shared, total;
    __host__ __device__ explicit MmaLayout(int R) {
        chunks = R / 64 + 1;
        q = 0;
        kv = chunks * kChunk;
        const int room = 227 * 1024 - 1024 - kv - kChunk - (int)sizeof(MmaShared);
        stages = room / (chunks * kChunk);
        stages = stages > kMaxStages ? kMaxStages : stages;
        p = kv + stages * chunks * kChunk;
        shared = p + kChunk;
        total = shared + (int)sizeof(MmaShared) + 1024;  // 1024: alignment of the base
    }
};

// The tiles of one worker, sequence by sequence.
struct Walk {
    int t, t1, b, before;
    Runs runs;
    __device__ bool more() const { return t < t1; }
};

struct Segment {
    SeqInfo seq;
    int nt;     // tiles of the whole sequence
    int first;  // first tile of this worker
    int end;
};

__device__ __forceinline__ Segment segment(const LatentArgs& a, const Walk& k, FastDiv by_tile) {
    Segment s;
    s.seq = latent_seq(a, k.b);
    s.nt = max(1, by_tile.up(s.seq.n));
    // the run's part of the sequence's places: `lead` of them, then its tiles
    s.first = max(0, k.t - k.before - a.lead);
    s.end = min(s.nt, k.t1 - k.before - a.lead);
    return s;
}
// To the next sequence; a run that ends before that one's first tile is over.
__device__ __forceinline__ void advance(const LatentArgs& a, Walk& k, const Segment& s) {
    k.before += a.lead + s.nt;
    k.t = min(k.before, k.t1);
    if (k.t1 <= k.before + a.lead) k.t = k.t1;
    ++k.b;
}

// Reads this lane's dims of the transposed output (a dim per lane and pair of
// chunks, a row per column), multiplies each row by its factor and hands it on.
template <typename Put>
__device__ __forceinline__ void store_rows(uint32_t tm, int pairs, int N, int nrows,
                                           const float* factor, int R, Put put) {
    for (int c = 0; c < nrows; c += 16) {
        float f[16];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const float4 x = *reinterpret_cast<const float4*>(factor + c + i);
            f[i] = x.x;
            f[i + 1] = x.y;
            f[i + 2] = x.z;
            f[i + 3] = x.w;
        }
        const int n = min(16, nrows - c);
#pragma unroll 2
        for (int j = 0; j < pairs; ++j) {
            float o[16];
            tmem_ld16(tm + j * N + c, o);
            tmem_wait_ld();
            const size_t at = (size_t)c * R + 128 * j;
            if (n == 16) {
#pragma unroll
                for (int i = 0; i < 16; ++i) put(at + i * R, o[i] * f[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (i < n) put(at + i * R, o[i] * f[i]);
            }
        }
    }
}

// mbar_wait by a whole converged warp: every branch is a vote, so that the
// compiler sees a uniform control flow behind it.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    unsigned long long since = 0;
    while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
        const unsigned long long now = global_timer_ns();
        if (since == 0) since = now;
        if (__any_sync(0xffffffffu, *abort_flag || now - since > kWaitLimitNs)) return false;
    }
    return true;
}

// A wait ran out: tells the others and waits for this warp's own MMAs.
__device__ __forceinline__ void drain(uint64_t* bar, int* abort_flag) {
    *reinterpret_cast<volatile int*>(abort_flag) = 1;
    __syncwarp();
    if (elect_one()) mma_commit(bar);
    __syncwarp();
    const unsigned long long since = global_timer_ns();
    while (!mbar_try_wait(bar, 0) && global_timer_ns() - since < kWaitLimitNs) {
    }
    __syncwarp();
}

__global__ void __maxnreg__(144)
latent_mma_kernel(const LatentArgs a, const int piece, const FastDiv by_tile, const __grid_constant__ CUtensorMap lmap,
                  const __grid_constant__ CUtensorMap rmap,
                  const __grid_constant__ CUtensorMap qlmap,
                  const __grid_constant__ CUtensorMap qrmap) {
    extern __shared__ __align__(1024) unsigned char raw[];
    unsigned char* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const MmaLayout L(a.R);
    MmaShared& sh = *reinterpret_cast<MmaShared*>(sm + L.shared);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = blockIdx.x, w = blockIdx.y;
    const int pairs = a.R / 128;
    const int KT = kTile / piece * piece;  // keys of a tile
    const int row0 = g * a.rpg, nrows = min(a.rpg, a.rows - row0);
    const int N = (a.rpg + 15) / 16 * 16;  // rows of the MMA
    const uint32_t stage_bytes = L.chunks * kChunk;

    if (tid == 0) {
        for (int s = 0; s < L.stages; ++s) {
            for (int j = 0; j < pairs; ++j) {
                mbar_init(&sh.full[s][j], 1);
                mbar_init(&sh.empty[s][j], 1);
            }
        }
        mbar_init(&sh.s_full[0], 2);
        mbar_init(&sh.s_full[1], 2);
        mbar_init(&sh.s_free[0], kSoftmax / 32);
        mbar_init(&sh.s_free[1], kSoftmax / 32);
        mbar_init(&sh.p_full, kSoftmax / 32);
        mbar_init(&sh.pv_done, 1);
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_free, 1);
        mbar_init(&sh.drain[0], 1);
        mbar_init(&sh.drain[1], 1);
        sh.abort = 0;
        fence_barrier_init();
    }
    if (warp == 4) tmem_alloc(&sh.tmem, kTmemCols);
    if (warp >= kCopyWarp && lane == 0) {
        prefetch_tensormap(&lmap);
        prefetch_tensormap(&rmap);
    }
    pdl_launch_dependents();
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const uint32_t tmem_s = tmem + 256;  // two score tiles behind the output
    volatile int* abort_flag = &sh.abort;

    Walk walk;
    uint32_t refused = 0;
    const Found f = block_find_strided<kThreads>(
        a.Q, sh.scratch,
        [&](int tot) {
            walk.runs = Runs(tot, used_workers(a, tot));
            return w < walk.runs.W ? walk.runs.start(w) : tot;
        },
        [&](int b) {
            const SeqInfo s = latent_seq(a, b);
            refused |= s.bad;
            return a.lead + max(1, by_tile.up(s.n));
        });
    if (refused && g == 0 && w == 0) report(a.dev_status, refused);
    const bool some = f.item < a.Q;
    walk.b = f.item;
    walk.before = f.before;
    walk.t = some ? walk.runs.start(w) : 0;
    walk.t1 = some ? walk.runs.start(w + 1) : 0;
    if (walk.t1 <= walk.before + a.lead) walk.t = walk.t1;  // no tile of its first sequence
    const int t0 = walk.t;
    bool bad = false;

    if (warp == kQueryWarp) {
        // ------------------------------------------------------------ queries
        // N rows from the group's first on.  Where the group has fewer, the rest are
        // other rows or zeros: their scores and outputs are never read.
        const uint64_t policy = policy_evict_first();
        int seg = 0;
        while (walk.more() && !bad) {
            const Segment s = segment(a, walk, by_tile);
            const int row = uniform(walk.b * a.rows + row0);
            if (seg > 0 && !warp_wait(&sh.q_free, (seg - 1) & 1, abort_flag)) {
                bad = true;
                break;
            }
            if (elect_one()) {
                mbar_arrive_expect_tx(&sh.q_full, (uint32_t)(N * 128 * L.chunks));
                for (int c = 0; c < 2 * pairs; ++c)
                    tma_g2s_3d(sm + L.q + c * kChunk, &qlmap, 0, row, c, &sh.q_full, policy);
                tma_g2s_3d(sm + L.q + 2 * pairs * kChunk, &qrmap, 0, row, 0, &sh.q_full, policy);
            }
            __syncwarp();
            advance(a, walk, s);
            ++seg;
        }
        if (seg > 0) {  // nothing of its own may be in flight when it leaves
            const unsigned long long since = global_timer_ns();
            while (!mbar_try_wait(&sh.q_full, (seg - 1) & 1) &&
                   global_timer_ns() - since < kWaitLimitNs) {
            }
        }
    } else if (warp >= kCopyWarp) {
        // ------------------------------------------------------------ copies
        // Warp j brings pair j of the chunks (the rotary chunk goes with pair 0) as
        // the values MMAs free it: one wait, one count and one copy take a warp
        // about 500 cycles from end to end, and four pairs by one warp set the
        // pace of the whole kernel.  Lane p looks up piece p (and p + 32) of a tile
        // before the wait and issues its copies: a box is one chunk of a piece, or a
        // pair of chunks of a whole tile.
        const int j = warp - kCopyWarp;
        const uint64_t policy = policy_evict_first();
        const int pieces = kTile / piece;
        const uint32_t bytes = (uint32_t)piece * 128u, total = bytes * (j == 0 ? 3u : 2u);
        unsigned char* dst = sm + L.kv + 2 * j * kChunk;
        unsigned char* rdst = sm + L.kv + 2 * pairs * kChunk;
        int it = 0, st = 0, par = 1;
        if (j >= pairs) walk.t = walk.t1;
        while (walk.more() && !bad) {
            const Segment s = segment(a, walk, by_tile);
            for (int k = s.first; k < s.end; ++k, ++it) {
                unsigned long long valid = 0;
                int src[2];  // first row of this lane's pieces in the cache, or -1
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int p = lane + 32 * u;
                    const int key = k * KT + p * piece;
                    src[u] = -1;
                    if (p < pieces && key < s.seq.n) {
                        const int page = a.by_page(key);
                        const int phys = __ldg(a.block_tables + (size_t)walk.b * a.cols +
                                               s.seq.col0 + page);
                        if (phys < 0 || phys >= a.NB) {
                            report(a.dev_status, KVD_DEV_BLOCK_RANGE);
                        } else {
                            src[u] = phys * a.BS + key - page * a.BS;
                            const int n = min(piece, s.seq.n - key);
                            valid |= (n == 64 ? ~0ull : (1ull << n) - 1ull) << (p * piece);
                        }
                    }
                }
                const int loads = __popc(__ballot_sync(0xffffffffu, src[0] >= 0)) +
                                  __popc(__ballot_sync(0xffffffffu, src[1] >= 0));
                if (j == 0) {
                    if (pieces > 1) {
#pragma unroll
                        for (int d = 16; d; d >>= 1)
                            valid |= __shfl_xor_sync(0xffffffffu, valid, d);
                    }
                    if (lane == 0) sh.valid[it % kValid] = valid;
                    __syncwarp();
                }
                uint64_t* full = &sh.full[st][j];
                if (it >= L.stages) {
                    // the stage is still in use: meanwhile the tile comes to L2
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        if (src[u] < 0) continue;
                        tma_prefetch_3d(&lmap, 0, src[u], 2 * j);
                        if (piece != kTile) tma_prefetch_3d(&lmap, 0, src[u], 2 * j + 1);
                        if (j == 0) tma_prefetch_3d(&rmap, 0, src[u], 0);
                    }
                    __syncwarp();
                    if (!warp_wait(&sh.empty[st][j], par, abort_flag)) {
                        bad = true;
                        break;
                    }
                }
                if (pieces == 1) {
                    const int row = uniform(src[0]);
                    unsigned char* x = dst + st * stage_bytes;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(full, loads * total);
                        if (row >= 0) {
                            tma_g2s_3d(x, &lmap, 0, row, 2 * j, full, policy);
                            if (piece != kTile)
                                tma_g2s_3d(x + kChunk, &lmap, 0, row, 2 * j + 1, full, policy);
                            if (j == 0)
                                tma_g2s_3d(rdst + st * stage_bytes, &rmap, 0, row, 0, full, policy);
                        }
                    }
                } else {
                    if (lane == 0) mbar_arrive_expect_tx(full, loads * total);
                    __syncwarp();
                    const uint32_t at = st * stage_bytes + lane * bytes;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        if (src[u] < 0) continue;
                        unsigned char* x = dst + at + u * 32 * bytes;
                        tma_g2s_3d(x, &lmap, 0, src[u], 2 * j, full, policy);
                        tma_g2s_3d(x + kChunk, &lmap, 0, src[u], 2 * j + 1, full, policy);
                        if (j == 0)
                            tma_g2s_3d(rdst + at + u * 32 * bytes, &rmap, 0, src[u], 0, full, policy);
                    }
                }
                __syncwarp();
                if (++st == L.stages) {
                    st = 0;
                    par ^= 1;
                }
            }
            advance(a, walk, s);
        }
        if (bad) {  // a wait ran out: leave only when the copies in flight have landed
            if (lane == 0) sh.abort = 1;
            const unsigned long long since = global_timer_ns();
            for (int i = max(0, it - L.stages); i < it; ++i)
                while (!mbar_try_wait(&sh.full[i % L.stages][j],
                                      (i / L.stages) & 1) &&
                       global_timer_ns() - since < kWaitLimitNs) {
                }
        }
    } else if (warp == 4) {
        // ------------------------------------------------------------ scores
        // Everything that an issue loop branches on or addresses with goes through
        // uniform(): MMA operands live in uniform registers, and with operands (or
        // a control flow) that the compiler cannot prove to be the same in all
        // lanes an MMA took 50 to 140 cycles to issue instead of 32 to 48.  Scores
        // and values have a warp each, so that neither waits for the other's turn.
        const uint32_t desc = mma_desc(kTile, kTile);
        const uint32_t q = uniform(smem_u32(sm + L.q)), kv = uniform(smem_u32(sm + L.kv));
        const uint32_t tm = uniform(tmem) + 256;
        int it = 0, st = 0, par = 0, seg = 0;
        while (uniform((int)walk.more()) && !bad) {
            const Segment s = segment(a, walk, by_tile);
            const int tiles = uniform(s.end - s.first);
            bad = !warp_wait(&sh.q_full, seg & 1, abort_flag);
            for (int k = 0; k < tiles && !bad; ++k, ++it) {
                const uint32_t d = tm + 64 * (it & 1);
                if (it > 1) bad = !warp_wait(&sh.s_free[it & 1], ((it >> 1) - 1) & 1, abort_flag);
                // pair by pair, as they arrive
                const uint32_t q_low = uniform(desc_low(q, 16));
                const uint32_t k_low = uniform(desc_low(kv + st * stage_bytes, 16));
#pragma unroll
                for (int j = 0; j < kMaxPairs; ++j) {
                    if (j >= pairs || bad) break;
                    if (!warp_wait(&sh.full[st][j], par, abort_flag)) {
                        bad = true;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t off = ((2 * j + (i >> 2)) * kChunk + (i & 3) * 32) >> 4;
                            mma_ss(d, desc_of(q_low + off), desc_of(k_low + off), desc,
                                   i > 0 || j > 0);
                        }
                        if (j == 0) {
                            const uint32_t rope = (2 * pairs * kChunk) >> 4;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mma_ss(d, desc_of(q_low + rope + 2 * i),
                                       desc_of(k_low + rope + 2 * i), desc, true);
                            // the copying warps' writes (which this warp has waited
                            // for) are ordered before the softmax's reads by an
                            // arrival of its own
                            mbar_arrive(&sh.s_full[it & 1]);
                        }
                        if (j + 1 == pairs) {
                            mma_commit(&sh.s_full[it & 1]);
                            if (k + 1 == tiles) mma_commit(&sh.q_free);
                        }
                    }
                    __syncwarp();
                }
                if (++st == L.stages) {
                    st = 0;
                    par ^= 1;
                }
            }
            advance(a, walk, s);
            ++seg;
        }
        if (bad) drain(&sh.drain[0], &sh.abort);
    } else if (warp == 5) {
        // ------------------------------------------------------------ values
        const uint32_t desc = mma_desc(128, N, kAMn);
        const uint32_t kv = uniform(smem_u32(sm + L.kv)), tm = uniform(tmem);
        const uint32_t p_low = uniform(desc_low(smem_u32(sm + L.p), 16));
        int it = 0, st = 0;
        while (uniform((int)walk.more()) && !bad) {
            const Segment s = segment(a, walk, by_tile);
            const int tiles = uniform(s.end - s.first);
            for (int k = 0; k < tiles && !bad; ++k, ++it) {
                const uint32_t v_low = uniform(desc_low(kv + st * stage_bytes, kChunk));
                if (!warp_wait(&sh.p_full, it & 1, abort_flag)) {
                    bad = true;
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < kMaxPairs; ++j) {
                        if (j >= pairs) break;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_ss(tm + j * N, desc_of(v_low + ((2 * j * kChunk + i * 2048) >> 4)),
                                   desc_of(p_low + i * 2), desc, i > 0 || k > 0);
                        mma_commit(&sh.empty[st][j]);
                    }
                    mma_commit(&sh.pv_done);
                }
                __syncwarp();
                if (++st == L.stages) st = 0;
            }
            advance(a, walk, s);
        }
        if (bad) drain(&sh.drain[1], &sh.abort);
    } else {
        // ------------------------------------------------------------ softmax
        // A 64-row accumulator lies on lanes 0-15 of every warp's quarter, and four
        // threads share a row (16 keys of it each): thread i has rows i / 4 and
        // i / 4 + 8 of its warp's sixteen.
        const int quad = lane & 3;
        const uint32_t quarter = (uint32_t)(32 * warp) << 16;
        const int rows[2] = {16 * warp + (lane >> 2), 16 * warp + (lane >> 2) + 8};
        const bool busy = 16 * warp < nrows;  // the warp has rows at all
        // The largest score is the largest product where the scale is positive;
        // products change sign where it is negative.
        const bool flip = a.qscale < 0.f;
        const float qs = fmaxf(fabsf(a.qscale), kTinyScale);
        // where this lane's row of a group of four 8 x 8 weight tiles goes
        const int prow = 16 * warp + 8 * ((lane >> 3) & 1) + (lane & 7);
        const uint32_t p_row = smem_u32(sm + L.p) + prow * 128;
        const uint32_t p_group = lane >> 4, p_swizzle = lane & 7;
        int it = 0, st = 0;
        while (walk.more()) {
            const Segment s = segment(a, walk, by_tile);
            int last[2];  // newest key that the row sees
            float m[2], l[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                last[h] = rows[h] < nrows ? s.seq.n - a.T + a.by_head(row0 + rows[h])
                                         : 0x3fffffff;
                m[h] = -INFINITY;
                l[h] = 0.f;
            }
            // newest key that every row of the warp sees
            const int all_see = __reduce_min_sync(0xffffffffu, min(last[0], last[1]));
            for (int k = s.first; k < s.end; ++k, ++it) {
                if (!mbar_wait(&sh.s_full[it & 1], (it >> 1) & 1, abort_flag)) bad = true;
                __syncwarp();
                tc_fence_after();
                float x[32];
                float mn[2] = {m[0], m[1]};
                bool need = false;
                const unsigned long long valid = sh.valid[it % kValid];
                if (busy) {
                    tmem_ld16x64(tmem_s + 64 * (it & 1) + quarter, reinterpret_cast<uint32_t*>(x));
                    tmem_wait_ld();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.s_free[it & 1]);  // one arrival a warp
                if (busy) {
                    if (flip) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = -x[i];
                    }
                    if (valid != ~0ull || k * KT + 63 > all_see) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int lim = last[h] - k * KT;  // keys 0 .. lim of the tile
                            const unsigned long long z =
                                (valid & (lim >= 63 ? ~0ull
                                          : lim < 0 ? 0ull
                                                    : (2ull << lim) - 1ull)) >> (2 * quad);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (!((z >> (8 * (i >> 1) + (i & 1))) & 1ull))
                                    x[4 * (i >> 1) + 2 * h + (i & 1)] = -INFINITY;
                        }
                    }
                    float mx[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mx[h][i] = fmaxf(fmaxf(x[4 * i + 2 * h], x[4 * i + 2 * h + 1]),
                                             fmaxf(x[4 * i + 16 + 2 * h], x[4 * i + 17 + 2 * h]));
                        mn[h] = fmaxf(fmaxf(mx[h][0], mx[h][1]), fmaxf(mx[h][2], mx[h][3]));
                    }
#pragma unroll
                    for (int d = 1; d < 4; d <<= 1)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            mn[h] = fmaxf(mn[h], __shfl_xor_sync(0xffffffffu, mn[h], d));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        mn[h] = fmaxf(m[h], mn[h] * qs);
                        if (k == s.first) m[h] = mn[h];
                        need |= rows[h] < nrows && mn[h] > m[h] + kSkip;
                    }
                }
                bool waited = false;
                if (bar_any(1, kSoftmax, need || bad)) {
                    if (it > 0 && !mbar_wait(&sh.pv_done, (it - 1) & 1, abort_flag)) bad = true;
                    waited = true;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const bool up = mn[h] > m[h] + kSkip;
                        const float fac = up ? exp2f(m[h] - mn[h]) : 1.f;
                        if (up) m[h] = mn[h];
                        l[h] *= fac;
                        if (quad == 0) sh.factor[rows[h]] = fac;
                    }
                    __syncwarp();
                    if (bar_any(1, kSoftmax, bad)) {
                        bad = true;
                        break;
                    }
                    tc_fence_after();
                    for (int c = 0; c < pairs * N; c += 16) {
                        float o[16];
                        tmem_ld16(tmem + c + quarter, o);
                        tmem_wait_ld();
                        const float* fac = sh.factor + c % N;
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] *= fac[i];
                        tmem_st16(tmem + c + quarter, o);
                    }
                    tmem_wait_st();
                }
                // Weights are rounded to bf16, what the matrix unit takes with bf16 values (each
                // is off by 2^-8 of itself at most); their sum keeps fp32.
                uint32_t p[2][8];
                if (busy) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float base = m[h] == -INFINITY ? 0.f : m[h];
                        float sum[2] = {0.f, 0.f};
#pragma unroll
                        for (int g8 = 0; g8 < 8; ++g8) {
                            const float e0 = fast_exp2(fmaf(x[4 * g8 + 2 * h], qs, -base));
                            const float e1 = fast_exp2(fmaf(x[4 * g8 + 2 * h + 1], qs, -base));
                            sum[g8 & 1] += e0 + e1;
                            p[h][g8] = pack_bf16(e0, e1);
                        }
                        l[h] += sum[0] + sum[1];
                    }
                }
                if (!waited && it > 0 && !mbar_wait(&sh.pv_done, (it - 1) & 1, abort_flag))
                    bad = true;
                __syncwarp();
                if (busy) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        stsm_x4(p_row + (((2 * i + p_group) ^ p_swizzle) << 4), p[0][2 * i],
                                p[1][2 * i], p[0][2 * i + 1], p[1][2 * i + 1]);
                }
                if (valid != ~0ull) {
                    // rows that hold no token of the sequence: a weight of zero does
                    // not keep what they contain (NaN) out of the sum
                    unsigned char* v = sm + L.kv + st * stage_bytes;
                    for (int i = tid; i < 2 * pairs * kTile * 8; i += kSoftmax) {
                        const int r = (i >> 3) & 63;
                        if (!((valid >> r) & 1ull))
                            *reinterpret_cast<uint4*>(v + (i >> 9) * kChunk + r * 128 +
                                                      ((i & 7) << 4)) = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_full);
                if (++st == L.stages) st = 0;
            }
            __syncwarp();
            if (bar_any(1, kSoftmax, bad)) {
                bad = true;
                break;
            }
            const int b = walk.b;
            const bool head = walk.t == t0;
            const int before = walk.before;
            advance(a, walk, s);
            const bool whole = s.first == 0 && s.end == s.nt;
            const size_t slot = ((size_t)w * a.groups + g) * 2 + (head ? 0 : 1);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
                // a scale of NaN (the weights above do without it): every query that sees a key
                if (a.qscale != a.qscale && l[h] != 0.f) l[h] = a.qscale;
                if (quad == 0) sh.factor[rows[h]] = l[h] == 0.f ? 0.f : 1.f / l[h];
                if (quad == 0 && rows[h] < nrows) {
                    const float z = l[h] > 0.f ? m[h] + log2f(l[h]) : (l[h] == 0.f ? -INFINITY : NAN);
                    if (!whole)
                        a.part_lse[slot * a.rpg + rows[h]] = z;
                    else if (a.lse_out)
                        a.lse_out[(size_t)b * a.rows + row0 + rows[h]] = z * kLn2;
                }
            }
            if (g == 0 && tid == 0 && s.first == 0)
                a.meta[b] = make_int4(w, walk.runs.worker_of(before + a.lead + s.nt - 1),
                                      head ? 0 : 1, 0);
            if (it > 0 && !mbar_wait(&sh.pv_done, (it - 1) & 1, abort_flag)) bad = true;
            __syncwarp();
            if (bar_any(1, kSoftmax, bad)) {
                bad = true;
                break;
            }
            tc_fence_after();
            // 32 lanes are 32 consecutive dims: every store is a whole 64- or
            // 128-byte line part
            const int d = 32 * warp + lane;
            if (whole) {
                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) +
                                   ((size_t)b * a.rows + row0) * a.R + d;
                store_rows(tmem + quarter, pairs, N, nrows, sh.factor, a.R, [&](size_t at, float y) {
                    o[at] = __float2bfloat16_rn(y);
                });
            } else {
                float* o = a.part_o + slot * a.rpg * a.R + d;
                store_rows(tmem + quarter, pairs, N, nrows, sh.factor, a.R,
                           [&](size_t at, float y) { o[at] = y; });
            }
            tc_fence_before();
        }
        if (bad) sh.abort = 1;
    }
    __syncthreads();
    if (tid == 0 && sh.abort) report(a.dev_status, KVD_DEV_TIMEOUT);
    if (warp == 4) tmem_free(tmem, kTmemCols);
}

}  // namespace

// Keys of a copy box: the largest divisor of the page size not above a tile.
static int latent_piece(int BS) {
    int t = BS < kTile ? BS : kTile;
    while (BS % t) --t;
    return t;
}

cudaError_t launch_latent_mma(const LatentArgs& a, cudaStream_t stream) {
    const int piece = latent_piece(a.BS), N = (a.rpg + 15) / 16 * 16;
    const long long rows = (long long)a.NB * a.BS, qrows = (long long)a.Q * a.rows;
    CUtensorMap lmap, rmap, qlmap, qrmap;
    cudaError_t e = encode_rows(&lmap, a.latent, a.R, a.R, rows, piece, piece == kTile ? 2 : 1);
    if (e == cudaSuccess) e = encode_rows(&rmap, a.rope, a.P, a.P, rows, piece, 1);
    if (e == cudaSuccess) e = encode_rows(&qlmap, a.q_latent, a.R, a.R, qrows, N, 1);
    if (e == cudaSuccess) e = encode_rows(&qrmap, a.q_rope, a.P, a.P, qrows, N, 1);
    if (e != cudaSuccess) return e;
    const MmaLayout L(a.R);
    e = cudaFuncSetAttribute(latent_mma_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             L.total);
    if (e != cudaSuccess) return e;
    return launch_pdl(latent_mma_kernel, dim3(a.groups, a.workers), dim3(kThreads), L.total, stream,
                      a, piece, FastDiv(kTile / piece * piece), lmap, rmap, qlmap, qrmap);
}

}  // namespace kvd
