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
// Warps 0-3: softmax (a row a thread, so no shuffles), rescaling, epilogue.
// Warp 4: tensor copies of the pages.  Warp 5: MMA issue; the scores of tile
// i + 1 are issued before the values of tile i, so they run during softmax i.
// The running output is rescaled only when some row's maximum rose by more
// than 8 (log2 units), as in the decode kernel: weights stay below 2^8.
#include "kvd_internal.h"
#include "latent_common.cuh"
#include "tcgen05_ptx.cuh"

namespace kvd {
namespace {

constexpr int kSoftmax = 128;            // threads of warps 0-3
constexpr int kThreads = kSoftmax + 64;
constexpr int kTile = 64;                // keys of an MMA tile, rows of the query tile
constexpr int kChunk = kTile * 128;      // bytes of 64 rows x 64 bf16
constexpr int kMaxStages = 4;
constexpr int kMaxPairs = 4;             // R / 128
constexpr uint32_t kTmemCols = 512;
constexpr float kSkip = 8.f;             // log2 units

struct MmaShared {
    uint64_t full[kMaxStages][kMaxPairs];
    uint64_t empty[kMaxStages];
    uint64_t s_full[2];
    uint64_t p_full, pv_done, q_full, drain;
    unsigned long long valid[kMaxStages];
    float factor[kTile];
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
    int tot, W;
    __device__ bool more() const { return t < t1; }
};

struct Segment {
    SeqInfo seq;
    int nt;     // tiles of the whole sequence
    int first;  // first tile of this worker
    int end;
};

__device__ __forceinline__ Segment segment(const LatentArgs& a, const Walk& k, int KT) {
    Segment s;
    s.seq = latent_seq(a, k.b);
    s.nt = max(1, (s.seq.n + KT - 1) / KT);
    s.first = k.t - k.before;
    s.end = min(s.nt, k.t1 - k.before);
    return s;
}
__device__ __forceinline__ void advance(Walk& k, const Segment& s) {
    k.t = k.before + s.end;
    k.before += s.nt;
    ++k.b;
}

__global__ void __launch_bounds__(kThreads, 1)
latent_mma_kernel(const LatentArgs a, const int piece, const __grid_constant__ CUtensorMap lmap,
                  const __grid_constant__ CUtensorMap rmap) {
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

    if (tid == 0) {
        for (int s = 0; s < L.stages; ++s) {
            for (int j = 0; j < pairs; ++j) mbar_init(&sh.full[s][j], 1);
            mbar_init(&sh.empty[s], 1);
        }
        mbar_init(&sh.s_full[0], 1);
        mbar_init(&sh.s_full[1], 1);
        mbar_init(&sh.p_full, kSoftmax);
        mbar_init(&sh.pv_done, 1);
        mbar_init(&sh.q_full, kSoftmax);
        mbar_init(&sh.drain, 1);
        sh.abort = 0;
        fence_barrier_init();
    }
    if (warp == 4) tmem_alloc(&sh.tmem, kTmemCols);
    if (warp == 5 && lane == 0) {
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
    walk.W = 1;
    const Found f = block_find<kThreads>(
        a.Q, sh.scratch,
        [&](int tot) {
            walk.W = used_workers(a, tot);
            return w < walk.W ? run_start(w, tot, walk.W) : tot;
        },
        [&](int b) {
            const SeqInfo s = latent_seq(a, b);
            if (s.bad && g == 0 && w == 0) report(a.dev_status, s.bad);
            return max(1, (s.n + KT - 1) / KT);
        });
    const bool some = f.item < a.Q;
    walk.b = f.item;
    walk.before = f.before;
    walk.tot = f.total;
    walk.t = some ? run_start(w, f.total, walk.W) : 0;
    walk.t1 = some ? run_start(w + 1, f.total, walk.W) : 0;
    const int t0 = walk.t;
    bool bad = false;

    if (warp == 4) {
        // ------------------------------------------------------------ copies
        const uint64_t policy = policy_evict_first();
        const int pieces = kTile / piece;
        const uint32_t bytes = (uint32_t)piece * 128u;
        int it = 0;
        while (walk.more() && !bad) {
            const Segment s = segment(a, walk, KT);
            for (int k = s.first; k < s.end; ++k, ++it) {
                const int st = it % L.stages, use = it / L.stages;
                if (use > 0 && !mbar_wait(&sh.empty[st], (use - 1) & 1, abort_flag)) bad = true;
                if (__any_sync(0xffffffffu, bad)) {
                    bad = true;
                    break;
                }
                unsigned long long valid = 0;
                int src[2];  // first row of this lane's pieces in the cache, or -1
                int loads = 0;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int p = lane + 32 * u;
                    const int key = k * KT + p * piece;
                    src[u] = -1;
                    if (p < pieces && key < s.seq.n) {
                        const int phys = __ldg(a.block_tables + (size_t)walk.b * a.cols +
                                               s.seq.col0 + key / a.BS);
                        if (phys < 0 || phys >= a.NB) {
                            report(a.dev_status, KVD_DEV_BLOCK_RANGE);
                        } else {
                            src[u] = phys * a.BS + key % a.BS;
                            const int n = min(piece, s.seq.n - key);
                            valid |= (n == 64 ? ~0ull : (1ull << n) - 1ull) << (p * piece);
                        }
                    }
                    loads += __popc(__ballot_sync(0xffffffffu, src[u] >= 0));
                }
#pragma unroll
                for (int d = 16; d; d >>= 1) valid |= __shfl_xor_sync(0xffffffffu, valid, d);
                if (lane == 0) {
                    sh.valid[st] = valid;
                    for (int j = 0; j < pairs; ++j)
                        mbar_arrive_expect_tx(&sh.full[st][j],
                                              (uint32_t)loads * bytes * (j == 0 ? 3u : 2u));
                }
                __syncwarp();
                unsigned char* base = sm + L.kv + st * L.chunks * kChunk;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (src[u] < 0) continue;
                    unsigned char* dst = base + (lane + 32 * u) * bytes;
                    for (int c = 0; c < 2 * pairs; ++c) {
                        tma_g2s_2d(dst + c * kChunk, &lmap, 64 * c, src[u], &sh.full[st][c >> 1],
                                   policy);
                        if (c == 1)
                            tma_g2s_2d(dst + 2 * pairs * kChunk, &rmap, 0, src[u],
                                       &sh.full[st][0], policy);
                    }
                }
            }
            advance(walk, s);
        }
        if (bad) {  // a wait ran out: leave only when the copies in flight have landed
            if (lane == 0) sh.abort = 1;
            for (int i = max(0, it - L.stages); i < it; ++i)
                for (int j = 0; j < pairs; ++j) {
                    const unsigned long long since = global_timer_ns();
                    while (!mbar_try_wait(&sh.full[i % L.stages][j], (i / L.stages) & 1) &&
                           global_timer_ns() - since < kWaitLimitNs) {
                    }
                }
        }
    } else if (warp == 5) {
        // ------------------------------------------------------------ MMA issue
        if (lane == 0) {
            const uint32_t sdesc = mma_desc(64, 64), odesc = mma_desc(128, N, kAMn);
            const uint32_t q = smem_u32(sm + L.q), kv = smem_u32(sm + L.kv), p = smem_u32(sm + L.p);
            // scores of tile `it`, the first of its segment if `fresh`
            auto scores = [&](int it, int seg, bool fresh) {
                const int st = it % L.stages;
                if (fresh && !mbar_wait(&sh.q_full, seg & 1, abort_flag)) return false;
                const uint32_t k = kv + st * L.chunks * kChunk, d = tmem_s + 64 * (it & 1);
                for (int j = 0; j < pairs; ++j) {
                    if (!mbar_wait(&sh.full[st][j], (it / L.stages) & 1, abort_flag)) return false;
                    tc_fence_after();
#pragma unroll
                    for (int i = 0; i < 12; ++i) {
                        if (j > 0 && i >= 8) break;
                        const int c = i < 8 ? 2 * j + (i >> 2) : 2 * pairs;
                        const uint32_t off = c * kChunk + (i & 3) * 32;
                        mma_ss(d, smem_desc(q + off, 16), smem_desc(k + off, 16), sdesc,
                               j > 0 || i > 0);
                    }
                }
                mma_commit(&sh.s_full[it & 1]);
                return true;
            };
            int it = 0, seg = 0;
            Segment s = walk.more() ? segment(a, walk, KT) : Segment{};
            if (walk.more()) bad = !scores(0, 0, true);
            while (walk.more() && !bad) {
                for (int k = s.first; k < s.end && !bad; ++k, ++it) {
                    // the next tile's scores first; the first of the next segment
                    // only behind this segment's last values, since they wait for
                    // other queries
                    if (k + 1 < s.end) bad = !scores(it + 1, seg, false);
                    if (bad || !mbar_wait(&sh.p_full, it & 1, abort_flag)) {
                        bad = true;
                        break;
                    }
                    tc_fence_after();
                    const int st = it % L.stages;
                    const uint32_t v = kv + st * L.chunks * kChunk;
                    for (int j = 0; j < pairs; ++j) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_ss(tmem + j * N, smem_desc(v + 2 * j * kChunk + i * 2048, kChunk),
                                   smem_desc(p + i * 32, 16), odesc, k > s.first || i > 0);
                    }
                    mma_commit(&sh.empty[st]);
                    mma_commit(&sh.pv_done);
                }
                if (bad) break;
                advance(walk, s);
                ++seg;
                if (walk.more()) {
                    s = segment(a, walk, KT);
                    bad = !scores(it, seg, true);
                }
            }
            if (bad) {
                sh.abort = 1;
                mma_commit(&sh.drain);
                const unsigned long long since = global_timer_ns();
                while (!mbar_try_wait(&sh.drain, 0) && global_timer_ns() - since < kWaitLimitNs) {
                }
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        // A 64-row accumulator lies on lanes 0-15 of every warp's quarter.
        const int row = 16 * warp + (lane & 15);
        const bool live = lane < 16 && row < nrows;
        const uint32_t quarter = (uint32_t)(32 * warp) << 16;
        const __nv_bfloat16* ql = static_cast<const __nv_bfloat16*>(a.q_latent);
        const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(a.q_rope);
        // Query rows of sequence b into the swizzled tile.  Rows at and behind
        // nrows are not written: their scores and outputs are never read.
        auto load_q = [&](int b) {
            const int vecs = L.chunks * 8;
            for (int i = tid; i < nrows * vecs; i += kSoftmax) {
                const int r = i / vecs, v = i % vecs, c = v >> 3, j = v & 7;
                const size_t at = (size_t)b * a.rows + row0 + r;
                const uint4 x = __ldg(reinterpret_cast<const uint4*>(
                    c < 2 * pairs ? ql + at * a.R + 8 * v : qr + at * 64 + 8 * j));
                *reinterpret_cast<uint4*>(sm + L.q + c * kChunk + r * 128 + ((j ^ (r & 7)) << 4)) = x;
            }
            fence_async_smem();
            mbar_arrive(&sh.q_full);
        };
        int it = 0;
        if (walk.more()) load_q(walk.b);
        while (walk.more()) {
            const Segment s = segment(a, walk, KT);
            // newest key that the row sees
            const int last = live ? s.seq.n - a.T + (row0 + row) / a.H : -1;
            float m = -INFINITY, l = 0.f;
            for (int k = s.first; k < s.end; ++k, ++it) {
                const int st = it % L.stages;
                const uint32_t par = (it / L.stages) & 1;
                if (!mbar_wait(&sh.full[st][0], par, abort_flag)) bad = true;
                if (!mbar_wait(&sh.s_full[it & 1], (it >> 1) & 1, abort_flag)) bad = true;
                __syncwarp();
                tc_fence_after();
                float x[kTile];
                tmem_ld32(tmem_s + 64 * (it & 1) + quarter, reinterpret_cast<uint32_t*>(x));
                tmem_ld32(tmem_s + 64 * (it & 1) + 32 + quarter,
                          reinterpret_cast<uint32_t*>(x + 32));
                tmem_wait_ld();
                const unsigned long long valid = sh.valid[st];
                const int lim = last - k * KT;  // keys 0 .. lim of the tile
                const unsigned long long sees =
                    valid & (lim >= 63 ? ~0ull : lim < 0 ? 0ull : (2ull << lim) - 1ull);
                float mt = -INFINITY;
                if (__all_sync(0xffffffffu, sees == ~0ull || !live)) {
#pragma unroll
                    for (int i = 0; i < kTile; ++i) {
                        x[i] *= a.qscale;
                        mt = fmaxf(mt, x[i]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kTile; ++i) {
                        x[i] = (sees >> i) & 1ull ? x[i] * a.qscale : -INFINITY;
                        mt = fmaxf(mt, x[i]);
                    }
                }
                const float mn = fmaxf(m, mt);
                const bool need = live && k > s.first && mn > m + kSkip;
                if (k == s.first) m = mn;
                bool waited = false;
                if (bar_any(1, kSoftmax, need || bad)) {
                    if (it > 0 && !mbar_wait(&sh.pv_done, (it - 1) & 1, abort_flag)) bad = true;
                    waited = true;
                    const float fac = need ? exp2f(m - mn) : 1.f;
                    if (need) m = mn;
                    l *= fac;
                    if (lane < 16) sh.factor[row] = fac;
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
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] *= sh.factor[c % N + i];
                        tmem_st16(tmem + c + quarter, o);
                    }
                    tmem_wait_st();
                }
                const float base = m == -INFINITY ? 0.f : m;
                uint32_t p[kTile / 2];
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < kTile; i += 2) {
                    const float e0 = fast_exp2(x[i] - base), e1 = fast_exp2(x[i + 1] - base);
                    sum += e0 + e1;
                    p[i / 2] = pack_bf16(e0, e1);
                }
                l += sum;
                if (!waited && it > 0 && !mbar_wait(&sh.pv_done, (it - 1) & 1, abort_flag))
                    bad = true;
                if (live) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        *reinterpret_cast<uint4*>(sm + L.p + row * 128 + ((j ^ (row & 7)) << 4)) =
                            make_uint4(p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]);
                }
                if (valid != ~0ull) {
                    // rows that hold no token of the sequence: a weight of zero does
                    // not keep what they contain (NaN) out of the sum
                    for (int j = 1; j < pairs; ++j)
                        if (!mbar_wait(&sh.full[st][j], par, abort_flag)) bad = true;
                    unsigned char* v = sm + L.kv + st * L.chunks * kChunk;
                    for (int i = tid; i < 2 * pairs * kTile * 8; i += kSoftmax) {
                        const int r = (i >> 3) & 63;
                        if (!((valid >> r) & 1ull))
                            *reinterpret_cast<uint4*>(v + (i >> 9) * kChunk + r * 128 +
                                                      ((i & 7) << 4)) = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_async_smem();
                tc_fence_before();
                mbar_arrive(&sh.p_full);
            }
            __syncwarp();
            if (bar_any(1, kSoftmax, bad)) {
                bad = true;
                break;
            }
            // the segment's score MMAs are complete: the next segment's queries may
            // replace its own
            const int b = walk.b;
            const bool head = walk.t == t0;
            const int before = walk.before;
            advance(walk, s);
            if (walk.more()) load_q(walk.b);
            if (it > 0 && !mbar_wait(&sh.pv_done, (it - 1) & 1, abort_flag)) bad = true;
            __syncwarp();
            if (bar_any(1, kSoftmax, bad)) {
                bad = true;
                break;
            }
            tc_fence_after();
            const bool whole = s.first == 0 && s.end == s.nt;
            const size_t slot = ((size_t)w * a.groups + g) * 2 + (head ? 0 : 1);
            if (lane < 16) sh.factor[row] = l == 0.f ? 0.f : 1.f / l;
            if (live) {
                const float z = l > 0.f ? m + log2f(l) : (l == 0.f ? -INFINITY : NAN);
                if (!whole)
                    a.part_lse[slot * a.rpg + row] = z;
                else if (a.lse_out)
                    a.lse_out[(size_t)b * a.rows + row0 + row] = z * kLn2;
            }
            if (g == 0 && tid == 0 && s.first == 0)
                a.meta[b] = make_int4(w, worker_of(before + s.nt - 1, walk.tot, walk.W),
                                      head ? 0 : 1, 0);
            bar_sync(1, kSoftmax);
            for (int j = 0; j < pairs; ++j) {
                const int d = 128 * j + 32 * warp + lane;
                for (int c = 0; c < nrows; c += 16) {
                    float o[16];
                    tmem_ld16(tmem + j * N + c + quarter, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (c + i >= nrows) continue;
                        const float y = o[i] * sh.factor[c + i];
                        if (whole)
                            static_cast<__nv_bfloat16*>(
                                a.out)[((size_t)b * a.rows + row0 + c + i) * a.R + d] =
                                __float2bfloat16_rn(y);
                        else
                            a.part_o[(slot * a.rpg + c + i) * a.R + d] = y;
                    }
                }
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
int latent_piece(int BS) {
    int t = BS < kTile ? BS : kTile;
    while (BS % t) --t;
    return t;
}

cudaError_t launch_latent_mma(const LatentArgs& a, const CUtensorMap& lmap, const CUtensorMap& rmap,
                              cudaStream_t stream) {
    const MmaLayout L(a.R);
    const cudaError_t e = cudaFuncSetAttribute(
        latent_mma_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L.total);
    if (e != cudaSuccess) return e;
    return launch_pdl(latent_mma_kernel, dim3(a.groups, a.workers), dim3(kThreads), L.total, stream,
                      a, latent_piece(a.BS), lmap, rmap);
}

}  // namespace kvd
