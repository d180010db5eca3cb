// latent_common.cuh -- what the latent-cache kernels share: the arguments of a
// call, the sequence checks, and the division of ragged sequences over a grid.
//
// Division of kvd_attend_latent.  The host knows the sizes but not the
// lengths, so every CTA derives its share on the device: the key tiles of all
// sequences form one line, cut into W equal runs, and worker w takes the tiles
// [w * tot / W, (w + 1) * tot / W), whichever sequences they belong to.  Only
// the first and the last sequence of a run can be shared with other workers,
// so a worker leaves at most two partial results (slots 2w and 2w + 1) and
// every other sequence of its run goes straight to the output.  A grid of one
// CTA per SM is then balanced to one tile, whatever the lengths are.  A sequence
// counts `lead` tiles more than it has, laid before its first one: what a run
// spends on starting and finishing it.
#pragma once

#include "../kvd_device.cuh"

namespace kvd {

constexpr int kLatentSMs = 152;  // SMs of a GB300: the workers of one call

// Division of n < 2^31 by a number that the host knows, 1 <= d < 2^31 (Granlund and
// Montgomery: a product's upper half, an addition and a shift).
struct FastDiv {
    uint32_t mul, shift;
    FastDiv() = default;
    explicit FastDiv(uint32_t d) {
        shift = 0;
        while ((1u << shift) < d) ++shift;
        mul = (uint32_t)((((1ull << shift) - d) << 32) / d + 1);
    }
    __device__ __forceinline__ int operator()(int n) const {
        return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift);
    }
    // n / d rounded up, for n >= 0
    __device__ __forceinline__ int up(int n) const { return n > 0 ? (*this)(n - 1) + 1 : 0; }
};

struct LatentArgs {
    const void* q_latent;   // [Q, T, H, R]
    const void* q_rope;     // [Q, T, H, P]
    const void* latent;     // [NB, BS, R]
    const void* rope;       // [NB, BS, P]
    const int32_t* block_tables;
    const int32_t* seq_lens;
    const int32_t* seq_offset;
    void* out;              // [Q, T, H, R]
    float* lse_out;         // [Q, T, H] or null
    int32_t* dev_status;
    int Q, T, H, NB, BS, cols, R, P;
    float qscale;           // scale * log2(e)
    int rows;               // T * H query rows of a sequence
    int groups, rpg;        // row groups of a sequence, rows per group
    int workers;            // W at most (the grid's x extent)
    int min_shift;          // 2^min_shift tiles are the fewest worth a worker of its own
    int lead;               // tiles that a sequence counts above its own
    FastDiv by_page, by_head;  // by BS, by H
    int4* meta;             // [Q] first worker, last worker, first slot's parity
    float* part_lse;        // [workers * groups * 2, rpg], log2 units
    float* part_o;          // [workers * groups * 2, rpg, R], normalised
};

// What the bf16 kernels take for a scale of zero, so that a masked score of -inf stays
// one: the smallest number, which makes any finite product less than 2^-21.
constexpr float kTinyScale = 1.4e-45f;

// A sequence's keys: count (0 if the sequence is refused), first table column.
struct SeqInfo {
    int n;
    int col0;
    uint32_t bad;
};

__device__ __forceinline__ SeqInfo latent_seq(const LatentArgs& a, int b) {
    SeqInfo s{0, 0, 0u};
    const int s0 = a.seq_lens[b], s1 = a.seq_lens[b + 1];
    const int off = a.seq_offset ? a.seq_offset[b] : 0;
    if ((b == 0 && s0 != 0) || s0 < 0 || s1 < s0) s.bad |= KVD_DEV_SEQLENS;
    const int col0 = off > 0 ? a.by_page(off) : 0;
    if (off < 0 || off != col0 * a.BS) s.bad |= KVD_DEV_SEQ_OFFSET;
    if (s.bad) return s;
    const int n = s1 - s0;
    if ((uint32_t)col0 + (uint32_t)a.by_page.up(n) > (uint32_t)a.cols) {
        s.bad |= KVD_DEV_TABLE_COLS;
        return s;
    }
    s.n = n;
    s.col0 = col0;
    return s;
}

// Finds the item of `target` in a line of items with
// count(b) places each (b < Q): item, the places before it, and the total.
// Every thread gets the result; item = Q if target is behind the line.  Up to
// kFindWarp items each warp finds it by itself (no barrier), above with the whole
// block, a thread's sum of counts ending at kMost.  `scratch`: kFindWords ints of shared
// memory.
constexpr int kFindWords = 40;
constexpr int kFindWarp = 128;
struct Found {
    int item;
    int before;
    int total;
};

template <int THREADS, int kMost = 0x7fffffff, typename Total, typename Count>
__device__ __forceinline__ Found block_find(int Q, int* scratch, Total target_of, Count count) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (Q <= kFindWarp) {
        constexpr int kPer = kFindWarp / 32;
        int c[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int b = lane * kPer + i;
            c[i] = b < Q ? count(b) : 0;
            sum += c[i];
        }
        int inc = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        const int total = __shfl_sync(0xffffffffu, inc, 31);
        const int target = target_of(total);
        int at = inc - sum, item = lane * kPer;
        const bool mine = target >= at && target < inc;
#pragma unroll
        for (int i = 0; i + 1 < kPer; ++i)
            if (mine && target >= at + c[i] && item == lane * kPer + i) {
                at += c[i];
                ++item;
            }
        const uint32_t who = __ballot_sync(0xffffffffu, mine);
        const int src = who ? __ffs(who) - 1 : 0;
        item = __shfl_sync(0xffffffffu, item, src);
        at = __shfl_sync(0xffffffffu, at, src);
        return Found{who ? item : Q, at, total};
    }
    const int per = (Q + THREADS - 1) / THREADS;
    const int lo = min(tid * per, Q), hi = min(lo + per, Q);
    int sum = 0;
    for (int b = lo; b < hi; ++b) sum = min(sum + count(b), kMost);
    int inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 31) scratch[warp] = inc;
    if (tid == 0) scratch[32] = Q;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        const int s = scratch[i];
        if (i < warp) before += s;
        total += s;
    }
    before += inc - sum;
    const int target = target_of(total);
    if (target >= before && target < before + sum) {
        int b = lo, at = before;
        while (b < hi) {
            const int c = count(b);
            if (target < at + c) break;
            at += c;
            ++b;
        }
        scratch[32] = b;
        scratch[33] = at;
    }
    __syncthreads();
    Found f{scratch[32], scratch[33], total};
    __syncthreads();
    return f;
}

// The same with item 32 i + lane as the lane's i-th, so that all counts cost one
// memory latency.  (kvd_attend_latent: 64 sequences 66.0 -> 63.8 us with the cheaper
// divisions, 8 sequences 15.8 -> 13.9.  kvd_attend_expanded, whose softmax has no
// registers left, lost 1 % to it.)
template <int THREADS, typename Total, typename Count>
__device__ __forceinline__ Found block_find_strided(int Q, int* scratch, Total target_of,
                                                    Count count) {
    if (Q > kFindWarp) return block_find<THREADS>(Q, scratch, target_of, count);
    const int lane = threadIdx.x & 31;
    constexpr int kPer = kFindWarp / 32;
    int c[kPer], inc[kPer], total = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) c[i] = 32 * i + lane < Q ? count(32 * i + lane) : 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        inc[i] = c[i];
        if (32 * i >= Q) continue;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc[i], d);
            if (lane >= d) inc[i] += o;
        }
        inc[i] += total;
        total = __shfl_sync(0xffffffffu, inc[i], 31);
    }
    const int target = target_of(total);
    int item = Q, at = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (32 * i >= Q) continue;
        const uint32_t who =
            __ballot_sync(0xffffffffu, target >= inc[i] - c[i] && target < inc[i]);
        if (who) {
            const int src = __ffs(who) - 1;
            item = 32 * i + src;
            at = __shfl_sync(0xffffffffu, inc[i] - c[i], src);
        }
    }
    return Found{item, at, total};
}

// `tot` tiles over W workers: worker w's run is [start(w), start(w + 1)), and the
// inverse.  start(w) = floor(w * tot / W) in 32 bits.
struct Runs {
    int tot, W, per, rest;
    Runs() = default;
    __device__ __forceinline__ Runs(int tot_, int W_) : tot(tot_), W(W_) {
        per = (uint32_t)tot / (uint32_t)W;
        rest = tot - per * W;
    }
    __device__ __forceinline__ int start(int w) const {
        return w * per + (int)((uint32_t)(w * rest) / (uint32_t)W);
    }
    __device__ __forceinline__ int worker_of(int tile) const {
        return (int)((((long long)tile + 1) * W - 1) / tot);
    }
};
// A worker per 2^min_shift places of the line (the `lead` ones, which hold no tile,
// counted), but kFewWorkers at least, or one a place where there are fewer: while there
// are few the merge of their partial rows is cheaper than a second tile (bf16: 1000
// tokens 11.8 us instead of 12.7 with 18 workers instead of 9, but 4000 tokens 16.1
// instead of 15.0 with 66 instead of 33).
constexpr int kFewWorkers = 32;
__device__ __forceinline__ int used_workers(const LatentArgs& a, int tot) {
    return max(1, min(a.workers,
                      max(((tot - 1) >> a.min_shift) + 1, min(tot, kFewWorkers))));
}

// Tensor map over `rows` bf16 rows of `stride` elements, of which the first
// `width` (a multiple of 64) are mapped: (64, rows, width / 64).  A box is
// box_chunks blocks of box_rows consecutive rows x 64 elements (128 bytes, under
// the 128-byte swizzle), one block behind the other.
cudaError_t encode_rows(CUtensorMap* map, const void* base, long long width, long long stride,
                        long long rows, int box_rows, int box_chunks);

// Merges the partial rows of sequences that several workers share.
cudaError_t launch_latent_combine(const LatentArgs& a, kvd_dtype dt, cudaStream_t stream);
cudaError_t launch_latent_mma(const LatentArgs& a, cudaStream_t stream);
cudaError_t launch_latent_simt(const LatentArgs& a, cudaStream_t stream);

struct ExpandedArgs {
    const void* q;       // [Nq, H, Dn + P]
    const void* kv;      // [Nk, H, Dn + Dv]
    const void* k_rope;  // [Nk, P]
    const int32_t* q_lens;
    const int32_t* k_lens;
    void* out;           // [Nq, H, Dv]
    float* lse_out;      // [Nq, H] or null
    int32_t* dev_status;
    int Q, Nq, Nk, H, Dn, Dv, P;
    float qscale;        // scale * log2(e)
    int causal;
    int span_log;        // log2 of the queries that a CTA of the bf16 kernel takes
};

// Queries and keys of one sequence.  A bad pair of q_lens leaves no queries, a
// bad pair of k_lens no keys.  falls: q_lens decreases here.
struct PackedSeq {
    int q0, nq, k0, nk;
    uint32_t bad;
    bool falls;
};

__device__ __forceinline__ PackedSeq packed_seq(const ExpandedArgs& a, int b) {
    PackedSeq s{0, 0, 0, 0, 0u, false};
    const int q0 = a.q_lens[b], q1 = a.q_lens[b + 1], k0 = a.k_lens[b], k1 = a.k_lens[b + 1];
    s.falls = q1 < q0;
    if ((b == 0 && q0 != 0) || q0 < 0 || s.falls || q1 > a.Nq) {
        s.bad = KVD_DEV_SEQLENS;
    } else {
        s.q0 = q0;
        s.nq = q1 - q0;
    }
    if ((b == 0 && k0 != 0) || k0 < 0 || k1 < k0 || k1 > a.Nk) {
        s.bad = KVD_DEV_SEQLENS;
    } else {
        s.k0 = k0;
        s.nk = k1 - k0;
    }
    return s;
}

// The sequence of a CTA's unit in the line of all units of 2^span_log queries, by the
// whole block.  The grid has units for Nq queries, one sequence each; a q_lens that
// decreases would give queries to several.  A pair that does takes more units than any
// grid has (2^23 queries in 16s and 2^14 sequences), so that nothing behind it is found,
// and has no queries itself: a sequence found may have none.  (A second search for such
// lengths, or a vote on them, cost good calls 1 %.)  `tell`: the CTA that reports.
template <int THREADS>
__device__ __forceinline__ Found packed_find(const ExpandedArgs& a, int* scratch, int unit,
                                             int span_log, bool tell) {
    constexpr int kBehindAll = 1 << 20;
    return block_find<THREADS, 2 * kBehindAll>(
        a.Q, scratch, [&](int) { return unit; },
        [&](int b) {
            const PackedSeq s = packed_seq(a, b);
            if (s.bad && tell) report(a.dev_status, s.bad);
            return s.falls ? kBehindAll : (s.nq + (1 << span_log) - 1) >> span_log;
        });
}

cudaError_t launch_expanded_mma(const ExpandedArgs& a, cudaStream_t stream);
cudaError_t launch_expanded_simt(const ExpandedArgs& a, cudaStream_t stream);

cudaError_t launch_append_latent(void* latent, void* rope, const void* latent_new,
                                 const void* rope_new, const int32_t* block_tables,
                                 const int32_t* seq_offset, const int32_t* new_lens,
                                 const int32_t* pos, int Q, int N, int NB, int BS, int cols,
                                 int latent_bytes, int rope_bytes, int32_t* dev_status,
                                 cudaStream_t stream);
cudaError_t launch_verify_drafts(const void* target, const void* draft, const int32_t* drafts,
                                 const float* u_accept, const float* u_sample,
                                 const int32_t* num_drafts, int32_t* tokens, int32_t* accepted,
                                 int Q, int T, int V, kvd_dtype dt, int32_t* dev_status,
                                 cudaStream_t stream);

}  // namespace kvd
