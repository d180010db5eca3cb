// serving_common.cuh -- what the serving-step kernels share: arguments, the
// division of shared prefixes over a grid, launchers.
//
// Division of kvd_attend_paged_prefix.  A segment is one tile of query rows of
// one kv head of one group (row = sequence of the group x query head of the kv
// head) with all key tiles of the group's prefix.  The host knows sizes, not
// lengths, so every CTA lays all segments' key tiles in one line on the device
// (a segment counts `lead` places more than it has, laid before its first tile:
// what starting and finishing it costs) and takes an equal run of it.  A segment
// that a worker holds whole goes to a row array of its own; of those that it
// shares there are two at most, one that began before its run (slot 2w) and one
// that goes on behind it (slot 2w + 1).
#pragma once

#include "../kvd_device.cuh"

namespace kvd {

constexpr int kServingSMs = 152;

struct PrefixArgs {
    const void* q;        // [Q, Hq, D]
    const void* k;        // [NB, BS, Hkv, D]
    const void* v;
    const int32_t* prefix_tables;  // [G, pcols]
    const int32_t* prefix_lens;    // [G]
    const int32_t* group_lens;     // [G + 1]
    void* out;            // [Q, Hq, D]
    float* lse_out;       // [Q, Hq] or null
    int32_t* dev_status;
    int Q, G, Hq, Hkv, g, NB, BS, pcols, D;
    float qscale;         // scale * log2(e)
    int rows, keys;       // of a tile
    int lead, workers;
    // SM microseconds that a place of the line costs, and a token of a sequence's own, and
    // the units of the attention over those: how many SMs the prefixes take while the
    // sequences' own keys go through the others (0: as many as there are)
    float place_cost, token_cost;
    int own_units;
    const int32_t* seq_lens;
    int4* meta;           // [Q + 1] first place, row tiles, key tiles, place in the group;
                          // last the line's length and the workers that share it
    float* part_lse;      // [2 * workers, rows] log2 units
    float* part_o;        // [2 * workers, rows, D], normalised
    float* whole_lse;     // [Q * Hq]
    float* whole_o;       // [Q * Hq, D]
    // the sequences' own keys: partial rows of the paged attention (natural log)
    const float* own_lse; // [Q * Hq, S]
    const float* own_o;   // [Q * Hq, S, D]
    int S;
    uint32_t* counters;   // of that attention: zero before it starts
};

constexpr int kMaxGroups = 1024;

// Groups of a call, in shared memory.
struct PrefixGroups {
    int start[kMaxGroups + 1];  // first sequence
    int base[kMaxGroups + 1];   // first place of the line
    int keys[kMaxGroups];       // of the prefix
    __device__ __forceinline__ int sequences(int i) const { return start[i + 1] - start[i]; }
};

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// The largest i < n with x[i] <= v (x ascending, x[0] <= v).
__device__ __forceinline__ int last_not_above(const int* x, int n, int v) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (x[mid] <= v)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// The line over W workers: worker w takes [start(w), start(w + 1)), start(w) = floor(w tot / W),
// in 32 bits (W is a few hundred, tot below 2^30).
struct PrefixRuns {
    int tot, W, per, rest;
    __device__ __forceinline__ PrefixRuns(int tot_, int W_) : tot(tot_), W(W_) {
        per = tot / W;
        rest = tot - per * W;
    }
    __device__ __forceinline__ int start(int w) const { return w * per + w * rest / W; }
    __device__ __forceinline__ int worker_of(int place) const {
        int w = min(W - 1, (int)((float)place * (float)W / (float)tot));  // or one beside it
        while (w > 0 && start(w) > place) --w;
        while (w + 1 < W && start(w + 1) <= place) ++w;
        return w;
    }
};

// The SMs that the prefixes take of a call's workers; every warp of every CTA gets the same.
// Two ways, by their estimated ends:
//  - Such a share that the other SMs are through the own tokens by the time the prefixes
//    end, so that nothing starts late.  A CTA's start and end take 8 us, a place 1.75, up to
//    place_cost as own tokens fill the memory's queues; an own unit's chain takes 9, each
//    further one of a CTA 1.5.
//  - Where own tokens are most of the work: SMs by the shares of the work, and the own units
//    that are left when the prefixes end over all SMs, a chain later.
// (The second way and an SM for two own units at most 76: 64 sequences behind 16384 tokens
// with up to 16 own ones 48.3 us, now 39.7; 64 in 4 groups behind 1024 to 4096 34.7, 31.0; 8
// behind 4096 22.0, 20.5; one behind 8192 24.3, 21.8; 64 to 1024 own ones the same.)
__device__ __forceinline__ int prefix_workers(const PrefixArgs& a, int tot, int own) {
    constexpr float kStart = 8.f, kChain = 9.f, kUnit = 1.5f, kPlace = 1.75f;
    const int lane = threadIdx.x & 31, most = min(a.workers, max(tot, 1));
    const float theirs = a.token_cost * (float)own, places = (float)max(tot, 1);
    const float place =
        kPlace + (a.place_cost - kPlace) * fminf(__fdividef(theirs, kPlace * places), 1.f);
    const int w = max(1, min(most, a.workers - 4 * lane));
    const float others = __fdividef(1.f, fmaxf((float)(a.workers - w), 0.5f));  // one over them
    const float prefix_end = kStart + place * ceilf(__fdividef(places, (float)w) - 0.01f);
    const float rounds = 0.5f * (float)a.own_units * others;  // two CTAs an SM
    const bool late = a.own_units <= 2 * kServingSMs && rounds > 1.f;  // a CTA a unit, not dealt
    const float own_end = kChain + (late ? prefix_end : kUnit * fmaxf(rounds - 1.f, 0.f)) + theirs * others;
    // the earliest end, in 2^-6 us, and of equal ones the smallest share
    const uint32_t end = (uint32_t)(fminf(fmaxf(prefix_end, own_end), 1e6f) * 64.f);
    const uint32_t best = __reduce_min_sync(0xffffffffu, end << 5 | (31 - lane));
    const float mine = a.place_cost * places, all = __fdividef(mine + theirs, (float)a.workers);
    if ((float)(best >> 5) <= 64.f * (kStart + all + kChain))
        return max(1, min(most, a.workers - 4 * (31 - (int)(best & 31u))));
    const int share = max(1, min(most, (int)(__fdividef(mine, all) + 0.5f)));
    return share > 1 && share < most ? share & ~1 : share;
}

// By all threads of a CTA: reads and checks the groups, lays out the line; returns its
// division.  The attention over the sequences' own keys, which is launched behind, runs
// beside this kernel: it may start from here on, when everything before both is complete
// and its counters are zero.
template <int THREADS>
__device__ __forceinline__ PrefixRuns prefix_setup(const PrefixArgs& a, PrefixGroups& t) {
    const int tid = threadIdx.x;
    if (blockIdx.x == 0) {
        if (tid < 2) {
            a.counters[tid] = 0;
            __threadfence();
        }
        __syncthreads();
    }
    pdl_launch_dependents();
    uint32_t bits = 0;
    bool bad = false;
    const int own = a.place_cost > 0.f ? a.seq_lens[a.Q] : 0;
    for (int i = tid; i <= a.G; i += THREADS) {
        const int s0 = a.G > 0 ? a.group_lens[i] : 0;
        t.start[i] = s0;
        if (i == 0 && s0 != 0) bad = true;
        if (i == a.G) continue;
        const int s1 = a.group_lens[i + 1];
        bad |= s0 < 0 || s1 < s0 || s1 > a.Q;
        int n = a.prefix_lens[i];
        if (n < 0) {
            bits |= KVD_DEV_SEQLENS;
            n = 0;
        } else if (n > 0 && (n - 1) / a.BS >= a.pcols) {
            bits |= KVD_DEV_TABLE_COLS;
            n = 0;
        }
        t.keys[i] = n;
    }
    if (bad) bits |= KVD_DEV_SEQLENS;
    if (bits && blockIdx.x == 0) report(a.dev_status, bits);
    bad = __syncthreads_or(bad);
    if (tid < 32) {
        int at = 0;
        for (int i0 = 0; i0 < a.G; i0 += 32) {
            const int i = i0 + tid;
            int c = 0;
            if (i < a.G && !bad) {
                const int kt = ceil_div(t.keys[i], a.keys);
                c = kt > 0 ? a.Hkv * ceil_div(t.sequences(i) * a.g, a.rows) * (kt + a.lead) : 0;
            }
            int inc = c;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, inc, d);
                if (tid >= d) inc += o;
            }
            if (i < a.G) t.base[i] = at + inc - c;
            at += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (tid == 0) t.base[a.G] = at;
    }
    __syncthreads();
    const int tot = t.base[a.G];
    return PrefixRuns(tot, own > 0 ? prefix_workers(a, tot, own) : min(a.workers, max(tot, 1)));
}

// The CTA's share of the meta rows, by `threads` of its threads (without groups t.base[G] is
// 0, and a bad group_lens leaves no places).
__device__ __forceinline__ void prefix_meta(const PrefixArgs& a, const PrefixGroups& t,
                                            const PrefixRuns& runs, int thread, int threads) {
    for (int q = blockIdx.x * threads + thread; q <= a.Q; q += gridDim.x * threads) {
        int4 m = make_int4(0, 0, 0, 0);
        if (q == a.Q) {
            m.x = runs.tot;
            m.y = runs.W;
        } else if (runs.tot > 0 && q < t.start[a.G]) {
            const int i = last_not_above(t.start, a.G, q);
            m = make_int4(t.base[i], ceil_div(t.sequences(i) * a.g, a.rows),
                          ceil_div(t.keys[i], a.keys), q - t.start[i]);
        }
        a.meta[q] = m;
    }
}

// The piece of a segment that a run holds.
struct PrefixPiece {
    int group, head, tile;  // tile: of the group's query rows
    int k0, k1;             // key tiles
    int slot;               // -1: the whole segment
    int next;               // the place behind it
};

// The piece at place p of the run [lo, hi) (p >= lo).
__device__ __forceinline__ PrefixPiece prefix_piece(const PrefixArgs& a, const PrefixGroups& t,
                                                    int w, int lo, int hi, int p) {
    PrefixPiece s;
    // the last group that starts at or before p: empty ones have no places
    s.group = last_not_above(t.base, a.G, p);
    const int kt = ceil_div(t.keys[s.group], a.keys), span = kt + a.lead;
    const int tiles = ceil_div(t.sequences(s.group) * a.g, a.rows);
    const int seg = (p - t.base[s.group]) / span, first = t.base[s.group] + seg * span;
    s.head = seg / tiles;
    s.tile = seg - s.head * tiles;
    s.k0 = max(0, lo - first - a.lead);
    s.k1 = min(kt, hi - first - a.lead);
    s.next = first + span;
    const int tile0 = first + a.lead;
    s.slot = s.k0 == 0 && s.k1 == kt ? -1 : 2 * w + (tile0 >= lo ? 1 : 0);
    return s;
}

// Rows of a copy box: the largest divisor of the page size not above a tile of 128 keys.
inline int prefix_piece_rows(int BS) {
    int t = BS < 128 ? BS : 128;
    while (BS % t) --t;
    return t;
}

cudaError_t launch_prefix_mma(const PrefixArgs& a, cudaStream_t stream);   // bf16
cudaError_t launch_prefix_simt(const PrefixArgs& a, cudaStream_t stream);  // fp32
cudaError_t launch_prefix_combine(const PrefixArgs& a, kvd_dtype dt, cudaStream_t stream);

struct PlanArgs {
    int32_t *block_tables, *pages_held, *free_pages, *free_count;
    const int32_t *kept_lens, *new_lens, *pos_base;
    int32_t *seq_lens, *slots, *positions;
    int32_t* dev_status;
    int Q, N, BS, cols, F;
};
cudaError_t launch_plan_pages(const PlanArgs& a, cudaStream_t stream);

struct RotateArgs {
    const void* x;            // [N, Hq + 2 Hkv, D]
    const void* q_weight;     // [D] or null
    const void* k_weight;
    const double* freqs;      // [Dr / 2]
    const int32_t* positions; // [N]
    const int32_t* slots;     // [N]
    void* q_out;              // [N, Hq, D]
    void* key_cache;
    void* value_cache;
    int32_t* dev_status;
    int N, Hq, Hkv, D, Dr;
    long long rows;           // NB * BS
    float stretch, eps;
};
cudaError_t launch_rotate(const RotateArgs& a, bool interleaved, kvd_dtype dt, cudaStream_t stream);

struct SampleArgs {
    const void* logits;       // [R, V]
    const float* temperature; // [R] or null
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    const float* u;           // [R], tokens only
    int32_t* tokens;          // [R], or null: probabilities
    void* probs;              // [R, V]
    int32_t* dev_status;
    int R, V;
    bool probs_bf16;
};
cudaError_t launch_sample(const SampleArgs& a, kvd_dtype dt, cudaStream_t stream);

}  // namespace kvd
