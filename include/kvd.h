/*
 * kvd.h -- C ABI of libkvd: decode-phase KV-cache attention on GB300 (sm_103a).
 *
 * One new query token per head attends over a KV cache of fixed capacity,
 * kept either as a static buffer with a 0/1 mask or as a paged cache
 * addressed through block tables.  Sources (page title, section):
 *
 *  [NPU]    "Intel NPU running LLMs" (OpenVINO community article 882):
 *           Part 1 "解决方案：预分配 + Attention Mask" -- static buffer of
 *           capacity MAX_PROMPT_LEN + MIN_RESPONSE_LEN (default 1024 + 128 =
 *           1152) with a 0/1 mask the length of the buffer, mask = 0 slots
 *           set to -inf before the softmax; Part 2 "NPUW 的核心设计" --
 *           update_kvcache_for writes only the new token's row at the next
 *           empty slot and bumps num_stored_tokens; Part 3 "Attention 在 NPU
 *           上的完整实现" -- decode is one query against N keys (incremental
 *           SDPA), tiles along the sequence merged exactly through a running
 *           output, max and sum (Flash SDPA path); Part 5 "当前限制" -- more
 *           tokens than the capacity is an error.
 *  [FlashMLA] "FlashMLA на Huawei Ascend: ядро разреженного внимания
 *           изнутри", "Математическая постановка" -- out = softmax(Q K^T *
 *           sm_scale) V per query token; "Ход вычислений" -- fp32 running
 *           max / sum / output and a log-sum-exp per row.
 *  [FlashMLA-KV] the same page, "Ограничение по деквантованию" -- decoding
 *           reads the KV cache in FP8, dequantises it to bf16 and feeds the
 *           matrix unit; "Оптимизация раскладки KV-кэша при decoding" -- a
 *           token's quantised values and its scale are stored side by side.
 *  [PyPTO]  "PyPTO 实现 AscendC GatherPaKvCache（Norm/ND 分支）" sections
 *           3.1-3.3 -- key_cache [num_blocks, block_size, heads, dim],
 *           int32 block_tables [Q, cols], cumsum seq_lens [Q+1] starting at
 *           0, optional seq_offset [Q] (multiple of block_size, selects the
 *           first table column), logical_block = t / block_size, slot =
 *           t % block_size, output row seq_lens[q] + t; section 7 -- only the
 *           cumsum form of seq_lens and int32 indices.
 *
 * Conventions for every entry point:
 *  - Tensors are caller-owned device memory, contiguous, row-major, in the
 *    layouts given per call.  The library never allocates, frees, copies to
 *    the host or synchronises; every call is asynchronous on `stream`.
 *  - Pointers to element data must be 16-byte aligned; byte masks and int32
 *    index arrays need only their natural alignment.
 *  - The return value reports errors the host can see (arguments, sizes,
 *    launch failures).  Errors that depend on device-resident data set bits
 *    in the optional caller-owned `dev_status` word (atomic OR, never cleared
 *    by the library); the offending element is skipped, never written out of
 *    bounds.  Nothing traps or aborts.
 *  - Every wait inside a kernel is bounded (about one second); a wait that
 *    runs out sets KVD_DEV_TIMEOUT and the kernel returns.
 *  - The caches are plain inputs/outputs of the calls: the caller owns them,
 *    starts a conversation by zeroing them and appends through kvd_append.
 */
#ifndef KVD_H
#define KVD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st* kvd_stream_t;

typedef enum {
    KVD_OK = 0,
    KVD_ERR_INVALID_ARG = 1,  /* null/misaligned pointer, bad size, bad combination */
    KVD_ERR_UNSUPPORTED = 2,  /* valid but not implemented (head_dim, dtype, group) */
    KVD_ERR_WORKSPACE = 3,    /* workspace missing or smaller than required */
    KVD_ERR_CUDA = 4          /* a CUDA runtime/driver call failed (see kvd_last_error) */
} kvd_status;

typedef enum { KVD_BF16 = 0, KVD_F32 = 1 } kvd_dtype;

/* Bits OR-ed into *dev_status by the kernels. */
#define KVD_DEV_POS_RANGE 1u     /* append position outside [0, capacity) */
#define KVD_DEV_BLOCK_RANGE 2u   /* block table entry outside [0, num_blocks) */
#define KVD_DEV_TABLE_COLS 4u    /* seq_offset/BS + ceil(len/BS) > table columns */
#define KVD_DEV_SEQLENS 8u       /* seq_lens not starting at 0, decreasing, or past total */
#define KVD_DEV_SEQ_OFFSET 16u   /* seq_offset negative or not a multiple of block_size */
#define KVD_DEV_TIMEOUT 32u      /* a bounded in-kernel wait ran out */
#define KVD_DEV_POINTER 64u      /* a pointer read from a device pointer array is null or misaligned */
#define KVD_DEV_TOKEN_RANGE 128u /* drafted token outside [0, V) */
#define KVD_DEV_PROBS 256u       /* no finite positive weight to sample a token from */
#define KVD_DEV_NO_PAGES 512u    /* the free list has too few pages, or no room for those given back */
#define KVD_DEV_PARAM 1024u      /* a row's sampling parameter is NaN or out of range */

/*
 * kvd_append -- [NPU] Part 2, update_kvcache_for: for every batch entry b
 * and kv head h, row pos[b] of k_cache[b, h] and v_cache[b, h] becomes
 * k_new[b, h] and v_new[b, h]; if `mask` is given, mask[b, pos[b]] = 1.
 *   k_cache, v_cache  [B, Hkv, C, D] of `dtype`          (in/out)
 *   k_new, v_new      [B, Hkv, D] of `dtype`             (in)
 *   pos               [B] int32, device                  (in)
 *   mask              [B, C] uint8 or NULL               (in/out)
 * A byte copy.  pos[b] outside [0, C) writes nothing for b and sets
 * KVD_DEV_POS_RANGE ([NPU] Part 5: over capacity is an error).
 * Errors: INVALID_ARG for null pointers, sizes < 1, D*elem not a multiple of
 * 16 bytes, misaligned data pointers.
 */
kvd_status kvd_append(void* k_cache, void* v_cache, const void* k_new, const void* v_new,
                      const int32_t* pos, uint8_t* mask, int B, int Hkv, int C, int D,
                      kvd_dtype dtype, int32_t* dev_status, kvd_stream_t stream);

/*
 * kvd_copy_prefix -- copy_kvcache, the prefill -> generate hand-over ([NPU]
 * Part 2 "NPUW 的核心设计", step 3: the prefill model's present K/V are copied
 * as the slice [0:N] into the generate model's past K/V, capacities 1024 and
 * 1152, all 32 layers x K and V at once).  For every layer l, batch entry b
 * and kv head h, rows [0, n[b]) of k_src[l][b, h] and v_src[l][b, h] become
 * the same rows of k_dst[l][b, h] and v_dst[l][b, h]; rows >= n[b] of the
 * destination are left alone.  If `masks` is given, masks[l][b, t] becomes
 * (t < n[b]) for every t < C_dst.
 *   k_src, v_src  device arrays of L pointers to [B, Hkv, C_src, D] of `dtype`
 *   k_dst, v_dst  device arrays of L pointers to [B, Hkv, C_dst, D]
 *   masks         device array of L pointers to [B, C_dst] uint8, or NULL
 *   n             [B] int32, device
 * One launch for all layers; a byte copy.  n[b] outside [0, min(C_src,
 * C_dst)] copies nothing for b (and leaves its masks) and sets
 * KVD_DEV_POS_RANGE; a null or non-16-byte-aligned pointer in an array skips
 * that layer and sets KVD_DEV_POINTER.
 * Errors: INVALID_ARG for null arrays, sizes < 1, D*elem not a multiple of 16
 * bytes, misaligned arrays; UNSUPPORTED for B*Hkv or L above 65535 / 32767.
 */
kvd_status kvd_copy_prefix(const void* const* k_src, const void* const* v_src, void* const* k_dst,
                           void* const* v_dst, uint8_t* const* masks, const int32_t* n, int L,
                           int B, int Hkv, int C_src, int C_dst, int D, kvd_dtype dtype,
                           int32_t* dev_status, kvd_stream_t stream);

/*
 * kvd_attend_masked -- decode attention over the static buffer ([NPU] Part 1
 * and Part 3; [FlashMLA] "Математическая постановка"):
 *   out[b, h, :] = sum_t w_t v[b, h/g, t, :] / sum_t w_t,
 *   w_t = exp(scale * q[b, h, :] . k[b, h/g, t, :] - max), over t with
 *   mask[b, t] != 0, g = Hq / Hkv (query head h reads kv head h / g).
 *   lse[b, h] = log sum_t exp(scale * q.k_t) (natural log).
 *   q         [B, Hq, D] of `dtype`
 *   k_cache   [B, Hkv, C, D], v_cache [B, Hkv, C, D] of `dtype`
 *   mask      [B, C] uint8, nonzero = valid; any content in mask = 0 slots
 *             (inf, NaN) is ignored; all-zero mask tiles are not read
 *   out       [B, Hq, D] of `dtype` (fp32 result rounded to nearest even)
 *   lse_out   [B, Hq] float or NULL
 * A row with no valid slot gives out = 0 and lse = -inf.
 * The sequence axis of every (batch entry, kv head) row is cut into splits
 * that a persistent grid takes from a work counter; each split keeps an fp32
 * running max / sum / output.  num_splits > 0 asks for about that many equal
 * splits (lengths rounded up to the kernel's tile, at most 4096 slots); 0
 * lets the library plan from the sizes, with smaller splits over the end of
 * the capacity.  With more than one split a second kernel merges the splits by
 * log-sum-exp (the kvd_combine formula).  Short buffers with num_splits = 0
 * (at most 8 splits of at most 384 slots per row, every split of every row
 * resident at once on the GPU) take one launch instead: a thread-block
 * cluster per row whose CTAs hold one split each and merge the row through
 * distributed shared memory (kvd_attend_masked_launches tells which).
 * Workspace: at least kvd_attend_masked_workspace_bytes(...) bytes (never
 * less than 256), 256-byte aligned, holding the work counters and the
 * partial rows.  Zero-fill it once before its first use; every call leaves
 * its counters at zero again, so calls ordered on one stream can reuse it
 * (calls that may overlap on the GPU must not share one).  After a call that
 * reported KVD_DEV_TIMEOUT, zero it again.
 * Supported: D in {64, 128}; dtype bf16 or f32; any Hq multiple of Hkv.
 */
size_t kvd_attend_masked_workspace_bytes(int B, int Hq, int Hkv, int C, int D, kvd_dtype dtype,
                                         int num_splits);
/* Kernel launches one kvd_attend_masked (or kvd_append_attend_masked with
 * Hq / Hkv <= 8) call makes for these sizes: 1 or 2; 0 for invalid sizes. */
int kvd_attend_masked_launches(int B, int Hq, int Hkv, int C, int D, kvd_dtype dtype,
                               int num_splits);
kvd_status kvd_attend_masked(const void* q, const void* k_cache, const void* v_cache,
                             const uint8_t* mask, void* out, float* lse_out, int B, int Hq,
                             int Hkv, int C, int D, float scale, kvd_dtype dtype, int num_splits,
                             void* workspace, size_t workspace_bytes, int32_t* dev_status,
                             kvd_stream_t stream);

/*
 * How a split attention call runs for given sizes (the *_plan queries), for a
 * caller that reads the workspace's partial rows or times the launches apart:
 *   splits            S of the split kernel: 1 = its units write the output
 *                     rows directly; > 1 = partial rows merged by log-sum-exp;
 *                     0 = the one-launch cluster kernel (no partial rows)
 *   launches          kernel launches of one call (1, or 2 when the combine
 *                     launch merges the splits)
 *   lse_offset, o_offset  with S > 1, the workspace byte offsets of part_lse
 *                     float [rows*Hq, S] and part_o float [rows*Hq, S, D] (the
 *                     kvd_combine layout); 0 otherwise
 *   counter_bytes     leading workspace bytes holding work counters (zero
 *                     before a call; every completed call leaves them zero)
 */
typedef struct {
    int32_t splits;
    int32_t launches;
    size_t lse_offset;
    size_t o_offset;
    size_t counter_bytes;
} kvd_plan;

/* kvd_attend_masked_plan -- kvd_plan of kvd_attend_masked (and of
 * kvd_append_attend_masked, kvd_attend_masked_partial) for these sizes.
 * Arguments and errors as for kvd_attend_masked. */
kvd_status kvd_attend_masked_plan(int B, int Hq, int Hkv, int C, int D, kvd_dtype dtype,
                                  int num_splits, kvd_plan* plan);

/*
 * kvd_attend_masked_partial -- the same attention as kvd_attend_masked, but
 * the output rows stay in fp32 whatever `dtype` is: out [B, Hq, D] float,
 * lse_out [B, Hq] float (required).  This is the partial result of one range
 * of a sequence's tokens ([NPU] Part 3, Flash SDPA path: each tile's output
 * is normalised over its own keys and carried with its max and sum), which
 * kvd_combine or kvd_combine_gathered merges exactly with the other
 * ranges' partials -- e.g. when the sequence axis of one long sequence is
 * spread over several GPUs, each holding a slice [B, Hkv, C_r, D] of the
 * cache and the matching slice [B, C_r] of the mask.  A range with no valid
 * slot gives out = 0 and lse = -inf (weight 0 in the merge).  Workspace,
 * splits and errors as for kvd_attend_masked.
 */
kvd_status kvd_attend_masked_partial(const void* q, const void* k_cache, const void* v_cache,
                                     const uint8_t* mask, float* out, float* lse_out, int B,
                                     int Hq, int Hkv, int C, int D, float scale, kvd_dtype dtype,
                                     int num_splits, void* workspace, size_t workspace_bytes,
                                     int32_t* dev_status, kvd_stream_t stream);

/*
 * kvd_attend_paged -- decode attention over the paged cache: for sequence q
 * the keys/values are the rows kvd_gather_paged would produce for q
 * ([PyPTO] 3.2), all valid, and q_in[q, h] attends over them with kv head
 * h / (Hq / Hkv).  The block-table indirection is resolved in the kernel.
 *   q_in         [Q, Hq, D] of `dtype`
 *   key_cache    [NB, BS, Hkv, D], value_cache [NB, BS, Hkv, D] of `dtype`
 *   block_tables [Q, cols] int32
 *   seq_lens     [Q + 1] int32, cumsum starting at 0
 *   seq_offset   [Q] int32 or NULL (zeros); first table column = seq_offset[q] / BS
 *   out          [Q, Hq, D] of `dtype`;  lse_out [Q, Hq] float or NULL
 * Device-detected errors (KVD_DEV_SEQLENS, SEQ_OFFSET, TABLE_COLS) make the
 * sequence empty (out = 0, lse = -inf); an out-of-range block id
 * (KVD_DEV_BLOCK_RANGE) drops that block's tokens.  A sequence of length 0
 * gives out = 0, lse = -inf.  One launch and a workspace as for
 * kvd_attend_masked (zero-filled before first use, left zeroed by each call).
 * Supported: D in {64, 128}; bf16 or f32; BS*Hkv*D*elem addressable by a
 * TMA tensor map (NB*BS < 2^31).
 */
/*
 * kvd_append_attend_masked -- one decode step over the static buffer: the
 * result of kvd_append(k_cache, v_cache, k_new, v_new, pos, mask) followed by
 * kvd_attend_masked(q, k_cache, v_cache, mask, ...) ([NPU] Part 2,
 * update_kvcache_for, then Part 3), with the append done inside the
 * attention launch when every kv head has a single group of query heads
 * (Hq / Hkv <= 8): the split holding pos[b] writes the new rows of its kv
 * head and kv head 0's split sets mask[b, pos[b]], before that split's tiles
 * are read.  Larger groups run the append kernel first.  Arguments as for
 * the two calls (k_new, v_new [B, Hkv, D] of `dtype`, pos [B] int32, mask
 * written); the caches, the mask and the output end exactly as after the two
 * calls.  pos[b] outside [0, C) writes nothing for b and sets
 * KVD_DEV_POS_RANGE; the attention then runs over the mask as it is.
 * Workspace: kvd_attend_masked_workspace_bytes.
 */
kvd_status kvd_append_attend_masked(const void* q, void* k_cache, void* v_cache, uint8_t* mask,
                                    const void* k_new, const void* v_new, const int32_t* pos,
                                    void* out, float* lse_out, int B, int Hq, int Hkv, int C,
                                    int D, float scale, kvd_dtype dtype, int num_splits,
                                    void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                    kvd_stream_t stream);

/*
 * kvd_attend_window -- sliding-window decode attention over the static
 * buffer ([NPU] Part 3, the sliding-window tile variant; Part 1 for the
 * mask): row b attends to the slots j with mask[b, j] != 0 and
 *   last[b] - W + 1 <= j <= last[b],
 * i.e. kvd_attend_masked with every mask slot outside the window taken as 0.
 *   q [B, Hq, D]; k_cache, v_cache [B, Hkv, C, D]; mask [B, C] uint8;
 *   last [B] int32, device (the window's newest slot, normally the slot the
 *   step appended); W >= 1 window slots; out, lse_out, scale, dtype,
 *   workspace, num_splits and dev_status as for kvd_attend_masked.
 * The splits are laid over each row's window only (from the 64-slot boundary
 * at or below last[b] - W + 1), so no slot outside it is scanned or read,
 * whatever C is.  last[b] outside [0, C): row b is empty (out = 0,
 * lse = -inf) and KVD_DEV_POS_RANGE is set.  Always the persistent split
 * kernel (the one-launch cluster kernel holds whole buffers); 1 or 2
 * launches (kvd_attend_window_plan).  Errors as for kvd_attend_masked, and
 * KVD_ERR_INVALID_ARG for W < 1 or a null `last`.
 */
size_t kvd_attend_window_workspace_bytes(int B, int Hq, int Hkv, int C, int D, int W,
                                         kvd_dtype dtype, int num_splits);
/* As kvd_attend_masked_plan, for kvd_attend_window and
 * kvd_append_attend_window (splits >= 1: never the one-launch kernel). */
kvd_status kvd_attend_window_plan(int B, int Hq, int Hkv, int C, int D, int W, kvd_dtype dtype,
                                  int num_splits, kvd_plan* plan);
kvd_status kvd_attend_window(const void* q, const void* k_cache, const void* v_cache,
                             const uint8_t* mask, const int32_t* last, void* out, float* lse_out,
                             int B, int Hq, int Hkv, int C, int D, int W, float scale,
                             kvd_dtype dtype, int num_splits, void* workspace,
                             size_t workspace_bytes, int32_t* dev_status, kvd_stream_t stream);
/*
 * kvd_append_attend_window -- one sliding-window decode step: the result of
 * kvd_append(k_cache, v_cache, k_new, v_new, pos, mask) followed by
 * kvd_attend_window(..., last = pos, W, ...), the append done inside the
 * attention launch as in kvd_append_attend_masked (Hq / Hkv <= 8; larger
 * groups run the append kernel first).  pos[b] outside [0, C): nothing is
 * written for b, row b is empty, KVD_DEV_POS_RANGE is set.  Workspace:
 * kvd_attend_window_workspace_bytes.
 */
kvd_status kvd_append_attend_window(const void* q, void* k_cache, void* v_cache, uint8_t* mask,
                                    const void* k_new, const void* v_new, const int32_t* pos,
                                    void* out, float* lse_out, int B, int Hq, int Hkv, int C,
                                    int D, int W, float scale, kvd_dtype dtype, int num_splits,
                                    void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                    kvd_stream_t stream);

/*
 * kvd_attend_indexed -- decode attention over a list of cache slots per batch
 * entry ([FlashMLA] "Математическая постановка": the indexer's top-k indices
 * pick the KV rows, P = Q . gathered^T, S = softmax(P * sm_scale),
 * out = S . gathered):
 *   out[b, h, :] = sum_j w_j v[b, h/g, indices[b, j], :] / sum_j w_j,
 *   w_j = exp(scale * q[b, h, :] . k[b, h/g, indices[b, j], :] - max), over
 *   the entries j with 0 <= indices[b, j] < C.
 *   q [B, Hq, D]; k_cache, v_cache [B, Hkv, C, D]; indices [B, topk] int32,
 *   device (-1 = unused entry); out [B, Hq, D]; lse_out [B, Hq] float or NULL
 * Every entry is one term of the softmax (a repeated slot counts once per
 * entry; the list order does not matter).  An entry outside [-1, C) is
 * skipped and sets KVD_DEV_POS_RANGE.  No valid entry: out = 0, lse = -inf.
 * The list is cut into splits of at most 128 entries that the persistent grid
 * takes from its work counter; the listed rows are gathered into shared
 * memory with 16-byte cp.async copies.
 * Workspace, num_splits and dtypes as for kvd_attend_masked (the list length
 * topk takes the place of the capacity).
 */
size_t kvd_attend_indexed_workspace_bytes(int B, int Hq, int Hkv, int topk, int D,
                                          kvd_dtype dtype, int num_splits);
/* As kvd_attend_masked_plan, for kvd_attend_indexed (the one-launch cluster
 * kernel is never used: splits >= 1). */
kvd_status kvd_attend_indexed_plan(int B, int Hq, int Hkv, int topk, int D, kvd_dtype dtype,
                                   int num_splits, kvd_plan* plan);
kvd_status kvd_attend_indexed(const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* indices, void* out, float* lse_out, int B, int Hq,
                              int Hkv, int C, int topk, int D, float scale, kvd_dtype dtype,
                              int num_splits, void* workspace, size_t workspace_bytes,
                              int32_t* dev_status, kvd_stream_t stream);

/*
 * Quantised KV rows ([FlashMLA-KV]; the scale granularity and encoding are
 * this library's reading, the page gives neither): one row of a kv head is
 *   bytes [0, D)        OCP FP8 E4M3 codes (bias 7, max 448, no infinities)
 *   bytes [D, D + 4)    the row's scale, fp32 little-endian
 *   bytes [D + 4, D+16) zero
 * so a cache is uint8 [B, Hkv, C, D + KVD_FP8_ROW_PAD] and element d of a row
 * is scale * E4M3(code[d]).  kvd_append_fp8 writes such rows; the attention
 * reads them directly (no bf16 copy of the cache exists).
 */
#define KVD_FP8_ROW_PAD 16

/*
 * kvd_append_fp8 -- kvd_append ([NPU] Part 2, update_kvcache_for) into
 * quantised caches: for every kv head h the new rows k_new[b, h, :],
 * v_new[b, h, :] ([B, Hkv, D], new_dtype bf16 or fp32, finite) are quantised
 *   amax = max_d |x_d|, scale = amax / 448, code_d = E4M3(x_d / scale)
 * (both divisions fp32 round-to-nearest; codes rounded to nearest even and
 * saturated at 448; amax = 0 gives scale 0 and zero codes) and written as
 * row pos[b] of k_cache / v_cache [B, Hkv, C, D + 16] (uint8); mask[b, pos[b]]
 * becomes 1 if mask is not NULL.  D is 64 or 128.  pos[b] outside [0, C)
 * writes nothing for b and sets KVD_DEV_POS_RANGE.
 */
kvd_status kvd_append_fp8(void* k_cache, void* v_cache, const void* k_new, const void* v_new,
                          const int32_t* pos, uint8_t* mask, int B, int Hkv, int C, int D,
                          kvd_dtype new_dtype, int32_t* dev_status, kvd_stream_t stream);

/*
 * kvd_attend_masked_fp8 -- kvd_attend_masked over quantised caches: the same
 * definition with every K/V element dequantised (scale * E4M3(code)).
 *   q [B, Hq, D] bf16; k_cache, v_cache uint8 [B, Hkv, C, D + 16] (rows as
 *   above); mask [B, C]; out [B, Hq, D] bf16; lse_out [B, Hq] float or NULL.
 * The tensor-core kernel never builds a dequantised copy: K codes meet q in
 * fp16 (q is converted to fp16, so |q| must stay below 65504) and each row's
 * scale multiplies its score; V codes meet the softmax weights in fp16, each
 * weight carrying its row's scale relative to a running power of two (row
 * scales must be finite and below 2^126).  D is 64 or 128; any Hq / Hkv (up
 * to 8 query heads per kv head in one group, larger groups are split).
 * Workspace and num_splits as for kvd_attend_masked (64-token tiles), short
 * buffers included: with num_splits = 0 they take the one-launch cluster
 * path.
 */
size_t kvd_attend_masked_fp8_workspace_bytes(int B, int Hq, int Hkv, int C, int D, int num_splits);
/* As kvd_attend_masked_plan, for kvd_attend_masked_fp8. */
kvd_status kvd_attend_masked_fp8_plan(int B, int Hq, int Hkv, int C, int D, int num_splits,
                                      kvd_plan* plan);
kvd_status kvd_attend_masked_fp8(const void* q, const void* k_cache, const void* v_cache,
                                 const uint8_t* mask, void* out, float* lse_out, int B, int Hq,
                                 int Hkv, int C, int D, float scale, int num_splits,
                                 void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                 kvd_stream_t stream);

/*
 * FP4 KV rows ([FlashMLA-KV], which names FP4 beside FP8; the granularity and
 * encoding are this library's reading, as for FP8): one row of a kv head is
 *   bytes [0, D/2)          OCP FP4 E2M1 codes, two per byte: element 2j in
 *                           the low nibble of byte j, 2j + 1 in the high one
 *                           (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6)
 *   bytes [D/2, D/2 + 4)    the row's scale, fp32 little-endian
 *   bytes [D/2 + 4, D/2+16) zero
 * so a cache is uint8 [B, Hkv, C, D/2 + KVD_FP4_ROW_PAD] and element d of a
 * row is scale * E2M1(code[d]).
 */
#define KVD_FP4_ROW_PAD 16

/*
 * kvd_append_fp4 -- kvd_append_fp8 with FP4 rows: per new row
 *   amax = max_d |x_d|, scale = amax / 6, code_d = E2M1(x_d / scale)
 * (both divisions fp32 round-to-nearest; codes rounded to the nearest
 * magnitude, ties to the even code, saturated at 6; amax = 0 gives scale 0
 * and zero codes), written as row pos[b] of k_cache / v_cache
 * [B, Hkv, C, D/2 + 16] (uint8).  Arguments, mask, D and errors as for
 * kvd_append_fp8.
 */
kvd_status kvd_append_fp4(void* k_cache, void* v_cache, const void* k_new, const void* v_new,
                          const int32_t* pos, uint8_t* mask, int B, int Hkv, int C, int D,
                          kvd_dtype new_dtype, int32_t* dev_status, kvd_stream_t stream);

/*
 * kvd_attend_masked_fp4 -- kvd_attend_masked over FP4 caches: the same
 * definition with every K/V element dequantised (scale * E2M1(code)).
 *   k_cache, v_cache uint8 [B, Hkv, C, D/2 + 16]; every other argument, the
 * precision rules (E2M1 codes are exact in fp16), workspace, plan and paths as
 * for kvd_attend_masked_fp8.
 */
size_t kvd_attend_masked_fp4_workspace_bytes(int B, int Hq, int Hkv, int C, int D, int num_splits);
/* As kvd_attend_masked_plan, for kvd_attend_masked_fp4. */
kvd_status kvd_attend_masked_fp4_plan(int B, int Hq, int Hkv, int C, int D, int num_splits,
                                      kvd_plan* plan);
kvd_status kvd_attend_masked_fp4(const void* q, const void* k_cache, const void* v_cache,
                                 const uint8_t* mask, void* out, float* lse_out, int B, int Hq,
                                 int Hkv, int C, int D, float scale, int num_splits,
                                 void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                 kvd_stream_t stream);

/*
 * Quantised rows in the paged layout and through index lists ([FlashMLA-KV]
 * "Оптимизация раскладки KV-кэша при decoding" keeps a token's quantised
 * values and scale side by side, on paged KV blocks).  The rows are those of
 * kvd_append_fp8 (RB = D + 16 bytes) and kvd_append_fp4 (RB = D/2 + 16); q
 * and out are bf16; D in {64, 128}; Hq / Hkv <= 8 query heads per kv head
 * share one tensor-core consumer pass, larger groups several.
 *
 * kvd_append_paged_fp8, kvd_append_paged_fp4 -- kvd_append_paged with the
 * quantisation of kvd_append_fp8 / kvd_append_fp4: the new rows k_new, v_new
 * [Q, Hkv, D] (new_dtype bf16 or fp32) quantised row by row and written as
 * whole rows of key_cache, value_cache uint8 [NB, BS, Hkv, RB] at token pos[q]
 * of sequence q, through the gather's index mapping ([PyPTO] 3.2).  Checks
 * and their status bits in kvd_append_paged's order (a refused sequence
 * writes nothing): pos[q] < 0 KVD_DEV_POS_RANGE, seq_offset[q] negative or
 * not a multiple of BS KVD_DEV_SEQ_OFFSET, a column at or beyond cols
 * KVD_DEV_TABLE_COLS, a block outside [0, NB) KVD_DEV_BLOCK_RANGE.
 */
kvd_status kvd_append_paged_fp8(void* key_cache, void* value_cache, const void* k_new,
                                const void* v_new, const int32_t* block_tables,
                                const int32_t* seq_offset, const int32_t* pos, int Q, int NB,
                                int BS, int cols, int Hkv, int D, kvd_dtype new_dtype,
                                int32_t* dev_status, kvd_stream_t stream);
kvd_status kvd_append_paged_fp4(void* key_cache, void* value_cache, const void* k_new,
                                const void* v_new, const int32_t* block_tables,
                                const int32_t* seq_offset, const int32_t* pos, int Q, int NB,
                                int BS, int cols, int Hkv, int D, kvd_dtype new_dtype,
                                int32_t* dev_status, kvd_stream_t stream);
/*
 * kvd_attend_paged_fp8, kvd_attend_paged_fp4 -- kvd_attend_paged over
 * quantised rows: key_cache, value_cache uint8 [NB, BS, Hkv, RB]; the same
 * definition with every K/V element dequantised (scale * code value), the
 * same sequence and block rules and status bits, and the precision rules of
 * kvd_attend_masked_fp8 / _fp4.  Tiles are whole-row TMA boxes of the largest
 * divisor of BS not above 64 rows; workspace and plan from the queries below
 * (splits >= 1).
 */
size_t kvd_attend_paged_fp8_workspace_bytes(int Q, int Hq, int Hkv, int BS, int cols, int D,
                                            int num_splits);
size_t kvd_attend_paged_fp4_workspace_bytes(int Q, int Hq, int Hkv, int BS, int cols, int D,
                                            int num_splits);
kvd_status kvd_attend_paged_fp8_plan(int Q, int Hq, int Hkv, int BS, int cols, int D,
                                     int num_splits, kvd_plan* plan);
kvd_status kvd_attend_paged_fp4_plan(int Q, int Hq, int Hkv, int BS, int cols, int D,
                                     int num_splits, kvd_plan* plan);
kvd_status kvd_attend_paged_fp8(const void* q, const void* key_cache, const void* value_cache,
                                const int32_t* block_tables, const int32_t* seq_lens,
                                const int32_t* seq_offset, void* out, float* lse_out, int Q,
                                int Hq, int Hkv, int NB, int BS, int cols, int D, float scale,
                                int num_splits, void* workspace, size_t workspace_bytes,
                                int32_t* dev_status, kvd_stream_t stream);
kvd_status kvd_attend_paged_fp4(const void* q, const void* key_cache, const void* value_cache,
                                const int32_t* block_tables, const int32_t* seq_lens,
                                const int32_t* seq_offset, void* out, float* lse_out, int Q,
                                int Hq, int Hkv, int NB, int BS, int cols, int D, float scale,
                                int num_splits, void* workspace, size_t workspace_bytes,
                                int32_t* dev_status, kvd_stream_t stream);
/*
 * kvd_attend_indexed_fp8, kvd_attend_indexed_fp4 -- kvd_attend_indexed over
 * quantised rows: k_cache, v_cache uint8 [B, Hkv, C, RB]; the same definition
 * (every entry with 0 <= indices[b, j] < C one softmax term, entries outside
 * [-1, C) skipped and reported) with every K/V element dequantised; the
 * listed rows are gathered whole (RB bytes) with 16-byte cp.async copies.
 * Precision rules of kvd_attend_masked_fp8 / _fp4; workspace and plan from
 * the queries below (splits of at most 128 entries).
 */
size_t kvd_attend_indexed_fp8_workspace_bytes(int B, int Hq, int Hkv, int topk, int D,
                                              int num_splits);
size_t kvd_attend_indexed_fp4_workspace_bytes(int B, int Hq, int Hkv, int topk, int D,
                                              int num_splits);
kvd_status kvd_attend_indexed_fp8_plan(int B, int Hq, int Hkv, int topk, int D, int num_splits,
                                       kvd_plan* plan);
kvd_status kvd_attend_indexed_fp4_plan(int B, int Hq, int Hkv, int topk, int D, int num_splits,
                                       kvd_plan* plan);
kvd_status kvd_attend_indexed_fp8(const void* q, const void* k_cache, const void* v_cache,
                                  const int32_t* indices, void* out, float* lse_out, int B,
                                  int Hq, int Hkv, int C, int topk, int D, float scale,
                                  int num_splits, void* workspace, size_t workspace_bytes,
                                  int32_t* dev_status, kvd_stream_t stream);
kvd_status kvd_attend_indexed_fp4(const void* q, const void* k_cache, const void* v_cache,
                                  const int32_t* indices, void* out, float* lse_out, int B,
                                  int Hq, int Hkv, int C, int topk, int D, float scale,
                                  int num_splits, void* workspace, size_t workspace_bytes,
                                  int32_t* dev_status, kvd_stream_t stream);

/*
 * kvd_attend_masked_noalloc -- the pages have no counterpart to this call; it
 * exists for callers that cannot allocate device memory.  Some host runtimes
 * own all device memory through their own allocator and hand a kernel library
 * only its input and output buffers; some enqueue paths may not allocate at
 * all; some latency-critical loops cannot afford cudaMalloc's implicit device
 * synchronisation.  Such callers cannot supply the workspace that
 * kvd_attend_masked needs once it splits the sequence axis.
 *
 * Same arguments, same result and the same kernels as kvd_attend_masked,
 * minus the workspace: the split scratch lives in an array of
 * KVD_NOALLOC_SCRATCH_BYTES built into the library, which every GPU that
 * loads the library holds until the process exits.  Nothing is allocated.
 *  - Sizes whose split scratch (kvd_attend_masked_workspace_bytes with the
 *    same arguments) exceeds KVD_NOALLOC_SCRATCH_BYTES are rejected with
 *    KVD_ERR_WORKSPACE and a message in kvd_last_error(); pass fewer splits
 *    (num_splits) or use kvd_attend_masked.
 *  - The first call in a device's context looks up the array's device
 *    address there (cudaGetSymbolAddress) and caches it per context; make
 *    that first call before any stream capture on that device (and again
 *    after a cudaDeviceReset, which loads the library's module anew).
 *  - All calls on a device share the one array, which keeps the last call's
 *    contents.  Each call first clears the array's work counters
 *    (kvd_plan.counter_bytes) with cudaMemsetAsync on `stream`
 *    (stream-ordered; no allocation), so a
 *    call whose launch gave up on a bounded wait (KVD_DEV_TIMEOUT) does not
 *    poison the next one.  Calls that may overlap on the GPU (other streams,
 *    unordered host threads) race on the array: the caller must order them.
 */
#define KVD_NOALLOC_SCRATCH_BYTES (8u << 20)
kvd_status kvd_attend_masked_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                     const uint8_t* mask, void* out, float* lse_out, int B,
                                     int Hq, int Hkv, int C, int D, float scale, kvd_dtype dtype,
                                     int num_splits, int32_t* dev_status, kvd_stream_t stream);

size_t kvd_attend_paged_workspace_bytes(int Q, int Hq, int Hkv, int BS, int cols, int D,
                                        kvd_dtype dtype, int num_splits);
/* As kvd_attend_masked_plan, for kvd_attend_paged (rows = sequences; the
 * one-launch cluster kernel is never used: splits >= 1). */
kvd_status kvd_attend_paged_plan(int Q, int Hq, int Hkv, int BS, int cols, int D, kvd_dtype dtype,
                                 int num_splits, kvd_plan* plan);
kvd_status kvd_attend_paged(const void* q_in, const void* key_cache, const void* value_cache,
                            const int32_t* block_tables, const int32_t* seq_lens,
                            const int32_t* seq_offset, void* out, float* lse_out, int Q, int Hq,
                            int Hkv, int NB, int BS, int cols, int D, float scale,
                            kvd_dtype dtype, int num_splits, void* workspace,
                            size_t workspace_bytes, int32_t* dev_status, kvd_stream_t stream);

/*
 * kvd_append_paged -- the step's KV append ([NPU] Part 2, update_kvcache_for)
 * into the paged cache, through the gather's index mapping ([PyPTO] 3.2):
 * token pos[q] of sequence q is written to
 *   key_cache[block_tables[q, seq_offset[q] / BS + pos[q] / BS], pos[q] % BS]
 * (all Hkv x D of it; value_cache likewise), i.e. where kvd_gather_paged and
 * kvd_attend_paged read token pos[q] of q once seq_lens counts it.
 *   key_cache, value_cache [NB, BS, Hkv, D] of `dtype`
 *   k_new, v_new [Q, Hkv, D] of `dtype`;  pos [Q] int32 (device)
 *   block_tables [Q, cols] int32;  seq_offset [Q] int32 or NULL (zeros)
 * A byte copy.  Device-detected errors skip that sequence (nothing written):
 * pos[q] < 0 (KVD_DEV_POS_RANGE), seq_offset negative or not a multiple of
 * BS (KVD_DEV_SEQ_OFFSET), table column past cols (KVD_DEV_TABLE_COLS), block
 * id outside [0, NB) (KVD_DEV_BLOCK_RANGE).  The caller keeps seq_lens.
 */
kvd_status kvd_append_paged(void* key_cache, void* value_cache, const void* k_new,
                            const void* v_new, const int32_t* block_tables,
                            const int32_t* seq_offset, const int32_t* pos, int Q, int NB, int BS,
                            int cols, int Hkv, int D, kvd_dtype dtype, int32_t* dev_status,
                            kvd_stream_t stream);

/*
 * kvd_gather_paged -- gather_pa_kv_cache, Norm/ND branch ([PyPTO] 3.2):
 * for every sequence q and t < seq_lens[q+1] - seq_lens[q]:
 *   phys = block_tables[q, seq_offset[q] / BS + t / BS]
 *   key_out[seq_lens[q] + t] = key_cache[phys, t % BS]   (all Hk x Dk)
 *   value_out[seq_lens[q] + t] = value_cache[phys, t % BS] (all Hv x Dv)
 *   key_cache [NB, BS, Hk, Dk], value_cache [NB, BS, Hv, Dv], elem_bytes 2 or 4
 *   key_out [total_tokens, Hk, Dk], value_out [total_tokens, Hv, Dv]
 * A byte copy (bit-exact).  total_tokens must equal seq_lens[Q] and is
 * passed from the host.  Device-detected errors (SEQLENS, SEQ_OFFSET,
 * TABLE_COLS) skip the whole sequence; BLOCK_RANGE skips that block's rows;
 * skipped rows are left untouched.  Rows must be whole multiples of 2 bytes.
 */
kvd_status kvd_gather_paged(const void* key_cache, const void* value_cache,
                            const int32_t* block_tables, const int32_t* seq_lens,
                            const int32_t* seq_offset, void* key_out, void* value_out, int Q,
                            int NB, int BS, int cols, int Hk, int Dk, int Hv, int Dv,
                            int total_tokens, int elem_bytes, int32_t* dev_status,
                            kvd_stream_t stream);

/*
 * kvd_combine -- log-sum-exp merge of partial results over disjoint key
 * ranges ([NPU] Part 3, Flash SDPA path: tiles merged exactly):
 *   LSE[r] = log sum_s exp(part_lse[r, s]),
 *   out[r, :] = sum_s exp(part_lse[r, s] - LSE[r]) * part_o[r, s, :]
 *   part_o [R, S, D] float (each normalised over its range), part_lse [R, S]
 *   float (natural log, -inf = empty range whose part_o is ignored)
 *   out [R, D] of out_dtype;  lse_out [R] float or NULL
 * All ranges empty: out = 0, LSE = -inf.  D a multiple of 4, at most 1024.
 */
kvd_status kvd_combine(const float* part_o, const float* part_lse, void* out, float* lse_out,
                       int R, int S, int D, kvd_dtype out_dtype, kvd_stream_t stream);

/*
 * kvd_combine_gathered -- kvd_combine over the exchange layout of a
 * sequence split across S ranks: `parts` float [S, R * (D + 1)] holds, for
 * range s, its R partial rows [R, D] followed by their R log-sum-exps
 * (kvd_attend_masked_partial writing out and lse_out into the two parts of
 * one rank's block), the blocks one after the other as an all-gather of the
 * blocks along the first axis leaves them.  Same formula, outputs and rules
 * as kvd_combine (range s of row r has part_o = parts[s, r*D : (r+1)*D] and
 * part_lse = parts[s, R*D + r]).
 */
kvd_status kvd_combine_gathered(const float* parts, void* out, float* lse_out, int R, int S,
                                int D, kvd_dtype out_dtype, kvd_stream_t stream);

/*
 * Latent caches.  One row a token, shared by all heads: R latent values, which
 * are the keys and the values at once, and P rotary key values.  The paged
 * cache is the one kvd_gather_paged reads with one head ([PyPTO] 3.1, 8.1):
 *   latent_cache [NB, BS, 1, R], rope_cache [NB, BS, 1, P] of `dtype`.
 * R in {128, 256, 384, 512}, P = 64.  The attention of such a cache has two
 * forms.  With the up-projections multiplied into the queries and the outputs
 * (absorbed), it runs over the rows themselves: kvd_attend_latent.  With the
 * rows gathered and expanded into keys and values per head, it is ordinary
 * attention whose rotary key part is shared: kvd_attend_expanded.
 */

/*
 * kvd_append_latent -- kvd_append_paged for latent rows, any number of new
 * tokens a sequence: row new_lens[q] + i of latent_new and rope_new is written
 * to token pos[q] + i of sequence q, 0 <= i < new_lens[q + 1] - new_lens[q],
 * i.e. to page block_tables[q, seq_offset[q] / BS + (pos[q] + i) / BS], slot
 * (pos[q] + i) % BS.
 *   latent_cache [NB, BS, 1, R], rope_cache [NB, BS, 1, P] of `dtype` (in/out)
 *   latent_new [N, R], rope_new [N, P] of `dtype`, packed
 *   new_lens [Q + 1] int32, cumsum starting at 0;  pos [Q] int32 (device)
 *   block_tables [Q, cols] int32;  seq_offset [Q] int32 or NULL (zeros)
 * A byte copy.  Rows at and behind new_lens[Q] go nowhere.  Device-detected
 * errors skip the row (nothing written): new_lens not starting at 0 (every row),
 * a pair past N (its rows; both KVD_DEV_SEQLENS), pos[q] < 0
 * (KVD_DEV_POS_RANGE), seq_offset negative or not a multiple of BS
 * (KVD_DEV_SEQ_OFFSET), table column past cols (KVD_DEV_TABLE_COLS), block id
 * outside [0, NB) (KVD_DEV_BLOCK_RANGE).  Where new_lens decreases
 * (KVD_DEV_SEQLENS) the rows below the smallest value that it falls to go where
 * they belong, the others to one sequence whose pair holds them, or nowhere.
 * With Q = 0 or N = 0 nothing is launched, and new_lens is not looked at.
 * Any R and P with rows of whole 16-byte vectors.
 */
kvd_status kvd_append_latent(void* latent_cache, void* rope_cache, const void* latent_new,
                             const void* rope_new, const int32_t* block_tables,
                             const int32_t* seq_offset, const int32_t* new_lens,
                             const int32_t* pos, int Q, int N, int NB, int BS, int cols, int R,
                             int P, kvd_dtype dtype, int32_t* dev_status, kvd_stream_t stream);

/*
 * kvd_attend_latent -- attention of the newest T tokens of every sequence over
 * the paged latent cache, the absorbed form ([FlashMLA] "Математическая
 * постановка": one KV row per token, the values its first R elements).  With
 * n = seq_lens[q + 1] - seq_lens[q] tokens in the cache (the T new ones among
 * them), query token t of sequence q and head h:
 *   s_k = scale * (q_latent[q, t, h, :] . latent_k + q_rope[q, t, h, :] . rope_k)
 *   out[q, t, h, :] = sum_k w_k latent_k / sum_k w_k,  w_k = exp(s_k - max)
 *   lse[q, t, h] = log sum_k exp(s_k),  over the tokens 0 <= k <= n - T + t
 * (token t of the newest T sees everything up to itself; T = 1: the whole
 * sequence).  A query with no such token (n - T + t < 0) gives out = 0,
 * lse = -inf.
 *   q_latent [Q, T, H, R], q_rope [Q, T, H, P] of `dtype`
 *   block_tables, seq_lens, seq_offset as for kvd_attend_paged
 *   out [Q, T, H, R] of `dtype`;  lse_out [Q, T, H] float or NULL
 * Slots of a page behind the sequence's end, and the rotary values of tokens
 * behind a query's own, may hold anything (inf, NaN) without reaching it.  The
 * latent rows of a sequence, which are values too, must be finite: one that is
 * not reaches all T queries of its sequence, also those that come before it.
 * bf16: scores, maxima and sums are held in fp32, the weights w_k are rounded to
 * bf16 before they multiply latent_k, and out is rounded once.
 * Device-detected errors as for kvd_attend_paged: KVD_DEV_SEQLENS, SEQ_OFFSET
 * and TABLE_COLS make the sequence empty, KVD_DEV_BLOCK_RANGE drops the
 * block's tokens.
 * Workspace: at least kvd_attend_latent_workspace_bytes(...) bytes, 256-byte
 * aligned; its contents do not matter before a call (no zero fill) and calls
 * that may overlap on the GPU must not share one.
 */
size_t kvd_attend_latent_workspace_bytes(int Q, int T, int H, int BS, int cols, int R, int P,
                                         kvd_dtype dtype);
kvd_status kvd_attend_latent(const void* q_latent, const void* q_rope, const void* latent_cache,
                             const void* rope_cache, const int32_t* block_tables,
                             const int32_t* seq_lens, const int32_t* seq_offset, void* out,
                             float* lse_out, int Q, int T, int H, int NB, int BS, int cols, int R,
                             int P, float scale, kvd_dtype dtype, void* workspace,
                             size_t workspace_bytes, int32_t* dev_status, kvd_stream_t stream);

/*
 * kvd_attend_expanded -- the expanded form, for prompts and chunks of them:
 * packed sequences, per-head keys and values that were expanded from gathered
 * latent rows (kv, as one projection leaves them: Dn key values, then Dv
 * values), the rotary key part shared by all heads.  With nq queries and nk
 * keys of sequence b, query i of head h sees the keys 0 <= j <= i + nk - nq
 * (causal from the end: the last query sees every key):
 *   s_j = scale * (q[i, h, :Dn] . kv[j, h, :Dn] + q[i, h, Dn:] . k_rope[j, :])
 *   out[i, h, :] = sum_j w_j kv[j, h, Dn:] / sum_j w_j,  w_j = exp(s_j - max)
 *   lse[i, h] = log sum_j exp(s_j)
 * With causal = 0 every query of b sees all nk keys.  A query that sees no
 * key gives out = 0, lse = -inf.
 *   q [Nq, H, Dn + P], kv [Nk, H, Dn + Dv], k_rope [Nk, P] of `dtype`
 *   q_lens, k_lens [Q + 1] int32, cumsum starting at 0 (device)
 *   out [Nq, H, Dv] of `dtype`;  lse_out [Nq, H] float or NULL
 * Rows of out and lse_out at and behind q_lens[Q] are left as they were; rows
 * of kv and k_rope of other sequences and behind k_lens[Q], and keys that a query
 * does not see, may hold anything (inf, NaN) without reaching it.  The values of
 * a sequence must be finite: one that is not may reach queries before it.
 * bf16: as for kvd_attend_latent, the weights are rounded to bf16 before they
 * multiply the values.
 * Device-detected errors: a bad pair of k_lens (not starting at 0, decreasing,
 * past Nk) makes the sequence's keys empty; a bad pair of q_lens skips its
 * queries, a decreasing one those of all sequences behind it too (rows that are
 * not computed are left as they were); both set KVD_DEV_SEQLENS.  With Q = 0 or
 * Nq = 0 nothing is launched, and the lengths are not looked at.
 * Supported: Dn, Dv in {64, 128}, P = 64.  Needs no workspace.
 */
kvd_status kvd_attend_expanded(const void* q, const void* kv, const void* k_rope,
                               const int32_t* q_lens, const int32_t* k_lens, void* out,
                               float* lse_out, int Q, int Nq, int Nk, int H, int Dn, int Dv, int P,
                               float scale, int causal, kvd_dtype dtype, int32_t* dev_status,
                               kvd_stream_t stream);

/*
 * kvd_verify_drafts -- drafted tokens against the target's probabilities, from
 * given random numbers.  Sequence q has m = num_drafts[q] drafts (T without
 * num_drafts) x_i = draft_tokens[q, i], drawn from draft_probs[q, i, :].
 *   draft i is accepted while  u_accept[q, i] * draft_probs[q, i, x_i] <
 *   target_probs[q, i, x_i]  (in 64 bits) and all drafts before it are;
 *   n = number of accepted drafts;
 *   one more token comes from the weights w_v = max(target_probs[q, n, v] -
 *   draft_probs[q, n, v], 0) if n < m (from target_probs[q, n, v] itself where
 *   these are all zero), w_v = target_probs[q, m, v] if n = m: the smallest v
 *   with w_0 + ... + w_v > u_sample[q] * (sum of w), the largest v with
 *   w_v > 0 where rounding leaves none.
 *   tokens[q, :] = x_0 .. x_{n-1}, that token, then -1;  accepted[q] = n.
 *   target_probs [Q, T + 1, V], draft_probs [Q, T, V] of `dtype`; they need
 *   not be normalised; NaN and negative weights count as zero
 *   draft_tokens [Q, T] int32;  u_accept [Q, T], u_sample [Q] float in [0, 1)
 *   num_drafts [Q] int32 or NULL;  tokens [Q, T + 1] int32;  accepted [Q] int32
 * T = 0 (a token without drafts) takes NULL for the drafts' arrays.  The
 * acceptance and the differences are exact to 64 bits; a sum is right to about
 * 2^-47 of itself (two fp32 words for 64 elements of a lane, 64 bits above), so
 * that only a draw closer than that to a border can differ from one in 64 bits.
 * Finite weights count whatever their sum.  Device-detected errors: a drafted
 * token outside [0, V) is rejected (KVD_DEV_TOKEN_RANGE); no weight above zero,
 * or an infinite one, gives the token -1 (KVD_DEV_PROBS); num_drafts[q] outside
 * [0, T] gives tokens -1 and accepted 0 (KVD_DEV_POS_RANGE).
 */
kvd_status kvd_verify_drafts(const void* target_probs, const void* draft_probs,
                             const int32_t* draft_tokens, const float* u_accept,
                             const float* u_sample, const int32_t* num_drafts, int32_t* tokens,
                             int32_t* accepted, int Q, int T, int V, kvd_dtype dtype,
                             int32_t* dev_status, kvd_stream_t stream);

/*
 * The serving step around the paged cache: pages and slots for the step's new
 * tokens (kvd_plan_pages), their queries, keys and values normed, rotated and
 * appended (kvd_rotate_append_paged), decode attention of sequences behind
 * shared prefixes (kvd_attend_paged_prefix), and the next tokens from the logits
 * (kvd_sample, or kvd_filter_probs in front of kvd_verify_drafts).
 */

/*
 * kvd_plan_pages -- pages, slots and positions from the requests' lengths,
 * without the host.  Sequence q keeps the kept_lens[q] first tokens that it has
 * in the cache (fewer than before where drafted tokens were rejected, 0 where a
 * request is over) and gets new_lens[q + 1] - new_lens[q] new ones; with
 *   need[q] = ceil((kept + new) / BS)
 * pages it gives pages back where it holds more and takes some where it holds
 * fewer:
 *  - first, all pages given back are pushed onto the free list, the last
 *    sequence's last column first;
 *  - then pages are taken from the list's end, the first sequence's first column
 *    first (so that taking and giving back the same pages leaves the list as it
 *    was), while they last: a sequence whose pages and those of all sequences
 *    before it are more than there are gets none (KVD_DEV_NO_PAGES).  One that
 *    needs more than cols pages asks for none; what was refused to one for want of
 *    pages does count against those behind it.
 *   block_tables [Q, cols] int32   columns [0, pages_held[q]) are q's (in/out)
 *   pages_held   [Q] int32         (in/out)
 *   free_pages   [F] int32, free_count [1] int32: the first free_count entries
 *                are free pages (in/out); F: at least all pages of the cache (NULL
 *                with F = 0)
 *   kept_lens    [Q] int32;  new_lens [Q + 1] int32, cumsum starting at 0
 *   pos_base     [Q] int32 or NULL (zeros): the position of q's first token (the
 *                length of a shared prefix before it)
 *   seq_lens     [Q + 1] int32 (out): cumsum of kept + new, as the attention
 *                calls take it
 *   slots, positions [N] int32 (out): token new_lens[q] + i of the packed new
 *                tokens is token t = kept + i of q,
 *                slot = block_tables[q, t / BS] * BS + t % BS, position =
 *                pos_base[q] + t; both -1 for tokens without a place: those of a
 *                refused sequence, and padding behind new_lens[Q]
 * A refused sequence keeps its pages and counts kept_lens[q] tokens: too few pages
 * left, or need above cols (KVD_DEV_TABLE_COLS).  A bad one is left alone and counts
 * none: kept_lens negative or more than its pages hold, pages_held outside [0,
 * cols], or kept + new past 2^31 - 1 (KVD_DEV_POS_RANGE).  One whose end in seq_lens
 * would pass 2^31 - 1, it and those before it counted, takes no pages and counts
 * none (KVD_DEV_SEQLENS); pages above its need[q] are given back all the same and no
 * longer held.  All sequences are refused, and none gives pages back, by a new_lens
 * that does not start at 0, decreases or passes N (KVD_DEV_SEQLENS) and by a
 * free_count outside [0, F] (KVD_DEV_POS_RANGE).  Where the list has no room for all
 * pages given back, none is (KVD_DEV_NO_PAGES).  A token whose page is negative or
 * whose slot is past 2^31 - 1 (KVD_DEV_BLOCK_RANGE), or whose position is outside 32
 * bits (KVD_DEV_POS_RANGE), has no place.  One launch, two for many tokens; runs
 * that change the same tables must be ordered.  Q at most 2^20, N at most 2^30.
 */
kvd_status kvd_plan_pages(int32_t* block_tables, int32_t* pages_held, int32_t* free_pages,
                          int32_t* free_count, const int32_t* kept_lens, const int32_t* new_lens,
                          const int32_t* pos_base, int32_t* seq_lens, int32_t* slots,
                          int32_t* positions, int Q, int N, int BS, int cols, int F,
                          int32_t* dev_status, kvd_stream_t stream);

/* How rotary frequencies are stretched for contexts longer than the trained one. */
typedef enum {
    KVD_ROPE_PLAIN = 0,  /* f_i = base^(-2 i / Dr) */
    KVD_ROPE_LINEAR = 1, /* f_i / factor: positions brought closer */
    KVD_ROPE_BASE = 2,   /* base * factor^(Dr / (Dr - 2)) in place of base */
    KVD_ROPE_PARTS = 3   /* frequencies that make more than `fast` turns over the
                            `trained` length stay, those below `slow` turns are divided
                            by factor, a linear mixture by turns between */
} kvd_rope_scaling;

/*
 * kvd_rotary_freqs -- the frequencies of Dr rotated dims, in radians a position,
 * into freqs [Dr / 2], HOST memory; the caller copies them to the device once.
 * factor > 0 (not used by PLAIN); trained > 0 and fast > slow > 0 for PARTS only.
 */
kvd_status kvd_rotary_freqs(double* freqs, int Dr, double base, kvd_rope_scaling scaling,
                            double factor, double trained, double fast, double slow);

/*
 * kvd_rotate -- norm and rotation of every head of N tokens:
 *   y = x * weight / sqrt(mean_D(x^2) + eps)        (y = x without a weight)
 *   pair i of the first Dr dims, (y_i, y_{i + Dr/2}), or (y_2i, y_{2i+1}) if
 *   `interleaved`, at position p = positions[n]:
 *     (a, b) -> (a c - b s, a s + b c),  c, s = rotary_scale * cos, sin(p freqs[i])
 *   dims at and behind Dr are not rotated (nor scaled).
 *   x, out [N, H, D] of `dtype` (out may be x), weight [D] of `dtype` or NULL
 *   freqs [Dr / 2] double, device (NULL with Dr = 0);  positions [N] int32
 * fp32 arithmetic, one rounding; the angle is taken in 64 bits, so that far
 * positions lose nothing.  A token at position -1 is left out (its row of out
 * stays as it was), other negative ones too and set KVD_DEV_POS_RANGE.
 * D in {64, 128}; Dr a multiple of 16, 0 <= Dr <= D.
 */
kvd_status kvd_rotate(const void* x, const void* weight, const double* freqs,
                      const int32_t* positions, void* out, int N, int H, int D, int Dr,
                      int interleaved, float rotary_scale, float eps, kvd_dtype dtype,
                      int32_t* dev_status, kvd_stream_t stream);

/*
 * kvd_rotate_append_paged -- kvd_rotate of a fused projection's queries and keys,
 * the keys and the (unchanged) values straight into the paged cache:
 *   qkv [N, Hq + 2 Hkv, D] of `dtype`: Hq queries, Hkv keys, Hkv values a token
 *   q_out [N, Hq, D];  key_cache, value_cache [NB, BS, Hkv, D] of `dtype`
 *   slots [N] int32: the token's row block * BS + slot of the caches, as
 *   kvd_plan_pages gives it
 * A token at position -1 is left out altogether; one with slot -1 has its queries
 * rotated and nothing appended.  Any other negative position, or a slot outside
 * [-1, NB * BS), counts as -1 and sets KVD_DEV_POS_RANGE or KVD_DEV_BLOCK_RANGE.
 * Two tokens with one slot leave one of them there.  Otherwise as kvd_rotate.
 */
kvd_status kvd_rotate_append_paged(const void* qkv, const void* q_weight, const void* k_weight,
                                   const double* freqs, const int32_t* positions,
                                   const int32_t* slots, void* q_out, void* key_cache,
                                   void* value_cache, int N, int Hq, int Hkv, int NB, int BS,
                                   int D, int Dr, int interleaved, float rotary_scale, float eps,
                                   kvd_dtype dtype, int32_t* dev_status, kvd_stream_t stream);

/*
 * kvd_attend_paged_prefix -- kvd_attend_paged for groups of sequences that share
 * a prefix, which is kept once and read once a group: the sequences group_lens[i]
 * <= q < group_lens[i + 1] attend over the first prefix_lens[i] tokens of the
 * pages prefix_tables[i, :], and then over their own tokens as in
 * kvd_attend_paged; one softmax over both.  Sequences behind group_lens[G] have
 * no prefix.
 *   q [Q, Hq, D], key_cache, value_cache [NB, BS, Hkv, D] of `dtype`
 *   prefix_tables [G, pcols], prefix_lens [G], group_lens [G + 1] (cumsum of the
 *   groups' sequences starting at 0) int32, device; NULL with G = 0
 *   block_tables [Q, cols], seq_lens [Q + 1], seq_offset, out, lse_out, scale as
 *   for kvd_attend_paged: a sequence's own tokens, none for some
 * Errors of a sequence's own pages as for kvd_attend_paged (its prefix still
 * counts).  Prefixes: a negative length (KVD_DEV_SEQLENS) or one past pcols pages
 * (KVD_DEV_TABLE_COLS) counts as none; an out-of-range block
 * (KVD_DEV_BLOCK_RANGE) drops its tokens; a group_lens that does not start at 0,
 * decreases or passes Q leaves every sequence without a prefix (KVD_DEV_SEQLENS).
 * A query without any key gives out = 0, lse = -inf.  Slots behind a prefix's or
 * a sequence's end may hold anything (inf, NaN).
 * bf16: the weights of a prefix's keys are rounded to bf16 before they multiply the
 * values (their sum keeps fp32), whatever Hq / Hkv; those of own keys as in
 * kvd_attend_paged, which rounds them from three query heads a kv head on.
 * Pays where a group's sequences times its prefix's tokens are above some 8000 (16000
 * where the caches do not come from L2); below, kvd_attend_paged over tables that
 * list the prefix's pages in front is up to 6 us faster.
 * Workspace: at least kvd_attend_paged_prefix_workspace_bytes(...) bytes, 256-byte
 * aligned; its contents do not matter before a call, and calls that may overlap
 * on the GPU must not share one.  D in {64, 128}; any Hq multiple of Hkv;
 * G at most 1024; pcols * BS at most 2^31 - 128.
 */
size_t kvd_attend_paged_prefix_workspace_bytes(int Q, int G, int Hq, int Hkv, int BS, int pcols,
                                               int cols, int D, kvd_dtype dtype);
kvd_status kvd_attend_paged_prefix(const void* q, const void* key_cache, const void* value_cache,
                                   const int32_t* prefix_tables, const int32_t* prefix_lens,
                                   const int32_t* group_lens, const int32_t* block_tables,
                                   const int32_t* seq_lens, const int32_t* seq_offset, void* out,
                                   float* lse_out, int Q, int G, int Hq, int Hkv, int NB, int BS,
                                   int pcols, int cols, int D, float scale, kvd_dtype dtype,
                                   void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                   kvd_stream_t stream);

/*
 * kvd_sample -- a token for each row of logits, from given random numbers.  With
 * T = temperature[r] and w_v = exp((l_v - max l) / T), logits in falling order
 * (equal ones by index, the lowest first):
 *   top-k:  the first top_k[r] tokens stay (all if top_k[r] <= 0 or > V);
 *   top-p:  of these, a token stays while the sum of the weights before it is
 *           below top_p[r] times their sum (all if top_p[r] >= 1);
 *   min-p:  of these, the tokens with w_v >= min_p[r] stay (all if min_p[r] <= 0;
 *           above 1 counts as 1);
 * the first always stays.  T = 0 keeps the first alone.  tokens[r] is the smallest
 * v whose running sum of the weights that stay, in index order, is above u[r] times
 * their sum.
 *   logits [R, V] of `dtype`;  temperature [R], top_p [R], min_p [R] float and
 *   top_k [R] int32, device, or NULL (1, all, all, all);  u [R] float in [0, 1)
 *   tokens [R] int32
 * NaN logits count as -inf; among infinite ones the weight is shared alike.
 * Weights are right to about 2^-28 of themselves, without a trend, and are summed as
 * whole multiples of 2^-42 of the largest, in any order to the same sum.  A multiple
 * is half of one off at most, but equal weights to the same side: a draw or a top-p
 * border that differs from one in 64 bits lies within 2^-28 + V 2^-43 of the sum (2^-23
 * for V = 2^20) of a token's border, and weights below 2^-43 of the largest count as
 * zero: such a token is not drawn.
 * A row without a logit above -inf gives -1 (KVD_DEV_PROBS); a NaN, a temperature
 * below 0 or above 1e30, or u outside [0, 1) gives -1 (KVD_DEV_PARAM).
 * V at most 2^20.
 */
kvd_status kvd_sample(const void* logits, const float* temperature, const int32_t* top_k,
                      const float* top_p, const float* min_p, const float* u, int32_t* tokens,
                      int R, int V, kvd_dtype dtype, int32_t* dev_status, kvd_stream_t stream);

/*
 * kvd_filter_probs -- the distributions that kvd_sample draws from: probs[r, v] =
 * w_v over the sum of the weights that stay, 0 for the others, as kvd_verify_drafts
 * takes them.  probs [R, V] of probs_dtype, not overlapping the logits; rows that
 * kvd_sample refuses are zero.  Weights that stay but are too small to be drawn keep
 * their probability (down to 2^-125 of the largest).  Otherwise as kvd_sample.
 */
kvd_status kvd_filter_probs(const void* logits, const float* temperature, const int32_t* top_k,
                            const float* top_p, const float* min_p, void* probs, int R, int V,
                            kvd_dtype dtype, kvd_dtype probs_dtype, int32_t* dev_status,
                            kvd_stream_t stream);

/* Human-readable name of a status code (static string). */
const char* kvd_status_string(kvd_status status);
/* Description of the last error returned on the calling thread (static per thread). */
const char* kvd_last_error(void);
/* Library ABI version: major * 10000 + minor * 100 + patch. */
int kvd_version(void);

#ifdef __cplusplus
}
#endif
#endif /* KVD_H */
