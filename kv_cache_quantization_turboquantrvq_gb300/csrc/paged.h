// paged.h - internal interface of the paged-cache operators (append, gather,
// attention over pages) between their C-ABI front end (paged_api.cpp) and the
// kernel translation units.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "launch.h"

namespace vq {

// ---------------------------------------------------------------- the cache
//
// One layer's pages: k_pages, v_pages [num_pages, Hkv, page_size, 128] of 16-bit
// entries or e4m3 codes; with codes, k_exp, v_exp [num_pages, Hkv, page_size]
// hold one exponent per token and head, biased by 127: value = code * 2^(exp - 127).
struct PagedCache {
    const void *k, *v;
    const uint8_t *ke, *ve;  // e4m3 only
    int num_pages, Hkv, page_shift;
};

// exponents of a row: the least e in [PG_EMIN, PG_EMAX] with max|x| <= 448 * 2^e
constexpr int PG_EMIN = -32, PG_EMAX = 64;

struct PagedAppendParams {
    PagedCache c;
    const void *k_in, *v_in;
    long long kst, ksh, vst, vsh;  // element strides of k_in, v_in: token, head
    const long long *slots;        // [T]
    int T;
    FastDiv divH;
};
cudaError_t launch_paged_append(const PagedAppendParams &p, int in_dtype, int cache_dtype, cudaStream_t stream);

struct PagedGatherParams {
    PagedCache c;
    const int32_t *table, *lens, *first;  // first may be null (0)
    void *k_out, *v_out;                  // [B, Hkv, S_out, 128], either may be null
    int B, max_pages, S_out;
    FastDiv divS, divH;
};
cudaError_t launch_paged_gather(const PagedGatherParams &p, int cache_dtype, int out_dtype, cudaStream_t stream);
cudaError_t paged_cache_take_device_error(unsigned *bits, cudaStream_t stream);

// ------------------------------------------------ keeping a part of the cache

struct PagedSelectParams {
    const float *weights;             // [num_pages, Hkv, page_size]
    const int32_t *table, *lens;
    int32_t *keep, *counts;           // [B, Hkv, budget], [B]
    int num_pages, Hkv, page_shift;
    int B, max_pages, budget, recent, sinks;
    int held;                         // weights of a CTA that stay in shared memory (set by the launcher)
};
cudaError_t launch_paged_select(const PagedSelectParams &p, cudaStream_t stream);

struct PagedCompactParams {
    PagedCache c;
    const int32_t *table, *keep, *counts, *first;  // first may be null (0)
    float *weights;                                // [num_pages, Hkv, page_size], may be null
    long long keep_b, keep_h;                      // strides of keep: sequence, head (0: one list for all heads)
    int B, max_pages, K;
};
cudaError_t launch_paged_compact(const PagedCompactParams &p, int cache_dtype, cudaStream_t stream);
cudaError_t paged_keep_take_device_error(unsigned *bits, cudaStream_t stream);

// ------------------------------------------------------------ the attention
//
// The new tokens of the sequences are cut into entries (tq consecutive tokens
// of one sequence, so tq * GQ query rows of one kv head); entry x kv head is an
// item, and an item's keys are cut into tiles of PG_TILE keys, the units of
// work.  All units of a launch lie in one line, ordered by entry, head, tile,
// and CTA c of G takes units [c U / G, (c + 1) U / G): an even share, whatever
// the mix of lengths.  An item cut by a CTA boundary leaves partial results (one
// slot for the item a CTA enters in the middle, one for the item it leaves
// unfinished), merged by the combine kernel in the order of the CTAs.
constexpr int PG_TILE = 128;
constexpr int PLAN_CTAS = 512;  // CTAs of a launch at most

struct PgEntry {     // 32 bytes, read as two int4
    int b, tok0, nt; // sequence, first query token (index into q), number of tokens
    int p0;          // position of the first token in its sequence (may be negative);
                     // of a tree, of the sequence's first drafted token
    int hi;          // keys [0, hi) are visible to some row
    int nsink;       // leading tiles that hold the first tokens kept by the window
    int tl;          // first tile after those
    int ntiles;      // tiles of the entry (at least 1)
};
struct PgStart {     // where a CTA starts: 48 bytes, read as three int4
    int ei, h, t;    // entry, kv head, tile
    int left;        // units of the CTA (0: nothing to do)
    PgEntry e;       // entry ei
};
// One class of entries (small: few rows; large: tensor-memory tiles): device arrays.
struct PgPlan {
    PgStart *start;    // [G]
    int4 *cmb;         // [G] what is merged at its start: parts (0: nothing), first token, tokens, head
    PgEntry *ent;
    long long *base;   // first unit of each entry
    float *part;       // [G][2] partial slots
    int cap, G, tq;    // entries that fit, CTAs, tokens per entry
};

// What the new tokens of a call are: each sequence's next ones in order, or a tree
// of drafts, in which a token sees its ancestors only; or (WEIGH) the next ones,
// whose softmax weights are added up too.
enum PgMode { PG_CHAIN, PG_TREE, PG_WEIGH };
constexpr int PG_TREE_MAX = 256, PG_TREE_WORDS = PG_TREE_MAX / 32;  // tokens of a tree

struct PagedAttendParams {
    CUtensorMap tmk, tmv, tmq;
    PagedCache c;
    const void *q;
    long long qst, qsh;          // element strides of q: token, head
    const int32_t *table, *cu, *lens;
    void *out;                   // [T, Hq, 128]
    int T, B, Hq, Hkv, GQ, max_pages, max_q;
    int window, sinks;           // window 0: all earlier keys
    int small_rows;              // sequences with at most this many query rows per kv head are small
    float qscale;                // softmax scale * log2(e)
    PgPlan small, large;         // cap 0: the class is not used
    unsigned long long *planned; // (both classes) `call` from when the plan is made until the merge
    unsigned long long call;     // a number of this call's own, not 0
    const int32_t *parents;      // [T] trees; null: no tree
    uint32_t *masks;             // [T][PG_TREE_WORDS] trees in the large class: the new tokens that a token sees
    int32_t *depth;              // [T] and its number of ancestors
    // (WEIGH)
    float *lse;                  // [Hkv, T, GQ] log2 of each query row's sum of 2^score; null: no weights
    float *scores;               // [B, Hkv, srows, keys] scores of single tokens, or sums over parts of a chunk
    int srows, keys;
    long long *wbase;            // [B + 1] units of weighing before each sequence of the large class
    float *weights;              // [num_pages, Hkv, page_size]
    float decay;
    int observe;                 // new tokens of a sequence that count, the last ones; 0: all
};
constexpr int PG_PARTS = 8;      // parts that a chunk's query rows are weighed in, at most
constexpr int PG_SROWS = 16;     // rows of a small item
constexpr int PG_LROWS = 256;    // rows of a large item (two tensor-memory tiles)
// Floats of a row's partial result.  A slot holds the rows' maxima, then their
// sums, then their outputs: of small items row by row, of large ones 32 rows by
// 32, and of those 8 columns after another, each [32 rows][8].
constexpr int PG_PART = 2 + 128;


// A launch that may start while the kernel before it in the stream still runs
// (it waits for that kernel's results by itself, pg_wait()).
template <class... A, class... B>
cudaError_t launch_early(void (*kern)(A...), dim3 grid, int threads, int smem, cudaStream_t stream, const B &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

cudaError_t launch_paged_plan(const PagedAttendParams &p, cudaStream_t stream);
cudaError_t launch_paged_small(const PagedAttendParams &p, int q_dtype, int cache_dtype, cudaStream_t stream);
cudaError_t launch_paged_large(const PagedAttendParams &p, int q_dtype, int cache_dtype, cudaStream_t stream);
cudaError_t paged_chunk_take_device_error(unsigned *bits, cudaStream_t stream);
cudaError_t launch_paged_weigh(const PagedAttendParams &p, int q_dtype, int cache_dtype, cudaStream_t stream);
cudaError_t launch_paged_weigh_update(const PagedAttendParams &p, cudaStream_t stream);
cudaError_t paged_weigh_take_device_error(unsigned *bits, cudaStream_t stream);
cudaError_t launch_paged_combine(const PagedAttendParams &p, int q_dtype, cudaStream_t stream);
cudaError_t paged_attend_take_device_error(unsigned *bits, cudaStream_t stream);

// Tensor map of pages [rows, 128]: 16-bit boxes of 64 columns, 8-bit boxes of
// 128 columns (128 bytes a row), `box_rows` rows, 128-byte swizzle.
bool encode_tmap_pages(CUtensorMap *map, const void *base, uint64_t rows, int elem_bytes, uint32_t box_rows);
// The same 16-bit rows as [2 halves, rows, 64]: a box holds `box_rows` rows of the
// first half, then of the second.
bool encode_tmap_halves(CUtensorMap *map, const void *base, uint64_t rows, uint32_t box_rows);
// A call's queries: boxes of 64 columns, the heads of a kv head, the tokens of a tile
// of 128 rows.
bool encode_tmap_queries(CUtensorMap *map, const PagedAttendParams &p);

}  // namespace vq
