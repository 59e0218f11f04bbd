/*
 * nvfp4_kv.h -- C ABI of the paged NVFP4 key/value cache: block tables and
 * slot maps built on the GPU, the quantising append (with the position rotation
 * on the way, where wanted), and attention over the cache (single tokens, a few
 * tokens a request, chunks and whole prompts; requests that share a prefix;
 * cross attention to an encoder's states).
 *
 * The cache holds keys and values in the library's NVFP4 (nvfp4.h): E2M1 codes
 * two per byte, one E4M3 scale per 16 consecutive elements of the head
 * dimension, one FP32 tensor scale for the keys (k_g) and one for the values
 * (v_g), both amax / 2688 of calibration data (nvfp4_global_scale).  Values
 * past a tensor scale's amax saturate.
 *
 * A pool of pages; page p holds page_size tokens of every kv head.  The bytes
 * of kv head h of page p start at p * page_stride + h * page_size * 9 D / 8:
 *     K codes   [page_size][D/2]      V codes   [page_size][D/2]
 *     K scales  [page_size][D/16]     V scales  [page_size][D/16]
 * (D = head_dim; element 2j of a row in the low nibble of byte j).  A token's
 * slot is page * page_size + its place in the page.
 *
 * Conventions are those of nvfp4.h: pointers are device memory of the current
 * device, work is queued on `stream`, nothing is allocated or synchronised,
 * host checks come before any launch, calls can be captured in CUDA graphs.
 * Descriptor structs are HOST memory, read during the call only.  Lengths,
 * tables and slots live on the device; what a kernel finds out of range there
 * (it never follows such an entry) sets NVFP4_DEVICE_KV_RANGE in the status
 * word (nvfp4_device_status).
 */
#ifndef NVFP4_KV_GB300_H
#define NVFP4_KV_GB300_H

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Status bit: a page id, slot or length out of range, a block table too short
 * for a request, or a free list that ran out. */
#define NVFP4_DEVICE_KV_RANGE 2u

typedef struct {
    void* pool;          /* num_pages pages, 16-byte aligned */
    const float* k_g;    /* [1] tensor scale of the keys */
    const float* v_g;    /* [1] tensor scale of the values */
    int64_t num_pages;   /* pages in the pool, at most 2^31 - 1 */
    int64_t page_stride; /* bytes from page to page: at least
                            nvfp4_kv_page_bytes(), a multiple of 16 */
    int32_t page_size;   /* tokens a page: 16, 32, 64, 128 or 256 */
    int32_t num_kv_heads;
    int32_t head_dim;    /* 64 or 128 */
} nvfp4_kv_cache;

/* Bytes of one page (num_kv_heads * page_size * 9 head_dim / 8), or minus a
 * status code.  Host only. */
int64_t nvfp4_kv_page_bytes(int64_t page_size, int64_t num_kv_heads, int64_t head_dim);

/*
 * Block tables and slot maps of one step.  Request r holds kv_len[r] tokens
 * and gets q_len[r] new ones.  With P = page_size:
 *     seq_len[r] = kv_len[r] + q_len[r]
 *     q_start    = exclusive prefix sum of q_len (reqs + 1 entries)
 *     new pages of r: ceil(seq_len[r] / P) - ceil(kv_len[r] / P), taken from
 *     free_pages in request order from index *free_head on and entered into
 *     block_table[r][ceil(kv_len[r] / P) ...]; the other entries stay
 *     *free_next = *free_head + all new pages
 * and for row t of the step's tokens (token i = t - q_start[r] of request r):
 *     positions[t] = kv_len[r] + i
 *     slots[t]     = block_table[r][positions[t] / P] * P + positions[t] % P
 * Rows from q_start[reqs] up to `tokens` (padding of a fixed-size batch) get
 * slot -1 and position 0.  The call changes nothing it reads but the new
 * table entries, so repeating it gives the same result.
 *   kv_len, q_len   int32 [reqs] (negative lengths count as 0)
 *   free_pages      int32 [num_free] page ids
 *   free_head       int32 [1], in;  free_next  int32 [1], out, not the same
 *   block_table     int32 [reqs][table_stride], max_blocks entries of a row used
 *   seq_len [reqs], q_start [reqs + 1], positions [tokens]  int32, out
 *   slots           int64 [tokens], out
 * A page past the end of the free list is entered as -1 and its tokens get
 * slot -1; tokens past max_blocks * P get slot -1, take no page, and seq_len
 * stops there; both set NVFP4_DEVICE_KV_RANGE, and so do more new tokens than `tokens`.
 * What is written (the outputs, the table) shares no memory with another operand
 * (NVFP4_ERR_INVALID_ARG): lengths are not updated in place.
 * Lengths may be any int32: positions, q_start and *free_next past 2^31 - 1 are
 * stored as 2^31 - 1.  reqs at most 16384
 * (NVFP4_ERR_UNSUPPORTED), tokens and max_blocks * P below 2^30.  options:
 * NVFP4_FLAG_PDL.  One kernel.
 */
int nvfp4_kv_tables(const int32_t* kv_len, const int32_t* q_len, int64_t reqs, int64_t page_size,
                    const int32_t* free_pages, int64_t num_free, const int32_t* free_head,
                    int32_t* block_table, int64_t table_stride, int64_t max_blocks,
                    int32_t* seq_len, int32_t* q_start, int64_t* slots, int32_t* positions,
                    int64_t tokens, int32_t* free_next, uint32_t options, void* stream);

/*
 * Quantise new keys and values into the cache: token t's heads go to slot
 * slots[t], by the block recipe of nvfp4.h with *k_g and *v_g (every byte has
 * one right value; k and v are finite, as there).  Slot -1 is skipped (padding); slots outside the pool are
 * skipped and set NVFP4_DEVICE_KV_RANGE.  No two tokens may have the same slot.
 *   k, v      [tokens][num_kv_heads][head_dim], FP32 (16-byte aligned), or
 *             BF16 with NVFP4_FLAG_X_BF16 (8-byte aligned); k_stride and
 *             v_stride elements from token to token (a multiple of 4): slices
 *             of a fused projection's rows need no copy
 *   slots     int64 [tokens]
 * options: NVFP4_FLAG_X_BF16, NVFP4_FLAG_PDL.  One kernel.
 */
int nvfp4_kv_append(const nvfp4_kv_cache* cache, const void* k, int64_t k_stride, const void* v,
                    int64_t v_stride, int64_t tokens, const int64_t* slots, uint32_t options,
                    void* stream);

/*
 * The append with the position rotation on the way: keys and queries are turned
 * by their token's angles, then keys and values quantised into the cache as by
 * nvfp4_kv_append and the queries written out.
 *
 * The first rotary_dim elements of a head are pairs (a, b), at i and i +
 * rotary_dim / 2 (interleaved: at 2 i and 2 i + 1), i < rotary_dim / 2.  With
 * (c, s) = (row[i], row[rotary_dim / 2 + i]) of the row positions[t] of `rotary`:
 *     a' = a c - b s,   b' = b c + a s
 * in FP32, each product and the difference or sum rounded by itself: every bit of a'
 * and b' has one right value, and so has every byte of the cache (the keys are not
 * rounded in between; k, v and the angles are finite).  Queries are rounded once, to
 * their own type.  The rest of a head, and the values, are not turned.
 * Rows with slot -1 are not appended (padding).  Rows with a position outside
 * [0, rotary_rows) are not appended either, their queries are zeros, and unless their slot is
 * -1 they set NVFP4_DEVICE_KV_RANGE; so do slots outside the pool, as in nvfp4_kv_append.
 * No two tokens may have the same slot.
 */
typedef struct {
    const void* q;            /* [tokens][num_q_heads][head_dim], the type and alignment of k */
    int64_t q_stride;         /* elements from token to token, a multiple of 4, here and below */
    int64_t num_q_heads;      /* 0: no queries (q and q_out are then not used); any number up to
                                 65536, not only multiples of the kv heads */
    void* q_out;              /* like q; q itself (the same address and stride) turns it in place,
                                 any other overlap with q, k, v or the rest is refused */
    int64_t q_out_stride;
    const void* k;            /* k, v as in nvfp4_kv_append */
    int64_t k_stride;
    const void* v;
    int64_t v_stride;
    int64_t tokens;
    const int64_t* slots;     /* int64 [tokens] */
    const int32_t* positions; /* int32 [tokens] */
    const float* rotary;      /* FP32 [rotary_rows][rotary_dim], 16-byte aligned */
    int64_t rotary_rows;
    int64_t rotary_stride;    /* elements from row to row, a multiple of 4 */
    int32_t rotary_dim;       /* a multiple of 32 (else NVFP4_ERR_UNSUPPORTED), at most head_dim */
    int32_t interleaved;      /* 0 or 1 */
} nvfp4_kv_rotary_args;

/* options: NVFP4_FLAG_X_BF16 (q, k, v and q_out), NVFP4_FLAG_PDL.  One kernel. */
int nvfp4_kv_append_rotary(const nvfp4_kv_cache* cache, const nvfp4_kv_rotary_args* args,
                           uint32_t options, void* stream);

/*
 * Attention of the step's queries over the cache.  Query row t belongs to
 * request r with q_start[r] <= t < q_start[r + 1] and has position
 * p = seq_len[r] - (q_start[r + 1] - t); it sees the keys j of its request
 * with 0 <= j <= p and, with a window W > 0, j > p - W.  For query head h,
 * reading kv head h / (num_q_heads / num_kv_heads):
 *     s_j = scale * q . K_j,  out = sum_j softmax(s)_j V_j,
 *     lse = ln sum_j exp(s_j)
 * A row that sees no key (an empty request, positions below 0) gets zeros and
 * lse = -inf.  Whatever the cache holds past a request's end, or before the first key that
 * a request's rows see, does not matter, nor do table entries of pages that lie there
 * wholly: pages that a window has left can be given to others.
 * Keys and values on a page that is not in the pool count as zeros
 * (NVFP4_DEVICE_KV_RANGE is set).
 * Scores, softmax statistics and sums are FP32; the cached values enter
 * exactly, FP32 queries and (for FP32 outputs) probabilities as two f16 terms
 * each, else probabilities as one f16.
 */
typedef struct {
    const void* q;              /* [tokens][num_q_heads][head_dim], FP32 (16-byte aligned) or
                                   BF16 (NVFP4_FLAG_X_BF16, 8-byte aligned) */
    int64_t q_stride;           /* elements from token to token, a multiple of 4 */
    int64_t num_q_heads;        /* a multiple of num_kv_heads */
    const int32_t* block_table; /* int32 [reqs][table_stride] */
    int64_t table_stride;
    int64_t max_blocks;         /* entries of a table row that may be used */
    const int32_t* seq_len;     /* int32 [reqs]: tokens in the cache, the new ones included */
    const int32_t* q_start;     /* int32 [reqs + 1], or NULL: tokens / reqs rows each */
    int64_t reqs;
    int64_t tokens;             /* query rows */
    int64_t max_q;              /* the most rows a request has (a hint for the
                                   choice of kernel: any value gives right results) */
    float scale;
    int64_t window;             /* 0: none */
    void* out;                  /* [tokens][num_q_heads][head_dim], FP32 or BF16
                                   (NVFP4_FLAG_Y_BF16), aligned like q */
    int64_t out_stride;         /* elements from token to token, a multiple of 4 */
    float* lse;                 /* FP32 [tokens][num_q_heads], or NULL */
} nvfp4_kv_attention_args;

/*
 * options: a kernel choice in the low byte --
 *   NVFP4_KERNEL_AUTO          the library's choice
 *   NVFP4_KERNEL_KV_ROWS       query rows as the narrow side of mma.sync tiles:
 *                              few rows a request; any dtype
 *   NVFP4_KERNEL_KV_TILE       tcgen05 tiles of 128 query rows: many rows a
 *                              request; BF16 queries and outputs only
 *                              (NVFP4_ERR_UNSUPPORTED otherwise)
 * -- OR-ed with NVFP4_FLAG_X_BF16, NVFP4_FLAG_Y_BF16, NVFP4_FLAG_PDL,
 * NVFP4_FLAG_ALL_ROWS.  Rows of no request (before q_start[0], from q_start[reqs]
 * on: the padding of a fixed-size batch; every row when reqs is 0) are left as
 * they are, or with NVFP4_FLAG_ALL_ROWS get zeros and lse = -inf.
 * The keys of all requests are one list of work that the SMs share equally:
 * a request cut between SMs is joined through the workspace in a fixed order
 * (results do not depend on timing).
 *   workspace  caller-owned, 16-byte aligned, its first
 *              NVFP4_KV_WORKSPACE_ZERO bytes ZERO before its first use (the rest
 *              is written before it is read); every completed call leaves them so,
 *              and it may serve any number of calls that do not overlap in time.
 *              With less than
 *              nvfp4_kv_attention_workspace_size() bytes (NULL with 0) no
 *              request is cut.
 * reqs at most 16384, num_q_heads / num_kv_heads at most 64, tokens below 2^24,
 * max_blocks * page_size below 2^30 (else NVFP4_ERR_UNSUPPORTED).  One kernel.
 */
#define NVFP4_KERNEL_KV_ROWS 1u
#define NVFP4_KERNEL_KV_TILE 2u
#define NVFP4_FLAG_ALL_ROWS 0x20000u
#define NVFP4_KV_WORKSPACE_ZERO 4096

int nvfp4_kv_attention(const nvfp4_kv_cache* cache, const nvfp4_kv_attention_args* args,
                       uint32_t options, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of nvfp4_kv_attention on the current device for this
 * head_dim (any shape), or minus a status code.  Host only. */
int64_t nvfp4_kv_attention_workspace_size(int64_t head_dim);

/*
 * Cross attention: every query row of request r sees all seq_len[r] tokens that the
 * cache holds for it (the states of an encoder, say), however many rows it has; with
 * seq_len[r] = 0 they get zeros and lse = -inf.  All else, the workspace too, as for
 * nvfp4_kv_attention; args->window is 0 (else NVFP4_ERR_INVALID_ARG).  out may be q itself (the
 * same address, type and stride); any other overlap of out or lse with q, the pool or each other
 * is refused.  One kernel.
 */
int nvfp4_kv_cross_attention(const nvfp4_kv_cache* cache, const nvfp4_kv_attention_args* args,
                             uint32_t options, void* workspace, size_t workspace_bytes,
                             void* stream);

/*
 * Causal attention of requests that share prefixes, each prefix read not for every request
 * but once a kv head for 256 rows (tokens times query heads of the kv head) of its requests on the
 * tcgen05 kernel, for 8, 16 or 32 of them on the rows kernel, which takes FP32 always and short groups:
 * the library chooses by the average rows of a group.  For few requests or a short prefix
 * nvfp4_kv_attention with tables that spell the prefix out is faster (single tokens, 32 query heads of 128
 * on 8 kv heads in BF16: 2 requests up to 8000 tokens, 8 up to 4000, 16 up to 2000, 64 up to 250; 14 query
 * heads of 64 on 2 in FP32: 8 requests up to 30000, 64 up to 8000).  Group g is the requests group_start[g] up to
 * group_start[g + 1]; their first prefix_len[g] tokens are the same and lie on the pages of
 * row g of the prefixes' table.  Lengths and positions count them: in args, seq_len[r] is the
 * whole length, and entry b of a request's own row of args->block_table holds the tokens
 * b * page_size and on.  Query rows see what they see in nvfp4_kv_attention, with key j of
 * request r read
 *     on the prefix's pages for j < prefix_len[g], on the request's own pages from there on
 * if all rows of r lie behind the prefix (seq_len[r] - rows >= prefix_len[g]); entries of
 * its own pages wholly before prefix_len[g] are not looked up then.  A request with a row
 * inside the prefix (an empty one, too) shares nothing: all of its keys are read on its own
 * pages, as by nvfp4_kv_attention.  Requests of no group share nothing.  A prefix need not
 * end with a page (the rest of its last page is a request's own page then), and may be
 * empty (0 or less).
 * args->window is 0 (else NVFP4_ERR_INVALID_ARG), tokens * num_q_heads below 2^31 (else
 * NVFP4_ERR_UNSUPPORTED); out as for nvfp4_kv_cross_attention.  Options, workspace, statuses and what
 * is done about bad entries as for nvfp4_kv_attention, for both tables; the kernel choice of the options is that
 * of both passes.
 */
typedef struct {
    const int32_t* block_table; /* int32 [groups][table_stride] */
    int64_t table_stride;
    int64_t max_blocks;         /* entries of a row that may be used */
    const int32_t* prefix_len;  /* int32 [groups] */
    const int32_t* group_start; /* int32 [groups + 1], ascending, or NULL: one group of all
                                   requests (groups is 1 then) */
    int64_t groups;             /* at most 16384; 0: nothing is shared */
    void* scratch;              /* nvfp4_kv_shared_scratch_size() bytes, 32-byte aligned, any contents,
                                   not used by another call at the same time */
    size_t scratch_bytes;
} nvfp4_kv_prefixes;

/* Two kernels, the prefixes and the requests' own keys, which join the two; with few rows a
 * request three: the own keys are taken beside the prefixes, and a third kernel joins. */
int nvfp4_kv_attention_shared(const nvfp4_kv_cache* cache, const nvfp4_kv_attention_args* args,
                              const nvfp4_kv_prefixes* prefixes, uint32_t options,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of nvfp4_kv_prefixes.scratch on the current device, or minus a status code (devices of
 * more than 256 SMs: NVFP4_ERR_UNSUPPORTED).  Host only. */
int64_t nvfp4_kv_shared_scratch_size(int64_t tokens, int64_t num_q_heads, int64_t head_dim);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_KV_GB300_H */
