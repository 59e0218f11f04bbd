// kv_api.cu -- the C ABI of the paged NVFP4 key/value cache
// (include/nvfp4_kv.h): argument checks, then launches on the caller's stream.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/nvfp4_kv.h"
#include "kernels.cuh"
#include "kv.cuh"
#include "launch_cache.cuh"

namespace {

using nvfp4::KvSees;

constexpr int64_t kMaxTokens = (int64_t)1 << 30;

int sm_count()
{
    return nvfp4::device_sm_count(nvfp4::current_device());
}

// Bytes of what one of two passes over `rows` rows leaves, but for KvParts::where; its sums begin
// on a sector's boundary.
int64_t pass_bytes(int64_t rows, int64_t dim)
{
    return ((rows + nvfp4::kv_part_total(sm_count())) * (dim * 4 + 8) + 31) / 32 * 32;
}

// Whether the tcgen05 kernel takes an attention call: its tiles of 128 rows and
// its start of some microseconds an item want many rows a request, and enough of
// them in all.  Measured both ways on GB300 (rows kernel / tile kernel, us): 64
// requests of 4000 tokens, 8 kv heads of 128, 32 rows a request 184 / 233, 48 rows 336 /
// 230; 16 of 1000, 32 rows 30 / 36, 48 rows 45 / 36; 16 of 8000, 4 kv heads of 64, 32 rows
// 35 / 53, 64 rows 54 / 52; one of 30000, 8 kv heads of 128, 128 rows 80 / 90, 256 rows
// 142 / 91; one of 2000, 256 rows 30 / 36.  (The last lies on the rule's border and goes to
// the slower one: neither lengths nor windows enter the rule, and one answer holds for
// all requests of a call, so that single tokens beside a prompt go with the prompt.)
// All keys (cross attention), requests x kv heads x rows on 100 / 1500 / 8000 states: of 128, 1 x 8 x 160 12 21
// 39 / 11 30 58; 4 x 8 x 48 11 25 49 / 10 30 54; 8 x 8 x 24 10 25 50 / 10 34 70; 8 x 8 x 36 11 32 84 / 10 34 69;
// 1 x 8 x 400 12 31 71 / 11 32 56; 32 x 8 x 36 35 83 295 / 16 60 204; of 64, 8 x 16 x 40 14 34 95 / 8 29 84; 64 x 4 x 40
// 27 56 189 / 13 43 153.
bool use_tile(int64_t reqs, int64_t heads, int64_t rows)
{
    return rows > 32 && reqs * heads * rows >= 2048;
}

// The same for a prefix that requests share: its parts are joined by another kernel, so that items
// cut between all SMs cost little.  `rows` is the average of the groups.  Measured both ways (rows kernel /
// tile kernel for the prefix, us a call; single tokens of 8 kv heads of 128, a prefix of 500 / 2000 / 8000 / 60000
// tokens).  One group of 16 rows 13.5 14 21 33 / 18 19 21 60, of 20 17 18 22 49 / 19 19 21 61, of 32 17 18 27 50 /
// 19 19 21 63, of 64 18 24 31 80 / 20 20 26 67; four of 16 rows 17 24 35 139 / 20 26 43 205, of 20 24 25 40 208 /
// 21 27 45 204, of 64 23 35 90 574 / 23 29 47 204; sixteen (up to 8000) of 16 rows 30 40 88 / 30 48 119, of 20 43 56
// 121 / 36 52 137, of 32 49 69 154 / 40 57 148, of 64 80 108 228 / 60 77 152.  4 kv heads of 64, one group: of 32
// rows 14 15 17 26 / 16 16 17 29, of 128 15 16 25 51 / 16 17 18 32.  264 rows of 4 kv heads (500, 4000, 30000) 28 34 91 /
// 24 27 48.  From 17 to 48 rows neither wins by much; the rows kernel's items grow from 16 to 32 rows there.  Uneven
// groups, 64 single tokens behind 8000 and 30 behind as many prefixes (13 rows on the average: the rows
// kernel): prefixes of 8000 154 / 202, of 500 89 / 63.
bool use_tile_for_prefix(int64_t rows)
{
    return rows > 16;
}

// The same for the keys behind a prefix, which the rows kernel takes beside the prefix's pass and
// leaves to the kernel that joins, while the tile kernel waits for the prefix and joins itself.
// Measured both ways (rows / tile for these keys, us a call; a prefix of 2000, 0 / 300 / 3000 tokens
// and the new ones behind it, by requests x kv heads x rows): 4 x 8 x 80 34 36 58 / 42 48 72; 4 x 8 x 160 46 50
// 77 / 45 57 76; 32 x 2 x 84 46 51 86 / 47 61 83; 32 x 4 x 48 37 43 69 / 33 50 67; 32 x 2 x 140 62 67 122 / 47 61 85;
// 32 x 8 x 80 100 115 258 / 72 92 168.
bool use_tile_behind(int64_t reqs, int64_t heads, int64_t rows)
{
    return rows > 32 && reqs * heads * rows >= 6144;
}

bool aligned(const void* p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

int from_cuda(cudaError_t e)
{
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

// log2 of a supported page size, or -1.
int page_shift(int64_t page_size)
{
    for (int s = 4; s <= 8; ++s)
        if (page_size == (int64_t)1 << s)
            return s;
    return -1;
}

// The bytes of an operand: `rows` runs of `size` bytes, `stride` apart.
struct Span {
    uintptr_t at;
    int64_t rows, stride, size;
    bool written;
};

template <typename T>
Span vec(const T* p, int64_t n, bool written)
{
    return {reinterpret_cast<uintptr_t>(p), 1, 0, n * (int64_t)sizeof(T), written};
}

// Whether a run of bytes meets any row of the other.
bool meets(const Span& run, const Span& rows)
{
    if (run.size == 0 || rows.size == 0 || rows.rows == 0)
        return false;
    const int64_t lo = (int64_t)(run.at - rows.at), hi = lo + run.size;
    if (hi <= 0 || rows.rows == 1)
        return hi > 0 && lo < rows.size;
    // the row that begins at or before lo, and the next
    const int64_t r = lo > 0 ? lo / rows.stride : 0;
    return (r < rows.rows && lo < r * rows.stride + rows.size) ||
           (r + 1 < rows.rows && hi > (r + 1) * rows.stride);
}

// Rows of `size` bytes of a tensor with token rows.
Span token_rows(const void* p, int64_t tokens, int64_t stride, int64_t elements, int item, bool written)
{
    return {reinterpret_cast<uintptr_t>(p), tokens, stride * item, elements * item, written};
}

// Whether two tensors with token rows share memory.  Rows of one stride (slices of one
// projection's rows) by their place in the stride, else by the ranges they lie in.
bool rows_meet(const Span& x, const Span& y)
{
    if (x.rows == 0 || y.rows == 0 || x.size == 0 || y.size == 0)
        return false;
    const uintptr_t x_end = x.at + (uintptr_t)((x.rows - 1) * x.stride + x.size);
    const uintptr_t y_end = y.at + (uintptr_t)((y.rows - 1) * y.stride + y.size);
    if (x_end <= y.at || y_end <= x.at)
        return false;
    if (x.rows == 1)
        return meets(x, y);
    if (y.rows == 1)
        return meets(y, x);
    if (x.stride != y.stride)
        return true;
    const int64_t d = (int64_t)(y.at - x.at) % x.stride;
    const int64_t place = d < 0 ? d + x.stride : d;  // of y's row in x's
    return place < x.size || place + y.size > x.stride;
}

int check_cache(const nvfp4_kv_cache* c, nvfp4::KvCache* out)
{
    if (c == nullptr)
        return NVFP4_ERR_INVALID_ARG;
    const int64_t bytes = nvfp4_kv_page_bytes(c->page_size, c->num_kv_heads, c->head_dim);
    if (bytes < 0)
        return (int)-bytes;
    if (c->num_pages < 0 || c->num_pages > INT32_MAX || c->page_stride < bytes ||
        (c->page_stride % 16) != 0)
        return NVFP4_ERR_INVALID_ARG;
    if (c->k_g == nullptr || c->v_g == nullptr || !aligned(c->k_g, 4) || !aligned(c->v_g, 4) ||
        (c->num_pages > 0 && c->pool == nullptr) || !aligned(c->pool, 16))
        return NVFP4_ERR_INVALID_ARG;
    *out = {static_cast<uint8_t*>(c->pool), c->k_g, c->v_g, c->num_pages, c->page_stride,
            page_shift(c->page_size), c->num_kv_heads, c->head_dim};
    return NVFP4_OK;
}

// The checks of an attention call, and its arguments as the kernels take them; `any`: there is
// something to do.
int check_attention(const nvfp4_kv_cache* cache, const nvfp4_kv_attention_args* args, uint32_t options,
                    const void* workspace, size_t workspace_bytes, nvfp4::KvAttnArgs* to, bool* any)
{
    nvfp4::KvAttnArgs& a = *to;
    *any = false;
    const int st = check_cache(cache, &a.c);
    if (st != NVFP4_OK)
        return st;
    if (args == nullptr || (options & ~(uint32_t)(NVFP4_KERNEL_MASK | NVFP4_FLAG_PDL |
                                                  NVFP4_FLAG_X_BF16 | NVFP4_FLAG_Y_BF16 |
                                                  NVFP4_FLAG_ALL_ROWS)) != 0)
        return NVFP4_ERR_INVALID_ARG;
    const nvfp4_kv_attention_args& r = *args;
    if (workspace == nullptr ? workspace_bytes != 0 : !aligned(workspace, 16))
        return NVFP4_ERR_INVALID_ARG;
    if (r.reqs < 0 || r.tokens < 0 || r.num_q_heads < 1 || (r.num_q_heads % a.c.heads) != 0 ||
        r.max_blocks < 0 || r.table_stride < r.max_blocks || r.max_q < 0 || r.window < 0 ||
        !(r.scale == r.scale) || (r.q_start == nullptr && r.reqs > 0 && (r.tokens % r.reqs) != 0))
        return NVFP4_ERR_INVALID_ARG;
    if (r.num_q_heads / a.c.heads > nvfp4::kKvMaxGroup || r.reqs > nvfp4::kKvMaxReqs ||
        r.tokens >= kMaxTokens / nvfp4::kKvMaxGroup ||
        r.max_blocks >= (kMaxTokens >> a.c.page_shift))
        return NVFP4_ERR_UNSUPPORTED;
    const uint32_t kern = options & NVFP4_KERNEL_MASK;
    const bool all_bf16 = (options & NVFP4_FLAG_X_BF16) && (options & NVFP4_FLAG_Y_BF16);
    if (kern != NVFP4_KERNEL_AUTO && kern != NVFP4_KERNEL_KV_ROWS &&
        !(kern == NVFP4_KERNEL_KV_TILE && all_bf16))
        return NVFP4_ERR_UNSUPPORTED;
    const bool all_rows = (options & NVFP4_FLAG_ALL_ROWS) != 0;
    if (r.tokens == 0 || (r.reqs == 0 && !all_rows))
        return NVFP4_OK;
    const bool q_bf16 = (options & NVFP4_FLAG_X_BF16) != 0;
    const bool out_bf16 = (options & NVFP4_FLAG_Y_BF16) != 0;
    const int64_t row = r.num_q_heads * a.c.dim;
    if (r.q == nullptr || r.out == nullptr || (r.reqs > 0 && r.seq_len == nullptr) ||
        (r.reqs > 0 && r.max_blocks > 0 && r.block_table == nullptr) || !aligned(r.q, q_bf16 ? 8 : 16) ||
        !aligned(r.out, out_bf16 ? 8 : 16) || !aligned(r.block_table, 4) ||
        !aligned(r.seq_len, 4) || !aligned(r.q_start, 4) || !aligned(r.lse, 4) ||
        (r.q_stride % 4) != 0 || (r.out_stride % 4) != 0 ||
        (r.tokens > 1 && (r.q_stride < row || r.out_stride < row)))
        return NVFP4_ERR_INVALID_ARG;
    a.q = r.q;
    a.q_stride = r.q_stride;
    a.table = r.block_table;
    a.table_stride = r.table_stride;
    a.max_blocks = (int32_t)r.max_blocks;
    a.seq_len = r.seq_len;
    a.q_start = r.q_start;
    a.q_per_req = (int32_t)(r.q_start || r.reqs == 0 ? 0 : r.tokens / r.reqs);
    a.reqs = (int32_t)r.reqs;
    a.tokens = (int32_t)r.tokens;
    a.max_q = (int32_t)(r.max_q < r.tokens ? r.max_q : r.tokens);
    a.group = (int32_t)(r.num_q_heads / a.c.heads);
    a.group_magic = (uint32_t)(((uint64_t)1 << 32) / (uint64_t)a.group + 1);
    a.scale_log2 = r.scale * 1.4426950408889634f;
    // a window past every length is none
    a.window = r.window >= kMaxTokens ? 0 : (int32_t)r.window;
    a.out = r.out;
    a.out_stride = r.out_stride;
    a.lse = r.lse;
    a.q_bf16 = q_bf16;
    a.out_bf16 = out_bf16;
    a.all_rows = all_rows;
    *any = true;
    return NVFP4_OK;
}

// Whether an attention call writes over what it, or another of its CTAs, reads.  In place is fine: a
// row's output is written once all CTAs that take a part of its keys have read the row, those of the
// prefix's pass, which takes all rows of a group, among them.
bool writes_over(const nvfp4::KvAttnArgs& a)
{
    const int64_t heads = (int64_t)a.c.heads * a.group, row = heads * a.c.dim;
    const Span q = token_rows(a.q, a.tokens, a.q_stride, row, a.q_bf16 ? 2 : 4, false);
    const Span out = token_rows(a.out, a.tokens, a.out_stride, row, a.out_bf16 ? 2 : 4, true);
    const Span pool = {reinterpret_cast<uintptr_t>(a.c.pool), a.c.num_pages, a.c.page_stride,
                       nvfp4_kv_page_bytes((int64_t)1 << a.c.page_shift, a.c.heads, a.c.dim), false};
    const Span lse = vec(a.lse, a.lse ? a.tokens * heads : 0, true);
    const bool in_place = a.out == a.q && a.out_bf16 == a.q_bf16 && (a.out_stride == a.q_stride || a.tokens == 1);
    return (!in_place && rows_meet(out, q)) || rows_meet(out, pool) || meets(lse, q) || meets(lse, out) ||
           meets(lse, pool);
}

template <KvSees S>
bool takes_tile(const nvfp4::KvAttnArgs& a, uint32_t options)
{
    const uint32_t kern = options & NVFP4_KERNEL_MASK;
    if (kern != NVFP4_KERNEL_AUTO || !a.q_bf16 || !a.out_bf16)
        return kern == NVFP4_KERNEL_KV_TILE;
    const int64_t rows = (int64_t)a.max_q * a.group;
    if (S == KvSees::kBehind)
        return use_tile_behind(a.reqs, a.c.heads, rows);
    return S == KvSees::kAll && a.keep.rows ? use_tile_for_prefix(rows) : use_tile(a.reqs, a.c.heads, rows);
}

template <KvSees S>
int launch_attention(nvfp4::KvAttnArgs& a, uint32_t options, void* workspace, size_t workspace_bytes,
                     void* stream)
{
    if (a.status == nullptr && nvfp4::device_status_address(&a.status) != cudaSuccess)
        return NVFP4_ERR_CUDA;
    const auto launch = takes_tile<S>(a, options) ? nvfp4::launch_kv_tile<S> : nvfp4::launch_kv_rows<S>;
    return from_cuda(launch(a, workspace, (int64_t)workspace_bytes, static_cast<cudaStream_t>(stream),
                            (options & NVFP4_FLAG_PDL) != 0));
}

}  // namespace

extern "C" {

int64_t nvfp4_kv_page_bytes(int64_t page_size, int64_t num_kv_heads, int64_t head_dim)
{
    if (page_size < 1 || num_kv_heads < 1 || num_kv_heads > 65536 || head_dim < 1)
        return -NVFP4_ERR_INVALID_ARG;
    const int shift = page_shift(page_size);
    if (shift < 0 || (head_dim != 64 && head_dim != 128))
        return -NVFP4_ERR_UNSUPPORTED;
    return num_kv_heads * nvfp4::kv_head_bytes(shift, (int)head_dim);
}

int nvfp4_kv_tables(const int32_t* kv_len, const int32_t* q_len, int64_t reqs, int64_t page_size,
                    const int32_t* free_pages, int64_t num_free, const int32_t* free_head,
                    int32_t* block_table, int64_t table_stride, int64_t max_blocks,
                    int32_t* seq_len, int32_t* q_start, int64_t* slots, int32_t* positions,
                    int64_t tokens, int32_t* free_next, uint32_t options, void* stream)
{
    if (reqs < 0 || tokens < 0 || num_free < 0 || max_blocks < 0 || table_stride < max_blocks ||
        page_size < 1 || (options & ~(uint32_t)NVFP4_FLAG_PDL) != 0)
        return NVFP4_ERR_INVALID_ARG;
    const int shift = page_shift(page_size);
    if (shift < 0 || reqs > nvfp4::kKvMaxReqs || tokens >= kMaxTokens ||
        max_blocks >= (kMaxTokens >> shift) || num_free > INT32_MAX)
        return NVFP4_ERR_UNSUPPORTED;
    if (free_head == nullptr || free_next == nullptr || free_head == free_next ||
        q_start == nullptr || (num_free > 0 && free_pages == nullptr) ||
        (reqs > 0 && (kv_len == nullptr || q_len == nullptr || seq_len == nullptr ||
                      (max_blocks > 0 && block_table == nullptr))) ||
        (tokens > 0 && (slots == nullptr || positions == nullptr)))
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned(kv_len, 4) || !aligned(q_len, 4) || !aligned(free_pages, 4) ||
        !aligned(free_head, 4) || !aligned(block_table, 4) || !aligned(seq_len, 4) ||
        !aligned(q_start, 4) || !aligned(slots, 8) || !aligned(positions, 4) ||
        !aligned(free_next, 4))
        return NVFP4_ERR_INVALID_ARG;
    // CTAs read the lengths and the free list while others write: nothing written may
    // share memory with another operand
    const Span table = {reinterpret_cast<uintptr_t>(block_table), max_blocks ? reqs : 0, 4 * table_stride,
                        4 * max_blocks, true};
    const Span v[] = {vec(kv_len, reqs, false),         vec(q_len, reqs, false),
                      vec(free_pages, num_free, false), vec(free_head, 1, false),
                      vec(seq_len, reqs, true),         vec(q_start, reqs + 1, true),
                      vec(slots, tokens, true),         vec(positions, tokens, true),
                      vec(free_next, 1, true)};
    for (const Span& x : v) {
        if (meets(x, table))
            return NVFP4_ERR_INVALID_ARG;
        for (const Span& y : v)
            if (x.written && &x != &y && meets(y, x))
                return NVFP4_ERR_INVALID_ARG;
    }
    unsigned* status = nullptr;
    const cudaError_t e = nvfp4::device_status_address(&status);
    if (e != cudaSuccess)
        return NVFP4_ERR_CUDA;
    const nvfp4::KvTablesArgs a = {kv_len, q_len, (int32_t)reqs, shift, free_pages, num_free,
                                   free_head, block_table, table_stride, (int32_t)max_blocks,
                                   seq_len, q_start, slots, positions, (int32_t)tokens, free_next,
                                   status};
    return from_cuda(nvfp4::launch_kv_tables(a, static_cast<cudaStream_t>(stream),
                                             (options & NVFP4_FLAG_PDL) != 0));
}

int nvfp4_kv_append(const nvfp4_kv_cache* cache, const void* k, int64_t k_stride, const void* v,
                    int64_t v_stride, int64_t tokens, const int64_t* slots, uint32_t options,
                    void* stream)
{
    nvfp4::KvAppendArgs a = {};
    const int st = check_cache(cache, &a.c);
    if (st != NVFP4_OK)
        return st;
    if (tokens < 0 || (options & ~(uint32_t)(NVFP4_FLAG_PDL | NVFP4_FLAG_X_BF16)) != 0)
        return NVFP4_ERR_INVALID_ARG;
    if (tokens >= kMaxTokens)
        return NVFP4_ERR_UNSUPPORTED;
    if (tokens == 0)
        return NVFP4_OK;
    const bool bf16 = (options & NVFP4_FLAG_X_BF16) != 0;
    const int64_t row = (int64_t)a.c.heads * a.c.dim;
    if (k == nullptr || v == nullptr || slots == nullptr || !aligned(k, bf16 ? 8 : 16) ||
        !aligned(v, bf16 ? 8 : 16) || !aligned(slots, 8) || (k_stride % 4) != 0 ||
        (v_stride % 4) != 0 || (tokens > 1 && (k_stride < row || v_stride < row)))
        return NVFP4_ERR_INVALID_ARG;
    if (nvfp4::device_status_address(&a.status) != cudaSuccess)
        return NVFP4_ERR_CUDA;
    a.k = k;
    a.v = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.slots = slots;
    a.tokens = tokens;
    return from_cuda(nvfp4::launch_kv_append(a, bf16, static_cast<cudaStream_t>(stream),
                                             (options & NVFP4_FLAG_PDL) != 0));
}

int nvfp4_kv_append_rotary(const nvfp4_kv_cache* cache, const nvfp4_kv_rotary_args* args,
                           uint32_t options, void* stream)
{
    nvfp4::KvRotaryArgs a = {};
    const int st = check_cache(cache, &a.c);
    if (st != NVFP4_OK)
        return st;
    if (args == nullptr || (options & ~(uint32_t)(NVFP4_FLAG_PDL | NVFP4_FLAG_X_BF16)) != 0)
        return NVFP4_ERR_INVALID_ARG;
    const nvfp4_kv_rotary_args& r = *args;
    if (r.tokens < 0 || r.num_q_heads < 0 || r.rotary_rows < 0 || r.rotary_dim < 1 ||
        r.rotary_dim > a.c.dim || r.rotary_stride < 0 || (r.interleaved & ~1) != 0)
        return NVFP4_ERR_INVALID_ARG;
    const int64_t pieces = (r.num_q_heads + a.c.heads) * (a.c.dim / 16);  // threads a token, at most
    if (r.tokens >= kMaxTokens || r.num_q_heads > 65536 || (r.rotary_dim % 32) != 0 ||
        r.rotary_rows > INT32_MAX || r.tokens * pieces >= ((int64_t)1 << 37))
        return NVFP4_ERR_UNSUPPORTED;
    if (r.tokens == 0)
        return NVFP4_OK;
    const bool bf16 = (options & NVFP4_FLAG_X_BF16) != 0, with_q = r.num_q_heads > 0;
    const uintptr_t to = bf16 ? 8 : 16;
    const int64_t row = (int64_t)a.c.heads * a.c.dim, q_row = r.num_q_heads * a.c.dim;
    if (r.k == nullptr || r.v == nullptr || r.slots == nullptr || r.positions == nullptr ||
        (r.rotary_rows > 0 && r.rotary == nullptr) || !aligned(r.k, to) || !aligned(r.v, to) ||
        !aligned(r.slots, 8) || !aligned(r.positions, 4) || !aligned(r.rotary, 16) ||
        (r.rotary_stride % 4) != 0 || (r.rotary_rows > 1 && r.rotary_stride < r.rotary_dim) ||
        (r.k_stride % 4) != 0 || (r.v_stride % 4) != 0 ||
        (r.tokens > 1 && (r.k_stride < row || r.v_stride < row)))
        return NVFP4_ERR_INVALID_ARG;
    if (with_q) {
        if (r.q == nullptr || r.q_out == nullptr || !aligned(r.q, to) || !aligned(r.q_out, to) ||
            (r.q_stride % 4) != 0 || (r.q_out_stride % 4) != 0 ||
            (r.tokens > 1 && (r.q_stride < q_row || r.q_out_stride < q_row)))
            return NVFP4_ERR_INVALID_ARG;
        // what other threads read meanwhile is not written over
        const int item = bf16 ? 2 : 4;
        const Span out = token_rows(r.q_out, r.tokens, r.q_out_stride, q_row, item, true);
        const bool in_place = r.q_out == r.q && (r.q_out_stride == r.q_stride || r.tokens == 1);
        const Span pool = {reinterpret_cast<uintptr_t>(a.c.pool), a.c.num_pages, a.c.page_stride,
                           nvfp4_kv_page_bytes(cache->page_size, a.c.heads, a.c.dim), true};
        if ((!in_place && rows_meet(out, token_rows(r.q, r.tokens, r.q_stride, q_row, item, false))) ||
            rows_meet(out, token_rows(r.k, r.tokens, r.k_stride, row, item, false)) ||
            rows_meet(out, token_rows(r.v, r.tokens, r.v_stride, row, item, false)) ||
            rows_meet(out, pool) || meets(vec(r.slots, r.tokens, false), out) ||
            meets(vec(r.positions, r.tokens, false), out) || meets(vec(a.c.k_g, 1, false), out) ||
            meets(vec(a.c.v_g, 1, false), out) ||
            rows_meet(out, token_rows(r.rotary, r.rotary_rows, r.rotary_stride, r.rotary_dim, 4, false)))
            return NVFP4_ERR_INVALID_ARG;
    }
    if (nvfp4::device_status_address(&a.status) != cudaSuccess)
        return NVFP4_ERR_CUDA;
    if (with_q) {
        a.q = r.q;
        a.q_out = r.q_out;
        a.q_stride = r.q_stride;
        a.q_out_stride = r.q_out_stride;
        a.q_heads = (int32_t)r.num_q_heads;
    }
    a.k = r.k;
    a.v = r.v;
    a.k_stride = r.k_stride;
    a.v_stride = r.v_stride;
    a.tokens = r.tokens;
    a.slots = r.slots;
    a.positions = r.positions;
    a.rotary = r.rotary;
    a.rotary_rows = r.rotary_rows;
    a.rotary_stride = r.rotary_stride;
    a.rot = r.rotary_dim;
    a.interleaved = r.interleaved;
    return from_cuda(nvfp4::launch_kv_rotary(a, bf16, static_cast<cudaStream_t>(stream),
                                             (options & NVFP4_FLAG_PDL) != 0));
}

int64_t nvfp4_kv_attention_workspace_size(int64_t head_dim)
{
    if (head_dim < 1)
        return -NVFP4_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128)
        return -NVFP4_ERR_UNSUPPORTED;
    const int64_t rows = nvfp4::kv_rows_workspace_bytes((int)head_dim);
    const int64_t tile = nvfp4::kv_tile_workspace_bytes((int)head_dim);
    return rows > tile ? rows : tile;
}

int nvfp4_kv_attention(const nvfp4_kv_cache* cache, const nvfp4_kv_attention_args* args,
                       uint32_t options, void* workspace, size_t workspace_bytes, void* stream)
{
    nvfp4::KvAttnArgs a = {};
    bool any;
    const int st = check_attention(cache, args, options, workspace, workspace_bytes, &a, &any);
    return st != NVFP4_OK || !any
               ? st
               : launch_attention<KvSees::kCausal>(a, options, workspace, workspace_bytes, stream);
}

int nvfp4_kv_cross_attention(const nvfp4_kv_cache* cache, const nvfp4_kv_attention_args* args,
                             uint32_t options, void* workspace, size_t workspace_bytes, void* stream)
{
    nvfp4::KvAttnArgs a = {};
    bool any;
    if (args != nullptr && args->window != 0)
        return NVFP4_ERR_INVALID_ARG;
    const int st = check_attention(cache, args, options, workspace, workspace_bytes, &a, &any);
    if (st == NVFP4_OK && any && writes_over(a))
        return NVFP4_ERR_INVALID_ARG;
    return st != NVFP4_OK || !any
               ? st
               : launch_attention<KvSees::kAll>(a, options, workspace, workspace_bytes, stream);
}

int64_t nvfp4_kv_shared_scratch_size(int64_t tokens, int64_t num_q_heads, int64_t head_dim)
{
    if (tokens < 0 || num_q_heads < 1 || head_dim < 1)
        return -NVFP4_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || tokens >= kMaxTokens || num_q_heads > (1 << 22) ||
        sm_count() > nvfp4::kKvMostSms)
        return -NVFP4_ERR_UNSUPPORTED;
    const int64_t rows = tokens * num_q_heads;
    return 2 * (pass_bytes(rows, head_dim) + rows * 4);
}

int nvfp4_kv_attention_shared(const nvfp4_kv_cache* cache, const nvfp4_kv_attention_args* args,
                              const nvfp4_kv_prefixes* prefixes, uint32_t options, void* workspace,
                              size_t workspace_bytes, void* stream)
{
    nvfp4::KvAttnArgs a = {};
    bool any;
    if (prefixes == nullptr || (args != nullptr && args->window != 0))
        return NVFP4_ERR_INVALID_ARG;
    const int st = check_attention(cache, args, options, workspace, workspace_bytes, &a, &any);
    if (st != NVFP4_OK)
        return st;
    const nvfp4_kv_prefixes& p = *prefixes;
    if (p.groups < 0 || p.max_blocks < 0 || p.table_stride < p.max_blocks ||
        (p.group_start == nullptr && p.groups > 1))
        return NVFP4_ERR_INVALID_ARG;
    if (p.groups > nvfp4::kKvMaxReqs || p.max_blocks >= (kMaxTokens >> a.c.page_shift) ||
        args->tokens * args->num_q_heads > INT32_MAX)
        return NVFP4_ERR_UNSUPPORTED;
    if (!any)
        return NVFP4_OK;
    if (writes_over(a))
        return NVFP4_ERR_INVALID_ARG;
    if (p.groups == 0 || a.reqs == 0)
        return launch_attention<KvSees::kCausal>(a, options, workspace, workspace_bytes, stream);
    const int64_t rows = (int64_t)a.tokens * args->num_q_heads;
    const int64_t scratch = nvfp4_kv_shared_scratch_size(a.tokens, args->num_q_heads, a.c.dim);
    if (scratch < 0)
        return (int)-scratch;
    if (p.prefix_len == nullptr || (p.max_blocks > 0 && p.block_table == nullptr) || p.scratch == nullptr ||
        !aligned(p.prefix_len, 4) || !aligned(p.block_table, 4) || !aligned(p.group_start, 4) ||
        !aligned(p.scratch, 32) || (int64_t)p.scratch_bytes < scratch)
        return NVFP4_ERR_INVALID_ARG;
    const int64_t parts = nvfp4::kv_part_total(sm_count());
    nvfp4::KvParts of[2];
    for (int i = 0; i < 2; ++i) {
        nvfp4::KvParts& x = of[i];
        uint8_t* at = static_cast<uint8_t*>(p.scratch) + i * pass_bytes(rows, a.c.dim);
        x.rows = reinterpret_cast<float*>(at);
        x.parts = x.rows + rows * a.c.dim;
        x.stats = reinterpret_cast<float2*>(x.parts + parts * a.c.dim);
        x.part_stats = x.stats + rows;
        x.total = parts;
        x.item_rows = 0;
        x.where = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(p.scratch) + 2 * pass_bytes(rows, a.c.dim)) +
                  i * rows;
    }
    a.groups = {p.group_start, p.prefix_len, (int32_t)p.groups, a.reqs, p.max_blocks << a.c.page_shift};
    nvfp4::KvAttnArgs g = a;
    g.table = p.block_table;
    g.table_stride = p.table_stride;
    g.max_blocks = (int32_t)p.max_blocks;
    g.seq_len = p.prefix_len;
    g.reqs = (int32_t)p.groups;
    // rows of a group, on the average
    g.max_q = (int32_t)((a.tokens + p.groups - 1) / p.groups);
    g.all_rows = 0;
    g.keep = of[0];
    const int first = launch_attention<KvSees::kAll>(g, options, workspace, workspace_bytes, stream);
    if (first != NVFP4_OK)
        return first;
    a.status = g.status;
    a.prefix = of[0];
    a.prefix.item_rows =
        takes_tile<KvSees::kAll>(g, options) ? nvfp4::kv_tile_item_rows() : nvfp4::kv_rows_item_rows(g);
    const bool joins = takes_tile<KvSees::kBehind>(a, options);
    if (!joins) {
        a.keep = of[1];
        a.keep.item_rows = nvfp4::kv_rows_item_rows(a);
    }
    const int second =
        launch_attention<KvSees::kBehind>(a, options | NVFP4_FLAG_PDL, workspace, workspace_bytes, stream);
    if (second != NVFP4_OK || joins)
        return second;
    return from_cuda(nvfp4::launch_kv_join(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
