// kv_api.cu -- the C ABI of the paged NVFP4 key/value cache
// (include/nvfp4_kv.h): argument checks, then launches on the caller's stream.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/nvfp4_kv.h"
#include "kernels.cuh"
#include "kv.cuh"

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 30;

// Whether the tcgen05 kernel takes an attention call: its tiles of 128 rows and
// its start of some microseconds an item want many rows a request, and enough of
// them in all.  Measured both ways on GB300 (rows kernel / tile kernel, us): 64
// requests of 4000 tokens, 8 kv heads of 128, 32 rows a request 184 / 233, 48 rows 336 /
// 230; 16 of 1000, 32 rows 30 / 36, 48 rows 45 / 36; 16 of 8000, 4 kv heads of 64, 32 rows
// 35 / 53, 64 rows 54 / 52; one of 30000, 8 kv heads of 128, 128 rows 80 / 90, 256 rows
// 142 / 91; one of 2000, 256 rows 30 / 36.  (The last lies on the rule's border and goes to
// the slower one: neither lengths nor windows enter the rule, and one answer holds for
// all requests of a call, so that single tokens beside a prompt go with the prompt.)
bool use_tile(int64_t reqs, int64_t heads, int64_t rows)
{
    return rows > 32 && reqs * heads * rows >= 2048;
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

// The bytes of a kv_tables operand: `rows` runs of `size` bytes, `stride` apart.
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
    if (nvfp4::device_status_address(&a.status) != cudaSuccess)
        return NVFP4_ERR_CUDA;
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
    const bool tile = kern == NVFP4_KERNEL_KV_TILE ||
                      (kern == NVFP4_KERNEL_AUTO && all_bf16 &&
                       use_tile(a.reqs, a.c.heads, (int64_t)a.max_q * a.group));
    const auto launch = tile ? nvfp4::launch_kv_tile : nvfp4::launch_kv_rows;
    return from_cuda(launch(a, workspace, (int64_t)workspace_bytes,
                            static_cast<cudaStream_t>(stream), (options & NVFP4_FLAG_PDL) != 0));
}

}  // extern "C"
