// gdn_kv_api.cu -- the C ABI's entries of the 8-bit paged cache, of its pages and of the draft
// check: host-side argument validation and launches.  No allocation, no
// synchronisation.
#include <algorithm>
#include <cmath>
#include <functional>

#include "gdn.h"
#include "gdn_host.cuh"
#include "gdn_internal.cuh"

using namespace gdn::host;

namespace {

constexpr int kMaxGroup = 64;       // query heads per kv head
constexpr int kMaxPages = 1 << 28;  // a pool whose lists of pages are counted in 31 bits
constexpr int kMaxCaches = 1024;    // layers that share a page table
constexpr int kMaxList = 1 << 30;   // entries of a list that kernels step through with 32-bit numbers
constexpr int kMaxVocab = 1 << 19;  // 2^19 weights of at most 2^43 stay below 2^63

// bytes from the first element of a strided [T][row] array of 16-bit values to its last
size_t span16(int32_t T, int64_t stride, size_t row) { return span(T, stride, row, 2); }

bool known_dim(const gdn_kv_cache* c) { return c->head_dim == 64 || c->head_dim == 128; }

bool known_page(int32_t tokens) { return tokens == 16 || tokens == 32 || tokens == 64 || tokens == 128; }

gdn_status check_cache(const gdn_kv_cache* c)
{
    if (!c) return fail(GDN_ERR_INVALID_ARG, "cache is NULL");
    if (c->heads < 1 || c->n_pages < 1) return fail(GDN_ERR_INVALID_ARG, "need heads >= 1 and n_pages >= 1 (heads=%d n_pages=%d)", c->heads, c->n_pages);
    if (c->heads > 1024) return fail(GDN_ERR_UNSUPPORTED, "heads=%d above 1024", c->heads);
    if (!known_dim(c)) return fail(GDN_ERR_UNSUPPORTED, "head_dim must be 64 or 128 (got %d)", c->head_dim);
    if (!known_page(c->page_tokens))
        return fail(GDN_ERR_UNSUPPORTED, "page_tokens must be 16, 32, 64 or 128 (got %d)", c->page_tokens);
    if (c->format != GDN_KV_INT8 && c->format != GDN_KV_E4M3) return fail(GDN_ERR_INVALID_ARG, "unknown cache format %d", c->format);
    const size_t codes = (size_t)c->n_pages * c->heads * c->page_tokens * c->head_dim, scales = (size_t)c->n_pages * c->heads * 4;
    const Buf bufs[] = {{c->k, codes, "cache k"}, {c->v, codes, "cache v"}, {c->k_scale, scales, "k_scale"}, {c->v_scale, scales, "v_scale"}};
    gdn_status st = check_bufs(bufs, 4);
    return st != GDN_OK ? st : check_disjoint(bufs, 4, nullptr, 0);
}

// the arguments that the append and the attention share
gdn_status check_kv_batch(const gdn_kv_cache* c, int32_t dtype, int32_t n_seq, int32_t T, const int32_t* cu, const int32_t* past,
                          const int32_t* table, int64_t table_stride, int32_t max_pages)
{
    gdn_status st;
    if ((st = check_cache(c)) != GDN_OK) return st;
    if (dtype != GDN_FP16 && dtype != GDN_BF16) return fail(GDN_ERR_INVALID_ARG, "unknown activation type %d", dtype);
    if ((st = check_batch(n_seq, T, cu)) != GDN_OK) return st;
    if (max_pages < 0 || table_stride < max_pages)
        return fail(GDN_ERR_INVALID_ARG, "need 0 <= max_pages <= page_table_stride (max_pages=%d stride=%lld)", max_pages, (long long)table_stride);
    // positions stay in 31 bits (the kernels clamp past to +-2^30)
    if ((int64_t)max_pages * c->page_tokens > (1 << 30)) return fail(GDN_ERR_UNSUPPORTED, "max_pages * page_tokens above 2^30");
    if (T > (1 << 29)) return fail(GDN_ERR_UNSUPPORTED, "total_tokens=%d above 2^29", T);
    if (n_seq > 0 && !past) return fail(GDN_ERR_INVALID_ARG, "past is NULL");
    if (n_seq > 0 && max_pages > 0 && !table) return fail(GDN_ERR_INVALID_ARG, "page_table is NULL");
    if (!aligned4(past) || !aligned4(table)) return fail(GDN_ERR_ALIGNMENT, "past or page_table not 4-byte aligned");
    return GDN_OK;
}

void fill(gdn::KvBatch& p, const gdn_kv_cache* c, int32_t dtype, int32_t n_seq, int32_t T, const int32_t* cu, const int32_t* past,
          const int32_t* table, int64_t table_stride, int32_t max_pages, int32_t hq, const uint16_t* q, int64_t q_stride)
{
    p.heads = c->heads; p.dim = c->head_dim; p.page = c->page_tokens; p.n_pages = c->n_pages; p.format = c->format;
    p.k = c->k; p.v = c->v; p.k_scale = c->k_scale; p.v_scale = c->v_scale;
    p.n_seq = n_seq; p.T = T; p.hq = hq; p.max_pages = max_pages;
    p.cu_seqlens = cu; p.past = past; p.table = table; p.table_stride = table_stride;
    p.q = q; p.q_stride = q_stride; p.bf16 = dtype == GDN_BF16;
}

}  // namespace

extern "C" {

gdn_status gdn_kv_append(const gdn_kv_cache* cache, int32_t dtype, int32_t n_seq, int32_t T, const int32_t* cu_seqlens,
                         const int32_t* past, const int32_t* page_table, int64_t page_table_stride, int32_t max_pages, int32_t hq,
                         const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                         const float* cos, const float* sin, int32_t rot_dim, int32_t n_pos, int32_t interleaved, uint16_t* q_out,
                         struct CUstream_st* stream)
{
    gdn_status st;
    if ((st = check_kv_batch(cache, dtype, n_seq, T, cu_seqlens, past, page_table, page_table_stride, max_pages)) != GDN_OK) return st;
    if (hq < 0) return fail(GDN_ERR_INVALID_ARG, "negative hq");
    if (hq > 65535) return fail(GDN_ERR_UNSUPPORTED, "hq=%d above 65535", hq);
    if (interleaved != 0 && interleaved != 1) return fail(GDN_ERR_INVALID_ARG, "interleaved must be 0 or 1");
    const size_t d = cache->head_dim, rowq = (size_t)hq * d, rowk = (size_t)cache->heads * d;
    if (rot_dim < 0 || rot_dim > cache->head_dim || rot_dim % 16) return fail(GDN_ERR_UNSUPPORTED, "rot_dim=%d must be a multiple of 16 up to head_dim", rot_dim);
    if (rot_dim > 0 && n_pos < 1) return fail(GDN_ERR_INVALID_ARG, "n_pos=%d: the rotation table is empty", n_pos);
    if (hq > 0 && (st = check_stride("q", q_stride, rowq, T)) != GDN_OK) return st;
    if ((st = check_stride("k", k_stride, rowk, T)) != GDN_OK) return st;
    if ((st = check_stride("v", v_stride, rowk, T)) != GDN_OK) return st;
    const size_t tt = (size_t)T, table_bytes = rot_dim > 0 && T > 0 ? (size_t)n_pos * (rot_dim / 2) * 4 : 0;
    const size_t codes = (size_t)cache->n_pages * rowk * cache->page_tokens, scales = (size_t)cache->n_pages * cache->heads * 4;
    const Buf ins[] = {{q, hq ? span16(T, q_stride, rowq) : 0, "q"}, {k, span16(T, k_stride, rowk), "k"}, {v, span16(T, v_stride, rowk), "v"},
                       {cos, table_bytes, "cos"}, {sin, table_bytes, "sin"}};
    const Buf outs[] = {{q_out, tt * rowq * 2, "q_out"}, {cache->k, codes, "cache k"}, {cache->v, codes, "cache v"},
                        {cache->k_scale, scales, "k_scale"}, {cache->v_scale, scales, "v_scale"}};
    if ((st = check_bufs(ins, 5)) != GDN_OK) return st;
    if ((st = check_bufs(outs, 1)) != GDN_OK) return st;
    if ((st = check_disjoint(outs, 5, ins, 5)) != GDN_OK) return st;
    if (T == 0) return GDN_OK;
    gdn::AppendParams p{};
    fill(p, cache, dtype, n_seq, T, cu_seqlens, past, page_table, page_table_stride, max_pages, hq, q, q_stride);
    p.k_new = k; p.v_new = v; p.k_stride = k_stride; p.v_stride = v_stride;
    p.cos = cos; p.sin = sin; p.rot = rot_dim; p.n_pos = n_pos; p.interleaved = interleaved; p.q_out = q_out;
    cudaError_t e = gdn::launch_kv_append(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_kv_append launch");
}

size_t gdn_kv_attn_workspace_bytes(const gdn_kv_cache* cache, int32_t n_seq, int32_t T, int32_t hq, int32_t max_pages)
{
    // shapes that gdn_kv_attn refuses have no layout
    if (!cache || cache->heads < 1 || !known_dim(cache) || !known_page(cache->page_tokens) || n_seq < 0 || T < 0) return 0;
    if (hq < cache->heads || hq % cache->heads || hq / cache->heads > kMaxGroup || max_pages < 0) return 0;
    gdn::KvBatch b{};
    fill(b, cache, GDN_FP16, n_seq, T, nullptr, nullptr, nullptr, 0, max_pages, hq, nullptr, 0);
    return gdn::kv_attn_workspace_bytes(b);
}

gdn_status gdn_kv_attn(const gdn_kv_cache* cache, int32_t dtype, int32_t n_seq, int32_t T, const int32_t* cu_seqlens,
                       const int32_t* past, const int32_t* page_table, int64_t page_table_stride, int32_t max_pages, int32_t hq,
                       const uint16_t* q, int64_t q_stride, float softmax_scale, uint16_t* y, void* workspace, size_t workspace_bytes,
                       struct CUstream_st* stream)
{
    gdn_status st;
    if ((st = check_kv_batch(cache, dtype, n_seq, T, cu_seqlens, past, page_table, page_table_stride, max_pages)) != GDN_OK) return st;
    if (hq < cache->heads || hq % cache->heads) return fail(GDN_ERR_INVALID_ARG, "hq=%d is not a multiple of heads=%d", hq, cache->heads);
    if (hq / cache->heads > kMaxGroup) return fail(GDN_ERR_UNSUPPORTED, "%d query heads per kv head, above %d", hq / cache->heads, kMaxGroup);
    if (hq > 65535) return fail(GDN_ERR_UNSUPPORTED, "hq=%d above 65535", hq);
    if (!std::isfinite(softmax_scale)) return fail(GDN_ERR_INVALID_ARG, "softmax_scale is not finite");
    const size_t row = (size_t)hq * cache->head_dim, tt = (size_t)T;
    if ((st = check_stride("q", q_stride, row, T)) != GDN_OK) return st;
    const size_t need = gdn_kv_attn_workspace_bytes(cache, n_seq, T, hq, max_pages);
    if (workspace_bytes < need || (need && !workspace)) return fail(GDN_ERR_WORKSPACE, "attention workspace %zu bytes, need %zu", workspace_bytes, need);
    const size_t codes = (size_t)cache->n_pages * cache->heads * cache->page_tokens * cache->head_dim;
    const size_t scales = (size_t)cache->n_pages * cache->heads * 4;
    const Buf ins[] = {{q, span16(T, q_stride, row), "q"}, {cache->k, codes, "cache k"}, {cache->v, codes, "cache v"},
                       {cache->k_scale, scales, "k_scale"}, {cache->v_scale, scales, "v_scale"}};
    const Buf outs[] = {{y, tt * row * 2, "y"}, {workspace, need, "workspace"}};
    if ((st = check_bufs(ins, 1)) != GDN_OK) return st;
    if ((st = check_bufs(outs, 2)) != GDN_OK) return st;
    if ((st = check_disjoint(outs, 2, ins, 5)) != GDN_OK) return st;
    if (T == 0) {  // nothing to compute; a failure record still starts clean
        cudaError_t e = workspace && workspace_bytes >= 4 ? cudaMemsetAsync(workspace, 0, 4, reinterpret_cast<cudaStream_t>(stream)) : cudaSuccess;
        return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_kv_attn workspace clear");
    }
    gdn::AttnParams p{};
    fill(p, cache, dtype, n_seq, T, cu_seqlens, past, page_table, page_table_stride, max_pages, hq, q, q_stride);
    p.scale = softmax_scale; p.y = y; p.workspace = workspace;
    cudaError_t e = gdn::launch_kv_attn(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_kv_attn launch");
}

gdn_status gdn_kv_attn_check(const void* workspace, struct CUstream_st* stream) { return read_failure_word(workspace, stream); }

namespace {

// lists of whole numbers: present and 4-byte aligned
gdn_status check_lists(const Buf* b, int n)
{
    for (int i = 0; i < n; ++i) {
        if (b[i].bytes == 0) continue;
        if (!b[i].p) return fail(GDN_ERR_INVALID_ARG, "%s is NULL", b[i].name);
        if (!aligned4(b[i].p)) return fail(GDN_ERR_ALIGNMENT, "%s is not 4-byte aligned", b[i].name);
    }
    return GDN_OK;
}

// a table's bytes, from its first entry to its last
size_t table_bytes(int32_t rows, int64_t stride, int32_t width) { return width > 0 ? span(rows, stride, width, 4) : 0; }

gdn_status check_table(const char* name, int32_t rows, int64_t stride, int32_t width)
{
    if (rows < 0) return fail(GDN_ERR_INVALID_ARG, "negative number of rows");
    if (stride < width) return fail(GDN_ERR_INVALID_ARG, "%s_stride=%lld is shorter than max_pages=%d", name, (long long)stride, width);
    if (stride > (1 << 30)) return fail(GDN_ERR_UNSUPPORTED, "%s_stride=%lld above 2^30", name, (long long)stride);
    if ((int64_t)rows * width > (1 << 30)) return fail(GDN_ERR_UNSUPPORTED, "more than 2^30 table entries");
    return GDN_OK;
}

gdn_status check_pool(int32_t n_pages, int32_t max_pages)
{
    if (n_pages < 1 || max_pages < 0) return fail(GDN_ERR_INVALID_ARG, "need n_pages >= 1 and max_pages >= 0 (n_pages=%d max_pages=%d)", n_pages, max_pages);
    if (n_pages > kMaxPages) return fail(GDN_ERR_UNSUPPORTED, "n_pages=%d above 2^28", n_pages);
    return GDN_OK;
}

size_t words(size_t n) { return align256(n * 4); }

}  // namespace

size_t gdn_kv_remap_workspace_bytes(int32_t n_pages, int32_t n_rows, int32_t max_pages)
{
    if (n_pages < 1 || n_pages > kMaxPages || n_rows < 0 || n_rows > kMaxList || max_pages < 0 || (int64_t)n_rows * max_pages > (1 << 30)) return 0;
    return words(1) + 2 * words(n_pages) + words(n_rows) + words(gdn::remap_sums(n_pages, n_rows));
}

gdn_status gdn_kv_remap(int32_t page_tokens, int32_t n_pages, int32_t max_pages, int32_t n_old, const int32_t* page_table,
                        int64_t page_table_stride, int32_t n_rows, const int32_t* parent, const int32_t* keep, const int32_t* need,
                        int32_t* table_out, int64_t table_out_stride, int32_t* copy_from, int32_t* copy_to, int32_t* info,
                        void* workspace, size_t workspace_bytes, struct CUstream_st* stream)
{
    gdn_status st;
    if (!known_page(page_tokens)) return fail(GDN_ERR_UNSUPPORTED, "page_tokens must be 16, 32, 64 or 128 (got %d)", page_tokens);
    if ((st = check_pool(n_pages, max_pages)) != GDN_OK) return st;
    if ((int64_t)max_pages * page_tokens > (1 << 30)) return fail(GDN_ERR_UNSUPPORTED, "max_pages * page_tokens above 2^30");
    if (n_rows > kMaxList) return fail(GDN_ERR_UNSUPPORTED, "n_rows=%d above 2^30", n_rows);
    if ((st = check_table("page_table", n_old, page_table_stride, max_pages)) != GDN_OK) return st;
    if ((st = check_table("table_out", n_rows, table_out_stride, max_pages)) != GDN_OK) return st;
    const size_t rows = (size_t)n_rows * 4, need_ws = gdn_kv_remap_workspace_bytes(n_pages, n_rows, max_pages);
    const Buf ins[] = {{page_table, table_bytes(n_old, page_table_stride, max_pages), "page_table"}, {parent, rows, "parent"},
                       {keep, rows, "keep"}, {need, rows, "need"}};
    const Buf outs[] = {{table_out, table_bytes(n_rows, table_out_stride, max_pages), "table_out"}, {copy_from, rows, "copy_from"},
                        {copy_to, rows, "copy_to"}, {info, 8, "info"}, {workspace, need_ws, "workspace"}};
    if ((st = check_lists(ins, 4)) != GDN_OK) return st;
    if ((st = check_lists(outs, 4)) != GDN_OK) return st;
    if (workspace_bytes < need_ws || !workspace) return fail(GDN_ERR_WORKSPACE, "remap workspace %zu bytes, need %zu", workspace_bytes, need_ws);
    if ((st = check_bufs(outs + 4, 1)) != GDN_OK) return st;
    if ((st = check_disjoint(outs, 5, ins, 4)) != GDN_OK) return st;
    gdn::RemapParams p{};
    p.n_old = n_old; p.n_rows = n_rows; p.max_pages = max_pages; p.n_pages = n_pages;
    for (p.page_shift = 4; (1 << p.page_shift) < page_tokens; ++p.page_shift) {}
    p.table = page_table; p.table_stride = page_table_stride; p.out_stride = table_out_stride;
    p.parent = parent; p.keep = keep; p.need = need; p.table_out = table_out;
    p.copy_from = copy_from; p.copy_to = copy_to; p.info = info;
    char* ws = static_cast<char*>(workspace);
    p.header = reinterpret_cast<int32_t*>(ws);
    p.owner = reinterpret_cast<int32_t*>(ws + words(1));
    p.free_list = reinterpret_cast<int32_t*>(ws + words(1) + words(n_pages));
    p.first = reinterpret_cast<int32_t*>(ws + words(1) + 2 * words(n_pages));
    p.sums = reinterpret_cast<int32_t*>(ws + words(1) + 2 * words(n_pages) + words(n_rows));
    cudaError_t e = gdn::launch_kv_remap(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_kv_remap launch");
}

size_t gdn_kv_compact_workspace_bytes(int32_t n_pages)
{
    return n_pages < 1 || n_pages > kMaxPages ? 0 : words(n_pages) + words(gdn::compact_sums(n_pages));
}

gdn_status gdn_kv_compact(int32_t n_pages, int32_t max_pages, int32_t n_rows, const int32_t* page_table, int64_t page_table_stride,
                          int32_t* table_out, int64_t table_out_stride, int32_t* copy_from, int32_t* copy_to, int32_t* info,
                          void* workspace, size_t workspace_bytes, struct CUstream_st* stream)
{
    gdn_status st;
    if ((st = check_pool(n_pages, max_pages)) != GDN_OK) return st;
    if ((st = check_table("page_table", n_rows, page_table_stride, max_pages)) != GDN_OK) return st;
    if ((st = check_table("table_out", n_rows, table_out_stride, max_pages)) != GDN_OK) return st;
    const size_t list = (size_t)(n_pages / 2) * 4, need_ws = gdn_kv_compact_workspace_bytes(n_pages);
    const Buf ins[] = {{page_table, table_bytes(n_rows, page_table_stride, max_pages), "page_table"}};
    const Buf outs[] = {{table_out, table_bytes(n_rows, table_out_stride, max_pages), "table_out"}, {copy_from, list, "copy_from"},
                        {copy_to, list, "copy_to"}, {info, 8, "info"}, {workspace, need_ws, "workspace"}};
    if ((st = check_lists(ins, 1)) != GDN_OK) return st;
    if ((st = check_lists(outs, 4)) != GDN_OK) return st;
    if (workspace_bytes < need_ws || !workspace) return fail(GDN_ERR_WORKSPACE, "compact workspace %zu bytes, need %zu", workspace_bytes, need_ws);
    if ((st = check_bufs(outs + 4, 1)) != GDN_OK) return st;
    // an entry is renamed by the thread that reads it
    const bool in_place = table_out == page_table && table_out_stride == page_table_stride;
    if ((st = check_disjoint(outs, 5, nullptr, 0)) != GDN_OK) return st;
    if ((st = check_disjoint(in_place ? outs + 1 : outs, in_place ? 4 : 5, ins, 1)) != GDN_OK) return st;
    gdn::CompactParams p{};
    p.n_rows = n_rows; p.max_pages = max_pages; p.n_pages = n_pages;
    p.table = page_table; p.table_stride = page_table_stride; p.out_stride = table_out_stride;
    p.table_out = table_out; p.copy_from = copy_from; p.copy_to = copy_to; p.info = info;
    p.name = static_cast<int32_t*>(workspace);
    p.sums = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + words(n_pages));
    cudaError_t e = gdn::launch_kv_compact(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_kv_compact launch");
}

gdn_status gdn_kv_copy(const gdn_kv_cache* caches, int32_t n_caches, int32_t n, const int32_t* copy_from, const int32_t* copy_to,
                       struct CUstream_st* stream)
{
    gdn_status st;
    if (n_caches < 0 || n < 0) return fail(GDN_ERR_INVALID_ARG, "negative n_caches or n");
    if (n_caches > kMaxCaches) return fail(GDN_ERR_UNSUPPORTED, "n_caches=%d above %d", n_caches, kMaxCaches);
    if (n > kMaxList) return fail(GDN_ERR_UNSUPPORTED, "n=%d above 2^30", n);
    if (n_caches > 0 && !caches) return fail(GDN_ERR_INVALID_ARG, "caches is NULL");
    const Buf lists[] = {{copy_from, (size_t)n * 4, "copy_from"}, {copy_to, (size_t)n * 4, "copy_to"}};
    if ((st = check_lists(lists, 2)) != GDN_OK) return st;
    Buf bufs[kMaxCaches * 4];
    for (int i = 0; i < n_caches; ++i) {
        const gdn_kv_cache &c = caches[i], &first = caches[0];
        if ((st = check_cache(&c)) != GDN_OK) return st;
        if (c.heads != first.heads || c.head_dim != first.head_dim || c.page_tokens != first.page_tokens || c.n_pages != first.n_pages ||
            c.format != first.format)
            return fail(GDN_ERR_INVALID_ARG, "cache %d has another shape or format than cache 0", i);
        const size_t codes = (size_t)c.n_pages * c.heads * c.page_tokens * c.head_dim, scales = (size_t)c.n_pages * c.heads * 4;
        const Buf b[] = {{c.k, codes, "cache k"}, {c.v, codes, "cache v"}, {c.k_scale, scales, "k_scale"}, {c.v_scale, scales, "v_scale"}};
        std::copy(b, b + 4, bufs + 4 * i);
    }
    for (int i = 0; i < n_caches * 4; ++i)
        for (const Buf& list : lists)
            if (overlap(bufs[i], list)) return fail(GDN_ERR_INVALID_ARG, "%s overlaps %s", list.name, bufs[i].name);
    // of buffers in the order of their addresses, if any two overlap then two neighbours do (all pairs of 1024 caches: 19 ms)
    std::sort(bufs, bufs + n_caches * 4, [](const Buf& a, const Buf& b) { return std::less<const void*>()(a.p, b.p); });
    for (int i = 0; i + 1 < n_caches * 4; ++i)
        if (overlap(bufs[i], bufs[i + 1])) return fail(GDN_ERR_INVALID_ARG, "%s overlaps %s", bufs[i].name, bufs[i + 1].name);
    if (n_caches == 0 || n == 0) return GDN_OK;
    gdn::CopyParams p{};
    p.n = n; p.n_pages = caches[0].n_pages; p.heads = caches[0].heads; p.from = copy_from; p.to = copy_to;
    p.page_bytes = (size_t)caches[0].heads * caches[0].page_tokens * caches[0].head_dim;
    for (int at = 0; at < n_caches; at += gdn::kCopyCaches) {
        p.n_caches = std::min(gdn::kCopyCaches, n_caches - at);
        for (int i = 0; i < p.n_caches; ++i) {
            const gdn_kv_cache& c = caches[at + i];
            p.cache[i] = {c.k, c.v, reinterpret_cast<uint32_t*>(c.k_scale), reinterpret_cast<uint32_t*>(c.v_scale)};
        }
        cudaError_t e = gdn::launch_kv_copy(p, reinterpret_cast<cudaStream_t>(stream));
        if (e != cudaSuccess) return cuda_fail(e, "gdn_kv_copy launch");
    }
    return GDN_OK;
}

gdn_status gdn_draft_verify(int32_t n_seq, int32_t max_draft, int32_t vocab, const float* p, int64_t p_stride, const float* q,
                            int64_t q_stride, const int32_t* draft, const int32_t* n_draft, const float* u, int32_t* accepted,
                            int32_t* next, struct CUstream_st* stream)
{
    if (n_seq < 0 || max_draft < 0) return fail(GDN_ERR_INVALID_ARG, "negative n_seq or max_draft");
    if (n_seq > 65535) return fail(GDN_ERR_UNSUPPORTED, "n_seq=%d above 65535", n_seq);
    if (vocab < 1) return fail(GDN_ERR_INVALID_ARG, "vocab=%d", vocab);
    if (vocab > kMaxVocab) return fail(GDN_ERR_UNSUPPORTED, "vocab=%d above %d", vocab, kMaxVocab);
    if (max_draft > 65535) return fail(GDN_ERR_UNSUPPORTED, "max_draft=%d above 65535", max_draft);
    if (p_stride < vocab || (max_draft > 0 && q_stride < vocab)) return fail(GDN_ERR_INVALID_ARG, "a row stride is shorter than vocab=%d", vocab);
    if (n_seq == 0) return GDN_OK;
    const size_t rows_p = (size_t)n_seq * (max_draft + 1), rows_q = (size_t)n_seq * max_draft;
    const Buf ins[] = {{p, ((rows_p - 1) * p_stride + vocab) * 4, "p"}, {q, rows_q ? ((rows_q - 1) * q_stride + vocab) * 4 : 0, "q"},
                       {draft, rows_q * 4, "draft"}, {u, rows_p * 4, "u"}, {n_draft, n_draft ? (size_t)n_seq * 4 : 0, "n_draft"}};
    const Buf outs[] = {{accepted, (size_t)n_seq * 4, "accepted"}, {next, (size_t)n_seq * 4, "next"}};
    for (const Buf& b : ins)
        if (b.bytes && !b.p) return fail(GDN_ERR_INVALID_ARG, "%s is NULL", b.name);
    for (const Buf& b : outs)
        if (!b.p) return fail(GDN_ERR_INVALID_ARG, "%s is NULL", b.name);
    for (const Buf& b : ins)
        if (b.bytes && !aligned4(b.p)) return fail(GDN_ERR_ALIGNMENT, "%s is not 4-byte aligned", b.name);
    for (const Buf& b : outs)
        if (!aligned4(b.p)) return fail(GDN_ERR_ALIGNMENT, "%s is not 4-byte aligned", b.name);
    gdn_status st = check_disjoint(outs, 2, ins, 5);
    if (st != GDN_OK) return st;
    gdn::VerifyParams vp{n_seq, max_draft, vocab, p, q, p_stride, q_stride, draft, n_draft, u, accepted, next};
    cudaError_t e = gdn::launch_verify(vp, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_draft_verify launch");
}

}  // extern "C"
