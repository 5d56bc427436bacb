// gdn_kv_api.cu -- the C ABI's entries of the 8-bit paged cache and of the draft
// check: host-side argument validation and launches.  No allocation, no
// synchronisation.
#include <cmath>

#include "gdn.h"
#include "gdn_host.cuh"
#include "gdn_internal.cuh"

using namespace gdn::host;

namespace {

constexpr int kMaxGroup = 64;       // query heads per kv head
constexpr int kMaxVocab = 1 << 19;  // 2^19 weights of at most 2^43 stay below 2^63

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// bytes from the first element of a strided [T][row] array of 16-bit values to its last
size_t span16(int32_t T, int64_t stride, size_t row) { return T > 0 ? ((size_t)(T - 1) * (size_t)stride + row) * 2 : 0; }

bool known_dim(const gdn_kv_cache* c) { return c->head_dim == 64 || c->head_dim == 128; }

bool known_page(const gdn_kv_cache* c)
{
    return c->page_tokens == 16 || c->page_tokens == 32 || c->page_tokens == 64 || c->page_tokens == 128;
}

gdn_status check_cache(const gdn_kv_cache* c)
{
    if (!c) return fail(GDN_ERR_INVALID_ARG, "cache is NULL");
    if (c->heads < 1 || c->n_pages < 1) return fail(GDN_ERR_INVALID_ARG, "need heads >= 1 and n_pages >= 1 (heads=%d n_pages=%d)", c->heads, c->n_pages);
    if (c->heads > 1024) return fail(GDN_ERR_UNSUPPORTED, "heads=%d above 1024", c->heads);
    if (!known_dim(c)) return fail(GDN_ERR_UNSUPPORTED, "head_dim must be 64 or 128 (got %d)", c->head_dim);
    if (!known_page(c))
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

gdn_status check_stride(const char* name, int64_t stride, size_t row)
{
    if (stride < (int64_t)row) return fail(GDN_ERR_INVALID_ARG, "%s_stride=%lld is shorter than a row of %zu", name, (long long)stride, row);
    if (stride % 8) return fail(GDN_ERR_ALIGNMENT, "%s_stride=%lld is not a multiple of 8", name, (long long)stride);
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
    if (hq > 0 && (st = check_stride("q", q_stride, rowq)) != GDN_OK) return st;
    if ((st = check_stride("k", k_stride, rowk)) != GDN_OK) return st;
    if ((st = check_stride("v", v_stride, rowk)) != GDN_OK) return st;
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
    if (!cache || cache->heads < 1 || !known_dim(cache) || !known_page(cache) || n_seq < 0 || T < 0) return 0;
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
    if ((st = check_stride("q", q_stride, row)) != GDN_OK) return st;
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
