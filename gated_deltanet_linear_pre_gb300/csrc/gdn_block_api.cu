// gdn_block_api.cu -- the C ABI's entries of what lies around the layers: host-side
// argument validation and launches.  No allocation, no synchronisation.
#include <cmath>

#include "gdn.h"
#include "gdn_host.cuh"
#include "gdn_internal.cuh"

using namespace gdn::host;

namespace {

bool known_rank(int32_t rank) { return rank >= 8 && rank <= 128 && rank % 8 == 0; }
bool known_width(int32_t d) { return d >= 8 && d <= 65536 && d % 8 == 0; }

// rows that stand no further apart than these entries take them
gdn_status check_near(const char* name, int64_t stride, size_t row, int32_t T)
{
    const gdn_status st = check_stride(name, stride, row, T);
    if (st == GDN_OK && stride > (1 << 30)) return fail(GDN_ERR_UNSUPPORTED, "%s_stride=%lld above 2^30", name, (long long)stride);
    return st;
}

}  // namespace

extern "C" {

gdn_status gdn_block_norm(int32_t x_dtype, int32_t dtype, int32_t T, int32_t width, const void* x, int64_t x_stride,
                          const uint16_t* y, int64_t y_stride, const uint16_t* gate, int64_t gate_stride, int32_t gate_kind,
                          float scale, const float* post_weight, const float* pre_weight, float eps, void* x_out, uint16_t* h,
                          struct CUstream_st* stream)
{
    if (dtype != GDN_FP16 && dtype != GDN_BF16) return fail(GDN_ERR_INVALID_ARG, "unknown activation type %d", dtype);
    if (x_dtype != dtype && x_dtype != GDN_FP32) return fail(GDN_ERR_INVALID_ARG, "x_dtype=%d is neither dtype=%d nor GDN_FP32", x_dtype, dtype);
    if (T < 0 || width < 1) return fail(GDN_ERR_INVALID_ARG, "total_tokens=%d width=%d", T, width);
    if (width % 8 || width > 16384) return fail(GDN_ERR_UNSUPPORTED, "width=%d must be a multiple of 8 up to 16384", width);
    if (gate_kind < GDN_GATE_NONE || gate_kind > GDN_GATE_SILU) return fail(GDN_ERR_INVALID_ARG, "unknown gate_kind %d", gate_kind);
    if (!std::isfinite(scale)) return fail(GDN_ERR_INVALID_ARG, "scale is not finite");
    if (!(eps > 0.0f) || !std::isfinite(eps)) return fail(GDN_ERR_INVALID_ARG, "eps must be above 0");
    if (T == 0) return GDN_OK;  // empty arrays may be NULL
    if (!x_out && !h) return fail(GDN_ERR_INVALID_ARG, "neither x_out nor h is wanted");
    if (!h != !pre_weight) return fail(GDN_ERR_INVALID_ARG, "h and pre_weight come together");
    if (!gate != (gate_kind == GDN_GATE_NONE)) return fail(GDN_ERR_INVALID_ARG, "gate and gate_kind=%d do not go together", gate_kind);
    if (!y && (gate || post_weight || x_out)) return fail(GDN_ERR_INVALID_ARG, "without y there is no gate, post_weight or x_out");
    gdn_status st;
    if ((st = check_near("x", x_stride, width, T)) != GDN_OK) return st;
    if (y && (st = check_near("y", y_stride, width, T)) != GDN_OK) return st;
    if (gate && gate_stride != 0 && (st = check_near("gate", gate_stride, width, T)) != GDN_OK) return st;
    const size_t row = (size_t)width, x_bytes = x_dtype == GDN_FP32 ? 4 : 2, weight = row * 4;
    const Buf ins[] = {{x, span(T, x_stride, row, x_bytes), "x"}, {y, y ? span(T, y_stride, row, 2) : 0, "y"},
                       {gate, gate ? span(T, gate_stride, row, 2) : 0, "gate"}, {post_weight, post_weight ? weight : 0, "post_weight"},
                       {pre_weight, pre_weight ? weight : 0, "pre_weight"}};
    const Buf outs[] = {{h, h ? span(T, width, row, 2) : 0, "h"}, {x_out, x_out ? span(T, width, row, x_bytes) : 0, "x_out"}};
    if ((st = check_bufs(ins, 5)) != GDN_OK) return st;
    if ((st = check_bufs(outs, 2)) != GDN_OK) return st;
    // x_out may be x itself: each thread has read what it writes
    const bool in_place = x_out == x && x_stride == width;
    if ((st = check_disjoint(outs, 2, in_place ? ins + 1 : ins, in_place ? 4 : 5)) != GDN_OK) return st;
    if (in_place && overlap(outs[0], ins[0])) return fail(GDN_ERR_INVALID_ARG, "h overlaps x");
    gdn::BlockNormParams p{};
    p.T = T; p.width = width; p.x32 = x_dtype == GDN_FP32; p.bf16 = dtype == GDN_BF16;
    p.x = x; p.x_stride = x_stride; p.y = y; p.y_stride = y_stride;
    p.gate = gate; p.gate_stride = gate_stride; p.gate_kind = gate_kind; p.scale = scale; p.eps = eps;
    p.post_weight = post_weight; p.pre_weight = pre_weight; p.x_out = x_out; p.h = h;
    cudaError_t e = gdn::launch_block_norm(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_block_norm launch");
}

size_t gdn_adapter_workspace_bytes(int32_t n_seq, int32_t T, int32_t rank, int32_t d_in)
{
    if (n_seq < 0 || n_seq > 65535 || T < 0 || (n_seq == 0 && T > 0) || !known_rank(rank) || !known_width(d_in)) return 0;
    if (T == 0) return 0;
    gdn::AdapterParams p{};
    p.n_seq = n_seq; p.T = T; p.rank = rank;
    return gdn::adapter_workspace(p, nullptr);
}

gdn_status gdn_adapter_add(int32_t dtype, int32_t n_seq, int32_t T, const int32_t* cu_seqlens, const int32_t* ids, int32_t n_adapters,
                           int32_t rank, const int32_t* ranks, const uint16_t* down, const uint16_t* up, const float* scales, int32_t d_in,
                           const uint16_t* x, int64_t x_stride, int32_t d_out, const uint16_t* y, int64_t y_stride, uint16_t* y_out,
                           int64_t y_out_stride, void* workspace, size_t workspace_bytes, struct CUstream_st* stream)
{
    gdn_status st;
    if (dtype != GDN_FP16 && dtype != GDN_BF16) return fail(GDN_ERR_INVALID_ARG, "unknown activation type %d", dtype);
    if ((st = check_batch(n_seq, T, cu_seqlens)) != GDN_OK) return st;
    if (n_adapters < 0) return fail(GDN_ERR_INVALID_ARG, "negative n_adapters");
    if (n_adapters > (1 << 20)) return fail(GDN_ERR_UNSUPPORTED, "n_adapters=%d above 2^20", n_adapters);
    if (!known_rank(rank)) return fail(GDN_ERR_UNSUPPORTED, "rank=%d must be a multiple of 8 up to 128", rank);
    if (!known_width(d_in) || !known_width(d_out)) return fail(GDN_ERR_UNSUPPORTED, "d_in=%d and d_out=%d must be multiples of 8 up to 65536", d_in, d_out);
    if ((st = check_near("x", x_stride, d_in, T)) != GDN_OK) return st;
    if ((st = check_near("y", y_stride, d_out, T)) != GDN_OK) return st;
    if ((st = check_near("y_out", y_out_stride, d_out, T)) != GDN_OK) return st;
    if (T == 0) return GDN_OK;  // empty arrays may be NULL
    const size_t n = (size_t)n_adapters, need = gdn_adapter_workspace_bytes(n_seq, T, rank, d_in);
    const Buf lists[] = {{ids, (size_t)n_seq * 4, "ids"}, {ranks, ranks ? n * 4 : 0, "ranks"}, {scales, n * 4, "scales"}};
    for (const Buf& b : lists) {
        if (b.bytes && !b.p) return fail(GDN_ERR_INVALID_ARG, "%s is NULL", b.name);
        if (b.bytes && !aligned4(b.p)) return fail(GDN_ERR_ALIGNMENT, "%s is not 4-byte aligned", b.name);
    }
    const Buf y_in{y, span(T, y_stride, d_out, 2), "y"}, out{y_out, span(T, y_out_stride, d_out, 2), "y_out"}, ws{workspace, need, "workspace"};
    const Buf arrays[] = {{x, span(T, x_stride, d_in, 2), "x"}, {down, n * rank * d_in * 2, "down"}, {up, n * rank * d_out * 2, "up"}, y_in, out};
    if ((st = check_bufs(arrays, 5)) != GDN_OK) return st;
    if (workspace_bytes < need || !workspace) return fail(GDN_ERR_WORKSPACE, "adapter workspace %zu bytes, need %zu", workspace_bytes, need);
    if ((st = check_bufs(&ws, 1)) != GDN_OK) return st;
    const Buf outs[] = {out, ws}, ins[] = {arrays[0], arrays[1], arrays[2], lists[0], lists[1], lists[2], y_in};
    // y_out may be y itself: a block has read what it writes
    const bool in_place = y_out == y && y_out_stride == y_stride;
    if ((st = check_disjoint(outs, 2, ins, in_place ? 6 : 7)) != GDN_OK) return st;
    if (in_place && overlap(ws, y_in)) return fail(GDN_ERR_INVALID_ARG, "workspace overlaps y");
    gdn::AdapterParams p{};
    p.n_seq = n_seq; p.T = T; p.n_adapters = n_adapters; p.rank = rank; p.d_in = d_in; p.d_out = d_out; p.bf16 = dtype == GDN_BF16;
    p.cu_seqlens = cu_seqlens; p.ids = ids; p.ranks = ranks; p.down = down; p.up = up; p.scales = scales;
    p.x = x; p.y = y; p.y_out = y_out; p.x_stride = x_stride; p.y_stride = y_stride; p.out_stride = y_out_stride;
    cudaError_t e = gdn::launch_adapter(p, workspace, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_adapter_add launch");
}

gdn_status gdn_adapter_check(const void* workspace, struct CUstream_st* stream)
{
    if (!workspace) return fail(GDN_ERR_INVALID_ARG, "workspace is NULL");
    int32_t status[2 * gdn::kAdapterCtas] = {};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemcpyAsync(status, workspace, sizeof status, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "reading the failure record");
    for (int32_t w : status)
        if (w) return fail(GDN_ERR_TIMEOUT, "a bounded wait in the kernels expired; outputs are invalid");
    return GDN_OK;
}

}  // extern "C"
