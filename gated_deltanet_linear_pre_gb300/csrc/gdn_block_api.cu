// gdn_block_api.cu -- the C ABI's entries of what lies around the layers: host-side
// argument validation and launches.  No allocation, no synchronisation.
#include <cmath>

#include "gdn.h"
#include "gdn_host.cuh"
#include "gdn_internal.cuh"

using namespace gdn::host;

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
    if ((st = check_stride("x", x_stride, width)) != GDN_OK) return st;
    if (y && (st = check_stride("y", y_stride, width)) != GDN_OK) return st;
    if (gate && gate_stride != 0 && (st = check_stride("gate", gate_stride, width)) != GDN_OK) return st;
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

}  // extern "C"
