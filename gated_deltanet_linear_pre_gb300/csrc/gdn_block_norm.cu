// gdn_block_norm.cu -- the residual stream between two blocks.
//
//   u  = y, over sqrt(mean(y^2) + eps) and times post_weight where there is one
//   x' = x + scale * act(gate) * u
//   h  = x' / sqrt(mean(x'^2) + eps) * pre_weight
//
// HBM-bound: a row is read once, held in registers in fp32 through both norms
// and written once.  h comes from x' before its rounding to x's type.
#include "gdn.h"
#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kRowWarps = 4;  // rows per block where one warp holds a row

// 8 values of the residual stream, fp32 or the activations' type, to fp32
template <bool X32, bool BF16>
__device__ __forceinline__ void load_x(const void* p, int64_t at, float (&x)[8])
{
    if (X32) {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
        const float4 a = __ldcs(f), b = __ldcs(f + 1);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        widen8<BF16>(__ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at)), x);
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 narrow8(const float (&x)[8])
{
    return make_uint4(narrow2<BF16>(x[0], x[1]), narrow2<BF16>(x[2], x[3]), narrow2<BF16>(x[4], x[5]), narrow2<BF16>(x[6], x[7]));
}

template <bool X32, bool BF16>
__device__ __forceinline__ void store_x(void* p, int64_t at, const float (&x)[8])
{
    if (X32) {
        float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
        __stcs(f, make_float4(x[0], x[1], x[2], x[3]));
        __stcs(f + 1, make_float4(x[4], x[5], x[6], x[7]));
    } else {
        __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at), narrow8<BF16>(x));
    }
}

__device__ __forceinline__ void load_weight(const float* w, int at, float (&x)[8])
{
    const float4* f = reinterpret_cast<const float4*>(w + at);
    const float4 a = __ldg(f), b = __ldg(f + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

__device__ __forceinline__ float gated(int kind, float g)
{
    return kind == GDN_GATE_LINEAR ? g : kind == GDN_GATE_SIGMOID ? sigmoidf_(g) : siluf_(g);
}

// Sum over the threads of a row: a warp, or the whole block.
template <bool WARP_ROW>
__device__ __forceinline__ float row_sum(float v, float* part)
{
    v = warp_sum(v);
    if (WARP_ROW) return v;
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < warps ? part[lane] : 0.0f);
}

// One row per warp, or per block; VPT vectors of 8 values a thread.
template <bool X32, bool BF16, bool WARP_ROW, int VPT>
__global__ void __launch_bounds__(WARP_ROW ? kRowWarps * 32 : 1024) block_norm_kernel(BlockNormParams p)
{
    __shared__ float part[2][32];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = WARP_ROW ? (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5) : blockIdx.x;
    const int lane = WARP_ROW ? threadIdx.x & 31 : threadIdx.x, lanes = WARP_ROW ? 32 : blockDim.x;
    if (row >= p.T) return;
    const float inv = 1.0f / (float)p.width;
    float x[VPT][8], u[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * lanes + lane) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = u[i][e] = 0.0f;
        if (c < p.width) {
            load_x<X32, BF16>(p.x, row * p.x_stride + c, x[i]);
            if (p.y) widen8<BF16>(__ldcs(reinterpret_cast<const uint4*>(p.y + row * p.y_stride + c)), u[i]);
        }
    }
    if (p.y) {
        if (p.post_weight) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(u[i][e], u[i][e], ss);
            const float r = rsqrtf(row_sum<WARP_ROW>(ss, part[0]) * inv + p.eps);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = (i * lanes + lane) * 8;
                if (c < p.width) {
                    float w[8];
                    load_weight(p.post_weight, c, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) u[i][e] = u[i][e] * r * w[e];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * lanes + lane) * 8;
            if (c < p.width) {
                if (p.gate_kind != GDN_GATE_NONE) {
                    float g[8];
                    widen8<BF16>(__ldg(reinterpret_cast<const uint4*>(p.gate + row * p.gate_stride + c)), g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) u[i][e] *= gated(p.gate_kind, g[e]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) x[i][e] = fmaf(p.scale, u[i][e], x[i][e]);
                if (p.x_out) store_x<X32, BF16>(p.x_out, row * p.width + c, x[i]);
            }
        }
    }
    if (!p.h) return;
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[i][e], x[i][e], ss);
    const float r = rsqrtf(row_sum<WARP_ROW>(ss, part[1]) * inv + p.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * lanes + lane) * 8;
        if (c < p.width) {
            float w[8];
            load_weight(p.pre_weight, c, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i][e] = x[i][e] * r * w[e];
            __stcs(reinterpret_cast<uint4*>(p.h + row * p.width + c), narrow8<BF16>(x[i]));
        }
    }
}

template <bool X32, bool BF16>
cudaError_t launch_typed(const BlockNormParams& p, cudaStream_t stream)
{
    const int vectors = p.width / 8;
    const auto row_warps = [&](auto kernel) {
        return launch_k(kernel, dim3((unsigned)((p.T + kRowWarps - 1) / kRowWarps)), dim3(kRowWarps * 32), 0, stream, true, p);
    };
    const auto row_blocks = [&](auto kernel, int vpt) {
        const int threads = ((vectors + vpt - 1) / vpt + 31) / 32 * 32;
        return launch_k(kernel, dim3((unsigned)p.T), dim3((unsigned)threads), 0, stream, true, p);
    };
    if (vectors <= 32) return row_warps(block_norm_kernel<X32, BF16, true, 1>);
    if (vectors <= 64) return row_warps(block_norm_kernel<X32, BF16, true, 2>);
    if (vectors <= 1024) return row_blocks(block_norm_kernel<X32, BF16, false, 1>, 1);
    return row_blocks(block_norm_kernel<X32, BF16, false, 2>, 2);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormParams& p, cudaStream_t stream)
{
    if (p.x32) return p.bf16 ? launch_typed<true, true>(p, stream) : launch_typed<true, false>(p, stream);
    return p.bf16 ? launch_typed<false, true>(p, stream) : launch_typed<false, false>(p, stream);
}

}  // namespace gdn
