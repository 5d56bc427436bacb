// gdn_block_norm.cu -- the residual stream between two blocks.
//
//   u  = y, over sqrt(mean(y^2) + eps) and times post_weight where there is one
//   x' = x + scale * act(gate) * u
//   h  = x' / sqrt(mean(x'^2) + eps) * pre_weight
//
// HBM-bound: a row is read once, held in registers through both norms and written
// once.  h comes from x' before its rounding to x's type.  A block takes one row,
// two vectors of 8 channels a thread, with all of the row's loads under way before
// the first sum; a warp takes it where it is short.  Measured, of what a plain copy
// reaches: 8192 tokens of 5120 channels (bf16, normed and gated by a sigmoid a token)
// 76 us, 81%; without norm and gate 4096 channels 42 us, 95%; 4001 tokens of 7176,
// fp32 stream, 64 us, 79%.  The first two stood at 126 and 98 us with one vector a
// thread, the gate loaded behind the first sum, expf and a full division; four
// vectors a thread took 93 (fewer threads to hide a row's two sums behind).
#include "gdn.h"
#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kRowWarps = 4;   // rows per block where one warp holds a row
constexpr int kFewRows = 304;  // rows that the SMs take two at a time

// 8 values of the residual stream, fp32 or the activations' type, as they were loaded
template <bool X32>
struct Raw {
    uint4 v[X32 ? 2 : 1];
};

template <bool X32>
__device__ __forceinline__ Raw<X32> load_x(const void* p, int64_t at)
{
    Raw<X32> r;
    const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + at * (X32 ? 4 : 2));
    r.v[0] = __ldcs(from);
    if (X32) r.v[X32] = __ldcs(from + 1);
    return r;
}

template <bool X32, bool BF16>
__device__ __forceinline__ void widen_x(const Raw<X32>& r, float (&x)[8])
{
    if (X32) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 w = r.v[X32 ? i : 0];
            x[4 * i] = __uint_as_float(w.x);
            x[4 * i + 1] = __uint_as_float(w.y);
            x[4 * i + 2] = __uint_as_float(w.z);
            x[4 * i + 3] = __uint_as_float(w.w);
        }
    } else {
        widen8<BF16>(r.v[0], x);
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

// A sigmoid is exp(g) / (1 + exp(g)), with g held below 80, where it is 1: the divisor stays in the approximate quotient's
// range (up to 2^126) and small sigmoids come out down to the type's least values (as 1 / (1 + exp(-g)) they were 0 below
// -87.3, where a y of 1e38 shows 60 of it).  The exponential is the hardware's where the stream has 16 bits, off by
// 2 + 1.173 |g| units of 2^-23 at most; the quotient by 2 units for either.
template <bool X32>
__device__ __forceinline__ float gated(int kind, float g)
{
    if (kind == GDN_GATE_LINEAR) return g;
    float low;  // NaN stays NaN
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(low) : "f"(g), "f"(80.0f));
    const float e = X32 ? expf(low) : __expf(low), s = __fdividef(e, 1.0f + e);
    return kind == GDN_GATE_SIGMOID ? s : g * s;
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

// One row per warp, or per block; VPT vectors of 8 values a thread, all of a row's loads under way at once.
template <bool X32, bool BF16, bool WARP_ROW, int VPT, int THREADS>
__global__ void __launch_bounds__(THREADS) block_norm_kernel(BlockNormParams p)
{
    __shared__ float part[2][32];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = WARP_ROW ? (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5) : blockIdx.x;
    const int lane = WARP_ROW ? threadIdx.x & 31 : threadIdx.x, lanes = WARP_ROW ? 32 : blockDim.x;
    if (row >= p.T) return;
    const float inv = 1.0f / (float)p.width;
    Raw<X32> raw[VPT];
    uint4 y[VPT], gate[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * lanes + lane) * 8;
        raw[i] = Raw<X32>{};
        y[i] = gate[i] = make_uint4(0, 0, 0, 0);
        if (c < p.width) {
            raw[i] = load_x<X32>(p.x, row * p.x_stride + c);
            if (p.y) y[i] = __ldcs(reinterpret_cast<const uint4*>(p.y + row * p.y_stride + c));
            if (p.gate) gate[i] = p.gate_stride ? __ldcs(reinterpret_cast<const uint4*>(p.gate + row * p.gate_stride + c))
                                                : __ldg(reinterpret_cast<const uint4*>(p.gate + c));
        }
    }
    float x[VPT][8];
    if (p.y) {
        float r = 1.0f;
        if (p.post_weight) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float u[8];
                widen8<BF16>(y[i], u);
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(u[e], u[e], ss);
            }
            r = rsqrtf(row_sum<WARP_ROW>(ss, part[0]) * inv + p.eps);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * lanes + lane) * 8;
            float u[8];
            widen8<BF16>(y[i], u);
            widen_x<X32, BF16>(raw[i], x[i]);
            if (c < p.width) {
                if (p.post_weight) {
                    float w[8];
                    load_weight(p.post_weight, c, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) u[e] = u[e] * r * w[e];
                }
                if (p.gate_kind != GDN_GATE_NONE) {
                    float g[8];
                    widen8<BF16>(gate[i], g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) u[e] *= gated<X32>(p.gate_kind, g[e]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) x[i][e] = fmaf(p.scale, u[e], x[i][e]);
                if (p.x_out) store_x<X32, BF16>(p.x_out, row * p.width + c, x[i]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) widen_x<X32, BF16>(raw[i], x[i]);
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
        return launch_k(kernel, dim3((unsigned)(((int64_t)p.T + kRowWarps - 1) / kRowWarps)), dim3(kRowWarps * 32), 0, stream, true, p);
    };
    const auto row_blocks = [&](auto kernel, int vpt) {
        const int threads = ((vectors + vpt - 1) / vpt + 31) / 32 * 32;
        return launch_k(kernel, dim3((unsigned)p.T), dim3((unsigned)threads), 0, stream, true, p);
    };
    if (vectors <= 32) return row_warps(block_norm_kernel<X32, BF16, true, 1, kRowWarps * 32>);
    if (vectors <= 64) return row_warps(block_norm_kernel<X32, BF16, true, 2, kRowWarps * 32>);
    // few rows: their latency, one vector a thread; many: bytes in flight (1000 rows of 4096: 5.4 us, 6.4 with one)
    if (p.T <= kFewRows && vectors <= 1024) return row_blocks(block_norm_kernel<X32, BF16, false, 1, 1024>, 1);
    if (vectors <= 512) return row_blocks(block_norm_kernel<X32, BF16, false, 2, 256>, 2);
    if (vectors <= 1024) return row_blocks(block_norm_kernel<X32, BF16, false, 2, 512>, 2);
    return row_blocks(block_norm_kernel<X32, BF16, false, 2, 1024>, 2);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormParams& p, cudaStream_t stream)
{
    if (p.x32) return p.bf16 ? launch_typed<true, true>(p, stream) : launch_typed<true, false>(p, stream);
    return p.bf16 ? launch_typed<false, true>(p, stream) : launch_typed<false, false>(p, stream);
}

}  // namespace gdn
