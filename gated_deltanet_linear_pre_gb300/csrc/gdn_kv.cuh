// gdn_kv.cuh -- device helpers shared by the kernels of the 8-bit paged cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "gdn_internal.cuh"

namespace gdn {

// Largest s in [0, n) with base(s) <= x, for a non-decreasing base with base(0) <= x; a whole warp
// searches 32-way, so a batch of 1024 sequences takes two dependent loads instead of ten.
template <typename F>
__device__ __forceinline__ int warp_find(int n, int64_t x, F base)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5;
        const int at = lo + lane * step;
        const bool below = at < hi && base(at) <= x;
        const int count = max(__popc(__ballot_sync(0xffffffffu, below)), 1);
        lo += (count - 1) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// past[s], kept where position arithmetic cannot leave 31 bits
__device__ __forceinline__ int past_at(const int32_t* past, int s) { return min(max(__ldg(past + s), -(1 << 30)), 1 << 30); }

__device__ __forceinline__ int page_shift(const KvBatch& p) { return 31 - __clz(p.page); }

// pool page of table entry `at` of sequence s, or -1 where there is none
__device__ __forceinline__ int page_at(const KvBatch& p, int s, int at)
{
    if (at < 0 || at >= p.max_pages) return -1;
    const int page = __ldg(p.table + (size_t)s * p.table_stride + at);
    return page < p.n_pages ? page : -1;
}

// 8 activations (16 bytes) to fp32; exact
template <bool BF16>
__device__ __forceinline__ void widen8(const uint4& w, float (&x)[8])
{
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF16) {
            x[2 * i] = __uint_as_float(r[i] << 16);
            x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

// two fp32 values to the activation type (round to nearest even), packed
template <bool BF16>
__device__ __forceinline__ uint32_t narrow2(float a, float b)
{
    if (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace gdn
