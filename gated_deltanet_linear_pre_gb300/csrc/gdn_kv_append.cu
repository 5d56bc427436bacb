// gdn_kv_append.cu -- rotation, 8-bit quantisation and paged storage of new keys
// and values, and rotation of the queries, in one launch.
//
// Mathematics.  x = R(position) k (pairs of channels turned by the table's angle, in fp32) or x = v.
// A page and head share one scale S, a power of two: S = max(S_old, 2^ceil(log2(max|x| / qmax))), and a
// code is x / S to nearest even.  Powers of two make three things exact: the division, the
// dequantisation, and the growth S / S_old by which earlier codes of the page are shifted when a larger
// value arrives; since every growth at least doubles S, the half steps lost at each of them add up to
// less than one step of the final S.
//
// Layout.  The unit of work is (page touched by a sequence, kv head, k or v): its scale is one maximum
// over the unit's rows, so no unit needs another's result and the call is one launch without
// atomics.  16 bytes per thread: D / 8 threads hold a row, and the partner channels of a rotation
// half a head apart come from another lane of the row by shuffles.  A sequence's pages get
// slots floor(cu[s] / P) + 2 s onwards: n tokens touch at most floor((n - 1) / P) + 2 pages, so
// floor(T / P) + 2 n_seq slots hold any batch without a prefix sum on the host.
#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// Rotates the 8 channels 8c .. 8c+7 that this lane holds of a row (lanes of a row are adjacent).
// `cs`, `sn`: the position's table rows.  Every product and sum is rounded to fp32 on its own: the
// result does not depend on how a compiler would contract them.
template <bool BF16>
__device__ __forceinline__ void rotate8(const uint4& raw, float (&x)[8], int c, int rot, int interleaved, const float* cs, const float* sn)
{
    if (rot == 0) return;
    const int half = rot >> 1;
    if (interleaved) {
        if (8 * c >= rot) return;
        const float4 co = __ldg(reinterpret_cast<const float4*>(cs) + c), si = __ldg(reinterpret_cast<const float4*>(sn) + c);
        const float cc[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a = x[2 * e], b = x[2 * e + 1];
            x[2 * e] = __fsub_rn(__fmul_rn(a, cc[e]), __fmul_rn(b, ss[e]));
            x[2 * e + 1] = __fadd_rn(__fmul_rn(b, cc[e]), __fmul_rn(a, ss[e]));
        }
        return;
    }
    const int shift = half >> 3;  // lanes between the two channels of a pair
    const bool first = c < shift, turned = c < 2 * shift;
    const int lane = threadIdx.x & 31;
    const int from = turned ? (first ? lane + shift : lane - shift) : lane;
    uint4 o;
    o.x = __shfl_sync(0xffffffffu, raw.x, from);
    o.y = __shfl_sync(0xffffffffu, raw.y, from);
    o.z = __shfl_sync(0xffffffffu, raw.z, from);
    o.w = __shfl_sync(0xffffffffu, raw.w, from);
    if (!turned) return;
    float other[8];
    widen8<BF16>(o, other);
    const int j = 8 * (first ? c : c - shift);
    const float4* cp = reinterpret_cast<const float4*>(cs + j);
    const float4* sp = reinterpret_cast<const float4*>(sn + j);
    const float4 c0 = __ldg(cp), c1 = __ldg(cp + 1), s0 = __ldg(sp), s1 = __ldg(sp + 1);
    const float cc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const float ss[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float own = __fmul_rn(x[e], cc[e]), cross = __fmul_rn(other[e], ss[e]);
        x[e] = first ? __fsub_rn(own, cross) : __fadd_rn(own, cross);
    }
}

// Smallest power of two not below amax / qmax, at least 2^-100; 0 for 0 and NaN for an infinity or NaN.
// 127 = 1.984375 x 2^6 and 448 = 1.75 x 2^8: the exponent is amax's less 6 or 8, one more where amax's
// mantissa exceeds qmax's.
template <bool E4M3>
__device__ __forceinline__ float scale_for(uint32_t amax_bits)
{
    if (amax_bits == 0) return 0.0f;
    if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
    const int e = (int)(amax_bits >> 23) - (E4M3 ? 8 : 6) + ((amax_bits & 0x7fffffu) > (E4M3 ? 0x600000u : 0x7e0000u) ? 1 : 0);
    return __uint_as_float((uint32_t)max(e, 27) << 23);
}

// 8 values times inv (a power of two) to codes, nearest even; |x inv| <= qmax
template <bool E4M3>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv)
{
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i] * inv, b = x[2 * i + 1] * inv;
        uint32_t pair;
        if (E4M3) pair = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
        else pair = ((uint32_t)__float2int_rn(a) & 0xffu) | (((uint32_t)__float2int_rn(b) & 0xffu) << 8);
        w[i >> 1] |= pair << (16 * (i & 1));
    }
    return make_uint2(w[0], w[1]);
}

template <bool E4M3>
__device__ __forceinline__ void decode8(const uint2& w, float (&x)[8])
{
    const uint32_t r[2] = {w.x, w.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t pair = (r[i >> 1] >> (16 * (i & 1))) & 0xffffu;
        if (E4M3) {
            const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)pair, __NV_E4M3)));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        } else {
            x[2 * i] = (float)(int8_t)(pair & 0xffu);
            x[2 * i + 1] = (float)(int8_t)(pair >> 8);
        }
    }
}

// One unit with UNIT threads (32: a warp; 256: the block).  The block form holds every row of a page in
// registers between the maximum and the codes (8 rows a thread at P = 128, D = 128); the warp form reads
// its rows twice, the second time from the first-level cache.
template <bool BF16, bool E4M3, int D, int UNIT>
__device__ __forceinline__ void store_unit(const AppendParams& p, int unit)
{
    constexpr int kRowLanes = D / 8, kRows = UNIT / kRowLanes;      // threads a row, rows a pass
    constexpr int kHeld = UNIT == 32 ? 1 : 128 / kRows;             // rows a thread holds (block form)
    const int tid = threadIdx.x % UNIT, c = tid % kRowLanes, r0 = tid / kRowLanes;
    const int slot = unit / (2 * p.heads), rest = unit - slot * 2 * p.heads;
    const int head = rest >> 1, is_v = rest & 1;
    const int shift = 31 - __clz(p.page);
    auto base = [&](int s) { return (cu_at(p.cu_seqlens, s, p.T) >> shift) + 2 * s; };
    const int s = warp_find(p.n_seq, slot, base);
    const int t0 = cu_at(p.cu_seqlens, s, p.T), n = cu_at(p.cu_seqlens, s + 1, p.T) - t0, first = past_at(p.past, s);
    const int at = (first >> shift) + slot - ((t0 >> shift) + 2 * s);
    // rows [lo, hi) of the page are this call's; tokens t0 + at * P - first + row
    const int lo = max(first - at * p.page, 0), hi = min(first + n - at * p.page, p.page);
    if (n <= 0 || lo >= hi) return;  // uniform over the unit
    const int page = page_at(p, s, at);
    if (page < 0) return;
    float* const scale_at = (is_v ? p.v_scale : p.k_scale) + (size_t)page * p.heads + head;
    uint8_t* const codes = (is_v ? p.v : p.k) + ((size_t)page * p.heads + head) * p.page * D + 8 * c;
    const uint16_t* const src = (is_v ? p.v_new : p.k_new) + (int64_t)(t0 + at * p.page - first) * (is_v ? p.v_stride : p.k_stride) + head * D + 8 * c;
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    const int rot = is_v ? 0 : p.rot, half = p.rot >> 1;
    const float before = lo > 0 ? *scale_at : 0.0f;

    // the rotated row `row` (valid where lo <= row < hi; other lanes of a warp take part in the shuffles)
    auto load = [&](int row, float (&x)[8]) {
        const bool mine = row >= lo && row < hi;
        const uint4 raw = mine ? __ldg(reinterpret_cast<const uint4*>(src + (int64_t)row * stride)) : make_uint4(0, 0, 0, 0);
        widen8<BF16>(raw, x);
        const int64_t at_pos = rot ? (int64_t)min(at * p.page + min(row, p.page - 1), p.n_pos - 1) * half : 0;
        rotate8<BF16>(raw, x, c, rot, p.interleaved, p.cos + at_pos, p.sin + at_pos);
        return mine;
    };

    float held[kHeld][8];
    uint32_t amax = 0;  // as bits: infinities and NaN come out largest
    const int rows = UNIT == 32 ? (hi - lo + kRows - 1) / kRows : kHeld;
    const int start = UNIT == 32 ? lo : 0;
#pragma unroll
    for (int i = 0; i < (UNIT == 32 ? 1 : kHeld); ++i) {
        if (UNIT == 32) {
            for (int j = 0; j < rows; ++j) {
                float x[8];
                if (load(start + j * kRows + r0, x))
#pragma unroll
                    for (int e = 0; e < 8; ++e) amax = max(amax, __float_as_uint(x[e]) & 0x7fffffffu);
            }
        } else if (i * kRows < p.page) {
            if (load(i * kRows + r0, held[i]))
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = max(amax, __float_as_uint(held[i][e]) & 0x7fffffffu);
        }
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    if (UNIT > 32) {
        __shared__ uint32_t part[kThreads / 32];
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) amax = max(amax, part[w]);
    }
    const float need = scale_for<E4M3>(amax);
    const float scale = (before != before || need != need) ? __uint_as_float(0x7fc00000u) : fmaxf(before, need);
    const float inv = scale > 0.0f ? __frcp_rn(scale) : 0.0f;  // exact: a power of two
    if (scale > before) {  // earlier rows move to the larger scale (before = 0: all their values are 0)
        const float ratio = before * inv;
        for (int row = r0; row < lo; row += kRows) {
            uint2* const w = reinterpret_cast<uint2*>(codes + (size_t)row * D);
            float x[8];
            decode8<E4M3>(*w, x);
            *w = encode8<E4M3>(x, ratio);
        }
    }
#pragma unroll
    for (int i = 0; i < (UNIT == 32 ? 1 : kHeld); ++i) {
        if (UNIT == 32) {
            for (int j = 0; j < rows; ++j) {
                float x[8];
                const int row = start + j * kRows + r0;
                if (load(row, x)) *reinterpret_cast<uint2*>(codes + (size_t)row * D) = scale > 0.0f ? encode8<E4M3>(x, inv) : make_uint2(0u, 0u);
            }
        } else if (i * kRows < p.page) {
            const int row = i * kRows + r0;
            if (row >= lo && row < hi) *reinterpret_cast<uint2*>(codes + (size_t)row * D) = scale > 0.0f ? encode8<E4M3>(held[i], inv) : make_uint2(0u, 0u);
        }
    }
    if (tid == 0) *scale_at = scale;
}

// blocks [0, unit_blocks) store pages; the others rotate queries, 16 bytes a thread
template <bool BF16, bool E4M3, int D, int UNIT>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(AppendParams p, int units, int unit_blocks)
{
    pdl_wait();
    pdl_launch_dependents();
    if ((int)blockIdx.x < unit_blocks) {
        const int unit = blockIdx.x * (kThreads / UNIT) + threadIdx.x / UNIT;
        if (unit < units) store_unit<BF16, E4M3, D, UNIT>(p, unit);
        return;
    }
    constexpr int kRowLanes = D / 8, kRows = kThreads / kRowLanes;
    const int64_t row = (int64_t)(blockIdx.x - unit_blocks) * kRows + threadIdx.x / kRowLanes;
    const int64_t last = (int64_t)p.T * p.hq - 1;
    const int64_t mine = min(row, last);  // lanes past the end repeat the last row: they take part in shuffles
    const int t = (int)(mine / p.hq), head = (int)(mine - (int64_t)t * p.hq), c = threadIdx.x % kRowLanes;
    // a warp's rows may belong to two sequences: each lane looks for its own
    int lo = 0, hi = p.n_seq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu_at(p.cu_seqlens, mid, p.T) <= t) lo = mid; else hi = mid;
    }
    const int pos = past_at(p.past, lo) + t - cu_at(p.cu_seqlens, lo, p.T);
    const uint4 raw = __ldg(reinterpret_cast<const uint4*>(p.q + (int64_t)t * p.q_stride + head * D + 8 * c));
    float x[8];
    widen8<BF16>(raw, x);
    const int64_t at_pos = p.rot ? (int64_t)min(max(pos, 0), p.n_pos - 1) * (p.rot >> 1) : 0;
    rotate8<BF16>(raw, x, c, p.rot, p.interleaved, p.cos + at_pos, p.sin + at_pos);
    if (row <= last) {
        const uint4 w = make_uint4(narrow2<BF16>(x[0], x[1]), narrow2<BF16>(x[2], x[3]), narrow2<BF16>(x[4], x[5]), narrow2<BF16>(x[6], x[7]));
        *reinterpret_cast<uint4*>(p.q_out + (mine * D + 8 * c)) = w;
    }
}

template <bool BF16, bool E4M3, int D>
cudaError_t launch(const AppendParams& p, cudaStream_t stream)
{
    // A warp per unit where sequences bring a few tokens each (a block would leave most of its
    // threads without a row), a block per unit where they fill pages.
    const bool warp_units = (int64_t)p.T <= 8 * (int64_t)p.n_seq;
    const int64_t units = ((int64_t)p.T / p.page + 2 * (int64_t)p.n_seq) * p.heads * 2;
    const int64_t per_block = warp_units ? kThreads / 32 : 1;
    const int64_t unit_blocks = (units + per_block - 1) / per_block;
    const int64_t q_blocks = ((int64_t)p.T * p.hq * (D / 8) + kThreads - 1) / kThreads;
    if (units > 0x7fffffff || unit_blocks + q_blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)(unit_blocks + q_blocks));
    if (warp_units) return launch_k(kv_append_kernel<BF16, E4M3, D, 32>, grid, dim3(kThreads), 0, stream, true, p, (int)units, (int)unit_blocks);
    return launch_k(kv_append_kernel<BF16, E4M3, D, kThreads>, grid, dim3(kThreads), 0, stream, true, p, (int)units, (int)unit_blocks);
}

template <bool BF16, bool E4M3>
cudaError_t launch_dim(const AppendParams& p, cudaStream_t stream)
{
    return p.dim == 64 ? launch<BF16, E4M3, 64>(p, stream) : launch<BF16, E4M3, 128>(p, stream);
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t stream)
{
    if (p.format == 1) return p.bf16 ? launch_dim<true, true>(p, stream) : launch_dim<false, true>(p, stream);
    return p.bf16 ? launch_dim<true, false>(p, stream) : launch_dim<false, false>(p, stream);
}

}  // namespace gdn
