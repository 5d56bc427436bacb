// gdn_kv_append.cu -- rotation, 8-bit quantisation and paged storage of new keys
// and values, and rotation of the queries, in one launch.
//
// Mathematics.  x = R(position) k (pairs of channels turned by the table's angle, in fp32) or x = v.
// A page and head share one scale S, a power of two: S = max(S_old, 2^ceil(log2(max|x| / qmax))), and a
// code is x / S to nearest even.  Powers of two make three things exact: the division, the
// dequantisation, and the growth S / S_old by which earlier codes of the page are shifted when a larger
// value arrives; since every growth at least doubles S, the half steps lost at each of them add up to
// less than one step of the final S.  A value that is not finite makes the page's scale NaN, whose bits keep
// S (of the finite values; their codes are as they would be without it) and the first row that holds one: an
// append that starts at or in front of that row, as after rejected drafts, finds the page as it was.
//
// Layout.  The unit of work is (page touched by a sequence, kv head, k or v): its scale is one maximum
// over the unit's rows, so no unit needs another's result and the call is one launch without
// atomics.  16 bytes per thread: D / 8 threads hold a row, and the partner channels of a rotation
// half a head apart come from another lane of the row by shuffles.  Queries go by (token, 4 heads): a
// lane's four loads are in flight together and share the angles it holds.  A sequence's pages get
// slots floor(cu[s] / P) + 2 s onwards: n tokens touch at most floor((n - 1) / P) + 2 pages, so
// floor(T / P) + 2 n_seq slots hold any batch without a prefix sum on the host.
//
// Bound and measured.  Large calls by HBM: every value is read once and written once.  8 prompts of 1 to 4096
// tokens (48 query and 16 kv heads of 128, fp16 to e4m3, pages of 64) take 189 us for 950 MB at the DRAM, 5.0
// TB/s; the bytes' floor is 150 us at 6.8 TB/s.  (Eight query heads a lane in place of four: 192 to 200 us.)  Small calls by
// one chain of loads (lengths, table entry, scale, values): a token for each of 64 sequences takes 3.7 us.
#include "gdn_kv.cuh"

namespace gdn {
namespace {

// The angles of the 8 channels 8c .. 8c+7 that this lane holds of a row at one position, and their
// rotation (lanes of a row are adjacent).  Every product and sum is rounded to fp32 on its own: the
// result does not depend on how a compiler would contract them.
struct Angles {
    float c[8], s[8];
    int from;      // lane of the partner channels (rotations of halves)
    bool turned, first;

    __device__ __forceinline__ Angles(const AppendParams& p, int lane8, int pos)
    {
        const int half = p.rot >> 1, lane = threadIdx.x & 31;
        const int64_t at = (int64_t)min(max(pos, 0), p.n_pos - 1) * half;
        if (p.interleaved) {  // 4 angles
            turned = 8 * lane8 < p.rot;
            first = true;
            from = lane;
            if (turned) {
                load4(p.cos + at + 4 * lane8, c);
                load4(p.sin + at + 4 * lane8, s);
            }
        } else {
            const int shift = half >> 3;  // lanes between the two channels of a pair
            first = lane8 < shift;
            turned = lane8 < 2 * shift;
            from = turned ? (first ? lane + shift : lane - shift) : lane;
            if (turned) {
                const int64_t j = at + 8 * (first ? lane8 : lane8 - shift);
                load4(p.cos + j, c);
                load4(p.cos + j + 4, c + 4);
                load4(p.sin + j, s);
                load4(p.sin + j + 4, s + 4);
            }
        }
    }
    static __device__ __forceinline__ void load4(const float* a, float* x)
    {
        const float4 v = __ldg(reinterpret_cast<const float4*>(a));
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    }
    // x: the row's values of this lane, raw their bits (whole warps call this together)
    template <bool BF16>
    __device__ __forceinline__ void turn(const uint4& raw, float (&x)[8], int interleaved) const
    {
        if (interleaved) {
            if (!turned) return;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float a = x[2 * e], b = x[2 * e + 1];
                x[2 * e] = __fsub_rn(__fmul_rn(a, c[e]), __fmul_rn(b, s[e]));
                x[2 * e + 1] = __fadd_rn(__fmul_rn(b, c[e]), __fmul_rn(a, s[e]));
            }
            return;
        }
        uint4 o;
        o.x = __shfl_sync(0xffffffffu, raw.x, from);
        o.y = __shfl_sync(0xffffffffu, raw.y, from);
        o.z = __shfl_sync(0xffffffffu, raw.z, from);
        o.w = __shfl_sync(0xffffffffu, raw.w, from);
        if (!turned) return;
        float other[8];
        widen8<BF16>(o, other);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float own = __fmul_rn(x[e], c[e]), cross = __fmul_rn(other[e], s[e]);
            x[e] = first ? __fsub_rn(own, cross) : __fadd_rn(own, cross);
        }
    }
};

// Smallest power of two not below amax / qmax, at least 2^-100; 0 for 0.
// 127 = 1.984375 x 2^6 and 448 = 1.75 x 2^8: the exponent is amax's less 6 or 8, one more where amax's
// mantissa exceeds qmax's.
template <bool E4M3>
__device__ __forceinline__ float scale_for(uint32_t amax_bits)
{
    if (amax_bits == 0) return 0.0f;
    const int e = (int)(amax_bits >> 23) - (E4M3 ? 8 : 6) + ((amax_bits & 0x7fffffu) > (E4M3 ? 0x600000u : 0x7e0000u) ? 1 : 0);
    return __uint_as_float((uint32_t)max(e, 27) << 23);
}

// The scale of a page that holds a value that is not finite: a NaN of 17 fixed bits, the exponent of the finite
// values' scale (8 bits) and the first such row (7).  Any other NaN says nothing of either.
constexpr uint32_t kNanScale = 0x7fd50000u, kNanScaleMask = 0xffff8000u;
constexpr int kNoRow = 1 << 30;
__device__ __forceinline__ float nan_scale(float scale, int row)
{
    return __uint_as_float(scale == scale ? kNanScale | ((__float_as_uint(scale) >> 23) << 7) | (uint32_t)row : 0x7fc00000u);
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

// One unit, by a warp or a block (THREADS).  The page's rows stay in registers (HELD a thread) between the
// maximum and the codes, or, HELD = 0, the call's few rows are read twice, the second time from the
// first-level cache.
template <bool BF16, bool E4M3, int D, int THREADS, int HELD>
__device__ __forceinline__ void store_unit(const AppendParams& p, int unit)
{
    constexpr bool kTwice = HELD == 0;
    constexpr int kRowLanes = D / 8, kRows = THREADS / kRowLanes;  // threads a row, rows a pass
    const int tid = threadIdx.x % THREADS, c = tid % kRowLanes, r0 = tid / kRowLanes;
    const int slot = unit / (2 * p.heads), rest = unit - slot * 2 * p.heads;
    const int is_v = rest >= p.heads, head = is_v ? rest - p.heads : rest;
    const int shift = page_shift(p);
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
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    const uint16_t* const src = (is_v ? p.v_new : p.k_new) + (int64_t)(t0 + at * p.page - first) * stride + head * D + 8 * c;
    const bool rotated = !is_v && p.rot > 0;
    float before = lo > 0 ? *scale_at : 0.0f;

    auto fetch = [&](int row) {
        return row >= lo && row < hi ? __ldg(reinterpret_cast<const uint4*>(src + (int64_t)row * stride)) : make_uint4(0u, 0u, 0u, 0u);
    };
    auto value = [&](int row, const uint4& raw, float (&x)[8]) {
        widen8<BF16>(raw, x);
        if (rotated) Angles(p, c, at * p.page + row).turn<BF16>(raw, x, p.interleaved);
    };
    // as bits: infinities and NaN come out largest.  Rows outside [lo, hi) do not count: the table's angles at
    // their positions may be anything, and make NaN of their zeros.
    auto largest = [&](uint32_t amax, int row, const float (&x)[8]) {
        if (row < lo || row >= hi) return amax;
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = max(amax, __float_as_uint(x[e]) & 0x7fffffffu);
        return amax;
    };
    auto drop = [](float (&x)[8]) {  // values that are not finite, as 0
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if ((__float_as_uint(x[e]) & 0x7fffffffu) >= 0x7f800000u) x[e] = 0.0f;
    };

    float held[kTwice ? 1 : HELD][8];
    uint32_t amax = 0;
    if constexpr (kTwice) {
        for (int row = lo + r0; row - r0 < hi; row += kRows) {
            float x[8];
            value(row, fetch(row), x);
            amax = largest(amax, row, x);
        }
    } else {
        uint4 raw[HELD];
#pragma unroll
        for (int i = 0; i < HELD; ++i) raw[i] = fetch(i * kRows + r0);
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            value(i * kRows + r0, raw[i], held[i]);
            amax = largest(amax, i * kRows + r0, held[i]);
        }
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    if constexpr (THREADS > 32) {
        __shared__ uint32_t part[THREADS / 32];
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) amax = max(amax, part[w]);
    }
    // the first row with a value that is not finite: an earlier call's, unless this one stores it anew, or this call's
    int bad = kNoRow;
    if (before != before) {
        const uint32_t bits = __float_as_uint(before);
        if ((bits & kNanScaleMask) == kNanScale) {
            before = __uint_as_float(((bits >> 7) & 0xffu) << 23);
            if ((int)(bits & 127u) < lo) bad = bits & 127u;
        }
    }
    const bool clean = amax < 0x7f800000u;  // uniform over the unit
    if (!clean) {  // once more, over the finite values
        amax = 0;
        int mine = kNoRow;
        auto finite = [&](int row, float (&x)[8]) {
            if (row < lo || row >= hi) return;
            if (largest(0, row, x) >= 0x7f800000u) mine = min(mine, row);
            drop(x);
            amax = largest(amax, row, x);
        };
        if constexpr (kTwice) {
            for (int row = lo + r0; row - r0 < hi; row += kRows) {
                float x[8];
                value(row, fetch(row), x);
                finite(row, x);
            }
        } else {
#pragma unroll
            for (int i = 0; i < HELD; ++i) finite(i * kRows + r0, held[i]);
        }
        amax = __reduce_max_sync(0xffffffffu, amax);
        mine = __reduce_min_sync(0xffffffffu, mine);
        if constexpr (THREADS > 32) {
            __shared__ uint32_t part[THREADS / 32];
            __shared__ int row_part[THREADS / 32];
            if ((threadIdx.x & 31) == 0) {
                part[threadIdx.x >> 5] = amax;
                row_part[threadIdx.x >> 5] = mine;
            }
            __syncthreads();
#pragma unroll
            for (int w = 0; w < THREADS / 32; ++w) {
                amax = max(amax, part[w]);
                mine = min(mine, row_part[w]);
            }
        }
        bad = min(bad, mine);
    }
    const float need = scale_for<E4M3>(amax);
    const float scale = before != before ? before : fmaxf(before, need);
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
    auto put = [&](int row, const float (&x)[8]) {
        if (row >= lo && row < hi)
            *reinterpret_cast<uint2*>(codes + (size_t)row * D) = scale > 0.0f ? encode8<E4M3>(x, inv) : make_uint2(0u, 0u);
    };
    if constexpr (kTwice) {
        for (int row = lo + r0; row - r0 < hi; row += kRows) {
            float x[8];
            value(row, fetch(row), x);
            if (!clean) drop(x);
            put(row, x);
        }
    } else {
#pragma unroll
        for (int i = 0; i < HELD; ++i) put(i * kRows + r0, held[i]);
    }
    if (tid == 0) *scale_at = bad == kNoRow ? scale : nan_scale(scale, bad);
}

// (token, kQueryHeads heads) by D / 8 lanes
constexpr int kQueryHeads = 4;
template <bool BF16, int D>
__device__ __forceinline__ void rotate_queries(const AppendParams& p, int64_t item, int64_t items, int chunks)
{
    constexpr int kRowLanes = D / 8;
    const int c = threadIdx.x % kRowLanes;
    const int64_t mine = min(item, items - 1);  // lanes past the end take part in shuffles
    const int t = (int)(mine / chunks), h0 = (int)(mine - (int64_t)t * chunks) * kQueryHeads;
    const uint16_t* src = p.q + (int64_t)t * p.q_stride + 8 * c;
    uint16_t* dst = p.q_out + (int64_t)t * p.hq * D + 8 * c;
    uint4 raw[kQueryHeads];
#pragma unroll
    for (int i = 0; i < kQueryHeads; ++i) raw[i] = h0 + i < p.hq ? __ldcs(reinterpret_cast<const uint4*>(src + (h0 + i) * D)) : make_uint4(0u, 0u, 0u, 0u);
    if (p.rot > 0) {
        // the warp looks for its first token; the others are the same or follow it
        int s = warp_find(p.n_seq, __shfl_sync(0xffffffffu, t, 0), [&](int i) { return cu_at(p.cu_seqlens, i, p.T); });
        while (s + 1 < p.n_seq && cu_at(p.cu_seqlens, s + 1, p.T) <= t) ++s;
        const Angles angles(p, c, past_at(p.past, s) + t - cu_at(p.cu_seqlens, s, p.T));
#pragma unroll
        for (int i = 0; i < kQueryHeads; ++i) {
            float x[8];
            widen8<BF16>(raw[i], x);
            angles.turn<BF16>(raw[i], x, p.interleaved);
            raw[i] = make_uint4(narrow2<BF16>(x[0], x[1]), narrow2<BF16>(x[2], x[3]), narrow2<BF16>(x[4], x[5]), narrow2<BF16>(x[6], x[7]));
        }
    }
    if (item < items)
#pragma unroll
        for (int i = 0; i < kQueryHeads; ++i)
            if (h0 + i < p.hq) __stcs(reinterpret_cast<uint4*>(dst + (h0 + i) * D), raw[i]);
}

// blocks [0, unit_blocks) store pages, the others rotate queries.  Two blocks an SM at least where a lane holds 8
// rows: at its own choice of 134 registers one fits (64 sequences of 1024 tokens, pages of 16, 8 heads: 356 us for 203).
template <bool BF16, bool E4M3, int D, int THREADS, int UNIT, int HELD>
__global__ void __launch_bounds__(THREADS, UNIT == 32 ? 2 : 1024 / THREADS) kv_append_kernel(AppendParams p, int units, int unit_blocks)
{
    pdl_wait();
    pdl_launch_dependents();
    if ((int)blockIdx.x < unit_blocks) {
        const int unit = blockIdx.x * (THREADS / UNIT) + threadIdx.x / UNIT;
        if (unit < units) store_unit<BF16, E4M3, D, UNIT, HELD>(p, unit);
        return;
    }
    const int chunks = (p.hq + kQueryHeads - 1) / kQueryHeads;
    const int64_t item = (int64_t)(blockIdx.x - unit_blocks) * (THREADS / (D / 8)) + threadIdx.x / (D / 8);
    rotate_queries<BF16, D>(p, item, (int64_t)p.T * chunks, chunks);
}

int64_t unit_count(const AppendParams& p) { return ((int64_t)p.T / p.page + 2 * (int64_t)p.n_seq) * p.heads * 2; }

constexpr int64_t kFewUnits = 8 * 152;  // two waves of four blocks on each of this GPU's 152 SMs

template <bool BF16, bool E4M3, int D, int THREADS, int UNIT, int HELD>
cudaError_t launch(const AppendParams& p, cudaStream_t stream)
{
    const int64_t units = unit_count(p), unit_blocks = (units + THREADS / UNIT - 1) / (THREADS / UNIT);
    const int64_t items = (int64_t)p.T * ((p.hq + kQueryHeads - 1) / kQueryHeads), per_block = THREADS / (D / 8);
    const int64_t q_blocks = (items + per_block - 1) / per_block;
    if (units > 0x7fffffff || unit_blocks + q_blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return launch_k(kv_append_kernel<BF16, E4M3, D, THREADS, UNIT, HELD>, dim3((unsigned)(unit_blocks + q_blocks)), dim3(THREADS), 0, stream, true, p,
                    (int)units, (int)unit_blocks);
}

template <bool BF16, bool E4M3, int D>
cudaError_t launch_page(const AppendParams& p, cudaStream_t stream)
{
    // Up to kFewUnits a call takes as long as a unit or two, above as long as all units together.
    //   Sequences that bring a few tokens: a warp per unit, which looks at those rows only.  64 sequences of 12
    //   tokens (pages of 64, 8 heads of 128) took 9.5 us by warps and 11.2 by blocks, of 16 11.8 and 12.0, of 32
    //   17.2 and 18.3; 8 sequences of 1 token 3.2 and 4.2, of 4 the same, of 8 5.5 and 4.0.
    //   Small pages, many units: again a warp, its lanes holding the whole page.  64 sequences of 1024 tokens in
    //   pages of 16 took 349 us by warps, 407 by blocks (366 with rows read twice), 8 of 16 tokens 5.7 and 3.6.
    //   Else a block, 256 threads with up to 4 rows each, 512 for pages of 16 Ki values.
    const bool few = unit_count(p) <= kFewUnits;
    if ((int64_t)p.T <= (few ? 4 : 16) * (int64_t)p.n_seq) return launch<BF16, E4M3, D, 256, 32, 0>(p, stream);
    const int lanes = p.page * (D / 8);
    if (lanes <= 256 && few) return launch<BF16, E4M3, D, 256, 256, 1>(p, stream);
    if (lanes == 128) return launch<BF16, E4M3, D, 256, 32, 4>(p, stream);
    if (lanes == 256) return launch<BF16, E4M3, D, 256, 32, 8>(p, stream);
    if (lanes == 512) return launch<BF16, E4M3, D, 256, 256, 2>(p, stream);
    if (lanes == 1024) return launch<BF16, E4M3, D, 256, 256, 4>(p, stream);
    return launch<BF16, E4M3, D, 512, 512, 4>(p, stream);
}

template <bool BF16, bool E4M3>
cudaError_t launch_dim(const AppendParams& p, cudaStream_t stream)
{
    return p.dim == 64 ? launch_page<BF16, E4M3, 64>(p, stream) : launch_page<BF16, E4M3, 128>(p, stream);
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t stream)
{
    if (p.format == 1) return p.bf16 ? launch_dim<true, true>(p, stream) : launch_dim<false, true>(p, stream);
    return p.bf16 ? launch_dim<true, false>(p, stream) : launch_dim<false, false>(p, stream);
}

}  // namespace gdn
