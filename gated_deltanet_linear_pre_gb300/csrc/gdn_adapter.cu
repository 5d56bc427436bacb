// gdn_adapter.cu -- low-rank adapters of many sequences added to a shared projection's output.
//
//   h[t]     = down[a] x[t]                          (rank values, fp32)
//   y_out[t] = y[t] + scale[a] * up[a]^T h[t]        a = the adapter of t's sequence
//
// Bound by HBM: x and y are read and y_out written once, an adapter's weights
// once for every 128 tokens that use them (from L2 after the first).  Two launches:
//   adapter_down  partial sums of h over ranges of x's channels, fp32, to the workspace
//   adapter_up    the partial sums added in order, the product with up, the sum with y
// A unit of work is 64 channels (of x, of y) for one tile of up to 128 tokens of
// one sequence; each of two CTAs an SM takes an equal range of all units, and cuts
// a tile where its range ends.  Tiles of more than 8 tokens go through the tensor
// cores (tcgen05, 16-bit operands, fp32 sums in TMEM), 64 channels a stage of a
// ring of 128-byte swizzled rows that cp.async fills; the others are sums on the
// CUDA cores straight from global memory, as their weights are read once.
// h enters its product as hi + lo in the weights' type: 16 bits of it in bf16, 21
// of its row's largest in fp16, far below the rounding of y_out.
#include <algorithm>
#include <type_traits>

#include "gdn_kv.cuh"
#include "umma.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;              // tokens
constexpr int kFew = 8;                 // tokens up to which a tile is summed on the CUDA cores, 4 at a time
constexpr int kK = 64;                  // channels of a unit: rows of 128 bytes in shared memory
constexpr int kRow = kK * 2;
constexpr int kCtas = kAdapterCtas;     // two on each of 152 SMs
constexpr int kLeast = 4;               // units that are worth a CTA
constexpr int kTokenBytes = kTile * kRow;

template <int R> constexpr int kStages = R > 64 ? 3 : 4;
template <int R> constexpr int kStageBytes = kTokenBytes + R * kRow;
// two CTAs an SM hold all of its TMEM: never room for a third
template <int R> constexpr size_t kSmem = 1024 + (kStages<R> * kStageBytes<R> < 80 << 10 ? 80 << 10 : kStages<R> * kStageBytes<R>);

// 16 bytes to shared memory, or zeros where there is nothing to read
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there)
{
    const int bytes = there ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// byte offset of 16-byte piece `piece` of a row in a tile swizzled over 128 bytes
__device__ __forceinline__ uint32_t place(int row, int piece) { return row * kRow + ((piece ^ (row & 7)) << 4); }

// Up to kTile tokens of one sequence.  Sequence s owns the slots from cu[s] / kTile + s on; T / kTile + n_seq
// slots cover any batch.
struct Tile {
    int start, n;   // first token, tokens (0: an empty slot)
    int id, rank;   // adapter (-1: none) and its rank
};

__device__ __forceinline__ Tile tile_of(const AdapterParams& p, int slot)
{
    const auto base = [&](int s) { return (int64_t)(cu_at(p.cu_seqlens, s, p.T) / kTile + s); };
    const int s = warp_find(p.n_seq, slot, base);
    const int first = cu_at(p.cu_seqlens, s, p.T), end = cu_at(p.cu_seqlens, s + 1, p.T);
    Tile t;
    const int64_t start = first + (slot - base(s)) * kTile;
    t.n = (int)max((int64_t)0, min((int64_t)kTile, end - start));
    t.start = t.n > 0 ? (int)start : 0;
    t.id = __ldg(p.ids + s);
    if (t.id < 0 || t.id >= p.n_adapters) t.id = -1;
    t.rank = t.id < 0 ? 0 : p.ranks ? min(max(__ldg(p.ranks + t.id), 0), p.rank) : p.rank;
    return t;
}

// What the CTA's threads share for the tensor cores.  Every wait is bounded; after one that has expired the
// rest of the call's waits are passed over and its outputs are invalid, which the CTA records.
struct Shared {
    uint64_t done[4];  // products of a chunk
    uint32_t tmem;
    int expired;
    float factor[kTile];
    float most[2][kTile];
};

__device__ __forceinline__ void wait_done(Shared& sm, uint32_t chunk)
{
    if (*(volatile int*)&sm.expired) return;
    if (!umma::mbar_wait(&sm.done[chunk & 3], (chunk >> 2) & 1)) *(volatile int*)&sm.expired = 1;
}

__device__ __forceinline__ void shared_begin(Shared& sm, int columns)
{
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) umma::mbar_init(&sm.done[i], 1);
        sm.expired = 0;
    }
    if (threadIdx.x < 32) umma::tmem_alloc(&sm.tmem, columns);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
}

// the CTA's record, and clean ones for CTAs that this call does not have
__device__ __forceinline__ void shared_end(Shared& sm, int columns, int32_t* status)
{
    umma::fence_before_sync();
    __syncthreads();
    if (threadIdx.x < 32) umma::tmem_dealloc(sm.tmem, columns);
    if (threadIdx.x == 0) status[blockIdx.x] = sm.expired;
    if (blockIdx.x == 0)
        for (int i = gridDim.x + threadIdx.x; i < kCtas; i += kThreads) status[i] = 0;
}

template <bool BF16, int M, int N>
constexpr uint32_t idesc(bool b_mn_major) { return BF16 ? umma::idesc_bf16(M, N, false, b_mn_major) : umma::idesc_f16(M, N, false, b_mn_major); }

// ---- down -----------------------------------------------------------------------

// h of up to NT tokens, channels [k_lo, k_hi): each warp two rows of `down` at a time
template <bool BF16, int NT>
__device__ __forceinline__ void down_few(const AdapterParams& p, const Tile& t, int k_lo, int k_hi, float* h)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kAhead = NT > 2 ? 2 : 4;  // steps of 256 channels loaded ahead: what 128 registers hold
    const uint16_t* x = p.x + (size_t)t.start * p.x_stride;
    for (int j = warp * 2; j < t.rank; j += kThreads / 16) {
        const uint16_t* w0 = p.down + ((size_t)t.id * p.rank + j) * p.d_in;
        const uint16_t* w1 = j + 1 < t.rank ? w0 + p.d_in : w0;
        float acc[2][NT] = {};
        for (int k0 = k_lo + lane * 8; k0 < k_hi; k0 += kAhead * 256) {
            uint4 a[kAhead], b[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (k0 + i * 256 < k_hi) {
                    a[i] = __ldg(reinterpret_cast<const uint4*>(w0 + k0 + i * 256));
                    b[i] = __ldg(reinterpret_cast<const uint4*>(w1 + k0 + i * 256));
                }
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (k0 + i * 256 < k_hi) {
                    float wa[8], wb[8];
                    widen8<BF16>(a[i], wa);
                    widen8<BF16>(b[i], wb);
#pragma unroll
                    for (int q = 0; q < NT; ++q) {
                        float v[8];
                        widen8<BF16>(__ldg(reinterpret_cast<const uint4*>(x + (size_t)min(q, t.n - 1) * p.x_stride + k0 + i * 256)), v);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            acc[0][q] = fmaf(wa[e], v[e], acc[0][q]);
                            acc[1][q] = fmaf(wb[e], v[e], acc[1][q]);
                        }
                    }
                }
        }
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float sum = warp_sum(acc[i][q]);
                if (lane == 0 && q < t.n && j + i < t.rank) h[(size_t)q * p.rank + j + i] = sum;
            }
    }
}

template <bool BF16, int R>
__device__ __forceinline__ void down_tile(const AdapterParams& p, const Tile& t, int c_lo, int c_hi, float* h, Shared& sm, uint32_t ring, uint32_t& at)
{
    constexpr int kS = kStages<R>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint16_t* x = p.x + (size_t)t.start * p.x_stride;
    const uint16_t* w = p.down + (size_t)t.id * p.rank * p.d_in;
    const uint32_t first = at;
    const auto load = [&](int c) {
        if (c < c_hi) {
            const uint32_t stage = ring + (first + c - c_lo) % kS * kStageBytes<R>;
            const int k = c * kK + (tid & 7) * 8;
            const bool there = k < p.d_in;
            for (int row = tid >> 3; row < t.n; row += kThreads / 8)
                copy16(stage + place(row, tid & 7), there ? x + (size_t)row * p.x_stride + k : p.x, there);
            for (int row = tid >> 3; row < t.rank; row += kThreads / 8)
                copy16(stage + kTokenBytes + place(row, tid & 7), there ? w + (size_t)row * p.d_in + k : p.x, there);
        }
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < kS - 1; ++i) load(c_lo + i);
    for (int c = c_lo; c < c_hi; ++c, ++at) {
        copies_wait<kS - 2>();
        umma::fence_proxy_async();
        __syncthreads();
        if (warp == 0) {
            umma::fence_after_sync();
            if (umma::elect_one()) {
                const uint32_t stage = ring + at % kS * kStageBytes<R>;
                const uint64_t da = umma::desc_sw128(stage, 16, 1024), db = umma::desc_sw128(stage + kTokenBytes, 16, 1024);
#pragma unroll
                for (int k = 0; k < kK / 16; ++k) umma::mma_bf16(sm.tmem, da + 2 * k, db + 2 * k, idesc<BF16, 128, R>(false), c > c_lo || k > 0);
                umma::commit(&sm.done[at & 3]);
            }
            __syncwarp();
        }
        // the stage of the chunk before this one is free once its products are done
        if (c > c_lo) wait_done(sm, at - 1);
        load(c + kS - 1);
    }
    wait_done(sm, at - 1);
    copies_wait<0>();
    umma::fence_after_sync();
    const int row = (warp & 3) * 32 + lane;
#pragma unroll
    for (int j = 0; j < R / 16; ++j)
        if ((j & 1) == warp >> 2 && j * 16 < t.rank) {
            float v[16];
            umma::tmem_ld16(sm.tmem + ((warp & 3) * 32 << 16) + j * 16, v);
            umma::tmem_wait_ld();
            float4* to = reinterpret_cast<float4*>(h + (size_t)row * p.rank + j * 16);
            if (row < t.n) {
                to[0] = make_float4(v[0], v[1], v[2], v[3]);
                to[1] = make_float4(v[4], v[5], v[6], v[7]);
                if (j * 16 + 8 < p.rank) {  // a row holds a multiple of 8
                    to[2] = make_float4(v[8], v[9], v[10], v[11]);
                    to[3] = make_float4(v[12], v[13], v[14], v[15]);
                }
            }
        }
    umma::fence_before_sync();
    __syncthreads();  // TMEM and the ring are free
}

template <bool BF16, int R>
__global__ void __launch_bounds__(kThreads, 2) adapter_down_kernel(const __grid_constant__ AdapterParams p)
{
    extern __shared__ unsigned char smem[];
    __shared__ Shared sm;
    constexpr int kColumns = R < 32 ? 32 : R;
    const uint32_t ring = (umma::smem_u32(smem) + 1023) & ~1023u;
    // In this order.  Nobody waits here for another kernel while it holds TMEM that the other has yet to get, and
    // the kernel behind this one, which starts when all CTAs have come by, may read what earlier launches wrote.
    pdl_wait();
    shared_begin(sm, kColumns);
    pdl_launch_dependents();
    uint32_t at = 0;  // chunks so far
    const int64_t total = (int64_t)p.slots * p.chunks_in, end = min(total, (int64_t)(blockIdx.x + 1) * p.share_in);
    for (int64_t u = (int64_t)blockIdx.x * p.share_in; u < end;) {
        const int slot = (int)(u / p.chunks_in), c_lo = (int)(u - (int64_t)slot * p.chunks_in);
        const int c_hi = (int)min((int64_t)p.chunks_in, c_lo + end - u);
        u += c_hi - c_lo;
        const Tile t = tile_of(p, slot);
        if (t.n == 0 || t.rank == 0) continue;
        const int part = blockIdx.x - (int)((int64_t)slot * p.chunks_in / p.share_in);
        float* h = p.h + ((size_t)part * p.T + t.start) * p.rank;
        if (t.n <= kFew) {
            const int k_lo = c_lo * kK, k_hi = min(p.d_in, c_hi * kK);
            for (Tile q = t; q.n > 0; q.start += 4, q.n -= 4, h += 4 * p.rank) {
                if (q.n == 1) down_few<BF16, 1>(p, q, k_lo, k_hi, h);
                else if (q.n == 2) down_few<BF16, 2>(p, q, k_lo, k_hi, h);
                else down_few<BF16, 4>(p, q, k_lo, k_hi, h);
            }
        } else {
            down_tile<BF16, R>(p, t, c_lo, c_hi, h, sm, ring, at);
        }
    }
    shared_end(sm, kColumns, p.status);
}

// ---- up -------------------------------------------------------------------------

constexpr int kColumnD = 128;  // TMEM: h in the first R columns, the products of two chunks from here on

// y_out of up to NT tokens, channels [o_lo, o_hi): each thread 8 channels at a time
template <bool BF16, int NT>
__device__ __forceinline__ void up_few(const AdapterParams& p, const Tile& t, int o_lo, int o_hi, const float* h, float scale)
{
    constexpr int kAhead = NT > 2 ? 4 : 8;  // rows of `up` loaded ahead: what 128 registers hold
    const uint16_t* w = p.up + (size_t)t.id * p.rank * p.d_out;
    for (int o = o_lo + threadIdx.x * 8; o < o_hi; o += kThreads * 8) {
        uint4 y[NT];
#pragma unroll
        for (int q = 0; q < NT; ++q) y[q] = __ldcs(reinterpret_cast<const uint4*>(p.y + (size_t)(t.start + min(q, t.n - 1)) * p.y_stride + o));
        float acc[NT][8] = {};
        for (int j = 0; j < t.rank; j += kAhead) {
            uint4 v[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) v[i] = j + i < t.rank ? __ldg(reinterpret_cast<const uint4*>(w + (size_t)(j + i) * p.d_out + o)) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                float f[8];
                widen8<BF16>(v[i], f);
#pragma unroll
                for (int q = 0; q < NT; ++q)
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[q][e] = fmaf(h[q * p.rank + j + i], f[e], acc[q][e]);
            }
        }
#pragma unroll
        for (int q = 0; q < NT; ++q)
            if (q < t.n) {
                float f[8];
                widen8<BF16>(y[q], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = fmaf(scale, acc[q][e], f[e]);
                __stcs(reinterpret_cast<uint4*>(p.y_out + (size_t)(t.start + q) * p.out_stride + o),
                       make_uint4(narrow2<BF16>(f[0], f[1]), narrow2<BF16>(f[2], f[3]), narrow2<BF16>(f[4], f[5]), narrow2<BF16>(f[6], f[7])));
            }
    }
}

// two values as hi + lo in the weights' type; what is not finite goes into hi alone
template <bool BF16>
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo)
{
    hi = narrow2<BF16>(a, b);
    float ha, hb;
    if (BF16) {
        ha = __uint_as_float(hi << 16);
        hb = __uint_as_float(hi & 0xffff0000u);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        ha = f.x;
        hb = f.y;
    }
    lo = narrow2<BF16>(isfinite(ha) ? a - ha : 0.0f, isfinite(hb) ? b - hb : 0.0f);
}

template <int N>
__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t (&v)[N])
{
    if constexpr (N == 4)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
    else if constexpr (N == 8)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                     "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    else
        umma::tmem_st16(at, v);
}

// h of a tile as the products' first operand: hi in TMEM columns [0, R / 2), lo behind it, two values a column.
// Two threads a row, each half of its columns.
template <bool BF16, int R>
__device__ __forceinline__ void operand(const AdapterParams& p, const Tile& t, int parts, Shared& sm)
{
    constexpr int kMine = R / 2, kAtOnce = kMine < 32 ? kMine : 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = warp >> 2, row = (warp & 3) * 32 + lane;
    const int col = half * kMine;
    float v[kMine];
#pragma unroll
    for (int j = 0; j < kMine; ++j) v[j] = 0.0f;
    if (row < t.n)
        for (int s = 0; s < parts; ++s) {
            const float4* src = reinterpret_cast<const float4*>(p.h + ((size_t)s * p.T + t.start + row) * p.rank + col);
#pragma unroll
            for (int j = 0; j < kMine; j += 4)
                if (col + j < t.rank) {  // a row holds a multiple of 8 values
                    const float4 f = src[j / 4];
                    v[j] += f.x;
                    v[j + 1] += f.y;
                    v[j + 2] += f.z;
                    v[j + 3] += f.w;
                }
        }
#pragma unroll
    for (int j = 0; j < kMine; ++j)
        if (col + j >= t.rank) v[j] = 0.0f;
    float inv = 1.0f, factor = __ldg(p.scales + t.id);
    if (!BF16) {
        // a row's largest value to [1, 2): fp16 has 5 bits of exponent
        float most = 0.0f;
#pragma unroll
        for (int j = 0; j < kMine; ++j) most = fmaxf(most, fabsf(v[j]));
        sm.most[half][row] = most;
        __syncthreads();
        most = fmaxf(sm.most[0][row], sm.most[1][row]);
        const int exponent = min(max((int)(__float_as_uint(most) >> 23) - 127, -126), 126);
        inv = __uint_as_float((uint32_t)(127 - exponent) << 23);
        factor *= __uint_as_float((uint32_t)(127 + exponent) << 23);
    }
    if (half == 0) sm.factor[row] = factor;
    const uint32_t to = sm.tmem + ((warp & 3) * 32 << 16) + col / 2;
#pragma unroll
    for (int j = 0; j < kMine; j += kAtOnce) {
        uint32_t hi[kAtOnce / 2], lo[kAtOnce / 2];
#pragma unroll
        for (int i = 0; i < kAtOnce / 2; ++i) split2<BF16>(v[j + 2 * i] * inv, v[j + 2 * i + 1] * inv, hi[i], lo[i]);
        tmem_st(to + j / 2, hi);
        tmem_st(to + R / 2 + j / 2, lo);
    }
    umma::tmem_wait_st();
    umma::fence_before_sync();
    __syncthreads();
}

template <bool BF16, int R>
__device__ __forceinline__ void up_tile(const AdapterParams& p, const Tile& t, int parts, int c_lo, int c_hi, Shared& sm, unsigned char* ring, uint32_t& at,
                                        bool& waited)
{
    constexpr int kS = kStages<R>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, half = warp >> 2;
    const int steps = (t.rank + 15) / 16;
    const uint32_t base = umma::smem_u32(ring);
    const uint16_t* w = p.up + (size_t)t.id * p.rank * p.d_out;
    const uint16_t* y = p.y + (size_t)t.start * p.y_stride;
    uint16_t* out = p.y_out + (size_t)t.start * p.out_stride;
    const uint32_t first = at;
    const auto load = [&](int c) {
        if (c < c_hi) {
            const uint32_t stage = base + (first + c - c_lo) % kS * kStageBytes<R>;
            const int o = c * kK + (tid & 7) * 8;
            const bool there = o < p.d_out;
            for (int row = tid >> 3; row < t.n; row += kThreads / 8)
                copy16(stage + place(row, tid & 7), there ? y + (size_t)row * p.y_stride + o : p.y, there);
            // rows behind the rank: zeros, as what was there may not be finite
            for (int row = tid >> 3; row < steps * 16; row += kThreads / 8) {
                const bool mine = there && row < t.rank;
                copy16(stage + kTokenBytes + place(row, tid & 7), mine ? w + (size_t)row * p.d_out + o : p.y, mine);
            }
        }
        copies_commit();
    };
    // y plus the products of chunk c, the `n`th of all: this warp's 32 rows and 32 channels
    const auto finish = [&](int c, uint32_t n) {
        wait_done(sm, n);
        umma::fence_after_sync();
        float v[32];
        umma::tmem_ld32(sm.tmem + ((warp & 3) * 32 << 16) + kColumnD + (n & 1) * kK + half * 32, v);
        umma::tmem_wait_ld();
        unsigned char* tile = ring + n % kS * kStageBytes<R>;
        const int row = (warp & 3) * 32 + lane;
        const float factor = sm.factor[row];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint4* q = reinterpret_cast<uint4*>(tile + place(row, half * 4 + i));
            float f[8];
            widen8<BF16>(*q, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = fmaf(factor, v[i * 8 + e], f[e]);
            *q = make_uint4(narrow2<BF16>(f[0], f[1]), narrow2<BF16>(f[2], f[3]), narrow2<BF16>(f[4], f[5]), narrow2<BF16>(f[6], f[7]));
        }
        __syncwarp();
        const int piece = half * 4 + (lane & 3), o = c * kK + piece * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (warp & 3) * 32 + i * 8 + (lane >> 2);
            if (r < t.n && o < p.d_out) __stcs(reinterpret_cast<uint4*>(out + (size_t)r * p.out_stride + o), *reinterpret_cast<const uint4*>(tile + place(r, piece)));
        }
        umma::fence_before_sync();
    };
#pragma unroll
    for (int i = 0; i < kS - 2; ++i) load(c_lo + i);
    if (!waited) pdl_wait();
    waited = true;
    operand<BF16, R>(p, t, parts, sm);
    for (int c = c_lo; c < c_hi; ++c, ++at) {
        copies_wait<kS - 3>();
        umma::fence_proxy_async();
        __syncthreads();
        if (warp == 0) {
            umma::fence_after_sync();
            if (umma::elect_one()) {
                const uint32_t d = sm.tmem + kColumnD + (at & 1) * kK;
                const uint64_t db = umma::desc_sw128(base + at % kS * kStageBytes<R> + kTokenBytes, 16, 1024);
                for (int k = 0; k < steps; ++k) umma::mma_ts(d, sm.tmem + 8 * k, db + k * (2048 >> 4), idesc<BF16, 128, kK>(true), k > 0);
                for (int k = 0; k < steps; ++k) umma::mma_ts(d, sm.tmem + R / 2 + 8 * k, db + k * (2048 >> 4), idesc<BF16, 128, kK>(true), 1);
                umma::commit(&sm.done[at & 3]);
            }
            __syncwarp();
        }
        // every warp is past the chunk before the last one: its stage is free
        load(c + kS - 2);
        if (c > c_lo) finish(c - 1, at - 1);
    }
    finish(c_hi - 1, at - 1);
    copies_wait<0>();
    __syncthreads();  // TMEM and the ring are free
}

template <bool BF16, int R>
__global__ void __launch_bounds__(kThreads, 2) adapter_up_kernel(const __grid_constant__ AdapterParams p)
{
    extern __shared__ unsigned char smem[];
    __shared__ Shared sm;
    __shared__ float few[kFew * R];
    constexpr int kColumns = 256;
    unsigned char* ring = smem + ((1024 - (umma::smem_u32(smem) & 1023)) & 1023);
    // all of adapter_down's CTAs have their TMEM, as those of this kernel when the next one starts
    shared_begin(sm, kColumns);
    pdl_launch_dependents();
    // y, up and the batch were there before adapter_down began; only its own sums have to be waited for
    bool waited = false;
    uint32_t at = 0;
    const int64_t total = (int64_t)p.slots * p.chunks_out, end = min(total, (int64_t)(blockIdx.x + 1) * p.share_out);
    for (int64_t u = (int64_t)blockIdx.x * p.share_out; u < end;) {
        const int slot = (int)(u / p.chunks_out), c_lo = (int)(u - (int64_t)slot * p.chunks_out);
        const int c_hi = (int)min((int64_t)p.chunks_out, c_lo + end - u);
        u += c_hi - c_lo;
        const Tile t = tile_of(p, slot);
        const int64_t first = (int64_t)slot * p.chunks_in;
        const int parts = (int)((first + p.chunks_in - 1) / p.share_in - first / p.share_in) + 1;
        const int o_lo = c_lo * kK, o_hi = min(p.d_out, c_hi * kK);
        if (t.rank > 0 && t.n > kFew) {
            up_tile<BF16, R>(p, t, parts, c_lo, c_hi, sm, ring, at, waited);
            continue;
        }
        if (!waited) pdl_wait();
        waited = true;
        if (t.rank > 0 && t.n > 0) {
            for (int i = threadIdx.x; i < t.n * p.rank; i += kThreads) {
                float v = 0.0f;
                if (i % p.rank < t.rank)
                    for (int s = 0; s < parts; ++s) v += p.h[((size_t)s * p.T + t.start) * p.rank + i];
                few[i] = v;
            }
            for (int i = t.n * p.rank + threadIdx.x; i < kFew * p.rank; i += kThreads) few[i] = 0.0f;
            __syncthreads();
            const float scale = __ldg(p.scales + t.id);
            const float* h = few;
            for (Tile q = t; q.n > 0; q.start += 4, q.n -= 4, h += 4 * p.rank) {
                if (q.n == 1) up_few<BF16, 1>(p, q, o_lo, o_hi, h, scale);
                else if (q.n == 2) up_few<BF16, 2>(p, q, o_lo, o_hi, h, scale);
                else up_few<BF16, 4>(p, q, o_lo, o_hi, h, scale);
            }
            __syncthreads();
        } else if (p.y_out != p.y) {
            const int vectors = (o_hi - o_lo) / 8;
            for (int i = threadIdx.x; i < t.n * vectors; i += kThreads) {
                const int row = t.start + i / vectors, o = o_lo + i % vectors * 8;
                __stcs(reinterpret_cast<uint4*>(p.y_out + (size_t)row * p.out_stride + o), __ldcs(reinterpret_cast<const uint4*>(p.y + (size_t)row * p.y_stride + o)));
            }
        }
    }
    if (!waited) pdl_wait();
    shared_end(sm, kColumns, p.status + kCtas);
}

template <bool BF16, int R>
cudaError_t launch_rank(const AdapterParams& p, unsigned ctas_in, unsigned ctas_out, cudaStream_t stream)
{
    cudaError_t e = cudaFuncSetAttribute(adapter_down_kernel<BF16, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem<R>);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(adapter_up_kernel<BF16, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem<R>);
    if (e == cudaSuccess) e = launch_k(adapter_down_kernel<BF16, R>, dim3(ctas_in), dim3(kThreads), kSmem<R>, stream, true, p);
    if (e == cudaSuccess) e = launch_k(adapter_up_kernel<BF16, R>, dim3(ctas_out), dim3(kThreads), kSmem<R>, stream, true, p);
    return e;
}

int64_t slots_of(int n_seq, int T) { return (int64_t)T / kTile + n_seq; }
int chunks_of(int width) { return (width + kK - 1) / kK; }
int64_t share_of(int64_t units) { return std::max<int64_t>(kLeast, (units + kCtas - 1) / kCtas); }
constexpr size_t kHeader = (2 * kCtas * 4 + 255) / 256 * 256;

}  // namespace

size_t adapter_workspace_bytes(int n_seq, int T, int rank, int d_in)
{
    // consecutive units of a tile lie in at most so many shares
    const int64_t chunks = chunks_of(d_in), share = share_of(slots_of(n_seq, T) * chunks), parts = (chunks + share - 2) / share + 1;
    return kHeader + (size_t)parts * T * rank * 4;
}

cudaError_t launch_adapter(AdapterParams p, void* workspace, cudaStream_t stream)
{
    p.slots = (int)slots_of(p.n_seq, p.T);
    p.chunks_in = chunks_of(p.d_in);
    p.chunks_out = chunks_of(p.d_out);
    const int64_t units_in = (int64_t)p.slots * p.chunks_in, units_out = (int64_t)p.slots * p.chunks_out;
    p.share_in = share_of(units_in);
    p.share_out = share_of(units_out);
    p.status = static_cast<int32_t*>(workspace);
    p.h = reinterpret_cast<float*>(static_cast<char*>(workspace) + kHeader);
    const unsigned ctas_in = (unsigned)((units_in + p.share_in - 1) / p.share_in), ctas_out = (unsigned)((units_out + p.share_out - 1) / p.share_out);
    const auto launch = [&](auto bf16) {
        constexpr bool kBf16 = decltype(bf16)::value;
        if (p.rank <= 16) return launch_rank<kBf16, 16>(p, ctas_in, ctas_out, stream);
        if (p.rank <= 32) return launch_rank<kBf16, 32>(p, ctas_in, ctas_out, stream);
        if (p.rank <= 64) return launch_rank<kBf16, 64>(p, ctas_in, ctas_out, stream);
        return launch_rank<kBf16, 128>(p, ctas_in, ctas_out, stream);
    };
    return p.bf16 ? launch(std::true_type{}) : launch(std::false_type{});
}

}  // namespace gdn
