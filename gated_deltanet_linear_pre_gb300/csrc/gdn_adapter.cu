// gdn_adapter.cu -- low-rank adapters of many sequences added to a shared projection's output.
//
//   h[t]     = down[a] x[t]                          (rank values, fp32)
//   y_out[t] = y[t] + scale[a] * up[a]^T h[t]        a = the adapter of t's sequence
//
// Bound by HBM: x and y are read and y_out written once, and every adapter's
// weights once for each tile of 64 tokens that uses them (from L2 after the
// first).  Two launches:
//   adapter_down  a (tile of a sequence's tokens, range of x's channels): partial
//                 sums of h, in fp32, to the workspace
//   adapter_up    a (tile, range of y's channels): the partial sums added in
//                 order, the product with up, and the sum with y
// Products are mma.sync on 16-bit operands with fp32 sums.  h enters the second
// product as hi + lo in the weights' type (16 bits of h in bf16, 21 of its row's
// largest in fp16), so its rounding is far below that of y_out.
#include <type_traits>

#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = 64;    // tokens
constexpr int kK = 64;       // channels of a stage: rows of 128 bytes in shared memory
constexpr int kRow = kK * 2;
constexpr int kStages = 4;

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16 bytes to shared memory, or zeros where there is nothing to read
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there)
{
    const int bytes = there ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// byte offset of 16-byte piece `piece` of a row: rows 8 apart share banks, the others do not
__device__ __forceinline__ uint32_t place(int row, int piece) { return row * kRow + ((piece ^ (row & 7)) << 4); }

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}

template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A block's tile: up to kTile tokens of one sequence.  Sequence s owns the slots from cu[s] / kTile + s on;
// T / kTile + n_seq slots cover any batch.
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

// The four warps over a tile's 16-token rows: m of them take different rows, the others share the rest of the work
__device__ __forceinline__ int row_groups(int n) { return n <= 16 ? 1 : n <= 32 ? 2 : 4; }

template <bool BF16, int R>
__global__ void __launch_bounds__(kThreads) adapter_down_kernel(const __grid_constant__ AdapterParams p)
{
    extern __shared__ __align__(128) unsigned char smem[];
    constexpr int kStage = (kTile + R) * kRow;
    pdl_wait();
    // behind the wait: whatever starts now may read what earlier launches wrote
    pdl_launch_dependents();
    const Tile t = tile_of(p, blockIdx.x);
    if (t.n == 0 || t.rank == 0) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int k_lo = blockIdx.y * p.split_k, k_hi = min(p.d_in, k_lo + p.split_k);
    const int chunks = (k_hi - k_lo + kK - 1) / kK;
    const uint32_t base = smem_u32(smem);
    const uint16_t* x = p.x + (size_t)t.start * p.x_stride;
    const uint16_t* w = p.down + (size_t)t.id * p.rank * p.d_in;

    const auto load = [&](int chunk) {
        if (chunk < chunks) {
            const uint32_t at = base + (chunk % kStages) * kStage;
            const int k = k_lo + chunk * kK + (tid & 7) * 8;
            const bool there = k < k_hi;
            for (int row = tid >> 3; row < t.n; row += kThreads / 8)
                copy16(at + place(row, tid & 7), there ? x + (size_t)row * p.x_stride + k : p.x, there);
            for (int row = tid >> 3; row < t.rank; row += kThreads / 8)
                copy16(at + kTile * kRow + place(row, tid & 7), there ? w + (size_t)row * p.d_in + k : p.x, there);
        }
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) load(i);

    const int groups = row_groups(t.n), m0 = warp % groups * 16, kg = warp / groups, kgs = 4 / groups;
    float acc[R / 8][4];
#pragma unroll
    for (int j = 0; j < R / 8; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
    for (int chunk = 0; chunk < chunks; ++chunk) {
        copies_wait<kStages - 2>();
        __syncthreads();
        load(chunk + kStages - 1);
        const uint32_t at = base + (chunk % kStages) * kStage;
        for (int kk = kg; kk < kK / 16; kk += kgs) {
            uint32_t a[4];
            ldmatrix4(a, at + place(m0 + (lane & 15), kk * 2 + (lane >> 4)));
#pragma unroll
            for (int j = 0; j < R / 16; ++j) {
                if (j * 16 < t.rank) {
                    uint32_t b[4];
                    ldmatrix4(b, at + kTile * kRow + place(j * 16 + (lane & 7) + (lane >> 4 << 3), kk * 2 + (lane >> 3 & 1)));
                    mma<BF16>(acc[2 * j], a, b[0], b[1]);
                    mma<BF16>(acc[2 * j + 1], a, b[2], b[3]);
                }
            }
        }
    }
    // warps that shared rows add up in shared memory, in order
    if (kgs > 1) {
        copies_wait<0>();
        float* part = reinterpret_cast<float*>(smem);  // [3 warps][R / 8][4][32]
        __syncthreads();
        if (kg > 0) {
#pragma unroll
            for (int j = 0; j < R / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) part[((warp - groups) * (R / 2) + j * 4 + e) * 32 + lane] = acc[j][e];
        }
        __syncthreads();
        if (kg > 0) return;
        for (int g = 1; g < kgs; ++g)
#pragma unroll
            for (int j = 0; j < R / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][e] += part[(((g - 1) * groups + warp) * (R / 2) + j * 4 + e) * 32 + lane];
    }
    float* h = p.h + ((size_t)blockIdx.y * p.T + t.start) * p.rank;
#pragma unroll
    for (int j = 0; j < R / 8; ++j) {
        const int col = j * 8 + (lane & 3) * 2;
        if (j * 8 < t.rank) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int row = m0 + half * 8 + (lane >> 2);
                if (row < t.n) *reinterpret_cast<float2*>(h + (size_t)row * p.rank + col) = make_float2(acc[j][half * 2], acc[j][half * 2 + 1]);
            }
        }
    }
}

__device__ __forceinline__ float max4(float v)
{
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
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

template <bool BF16, int R>
__global__ void __launch_bounds__(kThreads) adapter_up_kernel(const __grid_constant__ AdapterParams p)
{
    extern __shared__ __align__(128) unsigned char smem[];
    constexpr int kStage = (kTile + R) * kRow;
    pdl_launch_dependents();
    // y, up and the batch were there before adapter_down began; its own sums are waited for below
    const Tile t = tile_of(p, blockIdx.x);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int o_lo = blockIdx.y * p.split_o, o_hi = min(p.d_out, o_lo + p.split_o);
    if (t.n == 0 || t.rank == 0) {
        pdl_wait();
        if (p.y_out == p.y) return;
        for (int row = 0; row < t.n; ++row)
            for (int o = o_lo + tid * 8; o < o_hi; o += kThreads * 8)
                __stcs(reinterpret_cast<uint4*>(p.y_out + (size_t)(t.start + row) * p.out_stride + o),
                       __ldcs(reinterpret_cast<const uint4*>(p.y + (size_t)(t.start + row) * p.y_stride + o)));
        return;
    }
    const int chunks = (o_hi - o_lo + kK - 1) / kK, steps = (t.rank + 15) / 16;
    const uint32_t base = smem_u32(smem);
    const uint16_t* w = p.up + (size_t)t.id * p.rank * p.d_out;
    const uint16_t* y = p.y + (size_t)t.start * p.y_stride;
    uint16_t* out = p.y_out + (size_t)t.start * p.out_stride;

    const auto load = [&](int chunk) {
        if (chunk < chunks) {
            const uint32_t at = base + (chunk % kStages) * kStage;
            const int o = o_lo + chunk * kK + (tid & 7) * 8;
            const bool there = o < o_hi;
            for (int row = tid >> 3; row < t.n; row += kThreads / 8)
                copy16(at + place(row, tid & 7), there ? y + (size_t)row * p.y_stride + o : p.y, there);
            // rows behind the rank: zeros, as what was there may not be finite
            for (int row = tid >> 3; row < steps * 16; row += kThreads / 8) {
                const bool mine = there && row < t.rank;
                copy16(at + kTile * kRow + place(row, tid & 7), mine ? w + (size_t)row * p.d_out + o : p.y, mine);
            }
        }
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) load(i);

    const int groups = row_groups(t.n), m0 = warp % groups * 16, og = warp / groups, ogs = 4 / groups;
    pdl_wait();
    // h of this warp's 16 tokens, as the product's first operand
    uint32_t hi[R / 16][4], lo[R / 16][4];
    float factor[2];
    {
        float h[R / 16][8];  // [step][half * 4 + e]: rows m0 + lane / 4 + 8 * half, columns 2 (lane & 3) + {0, 1, 8, 9}
#pragma unroll
        for (int k = 0; k < R / 16; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) h[k][e] = 0.0f;
        for (int s = 0; s < p.splits; ++s) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int row = m0 + half * 8 + (lane >> 2);
                const float* src = p.h + ((size_t)s * p.T + t.start + row) * p.rank;
#pragma unroll
                for (int k = 0; k < R / 16; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int col = k * 16 + e * 8 + (lane & 3) * 2;
                        if (row < t.n && col < t.rank) {
                            const float2 v = *reinterpret_cast<const float2*>(src + col);
                            h[k][half * 4 + e * 2] += v.x;
                            if (col + 1 < t.rank) h[k][half * 4 + e * 2 + 1] += v.y;
                        }
                    }
            }
        }
        const float scale = __ldg(p.scales + t.id);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float inv = 1.0f;
            factor[half] = scale;
            if (!BF16) {
                // a row's largest value to [1, 2): fp16 has 5 bits of exponent
                float most = 0.0f;
#pragma unroll
                for (int k = 0; k < R / 16; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) most = fmaxf(most, fabsf(h[k][half * 4 + e]));
                most = max4(most);
                const int exponent = min(max((int)(__float_as_uint(most) >> 23) - 127, -126), 126);
                inv = __uint_as_float((uint32_t)(127 - exponent) << 23);
                factor[half] = scale * __uint_as_float((uint32_t)(127 + exponent) << 23);
            }
#pragma unroll
            for (int k = 0; k < R / 16; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    split2<BF16>(h[k][half * 4 + e * 2] * inv, h[k][half * 4 + e * 2 + 1] * inv, hi[k][e * 2 + half], lo[k][e * 2 + half]);
        }
    }
    const int per = kK / 8 / ogs;  // 8-channel pieces of a chunk that this warp takes: 8, 4 or 2
    for (int chunk = 0; chunk < chunks; ++chunk) {
        copies_wait<kStages - 2>();
        __syncthreads();
        load(chunk + kStages - 1);
        const uint32_t at = base + (chunk % kStages) * kStage;
        unsigned char* tile = smem + (chunk % kStages) * kStage;
        for (int j = og * per; j < (og + 1) * per; j += 2) {
            float acc[2][4] = {};
#pragma unroll
            for (int k = 0; k < R / 16; ++k) {
                if (k < steps) {
                    uint32_t b[4];
                    ldmatrix4_t(b, at + kTile * kRow + place(k * 16 + (lane & 15), j + (lane >> 4)));
                    mma<BF16>(acc[0], hi[k], b[0], b[1]);
                    mma<BF16>(acc[1], hi[k], b[2], b[3]);
                    mma<BF16>(acc[0], lo[k], b[0], b[1]);
                    mma<BF16>(acc[1], lo[k], b[2], b[3]);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int row = m0 + half * 8 + (lane >> 2);
                    uint32_t* v = reinterpret_cast<uint32_t*>(tile + place(row, j + i) + (lane & 3) * 4);
                    float a, b;
                    if (BF16) {
                        a = __uint_as_float(*v << 16);
                        b = __uint_as_float(*v & 0xffff0000u);
                    } else {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(v));
                        a = f.x;
                        b = f.y;
                    }
                    *v = narrow2<BF16>(fmaf(factor[half], acc[i][half * 2], a), fmaf(factor[half], acc[i][half * 2 + 1], b));
                }
        }
        __syncwarp();
        // this warp's rows and pieces, 16 bytes a lane
        const int o = o_lo + chunk * kK;
        for (int i = lane; i < 16 * per; i += 32) {
            const int row = m0 + i / per, piece = og * per + i % per;
            if (row < t.n && o + piece * 8 < o_hi)
                __stcs(reinterpret_cast<uint4*>(out + (size_t)row * p.out_stride + o + piece * 8), *reinterpret_cast<const uint4*>(tile + place(row, piece)));
        }
    }
}

template <bool BF16, int R>
cudaError_t launch_rank(const AdapterParams& p, unsigned tiles, cudaStream_t stream)
{
    constexpr size_t smem = (size_t)kStages * (kTile + R) * kRow;
    cudaError_t e = cudaFuncSetAttribute(adapter_down_kernel<BF16, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(adapter_up_kernel<BF16, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) e = launch_k(adapter_down_kernel<BF16, R>, dim3(tiles, (unsigned)p.splits), dim3(kThreads), smem, stream, true, p);
    if (e == cudaSuccess)
        e = launch_k(adapter_up_kernel<BF16, R>, dim3(tiles, (unsigned)((p.d_out + p.split_o - 1) / p.split_o)), dim3(kThreads), smem, stream, true, p);
    return e;
}

int64_t tiles_of(int n_seq, int T) { return (int64_t)T / kTile + n_seq; }

// ranges of `width` channels for a block each, in steps of kK, so that about four blocks an SM share the work
int split_of(int64_t tiles, int width, int least)
{
    const int64_t want = tiles > 0 ? (152 * 4 + tiles - 1) / tiles : 1;
    const int64_t most = (width + least - 1) / least, parts = want < most ? want : most;
    return (int)((width + parts * kK - 1) / (parts * kK)) * kK;
}

}  // namespace

size_t adapter_workspace_bytes(int n_seq, int T, int rank, int d_in)
{
    const int split = split_of(tiles_of(n_seq, T), d_in, 256);
    return (size_t)((d_in + split - 1) / split) * T * rank * 4;
}

cudaError_t launch_adapter(AdapterParams p, cudaStream_t stream)
{
    const int64_t tiles = tiles_of(p.n_seq, p.T);
    p.split_k = split_of(tiles, p.d_in, 256);
    p.splits = (p.d_in + p.split_k - 1) / p.split_k;
    p.split_o = split_of(tiles, p.d_out, 256);
    const auto launch = [&](auto bf16) {
        constexpr bool kBf16 = decltype(bf16)::value;
        if (p.rank <= 16) return launch_rank<kBf16, 16>(p, (unsigned)tiles, stream);
        if (p.rank <= 32) return launch_rank<kBf16, 32>(p, (unsigned)tiles, stream);
        if (p.rank <= 64) return launch_rank<kBf16, 64>(p, (unsigned)tiles, stream);
        return launch_rank<kBf16, 128>(p, (unsigned)tiles, stream);
    };
    return p.bf16 ? launch(std::true_type{}) : launch(std::false_type{});
}

}  // namespace gdn
