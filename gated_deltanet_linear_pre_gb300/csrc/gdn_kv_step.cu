// gdn_kv_step.cu -- attention of few query rows over the 8-bit paged cache (single
// tokens, drafted tokens), split over the key axis, and the join of its parts.
//
// Mathematics.  One pass over the keys with the softmax's running maximum m and sum l (base 2):
// p = 2^(x - m) with x = scale log2(e) q.k, o = sum p v, and o, l scaled by 2^(m_old - m_new) where a
// maximum grows.  Both products run on the tensor cores in their transposed forms, S^T = K q^T and
// O^T = V^T P^T (m16n8k16, fp16 operands, fp32 accumulators): keys and channels fill the 16-row side
// and 8 query rows the other, so 8 rows (a kv head's query heads, times drafted tokens) cost no more
// than one.  Codes become fp16 exactly (codes2); a page's k scale multiplies its scores in fp32 and its
// v scale its weights p.  The weights are rounded to fp16 as p r 2^14, r the page's v scale over the
// largest met so far: 11 bits down to weights 2^-28 of the largest, below which the error stays under
// 2^-39 of the largest v.  Queries are scaled by a power of two per row to below 2^15: exact for fp16
// and, less what is 2^-29 of the row's largest, for bf16.
//
// Bound.  HBM: every code is read once.  A warp takes 16 positions at a time straight from global memory
// into its registers (16-byte loads, whole 128-byte lines), the next 16 in flight while it works on
// these: the layout of the loads is chosen so that a lane's bytes are the operands it needs (K: 16
// channels of a row feed 4 K steps; V: the same 16 channels of 4 positions, whose byte pairs one
// byte permute interleaves), so nothing passes through shared memory.
#include "gdn_kv_attn.cuh"

namespace gdn {
namespace {

constexpr int kStepThreads = 256;
constexpr int kWarps = kStepThreads / 32;
constexpr float kWeightUnit = 16384.0f;  // 2^14

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8x8 transpose of 16-bit elements across the warp
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// streaming 16- or 8-byte loads of codes (read once)
__device__ __forceinline__ uint4 ld16(const uint8_t* a) { return __ldcs(reinterpret_cast<const uint4*>(a)); }
__device__ __forceinline__ uint2 ld8(const uint8_t* a) { return __ldcs(reinterpret_cast<const uint2*>(a)); }

// 16 positions of a kv head as one lane holds them: K rows g and g + 8, 16-byte chunks t (and t + 4);
// V rows 2t, 2t + 1, 2t + 8, 2t + 9, channels g (D / 8) onwards
template <int D>
struct Tile {
    uint32_t k[D / 64][2][4];
    uint32_t v[4][D / 32];
    float ks, vs;  // the page's scales
    int page;      // -1: not there, nothing is seen

    __device__ __forceinline__ void load(const KvBatch& p, int page_, int head, int in_page, int lane)
    {
        page = page_;
        const size_t at = (size_t)max(page_, 0) * p.heads + head;
        ks = __ldg(p.k_scale + at);
        vs = __ldg(p.v_scale + at);
        const size_t base = (at * p.page + in_page) * D;
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                const uint4 w = ld16(p.k + base + (g + 8 * r) * D + 64 * h + 16 * t);
                k[h][r][0] = w.x; k[h][r][1] = w.y; k[h][r][2] = w.z; k[h][r][3] = w.w;
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint8_t* a = p.v + base + (2 * t + (i & 1) + 8 * (i >> 1)) * D + g * (D / 8);
            if constexpr (D == 128) {
                const uint4 w = ld16(a);
                v[i][0] = w.x; v[i][1] = w.y; v[i][2] = w.z; v[i][3] = w.w;
            } else {
                const uint2 w = ld8(a);
                v[i][0] = w.x; v[i][1] = w.y;
            }
        }
    }
};

// shared memory: each warp's statistics and output of the unit in hand
template <int D, int NT>
struct StepSmem {
    static constexpr int R = 8 * NT, kStride = D + 4;
    float o[kWarps][R][kStride];
    float m[kWarps][R], l[kWarps][R], unit[kWarps];
    ScanSmem<kStepThreads> scan;
};

// row groups and key tiles of a sequence (a unit that sees nothing still writes its zeros: one tile)
template <int NT>
__device__ __forceinline__ void step_units(const KvBatch& p, const AttnSpace& a, int s, const SeqView& v, int& groups, int& tiles)
{
    constexpr int R = 8 * NT;
    const int64_t rows = (int64_t)v.n * (p.hq / p.heads);
    groups = is_long(p, a, s, v) ? 0 : (int)((rows + R - 1) / R);
    tiles = max((v.kv + kSub - 1) / kSub, 1);
}

template <int D, bool BF16, bool E4M3, int NT>
__global__ void __launch_bounds__(kStepThreads, NT == 1 ? 2 : 1) kv_step_kernel(AttnParams p, AttnSpace a)
{
    constexpr int R = 8 * NT, KS = D / 16, MT = D / 16;
    using Smem = StepSmem<D, NT>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int group = p.hq / p.heads, shift = 31 - __clz(p.page);
    pdl_wait();
    pdl_launch_dependents();

    // ---- this worker's range of the batch's tiles ----
    auto weight = [&](int s) {
        int groups, tiles;
        step_units<NT>(p, a, s, seq_view(p, s), groups, tiles);
        return (int64_t)p.heads * groups * tiles;
    };
    const int64_t total = scan_total<kStepThreads>(p.n_seq, weight, sm.scan);
    // at least two tiles a warp and worker: shorter ranges cost more to join than they save
    const int workers = (int)min((int64_t)gridDim.x, (total + 2 * kWarps - 1) / (2 * kWarps));
    if (blockIdx.x == 0 && tid == 0) {
        a.head->step_total = total;
        a.head->step_workers = workers;
        if (a.image_tiles == 0) a.head->error = 0u;  // else the image kernel cleared it
    }
    if ((int)blockIdx.x >= workers) return;
    const int64_t lo = cut_start(total, workers, blockIdx.x), hi = cut_start(total, workers, blockIdx.x + 1);
    int64_t before;
    int s = scan_find<kStepThreads>(p.n_seq, lo, weight, sm.scan, before);
    int64_t at = lo - before;  // tiles into sequence s

    // ---- the units of the range ----
    bool first_unit = true;
    for (int64_t x = lo; x < hi && s < p.n_seq; ++s) {
        const SeqView v = seq_view(p, s);
        int groups, tiles;
        step_units<NT>(p, a, s, v, groups, tiles);
        const int64_t units = (int64_t)p.heads * groups;
        for (int64_t unit = tiles ? at / tiles : 0; unit < units && x < hi; ++unit) {
            const int j0 = (int)(at - unit * tiles), j1 = (int)min((int64_t)tiles, j0 + (hi - x));
            at = (unit + 1) * tiles;
            x += j1 - j0;
            const int head = (int)(unit / groups), row0 = (int)(unit - (int64_t)head * groups) * R;
            const int rows = v.n * group;
            if (first_unit && tid == 0) a.step_cut[blockIdx.x] = Cut{s, head, row0, j0, tiles};

            // queries: B operands (row g of each 8), scaled per row; the factor goes into the row's score unit
            uint32_t qf[NT][KS][2];
            float coef[NT][2];
            int limit[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int row = row0 + 8 * nt + g;
                uint2 raw[KS];
                uint32_t amax = 0;
                const int i = row / group, qh = row - i * group;
                const uint16_t* src = p.q + (int64_t)(v.t0 + i) * p.q_stride + (head * group + qh) * D;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    raw[ks] = row < rows ? __ldg(reinterpret_cast<const uint2*>(src + 64 * (ks >> 2) + 16 * t + 4 * (ks & 3))) : make_uint2(0u, 0u);
                float f[KS][4];
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const uint32_t r2[2] = {raw[ks].x, raw[ks].y};
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (BF16) {
                            f[ks][2 * e] = __uint_as_float(r2[e] << 16);
                            f[ks][2 * e + 1] = __uint_as_float(r2[e] & 0xffff0000u);
                        } else {
                            const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&r2[e]));
                            f[ks][2 * e] = h.x;
                            f[ks][2 * e + 1] = h.y;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) amax = max(amax, __float_as_uint(f[ks][e]) & 0x7fffffffu);
                }
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                float mul, back;
                row_unit(amax, mul, back);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    qf[nt][ks][0] = narrow2<false>(f[ks][0] * mul, f[ks][1] * mul);
                    qf[nt][ks][1] = narrow2<false>(f[ks][2] * mul, f[ks][3] * mul);
                }
                const float unit_of = back * (p.scale * kLog2e) * kCodeUnit<E4M3>;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    coef[nt][e] = __shfl_sync(0xffffffffu, unit_of, (2 * t + e) * 4);
                    const int col = row0 + 8 * nt + 2 * t + e;
                    limit[nt][e] = col < rows ? v.first + col / group : -1;
                }
            }
            const int first_limit = v.first + row0 / group;  // the smallest of the unit's rows

            float o[NT][MT][4], m[NT][2], l[NT][2], unit_v = 0.0f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nt][mt][e] = 0.0f;
                m[nt][0] = m[nt][1] = -INFINITY;
                l[nt][0] = l[nt][1] = 0.0f;
            }

            auto work = [&](const Tile<D>& tile, int j) {
                float x2[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) x2[nt][0] = x2[nt][1] = x2[nt][2] = x2[nt][3] = 0.0f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const uint32_t r0 = tile.k[ks >> 2][0][ks & 3], r1 = tile.k[ks >> 2][1][ks & 3];
                    const uint32_t a[4] = {codes2<E4M3, false>(r0), codes2<E4M3, false>(r1), codes2<E4M3, true>(r0), codes2<E4M3, true>(r1)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816(x2[nt], a, qf[nt][ks][0], qf[nt][ks][1]);
                }
                const bool masked = j * kSub + kSub - 1 > first_limit || tile.page < 0;
                bool grew = false;
                float keep[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x2[nt][e] *= coef[nt][e & 1] * tile.ks;
                        if (masked && (tile.page < 0 || j * kSub + g + 8 * (e >> 1) > limit[nt][e & 1])) x2[nt][e] = -INFINITY;
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = fmaxf(x2[nt][e], x2[nt][2 + e]);
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        keep[nt][e] = 1.0f;
                        if (mx > m[nt][e]) {
                            keep[nt][e] = exp2f(m[nt][e] - mx);
                            m[nt][e] = mx;
                            grew = true;
                        }
                    }
                }
                // the v unit: the largest page scale met so far (a power of two)
                float up = 1.0f;
                if (tile.vs > unit_v) {
                    up = unit_v / tile.vs;
                    unit_v = tile.vs;
                    grew = true;
                }
                if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) l[nt][e] *= keep[nt][e];
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[nt][mt][e] *= keep[nt][e & 1] * up;
                    }
                }
                // (a page whose v are all 0 has scale 0; a NaN scale makes every weight NaN)
                const float r = unit_v > 0.0f ? tile.vs / unit_v * kWeightUnit : tile.vs;
                uint32_t b[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float mm = m[nt][e & 1];
                        w[e] = exp2f(x2[nt][e] - (mm == -INFINITY ? 0.0f : mm));
                        l[nt][e & 1] += w[e];
                        // a masked position has weight 0 even where its page's scale is NaN
                        w[e] = x2[nt][e] == -INFINITY ? 0.0f : w[e] * r;
                    }
                    b[nt][0] = transpose8x8(narrow2<false>(w[0], w[1]));
                    b[nt][1] = transpose8x8(narrow2<false>(w[2], w[3]));
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const uint32_t sel = mt & 1 ? 0x7362 : 0x5140;
                    const uint32_t y0 = __byte_perm(tile.v[0][mt >> 1], tile.v[1][mt >> 1], sel);
                    const uint32_t y1 = __byte_perm(tile.v[2][mt >> 1], tile.v[3][mt >> 1], sel);
                    const uint32_t a[4] = {codes2<E4M3, false>(y0), codes2<E4M3, true>(y0), codes2<E4M3, false>(y1), codes2<E4M3, true>(y1)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][mt], a, b[nt][0], b[nt][1]);
                }
            };

            // the warp's tiles of the unit, the next one's codes in flight and the page after that looked up
            auto page_of = [&](int j) { return j < j1 ? page_at(p, s, (j * kSub) >> shift) : -1; };
            const int in_mask = p.page - 1;
            int j = j0 + warp;
            if (j < j1) {
                Tile<D> t0, t1;
                t0.load(p, page_of(j), head, (j * kSub) & in_mask, lane);
                int next = page_of(j + kWarps);
                while (true) {
                    if (j + kWarps < j1) t1.load(p, next, head, ((j + kWarps) * kSub) & in_mask, lane);
                    next = page_of(j + 2 * kWarps);
                    work(t0, j);
                    j += kWarps;
                    if (j >= j1) break;
                    if (j + kWarps < j1) t0.load(p, next, head, ((j + kWarps) * kSub) & in_mask, lane);
                    next = page_of(j + 2 * kWarps);
                    work(t1, j);
                    j += kWarps;
                    if (j >= j1) break;
                }
            }

            // ---- join the warps ----
            __syncthreads();  // the last unit's values are read
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float sum = l[nt][e];
                    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                    const int row = 8 * nt + 2 * t + e;
                    if (g == 0) {
                        sm.m[warp][row] = m[nt][e];
                        sm.l[warp][row] = sum;
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; mt += 2)
                        *reinterpret_cast<float4*>(&sm.o[warp][row][g * (D / 8) + 2 * mt]) =
                            make_float4(o[nt][mt][e], o[nt][mt][2 + e], o[nt][mt + 1][e], o[nt][mt + 1][2 + e]);
                }
            }
            if (lane == 0) sm.unit[warp] = unit_v;
            __syncthreads();
            const bool whole = j0 == 0 && j1 == tiles;
            const int slot = 2 * blockIdx.x + (first_unit ? 0 : 1);
            for (int row = warp; row < R; row += kWarps) {
                if (row0 + row >= rows) break;
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm.m[w][row]);
                const float ref = top == -INFINITY ? 0.0f : top;
                constexpr int E = D / 32;
                float sum = 0.0f, acc[E];
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float f = exp2f(sm.m[w][row] - ref);
                    sum += f * sm.l[w][row];
                    const float fo = f * (sm.unit[w] > 0.0f ? sm.unit[w] * (kCodeUnit<E4M3> / kWeightUnit) : 1.0f);
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] += fo * sm.o[w][row][lane * E + e];
                }
                if (whole) {
                    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                    const int i = (row0 + row) / group, qh = row0 + row - i * group;
                    uint32_t* dst = reinterpret_cast<uint32_t*>(p.y + ((int64_t)(v.t0 + i) * p.hq + head * group + qh) * D + lane * E);
#pragma unroll
                    for (int e = 0; e < E; e += 2) dst[e / 2] = narrow2<BF16>(acc[e] * inv, acc[e + 1] * inv);
                } else {
                    if (lane == 0) a.step_stat[(size_t)slot * kStepMaxRows + row] = make_float2(top, sum);
                    float* dst = a.step_out + ((size_t)slot * kStepMaxRows + row) * D + lane * E;
#pragma unroll
                    for (int e = 0; e < E; ++e) dst[e] = acc[e];
                }
            }
            first_unit = false;
        }
        at = 0;
    }
}

// Block (w, row): where range w is the first that begins inside a unit, joins that unit's parts for one
// query row, in the order of their ranges.
constexpr int kJoinThreads = 128;
template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) kv_join_kernel(AttnParams p, AttnSpace a)
{
    constexpr int E = D / 32, W = kJoinThreads / 32;
    __shared__ float part[W][D], part_l[W], part_m[W];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, group = p.hq / p.heads;
    pdl_wait();
    pdl_launch_dependents();
    const int w = (int)blockIdx.x + 1, row = blockIdx.y;
    const int workers = a.head->step_workers;
    if (w >= workers) return;
    const Cut cut = a.step_cut[w];
    if (cut.j0 == 0) return;
    const int64_t total = a.head->step_total, begin = cut_start(total, workers, w) - cut.j0;
    if (cut_start(total, workers, w - 1) > begin) return;
    const int t0 = cu_at(p.cu_seqlens, cut.s, p.T), n = cu_at(p.cu_seqlens, cut.s + 1, p.T) - t0;
    if (cut.unit + row >= n * group) return;
    const int last = cut_of(total, workers, begin + cut.tiles - 1);
    float top = -INFINITY, sum = 0.0f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll 4
    for (int i = w - 1 + warp; i <= last; i += W) {
        // the unit is the first of every range but the one that it begins in the middle of
        const int slot = 2 * i + (cut_start(total, workers, i) >= begin ? 0 : 1);
        const float2 st = a.step_stat[(size_t)slot * kStepMaxRows + row];
        const float* src = a.step_out + ((size_t)slot * kStepMaxRows + row) * D + lane * E;
        const float next = fmaxf(top, st.x), ref = next == -INFINITY ? 0.0f : next;
        const float f0 = exp2f(top - ref), f1 = exp2f(st.x - ref);
        sum = sum * f0 + st.y * f1;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * f0 + src[e] * f1;
        top = next;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) part[warp][lane * E + e] = acc[e];
    if (lane == 0) {
        part_m[warp] = top;
        part_l[warp] = sum;
    }
    __syncthreads();
    if (tid >= D / 2) return;
    float m = -INFINITY, l = 0.0f, x0 = 0.0f, x1 = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) m = fmaxf(m, part_m[i]);
    const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const float f = exp2f(part_m[i] - ref);
        l += f * part_l[i];
        x0 += f * part[i][2 * tid];
        x1 += f * part[i][2 * tid + 1];
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int i = (cut.unit + row) / group, qh = cut.unit + row - i * group;
    reinterpret_cast<uint32_t*>(p.y + ((int64_t)(t0 + i) * p.hq + cut.head * group + qh) * D)[tid] = narrow2<BF16>(x0 * inv, x1 * inv);
}

template <int D, bool BF16, bool E4M3, int NT>
cudaError_t launch(const AttnParams& p, const AttnSpace& a, int sms, cudaStream_t stream)
{
    auto kernel = kv_step_kernel<D, BF16, E4M3, NT>;
    const size_t smem = sizeof(StepSmem<D, NT>);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int grid = min(sms * (NT == 1 ? 2 : 1), kStepMaxWorkers);
    e = launch_k(kernel, dim3(grid), dim3(kStepThreads), smem, stream, true, p, a);
    if (e != cudaSuccess) return e;
    if (grid == 1) return cudaSuccess;
    return launch_k(kv_join_kernel<D, BF16>, dim3(grid - 1, 8 * NT), dim3(kJoinThreads), 0, stream, true, p, a);
}

template <int D, bool BF16, bool E4M3>
cudaError_t launch_rows(const AttnParams& p, const AttnSpace& a, int sms, cudaStream_t stream)
{
    // query rows of an average sequence decide the tile: 8 rows as long as they hold them (two blocks an
    // SM), else 16 or 32 (a warp's codes serve more rows, at one block an SM)
    const int64_t rows = ((int64_t)p.T * (p.hq / p.heads) + p.n_seq - 1) / p.n_seq;
    if (rows <= 8) return launch<D, BF16, E4M3, 1>(p, a, sms, stream);
    if (rows <= 16) return launch<D, BF16, E4M3, 2>(p, a, sms, stream);
    return launch<D, BF16, E4M3, 4>(p, a, sms, stream);
}

template <int D>
cudaError_t launch_types(const AttnParams& p, const AttnSpace& a, int sms, cudaStream_t stream)
{
    if (p.format == 1) return p.bf16 ? launch_rows<D, true, true>(p, a, sms, stream) : launch_rows<D, false, true>(p, a, sms, stream);
    return p.bf16 ? launch_rows<D, true, false>(p, a, sms, stream) : launch_rows<D, false, false>(p, a, sms, stream);
}

}  // namespace

cudaError_t launch_kv_step(const AttnParams& p, const AttnSpace& a, int sms, cudaStream_t stream)
{
    return p.dim == 64 ? launch_types<64>(p, a, sms, stream) : launch_types<128>(p, a, sms, stream);
}

}  // namespace gdn
