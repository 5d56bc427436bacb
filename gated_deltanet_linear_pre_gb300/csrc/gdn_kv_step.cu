// gdn_kv_step.cu -- attention of few query rows over the 8-bit paged cache (single
// tokens, drafted tokens), split over the key axis.
//
// Mathematics.  One pass over the keys with the softmax's running maximum m and sum l (base 2):
// p = 2^(x - m) with x = scale log2(e) q.k, o = sum p v, and o, l scaled by 2^(m_old - m_new) where a
// maximum grows.  Both products run on the tensor cores in their transposed forms, S^T = K q^T and
// O^T = V^T P^T (m16n8k16, fp16 operands, fp32 accumulators): keys and channels fill the 16-row side
// and 8 query rows the other, so 8 rows (a kv head's query heads, times drafted tokens) cost no more
// than one.  Codes become fp16 exactly (codes2); a page's k scale multiplies its scores in fp32 and its
// v scale its weights p.  The reference m moves only where a score passes it by 8, so most tiles need no
// exchange between lanes: p stays below 2^8.  The weights are rounded to fp16 as p r 2^7, r the page's v
// scale over the largest met so far: 11 bits down to 2^-21 of the largest weight, below which the error
// stays under 2^-32 of the largest v.  Queries are scaled to fp16 by a power of two per row (row_unit).
//
// Bound.  HBM: every code is read once.  A warp takes 4 KB of codes at a time; a lane copies (cp.async)
// exactly the bytes that it will turn into its operands, into shared memory that only it reads, so the
// ring needs no barrier, the codes in flight cost no registers, and every copy of a warp covers whole
// 128-byte lines.  The bytes are chosen so that no exchange between lanes is needed: K, 16 channels of
// a row feed 4 K steps; V, the same 16 channels of 4 positions, whose byte pairs one byte permute
// interleaves.  (Codes held in registers from load to use took 98 us where the ring took 72; eight warps a CTA
// no less than four.)
//
// Measured, on cold caches: 64 sequences of 1 to 8192 positions (32 query heads over 4 of 128, e4m3) 63 us for
// 282 MB, 3 of 131001 (16 over 4 of 64, int8) 43 us for 201 MB: 4.5 and 4.7 TB/s of 6.8.  In between a range's
// first codes, some 6 us after the launch, and the first CTAs' ends HBM is busy; the last end 12 and 4 us behind
// the mean.
// (Long ranges first and short ones after them, for the SMs that end early: 70.0 for 71.0 us, and drafted
// tokens' 98 for 88, as a late CTA's start costs what the balance brings.)  37 sequences of up to 6 drafted
// tokens over 4100 positions (48 over 16) 71 us for 299 MB.
#include "gdn_kv_attn.cuh"

namespace gdn {
namespace {

constexpr int kStepThreads = 128;
constexpr int kWarps = kStepThreads / 32;
constexpr int kStages = 2;             // tiles of a warp in its ring
constexpr float kWeightUnit = 128.0f;  // 2^7
constexpr float kLazy = 8.0f;

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

template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src)
{
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// A tile of a kv head in a warp's ring, in parts of 16 positions, every lane's bytes at [..][lane]:
// K rows g and g + 8, 16-byte chunks t (and t + 4); V rows 2t, 2t + 1, 2t + 8, 2t + 9, channels g (D / 8)
// onwards
template <int D>
struct Tile {
    static constexpr int kParts = kStepTile<D> / kSub;
    uint4 k[kParts][D / 64][2][32];
    uint32_t v[kParts][4][32][D / 32];
};

// what a lane keeps of a tile on its way: each part's page (-1: not there) and scales
template <int D>
struct Pages {
    int page[Tile<D>::kParts];
    float ks[Tile<D>::kParts], vs[Tile<D>::kParts];
};

// a unit's cache as a lane reads it
template <int D>
struct Source {
    const uint8_t *k, *v;        // its bytes of row 0 of page 0
    const float *ks, *vs;
    const int32_t* table;
    int64_t page_bytes;
    int heads, n_pages, shift, mask;

    __device__ __forceinline__ Source(const KvBatch& p, int s, int head, int lane)
        : table(p.table + (size_t)s * p.table_stride), page_bytes((int64_t)p.heads * p.page * D), heads(p.heads), n_pages(p.n_pages),
          shift(page_shift(p)), mask(p.page - 1)
    {
        const int g = lane >> 2, t = lane & 3, at = head * p.page * D;
        k = p.k + at + g * D + 16 * t;
        v = p.v + at + 2 * t * D + g * (D / 8);
        ks = p.k_scale + head;
        vs = p.v_scale + head;
    }
    // the pages of tile j (pos < kv <= max_pages * page: the entries exist)
    __device__ __forceinline__ void look(int j, int kv, int (&page)[Tile<D>::kParts]) const
    {
#pragma unroll
        for (int i = 0; i < Tile<D>::kParts; ++i) {
            const int pos = j * kStepTile<D> + i * kSub;
            const int x = pos < kv ? __ldg(table + (pos >> shift)) : -1;
            page[i] = x < n_pages ? x : -1;
        }
    }
    __device__ __forceinline__ void load(Tile<D>& tile, Pages<D>& pages, const int (&page)[Tile<D>::kParts], int j, int lane) const
    {
#pragma unroll
        for (int i = 0; i < Tile<D>::kParts; ++i) {
            pages.page[i] = page[i];
            const int x = max(page[i], 0);  // (a missing page: any, its scores are masked)
            pages.ks[i] = __ldg(ks + (int64_t)x * heads);
            pages.vs[i] = __ldg(vs + (int64_t)x * heads);
            const int64_t at = x * page_bytes + ((j * kStepTile<D> + i * kSub) & mask) * D;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int h = 0; h < D / 64; ++h) copy_async<16>(&tile.k[i][h][r][lane], k + at + 8 * r * D + 64 * h);
#pragma unroll
            for (int r = 0; r < 4; ++r) copy_async<D / 8>(&tile.v[i][r][lane][0], v + at + ((r & 1) + 8 * (r >> 1)) * D);
        }
    }
};

template <int D, int NT>
struct StepSmem {
    static constexpr int R = 8 * NT, kStride = D + 4;
    union {
        Tile<D> ring[kWarps][kStages];
        float o[kWarps][R][kStride];  // each warp's output of the unit in hand, once its keys are done
        ScanSmem<kStepThreads> scan;  // before the first unit
    };
    uint2 q[NT][D / 16][32];          // queries as B operands: row g of each 8, K step, lane
    float coef[R];                    // a row's score unit
    int limit[R];                     // last position it sees
    float m[kWarps][R], l[kWarps][R], unit[kWarps];
};

// row groups and key tiles of a sequence (a unit that sees nothing still writes its zeros: one tile)
template <int D, int NT>
__device__ __forceinline__ void step_units(const KvBatch& p, const AttnSpace& a, int s, const SeqView& v, int& groups, int& tiles)
{
    constexpr int R = 8 * NT;
    const int64_t rows = (int64_t)v.n * (p.hq / p.heads);
    groups = is_long(p, a, s, v) ? 0 : (int)((rows + R - 1) / R);
    tiles = max((v.kv + kStepTile<D> - 1) / kStepTile<D>, 1);
}

template <int D, bool BF16, bool E4M3, int NT>
__global__ void __launch_bounds__(kStepThreads, step_ctas(8 * NT)) kv_step_kernel(AttnParams p, AttnSpace a)
{
    constexpr int R = 8 * NT, KS = D / 16, MT = D / 16;
    using Smem = StepSmem<D, NT>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int group = p.hq / p.heads;
    pdl_wait();
    pdl_launch_dependents();

    // ---- this worker's range of the batch's tiles ----
    auto weight = [&](int s) {
        int groups, tiles;
        step_units<D, NT>(p, a, s, seq_view(p, s), groups, tiles);
        return (int64_t)p.heads * groups * (a.whole_units ? 1 : tiles + kStepUnitCost);
    };
    const int64_t total = scan_total<kStepThreads>(p.n_seq, weight, sm.scan);
    // at least two tiles a warp beside a unit's constant: shorter ranges cost more to join than they save
    const int least = a.whole_units ? 1 : kStepUnitCost + 2 * kWarps;
    const int workers = (int)min((int64_t)gridDim.x, (total + least - 1) / least);
    if (blockIdx.x == 0 && tid == 0) {
        a.head->step_total = total;
        a.head->step_workers = workers;
        if (a.image_tiles == 0) a.head->error = 0u;  // else the image kernel cleared it
    }
    if ((int)blockIdx.x >= workers) return;
    const int64_t lo = cut_start(total, workers, blockIdx.x), hi = cut_start(total, workers, blockIdx.x + 1);
    int64_t before;
    int s = scan_find<kStepThreads>(p.n_seq, lo, weight, sm.scan, before);
    int64_t at = lo - before;  // cost into sequence s

    // ---- the units of the range ----
    bool first_unit = true;
    for (int64_t x = lo; x < hi && s < p.n_seq; ++s) {
        const SeqView v = seq_view(p, s);
        int groups, tiles;
        step_units<D, NT>(p, a, s, v, groups, tiles);
        const int64_t units = (int64_t)p.heads * groups;
        const int cost = a.whole_units ? 1 : tiles + kStepUnitCost;
        for (int64_t unit = at / cost; unit < units && x < hi; ++unit) {
            const int from = (int)(at - unit * cost), to = (int)min((int64_t)cost, from + (hi - x));
            const int j0 = a.whole_units ? 0 : max(from - kStepUnitCost, 0), j1 = a.whole_units ? tiles : to - kStepUnitCost;
            at = (unit + 1) * cost;
            x += to - from;
            const int head = (int)(unit / groups), row0 = (int)(unit - (int64_t)head * groups) * R;
            const int rows = v.n * group;
            if (first_unit && tid == 0) a.step_cut[blockIdx.x] = Cut{s, head, row0, j0, tiles, from, lo, v.t0, v.n, 0, 0};
            if (j1 <= 0) break;  // the range ends within the unit's constant

            // the warp's first tiles on their way
            constexpr int kParts = Tile<D>::kParts;
            const Source<D> src(p, s, head, lane);
            Tile<D>* const ring = sm.ring[warp];
            Pages<D> pages[kStages];
            int j = j0 + warp, look[kStages][kParts];  // pages looked up ahead of their tiles
#pragma unroll
            for (int i = 0; i < kStages; ++i) src.look(j + i * kWarps, j + i * kWarps < j1 ? v.kv : 0, look[i]);
            int(&next_page)[kParts] = look[kStages - 1];
            __syncthreads();  // the last unit's outputs and queries are read
#pragma unroll
            for (int i = 0; i < kStages - 1; ++i) {
                if (j + i * kWarps < j1) src.load(ring[i], pages[i], look[i], j + i * kWarps, lane);
                copy_commit();
            }

            // queries as B operands, scaled per row; the factor goes into the row's score unit
            for (int nt = warp; nt < NT; nt += kWarps) {
                const int row = row0 + 8 * nt + g, i = row / group, qh = row - i * group;
                const uint16_t* from = p.q + (int64_t)(v.t0 + i) * p.q_stride + (head * group + qh) * D;
                uint2 raw[KS];
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    raw[ks] = row < rows ? __ldg(reinterpret_cast<const uint2*>(from + 64 * (ks >> 2) + 16 * t + 4 * (ks & 3))) : make_uint2(0u, 0u);
                float f[KS][4];
                uint32_t amax = 0;
#pragma unroll
                for (int ks = 0; ks < KS; ks += 2) {
                    float y[8];
                    widen8<BF16>(make_uint4(raw[ks].x, raw[ks].y, raw[ks + 1].x, raw[ks + 1].y), y);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        f[ks + (e >> 2)][e & 3] = y[e];
                        amax = max(amax, __float_as_uint(y[e]) & 0x7fffffffu);
                    }
                }
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                float mul, back;
                row_unit(amax, mul, back);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    sm.q[nt][ks][lane] = make_uint2(narrow2<false>(f[ks][0] * mul, f[ks][1] * mul), narrow2<false>(f[ks][2] * mul, f[ks][3] * mul));
                if (t == 0) {
                    // a row that is not finite has no softmax; its scores alone might all be -infinity, as if masked
                    sm.coef[8 * nt + g] = amax < 0x7f800000u ? back * (p.scale * kLog2e) : __uint_as_float(0x7fffffffu);
                    sm.limit[8 * nt + g] = row < rows ? v.first + i : -1;
                }
            }
            __syncthreads();
            // up to 16 rows are held in registers (shared memory reads bound the kernel with the conversions)
            constexpr bool kHeld = NT <= 2;
            uint2 qb[kHeld ? NT : 1][kHeld ? KS : 1];
            if constexpr (kHeld)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) qb[nt][ks] = sm.q[nt][ks][lane];
            float coef[NT][2];
            int limit[NT][2];
            const int first_limit = v.first + row0 / group;  // the smallest of the unit's rows
            bool seen = false;                               // the warp has met a score
            float o[NT][MT][4], m[NT][2], l[NT][2], unit_v = 0.0f, inv_v = 0.0f;  // inv_v: kWeightUnit / unit_v
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nt][mt][e] = 0.0f;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    m[nt][e] = 0.0f;
                    l[nt][e] = 0.0f;
                    coef[nt][e] = sm.coef[8 * nt + 2 * t + e];
                    limit[nt][e] = sm.limit[8 * nt + 2 * t + e];
                }
            }

            // part `i` of a tile: positions pos onwards
            auto work = [&](const Tile<D>& tile, const Pages<D>& pg, int i, int pos) {
                float x[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.0f;
#pragma unroll
                for (int h = 0; h < D / 64; ++h) {
                    const uint4 w0 = tile.k[i][h][0][lane], w1 = tile.k[i][h][1][lane];
                    const uint32_t r0[4] = {w0.x, w0.y, w0.z, w0.w}, r1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t ka[4] = {codes2<E4M3, false>(r0[c]), codes2<E4M3, false>(r1[c]), codes2<E4M3, true>(r0[c]), codes2<E4M3, true>(r1[c])};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            uint2 b;
                            if constexpr (kHeld) b = qb[nt][4 * h + c];
                            else b = sm.q[nt][4 * h + c][lane];
                            mma16816(x[nt], ka, b.x, b.y);
                        }
                    }
                }
                const float vs = pg.vs[i];
                const bool there = pg.page[i] >= 0, masked = pos + kSub - 1 > first_limit || !there;
                float top = -INFINITY;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float c2[2] = {coef[nt][0] * pg.ks[i], coef[nt][1] * pg.ks[i]};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[nt][e] = fmaf(x[nt][e], c2[e & 1], -m[nt][e & 1]);  // m: 0 until the first score is seen
                        if (masked && (!there || pos + g + 8 * (e >> 1) > limit[nt][e & 1])) x[nt][e] = -INFINITY;
                        top = fmaxf(top, x[nt][e]);
                    }
                }
                // a score passes its row's reference by kLazy, or is the warp's first (a row that the first tile
                // with any score leaves out sees none of the later ones either): references move to the maxima
                const bool first = !seen && __any_sync(0xffffffffu, top > -INFINITY);
                const bool grows = there && vs > unit_v;
                if (__any_sync(0xffffffffu, top > kLazy) || first || grows) {
                    float up = 1.0f;
                    if (grows) {  // the v unit: the largest page scale met so far (a power of two)
                        up = unit_v * __frcp_rn(vs);
                        unit_v = vs;
                        inv_v = kWeightUnit * __frcp_rn(vs);
                    }
                    seen = seen || first;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float keep[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float mx = fmaxf(x[nt][e], x[nt][2 + e]);
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                            // by how much the reference moves (with the first scores, down as well as up)
                            const float by = mx > 0.0f || (first && mx > -INFINITY) ? mx : 0.0f;
                            keep[e] = first ? 1.0f : ex2(-by);
                            m[nt][e] += by;
                            l[nt][e] *= keep[e];
                            x[nt][e] -= by;
                            x[nt][2 + e] -= by;
                        }
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[nt][mt][e] *= keep[e & 1] * up;
                    }
                }
                // (a page whose v are all 0 has scale 0; a NaN scale makes every weight NaN)
                const float r = unit_v > 0.0f ? vs * inv_v : vs;
                uint32_t b[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        w[e] = ex2(x[nt][e]);
                        l[nt][e & 1] += w[e];
                        w[e] *= r;
                        // a masked position has weight 0 even where its page's scale is NaN
                        if (masked && x[nt][e] == -INFINITY) w[e] = 0.0f;
                    }
                    b[nt][0] = transpose8x8(narrow2<false>(w[0], w[1]));
                    b[nt][1] = transpose8x8(narrow2<false>(w[2], w[3]));
                }
                constexpr int W = D / 32;
                uint32_t vw[4][W];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
#pragma unroll
                    for (int y = 0; y < W; ++y) vw[c][y] = tile.v[i][c][lane][y];
                    // positions past the sequence's end hold anything: their codes count as 0
                    if (masked && (!there || pos + 2 * t + (c & 1) + 8 * (c >> 1) >= v.kv))
#pragma unroll
                        for (int y = 0; y < W; ++y) vw[c][y] = 0u;
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const uint32_t sel = mt & 1 ? 0x7362 : 0x5140;
                    const uint32_t y0 = __byte_perm(vw[0][mt >> 1], vw[1][mt >> 1], sel);
                    const uint32_t y1 = __byte_perm(vw[2][mt >> 1], vw[3][mt >> 1], sel);
                    const uint32_t va[4] = {codes2<E4M3, false>(y0), codes2<E4M3, true>(y0), codes2<E4M3, false>(y1), codes2<E4M3, true>(y1)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][mt], va, b[nt][0], b[nt][1]);
                }
            };

            // the warp's tiles of the unit: kStages - 1 ahead in flight, the pages of the next one looked up
            while (j < j1) {
#pragma unroll
                for (int i = 0; i < kStages; ++i) {
                    constexpr int ahead = kStages - 1;
                    const int to = (i + ahead) % kStages;
                    if (j + ahead * kWarps < j1) src.load(ring[to], pages[to], next_page, j + ahead * kWarps, lane);
                    copy_commit();
                    src.look(j + kStages * kWarps, j + kStages * kWarps < j1 ? v.kv : 0, next_page);
                    copy_wait<ahead>();
#pragma unroll
                    for (int part = 0; part < kParts; ++part) work(ring[i], pages[i], part, j * kStepTile<D> + part * kSub);
                    j += kWarps;
                    if (j >= j1) break;
                }
            }

            // ---- join the warps ----
            __syncthreads();  // every ring is done with
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
                        sm.m[warp][row] = sum == 0.0f ? -INFINITY : m[nt][e];
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
                    const float f = ex2(sm.m[w][row] - ref);
                    sum += f * sm.l[w][row];
                    const float fo = f * (sm.unit[w] > 0.0f ? sm.unit[w] * (1.0f / kWeightUnit) : 1.0f);
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

template <int D, bool BF16, bool E4M3, int NT>
cudaError_t launch(const AttnParams& p, const AttnSpace& a, int sms, cudaStream_t stream)
{
    auto kernel = kv_step_kernel<D, BF16, E4M3, NT>;
    const size_t smem = sizeof(StepSmem<D, NT>);
    static_assert(sizeof(StepSmem<D, NT>) <= 232448, "shared memory");
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    // no more workers than the call can have ranges: those without one would only look for it (one sequence of
    // 301 positions 10.8 -> 7.5 us)
    const double units = ((double)p.T * (p.hq / p.heads) / (8 * NT) + p.n_seq) * p.heads, tiles = (double)p.max_pages * p.page / kStepTile<D> + 1;
    const double most = a.whole_units ? units : units * (tiles + kStepUnitCost) / (kStepUnitCost + 2 * kWarps) + 1;
    const int grid = (int)min((double)step_grid(sms, 8 * NT), ceil(most));
    return launch_k(kernel, dim3(grid), dim3(kStepThreads), smem, stream, true, p, a);
}

template <int D, bool BF16, bool E4M3>
cudaError_t launch_rows(const AttnParams& p, const AttnSpace& a, int sms, cudaStream_t stream)
{
    const int rows = step_rows(p, a);
    if (rows == 8) return launch<D, BF16, E4M3, 1>(p, a, sms, stream);
    if (rows == 16) return launch<D, BF16, E4M3, 2>(p, a, sms, stream);
    return launch<D, BF16, E4M3, 4>(p, a, sms, stream);
}

template <int D>
cudaError_t launch_types(const AttnParams& p, const AttnSpace& a, int sms, cudaStream_t stream)
{
    if (p.format == 1) return p.bf16 ? launch_rows<D, true, true>(p, a, sms, stream) : launch_rows<D, false, true>(p, a, sms, stream);
    return p.bf16 ? launch_rows<D, true, false>(p, a, sms, stream) : launch_rows<D, false, false>(p, a, sms, stream);
}

}  // namespace

int step_rows(const AttnParams& p, const AttnSpace& a)
{
    // query rows of an average sequence decide the tile: 8 rows as long as they hold them, else 16 or 32
    // (a warp's codes serve more rows).  An average above kLongRows says that there are long sequences, which
    // the prompt kernel takes; those left here are then taken to bring single tokens.
    const int group = p.hq / p.heads;
    int64_t rows = ((int64_t)p.T * group + p.n_seq - 1) / p.n_seq;
    if (rows > a.most_rows) rows = group;
    return rows <= 8 ? 8 : rows <= 16 ? 16 : kStepMaxRows;
}

cudaError_t launch_kv_step(const AttnParams& p, const AttnSpace& a, int sms, cudaStream_t stream)
{
    return p.dim == 64 ? launch_types<64>(p, a, sms, stream) : launch_types<128>(p, a, sms, stream);
}

}  // namespace gdn
