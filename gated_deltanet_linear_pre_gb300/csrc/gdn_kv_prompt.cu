// gdn_kv_prompt.cu -- attention of many query rows over the 8-bit paged cache, on
// the tcgen05 tensor cores.
//
// Mathematics.  One pass over the keys per 128 query rows with the softmax's running maximum and sum:
// S = Q K^T and O += P V are 128 x 128 (x head_dim) products with fp32 accumulators in TMEM; a thread
// owns a query row.  P = 2^(x - m + 7), x = scale log2(e) q.k; the reference m moves, and O and l are
// rescaled, only where a tile's maximum passes it by 8 (a factor of 256): P stays below 2^15, and what is
// lost to fp16's smallest step is 2^-31 of the largest weight.  Weights are rounded to fp16 (11 bits),
// sums and statistics are fp32.  Queries are scaled to fp16 by a power of two per row (row_unit).
//
// Layout.  The tensor cores read 16-bit operands from shared memory, so the codes have to be unpacked
// somewhere.  Done by every CTA for itself, a 128-position tile would cost each about as many issue slots
// as a third of its softmax; instead one kernel unpacks each long sequence's cache once into images, in
// the 128-byte swizzled order (without swizzle the products run at two thirds of their rate), that a single
// bulk copy brings in: 4 bytes moved per code byte, a few
// per cent of a prompt's time.  An image holds code * (page scale / largest scale of the sequence and
// head) * kUp, exact for pages whose scale is at least 2^-15 (e4m3) or 2^-24 (int8) of the largest after
// the shift; the largest scale itself goes into the scores' unit and the outputs'.
//
// A CTA (640 threads, one per SM) holds two 128-row halves, so that one half's softmax runs under the
// other's products: warps 0-7 and 8-15 the rows (two threads a row, each half of a tile's columns: a tile's
// softmax takes less than the other half's 1024 tensor cycles only with four warps a scheduler), warp 16
// the copies, warp 17 the products (18 and 19 only make up the warpgroup whose registers the rows'
// threads get).  TMEM: S and O of each half, 512 columns at head_dim 128; the fp16 P of 64 keys takes the
// first 32 of their 64 score columns.
// Rows are (token, query head of the kv head): floor(128 / group) tokens a half.
#include "gdn_kv_attn.cuh"
#include "umma.cuh"

namespace gdn {
namespace {

constexpr int kImageThreads = 256;
constexpr int kThreads = 640;
constexpr int kLoadWarp = 16, kMmaWarp = 17;
// registers a thread, of the 96 that 640 threads are launched with: 512 x 104 + 128 x 64 = 640 x 96
constexpr int kSoftmaxRegs = 104, kOtherRegs = 64;
constexpr float kWeightShift = 7.0f;
constexpr float kLazy = 8.0f;

// images hold codes times kUp: up to 127 x 2^8 and 448 x 2^6
template <bool E4M3> constexpr float kUp = E4M3 ? 64.0f : 256.0f;

template <int D> constexpr uint32_t kTileBytes = kKeys * D * 2;

// byte offset of (position, channels 8 c8 .. + 7) in an image: planes of 64 channels, a position's 128 bytes
// of a plane a row, its 16-byte pieces swizzled
constexpr uint32_t kPlane = kKeys * 128;
__device__ __forceinline__ int image_off(int pos, int c8) { return (c8 >> 3) * (int)kPlane + pos * 128 + (((c8 & 7) ^ (pos & 7)) << 4); }

// ---- unpacking ------------------------------------------------------------------------
__device__ __forceinline__ int key_tiles(int kv) { return (kv + kKeys - 1) / kKeys; }

template <bool E4M3>
__device__ __forceinline__ uint4 unpack8(uint2 w, __half2 f)
{
    uint32_t r[4] = {codes2<E4M3, false>(w.x), codes2<E4M3, true>(w.x), codes2<E4M3, false>(w.y), codes2<E4M3, true>(w.y)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&r[i]), f);
        r[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// Each block takes an equal range of the (tile, kv head) items of all candidates, head fastest.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kImageThreads) kv_image_kernel(AttnParams p, AttnSpace a)
{
    __shared__ ScanSmem<kImageThreads> scan;
    __shared__ float top_k[kImageThreads / 32], top_v[kImageThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, shift = page_shift(p);
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x == 0 && tid == 0) a.head->error = 0u;
    auto weight = [&](int s) {
        const SeqView v = seq_view(p, s);
        return candidate(p, a, v) ? (int64_t)key_tiles(v.kv) : 0;
    };
    const int64_t tiles = scan_total<kImageThreads>(p.n_seq, weight, scan), items = tiles * p.heads;
    const int64_t lo = cut_start(items, gridDim.x, blockIdx.x), hi = cut_start(items, gridDim.x, blockIdx.x + 1);
    if (lo >= hi) return;
    int64_t before;
    int s = scan_find<kImageThreads>(p.n_seq, lo / p.heads, weight, scan, before);
    int64_t at = lo / p.heads - before;  // tile within the sequence
    int head = (int)(lo % p.heads);
    for (int64_t x = lo; x < hi && s < p.n_seq;) {
        const SeqView v = seq_view(p, s);
        const int n = candidate(p, a, v) ? key_tiles(v.kv) : 0;
        if (at >= n) {
            before += n;
            at = 0;
            ++s;
            continue;
        }
        // the sequence's images fit, every page is there; its largest scales (NaN ones apart)
        const int pages = (v.kv + p.page - 1) >> shift;
        float mk = 0.0f, mv = 0.0f;
        bool there = before + n <= a.image_tiles;
        for (int i = tid; i < pages; i += kImageThreads) {
            const int page = page_at(p, s, i);
            if (page < 0) {
                there = false;
            } else {
                mk = fmaxf(mk, __ldg(p.k_scale + (size_t)page * p.heads + head));
                mv = fmaxf(mv, __ldg(p.v_scale + (size_t)page * p.heads + head));
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, off));
            mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, off));
        }
        if (lane == 0) {
            top_k[warp] = mk;
            top_v[warp] = mv;
        }
        there = __syncthreads_and(there);
#pragma unroll
        for (int w = 0; w < kImageThreads / 32; ++w) {
            mk = fmaxf(mk, top_k[w]);
            mv = fmaxf(mv, top_v[w]);
        }
        if (at == 0 && tid == 0) {
            if (head == 0) {
                a.ok[s] = there;
                a.image_base[s] = there ? (int)before : 0;
            }
            if (there) a.norm[(size_t)before * p.heads + head] = make_float2(mk, mv);
        }
        if (there) {
            unsigned char* const img = a.images + ((size_t)(before + at) * p.heads + head) * (2 * kTileBytes<D>);
            // neighbouring lanes take neighbouring channels: whole rows of codes and of an image's planes
            for (int i = tid; i < kKeys * (D / 8); i += kImageThreads) {
                const int pos = i / (D / 8), c8 = i % (D / 8);
                const int at_pos = (int)at * kKeys + pos;
                uint4 wk = make_uint4(0u, 0u, 0u, 0u), wv = wk;
                if (at_pos < v.kv) {
                    const size_t row = (size_t)page_at(p, s, at_pos >> shift) * p.heads + head;
                    const size_t src = (row * p.page + (at_pos & (p.page - 1))) * D + 8 * c8;
                    const float ks = __ldg(p.k_scale + row), vs = __ldg(p.v_scale + row);
                    // (a scale of 0 may meet a largest one of 0; NaN scales stay NaN)
                    const float fk = ks == 0.0f ? 0.0f : ks / mk * kUp<E4M3>, fv = vs == 0.0f ? 0.0f : vs / mv * kUp<E4M3>;
                    wk = unpack8<E4M3>(__ldg(reinterpret_cast<const uint2*>(p.k + src)), __float2half2_rn(fk));
                    wv = unpack8<E4M3>(__ldg(reinterpret_cast<const uint2*>(p.v + src)), __float2half2_rn(fv));
                }
                *reinterpret_cast<uint4*>(img + image_off(pos, c8)) = wk;
                *reinterpret_cast<uint4*>(img + kTileBytes<D> + image_off(pos, c8)) = wv;
            }
        }
        __syncthreads();  // top_k, top_v read
        ++x;
        if (++head == p.heads) {
            head = 0;
            ++at;
        }
    }
}

// ---- the units of long sequences -----------------------------------------------------
// sum over i < n of floor((a i + b) / m), by exchanging the roles of a and m as in Euclid's algorithm
__device__ __forceinline__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b)
{
    int64_t sum = 0;
    while (n > 0) {
        sum += (n - 1) * n / 2 * (a / m) + n * (b / m);
        a %= m;
        b %= m;
        const int64_t y = a * n + b;
        if (y < m) break;
        n = y / m;
        b = y % m;
        const int64_t t = a;
        a = m;
        m = t;
    }
    return sum;
}

// tokens of a unit: two halves of floor(128 / group)
__device__ __forceinline__ int half_tokens(int group) { return (kUnitRows / 2) / group; }
// cost of the units before unit i of a (sequence, head) (none of them the last one)
__device__ __forceinline__ int64_t unit_prefix(const SeqView& v, int span, int i)
{
    return floor_sum(i, kKeys, span, (int64_t)v.first + span + kKeys - 1) + (int64_t)i * kPromptUnitCost;
}
__device__ __forceinline__ int unit_tiles(int first, int n, int span, int i) { return (first + min((i + 1) * span, n) + kKeys - 1) / kKeys; }

// A worker's units in order.  Each role walks them for itself, in shared memory: what a unit needs now and
// then is read where it is needed, and the registers of the tile loops hold none of it.
struct Walk {
    int s, head, i, units;    // sequence, kv head, unit; units of a (sequence, head)
    int t0, n, first;         // the sequence's tokens, its first one's position
    int image;                // image tile of its first positions
    int from, to;             // this worker's cost of the unit
    int j0, j1, tiles;        // and its tiles
    int opening;              // the range's first unit
    int64_t left;             // cost of the range from here on (0: no more units)

    __device__ void begin(const AttnParams& p, const AttnSpace& a, const Cut& c, int64_t cost, int span)
    {
        s = c.s;
        head = c.head;
        i = c.unit;
        from = c.from;
        left = cost;
        opening = 1;
        enter(p, a, span);
        here(span);
    }
    __device__ void enter(const AttnParams& p, const AttnSpace& a, int span)
    {
        const SeqView v = seq_view(p, s);
        t0 = v.t0;
        n = v.n;
        first = v.first;
        units = (n + span - 1) / span;
        image = a.image_base[s];
    }
    __device__ void here(int span)
    {
        tiles = unit_tiles(first, n, span, i);
        to = (int)min((int64_t)tiles + kPromptUnitCost, from + left);
        j0 = max(from - kPromptUnitCost, 0);
        j1 = to - kPromptUnitCost;
        if (j1 <= 0) left = 0;  // the range ends within the unit's constant
    }
    __device__ void next(const AttnParams& p, const AttnSpace& a, int span)
    {
        left -= to - from;
        opening = 0;
        from = 0;
        if (left <= 0) return;
        if (++i == units) {
            i = 0;
            if (++head == p.heads) {
                head = 0;
                do {
                    if (++s >= p.n_seq) {
                        left = 0;
                        return;
                    }
                } while (!is_long(p, a, s, seq_view(p, s)));
                enter(p, a, span);
            }
        }
        here(span);
    }
};

template <int D>
struct PromptSmem {
    static constexpr int kSlots = D == 128 ? 5 : 8;
    unsigned char q[2][kTileBytes<D>];
    unsigned char kv[kSlots][kTileBytes<D>];   // K and V images in turn
    uint64_t kv_full[kSlots], kv_empty[kSlots];
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2], drain;
    uint32_t tmem_base;
    int abort_flag;
    Cut start;
    Walk walk[4];                              // of the two halves, the copies and the products
    float other[2][2][128];                    // what a row's two threads tell each other
};
// the search for the range's start is over before the first copy lands where it keeps its sums
static_assert(sizeof(ScanSmem<kThreads>) <= kTileBytes<64>, "scan fits a ring slot");
static_assert(sizeof(PromptSmem<128>) <= 232448 && sizeof(PromptSmem<64>) <= 232448, "shared memory");

// barriers: of the two warps that hold the two halves of the same rows' columns (64 threads, ids 1-8), of a
// half's 256 threads (ids 9, 10)
__device__ __forceinline__ bool pair_any(int id, bool say)  // whether any of them says so
{
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"((uint32_t)say), "r"(id)
        : "memory");
    return any != 0;
}
__device__ __forceinline__ void pair_sync(int id) { asm volatile("barrier.cta.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void half_sync(int h) { asm volatile("barrier.cta.sync %0, 256;" ::"r"(9 + h) : "memory"); }

// Bounded wait (about two seconds of SM clock; abandoned once another warp of the CTA has given up); the
// warp agrees on the outcome and stays converged.
__device__ __forceinline__ bool wait_for(uint64_t* mbar, uint32_t parity, const volatile int* abort_flag)
{
    bool ok = umma::mbar_try_wait(mbar, parity);
    if (!ok) {
        const long long start = clock64();
        while (!(ok = umma::mbar_try_wait_suspend(mbar, parity, 20000u)))
            if (*abort_flag || clock64() - start > (4ll << 30)) break;
    }
    return __all_sync(0xffffffffu, ok);
}

// two fp32 operations an instruction
__device__ __forceinline__ uint64_t pair2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair2(uint64_t r, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

template <int D, bool BF16, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1) kv_prompt_kernel(AttnParams p, AttnSpace a)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    using Smem = PromptSmem<D>;
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    constexpr int kSlots = Smem::kSlots;
    constexpr uint32_t kTile = kTileBytes<D>;
    constexpr uint32_t kColS = 128, kColO = 256, kTmemCols = 512;  // S of half h at 128 h, O at 256 + D h
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = p.hq / p.heads, tokens = half_tokens(group), span = 2 * tokens;
    ScanSmem<kThreads>& scan = *reinterpret_cast<ScanSmem<kThreads>*>(sm.kv[0]);
    pdl_wait();
    pdl_launch_dependents();

    // ---- this worker's range ----
    auto weight = [&](int s) {
        const SeqView v = seq_view(p, s);
        if (!is_long(p, a, s, v)) return (int64_t)0;
        const int last = (v.n + span - 1) / span - 1;
        return p.heads * (unit_prefix(v, span, last) + unit_tiles(v.first, v.n, span, last) + kPromptUnitCost);
    };
    const int64_t total = scan_total<kThreads>(p.n_seq, weight, scan);
    const int workers = (int)min((int64_t)gridDim.x, total);
    if (blockIdx.x == 0 && tid == 0) {
        a.head->prompt_total = total;
        a.head->prompt_workers = workers;
    }
    if ((int)blockIdx.x >= workers) return;
    const int64_t lo = cut_start(total, workers, blockIdx.x), hi = cut_start(total, workers, blockIdx.x + 1);
    {
        int64_t before;
        const int s = scan_find<kThreads>(p.n_seq, lo, weight, scan, before);
        if (warp == 0) {
            const SeqView v = seq_view(p, s);
            const int units = (v.n + span - 1) / span;
            const int64_t per_head = unit_prefix(v, span, units - 1) + unit_tiles(v.first, v.n, span, units - 1) + kPromptUnitCost;
            const int head = (int)((lo - before) / per_head);
            const int64_t rest = lo - before - head * per_head;
            const int i = warp_find(units, rest, [&](int u) { return unit_prefix(v, span, u); });
            if (lane == 0) {
                const int from = (int)(rest - unit_prefix(v, span, i));
                sm.start = Cut{s, head, i, max(from - kPromptUnitCost, 0), unit_tiles(v.first, v.n, span, i), from, lo};
                a.prompt_cut[blockIdx.x] = sm.start;
            }
        }
    }
    if (warp == kMmaWarp) umma::tmem_alloc(&sm.tmem_base, kTmemCols);
    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            umma::mbar_init(&sm.kv_full[i], 1);
            umma::mbar_init(&sm.kv_empty[i], 1);
        }
        for (int h = 0; h < 2; ++h) {
            umma::mbar_init(&sm.q_full[h], 256);
            umma::mbar_init(&sm.s_full[h], 1);
            umma::mbar_init(&sm.p_full[h], 256);
            umma::mbar_init(&sm.o_full[h], 1);
        }
        umma::mbar_init(&sm.drain, 1);
        sm.abort_flag = 0;
    }
    __syncthreads();  // the range's start
    if (tid < 4) sm.walk[tid].begin(p, a, sm.start, hi - lo, span);
    umma::fence_proxy_async();  // the scan's shared memory goes to the copies
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = sm.tmem_base;
    const volatile int* abort_flag = &sm.abort_flag;

#define GDN_KV_WAIT(mbar, parity)                         \
    do {                                                  \
        if (!wait_for((mbar), (parity), abort_flag)) {    \
            if (lane == 0) {                              \
                sm.abort_flag = 1;                        \
                atomicOr(&a.head->error, kAttnTimeout);   \
            }                                             \
            goto done;                                    \
        }                                                 \
    } while (0)

    if (warp >= kLoadWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp > kMmaWarp) goto done;
    if (warp == kLoadWarp) {
        // ---- copies: K and V of each tile in turn through the ring ----
        Walk& w = sm.walk[2];
        uint32_t n = 0;  // copies issued
        while (w.left > 0) {
            const unsigned char* src = a.images + ((size_t)(w.image + w.j0) * p.heads + w.head) * (2 * kTile);
            const size_t stride = (size_t)p.heads * (2 * kTile);
            for (int j = 2 * (w.j1 - w.j0); j > 0; --j, ++n) {
                const uint32_t slot = n % kSlots;
                if (n >= kSlots && !wait_for(&sm.kv_empty[slot], (n / kSlots - 1) & 1, abort_flag)) {
                    if (lane == 0) {
                        sm.abort_flag = 1;
                        atomicOr(&a.head->error, kAttnTimeout);
                    }
                    goto copies_done;
                }
                if (lane == 0) {
                    umma::mbar_arrive_expect_tx(&sm.kv_full[slot], kTile);
                    umma::bulk_g2s(sm.kv[slot], j & 1 ? src + kTile : src, kTile, &sm.kv_full[slot]);
                }
                if (j & 1) src += stride;
            }
            __syncwarp();
            if (lane == 0) w.next(p, a, span);
            __syncwarp();
        }
    copies_done:
        // no copy may be in flight when the CTA leaves (copies end by themselves; the limit is a formality)
        for (uint32_t i = n > kSlots ? n - kSlots : 0; i < n; ++i)
            for (int k = 0; k < 1 << 20 && !umma::mbar_try_wait(&sm.kv_full[i % kSlots], (i / kSlots) & 1); ++k) {}
        goto done;
    }
    if (warp == kMmaWarp) {
        // ---- products, issued by lane 0 ----
        constexpr uint32_t id_s = umma::idesc_f16(128, kKeys, false, false);
        constexpr uint32_t id_o = umma::idesc_f16(128, D, false, true);  // V: channels (N) contiguous
        Walk& w = sm.walk[3];
        uint32_t n = 0;         // ring position of the current tile's K
        uint32_t q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
        // descriptors of the first tiles; the others lie a whole number of tiles behind them
        const uint64_t q_desc = umma::desc_sw128(umma::smem_u32(sm.q[0]), 16, 1024);
        const uint64_t k_desc = umma::desc_sw128(umma::smem_u32(sm.kv[0]), 16, 1024);
        const uint64_t v_desc = umma::desc_sw128(umma::smem_u32(sm.kv[0]), kPlane, 1024);
        auto scores = [&](int h, uint32_t at) {
            if (lane == 0) {
                const uint64_t da = q_desc + h * (kTile >> 4), db = k_desc + (at % kSlots) * (kTile >> 4);
#pragma unroll 4
                for (int ks = 0; ks < D / 16; ++ks) {  // 16 channels: 32 bytes of a plane's rows
                    const uint32_t step = (ks >> 2) * (kPlane >> 4) + 2 * (ks & 3);
                    umma::mma_bf16(tmem + h * kColS, da + step, db + step, id_s, ks != 0);
                }
                umma::commit(&sm.s_full[h]);
            }
            __syncwarp();
        };
        auto outputs = [&](int h, uint32_t at, bool start) {
            if (lane == 0) {
                const uint64_t db = v_desc + (at % kSlots) * (kTile >> 4);
#pragma unroll 4
                for (int ks = 0; ks < kKeys / 16; ++ks)  // 16 keys: two atoms of 8 rows
                    umma::mma_ts(tmem + kColO + h * D, tmem + h * kColS + 64 * (ks >> 2) + 8 * (ks & 3), db + ks * (2048 >> 4), id_o, !(start && ks == 0));
                umma::commit(&sm.o_full[h]);
            }
            __syncwarp();
        };
        auto release = [&](uint32_t at) {
            if (lane == 0) umma::commit(&sm.kv_empty[at % kSlots]);
            __syncwarp();
        };
        while (w.left > 0) {
            const bool both = (2 * w.i + 1) * tokens < w.n;  // the second half has rows
            GDN_KV_WAIT(&sm.kv_full[n % kSlots], (n / kSlots) & 1);
            GDN_KV_WAIT(&sm.q_full[0], q_phase[0]);
            q_phase[0] ^= 1u;
            umma::fence_after_sync();
            scores(0, n);
            if (both) {
                GDN_KV_WAIT(&sm.q_full[1], q_phase[1]);
                q_phase[1] ^= 1u;
                umma::fence_after_sync();
                scores(1, n);
            }
            release(n);
            const int count = w.j1 - w.j0;
            for (int j = 0; j < count; ++j, n += 2) {
                const bool again = j + 1 < count;
                GDN_KV_WAIT(&sm.kv_full[(n + 1) % kSlots], ((n + 1) / kSlots) & 1);
                GDN_KV_WAIT(&sm.p_full[0], p_phase[0]);
                p_phase[0] ^= 1u;
                umma::fence_after_sync();
                outputs(0, n + 1, j == 0);
                if (again) {
                    GDN_KV_WAIT(&sm.kv_full[(n + 2) % kSlots], ((n + 2) / kSlots) & 1);
                    scores(0, n + 2);
                }
                if (both) {
                    GDN_KV_WAIT(&sm.p_full[1], p_phase[1]);
                    p_phase[1] ^= 1u;
                    umma::fence_after_sync();
                    outputs(1, n + 1, j == 0);
                }
                release(n + 1);
                if (again) {
                    if (both) scores(1, n + 2);
                    release(n + 2);
                }
            }
            __syncwarp();
            if (lane == 0) w.next(p, a, span);
            __syncwarp();
        }
        goto done;
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // ---- softmax: a row's two threads share a tile's columns ----
        // A wait that expires is recorded and its warp goes on, with waits that no longer wait: a half's warps
        // meet at barriers, and every loop ends by itself.
        auto await = [&](uint64_t* mbar, uint32_t parity) {
            if (!wait_for(mbar, parity, abort_flag) && lane == 0) {
                sm.abort_flag = 1;
                atomicOr(&a.head->error, kAttnTimeout);
            }
        };
        const int h = warp >> 3, part = (warp >> 2) & 1, r = (warp & 3) * 32 + lane, pair = 1 + 4 * h + (warp & 3);
        Walk& w = sm.walk[h];
        float* const mine = &sm.other[h][part][r];
        const float* const others = &sm.other[h][part ^ 1][r];
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lane_off + h * kColS + 64 * part, t_o = tmem + lane_off + kColO + h * D + part * (D / 2);
        const int i_tok = r / group, qh = r - i_tok * group;
        uint32_t s_phase = 0, o_phase = 0;  // o_phase: parity of the next PV product's completion
        // 32 of the thread's scores, -infinity from the column after `last` on
        auto scores = [&](int c, bool ends, int last, float (&x)[32]) {
            umma::tmem_ld32(t_s + 32 * c, x);
            umma::tmem_wait_ld();
            if (ends)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (32 * c + e > last) x[e] = -INFINITY;
        };
        for (; w.left > 0; half_sync(h)) {
            // (a second half without rows does nothing)
            if ((2 * w.i + h) * tokens < w.n) {
            const int tok = (2 * w.i + h) * tokens + i_tok;
            const bool valid = i_tok < tokens && tok < w.n;
            // the row's channels to shared memory in fp16
            float coef;
            {
                constexpr int C = D / 16;  // 16-byte pieces a thread
                const uint16_t* src = p.q + (int64_t)(w.t0 + tok) * p.q_stride + (w.head * group + qh) * D + part * (D / 2);
                uint4 raw[C];
                uint32_t amax = 0;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    raw[c] = valid ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0u, 0u, 0u, 0u);
                    float x[8];
                    widen8<BF16>(raw[c], x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) amax = max(amax, __float_as_uint(x[e]) & 0x7fffffffu);
                }
                *mine = __uint_as_float(amax);
                pair_sync(pair);
                amax = max(amax, __float_as_uint(*others));
                float mul, back;
                row_unit(amax, mul, back);
                if (p.scale < 0.0f) mul = -mul;  // scores times |scale|: a row's largest is its maximum's
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    float x[8];
                    widen8<BF16>(raw[c], x);
                    *reinterpret_cast<uint4*>(sm.q[h] + image_off(r, part * C + c)) =
                        make_uint4(narrow2<false>(x[0] * mul, x[1] * mul), narrow2<false>(x[2] * mul, x[3] * mul),
                                   narrow2<false>(x[4] * mul, x[5] * mul), narrow2<false>(x[6] * mul, x[7] * mul));
                }
                umma::fence_proxy_async();
                umma::mbar_arrive(&sm.q_full[h]);
                const float2 norm = a.norm[(size_t)w.image * p.heads + w.head];
                // (above 0, so that a masked score of -infinity stays one whatever the scale)
                coef = fmaxf(back * (fabsf(p.scale) * kLog2e) * (norm.x * (1.0f / kUp<E4M3>)), 1e-35f);
            }
            // the last of the thread's columns that the row sees, in the tile in hand, and whether a tile ends
            // before the half's first row does
            int last = (valid ? w.first + tok : -1) - (w.j0 * kKeys + 64 * part);
            int spare = w.first + (2 * w.i + h) * tokens - (w.j0 * kKeys + kKeys - 1);
            float m = -INFINITY, l = 0.0f;
            const int count = w.j1 - w.j0;
#pragma unroll 1
            for (int j = 0; j < count; ++j, last -= kKeys, spare -= kKeys) {
                await(&sm.s_full[h], s_phase);
                s_phase ^= 1u;
                umma::fence_after_sync();
                // (32 of the thread's 64 scores at a time: all of them and their weights do not fit its registers)
                const bool ends = spare < 0;
                float x[32], top = -INFINITY;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    scores(c, ends, last, x);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) top = fmaxf(top, fmaxf(x[e], x[e + 1]));
                }
                top *= coef;
                if (pair_any(pair, top > m + kLazy)) {
                    *mine = top;
                    pair_sync(pair);
                    top = fmaxf(top, *others);
                    float f = 1.0f;
                    if (top > m + kLazy) {
                        f = ex2(m - top);
                        m = top;
                        l *= f;
                    }
                    if (j > 0 && __any_sync(0xffffffffu, f != 1.0f)) {  // O holds the products up to tile j - 1
                        await(&sm.o_full[h], o_phase ^ 1u);
                        umma::fence_after_sync();
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            float o[16];
                            uint32_t u[16];
                            umma::tmem_ld16(t_o + 16 * c, o);
                            umma::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e] * f);
                            umma::tmem_st16(t_o + 16 * c, u);
                        }
                    }
                }
                const float off = kWeightShift - (m == -INFINITY ? 0.0f : m);
                const uint64_t coef2 = pair2(coef, coef), off2 = pair2(off, off);
                uint64_t sum[2] = {0, 0};
                uint32_t u[16], u1[16];
                auto weights = [&](uint32_t (&to)[16]) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float w0, w1;
                        unpair2(fma2(pair2(x[2 * e], x[2 * e + 1]), coef2, off2), w0, w1);
                        w0 = ex2(w0);
                        w1 = ex2(w1);
                        sum[e & 1] = add2(sum[e & 1], pair2(w0, w1));
                        to[e] = narrow2<false>(w0, w1);
                    }
                };
                // the second 32 are still there; the first ones come again, then both go where those were
                weights(u1);
                scores(0, ends, last, x);
                umma::tmem_st16(t_s + 16, u1);
                weights(u);
                umma::tmem_st16(t_s, u);
                umma::tmem_wait_st();
                umma::fence_before_sync();
                umma::mbar_arrive(&sm.p_full[h]);
                float s0, s1;
                unpair2(add2(sum[0], sum[1]), s0, s1);
                l += s0 + s1;
                o_phase ^= 1u;
            }
            pair_sync(pair);  // the last tile's maxima are read
            *mine = l;
            pair_sync(pair);
            l += *others;
            pair_sync(pair);  // the sums are read
            await(&sm.o_full[h], o_phase ^ 1u);
            umma::fence_after_sync();
            const float unit = a.norm[(size_t)w.image * p.heads + w.head].y * (1.0f / kUp<E4M3>);
            const bool whole = w.j0 == 0 && w.j1 == w.tiles;
            const int slot = 2 * blockIdx.x + (w.opening ? 0 : 1), row = 128 * h + r;
            const float scale = whole ? (l == 0.0f ? 0.0f : unit / l) : unit;
            uint16_t* const dst = p.y + ((int64_t)(w.t0 + tok) * p.hq + w.head * group + qh) * D + part * (D / 2);
            if (!whole && part == 0) a.prompt_stat[(size_t)slot * kUnitRows + row] = make_float2(m, l);
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                float o[32];
                umma::tmem_ld32(t_o + 32 * c, o);
                umma::tmem_wait_ld();
                if (whole) {
                    if (valid)
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            *reinterpret_cast<uint4*>(dst + 32 * c + e) =
                                make_uint4(narrow2<BF16>(o[e] * scale, o[e + 1] * scale), narrow2<BF16>(o[e + 2] * scale, o[e + 3] * scale),
                                           narrow2<BF16>(o[e + 4] * scale, o[e + 5] * scale), narrow2<BF16>(o[e + 6] * scale, o[e + 7] * scale));
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        a.prompt_out[((size_t)slot * (D / 4) + part * (D / 8) + 8 * c + e / 4) * kUnitRows + row] =
                            make_float4(o[e] * scale, o[e + 1] * scale, o[e + 2] * scale, o[e + 3] * scale);
                }
            }
            umma::fence_before_sync();  // O read before the next unit's products (which wait for this thread's weights)
            }
            half_sync(h);  // the unit is read
            if (part == 0 && r == 0) w.next(p, a, span);
        }
    }
done:
    // every product issued has ended before TMEM and shared memory go
    __syncwarp();
    if (warp == kMmaWarp) {
        if (lane == 0) {
            umma::commit(&sm.drain);
            for (int k = 0; k < 1 << 20 && !umma::mbar_try_wait(&sm.drain, 0); ++k) {}
        }
        __syncwarp();
    }
    umma::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) umma::tmem_dealloc(tmem, kTmemCols);
#undef GDN_KV_WAIT
}

// Block (w, 32 rows): where range w is the first that begins inside a unit, joins that unit's parts.  Four
// threads share a row's channels.
constexpr int kJoinThreads = 128;
template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) kv_prompt_join_kernel(AttnParams p, AttnSpace a)
{
    const int group = p.hq / p.heads, tokens = half_tokens(group);
    pdl_wait();
    pdl_launch_dependents();
    const int w = (int)blockIdx.x + 1, workers = a.head->prompt_workers;
    if (w >= workers) return;
    const Cut cut = a.prompt_cut[w];
    const int64_t total = a.head->prompt_total, begin = cut.lo - cut.from, prev = a.prompt_cut[w - 1].lo;
    if (cut.j0 == 0 || prev > begin + kPromptUnitCost) return;
    const int last = cut_of(total, workers, begin + kPromptUnitCost + cut.tiles - 1);
    const int row = blockIdx.y * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
    const int h = row >> 7, r = row & 127, i_tok = r / group, qh = r - i_tok * group;
    const int t0 = cu_at(p.cu_seqlens, cut.s, p.T), n = cu_at(p.cu_seqlens, cut.s + 1, p.T) - t0;
    const int tok = (2 * cut.unit + h) * tokens + i_tok;
    if (i_tok >= tokens || tok >= n) return;
    constexpr int E = D / 16;  // float4s a thread
    float top = -INFINITY, sum = 0.0f;
    float4 acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = w - 1; i <= last; ++i) {
        const int slot = 2 * i + (i == w - 1 && prev < begin ? 1 : 0);
        const float2 st = a.prompt_stat[(size_t)slot * kUnitRows + row];
        const float next = fmaxf(top, st.x), ref = next == -INFINITY ? 0.0f : next;
        const float f0 = exp2f(top - ref), f1 = exp2f(st.x - ref);
        sum = sum * f0 + st.y * f1;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float4 o = a.prompt_out[((size_t)slot * (D / 4) + part * E + e) * kUnitRows + row];
            acc[e].x = acc[e].x * f0 + o.x * f1;
            acc[e].y = acc[e].y * f0 + o.y * f1;
            acc[e].z = acc[e].z * f0 + o.z * f1;
            acc[e].w = acc[e].w * f0 + o.w * f1;
        }
        top = next;
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint2* dst = reinterpret_cast<uint2*>(p.y + ((int64_t)(t0 + tok) * p.hq + cut.head * group + qh) * D) + part * E;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[e] = make_uint2(narrow2<BF16>(acc[e].x * inv, acc[e].y * inv), narrow2<BF16>(acc[e].z * inv, acc[e].w * inv));
}

template <int D, bool BF16, bool E4M3>
cudaError_t launch(const AttnParams& p, const AttnSpace& a, int sms, cudaStream_t stream)
{
    const int64_t items = (int64_t)a.image_tiles * p.heads;
    cudaError_t e = launch_k(kv_image_kernel<D, E4M3>, dim3((unsigned)(items < sms * 8 ? items : sms * 8)), dim3(kImageThreads), 0, stream, true, p, a);
    if (e != cudaSuccess) return e;
    auto kernel = kv_prompt_kernel<D, BF16, E4M3>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(PromptSmem<D>));
    if (e != cudaSuccess) return e;
    const int grid = sms < kPromptMaxWorkers ? sms : kPromptMaxWorkers;
    e = launch_k(kernel, dim3(grid), dim3(kThreads), sizeof(PromptSmem<D>), stream, true, p, a);
    if (e != cudaSuccess || grid == 1) return e;
    return launch_k(kv_prompt_join_kernel<D, BF16>, dim3(grid - 1, kUnitRows / 32), dim3(kJoinThreads), 0, stream, true, p, a);
}

template <int D>
cudaError_t launch_types(const AttnParams& p, const AttnSpace& a, int sms, cudaStream_t stream)
{
    if (p.format == 1) return p.bf16 ? launch<D, true, true>(p, a, sms, stream) : launch<D, false, true>(p, a, sms, stream);
    return p.bf16 ? launch<D, true, false>(p, a, sms, stream) : launch<D, false, false>(p, a, sms, stream);
}

}  // namespace

cudaError_t launch_kv_prompt(const AttnParams& p, const AttnSpace& a, int sms, cudaStream_t stream)
{
    return p.dim == 64 ? launch_types<64>(p, a, sms, stream) : launch_types<128>(p, a, sms, stream);
}

}  // namespace gdn
