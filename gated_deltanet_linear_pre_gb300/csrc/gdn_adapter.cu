// gdn_adapter.cu -- low-rank adapters of many sequences added to a shared projection's output.
//
//   h[t]     = down[a] x[t]                          (rank values, fp32)
//   y_out[t] = y[t] + scale[a] * up[a]^T h[t]        a = the adapter of t's sequence
//
// Bound by HBM: x and y are read and y_out written once, an adapter's weights
// once for every 128 tokens that use them (from L2 after the first).
//
// Tiles of a good many of up to 128 tokens go through the tensor cores, in two
// launches: adapter_down (h, fp32, to the workspace) and adapter_up (its product with
// up, and the sum with y).  A unit of work is 64 channels (of x, of y) of a tile.
// Each of 152 CTAs, one an SM, takes a range of all units of equal cost, cutting a
// tile where its range ends; a tile that lies in several ranges has its h in several
// sums, which adapter_up adds in order.  One warp copies (TMA boxes of 64 channels,
// into a ring of stages of 128-byte swizzled rows), far ahead of the others; one
// issues the products (tcgen05, 16-bit operands, fp32 sums in TMEM); eight, or in
// adapter_up two teams of eight in turn, take what comes of them on.  h enters its
// product there as hi + lo in the weights' type: 16 bits of it in bf16, 21 of its
// row's largest in fp16, far below the rounding of y_out.
//
// Smaller tiles (single tokens, drafts) read weights that nobody shares; what counts
// for them is the chain from the batch's lengths to the last store.  They take two
// kernels of their own, without rings or ranges, behind the others'; a small batch goes
// that way alone.
//
// Measured (one GB300; the floor is the bytes that have to move, at a plain copy's rate): 8 prompts of 1 to 4096 tokens,
// rank 64, 4096 to 6144, fp16 137 us, 78% of the floor's rate (298 in the first form, by mma.sync in tiles of 64 tokens);
// one token of 64 sequences, rank 16, 4096 to 10240, 8.7 us replayed (floor 2.8); a 3001-token prompt beside 39 drafts,
// ranks of 8 to 128, 2048 to 10240, 82 us (floor 25; 181 in the first form); 8192 tokens, 2048 to 10240, rank 16 74 us,
// 64 80, 128 95 (floor 55).  What is left: the start of either kernel (some 5 us: lengths, ranges, the first copies; h), and
// reads and writes mixed, 5.5 TB/s in adapter_up; where few tokens stand beside a prompt, few_down and few_up, which wait
// for the kernel in front of them.
#include <algorithm>
#include <type_traits>

#include "gdn_adapter_index.cuh"
#include "gdn_kv.cuh"
#include "gdn_tensor_map.cuh"
#include "umma.cuh"

namespace gdn {
namespace {

constexpr int kWorkers = 8;                          // warps
constexpr int kCopier = kWorkers;                    // the warp that copies
constexpr int kProduct = kWorkers + 1;               // the warp that issues products
constexpr int kThreads = (kProduct + 1) * 32;
// adapter_up has two teams of workers, which take its units in turn: a unit is a chain (product, TMEM, y, y_out).  One team:
// 8192 tokens, 2048 to 10240, rank 16 75.2 us for 73.6, rank 64 81.9 for 80.2, rank 128 96.3 for 95.3.
constexpr int kTeams = kAdapterTeams;
constexpr int kUpWorkers = kWorkers * kTeams;
constexpr int kUpThreads = (kUpWorkers + 2) * 32;
constexpr int kTile = kAdapterTile;
constexpr int kK = 64;                               // channels of a unit: rows of 128 bytes in shared memory
constexpr int kRow = kK * 2;
constexpr int kCtas = kAdapterCtas;
constexpr int kTokenBytes = kTile * kRow;
constexpr int kRing = 4;                             // slots of chunks' products in TMEM
static_assert(kRing % kTeams == 0, "a slot is always the same team's");
constexpr int kPartsOut = 16;                        // ranges of a tile's y at most, less one
constexpr uint32_t kPolls = 1u << 18;                // of a wait: some two seconds
constexpr int kColumnD = 256;                        // adapter_up's TMEM: h in the first R columns, products from here on

// Stages leave some L1: 8192 tokens, 2048 to 10240, rank 64, 6 stages 80.2 us, 5 81.6, 7 82.6; rank 128, 4 and 5 95.3, 3 102.9;
// 255 single tokens beside 1500, rank 128, 5120 to 5120, 4 114.1, 5 120.5
template <int R> constexpr int kStages = R > 64 ? 4 : R > 32 ? 6 : 7;
template <int R> constexpr int kStageBytes = kTokenBytes + R * kRow;
constexpr int kResultBytes = 32 * 64;                // a worker's part of a chunk of y_out, on its way out
template <int R> constexpr size_t kSmem = 1024 + kStages<R> * kStageBytes<R> + kUpWorkers * kResultBytes;

// tensor maps of the tokens (x or y): boxes of kTile rows; and of the weights: boxes of `rank` and of 8 rows
struct Maps {
    CUtensorMap tokens, weights, weights8;
};

__device__ __forceinline__ void workers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kUpWorkers * 32) : "memory"); }  // adapter_up's

// byte offset of 16-byte piece `piece` of a row in a tile swizzled over 128 bytes
__device__ __forceinline__ uint32_t place(int row, int piece) { return row * kRow + ((piece ^ (row & 7)) << 4); }

// ---- who does what --------------------------------------------------------------

// What a unit costs, in steps of some 2 ns: rows of 128 bytes copied and written, fitted to the time that a CTA took for
// ranges of one kind (8 prompts with rank 64, one with rank 72), with one team of workers; not fitted again since there are
// two.  A tile copies the rows of a whole one.
__device__ __forceinline__ int cost_in(int rank) { return rank > 0 ? 144 + rank : 0; }
__device__ __forceinline__ int cost_out(int rank, bool copied) { return rank > 0 ? 160 + 2 * rank : copied ? 192 : 0; }

template <bool IN>
__device__ __forceinline__ int unit_cost(const AdapterParams& p, int n, int rank)
{
    return n <= p.few ? 0 : IN ? cost_in(rank) : cost_out(rank, p.y_out != p.y);
}

__device__ __forceinline__ int rank_of(const AdapterParams& p, int s, int& id)
{
    id = __ldg(p.ids + s);
    if (id < 0 || id >= p.n_adapters) {
        id = -1;
        return 0;
    }
    return p.ranks ? min(max(__ldg(p.ranks + id), 0), p.rank) : p.rank;
}

template <bool IN>
__device__ __forceinline__ int64_t sequence_cost(const AdapterParams& p, int s)
{
    const int n = cu_at(p.cu_seqlens, s + 1, p.T) - cu_at(p.cu_seqlens, s, p.T);
    int id;
    const int rank = rank_of(p, s, id);
    return n <= 0 ? 0 : (IN ? p.chunks_in : p.chunks_out) * ((int64_t)(n / kTile) * unit_cost<IN>(p, kTile, rank) + unit_cost<IN>(p, n % kTile, rank));
}

// units [c_lo, c_hi) of one tile
struct Piece {
    int start, n, id, rank;
    int slot;               // the tile's own number, below T / kTile + n_seq
    int c_lo, c_hi;
    int cost;               // of a unit
    int64_t before;         // cost of all units in front of the tile
};

// Walks the tiles of a range of costs [lo, hi).  A whole warp, in step.
template <bool IN>
struct Walk {
    int s, k;               // the next sequence and its next tile
    int64_t at, lo, hi;     // cost of all units in front of that tile; the range

    __device__ bool next(const AdapterParams& p, Piece& t)
    {
        const int chunks = IN ? p.chunks_in : p.chunks_out;
        while (at < hi && s < p.n_seq) {
            if (k == 0) {   // pass over sequences that cost nothing, 32 at a time
                const int mine = s + (threadIdx.x & 31);
                const uint32_t some = __ballot_sync(0xffffffffu, mine < p.n_seq && sequence_cost<IN>(p, min(mine, p.n_seq - 1)) > 0);
                if (some == 0) {
                    s += 32;
                    continue;
                }
                s += __ffs(some) - 1;
            }
            const int first = cu_at(p.cu_seqlens, s, p.T), end = cu_at(p.cu_seqlens, s + 1, p.T);
            t.start = first + k * kTile;
            t.n = min(kTile, end - t.start);
            t.rank = rank_of(p, s, t.id);
            t.slot = first / kTile + s + k;
            t.cost = unit_cost<IN>(p, t.n, t.rank);
            t.before = at;
            if (t.start + t.n >= end) {
                ++s;
                k = 0;
            } else {
                ++k;
            }
            if (t.cost == 0) continue;
            const int whole = t.cost * chunks;  // below 2^20
            at += whole;
            t.c_lo = ((int)min(max(lo - t.before, (int64_t)0), (int64_t)whole) + t.cost - 1) / t.cost;
            t.c_hi = ((int)min(hi - t.before, (int64_t)whole) + t.cost - 1) / t.cost;
            if (t.c_lo < t.c_hi) return true;
        }
        return false;
    }
};

struct PlanSmem {
    int64_t warp_sum[2][kThreads / 32];
    AdapterStart start;
};

// Sum over the threads in front of this one, and over all
__device__ __forceinline__ int64_t block_exclusive(int64_t (&warp_sum)[kThreads / 32], int64_t v, int64_t& all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int64_t before = 0;
    all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        all += warp_sum[w];
    }
    return before + incl - v;
}

// Where this CTA's ranges of x's and of y's units begin; every CTA goes over all sequences, a run of them a thread.
// All threads.
__device__ __forceinline__ void find_starts(const AdapterParams& p, PlanSmem& sm, AdapterStart& out)
{
    const int each = (p.n_seq + kThreads - 1) / kThreads, first = min(p.n_seq, (int)threadIdx.x * each), last = min(p.n_seq, first + each);
    int64_t mine[2] = {0, 0}, total[2], at[2];
    for (int s = first; s < last; ++s) {
        mine[0] += sequence_cost<true>(p, s);
        mine[1] += sequence_cost<false>(p, s);
    }
    at[0] = block_exclusive(sm.warp_sum[0], mine[0], total[0]);
    at[1] = block_exclusive(sm.warp_sum[1], mine[1], total[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        AdapterStart& start = i ? out : sm.start;
        // a CTA is worth 4 units of the largest tiles, and a tile is cut into `parts` + 1 at most
        const int chunks = i ? p.chunks_out : p.chunks_in, parts = i ? kPartsOut : p.parts_in;
        const int most = i ? cost_out(p.rank, true) : cost_in(p.rank);
        const int64_t share = max((total[i] + kCtas - 1) / kCtas, (int64_t)most * max(4, (chunks + parts - 1) / parts)), lo = share * blockIdx.x;
        if (threadIdx.x == 0) {
            start.share = share;
            if (lo >= total[i]) start.s = p.n_seq;  // no work
        }
        if (lo < at[i] || lo >= at[i] + mine[i]) continue;
        for (int s = first; s < last; ++s) {
            const int64_t c = i ? sequence_cost<false>(p, s) : sequence_cost<true>(p, s);
            if (lo < at[i] + c) {
                int id;
                const int rank = rank_of(p, s, id);
                const int tile = chunks * (i ? unit_cost<false>(p, kTile, rank) : unit_cost<true>(p, kTile, rank));
                start.s = s;
                start.k = (int)((lo - at[i]) / tile);
                start.before = at[i] + (int64_t)start.k * tile;
                break;
            }
            at[i] += c;
        }
    }
}

// ---- hand-offs ------------------------------------------------------------------

// Every wait is bounded; after one that has expired the rest of the CTA's waits are passed over, no copy or product is
// begun any more, those under way are waited for, and the CTA records that the call's outputs are invalid.
// A barrier's parity tells two turns apart, no more, so nobody may fall a turn behind or run one ahead.  The copier and the
// product warp wait for every stage, in order; the product warp for every slot of products too.  A worker passes over
// the other team's units without a wait, and is held by its own: slots go to units in turn and kRing is a multiple of the
// teams, so a slot is always the same team's; a slot's next product waits for its 8 arrivals (d_empty), and a stage's
// next copy for those of the team whose unit it held (empty, with the product warp's).  A worker waits for its slot (d_full)
// before it looks at the stage, which was full before that product began and stays so until the worker's own arrival.
// adapter_down's workers wait for every tile's slot; its stages are freed by their products.
struct Shared {
    uint64_t full[8], empty[8];           // stages of the ring
    uint64_t d_full[kRing], d_empty[kRing];
    uint64_t h_full;                      // h is in TMEM (adapter_up)
    uint64_t last;                        // every product is done
    uint32_t tmem;
    int expired;
    float factor[kTile];
    float most[4][kTile];
};

__device__ __forceinline__ void wait(Shared& sm, uint64_t* mbar, uint32_t parity)
{
    volatile int* expired = &sm.expired;
    for (uint32_t i = 0; i < kPolls; ++i)
        if (umma::mbar_try_wait(mbar, parity) || *expired) return;
    *expired = 1;
}

__device__ __forceinline__ bool expired(Shared& sm) { return *(volatile int*)&sm.expired; }

// a wait for what this CTA has under way, which no other expired wait cuts short
__device__ __forceinline__ void drain(uint64_t* mbar, uint32_t parity)
{
    umma::mbar_wait(mbar, parity, kPolls);
}

__device__ __forceinline__ void shared_begin(Shared& sm, int columns, int empty_count, int workers)
{
    if (threadIdx.x == 0) {
        for (int i = 0; i < 8; ++i) {
            umma::mbar_init(&sm.full[i], 1);
            umma::mbar_init(&sm.empty[i], empty_count);
        }
        for (int i = 0; i < kRing; ++i) {
            umma::mbar_init(&sm.d_full[i], 1);
            umma::mbar_init(&sm.d_empty[i], kWorkers);
        }
        umma::mbar_init(&sm.h_full, workers);
        umma::mbar_init(&sm.last, 1);
        sm.expired = 0;
    }
    if (threadIdx.x < 32) umma::tmem_alloc(&sm.tmem, columns);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
}

__device__ __forceinline__ void shared_end(Shared& sm, int columns, int32_t* status)
{
    umma::fence_before_sync();
    __syncthreads();
    if (threadIdx.x < 32) umma::tmem_dealloc(sm.tmem, columns);
    if (threadIdx.x == 0) *status = sm.expired;
}

// A position in the ring of stages
template <int R>
struct Ring {
    uint32_t stage = 0, phase = 0;
    __device__ void next()
    {
        if (++stage == kStages<R>) {
            stage = 0;
            phase ^= 1;
        }
    }
};

// The copying warp: the stages of a piece, in order.  Rows of tokens behind the tile's own are its neighbours', and
// what comes of them goes nowhere.
template <int R>
__device__ __forceinline__ void copy_piece(const AdapterParams& p, const Piece& t, const Maps& maps, Shared& sm, uint32_t base, Ring<R>& at, uint32_t& issued)
{
    const int rows = t.rank == 0 ? 0 : t.rank <= 8 ? 8 : p.rank, row = t.rank > 0 ? t.id * p.rank : 0;
    for (int c = t.c_lo; c < t.c_hi; ++c, at.next()) {
        wait(sm, &sm.empty[at.stage], at.phase ^ 1);
        __syncwarp();
        if (__any_sync(0xffffffffu, expired(sm))) return;
#ifdef GDN_ADAPTER_SELFTEST_WITHHOLD_COPY
        if (issued++ == 0) continue;  // tests: the CTA's first copy is left out
        if (umma::elect_one()) {
#else
        ++issued;
        if (umma::elect_one()) {
#endif
            const uint32_t to = base + at.stage * kStageBytes<R>;
            uint64_t* full = &sm.full[at.stage];
            umma::mbar_arrive_expect_tx(full, kTokenBytes + rows * kRow);
            umma::tensor_g2s_2d(to, &maps.tokens, c * kK, t.start, full);
            if (rows) umma::tensor_g2s_2d(to + kTokenBytes, rows == 8 ? &maps.weights8 : &maps.weights, c * kK, row, full);
        }
        __syncwarp();
    }
}

template <bool BF16, int M, int N>
constexpr uint32_t idesc(bool b_mn_major) { return BF16 ? umma::idesc_bf16(M, N, false, b_mn_major) : umma::idesc_f16(M, N, false, b_mn_major); }

// ---- down -----------------------------------------------------------------------

template <bool BF16, int R>
__global__ void __launch_bounds__(kThreads, 1) adapter_down_kernel(const __grid_constant__ AdapterParams p, const __grid_constant__ Maps maps)
{
    extern __shared__ unsigned char smem[];
    __shared__ Shared sm;
    __shared__ PlanSmem plan;
    constexpr int kColumns = R * 2 < 32 ? 32 : R * 2;
    unsigned char* ring = smem + ((1024 - (umma::smem_u32(smem) & 1023)) & 1023);
    const uint32_t base = umma::smem_u32(ring);
    // In this order: nobody waits here for another kernel while it holds TMEM that the other has yet to get.
    pdl_wait();
    shared_begin(sm, kColumns, 1, kWorkers);  // a stage is free when its products are done
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    find_starts(p, plan, p.starts[blockIdx.x]);
    __syncthreads();
    const int64_t share = plan.start.share;
    Walk<true> walk{plan.start.s, plan.start.k, plan.start.before, share * blockIdx.x, share * (blockIdx.x + 1)};
    if (walk.s >= p.n_seq) walk.hi = walk.at;
    Piece t;
    if (warp < kWorkers) {
        uint32_t tiles = 0;
        while (walk.next(p, t)) {
            // the range that a tile begins in has its sums in the tokens' places, every other its own; [rank][tokens],
            // as a warp has a row a lane here and where it reads them (rows of `rank`, when there was one team: 89.9 us for
            // 86.0, 8192 tokens, rank 64)
            float* h = p.h + h_place(p.T, p.rank, blockIdx.x, t.start, t.before >= walk.lo);
            if (tid == 0 && t.c_lo == 0) {
                const int64_t at_last = t.before + (int64_t)(p.chunks_in - 1) * t.cost;
                int ends = blockIdx.x;
                for (int64_t hi = walk.hi; hi <= at_last; hi += share) ++ends;
                p.parts[t.slot] = make_int2(blockIdx.x, ends);
            }
            const uint32_t d = tiles & 1;
            wait(sm, &sm.d_full[d], (tiles >> 1) & 1);
            umma::fence_after_sync();
            const int row = (warp & 3) * 32 + lane;
#pragma unroll
            for (int j = 0; j < R / 16; ++j)
                if ((j & 1) == warp >> 2 && j * 16 < t.rank) {
                    float v[16];
                    umma::tmem_ld16(sm.tmem + ((warp & 3) * 32 << 16) + d * R + j * 16, v);
                    umma::tmem_wait_ld();
                    if (row < t.n)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (j * 16 + e < t.rank) h[(j * 16 + e) * t.n + row] = v[e];
                }
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(&sm.d_empty[d]);
            ++tiles;
        }
    } else if (warp == kCopier) {
        Ring<R> at;
        uint32_t issued = 0;
        while (!__any_sync(0xffffffffu, expired(sm)) && walk.next(p, t)) copy_piece<R>(p, t, maps, sm, base, at, issued);
        // no copy may be under way when the CTA leaves
        if (expired(sm))
            for (uint32_t i = issued > kStages<R> ? issued - kStages<R> : 0; i < issued; ++i) drain(&sm.full[i % kStages<R>], (i / kStages<R>) & 1);
    } else {
        Ring<R> at;
        uint32_t tiles = 0;
        while (walk.next(p, t)) {
            const uint32_t d = tiles & 1;
            if (tiles >= 2) wait(sm, &sm.d_empty[d], ((tiles >> 1) - 1) & 1);
            for (int c = t.c_lo; c < t.c_hi; ++c, at.next()) {
                wait(sm, &sm.full[at.stage], at.phase);
                umma::fence_after_sync();
                __syncwarp();
                if (__any_sync(0xffffffffu, expired(sm))) break;
                if (umma::elect_one()) {
                    const uint32_t stage = base + at.stage * kStageBytes<R>;
                    const uint64_t da = umma::desc_sw128(stage, 16, 1024), db = umma::desc_sw128(stage + kTokenBytes, 16, 1024);
#pragma unroll
                    for (int k = 0; k < kK / 16; ++k) umma::mma_bf16(sm.tmem + d * R, da + 2 * k, db + 2 * k, idesc<BF16, 128, R>(false), c > t.c_lo || k > 0);
                    umma::commit(&sm.empty[at.stage]);
                    if (c + 1 == t.c_hi) umma::commit(&sm.d_full[d]);
                }
                __syncwarp();
            }
            ++tiles;
        }
        // no product may be under way when the CTA leaves
        if (umma::elect_one()) umma::commit(&sm.last);
        __syncwarp();
        drain(&sm.last, 0);
    }
    shared_end(sm, kColumns, p.status + blockIdx.x);
}

// ---- up -------------------------------------------------------------------------

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
    if constexpr (N == 2)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1,%2};" ::"r"(at), "r"(v[0]), "r"(v[1]) : "memory");
    else if constexpr (N == 4)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
    else if constexpr (N == 8)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                     "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    else
        umma::tmem_st16(at, v);
}

// a load that stays in front of the next one, so that a batch of them is under way at once
// (else the compiler waits for each: 79 us for 70, a 3001-token prompt of rank 72 beside drafts); 0 where it is not wanted
__device__ __forceinline__ float load_now(const float* from, bool wanted)
{
    float v = 0.0f;
    asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %2, 0;\n@p ld.global.cg.f32 %0, [%1];\n}" : "+f"(v) : "l"(from), "r"((uint32_t)wanted) : "memory");
    return v;
}

// h of a tile as the products' first operand: hi in TMEM columns [0, R / 2), lo behind it, two values a column.
// The workers: two threads a row for each team, each a part of its columns.
template <bool BF16, int R>
__device__ __forceinline__ void operand(const AdapterParams& p, const Piece& t, int2 b, Shared& sm)
{
    constexpr int kParts = kAdapterParts, kMine = R / kParts, kAtOnce = kMine < 32 ? kMine : 32, kBlock = kMine < 8 ? kMine : 8;
    constexpr int kAhead = kMine >= 32 ? 1 : kMine >= 16 ? 2 : 4;  // ranges
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp >> 2, row = (warp & 3) * 32 + lane;
    const int col = part * kMine;
    float v[kMine];
#pragma unroll
    for (int j = 0; j < kMine; ++j) v[j] = 0.0f;
    const Steps steps(t.rank);
    for (int r = b.x; r <= b.y; r += kAhead) {
        float f[kAhead][kMine];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const float* src = p.h + h_place(p.T, p.rank, r + i, t.start, r + i == b.x) + row;
#pragma unroll
            for (int j = 0; j < kMine; j += kBlock) {
                const OperandRows rows(steps, t.rank, col + j);
                const int left = row < t.n && r + i <= b.y ? rows.left : 0;
#pragma unroll
                for (int e = 0; e < kBlock; ++e) f[i][j + e] = load_now(src + (rows.at + e) * t.n, e < left);
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int j = 0; j < kMine; ++j) v[j] += f[i][j];
    }
    float inv = 1.0f, factor = __ldg(p.scales + t.id);
    if (!BF16) {
        // A row's largest value to [2^14, 2^15): fp16 has 5 bits of exponent.  A value keeps 22 bits, or is off by half the
        // type's least step, 2^-25, which is 2^-39 of that largest (with the largest in [1, 2) values 2^14 below it came
        // out with the bits of the output, those 2^23 below with two).
        float most = 0.0f;
#pragma unroll
        for (int j = 0; j < kMine; ++j) most = fmaxf(most, fabsf(v[j]));
        sm.most[part][row] = most;
        workers_sync();
#pragma unroll
        for (int i = 0; i < kParts; ++i) most = fmaxf(most, sm.most[i][row]);
        const int exponent = max((int)(__float_as_uint(most) >> 23) - 127 - 14, -126);  // up to 114
        inv = __uint_as_float((uint32_t)(127 - exponent) << 23);
        factor *= __uint_as_float((uint32_t)(127 + exponent) << 23);
    }
    if (part == 0) sm.factor[row] = factor;
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
    workers_sync();  // the factors
    if (lane == 0) umma::mbar_arrive(&sm.h_full);
}

// A warp's part of a chunk from its stage to y_out, 64 bytes of 8 rows at a time
__device__ __forceinline__ void store_rows(const AdapterParams& p, const Piece& t, int c, const unsigned char* tile, uint16_t* out, int row, int piece)
{
    if (c * kK + piece * 8 >= p.d_out) return;
    const unsigned char* mine = tile + place(row, piece);  // rows 8 apart are swizzled alike
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (row + i * 8 < t.n) __stcs(reinterpret_cast<uint4*>(out + (size_t)(i * 8) * p.out_stride), *reinterpret_cast<const uint4*>(mine + i * 8 * kRow));
}

template <bool BF16, int R>
__global__ void __launch_bounds__(kUpThreads, 1) adapter_up_kernel(const __grid_constant__ AdapterParams p, const __grid_constant__ Maps maps)
{
    extern __shared__ unsigned char smem[];
    __shared__ Shared sm;
    constexpr int kColumns = 512;
    unsigned char* ring = smem + ((1024 - (umma::smem_u32(smem) & 1023)) & 1023);
    const uint32_t base = umma::smem_u32(ring);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // nobody waits for TMEM that this kernel holds in front of its wait: adapter_down has ended when few_down lets it start
    shared_begin(sm, kColumns, kWorkers + 1, kUpWorkers);  // a stage is free: its team is done with it, the product warp is past it
    pdl_wait();
    pdl_launch_dependents();
    const AdapterStart start = p.starts[blockIdx.x];
    const int64_t share = p.starts[0].share;
    Walk<false> walk{start.s, start.k, start.before, share * blockIdx.x, share * (blockIdx.x + 1)};
    if (walk.s >= p.n_seq) walk.hi = walk.at;
    Piece t;
    if (warp < kUpWorkers) {
        unsigned char* result = ring + kStages<R> * kStageBytes<R> + warp * kResultBytes;
        const int team = warp / kWorkers, half = warp >> 2 & 1, row0 = (warp & 3) * 32, row = row0 + lane, spot = row0 + (lane >> 2), piece = half * 4 + (lane & 3);
        Ring<R> at;
        uint32_t m = 0;  // chunks of products
        while (walk.next(p, t)) {
            uint16_t* out = p.y_out + (size_t)(t.start + spot) * p.out_stride + t.c_lo * kK + piece * 8;
            if (t.rank == 0) {  // y as it is
                for (int c = t.c_lo; c < t.c_hi; ++c, ++m, out += kK, at.next()) {
                    if (m % kTeams != team) continue;
                    const uint32_t d = m % kRing;
                    wait(sm, &sm.d_full[d], (m / kRing) & 1);
                    wait(sm, &sm.full[at.stage], at.phase);
                    store_rows(p, t, c, ring + at.stage * kStageBytes<R>, out, spot, piece);
                    __syncwarp();
                    if (lane == 0) {
                        umma::mbar_arrive(&sm.d_empty[d]);
                        umma::mbar_arrive(&sm.empty[at.stage]);
                    }
                }
                continue;
            }
            const int2 b = p.parts[t.slot];
            workers_sync();  // the last tile's factors are read, and its products done
            operand<BF16, R>(p, t, b, sm);
            const float factor = sm.factor[row];
            for (int c = t.c_lo; c < t.c_hi; ++c, ++m, out += kK, at.next()) {
                if (m % kTeams != team) continue;
                const uint32_t d = m % kRing;  // a slot is always the same team's
                wait(sm, &sm.d_full[d], (m / kRing) & 1);
                if (row0 < t.n) {
                    wait(sm, &sm.full[at.stage], at.phase);  // long since; y was copied by other threads
                    umma::fence_after_sync();
                    float v[32];
                    umma::tmem_ld32(sm.tmem + (row0 << 16) + kColumnD + d * kK + half * 32, v);
                    umma::tmem_wait_ld();
                    const unsigned char* tile = ring + at.stage * kStageBytes<R>;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float f[8];
                        widen8<BF16>(*reinterpret_cast<const uint4*>(tile + place(row, half * 4 + i)), f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] = fmaf(factor, v[i * 8 + e], f[e]);
                        *reinterpret_cast<uint4*>(result + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4)) =
                            make_uint4(narrow2<BF16>(f[0], f[1]), narrow2<BF16>(f[2], f[3]), narrow2<BF16>(f[4], f[5]), narrow2<BF16>(f[6], f[7]));
                    }
                    umma::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        umma::mbar_arrive(&sm.d_empty[d]);
                        umma::mbar_arrive(&sm.empty[at.stage]);
                    }
                    // 64 bytes of 8 rows at a time
                    if (c * kK + piece * 8 < p.d_out) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = i * 8 + (lane >> 2);
                            if (row0 + r < t.n)
                                __stcs(reinterpret_cast<uint4*>(out + (size_t)(i * 8) * p.out_stride),
                                       *reinterpret_cast<const uint4*>(result + r * 64 + (((lane & 3) ^ (r >> 1 & 3)) << 4)));
                        }
                    }
                    __syncwarp();  // the results are read
                } else if (lane == 0) {
                    umma::mbar_arrive(&sm.d_empty[d]);
                    umma::mbar_arrive(&sm.empty[at.stage]);
                }
            }
        }
    } else if (warp == kUpWorkers) {
        Ring<R> at;
        uint32_t issued = 0;
        while (!__any_sync(0xffffffffu, expired(sm)) && walk.next(p, t)) copy_piece<R>(p, t, maps, sm, base, at, issued);
        // no copy may be under way when the CTA leaves
        if (expired(sm))
            for (uint32_t i = issued > kStages<R> ? issued - kStages<R> : 0; i < issued; ++i) drain(&sm.full[i % kStages<R>], (i / kStages<R>) & 1);
    } else {
        Ring<R> at;
        uint32_t m = 0, tiles = 0;
        while (walk.next(p, t)) {
            if (t.rank == 0) {  // no products, the same hand-offs
                for (int c = t.c_lo; c < t.c_hi; ++c, ++m, at.next()) {
                    const uint32_t slot = m % kRing;
                    wait(sm, &sm.full[at.stage], at.phase);
                    if (m >= kRing) wait(sm, &sm.d_empty[slot], (m / kRing - 1) & 1);
                    if (lane == 0) {
                        umma::mbar_arrive(&sm.d_full[slot]);
                        umma::mbar_arrive(&sm.empty[at.stage]);
                    }
                }
                continue;
            }
            const Steps steps(t.rank);
            const int zeros = t.rank <= 8 ? 16 - t.rank : -t.rank & 7;  // rows behind the rank that a step takes in all the same
            wait(sm, &sm.h_full, tiles & 1);
            ++tiles;
            for (int c = t.c_lo; c < t.c_hi; ++c, ++m, at.next()) {
                const uint32_t slot = m % kRing;
                wait(sm, &sm.full[at.stage], at.phase);
                if (m >= kRing) wait(sm, &sm.d_empty[slot], (m / kRing - 1) & 1);
                // (rows 8 to 15 of an adapter of 8 are copied by nobody: once a stage is enough)
                if (zeros > 0 && ((t.rank & 7) || c - t.c_lo < kStages<R>)) {
                    uint4* rows = reinterpret_cast<uint4*>(ring + at.stage * kStageBytes<R> + kTokenBytes + t.rank * kRow);
                    for (int i = lane; i < zeros * (kRow / 16); i += 32) rows[i] = make_uint4(0, 0, 0, 0);
                    umma::fence_proxy_async();
                }
                umma::fence_after_sync();
                __syncwarp();
                if (__any_sync(0xffffffffu, expired(sm))) break;
                if (umma::elect_one()) {
                    const uint32_t d = sm.tmem + kColumnD + slot * kK;
                    const uint64_t db = umma::desc_sw128(base + at.stage * kStageBytes<R> + kTokenBytes, 16, 1024);
                    for (int k = 0; k < steps.count; ++k) {
                        const uint64_t rows = db + steps.first_row(k) * (kRow >> 4);
                        umma::mma_ts(d, sm.tmem + 8 * k, rows, idesc<BF16, 128, kK>(true), k > 0);
                        umma::mma_ts(d, sm.tmem + R / 2 + 8 * k, rows, idesc<BF16, 128, kK>(true), 1);
                    }
                    umma::commit(&sm.d_full[slot]);
                    umma::mbar_arrive(&sm.empty[at.stage]);
                }
                __syncwarp();
            }
        }
        // no product may be under way when the CTA leaves
        if (umma::elect_one()) umma::commit(&sm.last);
        __syncwarp();
        drain(&sm.last, 0);
    }
    shared_end(sm, kColumns, p.status + kCtas + blockIdx.x);
}

// rows of `width` 16-bit values, `stride` apart, in boxes of 64 of them by `box_rows` rows, swizzled over 128 bytes
bool encode_map(CUtensorMap& map, const void* rows, bool bf16, int width, int64_t n_rows, int64_t stride, int box_rows)
{
    const auto encode = tensor_map_encoder();
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)n_rows}, strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {kK, (cuuint32_t)box_rows}, ones[2] = {1, 1};
    return encode && encode(&map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(rows), dims, strides, box,
                            ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_maps(Maps& maps, const AdapterParams& p, const uint16_t* tokens, int64_t stride, const uint16_t* weights, int width)
{
    const int64_t rows = (int64_t)p.n_adapters * p.rank;
    // (without adapters nothing is read through the weights')
    return encode_map(maps.tokens, tokens, p.bf16, width, p.T, stride, kTile) &&
           (rows == 0 || (encode_map(maps.weights, weights, p.bf16, width, rows, width, p.rank) && encode_map(maps.weights8, weights, p.bf16, width, rows, width, 8)));
}

// ---- few tokens -------------------------------------------------------------------
//
// A block takes 4 tokens of a sequence and some channels, on the CUDA cores, each thread's loads all under way at once.
// Alone (ALONE, a small batch) they take every token, and split x's channels among blocks.  Beside the tensor
// cores' kernels they take the tiles that those leave: the order is adapter_down, few_down, adapter_up, few_up, each
// behind the end of the one before it.  (A few_down beside adapter_down, which did not wait for it, and a few_up that read
// y, `up` and h in front of its wait took 69 us for 82, a 3001-token prompt beside 39 drafts; but only a grid that waits is
// promised to see what was written before.  few_down by adapter_down's workers, idle until their first product: 81, and 78
// for 53 for 128 sequences of 12 tokens, rank 16.)
constexpr int kFewThreads = 128, kFewTile = 4;
constexpr int kFewRows = kFewThreads / 16;   // of `down`, two a warp
constexpr int kFewIn = 1024;                 // x's channels at a time
constexpr int kFewOut = kFewThreads * 8;
// Tokens up to which a tile goes this way: the weights are read for every 4 tokens, and the others' kernels copy whole
// tiles.  128 sequences of 12 tokens, 4096 to 10240: rank 16 53 us, 102 by the others; of 24 96 and 106; rank 64, of 12 134
// and 114 (replayed).
int few_tokens(int rank) { return rank <= 16 ? 24 : rank <= 32 ? 16 : 8; }

// up to kFewTile tokens of one sequence; n 0: an empty slot
template <bool ALONE>
__device__ __forceinline__ Piece few_tile(const AdapterParams& p, int slot)
{
    Piece t{};
    const int slots = p.few / kFewTile;
    const auto cu = [&](int i) { return cu_at(p.cu_seqlens, i, p.T); };
    int s = slot / slots, end;
    int64_t start;
    if (ALONE) {  // sequence s owns the slots from cu[s] / kFewTile + s on
        const auto base = [&](int i) { return (int64_t)(cu(i) / kFewTile + i); };
        s = warp_find(p.n_seq, slot, base);
        end = cu(s + 1);
        start = cu(s) + max((int64_t)0, slot - base(s)) * kFewTile;
    } else {      // p.few tokens' slots a sequence, for its last ones
        const int first = cu(s);
        end = cu(s + 1);
        const int rest = max(end - first, 0) % kTile;
        start = rest > p.few ? end : end - rest + slot % slots * kFewTile;
    }
    t.n = (int)max((int64_t)0, min((int64_t)kFewTile, end - start));
    t.start = t.n > 0 ? (int)start : 0;
    t.rank = rank_of(p, s, t.id);
    return t;
}

// two rows of `down` with up to NT tokens, channels [k_lo, k_hi)
template <bool BF16, int NT>
__device__ __forceinline__ void few_down(const AdapterParams& p, const Piece& t, int j, int k_lo, int k_hi, float* h)
{
    constexpr int kSteps = kFewIn / 256;
    const int lane = threadIdx.x & 31;
    const uint16_t* x = p.x + (size_t)t.start * p.x_stride;
    const uint16_t* w0 = p.down + ((size_t)t.id * p.rank + j) * p.d_in;
    const uint16_t* w1 = j + 1 < t.rank ? w0 + p.d_in : w0;
    float acc[2][NT] = {};
    for (int k0 = k_lo + lane * 8; k0 < k_hi; k0 += kFewIn) {
        uint4 a[kSteps][2];
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
            if (k0 + i * 256 < k_hi) {
                a[i][0] = __ldg(reinterpret_cast<const uint4*>(w0 + k0 + i * 256));
                a[i][1] = __ldg(reinterpret_cast<const uint4*>(w1 + k0 + i * 256));
            }
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
            if (k0 + i * 256 < k_hi) {
                float f[2][8];
                widen8<BF16>(a[i][0], f[0]);
                widen8<BF16>(a[i][1], f[1]);
#pragma unroll
                for (int q = 0; q < NT; ++q) {
                    float v[8];
                    widen8<BF16>(__ldg(reinterpret_cast<const uint4*>(x + (size_t)min(q, t.n - 1) * p.x_stride + k0 + i * 256)), v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        acc[0][q] = fmaf(f[0][e], v[e], acc[0][q]);
                        acc[1][q] = fmaf(f[1][e], v[e], acc[1][q]);
                    }
                }
            }
    }
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float sum = warp_sum(acc[r][q]);
            if (lane == 0 && q < t.n && j + r < t.rank) h[(size_t)q * p.rank + j + r] = sum;
        }
}

// grid: slots, groups of kFewRows rows, (alone) ranges of kFewIn channels
template <bool BF16, bool ALONE>
__global__ void __launch_bounds__(kFewThreads) few_down_kernel(const __grid_constant__ AdapterParams p)
{
    pdl_wait();
    pdl_launch_dependents();
    if (ALONE && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
        for (int i = threadIdx.x; i < 2 * kCtas; i += kFewThreads) p.status[i] = 0;  // nobody waits here
    const Piece t = few_tile<ALONE>(p, blockIdx.x);
    const int j = blockIdx.y * kFewRows + (threadIdx.x >> 5) * 2;
    if (t.n > 0 && j < t.rank) {
        const int k_lo = ALONE ? blockIdx.z * kFewIn : 0, k_hi = ALONE ? min(p.d_in, k_lo + kFewIn) : p.d_in;
        float* h = p.h + ((size_t)blockIdx.z * p.T + t.start) * p.rank;
        if (t.n == 1) few_down<BF16, 1>(p, t, j, k_lo, k_hi, h);
        else if (t.n == 2) few_down<BF16, 2>(p, t, j, k_lo, k_hi, h);
        else few_down<BF16, 4>(p, t, j, k_lo, k_hi, h);
    }
}

template <bool BF16, bool ALONE, int NT>
__device__ __forceinline__ void few_up(const AdapterParams& p, const Piece& t, int o, float* h)
{
    constexpr int kAhead = NT > 2 ? 8 : 16;  // rows of `up` loaded ahead
    const bool mine = o < p.d_out;
    const uint16_t* w = p.up + (size_t)t.id * p.rank * p.d_out + (mine ? o : 0);
    uint4 y[NT], v[kAhead];
    const auto load = [&](int j) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) v[i] = mine && j + i < t.rank ? __ldcg(reinterpret_cast<const uint4*>(w + (size_t)(j + i) * p.d_out)) : make_uint4(0, 0, 0, 0);
    };
#pragma unroll
    for (int q = 0; q < NT; ++q)
        y[q] = mine ? __ldcg(reinterpret_cast<const uint4*>(p.y + (size_t)(t.start + min(q, t.n - 1)) * p.y_stride + o)) : make_uint4(0, 0, 0, 0);
    load(0);
    const int splits = ALONE ? (p.d_in + kFewIn - 1) / kFewIn : 1;
    for (int i = threadIdx.x; i < kFewTile * 128; i += kFewThreads) {
        float sum = 0.0f;
        const int q = i >> 7, j = i & 127;
        if (q < t.n && j < t.rank)
            for (int s = 0; s < splits; ++s) sum += __ldcg(p.h + ((size_t)s * p.T + t.start + q) * p.rank + j);
        h[i] = sum;
    }
    __syncthreads();
    float acc[NT][8] = {};
    for (int j = 0; j < t.rank; j += kAhead) {
        if (j > 0) load(j);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            float f[8];
            widen8<BF16>(v[i], f);
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                const float x = h[q * 128 + min(j + i, 127)];  // (zero behind the rank, as v is)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[q][e] = fmaf(x, f[e], acc[q][e]);
            }
        }
    }
    const float scale = __ldcg(p.scales + t.id);
#pragma unroll
    for (int q = 0; q < NT; ++q)
        if (mine && q < t.n) {
            float f[8];
            widen8<BF16>(y[q], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = fmaf(scale, acc[q][e], f[e]);
            __stcs(reinterpret_cast<uint4*>(p.y_out + (size_t)(t.start + q) * p.out_stride + o),
                   make_uint4(narrow2<BF16>(f[0], f[1]), narrow2<BF16>(f[2], f[3]), narrow2<BF16>(f[4], f[5]), narrow2<BF16>(f[6], f[7])));
        }
}

// grid: slots, ranges of kFewOut channels
template <bool BF16, bool ALONE>
__global__ void __launch_bounds__(kFewThreads) few_up_kernel(const __grid_constant__ AdapterParams p)
{
    __shared__ float h[kFewTile * 128];
    pdl_wait();
    pdl_launch_dependents();
    const Piece t = few_tile<ALONE>(p, blockIdx.x);
    const int o = blockIdx.y * kFewOut + threadIdx.x * 8;
    if (t.n > 0 && t.rank > 0) {
        if (t.n == 1) few_up<BF16, ALONE, 1>(p, t, o, h);
        else if (t.n == 2) few_up<BF16, ALONE, 2>(p, t, o, h);
        else few_up<BF16, ALONE, 4>(p, t, o, h);
    } else if (p.y_out != p.y && o < p.d_out) {
        for (int q = 0; q < t.n; ++q)
            *reinterpret_cast<uint4*>(p.y_out + (size_t)(t.start + q) * p.out_stride + o) =
                __ldcg(reinterpret_cast<const uint4*>(p.y + (size_t)(t.start + q) * p.y_stride + o));
    }
}

template <bool BF16, bool ALONE>
cudaError_t launch_few_down(const AdapterParams& p, unsigned slots, cudaStream_t stream)
{
    const dim3 grid(slots, (unsigned)((p.rank + kFewRows - 1) / kFewRows), ALONE ? (unsigned)((p.d_in + kFewIn - 1) / kFewIn) : 1);
    return launch_k(few_down_kernel<BF16, ALONE>, grid, dim3(kFewThreads), 0, stream, true, p);
}

template <bool BF16, bool ALONE>
cudaError_t launch_few_up(const AdapterParams& p, unsigned slots, cudaStream_t stream)
{
    return launch_k(few_up_kernel<BF16, ALONE>, dim3(slots, (unsigned)((p.d_out + kFewOut - 1) / kFewOut)), dim3(kFewThreads), 0, stream, true, p);
}

// Whether a batch goes this way alone, long sequences too, by the products that it takes: the other kernels cost some 10 us
// whatever they do, and 2^27 products are about as much.  Replayed, alone and beside, us: 8 single tokens (rank 16, 5120 to
// 5120) 5.5 and 13.5; 64 with rank 64 17.5 and 20.8; a prompt of 400 tokens, rank 16, 13.0 and 31.5, of 800 21.7 and 21.3; 128
// single tokens, rank 64, 28.4 and 29.4; 64 and a chunk of 400, rank 128, 84 and 53; 255 and one of 1500, 288 and 114.
#ifdef GDN_ADAPTER_SELFTEST_NEVER_ALONE
constexpr int64_t kAloneWork = -1;  // tests: small batches through all kernels
#else
constexpr int64_t kAloneWork = 1 << 27;
#endif
bool goes_alone(const AdapterParams& p)
{
    const int64_t splits = (p.d_in + kFewIn - 1) / kFewIn;
    return (int64_t)p.T * p.rank * (p.d_in + p.d_out) <= kAloneWork && p.T * (splits - 1) <= kCtas * kTile;
}

template <bool BF16>
cudaError_t launch_alone(const AdapterParams& p, cudaStream_t stream)
{
    const unsigned slots = (unsigned)((int64_t)p.T / kFewTile + p.n_seq);
    const cudaError_t e = launch_few_down<BF16, true>(p, slots, stream);
    return e != cudaSuccess ? e : launch_few_up<BF16, true>(p, slots, stream);
}

template <bool BF16, int R>
cudaError_t launch_rank(const AdapterParams& p, cudaStream_t stream)
{
    Maps in{}, out{};
    if (!encode_maps(in, p, p.x, p.x_stride, p.down, p.d_in) || !encode_maps(out, p, p.y, p.y_stride, p.up, p.d_out)) return cudaErrorNotSupported;
    const unsigned slots = (unsigned)p.n_seq * (unsigned)(p.few / kFewTile);
    // adapter_up may start while few_down ends, but not in a batch of prompts.  Replayed, so and so, us: 8 prompts of 1 to 4096
    // tokens, rank 64, 4096 to 6144, 142 and 139; 3001 beside 40 drafts of 3, 2048 to 10240, 65.6 and 67.1; 255 single tokens
    // beside 1500 76.8 and 77.8.
    const bool early = p.T < (int64_t)kTile * p.n_seq;
    cudaError_t e = cudaFuncSetAttribute(adapter_down_kernel<BF16, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem<R>);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(adapter_up_kernel<BF16, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem<R>);
    if (e == cudaSuccess) e = launch_k(adapter_down_kernel<BF16, R>, dim3(kCtas), dim3(kThreads), kSmem<R>, stream, true, p, in);
    if (e == cudaSuccess) e = launch_few_down<BF16, false>(p, slots, stream);
    if (e == cudaSuccess) e = launch_k(adapter_up_kernel<BF16, R>, dim3(kCtas), dim3(kUpThreads), kSmem<R>, stream, early, p, out);
    if (e == cudaSuccess) e = launch_few_up<BF16, false>(p, slots, stream);
    return e;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

// status words, where the ranges of adapter_up begin, which ranges a tile's h is in, h
size_t adapter_workspace(AdapterParams& p, void* workspace)
{
    char* at = static_cast<char*>(workspace);
    size_t used = 0;
    const auto take = [&](size_t bytes) {
        char* mine = at + used;
        used += align256(bytes);
        return mine;
    };
    p.status = reinterpret_cast<int32_t*>(take(2 * kCtas * 4));
    p.starts = reinterpret_cast<AdapterStart*>(take(kCtas * sizeof(AdapterStart)));
    p.parts = reinterpret_cast<int2*>(take(((size_t)p.T / kTile + p.n_seq) * sizeof(int2)));
    p.h = reinterpret_cast<float*>(take(((size_t)p.T + kCtas * kTile) * p.rank * 4));
    return used;
}

cudaError_t launch_adapter(AdapterParams p, void* workspace, cudaStream_t stream)
{
    adapter_workspace(p, workspace);
    p.few = few_tokens(p.rank);
    p.chunks_in = (p.d_in + kK - 1) / kK;
    p.chunks_out = (p.d_out + kK - 1) / kK;
    // Each part of a tile's h takes adapter_up over a microsecond to add, each unit of a range adapter_down half of one:
    // about sqrt(units) / 2 parts are best where there are more CTAs than tiles (one prompt of 3001 tokens, rank 128, 2048
    // to 10240: 56.1 us, 66.0 with up to 16).
    for (p.parts_in = 2; 4 * p.parts_in * p.parts_in < p.chunks_in; ++p.parts_in) {}
    const auto launch = [&](auto bf16) {
        constexpr bool kBf16 = decltype(bf16)::value;
        if (goes_alone(p)) return launch_alone<kBf16>(p, stream);
        if (p.rank <= 16) return launch_rank<kBf16, 16>(p, stream);
        if (p.rank <= 32) return launch_rank<kBf16, 32>(p, stream);
        if (p.rank <= 64) return launch_rank<kBf16, 64>(p, stream);
        return launch_rank<kBf16, 128>(p, stream);
    };
    return p.bf16 ? launch(std::true_type{}) : launch(std::false_type{});
}

}  // namespace gdn
