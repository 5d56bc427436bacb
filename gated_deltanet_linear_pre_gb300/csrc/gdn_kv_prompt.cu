// gdn_kv_prompt.cu -- attention of many query rows over the 8-bit paged cache, on
// the tcgen05 tensor cores.
//
// Mathematics.  One pass over the keys per 128 query rows with the softmax's running maximum and sum:
// S = Q K^T and O += P V are 128 x 128 (x head_dim) products with fp32 accumulators in TMEM.
// P = 2^(x - m + 7), x = scale log2(e) q.k; the reference m moves, and O and l are rescaled, only where a
// tile's maximum passes it by 8 (a factor of 256): P stays below 2^15, and what is lost to fp16's smallest
// step is 2^-31 of the largest weight.  Weights are rounded to fp16 (11 bits), sums and statistics are fp32.
//
// Layout.  The tensor cores read 16-bit operands from shared memory, so the codes have to be unpacked
// somewhere.  Done by every CTA for itself, a 128-position tile would cost each about as many issue slots
// as a third of its softmax; instead one kernel unpacks each long sequence's cache once into images, in
// the 128-byte swizzled order (without swizzle the products ran 7% slower), that a single bulk copy brings
// in: 4 bytes moved per code byte, 10 us of the 73 that 2048 tokens from nothing take and 18 of the 790 of a
// 4001-token chunk behind 16500.  K takes the activations' type (both operands of a product have one), so
// queries go to shared memory as they are.  A bf16 image holds code * scale, exactly.  An fp16 image (V always) holds code *
// (page scale / largest scale of the sequence and head) * kUp, exact for pages whose scale is at least exact_ratio
// of the largest, which goes into the scores' unit and the outputs'.  A sequence with smaller ones takes the step
// kernel (1.0 ms for those 2048 tokens, 12 ms for the chunk): rows that see only those must not lose bits to pages
// that they do not see.  A page whose v scale is NaN has an image of zeros, since a weight of 0 times NaN would
// reach the rows that do not see it: the output code makes the rows that do see it NaN.  (A NaN k scale makes a
// column of scores NaN, which the mask replaces.)
//
// A CTA (608 threads, one per SM) holds two 128-row halves, so that one half's softmax runs under the
// other's products: warps 0-7 and 8-15 the rows (two threads a row, each half of a tile's columns: a tile's
// softmax takes less than the other half's 1024 tensor cycles only with four warps a scheduler), warp 16
// the copies, warp 17 the products, warp 18 the units ahead and their queries, which it brings in as soon as
// the last scores of the unit before are issued, under its softmax and its output (a tensor map's box of
// floor(128 / group) tokens by group heads by 64 channels is 128 swizzled rows as the products read them).
// TMEM: S and O of each half,
// 512 columns at head_dim 128; the fp16 P of 64 keys takes the first 32 of their 64 score columns.
// Rows are (token, query head of the kv head): floor(128 / group) tokens a half.
//
// Bound and measured.  By the tensor cores and what feeds them together: a tile of both halves is 2048 cycles of
// products, reads shared memory at its full 128 bytes a cycle for as long, and has 1024 cycles of exponentials a
// half.  A 4001-token chunk behind 16500 tokens (32 query heads over 4 of 128, beside three single tokens) takes
// 745 us, 1.6 PFLOP/s, 83% of the measured dense rate; 2048 tokens from nothing (48 over 16) 61 us, of which a
// CTA's start takes 6 and each of its units 3 between the last tile of one and the first of the next.  Tried and
// left out: 8 softmax warps of 208 registers (1090 us for the chunk's call, 790), a warp of products for each
// half (830), waits that spin (829 and more).
#include "gdn_kv_attn.cuh"
#include "gdn_tensor_map.cuh"
#include "umma.cuh"

namespace gdn {
namespace {

constexpr int kImageThreads = 256;
constexpr int kThreads = 608;
constexpr int kLoadWarp = 16, kMmaWarp = 17, kQueryWarp = 18;
constexpr float kWeightShift = 7.0f;
constexpr float kLazy = 8.0f;
constexpr float kLargeScore = 1048576.0f;   // 2^20: fp32 steps of 2^-3
constexpr float kHugeScore = 67108864.0f;   // 2^26: steps of 4 to 8

// images hold codes times kUp: up to 127 x 2^8 and 448 x 2^6
template <bool E4M3> constexpr float kUp = E4M3 ? 64.0f : 256.0f;

// the smallest quotient of two scales that leaves a code times kUp a whole number of fp16's least steps, 2^-24:
// int8 codes are multiples of 1, e4m3 ones of 2^-9
template <bool E4M3> constexpr float exact_ratio = 1.0f / (E4M3 ? 2097152.0f : 4294967296.0f);

template <int D> constexpr uint32_t kTileBytes = kKeys * D * 2;

// byte offset of (position, channels 8 c8 .. + 7) in an image: planes of 64 channels, a position's 128 bytes
// of a plane a row, its 16-byte pieces swizzled
constexpr uint32_t kPlane = kKeys * 128;
__device__ __forceinline__ int image_off(int pos, int c8) { return (c8 >> 3) * (int)kPlane + pos * 128 + (((c8 & 7) ^ (pos & 7)) << 4); }

// ---- unpacking ------------------------------------------------------------------------
__device__ __forceinline__ int key_tiles(int kv) { return (kv + kKeys - 1) / kKeys; }

// eight codes times f in fp16
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

// ---- the units of long sequences -----------------------------------------------------
// Sum over k < i of ceil((first + (k + 1) span) / 128): the sum of the numerators, rounded up, less the sum
// of their residues, which repeat with a period of at most 128.
__device__ __forceinline__ int64_t tiles_before(int first, int span, int i)
{
    const int64_t c = (int64_t)first + span + kKeys - 1;
    const int period = kKeys >> min(__ffs(span) - 1, 7);   // 128 / gcd(span, 128)
    const int g = kKeys / period, full = i / period;
    int64_t residues = (int64_t)full * (period * (int)(c & (g - 1)) + g * (period * (period - 1) / 2));
    int x = (int)((c + (int64_t)full * period * span) & (kKeys - 1));
    for (int k = full * period; k < i; ++k, x = (x + span) & (kKeys - 1)) residues += x;
    return (i * c + (int64_t)span * ((int64_t)i * (i - 1) / 2) - residues) / kKeys;
}
// cost of the units before unit i of a (sequence, head) (none of them the last one)
__device__ __forceinline__ int64_t unit_prefix(int first, int span, int i) { return tiles_before(first, span, i) + (int64_t)i * kPromptUnitCost; }
__device__ __forceinline__ int unit_tiles(int first, int n, int span, int i) { return (first + min((i + 1) * span, n) + kKeys - 1) / kKeys; }
__device__ __forceinline__ int64_t head_cost(const SeqView& v, int span)
{
    const int last = (v.n + span - 1) / span - 1;
    return unit_prefix(v.first, span, last) + unit_tiles(v.first, v.n, span, last) + kPromptUnitCost;
}

// Whether the units are not cut but handed out one by one, sequence after sequence, each with its longest
// units first.  A unit then begins, at the latest, when all before it have taken every worker's time, so the
// last one ends by the largest of (cost of the units before it) / workers + its own.  Within a sequence that
// is a concave function of the unit, with its largest value where a unit's cost is what the following
// unit's is less, times workers / heads.  Against it stands an equal share of a cut batch, with one more unit
// begun and ended, its parts and their join.  Cut and whole took (48 query heads over 16, e4m3, from empty)
// 44 and 35 us for 1024 tokens, 83 and 72 for 2048, 717 and 675 for 8192 (a share of 358 tiles); 1186 and 1113
// for 8 prompts of 1 to 4096; 788 and 861 for 4001 tokens behind 16500 (16 over 4), whose 500 equal units
// make 4 rounds of 152 CTAs out of 3.3, and which the bound leaves cut.
template <int THREADS>
__device__ __forceinline__ bool whole_units(const AttnParams& p, const AttnSpace& a, int span, int64_t total, int workers, ScanSmem<THREADS>& scan)
{
    if (p.n_seq > THREADS) return false;  // (scan.prefix holds the costs before the sequences of one chunk)
    const int64_t share = (total + workers - 1) / workers, most = share + share / 16 + kPromptCutCost;
    bool late = false;
    if ((int)threadIdx.x < p.n_seq) {
        const SeqView v = seq_view(p, threadIdx.x);
        if (candidate(p, a, v)) {
            const int units = (v.n + span - 1) / span;
            const int64_t at = (int64_t)span * workers / p.heads - kPromptUnitCost * kKeys - v.first;
            const int i = (int)max(min(at / span - 1, (int64_t)units - 1), (int64_t)0);
            const int64_t rest = p.heads * (head_cost(v, span) - unit_prefix(v.first, span, i));  // of unit i and the longer ones
            late = (scan.prefix[threadIdx.x] + rest) / workers + unit_tiles(v.first, v.n, span, i) + kPromptUnitCost > most;
        }
    }
    return !__syncthreads_or(late);
}

// The plan: the total cost of all candidates, and where each worker's range begins in it.  One block.
template <int THREADS>
__device__ __forceinline__ void plan(const AttnParams& p, const AttnSpace& a, int grid, ScanSmem<THREADS>& scan)
{
    const int span = 2 * half_tokens(p.hq / p.heads), tid = threadIdx.x;
    auto weight = [&](int s) {
        const SeqView v = seq_view(p, s);
        return candidate(p, a, v) ? p.heads * head_cost(v, span) : 0;
    };
    const int64_t total = scan_total<THREADS>(p.n_seq, weight, scan);
    int workers = (int)min((int64_t)grid, total);
    const bool whole = total > 0 && whole_units(p, a, span, total, workers, scan);
    if (whole) {  // units in the place of costs
        int64_t mine = 0, jobs;
        if (tid < p.n_seq) {
            const SeqView v = seq_view(p, tid);
            if (candidate(p, a, v)) mine = (int64_t)((v.n + span - 1) / span) * p.heads;
        }
        const int64_t before = block_scan<THREADS>(mine, scan, jobs);
        scan.prefix[tid] = before;
        if (tid == 0) scan.chunk[0] = jobs;
        workers = (int)min((int64_t)grid, jobs);
    }
    if (tid == 0) {
        a.head->prompt_total = total;
        a.head->prompt_workers = workers;
        a.head->prompt_whole = whole;
        a.head->prompt_next = workers;
    }
    int64_t base = 0, tiles = 0;
    __shared__ int image[THREADS];  // image tiles before each of the chunk's sequences
    for (int c = 0; c * THREADS < p.n_seq; ++c) {
        {
            const int s = c * THREADS + tid;
            int64_t mine = 0, sum;
            if (s < p.n_seq) {
                const SeqView v = seq_view(p, s);
                mine = candidate(p, a, v) ? key_tiles(v.kv) : 0;
            }
            const int64_t before = tiles + block_scan<THREADS>(mine, scan, sum);
            image[tid] = (int)min(before, (int64_t)a.image_tiles);
            tiles += sum;
        }
        if (c > 0) {
            const int s = c * THREADS + tid;
            int64_t sum;
            const int64_t before = block_scan<THREADS>(s < p.n_seq ? weight(s) : 0, scan, sum);
            __syncthreads();
            scan.prefix[tid] = before;
        }
        __syncthreads();
        const int64_t end = base + scan.chunk[c];
        for (int w = tid; w < workers; w += THREADS) {  // the workers whose range begins in this chunk
            const int64_t lo = whole ? w : cut_start(total, workers, w);
            if (lo < base || lo >= end) continue;
            int s = 0;
            for (int step = THREADS / 2; step > 0; step >>= 1)
                if (base + scan.prefix[s + step] <= lo) s += step;
            int64_t rest = lo - (base + scan.prefix[s]);
            s += c * THREADS;
            const SeqView v = seq_view(p, s);
            const int units = (v.n + span - 1) / span;
            if (whole) {
                const int i = units - 1 - (int)(rest / p.heads);
                a.prompt_cut[w] = Cut{s, (int)(rest % p.heads), i, 0, unit_tiles(v.first, v.n, span, i), 0, lo - rest, v.t0, v.n, v.first, image[s]};
                continue;
            }
            const int64_t per_head = head_cost(v, span);
            const int head = (int)(rest / per_head);
            rest -= head * per_head;
            // the unit: about half a tile's rounding a unit makes the prefix a quadratic, whose root is near
            const float qa = span / (2.0f * kKeys), qb = (v.first + 0.5f * span) / kKeys + 0.5f + kPromptUnitCost;
            int i = min(max((int)((sqrtf(qb * qb + 4.0f * qa * (float)rest) - qb) / (2.0f * qa)), 0), units - 1);
            int64_t at = unit_prefix(v.first, span, i);
            while (at > rest) at -= unit_tiles(v.first, v.n, span, --i) + kPromptUnitCost;
            while (i + 1 < units) {
                const int64_t next = at + unit_tiles(v.first, v.n, span, i) + kPromptUnitCost;
                if (next > rest) break;
                at = next;
                ++i;
            }
            const int from = (int)(rest - at);
            a.prompt_cut[w] = Cut{s, head, i, max(from - kPromptUnitCost, 0), unit_tiles(v.first, v.n, span, i), from, lo, v.t0, v.n, v.first, image[s - c * THREADS]};
        }
        base = end;
        __syncthreads();
    }
}

// A worker's units in order: those of its range, or, where units are handed out, one by one.
struct Walk {
    int s, head, i, units;  // sequence, kv head, unit; units of a (sequence, head)
    int t0, n, first;       // the sequence's tokens, its first one's position
    int image, ok;          // image tile of its first positions; 0: not a long sequence after all
    int from;               // cost of the unit before the range
    int64_t left;           // cost of the range from here on
    int64_t jobs;           // (handed out) units of the sequences before s

    // to the next unit, having used `cost` of this one; false at the range's end
    __device__ __forceinline__ bool next(const AttnParams& p, const AttnSpace& a, int span, int cost)
    {
        left -= cost;
        from = 0;
        if (left <= 0) return false;
        if (++i < units) return true;
        i = 0;
        if (++head < p.heads) return true;
        head = 0;
        for (;;) {  // (a candidate that has turned out otherwise keeps its place in the ranges)
            if (++s >= p.n_seq) return false;
            const SeqView v = seq_view(p, s);
            if (!candidate(p, a, v)) continue;
            t0 = v.t0;
            n = v.n;
            first = v.first;
            units = (n + span - 1) / span;
            ok = images_there(p, a, s);
            image = ok ? a.image_base[s] : 0;
            return true;
        }
    }
    // to unit `job` of those handed out, at or behind the one in hand; the whole warp calls it
    __device__ __forceinline__ bool take(const AttnParams& p, const AttnSpace& a, int span, int64_t job)
    {
        const int lane = threadIdx.x & 31;
        while (job >= jobs + (int64_t)units * p.heads) {  // 32 sequences at a time
            jobs += (int64_t)units * p.heads;
            const int at = s + 1 + lane;
            int64_t mine = 0;
            if (at < p.n_seq) {
                const SeqView v = seq_view(p, at);
                if (candidate(p, a, v)) mine = (int64_t)((v.n + span - 1) / span) * p.heads;
            }
            int64_t upto = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += o;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, job < jobs + upto);
            if (past == 0) {
                if (s + 33 >= p.n_seq) return false;
                jobs += __shfl_sync(0xffffffffu, upto, 31);
                s += 32;
                units = 0;
                continue;
            }
            const int found = __ffs(past) - 1;
            jobs += __shfl_sync(0xffffffffu, upto - mine, found);
            s += 1 + found;
            const SeqView v = seq_view(p, s);
            t0 = v.t0;
            n = v.n;
            first = v.first;
            units = (n + span - 1) / span;
            ok = images_there(p, a, s);
            image = ok ? a.image_base[s] : 0;
        }
        const int64_t in = job - jobs;
        i = units - 1 - (int)(in / p.heads);
        head = (int)(in % p.heads);
        from = 0;
        return true;
    }
};

// What the CTA's roles need of a unit; written ahead, into a ring.
constexpr int kUnits = 4;
struct Unit {
    int count;         // tiles (0: no more units)
    int tile;          // first of them among the image tiles, and
    int j0;            // in the sequence
    int head;
    int first;         // position of the sequence's first token
    int t0, n;         // its tokens
    int token;         // the unit's first one in the sequence
    int whole, slot;   // all of the unit's tiles; else where its part goes
    float score_unit, v_unit;  // value of a score's unit (base 2) and of an output's
    int nan_from;      // first position of a page whose v are NaN
};

// and in bf16
template <bool E4M3>
__device__ __forceinline__ uint4 unpack8_bf16(uint2 w, float f)
{
    uint32_t r[4] = {codes2<E4M3, false>(w.x), codes2<E4M3, true>(w.x), codes2<E4M3, false>(w.y), codes2<E4M3, true>(w.y)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&r[i]));
        r[i] = narrow2<true>(h.x * f, h.y * f);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// Block 0 makes the prompt kernel's plan; each of the others takes an equal range of the (kv head, tile)
// items of all candidates, tiles fastest: the largest scales are looked for once a (sequence, head).
template <int D, bool BF16, bool E4M3>
__global__ void __launch_bounds__(kImageThreads, 3) kv_image_kernel(AttnParams p, AttnSpace a, int prompt_grid)
{
    __shared__ ScanSmem<kImageThreads> scan;
    __shared__ uint32_t top_k[kImageThreads / 32], top_v[kImageThreads / 32], first_nan[kImageThreads / 32];
    __shared__ uint32_t low_k[kImageThreads / 32], low_v[kImageThreads / 32];
    struct Part {
        int64_t at;  // byte of its first code
        float k, v;
    };
    __shared__ Part parts[kKeys / kSub];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, shift = page_shift(p);
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x == 0) {
        if (tid == 0) a.head->error = 0u;
        plan<kImageThreads>(p, a, prompt_grid, scan);
        return;
    }
    auto weight = [&](int s) {
        const SeqView v = seq_view(p, s);
        return candidate(p, a, v) ? (int64_t)p.heads * key_tiles(v.kv) : 0;
    };
    const int64_t items = scan_total<kImageThreads>(p.n_seq, weight, scan);
    const int64_t lo = cut_start(items, gridDim.x - 1, blockIdx.x - 1), hi = cut_start(items, gridDim.x - 1, blockIdx.x);
    if (lo >= hi) return;
    int64_t before;
    int s = scan_find<kImageThreads>(p.n_seq, lo, weight, scan, before);
    const float sign = p.scale < 0.0f ? -1.0f : 1.0f;  // scores times |scale|: a row's largest is its maximum's
    int64_t at = lo - before;                          // item within the sequence
    for (int64_t x = lo; x < hi && s < p.n_seq; ++s) {
        const SeqView v = seq_view(p, s);
        if (!candidate(p, a, v)) continue;
        const int n = key_tiles(v.kv), pages = (v.kv + p.page - 1) >> shift;
        const int64_t base = before / p.heads;         // image tiles before the sequence's
        before += (int64_t)p.heads * n;
        for (int head = (int)(at / n); head < p.heads && x < hi; ++head) {
            // whether the sequence's images fit and every page is there; its largest and smallest scales (0 and NaN
            // apart, as bits: they are not below 0) and the first page whose v scale is NaN
            uint32_t k_bits = 0u, v_bits = 0u, k_low = 0x7f800000u, v_low = 0x7f800000u, nan_page = 0x7fffffffu;
            bool there = base + n <= a.image_tiles;
            for (int i = tid; i < pages; i += kImageThreads) {
                const int page = page_at(p, s, i);
                if (page < 0) {
                    there = false;
                } else {
                    const float ks = __ldg(p.k_scale + (size_t)page * p.heads + head), vs = __ldg(p.v_scale + (size_t)page * p.heads + head);
                    if (ks > 0.0f) {
                        k_bits = max(k_bits, __float_as_uint(ks));
                        k_low = min(k_low, __float_as_uint(ks));
                    }
                    if (vs > 0.0f) {
                        v_bits = max(v_bits, __float_as_uint(vs));
                        v_low = min(v_low, __float_as_uint(vs));
                    }
                    if (vs != vs) nan_page = min(nan_page, (uint32_t)i);
                }
            }
            k_bits = __reduce_max_sync(0xffffffffu, k_bits);
            v_bits = __reduce_max_sync(0xffffffffu, v_bits);
            k_low = __reduce_min_sync(0xffffffffu, k_low);
            v_low = __reduce_min_sync(0xffffffffu, v_low);
            nan_page = __reduce_min_sync(0xffffffffu, nan_page);
            if (lane == 0) {
                low_k[warp] = k_low;
                low_v[warp] = v_low;
                top_k[warp] = k_bits;
                top_v[warp] = v_bits;
                first_nan[warp] = nan_page;
            }
            there = __syncthreads_and(there);
#pragma unroll
            for (int w = 0; w < kImageThreads / 32; ++w) {
                k_bits = max(k_bits, top_k[w]);
                v_bits = max(v_bits, top_v[w]);
                k_low = min(k_low, low_k[w]);
                v_low = min(v_low, low_v[w]);
                nan_page = min(nan_page, first_nan[w]);
            }
            const float mk = __uint_as_float(k_bits), mv = __uint_as_float(v_bits);
            there = there && (BF16 || __uint_as_float(k_low) >= mk * exact_ratio<E4M3>) && __uint_as_float(v_low) >= mv * exact_ratio<E4M3>;
            const int first = (int)(at - (int64_t)head * n);
            const int behind = ok_stride(p.heads) - p.heads;
            if (first == 0 && head == 0 && tid < behind) a.ok[(size_t)s * ok_stride(p.heads) + p.heads + tid] = 1;
            if (first == 0 && tid == 0) {
                a.ok[(size_t)s * ok_stride(p.heads) + head] = there;
                if (head == 0) a.image_base[s] = there ? (int)base : 0;
                if (there) a.units[(size_t)base * p.heads + head] = HeadUnits{mk, mv, nan_page < (uint32_t)pages ? (int)nan_page << shift : 0x7fffffff, 0};
            }
            const int last = (int)min((int64_t)n, first + (hi - x));
            x += last - first;
            at = (int64_t)(head + 1) * n;
            for (int tile = first; there && tile < last; ++tile) {
                // where the tile's 16-position parts lie and their factors
                if (tid < kKeys / kSub) {
                    const int pos = tile * kKeys + tid * kSub;
                    Part part{-1, 0.0f, 0.0f};
                    if (pos < v.kv) {
                        const int64_t row = (int64_t)page_at(p, s, pos >> shift) * p.heads + head;
                        const float ks = __ldg(p.k_scale + row), vs = __ldg(p.v_scale + row);
                        part.at = (row * p.page + (pos & (p.page - 1))) * D;
                        // (a scale of 0 may meet a largest one of 0; a NaN k scale stays NaN)
                        part.k = (ks == 0.0f ? 0.0f : BF16 ? ks : ks / mk * kUp<E4M3>) * sign;
                        part.v = vs > 0.0f ? vs / mv * kUp<E4M3> : 0.0f;
                    }
                    parts[tid] = part;
                }
                __syncthreads();
                // neighbouring lanes take neighbouring channels: whole rows of codes and of an image's planes; a
                // thread's codes are all on their way before the first is unpacked
                constexpr int kTimes = kKeys * (D / 8) / kImageThreads, kStep = kImageThreads / (D / 8);
                const int pos0 = tid / (D / 8), c8 = tid % (D / 8);
                uint2 ck[kTimes], cv[kTimes];
#pragma unroll
                for (int i = 0; i < kTimes; ++i) {
                    const int pos = pos0 + i * kStep;
                    const int64_t src = parts[pos / kSub].at + (pos % kSub) * D + 8 * c8;
                    const bool in = tile * kKeys + pos < v.kv;
                    ck[i] = in ? __ldcs(reinterpret_cast<const uint2*>(p.k + src)) : make_uint2(0u, 0u);
                    cv[i] = in ? __ldcs(reinterpret_cast<const uint2*>(p.v + src)) : make_uint2(0u, 0u);
                }
                unsigned char* const img = a.images + ((size_t)(base + tile) * p.heads + head) * (2 * kTileBytes<D>);
#pragma unroll
                for (int i = 0; i < kTimes; ++i) {
                    const int pos = pos0 + i * kStep;
                    const bool in = tile * kKeys + pos < v.kv;  // (a NaN factor leaves what lies behind at 0)
                    const float fk = in ? parts[pos / kSub].k : 0.0f, fv = in ? parts[pos / kSub].v : 0.0f;
                    *reinterpret_cast<uint4*>(img + image_off(pos, c8)) = BF16 ? unpack8_bf16<E4M3>(ck[i], fk) : unpack8<E4M3>(ck[i], __float2half2_rn(fk));
                    *reinterpret_cast<uint4*>(img + kTileBytes<D> + image_off(pos, c8)) = unpack8<E4M3>(cv[i], __float2half2_rn(fv));
                }
                __syncthreads();  // parts read
            }
            __syncthreads();  // the warps' extremes read
        }
        at = 0;
    }
}

template <int D>
struct PromptSmem {
    static constexpr int kSlots = D == 128 ? 4 : 8;
    unsigned char q[2][kTileBytes<D>];
    unsigned char kv[kSlots][kTileBytes<D>];   // K and V images in turn
    Unit unit[kUnits];
    float other[2][2][128];                    // what a row's two threads tell each other
    uint64_t kv_full[kSlots], kv_empty[kSlots];
    uint64_t unit_full[kUnits], unit_empty[kUnits], q_full[kUnits][2];  // (by unit: no role can be two of a half's queries behind)
    uint64_t q_empty[2], s_full[2], p_full[2], o_full[2], drain;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(PromptSmem<128>) <= 232448 && sizeof(PromptSmem<64>) <= 232448, "shared memory");

// barriers of the two warps that hold the two halves of the same rows' columns (64 threads, ids 1-8)
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

// Bounded wait (about two seconds of SM clock; abandoned once another warp of the CTA has given up).  The
// warp agrees on the outcome and stays converged.
__device__ __noinline__ bool wait_long(uint64_t* mbar, uint32_t parity, const volatile int* abort_flag)
{
    bool ok = false;
    const long long start = clock64();
    while (!(ok = umma::mbar_try_wait_suspend(mbar, parity, 20000u)))
        if (*abort_flag || clock64() - start > (4ll << 30)) break;
    return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool wait_for(uint64_t* mbar, uint32_t parity, const volatile int* abort_flag)
{
    return __all_sync(0xffffffffu, umma::mbar_try_wait(mbar, parity)) || wait_long(mbar, parity, abort_flag);
}

// Whatever completes phase `parity` has ended (bounded, about half a second of SM clock; copies and products end by
// themselves).
__device__ __forceinline__ void drain(uint64_t* mbar, uint32_t parity)
{
    const long long start = clock64();
    while (!umma::mbar_try_wait_suspend(mbar, parity, 20000u) && clock64() - start < (1ll << 30)) {}
}

// 32 bytes, on a boundary of 32
__device__ __forceinline__ void store8(void* to, const uint32_t* w)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
                 "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
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
__global__ void __launch_bounds__(kThreads, 1) kv_prompt_kernel(AttnParams p, AttnSpace a, const __grid_constant__ CUtensorMap q_map)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    using Smem = PromptSmem<D>;
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    constexpr int kSlots = Smem::kSlots;
    constexpr uint32_t kTile = kTileBytes<D>;
    constexpr uint32_t kColS = 128, kColO = 256, kTmemCols = 512;  // S of half h at 128 h, O at 256 + 128 h
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int group = p.hq / p.heads, tokens = half_tokens(group);
    if (warp == kMmaWarp) umma::tmem_alloc(&sm.tmem_base, kTmemCols);
    if (warp == kQueryWarp && lane == 0) umma::prefetch_map(&q_map);
    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            umma::mbar_init(&sm.kv_full[i], 1);
            umma::mbar_init(&sm.kv_empty[i], 1);
        }
        for (int i = 0; i < kUnits; ++i) {
            umma::mbar_init(&sm.unit_full[i], 1);
            umma::mbar_init(&sm.unit_empty[i], 18);  // the softmax warps, the copies and the products
            umma::mbar_init(&sm.q_full[i][0], 1);
            umma::mbar_init(&sm.q_full[i][1], 1);
        }
        for (int h = 0; h < 2; ++h) {
            umma::mbar_init(&sm.q_empty[h], 1);
            umma::mbar_init(&sm.s_full[h], 1);
            umma::mbar_init(&sm.p_full[h], 256);
            umma::mbar_init(&sm.o_full[h], 1);
        }
        umma::mbar_init(&sm.drain, 1);
        sm.abort_flag = 0;
    }
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem_base, 0);
    const volatile int* abort_flag = &sm.abort_flag;
    pdl_wait();
    pdl_launch_dependents();

    // A wait that expires is recorded; its warp goes on or ends as its role allows.
    auto await = [&](uint64_t* mbar, uint32_t parity) {
        const bool ok = wait_for(mbar, parity, abort_flag);
        if (!ok && lane == 0) {
            sm.abort_flag = 1;
            atomicOr(&a.head->error, kAttnTimeout);
        }
        return ok;
    };
#define GDN_KV_WAIT(mbar, parity)                   \
    do {                                            \
        if (!await((mbar), (parity))) goto done;    \
    } while (0)

    // the unit in hand: ring place x % kUnits, its x / kUnits-th use
    auto unit_ready = [&](uint32_t x) { return await(&sm.unit_full[x % kUnits], (x / kUnits) & 1); };
    auto unit_done = [&](uint32_t x) {
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(&sm.unit_empty[x % kUnits]);
    };

    if (warp >= kLoadWarp) {
        if (warp >= kQueryWarp) {
            // ---- units and queries ----
            const int span = 2 * tokens, workers = a.head->prompt_workers;
            const bool handed = a.head->prompt_whole;
            const int64_t total = a.head->prompt_total;
            const Cut c = a.prompt_cut[blockIdx.x];  // (all these loads at once: what lies past the workers is not used)
            const int64_t next_lo = a.prompt_cut[min(blockIdx.x + 1, kPromptMaxWorkers - 1)].lo;
            uint32_t x = 0, q_use[2] = {0, 0};  // units, and queries of each half, brought in
            uint32_t q_armed[2] = {0, 0};       // units whose q_full of each half completes by itself
            bool more = (int)blockIdx.x < workers, first_unit = true;
            Walk w;
            if (more) {
                w.s = c.s;
                w.head = c.head;
                w.i = c.unit;
                w.t0 = c.t0;
                w.n = c.n;
                w.first = c.first;
                w.units = (c.n + span - 1) / span;
                w.ok = images_there(p, a, c.s);
                w.image = min(c.image, a.image_tiles - 1);
                w.from = c.from;
                w.left = handed ? (int64_t)1 << 62 : ((int)blockIdx.x + 1 < workers ? next_lo : total) - c.lo;
                w.jobs = c.lo;  // (handed out)
            }
            while (more) {
                const int tiles = unit_tiles(w.first, w.n, span, w.i);
                const int to = (int)min((int64_t)tiles + kPromptUnitCost, w.from + w.left);
                const int j0 = max(w.from - kPromptUnitCost, 0), count = to - kPromptUnitCost - j0;
                const HeadUnits of = a.units[(size_t)w.image * p.heads + w.head];
                if (count > 0 && w.ok) {  // (a range may end within a unit's constant)
                    if (x >= kUnits && !await(&sm.unit_empty[x % kUnits], (x / kUnits - 1) & 1)) goto queries_done;
                    const int token = w.i * span;
                    if (lane == 0) {
                        Unit& u = sm.unit[x % kUnits];
                        u.count = count;
                        u.tile = w.image + j0;
                        u.j0 = j0;
                        u.head = w.head;
                        u.first = w.first;
                        u.t0 = w.t0;
                        u.n = w.n;
                        u.token = token;
                        u.whole = count == tiles;
                        u.slot = 2 * blockIdx.x + (first_unit ? 0 : 1);  // (the range's first, were it one without images)
                        // (above 0, so that a masked score of -infinity stays one whatever the scale; the least fp32
                        // above it, so that bf16 scores of up to 2^127 times a softmax_scale of 0 are nothing)
                        u.score_unit = fmaxf(fabsf(p.scale) * kLog2e * (BF16 ? 1.0f : of.k * (1.0f / kUp<E4M3>)), __uint_as_float(1u));
                        u.v_unit = of.v * (1.0f / kUp<E4M3>);
                        u.nan_from = of.nan_from;
                        umma::mbar_arrive(&sm.unit_full[x % kUnits]);
                    }
                    for (int h = 0; h < 2; ++h) {
                        const int token0 = token + h * tokens;
                        const bool rows = token0 < w.n;  // (else a second half without rows)
                        if (rows) {
                            if (q_use[h] > 0 && !await(&sm.q_empty[h], (q_use[h] - 1) & 1)) goto queries_done;
                            ++q_use[h];
                        }
                        if (lane == 0) {
                            uint64_t* const full = &sm.q_full[x % kUnits][h];
                            if (rows) {
                                // (rows past the sequence's end are another's or zeros; what comes of them is not written)
                                umma::mbar_arrive_expect_tx(full, tokens * group * D * 2);
                                for (int plane = 0; plane < D / 64; ++plane)
                                    umma::tensor_g2s_3d(sm.q[h] + plane * kPlane, &q_map, 64 * plane, w.head * group, w.t0 + token0, full);
                            } else {
                                umma::mbar_arrive(full);
                            }
                        }
                        q_armed[h] = x + 1;
                    }
                    ++x;
                }
                first_unit = false;
                if (handed) {
                    // the next one once the last scores of this are under way: sooner would leave it to a busy CTA
                    if (q_use[0] > 0 && !await(&sm.q_empty[0], (q_use[0] - 1) & 1)) goto queries_done;
                    int job = lane == 0 ? atomicAdd(&a.head->prompt_next, 1) : 0;
                    more = w.take(p, a, span, __shfl_sync(0xffffffffu, job, 0));
                } else {
                    more = w.next(p, a, span, to - w.from);
                }
            }
            if (x >= kUnits && !await(&sm.unit_empty[x % kUnits], (x / kUnits - 1) & 1)) goto queries_done;
            if (lane == 0) {
                sm.unit[x % kUnits].count = 0;
                umma::mbar_arrive(&sm.unit_full[x % kUnits]);
            }
        queries_done:
            // no copy may be in flight when the CTA leaves: after an expired wait nobody else has waited for these
            for (int h = 0; h < 2; ++h)
                for (uint32_t i = q_armed[h] > kUnits ? q_armed[h] - kUnits : 0; i < q_armed[h]; ++i) drain(&sm.q_full[i % kUnits][h], (i / kUnits) & 1);
        } else if (warp == kLoadWarp) {
            // ---- copies: K and V of each tile in turn through the ring ----
            uint32_t n = 0;  // copies issued
            for (uint32_t x = 0; unit_ready(x); ++x) {
                const Unit& u = sm.unit[x % kUnits];
                const int count = u.count;
                if (count == 0) break;
                const unsigned char* src = a.images + ((size_t)u.tile * p.heads + u.head) * (2 * kTile);
                const size_t stride = (size_t)p.heads * (2 * kTile);
                unit_done(x);
                for (int j = 2 * count; j > 0; --j, ++n) {
                    const uint32_t slot = n % kSlots;
                    if (n >= kSlots && !await(&sm.kv_empty[slot], (n / kSlots - 1) & 1)) goto copies_done;
#ifdef GDN_KV_SELFTEST_WITHHOLD_COPY  // the failure report's test builds a library without each CTA's first copy
                    if (lane == 0 && n > 0) {
#else
                    if (lane == 0) {
#endif
                        umma::mbar_arrive_expect_tx(&sm.kv_full[slot], kTile);
                        umma::bulk_g2s(sm.kv[slot], j & 1 ? src + kTile : src, kTile, &sm.kv_full[slot]);
                    }
                    if (j & 1) src += stride;
                }
            }
        copies_done:
            for (uint32_t i = n > kSlots ? n - kSlots : 0; i < n; ++i) drain(&sm.kv_full[i % kSlots], (i / kSlots) & 1);
        } else {
            // ---- products, issued by one lane ----
            constexpr uint32_t id_s = BF16 ? umma::idesc_bf16(128, kKeys, false, false) : umma::idesc_f16(128, kKeys, false, false);
            constexpr uint32_t id_o = umma::idesc_f16(128, D, false, true);  // V: channels (N) contiguous
            // descriptors of the first tiles; the others lie a whole number of tiles behind them
            const uint64_t q_desc = umma::desc_sw128(umma::smem_u32(sm.q[0]), 16, 1024);
            const uint64_t k_desc = umma::desc_sw128(umma::smem_u32(sm.kv[0]), 16, 1024);
            const uint64_t v_desc = umma::desc_sw128(umma::smem_u32(sm.kv[0]), kPlane, 1024);
            uint32_t n = 0;  // ring position of the current tile's K
            uint32_t p_phase[2] = {0, 0};
            // (one lane, in a converged warp)
            auto scores = [&](int h, uint32_t at, bool last) {
                const uint64_t da = q_desc + h * (kTile >> 4), db = k_desc + (at % kSlots) * (kTile >> 4);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {  // 16 channels: 32 bytes of a plane's rows
                    const uint32_t step = (ks >> 2) * (kPlane >> 4) + 2 * (ks & 3);
                    umma::mma_bf16(tmem + h * kColS, da + step, db + step, id_s, ks != 0);
                }
                umma::commit(&sm.s_full[h]);
                if (last) umma::commit(&sm.q_empty[h]);
            };
            auto outputs = [&](int h, uint32_t at, bool start, bool last) {
                const uint64_t db = v_desc + (at % kSlots) * (kTile >> 4);
#pragma unroll
                for (int ks = 0; ks < kKeys / 16; ++ks)  // 16 keys: two atoms of 8 rows
                    umma::mma_ts(tmem + kColO + h * kColS, tmem + h * kColS + 64 * (ks >> 2) + 8 * (ks & 3), db + ks * (2048 >> 4), id_o, !(start && ks == 0));
                if (last) umma::commit(&sm.o_full[h]);
            };
            for (uint32_t x = 0; unit_ready(x); ++x) {
                const Unit& u = sm.unit[x % kUnits];
                const int count = __shfl_sync(0xffffffffu, u.count, 0);
                if (count == 0) break;
                const bool both = __shfl_sync(0xffffffffu, u.token + tokens < u.n, 0);  // the second half has rows
                GDN_KV_WAIT(&sm.kv_full[n % kSlots], (n / kSlots) & 1);
                GDN_KV_WAIT(&sm.q_full[x % kUnits][0], (x / kUnits) & 1);
                umma::fence_after_sync();
                if (umma::elect_one()) scores(0, n, count == 1);
                __syncwarp();
                if (both) {
                    GDN_KV_WAIT(&sm.q_full[x % kUnits][1], (x / kUnits) & 1);
                    umma::fence_after_sync();
                }
                if (umma::elect_one()) {
                    if (both) scores(1, n, count == 1);
                    umma::commit(&sm.kv_empty[n % kSlots]);
                }
                unit_done(x);
                // the copies that a tile's products read are waited for a tile ahead, while the tensor cores have work
                GDN_KV_WAIT(&sm.kv_full[(n + 1) % kSlots], ((n + 1) / kSlots) & 1);
                if (count > 1) GDN_KV_WAIT(&sm.kv_full[(n + 2) % kSlots], ((n + 2) / kSlots) & 1);
                for (int j = 0; j < count; ++j, n += 2) {
                    const bool last = j + 1 == count;
                    GDN_KV_WAIT(&sm.p_full[0], p_phase[0]);
                    p_phase[0] ^= 1u;
                    umma::fence_after_sync();
                    if (umma::elect_one()) {
                        outputs(0, n + 1, j == 0, last);
                        if (!last) scores(0, n + 2, j + 2 == count);
                    }
                    __syncwarp();
                    if (both) {
                        GDN_KV_WAIT(&sm.p_full[1], p_phase[1]);
                        p_phase[1] ^= 1u;
                        umma::fence_after_sync();
                    }
                    if (umma::elect_one()) {
                        if (both) outputs(1, n + 1, j == 0, last);
                        umma::commit(&sm.kv_empty[(n + 1) % kSlots]);
                        if (!last) {
                            if (both) scores(1, n + 2, j + 2 == count);
                            umma::commit(&sm.kv_empty[(n + 2) % kSlots]);
                        }
                    }
                    __syncwarp();
                    if (!last) {
                        GDN_KV_WAIT(&sm.kv_full[(n + 3) % kSlots], ((n + 3) / kSlots) & 1);
                        if (j + 2 < count) GDN_KV_WAIT(&sm.kv_full[(n + 4) % kSlots], ((n + 4) / kSlots) & 1);
                    }
                }
            }
        }
    } else {
        // ---- softmax: a row's two threads share a tile's columns ----
        // After a wait that has expired its warp goes on, with waits that no longer wait: the two warps of the
        // same rows meet at barriers, and the loops over tiles end by themselves.
        const int h = warp >> 3, part = (warp >> 2) & 1, r = (warp & 3) * 32 + lane, pair = 1 + 4 * h + (warp & 3);
        // this thread's score columns, and half of its row's outputs
        const uint32_t t_s = tmem + ((uint32_t)((warp & 3) * 32) << 16) + h * kColS + 64 * part, t_o = t_s + kColO - part * (64 - D / 2);
        uint32_t phase = 0, units = 0;  // parity of the next scores' completion; units whose output was waited for
        // 32 of the thread's scores, -infinity from the column after `last` on
        auto scores = [&](int c, int last, float (&x)[32]) {
            umma::tmem_ld32(t_s + 32 * c, x);
            umma::tmem_wait_ld();
            if (last < 32 * c + 31)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (32 * c + e > last) x[e] = -INFINITY;
        };
        for (uint32_t x_unit = 0;; ++x_unit) {
            const bool ready = unit_ready(x_unit);
            const Unit& u = sm.unit[x_unit % kUnits];
            // (both warps of a pair take the same way: they meet here)
            if (pair_any(pair, !ready) || u.count == 0) break;
            const int token0 = u.token + h * tokens;
            if (token0 < u.n) {  // (a second half without rows does nothing)
                const float coef = u.score_unit;
                // the last of the thread's columns that the row sees, in the tile in hand
                int last = -1;
                {
                    const int i_tok = r / group;
                    if (i_tok < tokens && token0 + i_tok < u.n) last = u.first + token0 + i_tok - (u.j0 * kKeys + 64 * part);
                }
                float m = -INFINITY, l = 0.0f;  // m: the reference, in units of the scores as they come
                // A weight's exponent is x mul + off, one fused operation with mul = coef and off = kWeightShift - m coef;
                // m moves where a score passes `most`.  The products lie up to half a step of theirs beside the
                // rounded ones in off, which for large scores would take a weight out of fp16's range.  So from
                // kLargeScore on m is the maximum itself, and from kHugeScore on, where the steps of fp32 scores and the
                // errors of their sums are far above a weight's range, mul is a power of two and the products exact.
                float most = -INFINITY, mul = coef;
                const float lazy = kLazy / coef;
                float off = kWeightShift;
                const int count = u.count;
#pragma unroll 1
                for (int j = 0; j < count; ++j, last -= kKeys) {
                    await(&sm.s_full[h], phase);
                    phase ^= 1u;
                    umma::fence_after_sync();
                    // (32 of the thread's 64 scores at a time: all of them and their weights do not fit its registers)
                    float x[32], top = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        scores(c, last, x);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) top = fmaxf(top, fmaxf(x[e], x[e + 1]));
                    }
                    if (pair_any(pair, top > most)) {
                        sm.other[h][part][r] = top;
                        pair_sync(pair);
                        top = fmaxf(top, sm.other[h][part ^ 1][r]);
                        float f = 1.0f;
                        if (top > most) {
                            f = ex2((m - top) * coef);
                            m = top;
                            l *= f;
                            const float size = fabsf(m * coef);
                            mul = size < kHugeScore ? coef : __uint_as_float(__float_as_uint(coef) & 0x7f800000u);
                            off = kWeightShift - m * mul;
                            most = size < kLargeScore ? m + lazy : m;
                        }
                        // O holds the products up to tile j - 1, which ended before this tile's scores
                        if (j > 0 && __any_sync(0xffffffffu, f != 1.0f)) {
#pragma unroll
                            for (int c = 0; c < D / 32; ++c) {
                                float o[16];
                                uint32_t w[16];
                                umma::tmem_ld16(t_o + 16 * c, o);
                                umma::tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * f);
                                umma::tmem_st16(t_o + 16 * c, w);
                            }
                        }
                    }
                    const uint64_t coef2 = pair2(mul, mul), off2 = pair2(off, off);
                    uint64_t sum[2] = {0, 0};
                    uint32_t u0[16], u1[16];
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
                    scores(0, last, x);
                    umma::tmem_st16(t_s + 16, u1);
                    weights(u0);
                    umma::tmem_st16(t_s, u0);
                    umma::tmem_wait_st();
                    umma::fence_before_sync();
                    umma::mbar_arrive(&sm.p_full[h]);
                    float s0, s1;
                    unpair2(add2(sum[0], sum[1]), s0, s1);
                    l += s0 + s1;
                }
                pair_sync(pair);  // the last tile's maxima are read
                sm.other[h][part][r] = l;
                pair_sync(pair);
                l += sm.other[h][part ^ 1][r];
                await(&sm.o_full[h], units & 1);
                ++units;
                umma::fence_after_sync();
                const int i_tok = r / group, tok = token0 + i_tok, qh = r - i_tok * group;
                const bool wide = (reinterpret_cast<uintptr_t>(p.y) & 31) == 0, whole = u.whole, valid = i_tok < tokens && tok < u.n;
                const int slot = u.slot, row = 128 * h + r;
                // (every row sees its own position: l is 0 only where all scores are -infinity, and y is NaN)
                float scale = whole ? u.v_unit / l : u.v_unit;
                if (u.first + tok >= u.nan_from) scale = __uint_as_float(0x7fffffffu);
                uint16_t* const dst = p.y + ((int64_t)(u.t0 + tok) * p.hq + u.head * group + qh) * D + part * (D / 2);
                if (!whole && part == 0) a.prompt_stat[(size_t)slot * kUnitRows + row] = make_float2(m * u.score_unit, l);
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    float o[32];
                    umma::tmem_ld32(t_o + 32 * c, o);
                    umma::tmem_wait_ld();
                    if (whole) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = narrow2<BF16>(o[2 * e] * scale, o[2 * e + 1] * scale);
                        if (valid) {
                            // a warp's rows lie apart, each store touches 32 lines: stores of 32 bytes where y
                            // allows (2048-token prompt 72.8 -> 70.6 us)
                            if (wide) {
                                store8(dst + 32 * c, w);
                                store8(dst + 32 * c + 16, w + 8);
                            } else {
#pragma unroll
                                for (int e = 0; e < 16; e += 4) *reinterpret_cast<uint4*>(dst + 32 * c + 2 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            a.prompt_out[((size_t)slot * (D / 4) + part * (D / 8) + 8 * c + e / 4) * kUnitRows + row] =
                                make_float4(o[e] * scale, o[e + 1] * scale, o[e + 2] * scale, o[e + 3] * scale);
                    }
                }
                umma::fence_before_sync();  // O read before the next unit's products (which wait for this thread's weights)
            }
            unit_done(x_unit);
        }
    }
done:
    // every product issued has ended before TMEM and shared memory go
    __syncwarp();
    if (warp == kMmaWarp) {
        if (umma::elect_one()) {  // (the lane that issued them)
            umma::commit(&sm.drain);
            drain(&sm.drain, 0);
        }
        __syncwarp();
    }
    umma::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) umma::tmem_dealloc(tmem, kTmemCols);
#undef GDN_KV_WAIT
}

template <int D, bool BF16, bool E4M3>
cudaError_t launch(const AttnParams& p, const AttnSpace& a, int sms, cudaStream_t stream)
{
    const int64_t items = (int64_t)a.image_tiles * p.heads;
    const int grid = prompt_grid(sms);
    cudaError_t e = launch_k(kv_image_kernel<D, BF16, E4M3>, dim3((unsigned)(items < sms * 3 ? items + 1 : sms * 3)), dim3(kImageThreads), 0, stream, true, p, a, grid);
    if (e != cudaSuccess) return e;
    auto kernel = kv_prompt_kernel<D, BF16, E4M3>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(PromptSmem<D>));
    if (e != cudaSuccess) return e;
    // queries as [token][head][channel]; a box is the tokens of half a unit, one kv head's heads, 64 channels
    const auto encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    CUtensorMap q_map;
    const int group = p.hq / p.heads;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.hq, (cuuint64_t)p.T}, strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)p.q_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)(kUnitRows / 2 / group)}, ones[3] = {1, 1, 1};
    if (encode(&q_map, BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<uint16_t*>(p.q), dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    return launch_k(kernel, dim3(grid), dim3(kThreads), sizeof(PromptSmem<D>), stream, true, p, a, q_map);
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
