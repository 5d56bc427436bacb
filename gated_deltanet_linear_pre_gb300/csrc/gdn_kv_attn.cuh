// gdn_kv_attn.cuh -- what the attention's kernels share: which sequences go which
// way, the split of a ragged batch into equal shares of work, and the workspace.
//
// Two ways through the cache.  Sequences with few query rows (tokens times query heads per kv head, up
// to kLongRows) go to the step kernel, which reads the codes themselves; the others are long: their
// cache is unpacked once to fp16 operand images, which the prompt kernel then reads for every 256 query
// rows.  A long sequence whose images would not be exact (exact_ratio), have no room or lack a page takes the
// step kernel too.  The choice is made per sequence on the device, so one call serves a batch that mixes prompts
// and single tokens, and a captured call follows its lengths.
//
// Work is counted in key tiles: a unit is (sequence, kv head, group of query rows) and costs the tiles
// that it sees and a constant for its beginning and end.  The units of a batch, end to end, are cut into
// equal ranges, one per worker (CTA), so that one long sequence and many short ones load the GPU alike.  A
// unit whose tiles lie in one range is finished by its worker; one that is cut leaves a partial (maximum,
// sum, output) per worker, and a last kernel joins them in the order of the ranges.  A range that ends
// within a unit's constant has none of its tiles.
#pragma once

#include "gdn_kv.cuh"

namespace gdn {

constexpr int kSub = 16;               // positions of a step tile's part (a page holds whole ones)
template <int D> constexpr int kStepTile = D == 128 ? kSub : 2 * kSub;  // positions of a step tile: 4 KB of codes
constexpr int kStepMaxRows = 32;       // query rows of a step unit, at most
constexpr int kStepMaxWorkers = 480;
constexpr int kStepUnitCost = 16;      // a step unit's beginning and end, in tiles
constexpr int kPromptUnitCost = 2;     // a prompt unit's
constexpr int kPromptCutCost = 6;      // what cutting the prompt units costs a worker, beside a sixteenth of
                                       // its share (whole_units)
constexpr int kKeys = 128;             // positions of a prompt tile
constexpr int kUnitRows = 256;         // query rows of a prompt unit: two halves of 128
constexpr int kPromptMaxWorkers = 160;
// Above this many query rows the prompt way is faster: 16 sequences of 8K positions (4 heads, e4m3) took
// 127 us by steps at 96 rows and 161 at 128, 137 and 135 us by images; 4 of 2000 26.7 and 29.5, 26.9 and 27.2.
constexpr int kLongRows = 96;
// Where the page table holds at most this many positions (times 128 / head_dim) step units stay whole, and no
// kernel joins them: a unit's last tiles take less than a second launch (64 sequences of 490 positions, 4 heads,
// 15.1 us whole and 18.1 cut; 16 heads 38.3 and 38.4, of lengths up to 500 30.1 and 27.6).  Twice as many where
// the (sequence, kv head) pairs are few (kWholeUnits): 16 sequences of 900 positions, 4 heads, 12.8 us whole and
// 16.7 cut, 38 of 1000 15.5 and 18.5; but 64 of lengths up to 1000 20.4 and 18.6.
constexpr int kWholePositions = 512;
constexpr int kWholeUnits = 152;  // (one for each SM of this GPU)
constexpr size_t kImageCap = (size_t)2 << 30;  // bytes of images; sequences past it take the step kernel

constexpr uint32_t kAttnTimeout = 1u;  // failure record: a bounded wait expired

// a sequence as the attention sees it
struct SeqView {
    int t0, n, first;  // its tokens of this call, the first one's position
    int kv;            // positions it may see
};

__device__ __forceinline__ SeqView seq_view(const KvBatch& p, int s)
{
    SeqView v;
    v.t0 = cu_at(p.cu_seqlens, s, p.T);
    v.n = max(cu_at(p.cu_seqlens, s + 1, p.T) - v.t0, 0);
    v.first = past_at(p.past, s);
    v.kv = min(max(v.first + v.n, 0), p.max_pages * p.page);
    return v;
}

// where the range of a worker begins: tile j0 of a unit of `tiles`
struct Cut {
    int s, head, unit, j0, tiles;  // unit: the step unit's first row, the prompt unit's index
    int from;                      // cost of the unit that lies before the range
    int64_t lo;                    // cost of all units that does
    int t0, n;                     // the sequence's tokens
    int first, image;              // (prompt) its first position and image tile
};

// what the images of a (sequence, kv head) leave out
struct alignas(16) HeadUnits {
    float k, v;    // largest scales
    int nan_from;  // first position of a page whose v scale is NaN: rows that see it are NaN
    int unused;
};

struct AttnHeader {
    uint32_t error;
    int step_workers, prompt_workers;
    int prompt_whole, prompt_next;  // prompt units are not cut but handed out one by one; the next one
    int64_t step_total, prompt_total;
};

// the workspace's parts (kv_attn.cu lays them out)
struct AttnSpace {
    AttnHeader* head;
    Cut* step_cut;         // [kStepMaxWorkers]
    float2* step_stat;     // [2 kStepMaxWorkers][kStepMaxRows]: maximum (base 2), sum; two per worker, the
    float* step_out;       //   range's first unit and its last;  [..][kStepMaxRows][dim]
    // the rest is there only where the batch may hold a long sequence (image_tiles > 0)
    uint8_t* ok;           // [n_seq][ok_stride(heads)] 1: the images of that head are written (1 behind the last)
    int* image_base;       // [n_seq] its first image tile
    HeadUnits* units;      // [image_tiles][heads], at the sequence's first tile
    Cut* prompt_cut;       // [kPromptMaxWorkers]
    float2* prompt_stat;   // [2 kPromptMaxWorkers][kUnitRows]
    float4* prompt_out;    // [2 kPromptMaxWorkers][dim / 4][kUnitRows]
    unsigned char* images; // [image_tiles][heads][2]: K and V operand images of 128 positions
    int image_tiles;
    int most_rows;         // sequences with more query rows are candidates for the prompt way
    int whole_units;       // step units are not cut: ranges of units, not of tiles
};

__device__ __forceinline__ bool candidate(const KvBatch& p, const AttnSpace& a, const SeqView& v)
{
    // (negative positions and positions past the table take the step kernel, which sees to them)
    return (int64_t)v.n * (p.hq / p.heads) > a.most_rows && v.first >= 0 && v.first + v.n <= p.max_pages * p.page;
}
__host__ __device__ constexpr int ok_stride(int heads) { return (heads + 15) & ~15; }
// whether the images of all heads of a candidate are written
__device__ __forceinline__ bool images_there(const KvBatch& p, const AttnSpace& a, int s)
{
    const uint4* row = reinterpret_cast<const uint4*>(a.ok + (size_t)s * ok_stride(p.heads));
    uint32_t all = 0x01010101u;
    for (int i = 0; i < ok_stride(p.heads) / 16; ++i) all &= row[i].x & row[i].y & row[i].z & row[i].w;
    return all == 0x01010101u;
}
__device__ __forceinline__ bool is_long(const KvBatch& p, const AttnSpace& a, int s, const SeqView& v) { return candidate(p, a, v) && images_there(p, a, s); }

// the cut of `total` tiles into `workers` ranges: start of range w, and the range that holds tile x
__device__ __forceinline__ int64_t cut_start(int64_t total, int workers, int w) { return total * w / workers; }
__device__ __forceinline__ int cut_of(int64_t total, int workers, int64_t x) { return (int)(((x + 1) * workers - 1) / total); }

// tokens of half a prompt unit: as many as fit 128 rows of (token, query head of the kv head)
__device__ __forceinline__ int half_tokens(int group) { return (kUnitRows / 2) / group; }

// ---- where a worker's range begins -------------------------------------------------
template <int THREADS>
struct ScanSmem {
    int64_t chunk[65536 / THREADS + 1];  // sums over every THREADS sequences (at most 65535 of them)
    int64_t prefix[THREADS + 1], warp_sum[THREADS / 32];
    int found;
};

// exclusive scan over the block; `total` for all
template <int THREADS>
__device__ __forceinline__ int64_t block_scan(int64_t mine, ScanSmem<THREADS>& sm, int64_t& total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t v = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += o;
    }
    __syncthreads();  // warp_sum free
    if (lane == 31) sm.warp_sum[warp] = v;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) v += sm.warp_sum[w];
        total += sm.warp_sum[w];
    }
    return v - mine;
}

// the sum of weight(s) over all sequences
template <int THREADS, typename F>
__device__ __forceinline__ int64_t scan_total(int n_seq, F weight, ScanSmem<THREADS>& sm)
{
    int64_t total = 0;
    for (int c = 0; c * THREADS < n_seq; ++c) {
        const int s = c * THREADS + threadIdx.x;
        int64_t sum;
        const int64_t before = block_scan<THREADS>(s < n_seq ? weight(s) : 0, sm, sum);
        if (c == 0) sm.prefix[threadIdx.x] = before;  // a single chunk needs no second look
        if (threadIdx.x == 0) sm.chunk[c] = sum;
        total += sum;
    }
    return total;
}

// the sequence that holds x (0 <= x < scan_total's result), and the sum before it
template <int THREADS, typename F>
__device__ __forceinline__ int scan_find(int n_seq, int64_t x, F weight, ScanSmem<THREADS>& sm, int64_t& before)
{
    __syncthreads();
    const int chunks = (n_seq + THREADS - 1) / THREADS;
    int64_t base = 0;
    int c = 0;
    while (c + 1 < chunks && base + sm.chunk[c] <= x) base += sm.chunk[c++];
    if (c > 0) {
        const int s = c * THREADS + threadIdx.x;
        int64_t sum;
        const int64_t b = block_scan<THREADS>(s < n_seq ? weight(s) : 0, sm, sum);
        sm.prefix[threadIdx.x] = b;
    }
    if (threadIdx.x == 0) {
        sm.prefix[THREADS] = sm.chunk[c];
        sm.found = 0;
    }
    __syncthreads();
    if (base + sm.prefix[threadIdx.x] <= x && x < base + sm.prefix[threadIdx.x + 1]) sm.found = threadIdx.x;
    __syncthreads();
    before = base + sm.prefix[sm.found];
    return c * THREADS + sm.found;
}

// ---- 8-bit codes to fp16 ------------------------------------------------------------
// Two codes, bytes 0 and 1 (HIGH: 2 and 3) of y, to a pair of fp16 values, exactly:
//   int8: 1024 + (code + 128) assembled as fp16 bits, less 1152;
//   e4m3: the hardware's conversion.
template <bool E4M3, bool HIGH>
__device__ __forceinline__ uint32_t codes2(uint32_t y)
{
    if (E4M3) {
        uint32_t h;
        if (HIGH) asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(h) : "r"(y));
        else asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(y));
        return h;
    }
    const uint32_t x = __byte_perm(y ^ 0x80808080u, 0x64646464u, HIGH ? 0x4342 : 0x4140);
    const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&x), __half2half2(__ushort_as_half((unsigned short)0x6480)));
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float ex2(float x)  // 2^x; results below 2^-126 are 0
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Power of two that brings a query row (the bits of its largest magnitude) to [2^14, 2^15), and its
// inverse: fp16 then holds a row of either type, exactly for fp16 and, less what is 2^-29 of the row's
// largest, for bf16.  Rows of zeros, infinities or NaN stay as they are.
__device__ __forceinline__ void row_unit(uint32_t amax, float& mul, float& back)
{
    const int e = (int)(amax >> 23);
    const int up = amax != 0 && e < 255 ? 141 - max(e, 41) : 0;
    mul = __uint_as_float((uint32_t)(127 + up) << 23);
    back = __uint_as_float((uint32_t)(127 - up) << 23);
}

constexpr float kLog2e = 1.4426950408889634f;

// CTAs an SM of the step kernel, and its CTAs.  Three with rings of two tiles a warp keep some 48 KB in flight
// beside the tiles in work, which is enough: with four and rings of three, requests only waited for one another
// (64 sequences of up to 8192 positions 71.2 -> 68.1 us, 3 of 131000 50.0 -> 45.5, 37 sequences of drafts 88.8 ->
// 81.6; two and rings of four: 66.4, 69.3 and 89.8), and three leave the registers for the queries.
constexpr int step_ctas(int rows) { return rows == kStepMaxRows ? 2 : 3; }
inline int step_grid(int sms, int rows) { return sms * step_ctas(rows) < kStepMaxWorkers ? sms * step_ctas(rows) : kStepMaxWorkers; }
inline int prompt_grid(int sms) { return sms < kPromptMaxWorkers ? sms : kPromptMaxWorkers; }

// the kernels' launches (gdn_kv_step.cu, gdn_kv_prompt.cu, gdn_kv_join.cu)
int step_rows(const AttnParams& p, const AttnSpace& a);  // query rows of a step unit
cudaError_t launch_kv_join(const AttnParams& p, const AttnSpace& a, int sms, cudaStream_t stream);
cudaError_t launch_kv_step(const AttnParams& p, const AttnSpace& a, int sms, cudaStream_t stream);
cudaError_t launch_kv_prompt(const AttnParams& p, const AttnSpace& a, int sms, cudaStream_t stream);

}  // namespace gdn
