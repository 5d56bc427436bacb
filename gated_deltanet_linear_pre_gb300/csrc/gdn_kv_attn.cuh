// gdn_kv_attn.cuh -- what the attention's kernels share: the split of a ragged
// batch into equal shares of work, and the workspace.
//
// Work is counted in key tiles: a unit is (sequence, kv head, group of query rows) and costs the
// sequence's tiles.  The units of a batch, end to end, are cut into equal ranges, one per worker (CTA),
// so that one long sequence and many short ones load the GPU alike, whatever the lengths; the cuts come
// from the device's own lengths and change with them between replays of a captured call.  A unit that
// lies in one range is finished by its worker; one that is cut leaves a partial (maximum, sum, output)
// per worker, and a last kernel joins them in order.
#pragma once

#include "gdn_kv.cuh"

namespace gdn {

constexpr int kStepThreads = 256;
constexpr int kSub = 16;              // positions of one step tile (a page holds whole ones)
constexpr int kStepMaxRows = 32;      // query rows of a step unit, at most
constexpr int kStepMaxWorkers = 512;

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

// the cut of `total` tiles into `workers` ranges: start of range w, and the range that holds tile x
__host__ __device__ __forceinline__ int64_t cut_start(int64_t total, int workers, int w) { return total * w / workers; }
__host__ __device__ __forceinline__ int cut_of(int64_t total, int workers, int64_t x) { return (int)(((x + 1) * workers - 1) / total); }

// workspace: header, first tile of every sequence, partial statistics and outputs (two per worker: the
// range's first unit and its last)
struct StepHeader {
    int64_t total;
    int workers;
};
constexpr size_t kStepHeader = 256;
struct StepSpace {
    StepHeader* head;
    int64_t* base;  // [n_seq]
    float2* stat;   // [2 * kStepMaxWorkers][kStepMaxRows]: maximum (base 2), sum
    float* out;     // [2 * kStepMaxWorkers][kStepMaxRows][dim]
};
__host__ __device__ __forceinline__ size_t step_base_bytes(int n_seq) { return ((size_t)n_seq * 8 + 255) & ~size_t(255); }
__host__ __device__ __forceinline__ StepSpace step_space(void* ws, int n_seq)
{
    unsigned char* w = static_cast<unsigned char*>(ws);
    StepSpace s;
    s.head = reinterpret_cast<StepHeader*>(w);
    s.base = reinterpret_cast<int64_t*>(w + kStepHeader);
    s.stat = reinterpret_cast<float2*>(w + kStepHeader + step_base_bytes(n_seq));
    s.out = reinterpret_cast<float*>(s.stat + 2 * kStepMaxWorkers * kStepMaxRows);
    return s;
}
__host__ __device__ __forceinline__ size_t step_space_bytes(int n_seq, int dim)
{
    return kStepHeader + step_base_bytes(n_seq) + (size_t)2 * kStepMaxWorkers * kStepMaxRows * (8 + (size_t)dim * 4);
}

// ---- 8-bit codes to fp16 ------------------------------------------------------------
// Two codes, bytes LO of y, to a pair of fp16 values.  Both conversions are exact and give finite
// values for every byte, so what lies behind a sequence's end in its last page can do no harm:
//   int8: 1024 + (code + 128) assembled as fp16 bits, less 1152;
//   e4m3: the sign, exponent and mantissa bits moved to their fp16 places, which is the value / 256
//         (subnormals included); the byte pattern of NaN, which no append writes, reads as 480 / 256.
template <bool E4M3, bool HIGH>
__device__ __forceinline__ uint32_t codes2(uint32_t y)
{
    if (E4M3) {
        const uint32_t x = __byte_perm(y, 0u, HIGH ? 0x3424 : 0x1404);
        return ((x >> 1) & 0x3f803f80u) | (x & 0x80008000u);
    }
    const uint32_t x = __byte_perm(y ^ 0x80808080u, 0x64646464u, HIGH ? 0x4342 : 0x4140);
    const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&x), __half2half2(__ushort_as_half((unsigned short)0x6480)));
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool E4M3>
constexpr float kCodeUnit = E4M3 ? 256.0f : 1.0f;  // value of a converted code of 1.0

}  // namespace gdn
