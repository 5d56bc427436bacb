// gdn_kv_join.cu -- the attention's last kernel: joins the parts of the units that the
// workers' ranges have cut.
//
// Mathematics.  A part is (m, l, o) over some of a row's keys, l = sum 2^(x - m) and o = sum 2^(x - m) v;
// the row's output is sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i with M the largest m_i.  Parts are taken in the
// order of their ranges, so the result does not depend on which finished first.
//
// Bound.  Latency: the parts (at most two a worker) were just written and lie in the second-level cache.  A
// decode step of 64 sequences spends 3 us here (5.4 where each block first listed all cut units).
#include "gdn_kv_attn.cuh"

namespace gdn {
namespace {

constexpr int kJoinThreads = 256;

// Of range w and 32 rows: where the range is the first that begins inside a unit, joins that unit's parts.
// Eight threads share a row's channels.
template <int D, bool BF16>
__device__ __forceinline__ void join_prompt(const AttnParams& p, const AttnSpace& a, int w, int eighth)
{
    const int group = p.hq / p.heads, tokens = half_tokens(group);
    const int workers = a.head->prompt_workers;
    if (w >= workers || a.head->prompt_whole) return;
    const Cut cut = a.prompt_cut[w];
    const int64_t total = a.head->prompt_total, begin = cut.lo - cut.from, prev = a.prompt_cut[w - 1].lo;
    if (cut.j0 == 0 || prev > begin + kPromptUnitCost || !images_there(p, a, cut.s)) return;
    const int last = cut_of(total, workers, begin + kPromptUnitCost + cut.tiles - 1);
    const int row = eighth * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
    const int h = row >> 7, r = row & 127, i_tok = r / group, qh = r - i_tok * group;
    const int t0 = cu_at(p.cu_seqlens, cut.s, p.T), n = cu_at(p.cu_seqlens, cut.s + 1, p.T) - t0;
    const int tok = (2 * cut.unit + h) * tokens + i_tok;
    if (i_tok >= tokens || tok >= n) return;
    constexpr int E = D / 32;  // float4s a thread
    float top = -INFINITY, sum = 0.0f;
    float4 acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
    for (int i = w - 1; i <= last; ++i) {
        const int slot = 2 * i + (i == w - 1 && prev < begin ? 1 : 0);
        const float2 st = a.prompt_stat[(size_t)slot * kUnitRows + row];
        const float next = fmaxf(top, st.x), ref = next == -INFINITY ? 0.0f : next;
        const float f0 = ex2(top - ref), f1 = ex2(st.x - ref);
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
    const float inv = 1.0f / sum;  // (0: every score is -infinity, and 0 x inv NaN)
    uint2* dst = reinterpret_cast<uint2*>(p.y + ((int64_t)(t0 + tok) * p.hq + cut.head * group + qh) * D) + part * E;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[e] = make_uint2(narrow2<BF16>(acc[e].x * inv, acc[e].y * inv), narrow2<BF16>(acc[e].z * inv, acc[e].w * inv));
}

// Of range w and a slice of the rows: where the range is the first that begins inside a unit, joins that
// unit's parts.  The fewer rows there are, the more warps share a row's parts.
template <int D, bool BF16>
__device__ __forceinline__ void join_steps(const AttnParams& p, const AttnSpace& a, int w, int row_lo, int row_hi)
{
    constexpr int E = D / 32, W = kJoinThreads / 32;
    __shared__ float part[W][D], part_l[W], part_m[W];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = p.hq / p.heads;
    const int workers = a.head->step_workers;
    const int64_t total = a.head->step_total, prev = a.step_cut[w - 1].lo;
    const Cut cut = a.step_cut[w];  // (past the workers: not used)
    const int64_t begin = cut.lo - cut.from;
    row_hi = min(row_hi, cut.n * group - cut.unit);
    if (w >= workers || cut.j0 == 0 || prev > begin + kStepUnitCost || row_lo >= row_hi) return;
    // the unit is the first of every range but the one that it begins in the middle of
    const int first_slot = 2 * (w - 1) + (prev < begin ? 1 : 0), last = cut_of(total, workers, begin + kStepUnitCost + cut.tiles - 1);
    int share = 1;  // warps a row
    while (2 * share * (row_hi - row_lo) <= W) share *= 2;
    for (int k0 = row_lo; k0 < row_hi; k0 += W / share) {
        const int row = k0 + warp / share, in_row = warp % share;
        const bool mine = row < row_hi;
        float top = -INFINITY, sum = 0.0f, acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.0f;
        if (mine)
#pragma unroll 4
            for (int i = w - 1 + in_row; i <= last; i += share) {
                const int slot = i == w - 1 ? first_slot : 2 * i;
                const float2 st = a.step_stat[(size_t)slot * kStepMaxRows + row];
                const float* src = a.step_out + ((size_t)slot * kStepMaxRows + row) * D + lane * E;
                const float next = fmaxf(top, st.x), ref = next == -INFINITY ? 0.0f : next;
                const float f0 = ex2(top - ref), f1 = ex2(st.x - ref);
                sum = sum * f0 + st.y * f1;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = acc[e] * f0 + src[e] * f1;
                top = next;
            }
        if (share > 1) {  // uniform over the block
            __syncthreads();  // the last round's parts are read
#pragma unroll
            for (int e = 0; e < E; ++e) part[warp][lane * E + e] = acc[e];
            if (lane == 0) {
                part_m[warp] = top;
                part_l[warp] = sum;
            }
            __syncthreads();
            if (in_row == 0) {
                float m = top;
                for (int i = 1; i < share; ++i) m = fmaxf(m, part_m[warp + i]);
                const float ref = m == -INFINITY ? 0.0f : m, f0 = ex2(top - ref);
                sum *= f0;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] *= f0;
                for (int i = 1; i < share; ++i) {
                    const float f = ex2(part_m[warp + i] - ref);
                    sum += f * part_l[warp + i];
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] += f * part[warp + i][lane * E + e];
                }
            }
        }
        if (!mine || in_row != 0) continue;
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const int i = (cut.unit + row) / group, qh = cut.unit + row - i * group;
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.y + ((int64_t)(cut.t0 + i) * p.hq + cut.head * group + qh) * D + lane * E);
#pragma unroll
        for (int e = 0; e < E; e += 2) dst[e / 2] = narrow2<BF16>(acc[e] * inv, acc[e + 1] * inv);
    }
}

// the first blocks join the step kernel's parts (`slices` of them a range), the others the prompt kernel's
// (eight a range)
template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads, 4) kv_join_kernel(AttnParams p, AttnSpace a, int step_blocks, int slices, int slice_rows)
{
    pdl_wait();
    pdl_launch_dependents();
    const int block = blockIdx.x;
    if (block < step_blocks) {
        const int slice = block % slices;
        join_steps<D, BF16>(p, a, 1 + block / slices, slice * slice_rows, (slice + 1) * slice_rows);
    } else {
        join_prompt<D, BF16>(p, a, 1 + (block - step_blocks) / 8, (block - step_blocks) & 7);
    }
}

}  // namespace

cudaError_t launch_kv_join(const AttnParams& p, const AttnSpace& a, int sms, cudaStream_t stream)
{
    // Few (sequence, kv head) pairs are cut into many parts each: four blocks share a unit's rows (the whole call
    // for one sequence of 4000 positions, 8 heads, 11.2 us, by one block 13.3; 3 of 131000 46.7 and 48.1).  With many
    // pairs the blocks that find nothing cost more (64 sequences, 4 heads, 69.1 us by four, 65.8 by one).
    constexpr int kFewPairs = 32;
    const int rows = step_rows(p, a), slices = (int64_t)p.n_seq * p.heads <= kFewPairs ? 4 : 1;
    const int step_blocks = a.whole_units ? 0 : slices * (step_grid(sms, rows) - 1);
    const dim3 grid(step_blocks + (a.image_tiles > 0 ? 8 * (prompt_grid(sms) - 1) : 0)), block(kJoinThreads);
    auto launch = [&](auto kernel) { return launch_k(kernel, grid, block, 0, stream, true, p, a, step_blocks, slices, rows / slices); };
    if (p.dim == 64) return p.bf16 ? launch(kv_join_kernel<64, true>) : launch(kv_join_kernel<64, false>);
    return p.bf16 ? launch(kv_join_kernel<128, true>) : launch(kv_join_kernel<128, false>);
}

}  // namespace gdn
