// gdn_kv_join.cu -- the attention's last kernel: joins the parts of the units that the
// workers' ranges have cut.
//
// Mathematics.  A part is (m, l, o) over some of a row's keys, l = sum 2^(x - m) and o = sum 2^(x - m) v;
// the row's output is sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i with M the largest m_i.  Parts are taken in the
// order of their ranges, so the result does not depend on which finished first.
//
// Bound.  Latency: the parts (at most two a worker) were just written and lie in the second-level cache.  A
// decode step of 64 sequences spends 9.5 us here on cold caches, about half of that in sequence.
#include "gdn_kv_attn.cuh"

namespace gdn {
namespace {

constexpr int kJoinThreads = 512;

// Of range w and 64 rows: where the range is the first that begins inside a unit, joins that unit's parts.
// Eight threads share a row's channels.
template <int D, bool BF16>
__device__ __forceinline__ void join_prompt(const AttnParams& p, const AttnSpace& a, int w, int quarter)
{
    const int group = p.hq / p.heads, tokens = half_tokens(group);
    const int workers = a.head->prompt_workers;
    if (w >= workers || a.head->prompt_whole) return;
    const Cut cut = a.prompt_cut[w];
    const int64_t total = a.head->prompt_total, begin = cut.lo - cut.from, prev = a.prompt_cut[w - 1].lo;
    if (cut.j0 == 0 || prev > begin + kPromptUnitCost || !a.ok[cut.s]) return;
    const int last = cut_of(total, workers, begin + kPromptUnitCost + cut.tiles - 1);
    const int row = quarter * 64 + (threadIdx.x & 63), part = threadIdx.x >> 6;
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
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint2* dst = reinterpret_cast<uint2*>(p.y + ((int64_t)(t0 + tok) * p.hq + cut.head * group + qh) * D) + part * E;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[e] = make_uint2(narrow2<BF16>(acc[e].x * inv, acc[e].y * inv), narrow2<BF16>(acc[e].z * inv, acc[e].w * inv));
}

// Joins the parts of the units that the ranges cut, in the order of the ranges.  Every block lists the cut
// units (where a range is the first that begins inside a unit's tiles) and takes its share of their rows;
// the fewer rows there are (one long sequence: few rows of many parts), the more warps share a row's parts.
template <int D, bool BF16>
__device__ __forceinline__ void join_steps(const AttnParams& p, const AttnSpace& a, int R, int block, int blocks)
{
    constexpr int E = D / 32, W = kJoinThreads / 32;
    struct Joint {
        int s, head, unit;
        int from, last, slot;  // its first and last range, the slot of the first part
    };
    __shared__ Joint joints[kStepMaxWorkers];
    __shared__ int counts[W];
    __shared__ float part[W][D], part_l[W], part_m[W];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, group = p.hq / p.heads;
    const int workers = a.head->step_workers;
    const int64_t total = a.head->step_total;
    int n = 0;
    for (int w0 = 1; w0 < workers; w0 += kJoinThreads) {
        const int w = w0 + tid;
        Cut cut{};
        int64_t begin = 0, prev = 0;
        bool is_first = false;
        if (w < workers) {
            cut = a.step_cut[w];
            begin = cut.lo - cut.from;
            prev = a.step_cut[w - 1].lo;
            is_first = cut.j0 > 0 && prev <= begin + kStepUnitCost;
        }
        const uint32_t vote = __ballot_sync(0xffffffffu, is_first);
        if (lane == 0) counts[warp] = __popc(vote);
        __syncthreads();
        int at = n + __popc(vote & ((1u << lane) - 1u));
        for (int i = 0; i < W; ++i) {
            if (i < warp) at += counts[i];
            n += counts[i];
        }
        if (is_first)
            // the unit is the first of every range but the one that it begins in the middle of
            joints[at] = Joint{cut.s, cut.head, cut.unit, w - 1, cut_of(total, workers, begin + kStepUnitCost + cut.tiles - 1),
                               2 * (w - 1) + (prev < begin ? 1 : 0)};
        __syncthreads();
    }
    const int items = n * R, per_block = (items + blocks - 1) / blocks;
    int share = W;  // warps a row
    while (share > 1 && share * per_block > W) share >>= 1;
    for (int k0 = block * per_block; k0 < min((block + 1) * per_block, items); k0 += W / share) {
        const int k = k0 + warp / share, in_row = warp % share;
        bool mine = k < min((block + 1) * per_block, items);
        const Joint u = joints[mine ? k / R : 0];
        const int row = k % R, t0 = cu_at(p.cu_seqlens, u.s, p.T);
        mine = mine && u.unit + row < (cu_at(p.cu_seqlens, u.s + 1, p.T) - t0) * group;
        float top = -INFINITY, sum = 0.0f, acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.0f;
        if (mine)
#pragma unroll 4
            for (int i = u.from + in_row; i <= u.last; i += share) {
                const int slot = i == u.from ? u.slot : 2 * i;
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
        const int i = (u.unit + row) / group, qh = u.unit + row - i * group;
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.y + ((int64_t)(t0 + i) * p.hq + u.head * group + qh) * D + lane * E);
#pragma unroll
        for (int e = 0; e < E; e += 2) dst[e / 2] = narrow2<BF16>(acc[e] * inv, acc[e + 1] * inv);
    }
}

// the first blocks join the step kernel's parts, the others the prompt kernel's (four blocks a range)
template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads, 2) kv_join_kernel(AttnParams p, AttnSpace a, int step_blocks, int step_rows)
{
    pdl_wait();
    pdl_launch_dependents();
    const int block = blockIdx.x;
    if (block < step_blocks) join_steps<D, BF16>(p, a, step_rows, block, step_blocks);
    else join_prompt<D, BF16>(p, a, 1 + (block - step_blocks) / 4, (block - step_blocks) & 3);
}

}  // namespace

cudaError_t launch_kv_join(const AttnParams& p, const AttnSpace& a, int sms, cudaStream_t stream)
{
    const int step_blocks = 2 * sms, rows = step_rows(p, a);
    const dim3 grid(step_blocks + (a.image_tiles > 0 ? 4 * (prompt_grid(sms) - 1) : 0)), block(kJoinThreads);
    if (p.dim == 64)
        return p.bf16 ? launch_k(kv_join_kernel<64, true>, grid, block, 0, stream, true, p, a, step_blocks, rows)
                      : launch_k(kv_join_kernel<64, false>, grid, block, 0, stream, true, p, a, step_blocks, rows);
    return p.bf16 ? launch_k(kv_join_kernel<128, true>, grid, block, 0, stream, true, p, a, step_blocks, rows)
                  : launch_k(kv_join_kernel<128, false>, grid, block, 0, stream, true, p, a, step_blocks, rows);
}

}  // namespace gdn
