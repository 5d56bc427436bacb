// gdn_verify.cu -- the check of drafted tokens against the target's probabilities.
//
// Mathematics.  Leading drafts are accepted while u q(x) < p(x); the token after them is drawn from
// the normalised positive part of p - q (from p after the last draft) by inverting its running sum at
// u W.  Weights are whole multiples of 2^-43 of a probability, so their sums are exact in 64 bits and
// do not depend on the order in which threads form them: the drawn index is the one that a sequential
// sum would give.  At most 2^19 weights of at most 2^43 stay below 2^63.
//
// Layout.  The call reads one row of p and one of q per sequence, once: HBM-bound for large batches and
// bound by latency for one sequence.  A cluster of 8 CTAs shares a sequence (one CTA per sequence
// would leave most SMs idle in small batches); each sums its part of the row in segments of 512
// weights, the CTAs exchange their totals through distributed shared memory, and the one CTA whose part
// holds the threshold finds its segment from the sums and reads those 512 weights again.  CTAs of 256
// threads: five share an SM, so that one's search for the first rejected draft and its exchange run under
// the others' loads (512 threads: 63 us where 256 take 47).
//
// Measured: 256 sequences of 131072 weights, 220 MB that no cache holds, 47 us, 4.7 TB/s (the floor is 39.5 us
// for what the call must read); one sequence 5.8 us: four dependent loads, two exchanges and the launch.
#include <cooperative_groups.h>

#include "gdn_internal.cuh"

namespace gdn {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCtas = 8;          // CTAs a sequence (the portable cluster size)
constexpr int kSegment = 512;     // weights a segment: 16 a lane
constexpr int kMaxSegments = ((1 << 19) / kCtas + kSegment - 1) / kSegment;

// floor(x 2^43) for x in [0, 1], from the number's bits: its 24-bit mantissa times or over a power of
// two (one 32 x 32 -> 64 multiply-add to a sum; a float-to-64-bit conversion runs at a fraction of that
// rate).  Below 2^-126 the mantissa's hidden bit is wrong, and shifted out.
__device__ __forceinline__ uint64_t weight(float x)
{
    const uint32_t bits = __float_as_uint(x), mantissa = (bits & 0x7fffffu) | 0x800000u;
    const int up = (int)(bits >> 23) - 107;  // 2^43 / 2^23 against the exponent's bias of 127
    return (uint64_t)(mantissa >> min(max(-up, 0), 31)) * (1u << max(up, 0));
}

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

struct Row {
    const float* p;
    const float* q;  // NULL: the weights are p's alone
    bool vec;        // both rows 16-byte aligned
    __device__ __forceinline__ uint64_t one(int i) const
    {
        return weight(__saturatef(__fsub_rn(__ldg(p + i), q ? __ldg(q + i) : 0.0f)));  // NaN saturates to 0
    }
    // the sum of a segment's weights from i on (0 from `end` on); a lane's own share of it
    __device__ __forceinline__ uint64_t share(int i, int end, int lane) const
    {
        uint64_t sum = 0;
        if (i + kSegment > end) {
            for (int k = i + lane; k < end; k += 32) sum += one(k);
        } else if (vec) {
            float4 a[kSegment / 128], b[kSegment / 128];
#pragma unroll
            for (int j = 0; j < kSegment / 128; ++j) {
                a[j] = __ldcs(reinterpret_cast<const float4*>(p + i + j * 128) + lane);
                b[j] = q ? __ldcs(reinterpret_cast<const float4*>(q + i + j * 128) + lane) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
            for (int j = 0; j < kSegment / 128; ++j)
                sum += (weight(__saturatef(__fsub_rn(a[j].x, b[j].x))) + weight(__saturatef(__fsub_rn(a[j].y, b[j].y)))) +
                       (weight(__saturatef(__fsub_rn(a[j].z, b[j].z))) + weight(__saturatef(__fsub_rn(a[j].w, b[j].w))));
        } else {
            float a[kSegment / 32], b[kSegment / 32];
#pragma unroll
            for (int j = 0; j < kSegment / 32; ++j) {
                a[j] = __ldcs(p + i + j * 32 + lane);
                b[j] = q ? __ldcs(q + i + j * 32 + lane) : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < kSegment / 32; ++j) sum += weight(__saturatef(__fsub_rn(a[j], b[j])));
        }
        return sum;
    }
};

struct Shared {
    uint64_t seg[kMaxSegments];
    uint64_t total;
    int accepted;
};

__global__ void __launch_bounds__(kThreads) __cluster_dims__(kCtas, 1, 1) verify_kernel(VerifyParams p)
{
    __shared__ Shared sm;
    cg::cluster_group cluster = cg::this_cluster();
    pdl_wait();
    pdl_launch_dependents();
    const int s = blockIdx.y, rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int count = p.n_draft ? min(max(__ldg(p.n_draft + s), 0), p.max_draft) : p.max_draft;
    const float* const u = p.u + (size_t)s * (p.max_draft + 1);
    const float* const p0 = p.p + (size_t)s * (p.max_draft + 1) * p.p_stride;
    const float* const q0 = p.q + (size_t)s * p.max_draft * p.q_stride;
    if (warp == 0) {  // every CTA finds the first draft that is not accepted, 32 drafts at a time
        // (a draft, its random number and the count are loaded together; then the two probabilities)
        int accepted = p.max_draft;
        for (int i0 = 0; i0 < p.max_draft; i0 += 32) {
            const int i = i0 + lane;
            bool ok = true;
            if (i < p.max_draft) {
                const int x = __ldg(p.draft + (size_t)s * p.max_draft + i);
                const float r = __ldg(u + i);
                const bool there = x >= 0 && x < p.vocab;
                const size_t at = there ? x : 0;
                ok = there && __fmul_rn(r, __ldg(q0 + (size_t)i * p.q_stride + at)) < __ldg(p0 + (size_t)i * p.p_stride + at);
            }
            const uint32_t bad = __ballot_sync(0xffffffffu, !ok);
            if (bad) {
                accepted = i0 + __ffs(bad) - 1;
                break;
            }
        }
        accepted = min(accepted, count);
        if (lane == 0) sm.accepted = accepted;
    }
    __syncthreads();
    const int accepted = sm.accepted;
    Row row;
    row.p = p0 + (size_t)accepted * p.p_stride;
    row.q = accepted < count ? q0 + (size_t)accepted * p.q_stride : nullptr;
    // this CTA's part of the vocabulary, a whole number of segments
    const int per = ((p.vocab + kCtas * kSegment - 1) / (kCtas * kSegment)) * kSegment;
    const int lo = min(rank * per, p.vocab), hi = min(lo + per, p.vocab), segments = (hi - lo + kSegment - 1) / kSegment;
    int token = -1;
    uint64_t before = 0, total = 0;
    for (int pass = 0; pass < 2; ++pass) {  // the second one where the residual has no mass: p itself
        row.vec = ((reinterpret_cast<uintptr_t>(row.p) | reinterpret_cast<uintptr_t>(row.q)) & 15u) == 0;
        for (int g = warp; g < segments; g += kWarps) {
            const uint64_t sum = warp_sum64(row.share(lo + g * kSegment, hi, lane));
            if (lane == 0) sm.seg[g] = sum;
        }
        __syncthreads();
        if (warp == 0) {
            uint64_t sum = 0;
            for (int g = lane; g < segments; g += 32) sum += sm.seg[g];
            sum = warp_sum64(sum);
            if (lane == 0) sm.total = sum;
        }
        cluster.sync();
        before = total = 0;
        for (int r = 0; r < kCtas; ++r) {
            const uint64_t t = *cluster.map_shared_rank(&sm.total, r);
            if (r < rank) before += t;
            total += t;
        }
        cluster.sync();  // totals read before they are written again, or their CTA leaves
        if (total != 0 || row.q == nullptr) break;
        row.q = nullptr;
    }
    if (tid == 0 && rank == 0) p.accepted[s] = accepted;
    if (total == 0) {
        if (tid == 0 && rank == 0) p.next[s] = -1;
        return;
    }
    // u outside [0, 1] or NaN counts as the nearest of 0 and 1
    const double x = __dmul_rn((double)fminf(fmaxf(__ldg(u + p.max_draft), 0.0f), 1.0f), __ull2double_rn(total));
    const uint64_t limit = min((uint64_t)__double2ull_rd(x), total - 1);
    if (warp != 0 || limit < before || limit >= before + sm.total) return;
    // the first segment whose running sum exceeds the limit, then the first weight in it
    uint64_t run = before;
    int g0 = 0;
    for (;; g0 += 32) {
        const uint64_t v = g0 + lane < segments ? sm.seg[g0 + lane] : 0;
        uint64_t incl = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint64_t o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        const uint32_t over = __ballot_sync(0xffffffffu, run + incl > limit);
        if (over || g0 + 32 >= segments) {
            const int f = over ? __ffs(over) - 1 : 31;
            run += __shfl_sync(0xffffffffu, incl - v, f);
            g0 += f;
            break;
        }
        run += __shfl_sync(0xffffffffu, incl, 31);
    }
    for (int j = 0; j < kSegment / 128; ++j) {
        const int i = lo + g0 * kSegment + j * 128 + lane * 4;
        uint64_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = i + e < hi ? row.one(i + e) : 0;
        uint64_t incl = (w[0] + w[1]) + (w[2] + w[3]);
        const uint64_t v = incl;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint64_t o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        const uint32_t over = __ballot_sync(0xffffffffu, run + incl > limit);
        if (over) {
            if (lane == __ffs(over) - 1) {
                uint64_t at = run + incl - v;
                int e = 0;
                while (e < 3 && (at += w[e]) <= limit) ++e;
                token = i + e;
                p.next[s] = token;
            }
            return;
        }
        run += __shfl_sync(0xffffffffu, incl, 31);
    }
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream)
{
    return launch_k(verify_kernel, dim3(kCtas, (unsigned)p.n_seq), dim3(kThreads), 0, stream, true, p);
}

}  // namespace gdn
