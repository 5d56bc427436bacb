// gdn_kv_copy.cu -- pages copied within the caches of all layers in one launch.
//
// HBM-bound.  A warp moves 4 KB at a time, 8 independent 16-byte loads a lane: 705 MB
// read and written in 110 us, 6.4 TB/s, 94% of what a plain copy reaches (12 layers,
// pages of 128 KB for keys and for values, 112 pairs among 125); 179 MB in 29 us, 6.2 TB/s.
// Lists may be mostly empty (gdn_kv_remap has an entry for every row): each
// block gathers the entries that name two pages, and all warps of the grid share
// the pieces of those pages, layer by layer.
#include <algorithm>

#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kPiece = 4096;      // bytes
constexpr int kVectors = kPiece / 16 / 32;
constexpr int kEntries = 1024;    // list entries looked at together

__global__ void __launch_bounds__(kThreads) kv_copy_kernel(const __grid_constant__ CopyParams p)
{
    __shared__ int2 pair[kEntries];
    __shared__ int found[kThreads / 32];
    pdl_launch_dependents();
    pdl_wait();
    constexpr int kWarps = kThreads / 32, kRounds = kEntries / kThreads;
    const int lane = threadIdx.x & 31, mine = threadIdx.x >> 5;
    const int64_t warp = (int64_t)blockIdx.x * kWarps + mine, warps = (int64_t)gridDim.x * kWarps;
    const int pieces = (int)((p.page_bytes + kPiece - 1) / kPiece), per_pair = p.n_caches * 2 * pieces;
    for (int base = 0; base < p.n; base += kEntries) {
        // the pairs in the list's order: every block has them in the same places
        int2 ab[kRounds];
        uint32_t good[kRounds];
        int count = 0;
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            const int at = base + (mine * kRounds + i) * 32 + lane;
            ab[i] = at < p.n ? make_int2(__ldg(p.from + at), __ldg(p.to + at)) : make_int2(-1, -1);
        }
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            const bool ok = ab[i].x >= 0 && ab[i].x < p.n_pages && ab[i].y >= 0 && ab[i].y < p.n_pages && ab[i].x != ab[i].y;
            good[i] = __ballot_sync(0xffffffffu, ok);
            count += __popc(good[i]);
        }
        if (lane == 0) found[mine] = count;
        __syncthreads();
        int at = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < mine) at += found[w];
            all += found[w];
        }
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            if (good[i] >> lane & 1) pair[at + __popc(good[i] & ((1u << lane) - 1))] = ab[i];
            at += __popc(good[i]);
        }
        __syncthreads();
        const int64_t units = (int64_t)all * per_pair;
        for (int64_t u = warp; u < units; u += warps) {
            const int2 move = pair[u / per_pair];
            const int rest = (int)(u % per_pair), piece = rest % pieces, side = rest / pieces % 2;
            const CopyParams::Cache& c = p.cache[rest / pieces / 2];
            const size_t off = (size_t)piece * kPiece;
            const int vectors = (int)(min((size_t)kPiece, p.page_bytes - off) / 16);
            uint8_t* codes = side ? c.v : c.k;
            const uint4* src = reinterpret_cast<const uint4*>(codes + (size_t)move.x * p.page_bytes + off);
            uint4* dst = reinterpret_cast<uint4*>(codes + (size_t)move.y * p.page_bytes + off);
            uint4 v[kVectors];
#pragma unroll
            for (int i = 0; i < kVectors; ++i)
                if (i * 32 + lane < vectors) v[i] = __ldcs(src + i * 32 + lane);
#pragma unroll
            for (int i = 0; i < kVectors; ++i)
                if (i * 32 + lane < vectors) __stcs(dst + i * 32 + lane, v[i]);
            if (piece == 0) {  // scales as bits: a NaN's say something
                uint32_t* scales = side ? c.v_scale : c.k_scale;
                for (int h = lane; h < p.heads; h += 32) scales[(size_t)move.y * p.heads + h] = scales[(size_t)move.x * p.heads + h];
            }
        }
        __syncthreads();  // pairs read before the next ones are written
    }
}

}  // namespace

cudaError_t launch_kv_copy(const CopyParams& p, cudaStream_t stream)
{
    const int64_t pieces = (int64_t)((p.page_bytes + kPiece - 1) / kPiece) * 2 * p.n_caches * p.n;
    const int64_t blocks = std::min<int64_t>(152 * 6, (pieces + kThreads / 32 - 1) / (kThreads / 32));
    return launch_k(kv_copy_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, stream, true, p);
}

}  // namespace gdn
