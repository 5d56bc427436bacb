// gdn_kv_attn.cu -- the attention call: its workspace and the order of its kernels.
#include "gdn_kv_attn.cuh"

namespace gdn {
namespace {

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// lays the workspace's parts out from `ws` (NULL: only the size counts)
size_t layout(const KvBatch& b, void* ws, AttnSpace& a)
{
    unsigned char* const base = static_cast<unsigned char*>(ws);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        unsigned char* r = base + at;
        at += up256(bytes);
        return r;
    };
    const size_t dim = b.dim, n = b.n_seq, group = b.hq / b.heads;
    a = AttnSpace{};
    a.head = reinterpret_cast<AttnHeader*>(take(sizeof(AttnHeader)));
    a.step_cut = reinterpret_cast<Cut*>(take(kStepMaxWorkers * sizeof(Cut)));
    a.step_stat = reinterpret_cast<float2*>(take((size_t)2 * kStepMaxWorkers * kStepMaxRows * 8));
    a.step_out = reinterpret_cast<float*>(take((size_t)2 * kStepMaxWorkers * kStepMaxRows * dim * 4));
    a.most_rows = 0x7fffffff;
    const int64_t whole = (int64_t)kWholePositions * (128 / b.dim) * ((int64_t)b.heads * b.n_seq <= kWholeUnits ? 2 : 1);
    a.whole_units = (int64_t)b.max_pages * b.page <= whole;
    // As many long sequences as the batch's tokens allow where every sequence has one at least, each as long as
    // the page table allows.  In a batch with many empty sequences there may be more: those without room for
    // images take the step kernel.  (Counting on empty ones would launch the prompt way's kernels, some 8 us, in
    // every decode step of a large batch.)
    const size_t extra = (size_t)b.T > n ? (size_t)b.T - n : 0, long_seqs = extra / (kLongRows / group);
    const size_t per_seq = ((size_t)b.max_pages * b.page + kKeys - 1) / kKeys;
    const size_t tile_bytes = (size_t)b.heads * 2 * kKeys * dim * 2;
    size_t tiles = (long_seqs < n ? long_seqs : n) * per_seq;
    if (tiles > kImageCap / tile_bytes) tiles = kImageCap / tile_bytes;
    if (tiles == 0) return at;
    a.image_tiles = (int)tiles;
    a.most_rows = kLongRows;
    a.ok = take(n * ok_stride(b.heads));
    a.image_base = reinterpret_cast<int*>(take(n * 4));
    a.units = reinterpret_cast<HeadUnits*>(take(tiles * b.heads * sizeof(HeadUnits)));
    a.prompt_cut = reinterpret_cast<Cut*>(take(kPromptMaxWorkers * sizeof(Cut)));
    a.prompt_stat = reinterpret_cast<float2*>(take((size_t)2 * kPromptMaxWorkers * kUnitRows * 8));
    a.prompt_out = reinterpret_cast<float4*>(take((size_t)2 * kPromptMaxWorkers * kUnitRows * dim * 4));
    a.images = take(tiles * tile_bytes);
    return at;
}

}  // namespace

size_t kv_attn_workspace_bytes(const KvBatch& b)
{
    AttnSpace a;
    return b.T > 0 ? layout(b, nullptr, a) : 0;
}

cudaError_t launch_kv_attn(const AttnParams& p, cudaStream_t stream)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    AttnSpace a;
    layout(p, p.workspace, a);
    if (a.image_tiles > 0 && (e = launch_kv_prompt(p, a, sms, stream)) != cudaSuccess) return e;
    if ((e = launch_kv_step(p, a, sms, stream)) != cudaSuccess) return e;
    return a.whole_units && a.image_tiles == 0 ? cudaSuccess : launch_kv_join(p, a, sms, stream);
}

}  // namespace gdn
