// gdn_internal.cuh -- declarations shared by the library's translation units.
// Nothing here is part of the public ABI (include/gdn.h is).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {

constexpr int kHeadDim = 128;  // dk == dv == 128: one head is 32 lanes x 4 channels
constexpr int kChunk = 64;     // tokens per scan chunk

// The scan's [K; Q] operand image of one (chunk slot, key head): 128 rows (the chunk's 64 k rows and
// 64 q rows, k first for chunks at an even index within their sequence, q first for odd ones) x 128
// columns, bf16 split into hi and lo planes, in 16 groups of 8 rows, each group its hi plane (2 KB,
// 16 no-swizzle core matrices along the columns) then its lo plane.  Byte offset of (row r, column k)
// in the hi plane; the lo plane is 2048 bytes behind.  Chunk slots: sequence s owns slots from
// cu[s] / 64 + s on.
constexpr size_t kKqImageBytes = 128 * 128 * 2 * 2;
__host__ __device__ __forceinline__ int kq_off(int r, int k)
{
    return (r >> 3) * 4096 + (k >> 3) * 128 + (r & 7) * 16 + (k & 7) * 2;
}

struct PreParams {
    int hk, hv, C, T, n_seq;
    float eps;
    const int32_t* cu_seqlens;
    const __half* qkv;
    const float* conv_w;
    const __half* hist_in;
    __half* hist_out;
    const __half* a;
    const __half* b;
    const float* A_log;
    const float* dt_bias;
    float* qn;
    float* kn;
    float* vc;
    float* glog;
    float* beta;
    // inside gdn_layer: q and k go straight into the scan's [K; Q] images (qn and kn unused); the
    // images of slot `slot`, key head j start at kq_images + (slot * hk + j) * kKqImageBytes
    unsigned char* kq_images;
    int hist_in_place;  // hist_out == hist_in: the history is written by a second launch after the conv
};

struct ScanParams {
    int hk, hv, T, n_seq;
    const int32_t* cu_seqlens;
    const float* qn;
    const float* kn;
    const float* vc;
    const float* glog;
    const float* beta;
    const float* S_in;
    float* S_out;
    float* o;
    void* workspace;
    size_t workspace_bytes;
    int withhold_first_copy;  // failure-report self-test only (gdn_scan_selftest_timeout)
    int prep_no_keepers;      // prep fallback self-test only (gdn_scan_selftest_one_taker)
    int withhold_flag;        // cross-kernel wait self-test only (gdn_scan_selftest_withhold_flag)
    int fast;                 // one-pass bf16 products (gdn_scan_fast / gdn_layer_fast)
    int prep_sms, prep_keep;  // SMs of the device; SMs whose prep CTAs stay after round one (set by launch_scan)
    int kq_written;           // the pre kernel wrote the [K; Q] images (qn and kn unused; gdn_layer)
};

struct PostParams {
    int hv, T;
    float eps;
    const float* o;
    const __half* z;
    const float* gamma;
    int out_f32;
    void* y;
};

// one decode step: one token per sequence, the three stages fused
struct StepParams {
    int hk, hv, C, n_seq;
    float eps;
    const __half* qkv;      // [n_seq][C]
    const float* conv_w;    // [C][4]
    const __half* hist_in;  // [n_seq][C][3]
    __half* hist_out;
    const __half* a;        // [n_seq][hv]
    const __half* b;
    const __half* z;        // [n_seq][hv][dv]
    const float* A_log;
    const float* dt_bias;
    const float* gamma;
    const float* S_in;      // [n_seq][hv][dk][dv]
    float* S_out;
    int out_f32;
    void* y;                // [n_seq][hv][dv]
};

// one layer's paged 8-bit cache and the batch that appends to it or reads it
struct KvBatch {
    int heads, dim, page, n_pages, format;  // page: tokens per page, a power of two
    uint8_t* k;
    uint8_t* v;
    float* k_scale;
    float* v_scale;
    int n_seq, T, hq, max_pages;
    const int32_t* cu_seqlens;
    const int32_t* past;
    const int32_t* table;
    int64_t table_stride;
    const uint16_t* q;
    int64_t q_stride;
    int bf16;  // activations: bf16, else fp16
};

struct AppendParams : KvBatch {
    const uint16_t* k_new;
    const uint16_t* v_new;
    int64_t k_stride, v_stride;
    const float* cos;
    const float* sin;
    int rot, n_pos, interleaved;
    uint16_t* q_out;
};

struct AttnParams : KvBatch {
    float scale;
    uint16_t* y;
    void* workspace;
};

struct VerifyParams {
    int n_seq, max_draft, vocab;
    const float* p;
    const float* q;
    int64_t p_stride, q_stride;
    const int32_t* draft;
    const int32_t* n_draft;
    const float* u;
    int32_t* accepted;
    int32_t* next;
};

// the residual stream between two blocks
struct BlockNormParams {
    int T, width;
    int x32, bf16;  // the stream in fp32; activations (and a 16-bit stream) in bf16, else fp16
    const void* x;
    int64_t x_stride;
    const uint16_t* y;  // nullptr: h from x alone
    int64_t y_stride;
    const uint16_t* gate;
    int64_t gate_stride;
    int gate_kind;
    float scale, eps;
    const float* post_weight;
    const float* pre_weight;
    void* x_out;   // nullptr: not wanted
    uint16_t* h;   // nullptr: not wanted
};

// the next step's page table from the last one's
struct RemapParams {
    int n_old, n_rows, max_pages, page_shift, n_pages;
    const int32_t* table;
    int64_t table_stride, out_stride;
    const int32_t* parent;
    const int32_t* keep;
    const int32_t* need;
    int32_t* table_out;
    int32_t* copy_from;
    int32_t* copy_to;
    int32_t* info;
    // workspace: the free pages' number; per page, who names it; the free pages; per row, its place among them
    int32_t* header;
    int32_t* owner;
    int32_t* free_list;
    int32_t* first;
    int32_t* sums;  // [remap_sums]
};

// pages renamed to the front of the pool
struct CompactParams {
    int n_rows, max_pages, n_pages;
    const int32_t* table;
    int64_t table_stride, out_stride;
    int32_t* table_out;
    int32_t* copy_from;  // [n_pages / 2]
    int32_t* copy_to;
    int32_t* info;
    int32_t* name;  // workspace: per page, its new number
    int32_t* sums;  // workspace: [compact_sums]
};

constexpr int kCopyCaches = 64;  // caches of one launch

struct CopyParams {
    struct Cache {
        uint8_t* k;
        uint8_t* v;
        uint32_t* k_scale;
        uint32_t* v_scale;
    };
    int n_caches, n, n_pages, heads;
    size_t page_bytes;  // of k, and of v
    const int32_t* from;
    const int32_t* to;
    Cache cache[kCopyCaches];
};

// words of the workspace for the counts of a large batch's blocks
size_t remap_sums(int n_pages, int n_rows);
size_t compact_sums(int n_pages);
cudaError_t launch_kv_remap(const RemapParams& p, cudaStream_t stream);
cudaError_t launch_kv_compact(const CompactParams& p, cudaStream_t stream);
cudaError_t launch_kv_copy(const CopyParams& p, cudaStream_t stream);

constexpr int kAdapterCtas = 152;

// where a CTA's range of units begins: a sequence (n_seq: no work), its tile, the cost of all units in front of that
// tile; the cost of a range (in the first CTA's)
struct AdapterStart {
    int64_t before, share;
    int s, k;
};

// the sequences' adapters added to a shared projection's output
struct AdapterParams {
    int n_seq, T, n_adapters, rank, d_in, d_out, bf16;
    const int32_t* cu_seqlens;
    const int32_t* ids;
    const int32_t* ranks;   // nullptr: all `rank`
    const uint16_t* down;   // [n_adapters][rank][d_in]
    const uint16_t* up;     // [n_adapters][rank][d_out]
    const float* scales;
    const uint16_t* x;
    const uint16_t* y;
    uint16_t* y_out;
    int64_t x_stride, y_stride, out_stride;
    int few;                    // tokens up to which a tile is not the tensor cores' (set by launch_adapter)
    int chunks_in, chunks_out, parts_in;  // units of a tile; ranges that one is cut into (set by launch_adapter)
    // workspace (set by launch_adapter): a word for each CTA of either kernel, 0 or a wait that has expired; per CTA, where
    // its range of y's units begins; per tile, the first and the last range of x's units that it lies in;
    // h [T + ranges * 128][rank]: what the range that a tile begins in summed, then what each of the others did (a tile's
    // tokens change places with its rank; the few tokens' do not)
    int32_t* status;
    AdapterStart* starts;
    int2* parts;
    float* h;
};

// lays the workspace out (p: n_seq, T, rank) and returns its bytes
size_t adapter_workspace(AdapterParams& p, void* workspace);
cudaError_t launch_adapter(AdapterParams p, void* workspace, cudaStream_t stream);
cudaError_t launch_block_norm(const BlockNormParams& p, cudaStream_t stream);
cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t stream);
size_t kv_attn_workspace_bytes(const KvBatch& b);
cudaError_t launch_kv_attn(const AttnParams& p, cudaStream_t stream);
cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream);

cudaError_t launch_pre(const PreParams& p, cudaStream_t stream);
cudaError_t launch_step(const StepParams& p, cudaStream_t stream);
size_t scan_workspace_bytes(int hk, int hv, int n_seq, int T);
size_t scan_kq_images_offset(int hk, int hv, int n_seq, int T);  // byte offset of the [K; Q] images in the workspace
cudaError_t launch_scan(const ScanParams& p, cudaStream_t stream);
cudaError_t launch_post(const PostParams& p, cudaStream_t stream);

// record the detail string returned by gdn_last_error_string on this thread
void set_last_error(const char* msg);

// ---- programmatic dependent launch ---------------------------------------------
// Kernels launched with launch_k(..., pdl = true) may start while the previous
// kernel on the stream is still draining.  Every block of every kernel calls
// pdl_wait() before its first read of global memory (a no-op when launched
// without the attribute), whoever wrote what it reads: only the grid that waits is
// promised to see earlier writes.  (scan_chain_kernel takes each chunk by its flag
// instead, and waits at its end.)  pdl_launch_dependents() comes early, which lets the
// next kernel's CTAs be scheduled once every CTA of this one has started.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... KArgs, typename... Args>
cudaError_t launch_k(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, bool pdl,
                     Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl ? attr : nullptr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- small device helpers ---------------------------------------------------
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// cu_seqlens[s] clamped into [0, T]: a malformed offsets array gives wrong
// results, never an out-of-bounds access
__device__ __forceinline__ int cu_at(const int32_t* cu, int s, int T)
{
    return min(max(__ldg(cu + s), 0), T);
}

__device__ __forceinline__ float sigmoidf_(float x) { return 1.0f / (1.0f + expf(-x)); }

__device__ __forceinline__ float siluf_(float x) { return x / (1.0f + expf(-x)); }

// SiLU with the fast exponential and reciprocal intrinsics (a few ulp; for
// x -> -inf the reciprocal of inf is 0, so the result goes to -0 cleanly)
__device__ __forceinline__ float silu_fast(float x) { return x * __fdividef(1.0f, 1.0f + __expf(-x)); }

}  // namespace gdn
