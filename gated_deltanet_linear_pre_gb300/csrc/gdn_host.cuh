// gdn_host.cuh -- host-side helpers of the ABI's translation units: status and
// error reporting, argument checks.  Defined in gdn_api.cu.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {
namespace host {

// record the detail string of this host thread's last error and return s
gdn_status fail(gdn_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// GDN_ERR_CUDA with the runtime's text; an error that spoils the context is kept for gdn_last_async_error
gdn_status cuda_fail(cudaError_t e, const char* what);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Buf {
    const void* p;
    size_t bytes;
    const char* name;
};

gdn_status check_batch(int32_t n_seq, int32_t T, const int32_t* cu);
// every non-empty buffer present and 16-byte aligned
gdn_status check_bufs(const Buf* b, int n);
bool overlap(const Buf& a, const Buf& b);
// no output may overlap another output or any input
gdn_status check_disjoint(const Buf* outs, int n_out, const Buf* ins, int n_in);

// T token rows of `row` elements, `stride` apart, read in 16-byte pieces
gdn_status check_stride(const char* name, int64_t stride, size_t row, int32_t T);
// bytes from the first element of a strided [T][row] array to its last
inline size_t span(int32_t T, int64_t stride, size_t row, size_t element)
{
    return T > 0 ? ((size_t)(T - 1) * (size_t)stride + row) * element : 0;
}

// a workspace's failure record, its first 4 bytes (synchronises the stream)
gdn_status read_failure_word(const void* word, struct CUstream_st* stream);

}  // namespace host
}  // namespace gdn
