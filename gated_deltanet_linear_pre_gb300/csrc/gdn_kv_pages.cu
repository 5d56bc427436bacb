// gdn_kv_pages.cu -- which pages a batch's sequences hold: the table of the next
// step from that of the last (gdn_kv_remap), pages renamed to the front of the
// pool (gdn_kv_compact).  Whole numbers only; no result depends on an order of
// threads.
//
// Both go through the same four phases over a word for every page of the pool:
//   clear  no page has a word
//   mark   every table entry leaves its word at its page (scattered stores, or a
//          minimum where rows compete for a page)
//   scan   running counts over the pages (and, for remap, over the rows)
//   fill   the new table, entry by entry
// A small batch's phases run in one launch of one cluster, whose CTAs exchange
// their counts: what bounds it is the chain of loads and barriers.  A large one's
// run in a launch each over the whole GPU, the scan in two: every block's count,
// then each block adds up those in front of it.  500 rows of 2048 entries over
// 914k pages take 31 us (90 with the scan by one cluster of 8).
#include <cooperative_groups.h>

#include <algorithm>

#include "gdn_internal.cuh"

namespace cg = cooperative_groups;

namespace gdn {
namespace {

constexpr int kThreads = 1024;
constexpr int kCluster = 8;
constexpr int kNone = 0x7fffffff;  // a page that no entry names
constexpr int kReader = -1;        // a page that some row reads on
constexpr int kSegment = 256;      // table entries a warp takes at a time
constexpr int kPer = kSegment / 32;
// Table entries and pages from which on each phase is a launch of its own.  256 rows of 128 entries take 13.0 us in one
// launch and 10.0 in five, 512 of 512 32 and 14 (replayed); a call from Python 29 and 40, 34 and 39.
constexpr int64_t kOneLaunch = 1 << 17;

struct Phases {
    static constexpr int kClear = 0, kMark = 1, kFill = 2;
};
constexpr int kBlockPages = kThreads * 4;  // of a large scan's block; of rows, kThreads

// this CTA's place among those that share a phase's work
struct Share {
    int part, parts;
    __device__ int64_t warp() const { return (int64_t)part * (blockDim.x >> 5) + (threadIdx.x >> 5); }
    __device__ int64_t warps() const { return (int64_t)parts * (blockDim.x >> 5); }
    __device__ int64_t thread() const { return (int64_t)part * blockDim.x + threadIdx.x; }
    __device__ int64_t threads() const { return (int64_t)parts * blockDim.x; }
};

struct ScanSmem {
    int warp_sum[2][32];
    int total[4];  // what the cluster's other CTAs read
};

__device__ __forceinline__ int warp_inclusive(int v)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += o;
    }
    return v;
}

// Sum of v over the threads in front of this one, and over all (kThreads threads); `turn` alternates
// between calls, which keeps one call's sums from the next one's.
__device__ __forceinline__ int block_exclusive(ScanSmem& sm, int v, int turn, int& all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int incl = warp_inclusive(v);
    if (lane == 31) sm.warp_sum[turn & 1][warp] = incl;
    __syncthreads();
    const int sums = warp_inclusive(sm.warp_sum[turn & 1][lane]);
    all = __shfl_sync(0xffffffffu, sums, 31);
    const int before = __shfl_sync(0xffffffffu, sums, warp > 0 ? warp - 1 : 0);
    return (warp > 0 ? before : 0) + incl - v;
}

// Sum of total[which] over the cluster's CTAs in front of this one, and over all
__device__ __forceinline__ int cluster_exclusive(ScanSmem& sm, int which, int& all)
{
    cg::cluster_group cluster = cg::this_cluster();
    int before = 0;
    all = 0;
    for (int r = 0; r < kCluster; ++r) {
        const int t = *cluster.map_shared_rank(&sm.total[which], r);
        if (r < (int)cluster.block_rank()) before += t;
        all += t;
    }
    return before;
}

// the range of n items that this CTA of the cluster scans, in steps of 4
__device__ __forceinline__ void scan_range(int n, int& lo, int& hi)
{
    const int rank = (int)cg::this_cluster().block_rank();
    const int64_t step = ((int64_t)n + kCluster * 4 - 1) / (kCluster * 4) * 4;
    lo = (int)min((int64_t)n, step * rank);
    hi = (int)min((int64_t)n, step * (rank + 1));
}

// pages at .. at + 3 (behind the pool: kNone - 1, neither free nor a page's word)
__device__ __forceinline__ int4 words_at(const int* words, int at, int hi)
{
    int4 w = make_int4(kNone - 1, kNone - 1, kNone - 1, kNone - 1);
    if (at < hi) w = __ldcg(reinterpret_cast<const int4*>(words + at));
    if (at + 1 >= hi) w.y = kNone - 1;
    if (at + 2 >= hi) w.z = kNone - 1;
    if (at + 3 >= hi) w.w = kNone - 1;
    return w;
}

// Sum of sums[0 .. block) and of all n, kThreads threads
__device__ __forceinline__ int sums_exclusive(ScanSmem& sm, const int* sums, int n, int block, int& turn, int& all)
{
    int before = 0, total = 0, mine, part;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int v = __ldcg(sums + i);
        total += v;
        if (i < block) before += v;
    }
    block_exclusive(sm, before, turn++, part);
    mine = part;
    block_exclusive(sm, total, turn++, all);
    return mine;
}

__device__ __forceinline__ void clear_words(int* words, int n, Share s)
{
    int4* v = reinterpret_cast<int4*>(words);
    const int vectors = (n + 3) / 4;
    for (int64_t i = s.thread(); i < vectors; i += s.threads()) v[i] = make_int4(kNone, kNone, kNone, kNone);
}

// ---- remap ----------------------------------------------------------------------

// what a row of the new table keeps and needs
struct Row {
    int parent, kept, end;  // entries kept from the parent's row, entries in all
    bool grows_inside;      // tokens will be written behind others in the last kept page
};

__device__ __forceinline__ Row row_of(const RemapParams& p, int r)
{
    Row w;
    w.parent = __ldg(p.parent + r);
    const int keep = min(max(__ldg(p.keep + r), 0), 1 << 30), need = min(max(__ldg(p.need + r), 0), 1 << 30);
    const int page = 1 << p.page_shift;
    w.kept = w.parent < 0 || w.parent >= p.n_old ? 0 : min((keep + page - 1) >> p.page_shift, p.max_pages);
    w.end = max(w.kept, min((need + page - 1) >> p.page_shift, p.max_pages));
    w.grows_inside = need > keep && w.kept > 0 && keep < ((int64_t)w.kept << p.page_shift);
    return w;
}

__device__ __forceinline__ int entry(const RemapParams& p, const Row& w, int at)
{
    const int e = __ldg(p.table + (size_t)w.parent * p.table_stride + at);
    return e >= 0 && e < p.n_pages ? e : -1;
}

__device__ __forceinline__ void remap_mark(const RemapParams& p, Share s)
{
    const int lane = threadIdx.x & 31;
    const int segments = (p.max_pages + kSegment - 1) / kSegment;
    const int64_t units = (int64_t)p.n_rows * segments;
    for (int64_t u = s.warp(); u < units; u += s.warps()) {
        const int r = (int)(u / segments), at0 = (int)(u % segments) * kSegment;
        const Row w = row_of(p, r);
        int e[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = at0 + i * 32 + lane;
            e[i] = at < w.kept ? entry(p, w, at) : -1;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (e[i] < 0) continue;
            // kReader is below every row's number: the store needs no minimum
            if (w.grows_inside && at0 + i * 32 + lane == w.kept - 1) atomicMin(p.owner + e[i], r);
            else __stcg(p.owner + e[i], kReader);
        }
    }
}

// pages that row r takes, and whether one of them is for a copy of its last kept page
__device__ __forceinline__ int wanted(const RemapParams& p, int r, bool& copied)
{
    const Row w = row_of(p, r);
    copied = false;
    if (w.grows_inside) {
        const int e = entry(p, w, w.kept - 1);
        copied = e >= 0 && __ldcg(p.owner + e) != r;
    }
    return w.end - w.kept + (copied ? 1 : 0);
}

__device__ __forceinline__ int frees(const int4& w) { return (w.x == kNone) + (w.y == kNone) + (w.z == kNone) + (w.w == kNone); }

__device__ __forceinline__ void remap_scan(const RemapParams& p, ScanSmem& sm)
{
    const int tid = threadIdx.x;
    int turn = 0, all, lo, hi, row_lo, row_hi;
    scan_range(p.n_pages, lo, hi);
    scan_range(p.n_rows, row_lo, row_hi);
    int count = 0, want = 0;
    bool copied;
    for (int at = lo + tid * 4; at < hi; at += kThreads * 4) count += frees(words_at(p.owner, at, hi));
    for (int r = row_lo + tid; r < row_hi; r += kThreads) want += wanted(p, r, copied);
    block_exclusive(sm, count, turn++, all);
    if (tid == 0) sm.total[0] = all;
    block_exclusive(sm, want, turn++, all);
    if (tid == 0) sm.total[1] = all;
    cg::this_cluster().sync();
    int n_free, n_wanted;
    int free_at = cluster_exclusive(sm, 0, n_free), want_at = cluster_exclusive(sm, 1, n_wanted);
    for (int base = lo; base < hi; base += kThreads * 4) {
        const int at = base + tid * 4;
        const int4 w = words_at(p.owner, at, hi);
        int k = free_at + block_exclusive(sm, frees(w), turn++, all);
        if (w.x == kNone) p.free_list[k++] = at;
        if (w.y == kNone) p.free_list[k++] = at + 1;
        if (w.z == kNone) p.free_list[k++] = at + 2;
        if (w.w == kNone) p.free_list[k++] = at + 3;
        free_at += all;
    }
    for (int base = row_lo; base < row_hi; base += kThreads) {
        const int r = base + tid;
        const int mine = r < row_hi ? wanted(p, r, copied) : 0;
        const int first = want_at + block_exclusive(sm, mine, turn++, all);
        if (r < row_hi) p.first[r] = copied ? ~first : first;
        want_at += all;
    }
    if (cg::this_cluster().block_rank() == 0 && tid == 0) {
        p.header[0] = n_free;
        p.info[0] = p.n_pages - n_free + min(n_wanted, n_free);
        p.info[1] = max(n_wanted - n_free, 0);
    }
}

// the scan of a large batch: blocks of pages, then blocks of rows
__device__ __forceinline__ int page_blocks(int n_pages) { return (n_pages + kBlockPages - 1) / kBlockPages; }

__device__ __forceinline__ void remap_count(const RemapParams& p, ScanSmem& sm)
{
    const int pages = page_blocks(p.n_pages), block = blockIdx.x;
    int mine = 0, all;
    bool copied;
    if (block < pages) {
        mine = frees(words_at(p.owner, block * kBlockPages + (int)threadIdx.x * 4, p.n_pages));
    } else {
        const int64_t r = (int64_t)(block - pages) * kThreads + threadIdx.x;
        if (r < p.n_rows) mine = wanted(p, (int)r, copied);
    }
    block_exclusive(sm, mine, 0, all);
    if (threadIdx.x == 0) p.sums[block] = all;
}

__device__ __forceinline__ void remap_list(const RemapParams& p, ScanSmem& sm)
{
    const int pages = page_blocks(p.n_pages), block = blockIdx.x;
    int turn = 0, all, total;
    if (block < pages) {
        int k = sums_exclusive(sm, p.sums, pages, block, turn, total);
        const int at = block * kBlockPages + (int)threadIdx.x * 4;
        const int4 w = words_at(p.owner, at, p.n_pages);
        k += block_exclusive(sm, frees(w), turn++, all);
        if (w.x == kNone) p.free_list[k++] = at;
        if (w.y == kNone) p.free_list[k++] = at + 1;
        if (w.z == kNone) p.free_list[k++] = at + 2;
        if (w.w == kNone) p.free_list[k++] = at + 3;
        if (block == 0) {
            int n_wanted;
            sums_exclusive(sm, p.sums + pages, (int)gridDim.x - pages, 0, turn, n_wanted);
            if (threadIdx.x == 0) {
                p.header[0] = total;
                p.info[0] = p.n_pages - total + min(n_wanted, total);
                p.info[1] = max(n_wanted - total, 0);
            }
        }
    } else {
        const int first = sums_exclusive(sm, p.sums + pages, (int)gridDim.x - pages, block - pages, turn, total);
        const int64_t r = (int64_t)(block - pages) * kThreads + threadIdx.x;
        bool copied = false;
        const int mine = r < p.n_rows ? wanted(p, (int)r, copied) : 0;
        const int at = first + block_exclusive(sm, mine, turn++, all);
        if (r < p.n_rows) p.first[r] = copied ? ~at : at;
    }
}

__device__ __forceinline__ void remap_fill(const RemapParams& p, Share s)
{
    const int lane = threadIdx.x & 31;
    const int segments = max(1, (p.max_pages + kSegment - 1) / kSegment);
    const int64_t units = (int64_t)p.n_rows * segments;
    const int n_free = __ldcg(p.header);
    for (int64_t u = s.warp(); u < units; u += s.warps()) {
        const int r = (int)(u / segments), at0 = (int)(u % segments) * kSegment;
        const Row w = row_of(p, r);
        const int code = __ldcg(p.first + r);
        const bool copied = code < 0;
        const int first = copied ? ~code : code;
        const int copy = copied && first < n_free ? __ldcg(p.free_list + first) : -1;
        if (at0 == 0 && lane == 0) {
            p.copy_from[r] = copy >= 0 ? entry(p, w, w.kept - 1) : -1;
            p.copy_to[r] = copy;
        }
        int e[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = at0 + i * 32 + lane;
            e[i] = -1;
            if (at < w.kept) {
                e[i] = copied && at == w.kept - 1 ? copy : entry(p, w, at);
            } else if (at < w.end) {
                const int k = first + (copied ? 1 : 0) + at - w.kept;
                if (k < n_free) e[i] = __ldcg(p.free_list + k);
            }
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = at0 + i * 32 + lane;
            if (at < p.max_pages) p.table_out[(size_t)r * p.out_stride + at] = e[i];
        }
    }
}

// ---- compact --------------------------------------------------------------------

__device__ __forceinline__ int entry(const CompactParams& p, int64_t r, int at)
{
    const int e = p.table[(size_t)r * p.table_stride + at];  // may be the table that fill writes
    return e >= 0 && e < p.n_pages ? e : -1;
}

template <bool FILL>
__device__ __forceinline__ void compact_entries(const CompactParams& p, Share s)
{
    const int lane = threadIdx.x & 31;
    const int segments = (p.max_pages + kSegment - 1) / kSegment;
    const int64_t units = (int64_t)p.n_rows * segments;
    for (int64_t u = s.warp(); u < units; u += s.warps()) {
        const int64_t r = u / segments;
        const int at0 = (int)(u % segments) * kSegment;
        int e[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = at0 + i * 32 + lane;
            e[i] = at < p.max_pages ? entry(p, r, at) : -1;
        }
        if (FILL) {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (e[i] >= 0) e[i] = __ldcg(p.name + e[i]);
            // (a large batch's moved pages: their place in the list)
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int at = at0 + i * 32 + lane;
                if (at < p.max_pages && e[i] < -1) e[i] = __ldcg(p.copy_to + (-2 - e[i]));
            }
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = at0 + i * 32 + lane;
            if (FILL) {
                if (at < p.max_pages) p.table_out[(size_t)r * p.out_stride + at] = e[i];
            } else if (e[i] >= 0) {
                __stcg(p.name + e[i], e[i]);
            }
        }
    }
}

// Page `at` with word w: 1 in the low half where it is in use at or behind `used`, 1 in the high half
// where it is a hole in front of it.  (kNone - 1, behind the pool, is neither: `real` says so.)
__device__ __forceinline__ int moved_or_hole(int w, int at, int used)
{
    if (w == kNone - 1) return 0;
    return at >= used ? (w != kNone ? 1 : 0) : (w == kNone ? 1 << 16 : 0);
}

__device__ __forceinline__ void compact_scan(const CompactParams& p, ScanSmem& sm)
{
    const int tid = threadIdx.x;
    cg::cluster_group cluster = cg::this_cluster();
    int turn = 0, all, lo, hi;
    scan_range(p.n_pages, lo, hi);
    int count = 0;
    for (int at = lo + tid * 4; at < hi; at += kThreads * 4) count += frees(words_at(p.name, at, hi));
    block_exclusive(sm, count, turn++, all);
    const int my_free = all;
    if (tid == 0) sm.total[0] = all;
    cluster.sync();
    int n_free;
    cluster_exclusive(sm, 0, n_free);
    const int used = p.n_pages - n_free;
    // pages to move and holes of this range: known, but for the range that `used` falls into
    int moved = lo >= used ? hi - lo - my_free : 0, holes = hi <= used ? my_free : 0;
    if (lo < used && used < hi) {
        int m = 0, h = 0;
        for (int at = lo + tid * 4; at < hi; at += kThreads * 4) {
            const int4 w = words_at(p.name, at, hi);
            const int c = moved_or_hole(w.x, at, used) + moved_or_hole(w.y, at + 1, used) + moved_or_hole(w.z, at + 2, used) +
                          moved_or_hole(w.w, at + 3, used);
            m += c & 0xffff;
            h += c >> 16;
        }
        block_exclusive(sm, m, turn++, moved);
        block_exclusive(sm, h, turn++, holes);
    }
    if (tid == 0) {
        sm.total[1] = moved;
        sm.total[2] = holes;
    }
    cluster.sync();
    int n_moved, n_holes;
    int from = cluster_exclusive(sm, 1, n_moved), to = cluster_exclusive(sm, 2, n_holes);
    for (int base = lo; base < hi; base += kThreads * 4) {
        const int at = base + tid * 4;
        const int4 w = words_at(p.name, at, hi);
        const int c[4] = {moved_or_hole(w.x, at, used), moved_or_hole(w.y, at + 1, used), moved_or_hole(w.z, at + 2, used),
                          moved_or_hole(w.w, at + 3, used)};
        // at most 4096 of either: the halves stay apart
        const int k = block_exclusive(sm, c[0] + c[1] + c[2] + c[3], turn++, all);
        int f = from + (k & 0xffff), t = to + (k >> 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (c[i] & 0xffff) p.copy_from[f++] = at + i;
            if (c[i] >> 16) p.copy_to[t++] = at + i;
        }
        from += all & 0xffff;
        to += all >> 16;
    }
    cluster.sync();  // the lists are whole; as many holes as pages to move
    const Share s{(int)cluster.block_rank(), kCluster};
    for (int64_t i = s.thread(); i < n_moved; i += s.threads()) p.name[__ldcg(p.copy_from + i)] = __ldcg(p.copy_to + i);
    for (int64_t i = n_moved + s.thread(); i < p.n_pages / 2; i += s.threads()) p.copy_from[i] = p.copy_to[i] = -1;
    if (s.part == 0 && tid == 0) {
        p.info[0] = used;
        p.info[1] = n_moved;
    }
}

__device__ __forceinline__ void compact_count(const CompactParams& p, ScanSmem& sm)
{
    int all;
    const int at = blockIdx.x * kBlockPages + (int)threadIdx.x * 4;
    block_exclusive(sm, min(4, max(0, p.n_pages - at)) - frees(words_at(p.name, at, p.n_pages)), 0, all);
    if (threadIdx.x == 0) p.sums[blockIdx.x] = all;
}

__device__ __forceinline__ void compact_list(const CompactParams& p, ScanSmem& sm)
{
    const int tid = threadIdx.x, block = blockIdx.x;
    int turn = 0, all, used;
    const int before = sums_exclusive(sm, p.sums, (int)gridDim.x, block, turn, used);
    // pages in use in front of `used`: the blocks there, and the block that it falls into up to it
    int below, unused, cut = 0;
    const int edge = used / kBlockPages;
    below = sums_exclusive(sm, p.sums, (int)gridDim.x, edge, turn, unused);
    {
        const int at = edge * kBlockPages + tid * 4;
        const int4 w = words_at(p.name, at, min(used, p.n_pages));
        if (at < used) cut = min(4, used - at) - frees(w);
        block_exclusive(sm, cut, turn++, all);
        below += all;
    }
    const int n_moved = used - below, lo = block * kBlockPages, at = lo + tid * 4;
    const int4 w = words_at(p.name, at, p.n_pages);
    const int c[4] = {moved_or_hole(w.x, at, used), moved_or_hole(w.y, at + 1, used), moved_or_hole(w.z, at + 2, used), moved_or_hole(w.w, at + 3, used)};
    const int k = block_exclusive(sm, c[0] + c[1] + c[2] + c[3], turn++, all);
    // pages to move in front of this block, and holes
    int f = max(before - below, 0) + (k & 0xffff), t = min(lo, used) - min(before, below) + (k >> 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (c[i] & 0xffff) {
            p.copy_from[f] = at + i;
            p.name[at + i] = -2 - f++;
        }
        if (c[i] >> 16) p.copy_to[t++] = at + i;
    }
    for (int64_t i = (int64_t)block * kThreads + tid; i < p.n_pages / 2; i += (int64_t)gridDim.x * kThreads)
        if (i >= n_moved) p.copy_from[i] = p.copy_to[i] = -1;
    if (block == 0 && tid == 0) {
        p.info[0] = used;
        p.info[1] = n_moved;
    }
}

// ---- launches -------------------------------------------------------------------

__device__ __forceinline__ void clear(const RemapParams& p, Share s) { clear_words(p.owner, p.n_pages, s); }
__device__ __forceinline__ void mark(const RemapParams& p, Share s) { remap_mark(p, s); }
__device__ __forceinline__ void scan(const RemapParams& p, ScanSmem& sm) { remap_scan(p, sm); }
__device__ __forceinline__ void fill(const RemapParams& p, Share s) { remap_fill(p, s); }
__device__ __forceinline__ void clear(const CompactParams& p, Share s) { clear_words(p.name, p.n_pages, s); }
__device__ __forceinline__ void mark(const CompactParams& p, Share s) { compact_entries<false>(p, s); }
__device__ __forceinline__ void scan(const CompactParams& p, ScanSmem& sm) { compact_scan(p, sm); }
__device__ __forceinline__ void fill(const CompactParams& p, Share s) { compact_entries<true>(p, s); }

__device__ __forceinline__ void count(const RemapParams& p, ScanSmem& sm) { remap_count(p, sm); }
__device__ __forceinline__ void list(const RemapParams& p, ScanSmem& sm) { remap_list(p, sm); }
__device__ __forceinline__ void count(const CompactParams& p, ScanSmem& sm) { compact_count(p, sm); }
__device__ __forceinline__ void list(const CompactParams& p, ScanSmem& sm) { compact_list(p, sm); }

// all phases in one cluster
template <typename Params>
__global__ void __cluster_dims__(kCluster) __launch_bounds__(kThreads) pages_cluster_kernel(Params p)
{
    __shared__ ScanSmem sm;
    pdl_launch_dependents();
    pdl_wait();
    cg::cluster_group cluster = cg::this_cluster();
    const Share s{(int)cluster.block_rank(), kCluster};
    clear(p, s);
    cluster.sync();
    mark(p, s);
    cluster.sync();
    scan(p, sm);
    cluster.sync();  // also: no CTA leaves before its totals have been read
    fill(p, s);
}

// one phase over the whole GPU
template <typename Params, int PHASE>
__global__ void __launch_bounds__(256) pages_phase_kernel(Params p)
{
    pdl_launch_dependents();
    pdl_wait();
    const Share s{(int)blockIdx.x, (int)gridDim.x};
    if (PHASE == Phases::kClear) clear(p, s);
    if (PHASE == Phases::kMark) mark(p, s);
    if (PHASE == Phases::kFill) fill(p, s);
}

// the scan's two halves, a block for every kBlockPages pages and, for remap, kThreads rows
template <typename Params, bool LIST>
__global__ void __launch_bounds__(kThreads) pages_scan_kernel(Params p)
{
    __shared__ ScanSmem sm;
    pdl_launch_dependents();
    pdl_wait();
    if (LIST) list(p, sm);
    else count(p, sm);
}

int row_blocks(const RemapParams& p) { return (p.n_rows + kThreads - 1) / kThreads; }
int row_blocks(const CompactParams&) { return 0; }

template <typename Params>
cudaError_t launch_pages(const Params& p, cudaStream_t stream)
{
    const int64_t cells = (int64_t)p.n_rows * p.max_pages;
    if (cells + p.n_pages < kOneLaunch) return launch_k(pages_cluster_kernel<Params>, dim3(kCluster), dim3(kThreads), 0, stream, true, p);
    // a warp for every kSegment entries of a row, or every 512 words, and at most 8 blocks of 8 warps on an SM
    const int64_t units = (int64_t)p.n_rows * ((p.max_pages + kSegment - 1) / kSegment), most = 152 * 8;
    const auto blocks = [&](int64_t warps) { return dim3((unsigned)std::min(most, std::max<int64_t>(1, (warps + 7) / 8))); };
    const dim3 scans((unsigned)(((int64_t)p.n_pages + kBlockPages - 1) / kBlockPages + row_blocks(p)));
    cudaError_t e = launch_k(pages_phase_kernel<Params, Phases::kClear>, blocks(p.n_pages / 512), dim3(256), 0, stream, true, p);
    if (e == cudaSuccess) e = launch_k(pages_phase_kernel<Params, Phases::kMark>, blocks(units), dim3(256), 0, stream, true, p);
    if (e == cudaSuccess) e = launch_k(pages_scan_kernel<Params, false>, scans, dim3(kThreads), 0, stream, true, p);
    if (e == cudaSuccess) e = launch_k(pages_scan_kernel<Params, true>, scans, dim3(kThreads), 0, stream, true, p);
    if (e == cudaSuccess) e = launch_k(pages_phase_kernel<Params, Phases::kFill>, blocks(units), dim3(256), 0, stream, true, p);
    return e;
}

}  // namespace

size_t remap_sums(int n_pages, int n_rows) { return ((size_t)n_pages + kBlockPages - 1) / kBlockPages + ((size_t)n_rows + kThreads - 1) / kThreads; }
size_t compact_sums(int n_pages) { return ((size_t)n_pages + kBlockPages - 1) / kBlockPages; }

cudaError_t launch_kv_remap(const RemapParams& p, cudaStream_t stream) { return launch_pages(p, stream); }
cudaError_t launch_kv_compact(const CompactParams& p, cudaStream_t stream) { return launch_pages(p, stream); }

}  // namespace gdn
