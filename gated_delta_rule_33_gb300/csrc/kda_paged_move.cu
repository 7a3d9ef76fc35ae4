// kda_paged_move.cu -- keys and values of a paged cache moved within it: the accepted path of a
// tree of drafted tokens to where the context ends, and the pages of a fork.
//
// Copies: every row is read once and written once, 4 bytes a value (2 for an 8-bit cache), and
// a call moves little: what counts is the chain of loads (offsets, word, table, row), which
// thousands of threads walk side by side.  A thread moves one 16-byte piece of a row for all
// rows of a path.
#include "kda_tree.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 8;  // rows of a path that a thread has in flight

// Where a piece of a slot's row lies, or -1 where its page is not one of the cache's.
struct Place {
    const PagedView &cache;
    int64_t piece;

    __device__ __forceinline__ Place(const PagedView &c, uint32_t u, FastDiv head_pieces) : cache(c) {
        uint32_t h, at;
        head_pieces.divmod(u, h, at);
        piece = h * cache.head_stride + at * 16;
    }
    __device__ __forceinline__ int64_t operator()(int page, uint32_t in_page) const {
        if (page < 0 || page >= cache.num_pages) return -1;
        return page * cache.page_stride + in_page * cache.token_stride + piece;
    }
};

// blockIdx: (pieces of a row, request, keys or values).  The r-th node of the path goes to
// position C + r, C = seq_len - n: never behind its own place, and in order, so a place is
// read before a later row goes there: a thread reads rows in order, kAhead at a time, and
// writes them after.
__global__ void __launch_bounds__(kThreads) compact_kernel(
    const PagedView cache, const int32_t *block_table, int max_pages, const int32_t *seq_lens,
    const int32_t *cu, const uint64_t *ancestors, const int32_t *last, int64_t N, int max_nodes,
    uint32_t row_pieces, FastDiv head_pieces, int32_t *kept_lens, unsigned int *err) {
    wait_for_kernel_before();
    const int b = blockIdx.y;
    const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
    const bool speaks = blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0;
    const TreeRows t = tree_rows(cu, b, N, max_nodes);
    const int len = seq_lens[b], end = last[b];
    const bool fits = len >= t.rows && len <= static_cast<int64_t>(max_pages) * cache.page.d;
    const bool bad = t.bad || !fits || end >= t.n;
    const int context = fits ? len - t.rows : 0;
    uint64_t path = 0;
    if (!bad && end >= 0) path = path_of(ancestors[t.first + end], end);
    if (speaks) {
        if (bad) record_device_error(err, kDevInvalidArg);
        if (kept_lens != nullptr) kept_lens[b] = context + __popcll(path);
    }
    if (u >= row_pieces) return;
    // nodes 0 .. r-1 that are all on the path are where they belong
    const int settled = __ffsll(static_cast<long long>(~path)) - 1;
    int to = settled < 0 ? kTreeNodes : settled;
    if (to >= kTreeNodes) return;
    path &= ~bits_below(to);
    const Place place(cache, u, head_pieces);
    uint8_t *data = blockIdx.z != 0 ? cache.v : cache.k;
    const int32_t *row = block_table + static_cast<int64_t>(b) * max_pages;
    auto at = [&](int node) {
        uint32_t page, in_page;
        cache.page.divmod(static_cast<uint32_t>(context + node), page, in_page);
        return place(row[page], in_page);
    };
    while (path != 0) {
        uint4 x[kAhead];
        int64_t dst[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            dst[i] = -1;
            if (path != 0) {
                const int node = __ffsll(static_cast<long long>(path)) - 1;
                path &= path - 1;
                const int64_t src = at(node);
                dst[i] = at(to++);
                if (src < 0 || dst[i] < 0) {
                    dst[i] = -1;
                    record_device_error(err, kDevInvalidArg);
                } else {
                    x[i] = *reinterpret_cast<const uint4 *>(data + src);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (dst[i] >= 0) *reinterpret_cast<uint4 *>(data + dst[i]) = x[i];
    }
}

// blockIdx: (copy, keys or values, kAhead rows).  The block's threads move the rows' pieces.
__global__ void __launch_bounds__(kThreads) copy_kernel(const int32_t *copies, const PagedView cache,
                                                        FastDiv row_pieces, FastDiv head_pieces,
                                                        unsigned int *err) {
    wait_for_kernel_before();
    const int32_t *c = copies + 3 * static_cast<int64_t>(blockIdx.x);
    const int from = c[0], to = c[1], rows = c[2];
    if (rows == 0) return;
    if (from < 0 || from >= cache.num_pages || to < 0 || to >= cache.num_pages || rows < 0 ||
        rows > static_cast<int>(cache.page.d)) {
        if (threadIdx.x == 0) record_device_error(err, kDevInvalidArg);
        return;
    }
    if (from == to) return;
    uint8_t *data = blockIdx.y != 0 ? cache.v : cache.k;
    const uint32_t row = row_pieces.d;
    for (uint32_t r0 = blockIdx.z * kAhead; r0 < static_cast<uint32_t>(rows); r0 += gridDim.z * kAhead) {
        for (uint32_t u = threadIdx.x; u < row; u += kThreads) {
            const Place place(cache, u, head_pieces);
            uint4 x[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (r0 + i < static_cast<uint32_t>(rows))
                    x[i] = load_once(reinterpret_cast<const uint4 *>(data + place(from, r0 + i)));
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (r0 + i < static_cast<uint32_t>(rows))
                    *reinterpret_cast<uint4 *>(data + place(to, r0 + i)) = x[i];
        }
    }
}

}  // namespace

cudaError_t launch_paged_compact(const PagedView &cache, const int32_t *block_table, int max_pages,
                                 const int32_t *seq_lens, const int32_t *cu,
                                 const uint64_t *ancestors, const int32_t *last, int B, int64_t N,
                                 int max_nodes, int32_t *kept_lens, unsigned int *err,
                                 cudaStream_t s) {
    const uint32_t head = static_cast<uint32_t>(cache.head_dim) * (cache.fp8 ? 1 : 2) / 16;
    const uint32_t row = head * cache.heads;
    const dim3 grid((row + kThreads - 1) / kThreads, B, 2);
    return launch_early(compact_kernel, grid, kThreads, 0, s, cache, block_table, max_pages,
                        seq_lens, cu, ancestors, last, N, max_nodes, row, FastDiv(head), kept_lens,
                        err);
}

cudaError_t launch_paged_copy(const int32_t *copies, int n, const PagedView &cache,
                              unsigned int *err, cudaStream_t s) {
    const uint32_t head = static_cast<uint32_t>(cache.head_dim) * (cache.fp8 ? 1 : 2) / 16;
    const uint32_t groups = (cache.page.d + kAhead - 1) / kAhead;
    return launch_early(copy_kernel, dim3(n, 2, groups < 1024 ? groups : 1024), kThreads, 0, s, copies, cache,
                        FastDiv(head * cache.heads), FastDiv(head), err);
}

}  // namespace kda
