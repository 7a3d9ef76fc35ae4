// kda_tree.cuh -- what the operators over trees of drafted tokens share: a request's rows and
// paths, and the launchers of their entry points.
//
// Request b has n = cu[b + 1] - cu[b] <= kTreeNodes nodes, rows cu[b] .. of the token tensors.
// The word of node i says which nodes of its request it sees; the set bits below bit i are its
// ancestors, nearest first from the top.
#pragma once

#include "kda_internal.cuh"
#include "kda_paged.cuh"

namespace kda {

constexpr int kTreeNodes = 64;

// Requests whose pages a release takes as one list, with 32-bit places in it.
constexpr int kReleaseRequests = 1024;

struct TreeRows {
    int64_t first;  // row of node 0
    int n;          // nodes; 0 where there is nothing to do
    int rows;       // rows to write: n, or those of a request with too many (zeros)
    bool bad;       // to be reported
};

// Offsets that lie outside the N rows, or go back, leave their request out; one of more than
// max_nodes rows has no nodes.
__device__ __forceinline__ TreeRows tree_rows_between(int64_t lo, int64_t hi, int64_t N, int max_nodes) {
    if (lo < 0 || hi < lo || hi > N) return {0, 0, 0, true};
    const int64_t n = hi - lo;
    const bool ok = n <= max_nodes;
    return {lo, ok ? static_cast<int>(n) : 0, static_cast<int>(n), !ok};
}
__device__ __forceinline__ TreeRows tree_rows(const int32_t *cu, int b, int64_t N, int max_nodes) {
    return tree_rows_between(cu[b], cu[b + 1], N, max_nodes);
}

__device__ __forceinline__ uint64_t bits_below(int i) {
    return i >= 64 ? ~uint64_t{0} : (uint64_t{1} << i) - 1;
}

// The nodes of the path that ends at node i, i among them.
__device__ __forceinline__ uint64_t path_of(uint64_t word, int i) {
    return (word & bits_below(i)) | (uint64_t{1} << i);
}

__device__ __forceinline__ int top_bit(uint64_t x) { return 63 - __clzll(static_cast<long long>(x)); }

struct TreeStep {   // the operands of the recurrence over trees
    const __nv_bfloat16 *q, *k, *v;
    const float *g, *beta;
    void *pool;
    const int32_t *slots;  // or null: slot b
    int num_slots;
    const int32_t *cu;
    const uint64_t *ancestors;
    const int32_t *last;   // of the commit
    int B, H, max_nodes;
    int64_t N;
    float scale;
    void *o;
    float *u;
    unsigned int *err;
};

cudaError_t launch_tree_decode(const TreeStep &a, bool state_bf16, bool o_bf16, int num_sms,
                               cudaStream_t s);
cudaError_t launch_tree_commit(const TreeStep &a, bool state_bf16, cudaStream_t s);

struct TreeConv {
    const __nv_bfloat16 *x[3];
    const float *w[3];
    __nv_bfloat16 *y[3];
    __nv_bfloat16 *pool;
    const int32_t *slots;
    int num_slots;
    const int32_t *cu;
    const uint64_t *ancestors;
    const int32_t *last;   // of the commit
    int B, C, max_nodes;
    int64_t N;
    unsigned int *err;
};

cudaError_t launch_tree_conv(const TreeConv &a, int num_sms, cudaStream_t s);
cudaError_t launch_tree_conv_commit(const TreeConv &a, cudaStream_t s);

struct TreeAttention {
    const __nv_bfloat16 *q;
    int64_t q_row_stride;
    PagedView cache;
    const int32_t *block_table;
    int max_pages;
    const int32_t *seq_lens, *cu;
    const uint64_t *ancestors;
    int B, q_heads, group, max_nodes;
    int64_t N;
    float scale;
    __nv_bfloat16 *o;
    float *lse;
    uint8_t *workspace;
    unsigned int *err;
};

size_t paged_tree_workspace_bytes(int B, int max_nodes, int q_heads, int kv_heads, int head_dim);
cudaError_t launch_paged_tree_decode(const TreeAttention &a, int num_sms, cudaStream_t s);

cudaError_t launch_paged_compact(const PagedView &cache, const int32_t *block_table, int max_pages,
                                 const int32_t *seq_lens, const int32_t *cu,
                                 const uint64_t *ancestors, const int32_t *last, int B, int64_t N,
                                 int max_nodes, int32_t *kept_lens, unsigned int *err,
                                 cudaStream_t s);
cudaError_t launch_paged_copy(const int32_t *copies, int n, const PagedView &cache,
                              unsigned int *err, cudaStream_t s);
cudaError_t launch_page_fork(const int32_t *src, const int32_t *dst, int forks, int32_t *seq_lens,
                             const int32_t *free_pages, int num_free, int32_t *block_table,
                             int max_pages, int B, int page_size, int num_pages, int32_t *shares,
                             int32_t *copies, int32_t *pages_used, unsigned int *err,
                             cudaStream_t s);
cudaError_t launch_page_release(const int32_t *seq_lens, const int32_t *kept_lens,
                                const int32_t *block_table, int max_pages, int B, int page_size,
                                int num_pages, int32_t *shares, int32_t *freed, int max_freed,
                                int32_t *num_freed, unsigned int *err, cudaStream_t s);

}  // namespace kda
