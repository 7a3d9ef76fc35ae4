// kda_page_share.cu -- requests that share pages: forks, and what requests give back.
//
// shares[p] counts the holders of page p beyond the first.  A fork holds its source's full
// pages (shares + 1 each) and a page of its own for the rest, which is copied; a page that is
// given back has one share less, or is free.  Both calls touch a few bytes a page: latency.
#include "kda_tree.cuh"

namespace kda {
namespace {

constexpr int kForkThreads = 128;
constexpr int kThreads = kReleaseRequests;
constexpr int kRangePages = 1 << 20;  // pages whose bits fit shared memory (128 KB)
constexpr int kRanks = 8;             // blocks of a release of many requests, a cluster
// Up to these, one block: 16 requests' 60 pages each take it 6.9 us, a cluster 7.6; 64 requests' 12.4
// and 7.9, 256 requests' 35 and 11.5.
constexpr int kFewRequests = 16;

// The pages of a length.
__device__ __forceinline__ int pages_of(int n, const FastDiv &page) {
    const uint32_t full = page.div(n);
    return static_cast<int>(full + (full * page.d != static_cast<uint32_t>(n) ? 1 : 0));
}

// Whether fork f takes a page, its source's length being good.
__device__ __forceinline__ bool takes_page(int src, int B, const int32_t *seq_lens, int64_t room,
                                           const FastDiv &page) {
    if (src < 0 || src >= B) return false;
    const int n = seq_lens[src];
    return n >= 0 && n <= room && n - static_cast<int>(page.div(n)) * static_cast<int>(page.d) != 0;
}

// One block a fork; each looks over all forks for its place in the free list and for those
// that would write what it reads.  Lengths are written for destinations alone, which are no
// served fork's source.
__global__ void __launch_bounds__(kForkThreads) fork_kernel(
    const int32_t *src, const int32_t *dst, int forks, int32_t *seq_lens, const int32_t *free_pages,
    int num_free, int32_t *block_table, int max_pages, int B, FastDiv page, int num_pages,
    int32_t *shares, int32_t *copies, int32_t *pages_used, unsigned int *err) {
    __shared__ int s_before, s_all, s_clash;
    wait_for_kernel_before();
    const int f = blockIdx.x, tid = threadIdx.x;
    const int from = src[f], to = dst[f];
    const int64_t room = static_cast<int64_t>(max_pages) * page.d;
    if (tid == 0) s_before = s_all = s_clash = 0;
    __syncthreads();
    int before = 0, all = 0;
    bool clash = false;
    for (int i = tid; i < forks; i += kForkThreads) {
        const int x = src[i];
        const int takes = takes_page(x, B, seq_lens, room, page);
        all += takes;
        if (i < f) before += takes;
        clash |= x == to || (i < f && dst[i] == to);
    }
    before = __reduce_add_sync(0xffffffffu, before);
    all = __reduce_add_sync(0xffffffffu, all);
    if ((tid & 31) == 0) {
        atomicAdd(&s_before, before);
        atomicAdd(&s_all, all);
    }
    if (clash) s_clash = 1;
    __syncthreads();
    if (f == 0 && tid == 0) *pages_used = min(s_all, num_free);
    const bool takes = takes_page(from, B, seq_lens, room, page);
    const int n = from >= 0 && from < B ? seq_lens[from] : -1;
    const bool served = n >= 0 && n <= room && to >= 0 && to < B && s_clash == 0 &&
                        (!takes || s_before < num_free);
    const int full = served ? static_cast<int>(page.div(n)) : 0;
    const int32_t *theirs = block_table + static_cast<int64_t>(from) * max_pages;
    int32_t *ours = block_table + static_cast<int64_t>(to) * max_pages;
    if (tid == 0) {
        int a = -1, c = -1, rows = 0;
        if (!served) {
            record_device_error(err, kDevInvalidArg);
        } else {
            seq_lens[to] = n;
            if (takes) {
                a = theirs[full];
                c = free_pages[s_before];
                rows = n - full * static_cast<int>(page.d);
                ours[full] = c;
                if (a < 0 || a >= num_pages || c < 0 || c >= num_pages) {
                    record_device_error(err, kDevInvalidArg);
                    a = c = -1;
                    rows = 0;
                }
            }
        }
        copies[3 * static_cast<int64_t>(f)] = a;
        copies[3 * static_cast<int64_t>(f) + 1] = c;
        copies[3 * static_cast<int64_t>(f) + 2] = rows;
    }
    for (int i = tid; i < full; i += kForkThreads) {
        const int p = theirs[i];
        ours[i] = p;
        if (p >= 0 && p < num_pages) atomicAdd(shares + p, 1);
        else record_device_error(err, kDevInvalidArg);
    }
}

// The sum over the threads before this one, and over all; every thread of the block calls it.
__device__ __forceinline__ int scan_block(int x, int *s_warp, int &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int sum = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    const int w = s_warp[lane];
    int before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
    all = __reduce_add_sync(0xffffffffu, w);
    return before + sum - x;
}

// The blocks of a cluster meet; what they wrote before is seen by all of them.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this block's shared `p` in block `rank` of its cluster.
__device__ __forceinline__ uint32_t in_block(const void *p, int rank) {
    uint32_t x;
    asm("mapa.shared::cluster.u32 %0, %1, %2;"
        : "=r"(x)
        : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    return x;
}

// One cluster.  A page that nobody else holds falls to -1 by the thread that gives it back last,
// which marks it in a bitmap in shared memory, a slice in each block; the marked pages are then
// listed in order, so the list does not depend on which thread that was.  The pages are a chain of
// trips each (search, table, share), so the number of threads that walk them counts: 8 blocks give
// 340 of 1024 requests back in 11 us where one took 26 (both cold).
__global__ void __launch_bounds__(kThreads) release_kernel(
    const int32_t *seq_lens, const int32_t *kept_lens, const int32_t *block_table, int max_pages,
    int B, FastDiv page, int num_pages, int32_t *shares, int32_t *freed, int max_freed,
    int32_t *num_freed, int words, unsigned int *err) {
    extern __shared__ uint32_t s_free[];  // [words], of this block's slice
    __shared__ int s_warp[32], s_off[kThreads], s_first[kThreads], s_count;
    wait_for_kernel_before();
    const int tid = threadIdx.x, rank = blockIdx.x, ranks = gridDim.x;
    const int64_t room = static_cast<int64_t>(max_pages) * page.d;
    int listed = 0;
    for (int64_t range = 0; range < num_pages; range += kRangePages) {
        const int base = static_cast<int>(range);
        for (int i = tid; i < words; i += kThreads) s_free[i] = 0;
        cluster_sync();
        for (int b0 = 0; b0 < B; b0 += kThreads) {
            // the pages of up to kThreads requests, as one list
            int count = 0, first = 0;
            if (b0 + tid < B) {
                const int n = seq_lens[b0 + tid], m = kept_lens[b0 + tid];
                if (m < 0 || n < m || n > room) {
                    if (rank == 0) record_device_error(err, kDevInvalidArg);
                } else {
                    first = pages_of(m, page);
                    count = pages_of(n, page) - first;
                }
            }
            int all;
            const int off = scan_block(count, s_warp, all);
            s_off[tid] = off;
            s_first[tid] = first;
            __syncthreads();
            for (int e = rank * kThreads + tid; e < all; e += ranks * kThreads) {
                int lo = 0;  // the last request whose pages begin at e or before
#pragma unroll
                for (int step = kThreads / 2; step > 0; step >>= 1)
                    if (s_off[lo + step] <= e) lo += step;
                const int p = block_table[static_cast<int64_t>(b0 + lo) * max_pages + s_first[lo] +
                                          (e - s_off[lo])];
                if (p < 0 || p >= num_pages) {
                    record_device_error(err, kDevInvalidArg);
                } else if (p >= base && p - base < kRangePages) {
                    const int held = atomicSub(shares + p, 1);
                    if (held == 0) {
                        const int word = (p - base) >> 5, owner = word / words;
                        asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(
                                         in_block(s_free + (word - owner * words), owner)),
                                     "r"(1u << ((p - base) & 31))
                                     : "memory");
                    } else if (held < 0) {  // given back more often than held
                        atomicAdd(shares + p, 1);
                        record_device_error(err, kDevInvalidArg);
                    }
                }
            }
            __syncthreads();
        }
        cluster_sync();
        // the pages marked in the slices before this one's, and in all
        int mine = 0;
        for (int i = tid; i < words; i += kThreads) mine += __popc(s_free[i]);
        scan_block(mine, s_warp, mine);
        if (tid == 0) s_count = mine;
        cluster_sync();
        int first = listed;
        for (int r = 0; r < ranks; ++r) {
            int count;
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(count) : "r"(in_block(&s_count, r)) : "memory");
            if (r < rank) first += count;
            listed += count;
        }
        for (int w0 = 0; w0 < words; w0 += kThreads) {
            uint32_t bits = w0 + tid < words ? s_free[w0 + tid] : 0;
            int all;
            int at = first + scan_block(__popc(bits), s_warp, all);
            while (bits != 0) {
                const int p = base + (rank * words + w0 + tid) * 32 + __ffs(static_cast<int>(bits)) - 1;
                bits &= bits - 1;
                shares[p] = 0;
                if (at < max_freed) freed[at] = p;
                else record_device_error(err, kDevInvalidArg);
                ++at;
            }
            first += all;
            __syncthreads();
        }
    }
    cluster_sync();  // (nobody leaves while its count may be read)
    if (rank == 0 && tid == 0) *num_freed = min(listed, max_freed);
}

}  // namespace

cudaError_t launch_page_fork(const int32_t *src, const int32_t *dst, int forks, int32_t *seq_lens,
                             const int32_t *free_pages, int num_free, int32_t *block_table,
                             int max_pages, int B, int page_size, int num_pages, int32_t *shares,
                             int32_t *copies, int32_t *pages_used, unsigned int *err,
                             cudaStream_t s) {
    if (forks == 0) return cudaMemsetAsync(pages_used, 0, 4, s);
    return launch_early(fork_kernel, dim3(forks), kForkThreads, 0, s, src, dst, forks, seq_lens,
                        free_pages, num_free, block_table, max_pages, B, FastDiv(page_size),
                        num_pages, shares, copies, pages_used, err);
}

cudaError_t launch_page_release(const int32_t *seq_lens, const int32_t *kept_lens,
                                const int32_t *block_table, int max_pages, int B, int page_size,
                                int num_pages, int32_t *shares, int32_t *freed, int max_freed,
                                int32_t *num_freed, unsigned int *err, cudaStream_t s) {
    const int ranks = B <= kFewRequests ? 1 : kRanks;
    const int all = ((num_pages < kRangePages ? num_pages : kRangePages) + 31) / 32;
    const int words = (all + ranks - 1) / ranks, smem = words * 4;
    cudaError_t e = cudaSuccess;
    if (smem > 32 * 1024)
        e = ensure_dynamic_smem(reinterpret_cast<const void *>(&release_kernel), kRangePages / 8);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = ranks;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ranks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attrs;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, release_kernel, seq_lens, kept_lens, block_table, max_pages, B,
                              FastDiv(page_size), num_pages, shares, freed, max_freed, num_freed,
                              words, err);
}

}  // namespace kda
