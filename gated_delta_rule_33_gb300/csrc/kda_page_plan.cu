// kda_page_plan.cu -- block tables and slot maps from request lengths.
//
// The whole step is two exclusive prefix sums over the requests (new tokens:
// the rows of cu_seqlens; pages needed: the place in the free list) and a map
// from each new token to its request.  One launch: a CTA owns 1024 or 2048
// consecutive tokens and scans the requests itself, in tiles of as many, until the
// sum passes its tokens (B is at most some thousands, 8 bytes each, out of L2; a second
// launch or a look-back over other CTAs' sums would cost more than the scan).
// A request that meets the CTA's tokens leaves its record at the place of its
// first token there; starts are distinct, so a running maximum over the
// places then gives every token its request without a search.  A page's table
// entry is written by the token at offset 0 of it: each page taken has one.
// Bound: latency, the launch and two trips to memory (lengths, then page numbers).
#include "kda_internal.cuh"
#include "kda_paged.cuh"

namespace kda {
namespace {

constexpr int kItems = 4;                  // requests, then tokens, per thread
// Sums stop here.  One more token or page than this is past every list (both
// are shorter), and two such sums still fit 32 bits.
constexpr uint32_t kMany = 0x7fffffff;

__device__ __forceinline__ uint32_t add(uint32_t x, uint32_t y) { return min(x + y, kMany); }

// Four consecutive values of a list of n; zeros past its end.
__device__ __forceinline__ int4 load4(const int32_t *p, int64_t i, int64_t n) {
    if (i + 4 <= n) return *reinterpret_cast<const int4 *>(p + i);
    return make_int4(i < n ? p[i] : 0, i + 1 < n ? p[i + 1] : 0, i + 2 < n ? p[i + 2] : 0, 0);
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) plan_kernel(
    const int32_t *cached_lens, const int32_t *new_lens, const int32_t *free_pages, int num_free,
    int32_t *block_table, int max_pages, int B, FastDiv page, int num_pages, int32_t *seq_lens,
    int32_t *cu_seqlens, int32_t *slot_map, int64_t N, int32_t *pages_used, unsigned int *err) {
    constexpr int kTile = kThreads * kItems, kWarps = kThreads / 32;
    // a request at its first token in the CTA's range: its first row (which may lie before
    // the range) and tokens, its cached tokens, its place in the free list; its number, -1
    // where it is refused, -2 where no request starts
    __shared__ int s_cu[kTile], s_count[kTile], s_cached[kTile], s_off[kTile];
    __shared__ __align__(16) int s_b[kTile];  // read four at a time
    __shared__ uint32_t s_tok[kWarps], s_pg[kWarps];
    __shared__ int s_max[kWarps];
    __shared__ int s_used;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool writer = blockIdx.x == 0;   // of what there is one of per request
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTile;
    const int64_t t1 = t0 + kTile < N ? t0 + kTile : N;
    const int64_t cap = static_cast<int64_t>(max_pages) * page.d;
    wait_for_kernel_before();
    auto pages_of = [&](int n) { return n <= 0 ? 0 : static_cast<int>(page.div(n - 1)) + 1; };

    int4 c4 = load4(cached_lens, tid * kItems, B), n4 = load4(new_lens, tid * kItems, B);
#pragma unroll
    for (int i = 0; i < kItems; ++i) s_b[tid + i * kThreads] = -2;
    if (tid == 0) s_used = 0;

    uint32_t run_tok = 0, run_pg = 0;
    for (int64_t base = 0; base < B; base += kTile) {
        if (!writer && run_tok >= t1) break;
        const int c[kItems] = {c4.x, c4.y, c4.z, c4.w};
        int n[kItems] = {n4.x, n4.y, n4.z, n4.w}, need[kItems];
        bool ok[kItems];
        uint32_t tok = 0, pg = 0;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int64_t total = static_cast<int64_t>(c[i]) + n[i];
            ok[i] = c[i] >= 0 && n[i] >= 0 && total <= cap && total <= INT32_MAX;
            need[i] = ok[i] ? pages_of(static_cast<int>(total)) - pages_of(c[i]) : 0;
            n[i] = n[i] > 0 ? n[i] : 0;
            tok = add(tok, n[i]);
            pg = add(pg, need[i]);
        }
        if (base + kTile < B) {
            c4 = load4(cached_lens, base + kTile + tid * kItems, B);
            n4 = load4(new_lens, base + kTile + tid * kItems, B);
        }
        // prefix sums over the tile
        uint32_t itok = tok, ipg = pg;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, itok, d);
            const uint32_t y = __shfl_up_sync(0xffffffffu, ipg, d);
            if (lane >= d) {
                itok = add(itok, x);
                ipg = add(ipg, y);
            }
        }
        if (lane == 31) {
            s_tok[warp] = itok;
            s_pg[warp] = ipg;
        }
        // the sums before this thread's requests (not itok - tok: a sum may have stopped)
        uint32_t cu = __shfl_up_sync(0xffffffffu, itok, 1), off = __shfl_up_sync(0xffffffffu, ipg, 1);
        if (lane == 0) cu = off = 0;
        __syncthreads();
        uint32_t before_tok = run_tok, before_pg = run_pg;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const uint32_t x = s_tok[w], y = s_pg[w];
            if (w < warp) {
                before_tok = add(before_tok, x);
                before_pg = add(before_pg, y);
            }
            run_tok = add(run_tok, x);
            run_pg = add(run_pg, y);
        }
        cu = add(cu, before_tok);
        off = add(off, before_pg);
        __syncthreads();  // s_tok / s_pg are rewritten by the next tile
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int64_t b = base + tid * kItems + i;
            if (b < B) {
                const int64_t end = static_cast<int64_t>(cu) + n[i];
                const bool served =
                    ok[i] && (need[i] == 0 || static_cast<int64_t>(off) + need[i] <= num_free) &&
                    (n[i] == 0 || end <= N);
                if (writer) {
                    seq_lens[b] = served ? c[i] + n[i] : (c[i] >= 0 && c[i] <= cap ? c[i] : 0);
                    cu_seqlens[b + 1] = static_cast<int32_t>(end < N ? end : N);
                    if (!served) record_device_error(err, kDevInvalidArg);
                    else if (need[i] > 0) atomicMax(&s_used, static_cast<int>(off) + need[i]);
                }
                if (n[i] > 0 && cu < t1 && end > t0) {
                    const int at = static_cast<int>((cu > t0 ? cu : t0) - t0);
                    s_cu[at] = static_cast<int>(cu);
                    s_count[at] = n[i];
                    s_cached[at] = c[i];
                    s_off[at] = static_cast<int>(off);
                    s_b[at] = served ? static_cast<int>(b) : -1;
                }
            }
            cu = add(cu, n[i]);
            off = add(off, need[i]);
        }
    }
    __syncthreads();
    if (writer && tid == 0) {
        cu_seqlens[0] = 0;
        *pages_used = s_used;
    }

    // running maximum of the starts (place + 1) over the CTA's tokens
    const int4 here = *reinterpret_cast<const int4 *>(s_b + tid * kItems);
    const int starts[kItems] = {here.x, here.y, here.z, here.w};
    int from[kItems];
    int m = 0;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        if (starts[i] >= -1) m = tid * kItems + i + 1;
        from[i] = m;
    }
    int im = m;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, im, d);
        if (lane >= d) im = max(im, x);
    }
    if (lane == 31) s_max[warp] = im;
    __syncthreads();
    int before = __shfl_up_sync(0xffffffffu, im, 1);
    if (lane == 0) before = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        if (w < warp) before = max(before, s_max[w]);

    const int64_t t = t0 + tid * kItems;
    int p[kItems];
    uint32_t r[kItems];
    bool placed[kItems];
    int64_t taken[kItems];  // the table's entry for a page that the token begins, -1: none
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int at = max(from[i], before) - 1;
        placed[i] = false;
        p[i] = -1;
        taken[i] = -1;
        if (t + i >= t1 || at < 0) continue;
        const int b = s_b[at], cached = s_cached[at];
        const int64_t j = t + i - s_cu[at];
        if (b < 0 || j >= s_count[at]) continue;
        placed[i] = true;
        uint32_t idx;
        page.divmod(static_cast<uint32_t>(cached + j), idx, r[i]);
        const int64_t entry = static_cast<int64_t>(b) * max_pages + idx;
        const int held = pages_of(cached);
        if (static_cast<int>(idx) < held) {
            p[i] = block_table[entry];
        } else {
            p[i] = free_pages[s_off[at] + static_cast<int>(idx) - held];
            if (r[i] == 0) taken[i] = entry;
        }
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i)
        if (taken[i] >= 0) block_table[taken[i]] = p[i];
    int slot[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        slot[i] = -1;
        if (!placed[i]) continue;
        if (p[i] >= 0 && p[i] < num_pages)
            slot[i] = static_cast<int>(static_cast<uint32_t>(p[i]) * page.d + r[i]);
        else
            record_device_error(err, kDevInvalidArg);
    }
    if (t + kItems <= t1) {
        *reinterpret_cast<int4 *>(slot_map + t) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
#pragma unroll
        for (int i = 0; i < kItems; ++i)
            if (t + i < t1) slot_map[t + i] = slot[i];
    }
}

}  // namespace

cudaError_t launch_page_plan(const int32_t *cached_lens, const int32_t *new_lens,
                             const int32_t *free_pages, int num_free, int32_t *block_table,
                             int max_pages, int B, int page_size, int num_pages,
                             int32_t *seq_lens, int32_t *cu_seqlens, int32_t *slot_map, int64_t N,
                             int32_t *pages_used, unsigned int *err, cudaStream_t s) {
    // 512 threads scan 2048 requests at once; up to half as many are done sooner by 256,
    // whose barriers are cheaper (2048 requests, 260 thousand tokens: 6.8 us, 9.0 with 256;
    // 8 requests: 3.7 us, 4.4 with 512)
    auto kern = B <= 1024 ? plan_kernel<256> : plan_kernel<512>;
    const int threads = B <= 1024 ? 256 : 512, tile = threads * kItems;
    const int64_t ctas = N > 0 ? (N + tile - 1) / tile : 1;
    return launch_early(kern, dim3(static_cast<unsigned>(ctas)), threads, 0, s, cached_lens, new_lens,
                        free_pages, num_free, block_table, max_pages, B,
                        FastDiv(static_cast<uint32_t>(page_size)), num_pages, seq_lens, cu_seqlens,
                        slot_map, N, pages_used, err);
}

}  // namespace kda
