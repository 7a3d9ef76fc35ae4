// kda_page_plan.cu -- block tables and slot maps from request lengths.
//
// The whole step is two exclusive prefix sums over the requests (new tokens:
// the rows of cu_seqlens; pages needed: the place in the free list) and a map
// from each new token to its request.  One launch: a CTA owns 1024 consecutive
// tokens and scans the requests itself, in tiles of 1024, until the sum passes
// its tokens (B is at most some thousands, 8 bytes each, out of L2; a second
// launch or a look-back over other CTAs' sums would cost more than the scan).
// A request that meets the CTA's tokens leaves its record at the place of its
// first token there; starts are distinct, so a running maximum over the 1024
// places then gives every token its request without a search.  A page's table
// entry is written by the token at offset 0 of it: each page taken has one.
#include "kda_internal.cuh"
#include "kda_paged.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kItems = 4;                  // requests, then tokens, per thread
constexpr int kTile = kThreads * kItems;
constexpr int kWarps = kThreads / 32;

struct Start {       // a request at its first token in the CTA's range
    int cu, count;   // its first row (may lie before the range) and its tokens
    int cached;
    int off, held;   // its place in the free list; its pages before the step
    int b;           // -1: refused
};

__global__ void __launch_bounds__(kThreads) plan_kernel(
    const int32_t *__restrict__ cached_lens, const int32_t *__restrict__ new_lens,
    const int32_t *__restrict__ free_pages, int num_free, int32_t *block_table, int max_pages,
    int B, FastDiv page, int num_pages, int32_t *__restrict__ seq_lens,
    int32_t *__restrict__ cu_seqlens, int32_t *__restrict__ slot_map, int64_t N,
    int32_t *__restrict__ pages_used, unsigned int *err) {
    __shared__ Start s_start[kTile];
    __shared__ int s_has[kTile];           // place + 1 where a request starts, else 0
    __shared__ int64_t s_tok[kWarps], s_pg[kWarps];
    __shared__ int s_max[kWarps];
    __shared__ int s_used;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool writer = blockIdx.x == 0;   // of what there is one of per request
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTile;
    const int64_t t1 = t0 + kTile < N ? t0 + kTile : N;
    const int64_t cap = static_cast<int64_t>(max_pages) * page.d;

#pragma unroll
    for (int i = 0; i < kItems; ++i) s_has[tid + i * kThreads] = 0;
    if (tid == 0) s_used = 0;
    __syncthreads();

    int64_t run_tok = 0, run_pg = 0;
    for (int64_t base = 0; base < B; base += kTile) {
        if (!writer && run_tok >= t1) break;
        int c[kItems], n[kItems], need[kItems];
        bool ok[kItems];
        int64_t tok = 0, pg = 0;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int64_t b = base + tid * kItems + i;
            c[i] = b < B ? cached_lens[b] : 0;
            n[i] = b < B ? new_lens[b] : 0;
            ok[i] = c[i] >= 0 && n[i] >= 0 && static_cast<int64_t>(c[i]) + n[i] <= cap;
            n[i] = n[i] > 0 ? n[i] : 0;
            need[i] = 0;
            // c + n <= max_pages * page_size, which need not fit an int: the page
            // count of a sum past 2^31 - 1 is refused below through num_pages
            if (ok[i]) {
                const int64_t total = static_cast<int64_t>(c[i]) + n[i];
                ok[i] = total <= INT32_MAX;
                if (ok[i])
                    need[i] = static_cast<int>(
                        (total == 0 ? 0 : page.div(static_cast<uint32_t>(total - 1)) + 1) -
                        (c[i] == 0 ? 0 : page.div(static_cast<uint32_t>(c[i] - 1)) + 1));
            }
            tok += n[i];
            pg += need[i];
        }
        // exclusive prefix sums over the tile
        int64_t itok = tok, ipg = pg;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t a = __shfl_up_sync(0xffffffffu, itok, d);
            const int64_t e = __shfl_up_sync(0xffffffffu, ipg, d);
            if (lane >= d) {
                itok += a;
                ipg += e;
            }
        }
        if (lane == 31) {
            s_tok[warp] = itok;
            s_pg[warp] = ipg;
        }
        __syncthreads();
        int64_t cu = run_tok + itok - tok, off = run_pg + ipg - pg;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) {
                cu += s_tok[w];
                off += s_pg[w];
            }
            run_tok += s_tok[w];
            run_pg += s_pg[w];
        }
        __syncthreads();  // s_tok / s_pg are rewritten by the next tile
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int64_t b = base + tid * kItems + i;
            if (b < B) {
                const bool served = ok[i] && (need[i] == 0 || off + need[i] <= num_free) &&
                                    (n[i] == 0 || cu + n[i] <= N);
                if (writer) {
                    seq_lens[b] = served ? c[i] + n[i] : (c[i] >= 0 && c[i] <= cap ? c[i] : 0);
                    const int64_t end = cu + n[i];
                    cu_seqlens[b + 1] = static_cast<int32_t>(end < N ? end : N);
                    if (!served) record_device_error(err, kDevInvalidArg);
                    else if (need[i] > 0) atomicMax(&s_used, static_cast<int>(off + need[i]));
                }
                if (n[i] > 0 && cu < t1 && cu + n[i] > t0) {
                    const int at = static_cast<int>((cu > t0 ? cu : t0) - t0);
                    Start &st = s_start[at];
                    st.cu = static_cast<int>(cu);
                    st.count = n[i];
                    st.cached = c[i];
                    st.off = served ? static_cast<int>(off) : 0;
                    st.held = c[i] <= 0 ? 0 : static_cast<int>(page.div(c[i] - 1) + 1);
                    st.b = served ? static_cast<int>(b) : -1;
                    s_has[at] = at + 1;
                }
            }
            cu += n[i];
            off += need[i];
        }
    }
    __syncthreads();
    if (writer && tid == 0) {
        cu_seqlens[0] = 0;
        *pages_used = s_used;
    }

    // running maximum of the starts over the CTA's tokens
    int at[kItems];
    int m = 0;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int h = s_has[tid * kItems + i];
        m = h > m ? h : m;
        at[i] = m;
    }
    int im = m;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, im, d);
        if (lane >= d && a > im) im = a;
    }
    if (lane == 31) s_max[warp] = im;
    __syncthreads();
    int before = __shfl_up_sync(0xffffffffu, im, 1);
    if (lane == 0) before = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        if (w < warp && s_max[w] > before) before = s_max[w];

    int slot[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int64_t t = t0 + tid * kItems + i;
        const int from = at[i] > before ? at[i] : before;
        slot[i] = -1;
        if (t >= t1 || from == 0) continue;
        const Start &st = s_start[from - 1];
        const int64_t j = t - st.cu;
        if (st.b < 0 || j >= st.count) continue;
        uint32_t idx, r;
        page.divmod(static_cast<uint32_t>(st.cached + j), idx, r);
        const int64_t entry = static_cast<int64_t>(st.b) * max_pages + idx;
        int p;
        if (static_cast<int>(idx) < st.held) {
            p = block_table[entry];
        } else {
            p = free_pages[st.off + static_cast<int>(idx) - st.held];
            if (r == 0) block_table[entry] = p;
        }
        if (p >= 0 && p < num_pages)
            slot[i] = static_cast<int>(static_cast<uint32_t>(p) * page.d + r);
        else
            record_device_error(err, kDevInvalidArg);
    }
    const int64_t t = t0 + tid * kItems;
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
    const int64_t ctas = N > 0 ? (N + kTile - 1) / kTile : 1;
    plan_kernel<<<static_cast<unsigned>(ctas), kThreads, 0, s>>>(
        cached_lens, new_lens, free_pages, num_free, block_table, max_pages, B,
        FastDiv(static_cast<uint32_t>(page_size)), num_pages, seq_lens, cu_seqlens, slot_map, N,
        pages_used, err);
    return cudaGetLastError();
}

}  // namespace kda
