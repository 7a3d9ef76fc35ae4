// kda_paged_tree.cuh -- softmax attention of a tree of drafted tokens per sequence over a paged
// key-value cache that holds the drafted tokens' keys and values too.
//
// Node i of a sequence with L keys, n of them drafted, sees the C = L - n keys of the context
// and the drafted key j (at position C + j) where bit j of its word is set:
//
//   s_j = scale <q_i, k_j>,  m = max_j s_j,  l = sum_j e^{s_j - m}
//   o = sum_j e^{s_j - m} v_j / l,  lse = m + log l
//
// over the keys j that it sees; a node that sees none has o = 0 and lse = -inf.  Powers of two
// throughout: the scores carry log2 e.
//
// Bound: a key and a value are 4 D bytes (2 D in 8 bits) and meet R = n G rows (G query heads
// to a key head) in 4 D R flops: HBM up to some R = 300 of them (150), the tensor cores' full
// rate beyond.  That rate needs tcgen05: the rows are the 128 rows of a product, the keys
// (then the channels) its columns.
//
// Split.  A unit is (sequence, key head, up to kM x 128 rows); its keys are cut in tiles of 128
// (64 at 256 channels).  The tiles of all units form one list, of which each CTA, one an SM,
// takes an equal, contiguous piece; what is cut between CTAs is joined by a second, small
// kernel that is set up with the first.
//
// A CTA.  Two warps copy the keys and two the values of its piece into two rings, rows swizzled
// as the products read them: by TMA boxes of a page's keys, one instruction for up to 64 of
// them (16-byte copies took the warps longer than a product), or 16 bytes at a time where pages
// do not divide so or a tile is not full.  An 8-bit cache comes raw and is widened to fp16, which
// holds every e4m3 value.  Two warps issue the products: S = Q K^T from shared memory into one of
// two to four score buffers in tensor memory, and O += P V with P from there and V from shared
// memory.  Two warpgroups turn scores into weights in place, a thread a row (a lane of tensor
// memory), each every second step, so that one's exponentials run beside the other's loads and
// maxima.  A row's weights are relative to a reference that follows its maximum only when that has
// grown by 2^7 (2^3 over an 8-bit cache): O is then rescaled, which waits for the last product (at
// every growth, some row of a warp would grow in most tiles).
//
// Measured (floor): 1 request of 8 nodes, 301 keys 13.5 us; 32 requests of 16 nodes, 500-6000 keys, 8
// heads to each of 8 key heads 81 us (48); 64 of 1-21 nodes over 8 bits 265 us (68); 12 of 64 nodes,
// 12 heads to a key head 230-237 us (87).  The second case at 64 channels 64 us (24), at 256 151 us (97);
// over 8 bits 69 (13), 99 (26) and 172 us (51).  The tensor cores are busy for 40 to 50 % of it: what bounds
// it is the chain from scores over weights (2.4k cycles a tile) to outputs, as long as two products,
// with the score buffers that tensor memory has room for.  Half of a step's keys for each warpgroup, or a
// quarter for each of four, was slower (85 and 93 us in the second case).
//
// Precision: scores, maxima and sums in fp32.  For the product with the values a weight is two
// words: bf16 numbers, 16 bits together (one would leave up to 2^-8 of every weight, as much as
// the output's own rounding); over an 8-bit cache fp16 numbers of the weight times 2^12, which
// keep it to 2^-37 of the largest, with the queries scaled to fp16's range by a power of
// two a row.  The products' sums in tensor memory are cut off at each step of 16 keys:
// 2^-24 of the sum, below the output's rounding by far.
//
// What is not finite.  A weight of 0 times an infinite or NaN value is NaN, and so is 0 (a
// weight's second word) times an infinite one.  So a row whose output is not finite although
// its weights are is computed again over the keys that it sees (row_again), in 8 channels at a time:
// that of a whole unit by the warps that had it, once the CTA has nothing else to do, that of
// a cut one by the second kernel.  In neither place does another warp wait for it with a limit.  (One NaN
// that 64 nodes x 8 heads see in 8192 keys, beside 64 short requests: 45 ms.)
#pragma once

#include <cfloat>

#include <cuda_fp16.h>

#include "kda_chunk_common.cuh"
#include "kda_f32x2.cuh"
#include "kda_sm100.cuh"
#include "kda_tree.cuh"

namespace kda {
namespace treeatt {

using namespace sm100;

constexpr int kMaxCtas = 160;  // sizes the workspace; more SMs stay idle
constexpr int kSoftWarps = 8, kCopyWarps = 4;
constexpr int kThreads = 512;   // four warpgroups: weights (two), copies, products (one thread)
// Their registers, of the 512 x 128 that the block is launched with: 2 x 176 + 96 + 56 = 504.
constexpr int kSoftRegs = 176, kCopyRegs = 96, kProductRegs = 56;
static_assert(2 * kSoftRegs + kCopyRegs + kProductRegs <= 512, "registers of the block");
constexpr uint32_t kMaxPolls = 1u << 20;

__host__ __device__ constexpr int min_of(int a, int b) { return a < b ? a : b; }

// m tiles of a unit: two where a sequence may have more than 128 rows and tensor memory has
// room (2 x 128 columns of scores, 128 a tile of outputs).
inline int m_tiles(int max_nodes, int group, int head_dim) {
    return head_dim <= 128 && static_cast<int64_t>(max_nodes) * group > 128 ? 2 : 1;
}

inline size_t slot_bytes(int m, int head_dim) {
    return static_cast<size_t>(m) * 128 * (head_dim + 2) * 4;
}

struct Args {
    TreeAttention t;
    FastDiv group;
    float *ml;   // [CTAs][2][rows][2]
    float *cut;  // [CTAs][2][D / 4][rows][4]
    // the cache's halves as [pages][heads][tokens][channels]: boxes of `box` tokens of a page
    CUtensorMap map_k, map_v;
    int box;
};

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int kD_, bool kFp8_, int kM_>
struct Shape {
    static constexpr int kD = kD_, kM = kM_;
    static constexpr bool kFp8 = kFp8_;
    static constexpr int kRows = kM * 128;
    static constexpr int kKeys = kD == 256 ? 64 : 128;
    static constexpr int kTile = kKeys * kD * 2;  // as an operand
    // places in the list of a tile of one m tile, of two, and of beginning and ending a unit
    static constexpr int kOneCost = kM == 1 ? 1 : 2, kTwoCost = 3, kUnitCost = kM == 1 ? 3 : 10;
    static constexpr int kRaw = kTile / 2;        // of an 8-bit cache, as copied
    static constexpr int kQ = kRows * kD * 2;
    static constexpr int kRoom = 224 * 1024 - kQ;
    // rings of operands, and of raw tiles of keys and of values, in flight between copy and widening
    static constexpr int kOps = kRoom / kTile;
    static constexpr int kNK = kFp8 ? (kD == 256 ? 1 : 2) : min_of(6, (kOps + 1) / 2);
    static constexpr int kNV = kFp8 ? (kTile <= 16 * 1024 ? 2 : 1) : min_of(6, kOps / 2);
    static constexpr int kNR = kFp8 ? min_of(4, (kRoom - (kNK + kNV) * kTile) / kRaw / 2) : 0;
    static constexpr int kOffK = kQ, kOffV = kOffK + kNK * kTile, kOffRaw = kOffV + kNV * kTile;
    static constexpr int kOffSmall = kOffRaw + 2 * kNR * kRaw;
    // score buffers in tensor memory, then the outputs
    static constexpr int kBufs = min_of(4, (512 - kM * kD) / kKeys), kColO = kBufs * kKeys;
    // a row's reference follows its maximum when that has grown by 2^kSlack; weights are
    // 2^kShift times themselves (fp16 ends at 2^16)
    static constexpr float kSlack = kFp8 ? 3.f : 7.f, kShift = kFp8 ? 12.f : 0.f;
    static_assert(kBufs >= 2, "tensor memory");
    static_assert(!kFp8 || kNR >= 2, "tiles in flight");

    // tiles whose rows' validity is kept: more than lie between a copy and its weights
    static constexpr int kTilesAhead = 16;
    static_assert(kTilesAhead > kNK + kNR + kBufs, "tiles ahead");

    struct Small {  // what lies behind the tiles
        uint64_t qfull, kfull[kNK], kempty[kNK], vfull[kNV], vempty[kNV], sfull[kBufs], pfull[kBufs][2], pfree[kBufs], scored, done, ofree, drain[2];
        int64_t warp_sum[kThreads / 32], place[2];
        // by row: the reference that a warpgroup hands to the other (top[0]), and what they exchange in the end
        float top[2][128];
        // by row: the halves' largest queries of the next unit.  Apart from `top`: one warpgroup comes to
        // them while the other still reads its last step's reference.
        float q_top[2][128];
        uint64_t raw[2][2][kNR > 0 ? kNR : 1];  // keys and values, halves of rows
        uint32_t valid[kTilesAhead][kKeys / 32];  // which rows of a tile are keys
        uint32_t tmem;
        int begin[kSoftWarps][4];                 // where the CTA's piece begins: a warp's copy
        int64_t places[kSoftWarps];
    };
    static constexpr int kSmem = kOffSmall + static_cast<int>(sizeof(Small));
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^e, -126 <= e <= 127 (a power further out is taken in two factors).
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((e + 127) << 23); }

// x, or the least normal number where x is below it; a NaN stays.
__device__ __forceinline__ float at_least_normal(float x) { return x < FLT_MIN ? FLT_MIN : x; }

template <bool kF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (kF16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}
template <bool kF16>
__device__ __forceinline__ float2 unpack2(uint32_t x) {
    if constexpr (kF16) return __half22float2(*reinterpret_cast<const __half2 *>(&x));
    else return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x) {
    uint32_t y;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(static_cast<uint16_t>(x)));
    return y;
}

// ---- a row in fp32 arithmetic --------------------------------------------------------------

// Eight neighbouring values of a row, widened.
template <bool kFp8>
__device__ __forceinline__ void load_eight(const uint8_t *p, float (&y)[8]) {
    uint32_t w[4];
    if constexpr (kFp8) {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        w[0] = e4m3x2_to_f16x2(x.x);
        w[1] = e4m3x2_to_f16x2(x.x >> 16);
        w[2] = e4m3x2_to_f16x2(x.y);
        w[3] = e4m3x2_to_f16x2(x.y >> 16);
    } else {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        w[0] = x.x;
        w[1] = x.y;
        w[2] = x.z;
        w[3] = x.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<kFp8>(w[i]);
        y[2 * i] = f.x;
        y[2 * i + 1] = f.y;
    }
}

// The average of values over two sets of keys, weights relative to references.  (Averages, so that they
// are as large as the values.)
__device__ __forceinline__ void join_averages(float &m, float &l, float (&acc)[8], float m1, float l1, const float (&acc1)[8]) {
    const float to = m1 > m || m1 != m1 ? m1 : m, ref = to == -INFINITY ? 0.f : to;
    const float w = l * exp2f(m - ref), w1 = l1 * exp2f(m1 - ref);
    m = to;
    l = w + w1;
    if (l == 0.f) return;
    const float part = w / l, part1 = w1 / l;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = part * acc[i] + part1 * acc1[i];
}

// Channels d .. d + 7 of a row's output, by one warp, in fp32 arithmetic over the keys that the row
// sees: each lane has every 32nd of them.  s_q: [kD], the warp's.
template <int kD, bool kFp8>
__device__ __noinline__ void row_again(const TreeAttention &a, int b, int64_t row, int qh, int n, int len, int d,
                                       float *s_q) {
    constexpr int kSize = kFp8 ? 1 : 2;
    const int lane = threadIdx.x & 31, h = qh / a.group, context = len - n;
    const uint64_t word = a.ancestors[row];
    const float c = a.scale * kLog2e * (a.cache.k_scale != nullptr ? a.cache.k_scale[h] : 1.f);
    for (int i = lane; i < kD; i += 32)
        s_q[i] = __bfloat162float(a.q[row * a.q_row_stride + qh * kD + i]);
    __syncwarp();
    float m = -INFINITY, l = 0.f, acc[8] = {};
    for (uint32_t j = lane; j < static_cast<uint32_t>(len); j += 32) {
        const int drafted = static_cast<int>(j) - context;
        if (drafted >= 0 && !((word >> drafted) & 1)) continue;
        uint32_t idx, in_page;
        a.cache.page.divmod(j, idx, in_page);
        const int page = a.block_table[static_cast<int64_t>(b) * a.max_pages + idx];
        if (page < 0 || page >= a.cache.num_pages) continue;
        const int64_t off = page * a.cache.page_stride + in_page * a.cache.token_stride + h * a.cache.head_stride;
        float s = 0.f, x[8];
#pragma unroll 4
        for (int i = 0; i < kD; i += 8) {
            load_eight<kFp8>(a.cache.k + off + i * kSize, x);
#pragma unroll
            for (int k = 0; k < 8; ++k) s += s_q[i + k] * x[k];
        }
        load_eight<kFp8>(a.cache.v + off + d * kSize, x);
        s *= c;
        // (a score of -inf has no weight)
        join_averages(m, l, acc, s, s == -INFINITY ? 0.f : 1.f, x);
    }
#pragma unroll 1
    for (int x = 16; x > 0; x >>= 1) {
        float other[8];
        const float m1 = __shfl_xor_sync(0xffffffffu, m, x), l1 = __shfl_xor_sync(0xffffffffu, l, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) other[i] = __shfl_xor_sync(0xffffffffu, acc[i], x);
        join_averages(m, l, acc, m1, l1, other);
    }
    if (lane == 0) {
        const float vs = a.cache.v_scale != nullptr ? a.cache.v_scale[h] : 1.f;
        uint32_t y[4];
#pragma unroll
        for (int i = 0; i < 8; i += 2) y[i / 2] = l == 0.f ? 0u : pack2<false>(acc[i] * vs, acc[i + 1] * vs);
        *reinterpret_cast<uint4 *>(a.o + (row * a.q_heads + qh) * kD + d) = make_uint4(y[0], y[1], y[2], y[3]);
    }
    __syncwarp();
}

// ---- the list of tiles ---------------------------------------------------------------------

// a / b, both 0 or above: in 32 bits where they fit, which nearly all lists do.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// A place in the list, and the way from there.  A unit takes kUnitCost places of the list, then as
// many for each of its tiles as they cost (measured: a tile of two m tiles takes one and a half
// times one's; beginning and ending a unit takes three).
template <class S>
struct Cursor {
    int b, h, rg;
    int n, len, rows, groups, tiles;  // of the sequence; rows = n G
    int64_t first;                    // its first row
    int at;                           // place in the unit
    int t, t1;                        // the tiles taken of it
    int64_t left;                     // places to take

    __device__ __forceinline__ void request(const TreeAttention &a, int i) {
        b = i;
        const TreeRows r = tree_rows(a.cu, b, a.N, a.max_nodes);
        len = a.seq_lens[b];
        first = r.first;
        n = r.n;
        if (len < n || len > static_cast<int64_t>(a.max_pages) * a.cache.page.d) n = 0;
        measure(a);
    }
    // The request of lane `src`'s cursor.
    __device__ __forceinline__ void request_of(const TreeAttention &a, int src, int i) {
        b = i;
        first = __shfl_sync(0xffffffffu, static_cast<int>(first), src);
        n = __shfl_sync(0xffffffffu, n, src);
        len = __shfl_sync(0xffffffffu, len, src);
        measure(a);
    }
    __device__ __forceinline__ void measure(const TreeAttention &a) {
        rows = n * a.group;
        groups = (rows + S::kRows - 1) / S::kRows;
        tiles = n == 0 ? 0 : static_cast<int>((static_cast<uint32_t>(len) + S::kKeys - 1) / S::kKeys);
    }
    // m tiles of the sequence's i-th group of rows, places of a tile of them and of their unit
    __device__ __forceinline__ int m_tiles(int i) const { return S::kM == 2 && rows - i * S::kRows > 128 ? 2 : 1; }
    __device__ __forceinline__ int cost(int i) const { return m_tiles(i) == 2 ? S::kTwoCost : S::kOneCost; }
    __device__ __forceinline__ int64_t unit(int i) const {
        return static_cast<int64_t>(tiles) * cost(i) + S::kUnitCost;
    }
    __device__ __forceinline__ int64_t head() const {
        return (groups - 1) * unit(0) + unit(groups - 1);  // all groups but the last are full
    }
    __device__ __forceinline__ int64_t places(const TreeAttention &a) const {
        return tiles == 0 ? 0 : a.cache.heads * head();
    }
    // Place `i` of the sequence's part of the list.
    __device__ __forceinline__ void seek(int64_t i) {
        h = static_cast<int>(quotient(i, head()));
        i -= h * head();
        rg = groups == 1 ? 0 : min(static_cast<int>(quotient(i, unit(0))), groups - 1);
        at = static_cast<int>(i - rg * unit(0));
    }
    __device__ __forceinline__ void next_unit(const TreeAttention &a) {
        at = 0;
        if (++rg < groups) return;
        rg = 0;
        if (++h < a.cache.heads) return;
        h = 0;
        do request(a, b + 1);  // (there is one: places are left)
        while (tiles == 0);
    }
    // The first tile that begins at place i of the unit or behind it.
    __device__ __forceinline__ int tile_at(int i) const {
        return (max(i - S::kUnitCost, 0) + cost(rg) - 1) / cost(rg);
    }
    // The next tiles [t, t1) of one unit; false at the end.
    __device__ __forceinline__ bool take(const TreeAttention &a) {
        while (left > 0) {
            const int end = static_cast<int>(unit(rg));
            if (at == end) {
                next_unit(a);
                continue;
            }
            const int to = static_cast<int>(min(static_cast<int64_t>(end), at + left));
            t = tile_at(at);
            t1 = tile_at(to);
            left -= to - at;
            at = to;
            if (t1 > t) return true;
        }
        return false;
    }
};

// The block's way through the list; every thread of the block calls it.  begin(c): the first
// place of piece c.
struct List {
    int64_t total;
    int pieces;

    __device__ __forceinline__ int64_t begin(int64_t c) const { return quotient(total * c, pieces); }
    __device__ __forceinline__ int piece_of(int64_t at) const {
        return static_cast<int>(quotient((at + 1) * pieces - 1, total));
    }
};

template <class S, int kWarps>
__device__ __forceinline__ int64_t scan_sum(int64_t x, int64_t *s_warp, int64_t &before) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t sum = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    int64_t all = 0;
    before = sum - x;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const int64_t y = s_warp[w];
        if (w < warp) before += y;
        all += y;
    }
    return all;
}

// A tile begins in every piece that lies within a unit's tiles: the join counts on it.
template <class S>
__device__ __forceinline__ void cut_list(List &list, int ctas) {
    const int64_t most = quotient(list.total, S::kM == 1 ? S::kOneCost : S::kTwoCost);
    list.pieces = static_cast<int>(most < ctas ? (most < 1 ? 1 : most) : ctas);
}

// The list, and where place `at(list)` of it lies: c, or false past the end.  s_place: shared.
template <class S, int kWarps, class At>
__device__ __forceinline__ bool find_place(const TreeAttention &a, int ctas, int64_t *s_warp,
                                           int64_t (&s_place)[2], At at, List &list, Cursor<S> &c) {
    const int tid = threadIdx.x, lane = tid & 31;
    list.total = 0;
    if (a.B <= 32) {  // every warp by itself, a lane a request: no barriers, one trip to memory
        int64_t mine = 0;
        c.n = c.len = 0;
        c.first = 0;
        if (lane < a.B) {
            c.request(a, lane);
            mine = c.places(a);
        }
        int64_t end = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, end, d);
            if (lane >= d) end += y;
        }
        list.total = __shfl_sync(0xffffffffu, end, 31);
        cut_list<S>(list, ctas);
        const int64_t place = at(list);
        const uint32_t there = __ballot_sync(0xffffffffu, place >= end - mine && place < end);
        if (there == 0) return false;
        const int src = __ffs(static_cast<int>(there)) - 1;
        const int64_t before = __shfl_sync(0xffffffffu, end - mine, src);
        c.request_of(a, src, src);
        c.seek(place - before);
        return true;
    }
    constexpr int kStep = kWarps * 32;
    int64_t mine = 0, before = 0;
    for (int b0 = 0; b0 < a.B; b0 += kStep) {
        mine = 0;
        if (b0 + tid < a.B) {
            c.request(a, b0 + tid);
            mine = c.places(a);
        }
        list.total += scan_sum<S, kWarps>(mine, s_warp, before);
    }
    cut_list<S>(list, ctas);
    if (tid == 0) s_place[0] = -1;
    __syncthreads();
    const int64_t place = at(list);
    int64_t base = 0;
    for (int b0 = 0; b0 < a.B; b0 += kStep) {
        if (a.B > kStep) {  // else the first pass's values stand
            mine = 0;
            if (b0 + tid < a.B) {
                c.request(a, b0 + tid);
                mine = c.places(a);
            }
            const int64_t all = scan_sum<S, kWarps>(mine, s_warp, before);
            before += base;
            base += all;
        }
        if (b0 + tid < a.B && place >= before && place < before + mine) {
            s_place[0] = b0 + tid;
            s_place[1] = place - before;
        }
    }
    __syncthreads();
    if (s_place[0] < 0) return false;
    c.request(a, static_cast<int>(s_place[0]));
    c.seek(s_place[1]);
    return true;
}

// ---- products ------------------------------------------------------------------------------

// D[tmem] (+)= A[tmem] * B[smem], 16-bit operands of one type, fp32 sums; by one lane of a
// converged warp.
__device__ __forceinline__ void mma_f16_ts_w(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrives on `bar` when this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// 16 bytes to shared memory, or zeros (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0)
                 : "memory");
}

// A box of a page to shared memory; x a multiple of 64 elements.
__device__ __forceinline__ void load_box(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int token,
                                         int head, int page) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(token), "r"(head), "r"(page), "r"(smem_addr(bar))
        : "memory");
}

// The two warps of a lane quarter.
__device__ __forceinline__ void pair_barrier(int quarter) {
    asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
}
// One of them (of warpgroup wg) waits for what the other has done; the other says so.
__device__ __forceinline__ void pair_wait(int quarter, int wg) {
    asm volatile("bar.sync %0, 64;" ::"r"(5 + wg * 4 + quarter) : "memory");
}
__device__ __forceinline__ void pair_arrive(int quarter, int wg) {
    asm volatile("bar.arrive %0, 64;" ::"r"(5 + (wg ^ 1) * 4 + quarter) : "memory");
}

template <int kRegs>
__device__ __forceinline__ void take_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void leave_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Which of the 64 keys from drafted place d (below 0: still context) on a word sees.
__device__ __forceinline__ uint64_t seen_from(uint64_t word, int d) {
    if (d <= -64) return ~uint64_t{0};
    if (d < 0) return (word << -d) | bits_below(-d);
    return d >= 64 ? 0 : word >> d;
}

// A wait, by a whole warp, whose lanes agree and go on together.  One that runs out is an
// error, and the role that waited ends (the others' waits run out too).
struct Waits {
    unsigned int *err;
    bool ok;

    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) {
        if (ok && !mbar_wait_bounded(bar, parity, kMaxPolls)) {
            record_device_error(err, kDevTimeout);
            ok = false;
        }
        ok = __all_sync(0xffffffffu, ok);
        return ok;
    }
};

// ---- the kernel ------------------------------------------------------------------------------

template <class S>
__global__ void __launch_bounds__(kThreads, 1) tree_attention_kernel(const __grid_constant__ Args args) {
    constexpr int kD = S::kD, kM = S::kM, kKeys = S::kKeys;
    constexpr bool kFp8 = S::kFp8;
    constexpr int kWarps = kThreads / 32;
    extern __shared__ __align__(1024) uint8_t smem[];  // swizzled tiles: 1024-byte groups of rows
    typename S::Small &sm = *reinterpret_cast<typename S::Small *>(smem + S::kOffSmall);
    const TreeAttention &a = args.t;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = smem_addr(smem);

    if (warp == kSoftWarps + kCopyWarps) tmem_alloc(&sm.tmem, 512);
    if (tid == 32 && args.box > 0) {
        prefetch_tmap(&args.map_k);
        prefetch_tmap(&args.map_v);
    }
    if (tid == 0) {
        mbar_init(&sm.qfull, kFp8 ? kSoftWarps : 64);
        for (int i = 0; i < S::kNK; ++i) {
            // two warps' threads when they have widened their rows; else their copies, and a
            // thread of each for what it has said beside them
            mbar_init(&sm.kfull[i], kFp8 ? 64 : 66);
            mbar_init(&sm.kempty[i], 1);
        }
        for (int i = 0; i < S::kNV; ++i) {
            mbar_init(&sm.vfull[i], kFp8 ? 64 : 66);
            mbar_init(&sm.vempty[i], 1);
        }
        for (int i = 0; i < 4 * S::kNR; ++i) mbar_init(&sm.raw[0][0][0] + i, 33);
        for (int i = 0; i < S::kBufs; ++i) {
            mbar_init(&sm.sfull[i], 1);
            mbar_init(&sm.pfull[i][0], kSoftWarps / 2);
            mbar_init(&sm.pfull[i][1], kSoftWarps / 2);
            mbar_init(&sm.pfree[i], 1);
        }
        mbar_init(&sm.scored, 1);
        mbar_init(&sm.done, 1);
        mbar_init(&sm.ofree, kSoftWarps);
        mbar_init(&sm.drain[0], 1);
        mbar_init(&sm.drain[1], 1);
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    wait_for_kernel_before();

    List list;
    Cursor<S> at = {};
    if (find_place<S, kWarps>(a, gridDim.x, sm.warp_sum, sm.place, [&](const List &l) {
            return static_cast<int>(blockIdx.x) < l.pieces ? l.begin(blockIdx.x) : l.total;
        }, list, at))
        at.left = list.begin(blockIdx.x + int64_t{1}) - list.begin(blockIdx.x);

    if (warp < kSoftWarps) {
        // ---- queries in, weights, outputs ------------------------------------------------
        take_registers<kSoftRegs>();
        // (A wait that runs out ends no loop here: the other warpgroup's warps count on this one's.)
        Waits wait = {a.err, true};
        const int wg = warp >> 2, quarter = warp & 3, lrow = quarter * 32 + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        uint32_t step = 0, tiles_done = 0, units = 0;
        // Queries for an 8-bit cache, as fp16: a unit's, this lane's half of its rows, scaled by a
        // power of two that puts a row's largest value below 2^15; exps: those powers.
        int exps[kM], exps_next[kM];
        auto queries = [&](const Cursor<S> &u, int (&exps)[kM]) {
            constexpr int kPieces = kD / 16;  // 16-byte pieces of half a row
#pragma unroll
            for (int t = 0; t < kM; ++t) {
                const int rr = u.rg * S::kRows + t * 128 + lrow;
                exps[t] = 0;
                if (rr - lane >= u.rows) continue;
                const bool real = rr < u.rows;
                uint32_t node, head;
                args.group.divmod(rr, node, head);
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    a.q + (real ? (u.first + node) * a.q_row_stride + (u.h * a.group + static_cast<int>(head)) * kD : 0) +
                    wg * (kD / 2));
                uint32_t top = 0;
                if (real)
#pragma unroll 4
                    for (int i = 0; i < kPieces; ++i) {
                        const uint4 x = src[i];
                        for (const uint32_t y : {x.x, x.y, x.z, x.w})
                            top = max(top, max(y & 0x7fff0000u, (y << 16) & 0x7fff0000u));
                    }
                sm.q_top[wg][lrow] = __uint_as_float(top);
                pair_barrier(quarter);
                top = max(top, __float_as_uint(sm.q_top[wg ^ 1][lrow]));
                pair_barrier(quarter);
                exps[t] = min(max(static_cast<int>(top >> 23), 15), 254) - 127 - 14;
                const float up = power_of_two(-exps[t]);
                if (real)
#pragma unroll 4
                    for (int i = 0; i < kPieces; ++i) {
                        uint4 x = src[i];
                        uint32_t *y = reinterpret_cast<uint32_t *>(&x);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 f = unpack2<false>(y[k]);
                            y[k] = pack2<true>(f.x * up, f.y * up);
                        }
                        const int ch = wg * kPieces + i;
                        *reinterpret_cast<uint4 *>(smem + t * (128 * kD * 2) + (ch >> 3) * (128 * 128) + lrow * 128 +
                                                   (((ch & 7) ^ (lrow & 7)) << 4)) = x;
                    }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.qfull);
        };
        if (lane == 0) {
            int *begin = sm.begin[warp];
            begin[0] = at.b;
            begin[1] = at.h;
            begin[2] = at.rg;
            begin[3] = at.at;
            sm.places[warp] = at.left;
        }
        bool again = false;  // a row of the warp's, of a whole unit, is not finite although its weights are
        bool more = at.take(a);
        if (kFp8 && more) queries(at, exps);
        while (more) {
            const int m_used = at.m_tiles(at.rg);
            const int tiles = at.t1 - at.t, steps = tiles * m_used;
            // This warpgroup has every second step: of two m tiles always the same one, of one
            // every second tile.
            const int i0 = (step + wg) & 1, mt = m_used == 1 ? 0 : i0;
            const int rr = at.rg * S::kRows + mt * 128 + lrow;  // this lane's row
            const bool some = rr - lane < at.rows, real = rr < at.rows;
            uint32_t node, head;
            args.group.divmod(rr, node, head);
            const int64_t row = at.first + node;
            const int qh = at.h * a.group + static_cast<int>(head);
            const uint64_t word = real ? a.ancestors[row] & bits_below(at.n) : 0;
            // what turns the row's products into scores: above 0 (the queries of a negative scale
            // are negated by the product)
            float c = at_least_normal(fabsf(a.scale * kLog2e * (a.cache.k_scale != nullptr ? a.cache.k_scale[at.h] : 1.f)));
            if constexpr (kFp8) c = at_least_normal(c * power_of_two(mt == 0 ? exps[0] : exps[kM - 1]));
            float m = -INFINITY, l = 0.f;
            Cursor<S> next = at;
            more = next.take(a);

            for (int i = i0; i < steps; i += 2) {
                const int tile = m_used == 1 ? i : i >> 1;
                const uint32_t g = step + i, buf = g % S::kBufs;
                wait(&sm.sfull[buf], (g / S::kBufs) & 1);
                if (some) {
                    tc_fence_after();
                    const uint32_t cols = lanes + buf * kKeys;
                    // the keys that the row sees, where that is not all of them
                    const uint32_t *v = sm.valid[(tiles_done + tile) % S::kTilesAhead];
                    const int d = (at.t + tile) * kKeys - (at.len - at.n);
                    bool all = true;
#pragma unroll
                    for (int k = 0; k < kKeys / 32; ++k) all &= v[k] == 0xffffffffu;
                    if (d + kKeys > 0 || !all) {
#pragma unroll 1
                        for (int k = 0; k < kKeys / 32; ++k) {
                            uint32_t seen = v[k];
                            if (d + 32 * (k + 1) > 0) seen &= static_cast<uint32_t>(seen_from(word, d + 32 * k));
                            float s[32];
                            tmem_ld32(cols + 32 * k, s);
                            tmem_wait_ld();
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                if (!((seen >> x) & 1)) s[x] = -INFINITY;
                            tmem_st32(cols + 32 * k, s);
                        }
                        tmem_wait_st();
                    }
                    float top = -INFINITY, top1 = -INFINITY;
#pragma unroll
                    for (int k = 0; k < kKeys / 64; ++k) {
                        float s0[32], s1[32];
                        tmem_ld32(cols + 64 * k, s0);
                        tmem_ld32(cols + 64 * k + 32, s1);
                        tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 32; x += 2) {
                            top = fmaxf(fmaxf(top, s0[x]), s0[x + 1]);
                            top1 = fmaxf(fmaxf(top1, s1[x]), s1[x + 1]);
                        }
                    }
                    top = fmaxf(top, top1) * c;
                    // one m tile: the reference is the other warpgroup's of the step before
                    if (m_used == 1 && i > 0) {
                        pair_wait(quarter, wg);
                        const float other = sm.top[0][lrow];
                        if (other > m) {
                            if (i > 1) l *= ex2(m - other);
                            m = other;
                        }
                    }
                    const bool first = i < m_used;
                    // (where one row of the warp is rescaled, all that have grown at all are; lanes without a
                    // row have scores of whatever lay where their queries would)
                    const bool rescale = __any_sync(0xffffffffu, real && top > m + S::kSlack) && !first;
                    const bool grown = top > m && (first || rescale);
                    const float to = grown ? top : m;
                    const float ref = to == -INFINITY ? 0.f : to;
                    if (m_used == 1 && i + 1 < steps) {
                        sm.top[0][lrow] = to;
                        pair_arrive(quarter, wg);
                    }
                    if (rescale) {
                        const float keep = grown ? ex2(m - ref) : 1.f;
                        l *= keep;
                        const uint32_t q = g - m_used;  // the last product of these rows
                        wait(&sm.pfree[q % S::kBufs], (q / S::kBufs) & 1);
                        tc_fence_after();
#pragma unroll 1
                        for (int k = 0; k < kD / 32; ++k) {
                            float o[32];
                            const uint32_t oc = lanes + S::kColO + mt * kD + 32 * k;
                            tmem_ld32(oc, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int x = 0; x < 32; ++x) o[x] *= keep;
                            tmem_st32(oc, o);
                        }
                    }
                    m = to;
                    const uint64_t c2 = f2(c, c), off2 = f2(S::kShift - ref, S::kShift - ref);
                    uint64_t sum2 = 0;
#pragma unroll 1
                    for (int k = 0; k < kKeys / 32; ++k) {
                        float s[32], hi[16], lo[16];
                        tmem_ld32(cols + 32 * k, s);
                        tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            const float2 e = f2_split(f2_fma(f2(s[2 * x], s[2 * x + 1]), c2, off2));
                            const float p0 = ex2(e.x), p1 = ex2(e.y);
                            const uint64_t p2 = f2(p0, p1);
                            sum2 = f2_add(sum2, p2);
                            uint32_t h;
                            float2 y;  // the first words' values
                            if constexpr (kFp8) {
                                h = pack2<true>(p0, p1);
                                y = unpack2<true>(h);
                            } else {  // cut off: the second word holds what remains, and its rounding
                                h = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
                                y = make_float2(__uint_as_float(__float_as_uint(p0) & 0xffff0000u),
                                                __uint_as_float(__float_as_uint(p1) & 0xffff0000u));
                            }
                            const float2 rest = f2_split(f2_sub(p2, f2(y.x, y.y)));
                            hi[x] = __uint_as_float(h);
                            lo[x] = __uint_as_float(pack2<kFp8>(rest.x, rest.y));
                        }
                        // a weight's two words take its score's place
                        tmem_st16(cols + 32 * k, hi);
                        tmem_st16(cols + 32 * k + 16, lo);
                        if (k + 1 == kKeys / 64 || k + 1 == kKeys / 32) {
                            // half the keys' weights: their product may begin
                            tmem_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&sm.pfull[buf][k + 1 == kKeys / 64 ? 0 : 1]);
                        }
                    }
                    const float2 sum = f2_split(sum2);
                    l += sum.x + sum.y;
                } else {
                    if (lane < 2) mbar_arrive(&sm.pfull[buf][lane]);
                    __syncwarp();
                }
            }
            step += steps;
            tiles_done += tiles;
            if constexpr (kFp8) {
                // while this unit's last products run: its scores are all there, so nothing reads
                // its queries any more
                wait(&sm.scored, units & 1);
                if (more) queries(next, exps_next);
            }

            // outputs: a whole unit's to o, a cut one's to the workspace.  Of two m tiles a
            // warpgroup has its own, of one half the channels.
            wait(&sm.done, units & 1);
            ++units;
            const bool whole = at.t == 0 && at.t1 == at.tiles;
            const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (at.t == 0 ? 1 : 0);
            const float vs = a.cache.v_scale != nullptr ? a.cache.v_scale[at.h] : 1.f;
            if (some) {
                tc_fence_after();
                if (m_used == 1) {  // the two warpgroups' sums, by the later reference
                    sm.top[wg][lrow] = m;
                    pair_barrier(quarter);
                    const float to = fmaxf(m, sm.top[wg ^ 1][lrow]);
                    pair_barrier(quarter);
                    sm.top[wg][lrow] = l * ex2(m - (to == -INFINITY ? 0.f : to));
                    pair_barrier(quarter);
                    l = sm.top[0][lrow] + sm.top[1][lrow];
                    m = to;
                    pair_barrier(quarter);
                }
                const int d0 = m_used == 1 ? wg * (kD / 2) : 0, d1 = m_used == 1 ? d0 + kD / 2 : kD;
                const float f = l == 0.f ? 0.f : 1.f / l;
                float nan = 0.f;
                const int64_t out = row * a.q_heads + qh;
#pragma unroll 1
                for (int d = d0; d < d1; d += 32) {
                    float o[32];
                    tmem_ld32(lanes + S::kColO + mt * kD + d, o);
                    tmem_wait_ld();
                    if (whole) {
                        uint32_t y[16];
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            nan = fmaf(o[k], 0.f, fmaf(o[k + 1], 0.f, nan));
                            y[k / 2] = l == 0.f ? 0u : pack2<false>(o[k] * f * vs, o[k + 1] * f * vs);
                        }
                        if (real)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                reinterpret_cast<uint4 *>(a.o + out * kD + d)[k] =
                                    make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            reinterpret_cast<float4 *>(args.cut)[(slot * (kD / 4) + d / 4 + k) * S::kRows +
                                                                 mt * 128 + lrow] =
                                make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                    }
                }
                tc_fence_before();
                if (whole) {
                    if (real && d0 == 0 && a.lse != nullptr)
                        a.lse[out] = l == 0.f ? -INFINITY : (m + log2f(l) - S::kShift) * kLn2;
                    again |= __any_sync(0xffffffffu, real && nan != 0.f && l * 0.f == 0.f && l != 0.f);
                } else if (d0 == 0) {
                    reinterpret_cast<float2 *>(args.ml)[slot * S::kRows + mt * 128 + lrow] = make_float2(m, l);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.ofree);
            at = next;
            if constexpr (kFp8)
#pragma unroll
                for (int t = 0; t < kM; ++t) exps[t] = exps_next[t];
        }
        // What is not finite is computed again when the piece is done: it may take long, and no other
        // warp waits with a limit now.  (The queries' place is free.)
        if (again) {
            const int *begin = sm.begin[warp];
            at.request(a, begin[0]);
            at.h = begin[1];
            at.rg = begin[2];
            at.at = begin[3];
            at.left = sm.places[warp];
            step = 0;
            while (at.take(a)) {
                const int m_used = at.m_tiles(at.rg), mt = m_used == 1 ? 0 : (step + wg) & 1;
                step += (at.t1 - at.t) * m_used;
                if (at.t != 0 || at.t1 != at.tiles) continue;
                const int d0 = m_used == 1 ? wg * (kD / 2) : 0, d1 = m_used == 1 ? d0 + kD / 2 : kD;
                const int rr = at.rg * S::kRows + mt * 128 + lrow;
                uint32_t node, head;
                args.group.divmod(rr, node, head);
                const int64_t row = at.first + node;
                const int qh = at.h * a.group + static_cast<int>(head);
                for (int d = d0; d < d1; d += 8) {
                    bool bad = false;
                    if (rr < at.rows) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(a.o + (row * a.q_heads + qh) * kD + d);
                        for (const uint32_t y : {x.x, x.y, x.z, x.w})
                            bad |= (y & 0x7f80u) == 0x7f80u || (y & 0x7f800000u) == 0x7f800000u;
                    }
                    for (uint32_t rows = __ballot_sync(0xffffffffu, bad); rows != 0; rows &= rows - 1) {
                        const int src = __ffs(static_cast<int>(rows)) - 1;
                        row_again<kD, kFp8>(a, at.b, __shfl_sync(0xffffffffu, row, src),
                                            __shfl_sync(0xffffffffu, qh, src), at.n, at.len, d,
                                            reinterpret_cast<float *>(smem) + warp * kD);
                    }
                }
            }
        }
    } else if (warp < kSoftWarps + kCopyWarps) {
        // ---- keys and values in --------------------------------------------------------------
        // Two warps copy keys, two values; each half of a tile's rows.
        leave_registers<kCopyRegs>();
        Waits wait = {a.err, true};
        const int cw = warp - kSoftWarps, half = cw & 1;
        const bool is_v = cw >= 2;
        const uint8_t *data = is_v ? a.cache.v : a.cache.k;
        const CUtensorMap *map = is_v ? &args.map_v : &args.map_k;
        uint64_t *full = is_v ? sm.vfull : sm.kfull, *empty = is_v ? sm.vempty : sm.kempty;
        const uint32_t slots = is_v ? S::kNV : S::kNK, ops = is_v ? S::kOffV : S::kOffK;
        constexpr int kRowsOfWarp = kKeys / 2, kLaneRows = kRowsOfWarp / 32;
        constexpr int kRowBytes = kD * (kFp8 ? 1 : 2);
        constexpr int kPieces = kRowBytes / 16;          // lanes to a row
        constexpr int kAtOnce = 32 / kPieces;            // rows of a warp's copy
        constexpr int kTurns = kRowsOfWarp / kAtOnce;
        constexpr int kBlocks = kFp8 ? 1 : kD / 64;      // boxes beside one another
        const int sub = lane / kPieces, ch = lane % kPieces, row0 = half * kRowsOfWarp;
        const int box = args.box;                        // keys of a box; 0: none
        uint32_t made = 0, widened = 0;                  // tiles
        int page[kLaneRows];                             // of this lane's rows of the next tile
        uint32_t in_page[kLaneRows];
        bool held[kLaneRows];
        auto find_pages = [&](int tile) {
#pragma unroll
            for (int i = 0; i < kLaneRows; ++i) {
                const uint32_t j = static_cast<uint32_t>(tile) * kKeys + row0 + lane + 32 * i;
                uint32_t idx;
                a.cache.page.divmod(j, idx, in_page[i]);
                held[i] = j < static_cast<uint32_t>(at.len);
                page[i] = held[i] ? a.block_table[static_cast<int64_t>(at.b) * a.max_pages + idx] : -1;
            }
        };
        // a raw tile's rows, widened into their place as an operand (8-bit cache)
        auto widen = [&]() {
            if constexpr (kFp8) {
                const uint32_t slot = widened % slots, raw_slot = widened % S::kNR;
                if (!wait(&sm.raw[is_v][half][raw_slot], (widened / S::kNR) & 1)) return;
                if (!wait(&empty[slot], ((widened / slots) & 1) ^ 1)) return;
                const uint8_t *raw = smem + S::kOffRaw + (is_v * S::kNR + raw_slot) * S::kRaw + half * (S::kRaw / 2);
                uint8_t *to = smem + ops + slot * S::kTile;
                // (neighbouring blocks of 64 channels in turn, so that 8 lanes meet every bank once)
                const int swap = (ch >> 2) & 1;
                constexpr int kBatch = kTurns < 8 ? kTurns : 8;
#pragma unroll
                for (int k0 = 0; k0 < kTurns; k0 += kBatch) {
                    uint4 x[kBatch];  // loads first: a store might alias them
#pragma unroll
                    for (int k = 0; k < kBatch; ++k)
                        x[k] = *reinterpret_cast<const uint4 *>(raw + ((k0 + k) * 32 + lane) * 16);
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        const int r = row0 + (k0 + k) * kAtOnce + sub;
                        uint4 y0, y1;
                        y0.x = e4m3x2_to_f16x2(x[k].x);
                        y0.y = e4m3x2_to_f16x2(x[k].x >> 16);
                        y0.z = e4m3x2_to_f16x2(x[k].y);
                        y0.w = e4m3x2_to_f16x2(x[k].y >> 16);
                        y1.x = e4m3x2_to_f16x2(x[k].z);
                        y1.y = e4m3x2_to_f16x2(x[k].z >> 16);
                        y1.z = e4m3x2_to_f16x2(x[k].w);
                        y1.w = e4m3x2_to_f16x2(x[k].w >> 16);
                        uint8_t *row = to + (ch >> 2) * (kKeys * 128) + r * 128;
                        const int c0 = ((2 * ch + swap) & 7) ^ (r & 7);
                        *reinterpret_cast<uint4 *>(row + (c0 << 4)) = swap ? y1 : y0;
                        *reinterpret_cast<uint4 *>(row + ((c0 ^ 1) << 4)) = swap ? y0 : y1;
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(&full[slot]);
                ++widened;
                __syncwarp();
            }
        };
        bool more = at.take(a);
        if (more) find_pages(at.t);
        while (more && wait.ok) {
            const int t1 = at.t1;
            for (int tile = at.t; tile < t1 && wait.ok; ++tile, ++made) {
                const int h = at.h;
                bool whole = box > 0;
                int64_t off[kLaneRows];
                int box_page = 0, box_row = 0;  // of this lane's box
                const int mine = lane / kBlocks * box;
#pragma unroll
                for (int i = 0; i < kLaneRows; ++i) {
                    const bool ok = page[i] >= 0 && page[i] < a.cache.num_pages;
                    if (held[i] && !ok) record_device_error(a.err, kDevInvalidArg);
                    off[i] = ok ? page[i] * a.cache.page_stride + in_page[i] * a.cache.token_stride +
                                      h * a.cache.head_stride
                                : -1;
                    const uint32_t valid = __ballot_sync(0xffffffffu, ok);
                    whole &= valid == 0xffffffffu;
                    if (!is_v && lane == 0) sm.valid[made % S::kTilesAhead][half * kLaneRows + i] = valid;
                    const int p = __shfl_sync(0xffffffffu, page[i], mine & 31);
                    const int q = __shfl_sync(0xffffffffu, static_cast<int>(in_page[i]), mine & 31);
                    if (i == mine >> 5) {
                        box_page = p;
                        box_row = q;
                    }
                }
                // the next tile's pages, ahead of this one's copies
                if (tile + 1 < t1) {
                    find_pages(tile + 1);
                } else {
                    more = at.take(a);
                    if (more) find_pages(at.t);
                }
                uint64_t *bar;
                uint32_t to, row_pitch;  // where the warp's rows go
                if constexpr (kFp8) {
                    const uint32_t slot = made % S::kNR;
                    bar = &sm.raw[is_v][half][slot];
                    to = S::kOffRaw + (is_v * S::kNR + slot) * S::kRaw + half * (S::kRaw / 2);
                    row_pitch = kD;
                } else {
                    const uint32_t slot = made % slots;
                    if (!wait(&empty[slot], ((made / slots) & 1) ^ 1)) break;
                    bar = &full[slot];
                    to = ops + slot * S::kTile + row0 * 128;
                    row_pitch = 128;
                }
                if (whole) {
                    // every row is a key: boxes of keys, by the tensor map
                    if (lane == 0) mbar_arrive_expect_tx(bar, kRowsOfWarp * kRowBytes);
                    __syncwarp();
                    if (mine < kRowsOfWarp)
                        load_box(smem + to + lane % kBlocks * (kKeys * 128) + mine * row_pitch, map, bar,
                                 lane % kBlocks * 64, box_row, h, box_page);
                    mbar_arrive(bar);
                } else {
                    // row by row, zeros where there is no key
#pragma unroll 1
                    for (int k0 = 0; k0 < kTurns; k0 += 4) {
                        int64_t from[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int r = (k0 + k) * kAtOnce + sub;
                            from[k] = __shfl_sync(0xffffffffu, off[0], r & 31);
                            if constexpr (kLaneRows == 2) {
                                const int64_t x = __shfl_sync(0xffffffffu, off[1], r & 31);
                                if (r >= 32) from[k] = x;
                            }
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int r = (k0 + k) * kAtOnce + sub;
                            uint32_t dst = base + to + r * row_pitch;
                            if constexpr (kFp8) dst += ch * 16;
                            else dst += (ch >> 3) * (kKeys * 128) + (((ch & 7) ^ (r & 7)) << 4);
                            copy16(dst, data + (from[k] < 0 ? 0 : from[k] + ch * 16), from[k] >= 0);
                        }
                    }
                    copies_arrive(bar);
                    if (lane == 0) mbar_arrive(bar);
                }
                if (kFp8 && made + 1 >= S::kNR) widen();
            }
        }
        while (kFp8 && widened < made && wait.ok) widen();
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (!wait.ok) {  // boxes that nobody waits for any more
            const uint32_t ring = kFp8 ? S::kNR : slots;
            for (uint32_t i = made < ring ? 0 : made - ring; i < made; ++i)
                mbar_wait_bounded(kFp8 ? &sm.raw[is_v][half][i % ring] : &full[i % ring], (i / ring) & 1, kMaxPolls);
        }
    } else {
        // ---- products ------------------------------------------------------------------------
        // One warp issues the scores', the next the outputs': each spends more time on its waits
        // and its instructions' way to the SM than a product takes.
        leave_registers<kProductRegs>();
        constexpr uint32_t kFmt = kFp8 ? kFmtF16 : kFmtBF16;
        Waits wait = {a.err, true};
        if (warp == kSoftWarps + kCopyWarps) {
            uint32_t step = 0, made = 0, units = 0;
            while (at.take(a) && wait.ok) {
                const bool negate = a.scale * (a.cache.k_scale != nullptr ? a.cache.k_scale[at.h] : 1.f) < 0.f;
                const uint32_t id = negate ? instr_desc(128, kKeys, kFmt, 0, 0, 1) : instr_desc(128, kKeys, kFmt, 0, 0);
                const int m_used = at.m_tiles(at.rg);
                wait(&sm.qfull, units & 1);
                for (int tile = at.t; tile < at.t1 && wait.ok; ++tile, ++made) {
                    const uint32_t ks = made % S::kNK;
                    if (!wait(&sm.kfull[ks], (made / S::kNK) & 1)) break;
                    // the copies wrote by the generic proxy, the product reads by the async one
                    fence_proxy_async_smem();
                    for (int t = 0; t < m_used; ++t, ++step) {
                        // the weights in this buffer have met their values
                        const uint32_t buf = step % S::kBufs;
                        if (!wait(&sm.pfree[buf], ((step / S::kBufs) & 1) ^ 1)) break;
                        tc_fence_after();
                        const uint32_t d = tmem + buf * kKeys;
                        const uint64_t qd = smem_desc(base + t * (128 * kD * 2), 16, 1024, kSwizzle128B);
                        const uint64_t kd = smem_desc(base + S::kOffK + ks * S::kTile, 16, 1024, kSwizzle128B);
#pragma unroll 1
                        for (int k = 0; k < kD / 64; ++k)  // (short code: the warps share its cache)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                mma_f16_ss_w(d, qd + (k * (128 * 128) + j * 32) / 16,
                                             kd + (k * (kKeys * 128) + j * 32) / 16, id, k + j > 0);
                        mma_commit_w(&sm.sfull[buf]);
                    }
                    mma_commit_w(&sm.kempty[ks]);
                }
                mma_commit_w(&sm.scored);
                ++units;
            }
        } else if (warp == kSoftWarps + kCopyWarps + 1) {
            constexpr uint32_t kId = instr_desc(128, kD, kFmt, 0, 1);
            uint32_t step = 0, made = 0, units = 0;
            while (at.take(a) && wait.ok) {
                const int m_used = at.m_tiles(at.rg);
                // the last unit's outputs have been read
                if (!wait(&sm.ofree, (units & 1) ^ 1)) break;
                ++units;
                for (int tile = at.t; tile < at.t1 && wait.ok; ++tile, ++made) {
                    const uint32_t vs = made % S::kNV;
                    if (!wait(&sm.vfull[vs], (made / S::kNV) & 1)) break;
                    fence_proxy_async_smem();
                    for (int t = 0; t < m_used; ++t, ++step) {
                        const uint32_t buf = step % S::kBufs;
                        const uint32_t d = tmem + S::kColO + t * kD, p = tmem + buf * kKeys;
                        const uint64_t vd = smem_desc(base + S::kOffV + vs * S::kTile, kKeys * 128, 1024, kSwizzle128B);
#pragma unroll 1
                        for (int k = 0; k < kKeys / 32; ++k) {
                            if (k % (kKeys / 64) == 0) {
                                if (!wait(&sm.pfull[buf][k / (kKeys / 64)], (step / S::kBufs) & 1)) break;
                                tc_fence_after();
                            }
#pragma unroll
                            for (int j = 0; j < 4; ++j)  // two groups of 16 keys, two words
                                mma_f16_ts_w(d, p + 32 * k + (j & 1) * 8 + (j >> 1) * 16,
                                             vd + (32 * k + (j & 1) * 16) * 128 / 16, kId, k + j > 0 || tile > at.t);
                        }
                        if (!wait.ok) break;
                        mma_commit_w(&sm.pfree[buf]);
                    }
                    mma_commit_w(&sm.vempty[vs]);
                }
                mma_commit_w(&sm.done);
            }
        } else if (!kFp8) {
            // Queries in, by two warps: a unit's when the last one's scores are all there; their
            // rows are called into L2 before.
            const int qw = warp - kSoftWarps - kCopyWarps - 2;
            constexpr int kLanes = kD / 8, kAtOnce = 32 / kLanes;  // lanes to a row, rows of a warp
            const int sub = lane / kLanes, ch = lane % kLanes;     // ch: 16-byte piece
            uint32_t units = 0;
            while (at.take(a) && wait.ok) {
                const int row0 = at.rg * S::kRows, rows = min(at.rows - row0, S::kRows);
                auto source = [&](int r) {  // this lane's piece of row r
                    uint32_t node, head;
                    args.group.divmod(row0 + r, node, head);
                    return reinterpret_cast<const uint4 *>(a.q + (at.first + node) * a.q_row_stride +
                                                           (at.h * a.group + static_cast<int>(head)) * kD) + ch;
                };
                auto place = [&](int r) {
                    return (r >> 7) * (128 * kD * 2) + (ch >> 3) * (128 * 128) + (r & 127) * 128 + (((ch & 7) ^ (r & 7)) << 4);
                };
                if (ch % 8 == 0)
                    for (int r = qw * kAtOnce + sub; r < rows; r += 2 * kAtOnce)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(source(r)));
                if (units > 0 && !wait(&sm.scored, (units - 1) & 1)) break;
#pragma unroll 4
                for (int r = qw * kAtOnce + sub; r < rows; r += 2 * kAtOnce)
                    copy16(base + place(r), reinterpret_cast<const uint8_t *>(source(r)), true);
                copies_arrive(&sm.qfull);
                ++units;
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
        if (warp <= kSoftWarps + kCopyWarps + 1) {
            // nothing is in flight when tensor memory is given back
            uint64_t *drain = &sm.drain[warp - kSoftWarps - kCopyWarps];
            mma_commit_w(drain);
            mbar_wait_bounded(drain, 0, kMaxPolls);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kSoftWarps + kCopyWarps) tmem_dealloc(tmem, 512);
}

// Joins the parts of the unit that CTA blockIdx.x of the first kernel began and did not finish:
// its slot 1, and slot 0 of the CTAs after it up to the last.  A thread has one row and 8
// channels (blockIdx.y).  Blocks (c, 0) also look after sequences that have no keys.
template <class S>
__global__ void __launch_bounds__(S::kRows) tree_join_kernel(const __grid_constant__ Args args, int ctas) {
    constexpr int kD = S::kD, kWarps = S::kRows / 32;
    __shared__ int64_t s_warp[kWarps], s_place[2];
    __shared__ float s_q[kWarps][kD];
    const TreeAttention &a = args.t;
    const int tid = threadIdx.x, c0 = blockIdx.x;
    // (this kernel is set up once the first one's blocks have all waited for what was before
    // them, so the lengths, which the first one does not write, may be read here)
    List list;
    Cursor<S> cut = {};
    int parts = 0;
    if (find_place<S, kWarps>(a, ctas, s_warp, s_place, [&](const List &l) {
            return c0 < l.pieces ? l.begin(c0 + int64_t{1}) : l.total;
        }, list, cut)) {
        // the places where the unit's first and last tiles begin
        const int64_t first = list.begin(c0 + int64_t{1}) - cut.at + S::kUnitCost,
                      last = first + static_cast<int64_t>(cut.tiles - 1) * cut.cost(cut.rg);
        const int done = cut.tile_at(cut.at);  // tiles that begin before the next piece
        if (done > 0 && done < cut.tiles && first >= list.begin(c0)) parts = list.piece_of(last) - c0 + 1;
    }
    wait_for_kernel_before();
    const int r = cut.rg * S::kRows + tid;
    if (parts > 0) {
        const bool real = r < cut.rows;
        uint32_t node, g;
        args.group.divmod(r, node, g);
        const int64_t row = cut.first + node;
        const int qh = cut.h * a.group + static_cast<int>(g), d = blockIdx.y * 8;
        auto slot = [&](int i) { return static_cast<int64_t>(c0 + i) * 2 + (i == 0 ? 1 : 0); };
        float m = -INFINITY, l = 0.f, acc[8] = {}, nan = 0.f;
        if (real) {
            // four parts at a time, one trip to memory for them
            for (int i0 = 0; i0 < parts; i0 += 4) {
                float2 x[4];
                float4 y[4], z[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = make_float2(-INFINITY, 0.f);
                    y[i] = z[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i0 + i >= parts) continue;
                    x[i] = reinterpret_cast<const float2 *>(args.ml)[slot(i0 + i) * S::kRows + tid];
                    const float4 *p = reinterpret_cast<const float4 *>(args.cut) +
                                      (slot(i0 + i) * (kD / 4) + d / 4) * S::kRows + tid;
                    y[i] = p[0];
                    z[i] = p[S::kRows];
                }
                const float to = fmaxf(fmaxf(fmaxf(m, x[0].x), x[1].x), fmaxf(x[2].x, x[3].x));
                const float ref = to == -INFINITY ? 0.f : to, keep = ex2(m - ref);
                m = to;
                l *= keep;
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[k] *= keep;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float w = ex2(x[i].x - ref);
                    l += w * x[i].y;
                    acc[0] += w * y[i].x;
                    acc[1] += w * y[i].y;
                    acc[2] += w * y[i].z;
                    acc[3] += w * y[i].w;
                    acc[4] += w * z[i].x;
                    acc[5] += w * z[i].y;
                    acc[6] += w * z[i].z;
                    acc[7] += w * z[i].w;
                }
            }
            const float vs = a.cache.v_scale != nullptr ? a.cache.v_scale[cut.h] : 1.f;
            const float f = l == 0.f ? 0.f : 1.f / l;
            const int64_t out = row * a.q_heads + qh;
            uint32_t y[4];
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                nan = fmaf(acc[k], 0.f, fmaf(acc[k + 1], 0.f, nan));
                y[k / 2] = l == 0.f ? 0u : pack2<false>(acc[k] * f * vs, acc[k + 1] * f * vs);
            }
            *reinterpret_cast<uint4 *>(a.o + out * kD + d) = make_uint4(y[0], y[1], y[2], y[3]);
            if (a.lse != nullptr && blockIdx.y == 0)
                a.lse[out] = l == 0.f ? -INFINITY : (m + log2f(l) - S::kShift) * kLn2;
        }
        uint32_t again = __ballot_sync(0xffffffffu, real && nan != 0.f && l * 0.f == 0.f && l != 0.f);
        while (again != 0) {
            const int src = __ffs(static_cast<int>(again)) - 1;
            again &= again - 1;
            row_again<kD, S::kFp8>(a, cut.b, __shfl_sync(0xffffffffu, row, src),
                                   __shfl_sync(0xffffffffu, qh, src), cut.n, cut.len, d, s_q[tid >> 5]);
        }
    }
    if (blockIdx.y != 0) return;
    for (int b = c0; b < a.B; b += gridDim.x) {
        const TreeRows t = tree_rows(a.cu, b, a.N, a.max_nodes);
        const int len = a.seq_lens[b];
        const bool fits = len >= t.rows && len <= static_cast<int64_t>(a.max_pages) * a.cache.page.d;
        if (!t.bad && fits) continue;
        if (tid == 0) record_device_error(a.err, kDevInvalidArg);
        const int64_t rows = static_cast<int64_t>(t.rows) * a.q_heads, o0 = t.first * a.q_heads;
        for (int64_t i = tid; i < rows * (kD / 8); i += S::kRows)
            reinterpret_cast<uint4 *>(a.o + o0 * kD)[i] = make_uint4(0, 0, 0, 0);
        if (a.lse != nullptr)
            for (int64_t i = tid; i < rows; i += S::kRows) a.lse[o0 + i] = -INFINITY;
    }
}

// The cache's halves for boxes of keys, where its pages can be cut in boxes of 8 keys (a swizzled
// group of rows) or more.  Otherwise, and where the driver refuses, rows are copied one by one.
template <class S>
void make_maps(Args &a) {
    constexpr int kSize = S::kFp8 ? 1 : 2;
    const PagedView &c = a.t.cache;
    a.box = 0;
    int box = S::kKeys / 2;
    while (c.page.d % static_cast<uint32_t>(box) != 0) box /= 2;
    const chunk::EncodeTiledFn fn = chunk::encode_fn();
    if (box < 8 || fn == nullptr) return;
    const cuuint64_t dims[4] = {S::kD, c.page.d, static_cast<cuuint64_t>(c.heads),
                                static_cast<cuuint64_t>(c.num_pages)};
    // (the stride of a single entry is not given, and never taken)
    auto stride = [](int64_t x) { return static_cast<cuuint64_t>(x > 0 ? x : S::kD * kSize); };
    const cuuint64_t strides[3] = {stride(c.token_stride), stride(c.head_stride), stride(c.page_stride)};
    const cuuint32_t boxes[4] = {static_cast<cuuint32_t>(S::kFp8 ? S::kD : 64), static_cast<cuuint32_t>(box), 1, 1};
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    auto make = [&](CUtensorMap *map, void *data) {
        return fn(map, S::kFp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, data, dims,
                  strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  S::kFp8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (make(&a.map_k, c.k) && make(&a.map_v, c.v)) a.box = box;
}

template <class S>
cudaError_t launch_shape(Args a, int ctas, cudaStream_t s) {
    make_maps<S>(a);
    const cudaError_t e =
        ensure_dynamic_smem(reinterpret_cast<const void *>(&tree_attention_kernel<S>), S::kSmem);
    if (e != cudaSuccess) return e;
    const cudaError_t e1 = launch_early(tree_attention_kernel<S>, dim3(ctas), kThreads, S::kSmem, s, a);
    if (e1 != cudaSuccess) return e1;
    return launch_early(tree_join_kernel<S>, dim3(ctas, S::kD / 8), S::kRows, 0, s, a, ctas);
}

}  // namespace

// Instantiated for each head_dim in a file of its own: they compile side by side.
template <int kD>
cudaError_t launch_dim(const Args &a, int m, int ctas, cudaStream_t s) {
    if constexpr (kD <= 128)
        if (m == 2)
            return a.t.cache.fp8 ? launch_shape<Shape<kD, true, 2>>(a, ctas, s)
                                 : launch_shape<Shape<kD, false, 2>>(a, ctas, s);
    return a.t.cache.fp8 ? launch_shape<Shape<kD, true, 1>>(a, ctas, s)
                         : launch_shape<Shape<kD, false, 1>>(a, ctas, s);
}

}  // namespace treeatt
}  // namespace kda
