// kda_paged_decode.cu -- softmax attention of one new token per sequence over a
// paged key-value cache.
//
//   s_j = scale <q, k_j>,  m = max_j s_j,  l = sum_j e^{s_j - m}
//   o = sum_j e^{s_j - m} v_j / l,  lse = m + log l
//
// and over any partition of the keys, from the parts' (m_i, l_i, a_i) with
// a_i = sum e^{s_j - m_i} v_j:  m = max m_i,  l = sum e^{m_i - m} l_i,
// o = sum e^{m_i - m} a_i / l.  Powers of two throughout: the scores carry log2 e.
//
// Bound: every key and value is read once, 4 G flops for the 2 (or 4) bytes of
// a value at G query heads to a key head: HBM up to G = 100.  So what matters is
// that every SM has copies in flight from the first microsecond to the last,
// whatever the lengths.
//
// Split.  A unit is (sequence, key head, group of 16 query heads); its keys are
// cut in tiles of 8 KB of keys and values (16 KB at 256 channels in bf16).  The
// tiles of all units form one list, and each warp of the grid takes an equal,
// contiguous piece of it: long sequences are cut, short ones share a warp, and
// no warp has more than one tile more than another.  A piece ends in at most two
// cut units; their parts are joined within the CTA through shared memory, and
// what is cut between CTAs by a second, small kernel that is launched with the
// first and waits for it (programmatic dependent launch).
//
// A warp copies its own tiles, by 16-byte cp.async into its own ring of tiles
// (no barrier between warps), two ahead of the one it computes; the page numbers
// of a tile are read one tile earlier still.  Rows are swizzled (16-byte pieces
// xor row) so that ldmatrix meets no bank twice.  The products run on the warp's
// matrix instructions with the query heads as the 16 rows: S = Q K^T, then P V
// with S's accumulator layout as the left operand, so the weights never leave
// the registers.  (tcgen05.mma wants 64 or 128 rows: it would idle on 16, and the
// tensor pipe is not what binds here.)
//
// Precision: scores, maxima, sums and outputs in fp32.  For the product with the
// values a weight is two bf16 numbers, 16 bits together: one would leave up to
// 2^-8 of every weight, as much as the rounding of a bf16 output and far more
// than an fp32 one may lose, and the second product is free here (see Bound).  An 8-bit
// cache is widened to fp16, which holds every e4m3 value; the queries are scaled
// by a power of two for each row, so that fp16 holds their bf16 values too, and
// the weights are two fp16 numbers, times 2^15 to keep small ones normal.
#include <cuda_fp16.h>

#include "kda_internal.cuh"
#include "kda_paged.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace {

constexpr int kRows = 16;       // query heads of a unit
constexpr int kMaxCtas = 160;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int kD, bool kFp8>
struct Shape {
    static constexpr int kRowBytes = kD * (kFp8 ? 1 : 2);
    static constexpr int kKeys = kRowBytes >= 256 ? 16 : 4096 / kRowBytes;  // keys of a tile
    static constexpr int kHalf = kKeys * kRowBytes;                        // its keys, in bytes
    static constexpr int kWarps = kHalf > 4096 ? 4 : 8;
    static constexpr int kStages = 3;
    static constexpr int kRing = kStages * 2 * kHalf;                      // a warp's ring
    static constexpr int kPad = kD + 8;                                    // floats of a part's row
    static_assert(kRows * kPad * 4 <= kRing, "a part must fit a warp's ring");
};

// What is cut at a CTA's ends: its first unit's part (begun by an earlier CTA)
// in slot 0, its last unit's (begun here, not finished) in slot 1.
struct CutMeta {
    int64_t unit;  // -1: none
    int ends;      // the unit's last key is in this part
    int pad;
};

struct Layout {  // of the workspace
    CutMeta *meta;   // [ctas][2]
    float *ml;       // [ctas][2][kRows][2]
    float *cut;      // [ctas][2][kRows][D]
    float *head;     // [ctas][warps][kRows][D]: a warp's first part, until its CTA joins it
};

__host__ __device__ inline size_t align256(size_t x) { return (x + 255) & ~size_t{255}; }

inline size_t layout_bytes(int head_dim, uint8_t *base, Layout *l) {
    size_t at = 0;
    const size_t part = static_cast<size_t>(kRows) * head_dim * 4;
    const size_t meta = at;
    at = align256(at + kMaxCtas * 2 * sizeof(CutMeta));
    const size_t ml = at;
    at = align256(at + kMaxCtas * 2 * kRows * 2 * 4);
    const size_t cut = at;
    at = align256(at + kMaxCtas * 2 * part);
    const size_t head = at;
    at = align256(at + kMaxCtas * 8 * part);
    if (l != nullptr) {
        l->meta = reinterpret_cast<CutMeta *>(base + meta);
        l->ml = reinterpret_cast<float *>(base + ml);
        l->cut = reinterpret_cast<float *>(base + cut);
        l->head = reinterpret_cast<float *>(base + head);
    }
    return at;
}

struct Args {
    const __nv_bfloat16 *q;
    int64_t q_row_stride;
    PagedView cache;
    const int32_t *block_table;
    int max_pages;
    const int32_t *seq_lens;
    int B, q_heads, group, head_tiles;
    float scale;
    void *o;
    int o_bf16;
    float *lse;
    Layout ws;
    unsigned int *err;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// c (16 x 8, fp32) += a (16 x 16) b (16 x 8), bf16 or fp16 operands.
template <bool kF16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
    if constexpr (kF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two e4m3 values (the low or high half of x) as two fp16 values: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t x) {
    uint32_t y;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(x));
    return y;
}

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
    else return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&x));
}

// Byte offset of 16-byte piece `c` of row `r` of a tile half.
template <int kRowBytes>
__device__ __forceinline__ uint32_t piece(uint32_t r, uint32_t c) {
    if constexpr (kRowBytes >= 128) return r * kRowBytes + ((c ^ (r & 7)) << 4);
    else return (r >> 1) * 128 + (((((r & 1) << 2) | c) ^ ((r >> 1) & 7)) << 4);
}

__device__ __forceinline__ int valid_len(const Args &a, int b) {
    const int n = __ldg(a.seq_lens + b);
    return n < 0 || n > static_cast<int64_t>(a.max_pages) * a.cache.page.d ? 0 : n;
}

// A place in the list of tiles.
template <int kKeys>
struct Cursor {
    int b, u, t;    // sequence, unit of the sequence, tile of the unit
    int len, tiles;

    __device__ __forceinline__ void set_len(int n) {
        len = n;
        tiles = static_cast<int>((static_cast<uint32_t>(n) + kKeys - 1) / kKeys);
    }
    __device__ __forceinline__ void next(const Args &a, int units) {
        if (++t < tiles) return;
        t = 0;
        if (++u < units) return;
        u = 0;
        do {
            if (++b >= a.B) {
                tiles = len = 0;
                return;
            }
            set_len(valid_len(a, b));
        } while (tiles == 0);
    }
};

// A part of a unit as a warp leaves it for its CTA.
struct Part {
    int64_t unit;    // b * units + u; -1: none
    int starts, ends;
    int in_global;   // its sums are in the workspace (else in the warp's ring)
    int pad;
};

__device__ __forceinline__ void write_out(const Args &a, int64_t at, float4 x) {
    if (a.o_bf16) {
        uint2 w;
        w.x = pack2<false>(x.x, x.y);
        w.y = pack2<false>(x.z, x.w);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + at) = w;
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + at) = x;
    }
}

template <int kD, bool kFp8>
__global__ void __launch_bounds__(Shape<kD, kFp8>::kWarps * 32, 1)
    paged_decode_kernel(const Args a) {
    using S = Shape<kD, kFp8>;
    constexpr int kWarps = S::kWarps, kThreads = kWarps * 32, kKeys = S::kKeys;
    constexpr int kNT = kKeys / 8;        // score tiles of 8 keys
    constexpr int kOT = kD / 8;           // output tiles of 8 channels
    constexpr int kPieces = S::kRowBytes / 16;
    constexpr int kParts = 2 * kWarps;
    constexpr bool kF16 = kFp8;

    extern __shared__ __align__(1024) uint8_t s_ring[];
    __shared__ int64_t s_scan[kWarps];
    __shared__ Cursor<kKeys> s_start[kWarps];
    __shared__ uint64_t s_valid[kWarps][S::kStages];
    __shared__ Part s_part[kParts];
    __shared__ float s_m[kParts][kRows], s_l[kParts][kRows];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, tq = lane & 3;
    const int units = a.cache.heads * a.head_tiles;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the list: tiles before each sequence, and where this CTA's warps begin ----------
    const int chunk = (a.B + kThreads - 1) / kThreads;
    const int b_lo = min(a.B, tid * chunk), b_hi = min(a.B, b_lo + chunk);
    int64_t mine = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        const int n = __ldg(a.seq_lens + b);
        const int v = valid_len(a, b);
        if (n != v && blockIdx.x == 0) record_device_error(a.err, kDevInvalidArg);
        mine += (static_cast<uint32_t>(v) + kKeys - 1) / kKeys;
    }
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += x;
    }
    if (lane == 31) s_scan[warp] = incl;
    if (lane == 0) s_start[warp].b = -1;
    if (tid < kParts) s_part[tid].unit = -1;
    __syncthreads();
    int64_t before = (incl - mine), total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
    }
    before *= units;
    total *= units;
    // as many CTAs as leave a tile to each warp, all of the grid for longer lists
    const int64_t want = (total + kWarps - 1) / kWarps;
    const int64_t ctas = want < gridDim.x ? want : gridDim.x;
    const int64_t pieces_of = ctas * kWarps;
    if (blockIdx.x < ctas && mine > 0) {
        for (int w = 0; w < kWarps; ++w) {
            const int64_t start = (static_cast<int64_t>(blockIdx.x) * kWarps + w) * total / pieces_of;
            if (start < before || start >= before + mine * units) continue;
            int64_t left = start - before;
            int b = b_lo;
            Cursor<kKeys> c;
            for (;; ++b) {
                c.set_len(valid_len(a, b));
                const int64_t here = static_cast<int64_t>(c.tiles) * units;
                if (left < here) break;
                left -= here;
            }
            c.b = b;
            c.u = static_cast<int>(left / c.tiles);
            c.t = static_cast<int>(left - static_cast<int64_t>(c.u) * c.tiles);
            s_start[w] = c;
        }
    }
    __syncthreads();

    // ---- a warp's piece --------------------------------------------------------------------
    const uint32_t ring = sm100::smem_addr(s_ring) + warp * S::kRing;
    int64_t remaining = 0;
    if (blockIdx.x < ctas) {
        const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
        remaining = (w + 1) * total / pieces_of - w * total / pieces_of;
    }
    if (remaining > 0) {
        Cursor<kKeys> cur = s_start[warp], pre = cur;
        int64_t to_copy = remaining;

        // the page of this lane's row (two rows where a tile has 64 keys) of tile `pre`
        constexpr int kLaneRows = kKeys > 32 ? 2 : 1;
        int page[kLaneRows];
        bool held[kLaneRows];  // the row is a key of the sequence
        uint32_t in_page[kLaneRows];
        auto read_pages = [&]() {
#pragma unroll
            for (int i = 0; i < kLaneRows; ++i) {
                const uint32_t r = lane + 32 * i;
                const uint32_t j = static_cast<uint32_t>(pre.t) * kKeys + r;
                uint32_t idx;
                a.cache.page.divmod(j, idx, in_page[i]);
                held[i] = r < kKeys && j < static_cast<uint32_t>(pre.len);
                page[i] = -1;
                if (held[i])
                    page[i] = __ldg(a.block_table + static_cast<int64_t>(pre.b) * a.max_pages + idx);
            }
        };
        auto copy_tile = [&](int stage) {
            if (to_copy > 0) {
                --to_copy;
                const int h = pre.u / a.head_tiles;
                int64_t off[kLaneRows];
                uint64_t valid = 0;
#pragma unroll
                for (int i = 0; i < kLaneRows; ++i) {
                    const bool ok = page[i] >= 0 && page[i] < a.cache.num_pages;
                    if (!ok && held[i]) record_device_error(a.err, kDevInvalidArg);
                    off[i] = ok ? page[i] * a.cache.page_stride + in_page[i] * a.cache.token_stride +
                                      h * a.cache.head_stride
                                : -1;
                    valid |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, ok)) << (32 * i);
                }
                if (lane == 0) s_valid[warp][stage] = valid;
                const uint32_t to = ring + stage * 2 * S::kHalf;
#pragma unroll
                for (int i = 0; i < kKeys * kPieces / 32; ++i) {
                    const uint32_t flat = i * 32 + lane;
                    const uint32_t r = flat / kPieces, c = flat % kPieces;
                    const int64_t o = __shfl_sync(
                        0xffffffffu, off[kLaneRows > 1 ? (i * 32 / kPieces) / 32 : 0], r & 31);
                    const uint32_t dst = to + piece<S::kRowBytes>(r, c);
                    const int64_t src = (o < 0 ? 0 : o) + c * 16;
                    const int bytes = o < 0 ? 0 : 16;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                                 "l"(a.cache.k + src), "r"(bytes)
                                 : "memory");
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + S::kHalf),
                                 "l"(a.cache.v + src), "r"(bytes)
                                 : "memory");
                }
                pre.next(a, units);
                if (to_copy > 0) read_pages();
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        read_pages();
#pragma unroll
        for (int s = 0; s < S::kStages - 1; ++s) copy_tile(s);

        uint32_t qf[kD / 16][4];
        float acc[kOT][4], m[2], l[2], sc[2];
        int begun = cur.t;  // the part's first tile
        int stage = 0;
        bool fresh = true;
        while (remaining > 0) {
            const int h = cur.u / a.head_tiles, row0 = (cur.u - h * a.head_tiles) * kRows;
            const int rows = min(kRows, a.group - row0);
            if (fresh) {
                fresh = false;
                // the unit's queries as the left operand; rows past the group are zero
                const __nv_bfloat16 *q = a.q + cur.b * a.q_row_stride +
                                         (static_cast<int64_t>(h) * a.group + row0) * kD;
                const bool r0 = g < rows, r1 = g + 8 < rows;
                const float base = a.scale * kLog2e *
                                   (a.cache.k_scale == nullptr ? 1.f : __ldg(a.cache.k_scale + h));
                sc[0] = sc[1] = base;
                if constexpr (kFp8) {
                    // channels 16 c + 4 tq .. + 3, as the widened keys have them
                    uint2 x[2][kD / 16];
                    float top[2] = {0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < kD / 16; ++c) {
                        const uint2 z = make_uint2(0, 0);
                        const int at = 16 * c + 4 * tq;
                        x[0][c] = r0 ? __ldg(reinterpret_cast<const uint2 *>(q + g * kD + at)) : z;
                        x[1][c] = r1 ? __ldg(reinterpret_cast<const uint2 *>(q + (g + 8) * kD + at)) : z;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 lo = unpack2<false>(x[i][c].x), hi = unpack2<false>(x[i][c].y);
                            top[i] = fmaxf(fmaxf(top[i], fmaxf(fabsf(lo.x), fabsf(lo.y))),
                                           fmaxf(fabsf(hi.x), fabsf(hi.y)));
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
                        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
                        // 2^e with the row's largest value in [2^13, 2^14) after it; an
                        // infinite or zero row is left as it is
                        int e = 13 - (static_cast<int>((__float_as_uint(top[i]) >> 23) & 0xff) - 127);
                        if (!(top[i] > 0.f) || isinf(top[i])) e = 0;
                        // in two steps: 2^e itself may not be a float
                        const float f1 = exp2f(static_cast<float>(e / 2));
                        const float f2 = exp2f(static_cast<float>(e - e / 2));
                        sc[i] = base / f1 / f2;
#pragma unroll
                        for (int c = 0; c < kD / 16; ++c) {
                            float2 lo = unpack2<false>(x[i][c].x), hi = unpack2<false>(x[i][c].y);
                            qf[c][i] = pack2<true>(lo.x * f1 * f2, lo.y * f1 * f2);
                            qf[c][i + 2] = pack2<true>(hi.x * f1 * f2, hi.y * f1 * f2);
                        }
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < kD / 16; ++c) {
                        const __nv_bfloat16 *x = q + 16 * c + 2 * tq;
                        qf[c][0] = r0 ? __ldg(reinterpret_cast<const uint32_t *>(x + g * kD)) : 0;
                        qf[c][1] = r1 ? __ldg(reinterpret_cast<const uint32_t *>(x + (g + 8) * kD)) : 0;
                        qf[c][2] = r0 ? __ldg(reinterpret_cast<const uint32_t *>(x + g * kD + 8)) : 0;
                        qf[c][3] = r1 ? __ldg(reinterpret_cast<const uint32_t *>(x + (g + 8) * kD + 8)) : 0;
                    }
                }
                begun = cur.t;
                m[0] = m[1] = -INFINITY;
                l[0] = l[1] = 0.f;
#pragma unroll
                for (int i = 0; i < kOT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
            }
            asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 2) : "memory");
            __syncwarp();  // the tile is in, and the one before it is read by every lane
            copy_tile(stage == 0 ? S::kStages - 1 : stage - 1);
            const uint32_t kt = ring + stage * 2 * S::kHalf, vt = kt + S::kHalf;

            // scores: rows g, g + 8; keys 8 n + 2 tq, + 1
            float s[kNT][4];
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
                s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
                for (int c = 0; c < kPieces; c += 4) {
                    uint32_t r[4];
                    ldsm4(r, kt + piece<S::kRowBytes>(8 * n + (lane & 7), c + (lane >> 3)));
                    if constexpr (kFp8) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma<kF16>(s[n], qf[c + i], e4m3x2_to_f16x2(r[i] & 0xffff),
                                      e4m3x2_to_f16x2(r[i] >> 16));
                    } else {
                        mma<kF16>(s[n], qf[c / 2], r[0], r[1]);
                        mma<kF16>(s[n], qf[c / 2 + 1], r[2], r[3]);
                    }
                }
            }
            const uint64_t valid = s_valid[warp][stage];
            constexpr uint64_t kAll = kKeys == 64 ? ~uint64_t{0} : (uint64_t{1} << (kKeys & 63)) - 1;
            float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[n][i] *= sc[i >> 1];
            }
            if (valid != kAll) {
#pragma unroll
                for (int n = 0; n < kNT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!(valid >> (8 * n + 2 * tq + (i & 1)) & 1)) s[n][i] = -INFINITY;
            }
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
                mt[0] = fmaxf(mt[0], fmaxf(s[n][0], s[n][1]));
                mt[1] = fmaxf(mt[1], fmaxf(s[n][2], s[n][3]));
            }
            float ref[2];
            bool grew = false;
            float shrink[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mt[i] = fmaxf(mt[i], __shfl_xor_sync(0xffffffffu, mt[i], 1));
                mt[i] = fmaxf(mt[i], __shfl_xor_sync(0xffffffffu, mt[i], 2));
                const float mn = fmaxf(m[i], mt[i]);
                ref[i] = mn == -INFINITY ? 0.f : mn;
                shrink[i] = ex2(m[i] - ref[i]);
                grew |= mn > m[i];
                m[i] = mn;
            }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int i = 0; i < 2; ++i) l[i] *= shrink[i];
#pragma unroll
                for (int n = 0; n < kOT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[n][i] *= shrink[i >> 1];
            }
            // weights, and their product with the values 16 keys at a time
            constexpr float kUp = kF16 ? 32768.f : 1.f;
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk) {
                uint32_t p[4], p2[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // j: rows g (even) or g + 8 (odd), keys of the first or second 8
                    const int n = 2 * kk + (j >> 1), i = j & 1;
                    float x = ex2(s[n][2 * i] - ref[i]), y = ex2(s[n][2 * i + 1] - ref[i]);
                    l[i] += x + y;
                    x *= kUp;
                    y *= kUp;
                    p[j] = pack2<kF16>(x, y);
                    const float2 hi = unpack2<kF16>(p[j]);
                    p2[j] = pack2<kF16>(x - hi.x, y - hi.y);
                }
                const uint32_t vr = 16 * kk + (lane & 15);
#pragma unroll
                for (int c = 0; c < kPieces; c += 2) {
                    uint32_t r[4];
                    // pieces c (r[0], r[1]) and c + 1, keys 0-7 and 8-15 of the 16
                    ldsm4_trans(r, vt + piece<S::kRowBytes>(vr, c + (lane >> 4)));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if constexpr (kFp8) {
                            // bytes: channel 2 g and 2 g + 1 of key 2 tq, then of key 2 tq + 1
                            const uint32_t x = __byte_perm(r[2 * i], 0, 0x3120);
                            const uint32_t y = __byte_perm(r[2 * i + 1], 0, 0x3120);
                            const uint32_t e0 = e4m3x2_to_f16x2(x & 0xffff), o0 = e4m3x2_to_f16x2(x >> 16);
                            const uint32_t e1 = e4m3x2_to_f16x2(y & 0xffff), o1 = e4m3x2_to_f16x2(y >> 16);
                            mma<kF16>(acc[2 * (c + i)], p, e0, e1);
                            mma<kF16>(acc[2 * (c + i) + 1], p, o0, o1);
                            mma<kF16>(acc[2 * (c + i)], p2, e0, e1);
                            mma<kF16>(acc[2 * (c + i) + 1], p2, o0, o1);
                        } else {
                            mma<kF16>(acc[c + i], p, r[2 * i], r[2 * i + 1]);
                            mma<kF16>(acc[c + i], p2, r[2 * i], r[2 * i + 1]);
                        }
                    }
                }
            }

            // ---- the end of a unit, or of the piece
            --remaining;
            const bool ends = cur.t == cur.tiles - 1;
            if (ends || remaining == 0) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
                    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
                }
                const bool whole = ends && begun == 0;
                const int64_t unit = static_cast<int64_t>(cur.b) * units + cur.u;
                const int64_t out_row = static_cast<int64_t>(cur.b) * a.q_heads + h * a.group + row0;
                float *part = nullptr;
                int pitch = kD;
                if (!whole) {
                    const int at = 2 * warp + (remaining == 0 ? 1 : 0);
                    if (remaining == 0) {
                        asm volatile("cp.async.wait_all;" ::: "memory");
                        __syncwarp();  // the ring is free: the part goes there
                        part = reinterpret_cast<float *>(s_ring + warp * S::kRing);
                        pitch = S::kPad;
                    } else {
                        part = a.ws.head + (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kRows * kD;
                    }
                    if (tq == 0) {
                        s_m[at][g] = m[0];
                        s_m[at][g + 8] = m[1];
                        s_l[at][g] = l[0];
                        s_l[at][g + 8] = l[1];
                    }
                    if (lane == 0) {
                        s_part[at].unit = unit;
                        s_part[at].starts = begun == 0;
                        s_part[at].ends = ends;
                        s_part[at].in_global = remaining != 0;
                    }
                }
                const float vs = (a.cache.v_scale == nullptr ? 1.f : __ldg(a.cache.v_scale + h)) / kUp;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = g + 8 * i;
                    if (row >= rows) continue;
                    const float f = whole ? (l[i] == 0.f ? 0.f : vs / l[i]) : vs;
                    if (whole && tq == 0 && a.lse != nullptr)
                        a.lse[out_row + row] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
                    if constexpr (kFp8) {
#pragma unroll
                        for (int c = 0; c < kD / 16; ++c) {
                            const float4 x = make_float4(acc[2 * c][2 * i] * f, acc[2 * c + 1][2 * i] * f,
                                                         acc[2 * c][2 * i + 1] * f,
                                                         acc[2 * c + 1][2 * i + 1] * f);
                            const int d = 16 * c + 4 * tq;
                            if (whole) write_out(a, (out_row + row) * kD + d, x);
                            else *reinterpret_cast<float4 *>(part + row * pitch + d) = x;
                        }
                    } else {
#pragma unroll
                        for (int n = 0; n < kOT; ++n) {
                            const float x = acc[n][2 * i] * f, y = acc[n][2 * i + 1] * f;
                            const int d = 8 * n + 2 * tq;
                            if (!whole) {
                                *reinterpret_cast<float2 *>(part + row * pitch + d) = make_float2(x, y);
                            } else if (a.o_bf16) {
                                *reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(a.o) +
                                                              (out_row + row) * kD + d) = pack2<false>(x, y);
                            } else {
                                *reinterpret_cast<float2 *>(static_cast<float *>(a.o) +
                                                            (out_row + row) * kD + d) = make_float2(x, y);
                            }
                        }
                    }
                }
                fresh = true;
            }
            cur.next(a, units);
            stage = stage == S::kStages - 1 ? 0 : stage + 1;
        }
    }
    __syncthreads();

    // ---- joining the CTA's parts: runs of one unit, in the list's order ------------------
    if (tid < 2) a.ws.meta[blockIdx.x * 2 + tid].unit = -1;
    __syncthreads();
    for (int e0 = 0; e0 < kParts;) {
        const int64_t unit = s_part[e0].unit;
        if (unit < 0) {
            ++e0;
            continue;
        }
        int e1 = e0 + 1, last = e0;  // the run is e0 .. e1 - 1 (places without a part among them)
        while (e1 < kParts && (s_part[e1].unit < 0 || s_part[e1].unit == unit)) {
            if (s_part[e1].unit == unit) last = e1;
            ++e1;
        }
        const bool starts = s_part[e0].starts, ends = s_part[last].ends;
        const int b = static_cast<int>(unit / units), u = static_cast<int>(unit - static_cast<int64_t>(b) * units);
        const int h = u / a.head_tiles, row0 = (u - h * a.head_tiles) * kRows;
        const int rows = min(kRows, a.group - row0);
        const int64_t out_row = static_cast<int64_t>(b) * a.q_heads + h * a.group + row0;
        const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (starts ? 1 : 0);
        for (int i = tid; i < rows * (kD / 4); i += kThreads) {
            const int row = i / (kD / 4), d = i % (kD / 4) * 4;
            float mm = -INFINITY;
            for (int e = e0; e <= last; ++e)
                if (s_part[e].unit == unit) mm = fmaxf(mm, s_m[e][row]);
            const float ref = mm == -INFINITY ? 0.f : mm;
            float ll = 0.f;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int e = e0; e <= last; ++e) {
                if (s_part[e].unit != unit) continue;
                const float w = ex2(s_m[e][row] - ref);
                const float *part =
                    s_part[e].in_global
                        ? a.ws.head + ((static_cast<int64_t>(blockIdx.x) * kWarps + (e >> 1)) * kRows + row) * kD
                        : reinterpret_cast<const float *>(s_ring + (e >> 1) * S::kRing) + row * S::kPad;
                const float4 y = *reinterpret_cast<const float4 *>(part + d);
                ll += w * s_l[e][row];
                x.x += w * y.x;
                x.y += w * y.y;
                x.z += w * y.z;
                x.w += w * y.w;
            }
            if (starts && ends) {
                const float f = ll == 0.f ? 0.f : 1.f / ll;
                write_out(a, (out_row + row) * kD + d,
                          make_float4(x.x * f, x.y * f, x.z * f, x.w * f));
                if (d == 0 && a.lse != nullptr)
                    a.lse[out_row + row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
            } else {
                *reinterpret_cast<float4 *>(a.ws.cut + (slot * kRows + row) * kD + d) = x;
                if (d == 0) {
                    a.ws.ml[(slot * kRows + row) * 2] = mm;
                    a.ws.ml[(slot * kRows + row) * 2 + 1] = ll;
                }
            }
        }
        if (tid == 0 && !(starts && ends)) {
            a.ws.meta[slot].unit = unit;
            a.ws.meta[slot].ends = ends;
        }
        e0 = last + 1;
    }

    // ---- sequences without keys ----------------------------------------------------------
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (valid_len(a, b) > 0) continue;
        for (int i = tid; i < a.q_heads * (kD / 4); i += kThreads)
            write_out(a, static_cast<int64_t>(b) * a.q_heads * kD + i * 4, make_float4(0.f, 0.f, 0.f, 0.f));
        if (a.lse != nullptr)
            for (int i = tid; i < a.q_heads; i += kThreads)
                a.lse[static_cast<int64_t>(b) * a.q_heads + i] = -INFINITY;
    }
}

// Joins the parts of the unit that CTA blockIdx.x of the first kernel began and
// did not finish: its slot 1 and slot 0 of the CTAs after it, up to the last.
template <int kD>
__global__ void __launch_bounds__(256) join_kernel(const Args a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c0 = blockIdx.x;
    const CutMeta first = a.ws.meta[c0 * 2 + 1];
    if (first.unit < 0) return;
    const int units = a.cache.heads * a.head_tiles;
    const int b = static_cast<int>(first.unit / units);
    const int u = static_cast<int>(first.unit - static_cast<int64_t>(b) * units);
    const int h = u / a.head_tiles, row0 = (u - h * a.head_tiles) * kRows;
    const int rows = min(kRows, a.group - row0);
    const int64_t out_row = static_cast<int64_t>(b) * a.q_heads + h * a.group + row0;
    int c1 = c0 + 1;  // the last part's CTA
    while (c1 < gridDim.x - 1 && a.ws.meta[c1 * 2].ends == 0) ++c1;
    for (int i = threadIdx.x; i < rows * (kD / 4); i += blockDim.x) {
        const int row = i / (kD / 4), d = i % (kD / 4) * 4;
        float mm = -INFINITY, ll = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = c0; c <= c1; ++c) {
            const int64_t slot = static_cast<int64_t>(c) * 2 + (c == c0 ? 1 : 0);
            const float mc = a.ws.ml[(slot * kRows + row) * 2], lc = a.ws.ml[(slot * kRows + row) * 2 + 1];
            const float4 y = *reinterpret_cast<const float4 *>(a.ws.cut + (slot * kRows + row) * kD + d);
            const float mn = fmaxf(mm, mc), ref = mn == -INFINITY ? 0.f : mn;
            const float f = ex2(mm - ref), w = ex2(mc - ref);
            ll = ll * f + lc * w;
            x.x = x.x * f + y.x * w;
            x.y = x.y * f + y.y * w;
            x.z = x.z * f + y.z * w;
            x.w = x.w * f + y.w * w;
            mm = mn;
        }
        const float f = ll == 0.f ? 0.f : 1.f / ll;
        write_out(a, (out_row + row) * kD + d, make_float4(x.x * f, x.y * f, x.z * f, x.w * f));
        if (d == 0 && a.lse != nullptr)
            a.lse[out_row + row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
    }
}

template <int kD, bool kFp8>
cudaError_t launch_shape(const Args &a, int ctas, cudaStream_t s) {
    using S = Shape<kD, kFp8>;
    constexpr int kSmem = S::kWarps * S::kRing;
    const cudaError_t e = ensure_dynamic_smem(
        reinterpret_cast<const void *>(&paged_decode_kernel<kD, kFp8>), kSmem);
    if (e != cudaSuccess) return e;
    paged_decode_kernel<kD, kFp8><<<ctas, S::kWarps * 32, kSmem, s>>>(a);
    const cudaError_t e1 = cudaGetLastError();
    if (e1 != cudaSuccess) return e1;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<kD>, a);
}

template <int kD>
cudaError_t launch_dim(const Args &a, int ctas, cudaStream_t s) {
    return a.cache.fp8 ? launch_shape<kD, true>(a, ctas, s) : launch_shape<kD, false>(a, ctas, s);
}

}  // namespace

size_t paged_decode_workspace_bytes(int, int, int, int head_dim) {
    return layout_bytes(head_dim, nullptr, nullptr);
}

cudaError_t launch_paged_decode(const __nv_bfloat16 *q, int64_t q_row_stride,
                                const PagedView &cache, const int32_t *block_table, int max_pages,
                                const int32_t *seq_lens, int B, int q_heads, float scale, void *o,
                                bool o_bf16, float *lse, void *workspace, unsigned int *err,
                                int num_sms, cudaStream_t s) {
    Args a;
    a.q = q;
    a.q_row_stride = q_row_stride;
    a.cache = cache;
    a.block_table = block_table;
    a.max_pages = max_pages;
    a.seq_lens = seq_lens;
    a.B = B;
    a.q_heads = q_heads;
    a.group = q_heads / cache.heads;
    a.head_tiles = (a.group + kRows - 1) / kRows;
    a.scale = scale;
    a.o = o;
    a.o_bf16 = o_bf16;
    a.lse = lse;
    a.err = err;
    layout_bytes(cache.head_dim, static_cast<uint8_t *>(workspace), &a.ws);
    const int ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
    return cache.head_dim == 64    ? launch_dim<64>(a, ctas, s)
           : cache.head_dim == 128 ? launch_dim<128>(a, ctas, s)
                                   : launch_dim<256>(a, ctas, s);
}

}  // namespace kda
