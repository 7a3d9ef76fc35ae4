// kda_paged_decode.cuh -- softmax attention of one new token per sequence over a
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
// a value at G query heads to a key head: HBM up to G = 100, had the tensor cores' full
// rate.  So what matters is that every SM has copies in flight from the first microsecond
// to the last, whatever the lengths, and that a warp's instructions for a tile take less
// time than its copy.  Measured, 8 query heads to a key head of 128: 64 sequences of 16 to
// 16384 keys 129 us (92 % of HBM), one of 262149 keys 163 us (97 %), 256 of 3500 to 8192 in
// 8 bits 453 us (100 %).  16 heads over 8 bits (73 %) and 24 or more (32: 67 %) are bound by
// the warps' instructions.
//
// Split.  A unit is (sequence, key head, group of 8, 16, 24 or 32 query heads); its keys
// are cut in tiles of 4 KB of keys and 4 KB of values (2 KB each for 24 or 32 heads,
// but 16 keys at least: 8 KB at 256 channels in bf16, 4 KB at 128).  The tiles of all
// units form one list; each CTA takes an equal, contiguous piece of it and each warp an
// equal part of that: long sequences are cut, short ones share a warp.  A warp's part ends in at most two cut units;
// their parts are joined within the CTA through shared memory, and what is cut
// between CTAs by a second, small kernel that is launched with the first and
// waits for it (programmatic dependent launch; a join by the CTA that is last to write
// its part ends 2 us later: fences and a count cost more than the kernel).  Where the
// block table has no room for long sequences, the pieces are moved to the units' ends
// instead, and the second kernel is not launched.
//
// A warp copies its own tiles, by 16-byte cp.async into its own ring of tile
// halves (no barrier between warps); the page numbers of a tile are read one tile
// earlier.  Rows are swizzled (16-byte pieces xor row) so that ldmatrix meets no
// bank twice.  The products run on the warp's matrix instructions with the keys
// (then the channels) as the 16 rows and 8 query heads as the columns:
// S^T = K Q^T, O^T += V^T P^T, so that no row of the operand that is loaded is
// padding; the weights turn from accumulator to right operand by transposing
// 8 x 8 blocks in registers (movmatrix).  (tcgen05.mma takes 64 or 128 rows from
// shared memory and would need the weights there; at 8 heads the tensor pipe is 14 %
// busy, 28 % over 8 bits; at 16 over 8 bits 41 %.)
//
// Precision: scores, maxima, sums and outputs in fp32.  For the product with the
// values a weight is a sum of bf16 numbers: two, 16 bits together, for a bf16
// output (one would leave up to 2^-8 of every weight, as much as the output's own
// rounding), three, 24 bits, for an fp32 one; the products are free here (see
// Bound).  The matrix instructions cut their sums off instead of rounding them,
// which adds up over a warp's tiles (4e-5 over 300; fp32 arithmetic 5e-7): an fp32
// output, and a bf16 one of up to 8 heads, takes each tile's products in a sum of their
// own and adds it in fp32.  A bf16 output of more heads does not, where that costs up to
// 12 % (32 heads 205 and 230 us; 8 heads 140.4 and 140.9).
// An 8-bit cache is widened to fp16, which holds every e4m3 value; the
// queries are scaled by a power of two for each head, so that fp16 holds their bf16
// values too, and the weights are two fp16 numbers, 22 bits, of the weight times 2^13
// (2^12).  fp16 ends at 2^-24, so these words keep a weight to 2^-38 of the largest,
// which a bf16 output covers.  For an fp32 output the second word is 2^12 times larger,
// its products have a sum of their own in each tile, and a weight is kept to 2^-49 of
// the largest (fp32 outputs of 16 heads over 8 bits 189.6 us without that, 195.7 with
// it; 8 heads of 256 153 and 161).  The sums of the weights are fp32 throughout.
#pragma once

#include <cfloat>

#include <cuda_fp16.h>

#include "kda_internal.cuh"
#include "kda_paged.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace paged {

constexpr int kMaxCtas = 160;  // sizes the workspace and the join's weights; more SMs stay idle
constexpr int kMaxWarps = 12;
constexpr int kMaxSide = 4;   // key heads side by side

// What is cut at a CTA's ends: its first unit's part (begun by an earlier CTA)
// in slot 0, its last unit's (begun here, not finished) in slot 1.
struct Layout {      // of the workspace
    float *ml;       // [ctas][2][side][heads][2], side: key heads side by side (see List)
    float *cut;      // [ctas][2][side][heads][D]
    float *head;     // [ctas][warps][heads][D]: a warp's first part, until its CTA joins it
};

inline size_t align256(size_t x) { return (x + 255) & ~size_t{255}; }

inline size_t layout_bytes(int heads, int head_dim, uint8_t *base, Layout *l) {
    const size_t part = static_cast<size_t>(heads) * head_dim * 4;
    const size_t cut = align256(static_cast<size_t>(kMaxCtas) * 2 * kMaxSide * heads * 2 * 4);
    const size_t head = align256(cut + kMaxCtas * 2 * kMaxSide * part);
    if (l != nullptr) {
        l->ml = reinterpret_cast<float *>(base);
        l->cut = reinterpret_cast<float *>(base + cut);
        l->head = reinterpret_cast<float *>(base + head);
    }
    return head + kMaxCtas * kMaxWarps * part;
}

// Query heads of a unit: all of a group of up to 32 (16 at 256 channels), in eights, so
// that its keys are read once; of a larger group as many as share its units evenly.
inline int unit_heads(int group, int head_dim) {
    const int most = head_dim == 256 ? 16 : 32, units = (group + most - 1) / most;
    return (group + units * 8 - 1) / (units * 8) * 8;
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
    float *lse;
    Layout ws;
    unsigned int *err;
    int side_log;  // key heads that may go side by side (see List), as a power of two
};

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kSideTiles = 8;  // heads go side by side in lists of so many tiles a warp

constexpr int max_of(int a, int b) { return a > b ? a : b; }

// kN: groups of 8 query heads in a unit.  kWide: fp32 outputs.  Warps: as many as the
// accumulators (kD / 4 * kN registers a lane) leave registers for, so that one warp's
// instructions overlap another's waits (24 heads of 64: 118 us with 8, 110 with 12; now 104).
template <int kD_, bool kFp8_, int kN_, bool kWide_>
struct Shape {
    static constexpr int kD = kD_, kN = kN_;
    static constexpr bool kFp8 = kFp8_, kWide = kWide_;
    static constexpr int kRowBytes = kD * (kFp8 ? 1 : 2);
    // keys of a tile: 4 KB of them, 2 KB where 24 or 32 heads' scores would fill the registers,
    // but 16, the rows of a product, in any case (8 KB of 256 channels in bf16; of 128, 4 KB)
    static constexpr int kKeys = max_of(16, (kN >= 3 ? 2048 : 4096) / kRowBytes);
    static constexpr int kHalf = kKeys * kRowBytes;                        // its keys, in bytes
    static constexpr int kWarps = kD == 256 || kN == 4 || (kN == 3 && kD == 128) ? 8 : 12;
    static_assert(kWarps % kMaxSide == 0, "heads side by side share the warps evenly");
    // halves of a warp's ring: one that is read, and 96 KB in flight an SM in the others
    // (more gain nothing, and keep the SMs further apart: one sequence of 262149 keys 168 us
    // at 96, 181 at 144 KB; 24 heads of 64 104.0 and 104.6), but two of them in any case
    // (128 KB at 256 channels in bf16)
    static constexpr int kSlots = max_of(2, 96 * 1024 / (kWarps * kHalf)) + 1;
    // key heads may go side by side (see List): short rows, and HBM-bound
    static constexpr bool kSide = kRowBytes < 256 && (kD == 64 || kN == 1);
    static constexpr int kHeads = 8 * kN;
    // each tile's products in sums of their own (see Precision)
    static constexpr bool kApart = kWide || kN == 1;
    static constexpr int kPitch = kD + 4;                                  // floats of a part's row
    // the ring takes the warp's last part in the end
    static constexpr int kRing = max_of(kSlots * kHalf, (kHeads * kPitch * 4 + 1023) / 1024 * 1024);
    // The queries lie beside the ring, as operands, where they would fill the registers (32
    // heads of 128: 251 us with spills, 208 so, now 205; 16 over 8 bits: 200 and 185).
    static constexpr int kQBytes = kD / 16 * kN * 256;
    static constexpr bool kQShared = kD * kN >= 256 && kWarps * (kRing + kQBytes) <= 220 * 1024;
    static constexpr int kQ = kQShared ? kQBytes : 0;
    static constexpr int kSmem = kWarps * (kRing + kQ);
    static_assert(kSlots >= 3 && kSlots <= 7, "the masks' ring holds the tiles in flight");
};

// x, or the least normal number where x is below it; a NaN stays (fmaxf would drop it).
__device__ __forceinline__ float at_least_normal(float x) { return x < FLT_MIN ? FLT_MIN : x; }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The largest of three, NaN where one of them is.
__device__ __forceinline__ float max3_nan(float x, float y, float z) {
    float m;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
    return m;
}

// Volatile: they stay between the wait for a tile and the copy that replaces it.
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// The transpose of an 8 x 8 matrix of 16-bit values, a row to four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// c (16 x 8, fp32) += a (16 x 16) b (16 x 8), bf16 or fp16 operands.
template <bool kF16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
    if constexpr (kF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two e4m3 values as two fp16 values: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x) {
    uint32_t y;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(static_cast<uint16_t>(x)));
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

// n / d, n >= 0, d > 0: by 32 bits where they hold n (a 64-bit division is a call).
__device__ __forceinline__ int64_t div64(int64_t n, uint32_t d) {
    if (n >> 32 == 0) return static_cast<uint32_t>(n) / d;
    return static_cast<uint64_t>(n) / d;
}

__device__ __forceinline__ int valid_len(const Args &a, int b) {
    const int n = a.seq_lens[b];
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
    int b, u;        // b = -1: none
    int starts, ends;
    int in_global;   // its sums are in the workspace (else in the warp's ring)
};

// A part's sums, and the parts of one unit, when a CTA joins them.
struct PartAt {
    const float *sums;  // [heads][pitch], shared or global
    int pitch, part, run;
};
struct Run {
    int begin, end;     // parts
    int rows, whole;    // query heads; the unit's first and last keys are among them
    int64_t out_row, slot;
};

// Where a unit's queries and outputs are.
struct UnitRows {
    int h, rows;      // key head; query heads
    int64_t out_row;  // the first of them in [B, q_heads]

    __device__ __forceinline__ UnitRows(const Args &a, int b, int u, int heads) {
        h = u / a.head_tiles;
        const int row0 = (u - h * a.head_tiles) * heads;
        rows = min(heads, a.group - row0);
        out_row = static_cast<int64_t>(b) * a.q_heads + h * a.group + row0;
    }
};

template <bool kWide>
__device__ __forceinline__ void write_out(const Args &a, int64_t at, float4 x) {
    if constexpr (!kWide) {
        uint2 w;
        w.x = pack2<false>(x.x, x.y);
        w.y = pack2<false>(x.z, x.w);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + at) = w;
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + at) = x;
    }
}

__device__ __forceinline__ void write_lse(const Args &a, int64_t row, float m, float l) {
    if (a.lse != nullptr) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// 16 bytes to shared memory, or zeros (nothing is read then).  Evicted from L2
// first: a key is read once, and what else is there (weights, code) is not.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src, bool real) {
    asm volatile("{\n\t.reg .b64 pol;\n\tcreatepolicy.fractional.L2::evict_first.b64 pol, 1.0;\n\t"
                 "cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, pol;\n\t}" ::"r"(dst),
                 "l"(src), "r"(real ? 16 : 0)
                 : "memory");
}

// The tiles that a warp copies: its part of the list, one half at a time.
// kOnePage: a tile never spans two pages.
template <class S, bool kOnePage>
struct Copier {
    static constexpr int kKeys = S::kKeys, kPieces = S::kRowBytes / 16;
    static constexpr int kLaneRows = !kOnePage && kKeys > 32 ? 2 : 1;
    static constexpr int kCopies = S::kHalf / 512;           // 16-byte copies of a lane
    Cursor<kKeys> at;
    int side_log, side;                                      // the list's, and this warp's head
    int64_t left;                                            // tiles to begin
    int page[kLaneRows];                                     // of this lane's rows of tile `at`
    bool held[kLaneRows];                                    // the row is a key of the sequence
    uint32_t in_page[kLaneRows];
    // the tile whose values are next: where its rows are
    int64_t off[kLaneRows];                                  // kOnePage: of row 0
    int rows;                                                // rows to copy, the rest 0; -1: no tile

    __device__ __forceinline__ void read_pages(const Args &a, int lane) {
#pragma unroll
        for (int i = 0; i < kLaneRows; ++i) {
            const uint32_t r = kOnePage ? 0 : lane + 32 * i;
            const uint32_t j = static_cast<uint32_t>(at.t) * kKeys + r;
            uint32_t idx;
            a.cache.page.divmod(j, idx, in_page[i]);
            held[i] = r < kKeys && j < static_cast<uint32_t>(at.len);
            page[i] = -1;
            if (held[i])
                page[i] = a.block_table[static_cast<int64_t>(at.b) * a.max_pages + idx];
        }
    }

    __device__ __forceinline__ void begin(const Args &a, const Cursor<kKeys> &c, int64_t tiles,
                                          int log, int head, int lane) {
        at = c;
        side_log = log;
        side = head;
        left = tiles;
        read_pages(a, lane);
    }

    // Copies the keys of the next tile to the slot; mask: which of its rows are keys.
    __device__ __forceinline__ void keys(const Args &a, int units, int lane, uint32_t to,
                                         uint64_t *mask) {
        rows = -1;
        if (left > 0) {
            uint64_t valid = 0;
            const int u = S::kSide ? (at.u << side_log) + side : at.u;
            const int64_t h = (a.head_tiles == 1 ? u : u / a.head_tiles) * a.cache.head_stride;
            if constexpr (kOnePage) {
                const bool ok = page[0] >= 0 && page[0] < a.cache.num_pages;
                if (!ok) record_device_error(a.err, kDevInvalidArg);
                rows = ok ? min(kKeys, at.len - at.t * kKeys) : 0;
                off[0] = ok ? page[0] * a.cache.page_stride + in_page[0] * a.cache.token_stride + h : 0;
                valid = rows == 64 ? ~uint64_t{0} : (uint64_t{1} << rows) - 1;
            } else {
                rows = kKeys;
#pragma unroll
                for (int i = 0; i < kLaneRows; ++i) {
                    const bool ok = page[i] >= 0 && page[i] < a.cache.num_pages;
                    if (!ok && held[i]) record_device_error(a.err, kDevInvalidArg);
                    off[i] = ok ? page[i] * a.cache.page_stride + in_page[i] * a.cache.token_stride + h
                                : -1;
                    valid |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, ok)) << (32 * i);
                }
            }
            if (lane == 0) *mask = valid;
            copy(a, a.cache.k, lane, to);
            at.next(a, units);
            if (--left > 0) read_pages(a, lane);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }

    // Copies the values of the tile whose keys were last.
    __device__ __forceinline__ void values(const Args &a, int lane, uint32_t to) {
        if (rows >= 0) copy(a, a.cache.v, lane, to);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }

    __device__ __forceinline__ void copy(const Args &a, const uint8_t *src, int lane, uint32_t to) {
        const uint32_t r0 = lane / kPieces, c = lane % kPieces;
        if constexpr (kOnePage) {
            constexpr uint32_t kStep = 32 / kPieces;     // rows of one copy of the warp
            const uint8_t *p = src + off[0] + r0 * a.cache.token_stride + c * 16;
            const int64_t step = kStep * a.cache.token_stride;
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int r = i * kStep + r0;
                copy16(to + piece<S::kRowBytes>(r, c), r < rows ? p : src, r < rows);
                p += step;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const uint32_t r = i * 32 / kPieces + r0;
                const int64_t o = __shfl_sync(
                    0xffffffffu, off[kLaneRows > 1 ? (i * 32 / kPieces) / 32 : 0], r & 31);
                copy16(to + piece<S::kRowBytes>(r, c), src + (o < 0 ? 0 : o) + c * 16, o >= 0);
            }
        }
    }
};

// The place of position pos < the total of the list; called by a whole warp, whose lanes
// hold the sequences from b_lo on, at positions before .. after - 1.  Not inlined: it is
// wanted three times, and short calls wait for instructions more than for anything.
template <int kKeys>
__device__ __noinline__ Cursor<kKeys> find_tile(const Args &a, int units, int64_t pos, int b_lo,
                                                int64_t before, int64_t after) {
    Cursor<kKeys> c;
    c.b = c.u = c.t = c.len = 0;
    const bool owner = pos >= before && pos < after;
    if (owner) {
        int64_t left = pos - before;
        for (c.b = b_lo;; ++c.b) {
            c.set_len(valid_len(a, c.b));
            const int64_t here = static_cast<int64_t>(c.tiles) * units;
            if (left < here) break;
            left -= here;
        }
        c.u = static_cast<int>(div64(left, c.tiles));
        c.t = static_cast<int>(left - static_cast<int64_t>(c.u) * c.tiles);
    }
    const int src = 31 - __clz(__ballot_sync(0xffffffffu, owner));
    c.b = __shfl_sync(0xffffffffu, c.b, src);
    c.u = __shfl_sync(0xffffffffu, c.u, src);
    c.t = __shfl_sync(0xffffffffu, c.t, src);
    c.set_len(__shfl_sync(0xffffffffu, c.len, src));
    return c;
}

// The list of tiles and its pieces, as a warp sees it: every warp sums the lengths for
// itself (they come out of L1 after the first), lane i over sequences
// i ceil(B / 32) .. , so that no barrier precedes the first copy.
//
// Where a token's rows lie head by head and are short (64 or 128 bytes), warps that read one
// head's take a part of each DRAM burst and page.  In long lists 2 or 4 neighbouring key
// heads then go side by side: a place of the list is a tile of each of them, and warp w of
// a CTA walks the CTA's piece for head w mod 2 or 4, so that the CTA's warps read
// neighbouring rows at nearly the same time.
template <class S>
struct List {
    static constexpr int kKeys = S::kKeys, kWarps = S::kWarps;
    int64_t before, after;   // positions of the list in this lane's sequences
    int64_t total, q, r;     // CTA i's piece: q positions, one more in the first r
    int b_lo, units;         // units of a sequence (of the heads side by side, each)
    int many_log;            // side by side, as a power of two
    int filled, filled_before;  // sequences with keys: this lane's, and before them
    uint32_t ctas;           // that have a piece
    bool one_each, whole;    // pieces are units, or end where units end

    static __device__ __forceinline__ uint32_t tiles_of(const Args &a, int b) {
        return (static_cast<uint32_t>(valid_len(a, b)) + kKeys - 1) / kKeys;
    }

    __device__ __forceinline__ List(const Args &a, int lane, int grid) {
        const int chunk = (a.B + 31) / 32;
        b_lo = min(a.B, lane * chunk);
        const int b_hi = min(a.B, b_lo + chunk);
        int64_t mine = 0;
        uint32_t longest = 0;
        filled = 0;
#pragma unroll 4
        for (int b = b_lo; b < b_hi; ++b) {
            const uint32_t n = tiles_of(a, b);
            mine += n;
            filled += n > 0;
            longest = max(longest, n);
        }
        before = mine;
        filled_before = filled;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, before, d);
            const int y = __shfl_up_sync(0xffffffffu, filled_before, d);
            if (lane >= d) {
                before += x;
                filled_before += y;
            }
        }
        longest = __reduce_max_sync(0xffffffffu, longest);
        const int64_t tiles = __shfl_sync(0xffffffffu, before, 31);
        units = a.cache.heads * a.head_tiles;
        many_log = tiles * units >= kSideTiles * kWarps * static_cast<int64_t>(grid) ? a.side_log : 0;
        units >>= side_log();
        total = tiles * units;
        const int sequences = __shfl_sync(0xffffffffu, filled_before, 31);
        filled_before -= filled;
        before = (before - mine) * units;
        after = before + mine * units;
        // Whole units to a CTA where that makes no CTA's load larger by more than two tiles a
        // warp (0.2 us a tile; joining between CTAs costs some 5 us, with its launch): one
        // unit each where there are few, pieces moved back to a unit's start where units
        // are short.
        const int64_t all_units = static_cast<int64_t>(sequences) * units;
        one_each = all_units <= grid && longest <= div64(total, grid) + 2 * warps();
        whole = one_each || longest <= 2 * warps();
        // as many CTAs as leave a tile to each warp (a unit to each CTA), all of the
        // grid for longer lists
        const int64_t want = whole ? all_units : div64(total + warps() - 1, warps());
        ctas = static_cast<uint32_t>(want < grid ? want : grid);
        q = ctas == 0 ? 0 : div64(total, ctas);
        r = total - q * ctas;
    }

    __device__ __forceinline__ int side_log() const { return S::kSide ? many_log : 0; }
    // a CTA's warps for each of the heads side by side
    __device__ __forceinline__ int warps() const { return kWarps >> side_log(); }

    // The place of position pos < total; called by a whole warp.
    __device__ __forceinline__ Cursor<kKeys> find(const Args &a, int64_t pos) const {
        return find_tile<kKeys>(a, units, pos, b_lo, before, after);
    }

    // Where an even piece begins, and which holds a position (not `whole`).
    __device__ __forceinline__ int64_t even_begin(int64_t cta) const { return cta * q + min(cta, r); }
    __device__ __forceinline__ int even_piece_of(int64_t pos) const {
        const int64_t longer = r * (q + 1);
        return static_cast<int>(pos < longer ? div64(pos, static_cast<uint32_t>(q + 1))
                                             : r + div64(pos - longer, static_cast<uint32_t>(q)));
    }

    // CTA `cta`'s piece, cta < ctas; called by a whole warp.
    __device__ __forceinline__ void piece(const Args &a, uint32_t cta, int64_t &lo, int64_t &hi) const {
        if (one_each) {
            // unit `cta`: of the sequence before which there are `skip` with keys
            const int skip = cta / units, u = cta - skip * units;
            const bool owner = skip >= filled_before && skip < filled_before + filled;
            if (owner) {
                int left = skip - filled_before;
                lo = before;
                for (int b = b_lo;; ++b) {
                    hi = tiles_of(a, b);
                    if (hi > 0 && --left < 0) break;
                    lo += hi * units;
                }
                lo += u * hi;
                hi += lo;
            }
            const int src = 31 - __clz(__ballot_sync(0xffffffffu, owner));
            lo = __shfl_sync(0xffffffffu, lo, src);
            hi = __shfl_sync(0xffffffffu, hi, src);
            return;
        }
        lo = even_begin(cta);
        hi = even_begin(cta + int64_t{1});
        if (whole) {
            if (hi < total) hi -= find(a, hi).t;
            lo -= find(a, lo).t;
        }
    }
};

__device__ __forceinline__ bool any_nonfinite(uint32_t two_bf16) {
    return (two_bf16 & 0x7f80u) == 0x7f80u || (two_bf16 & 0x7f800000u) == 0x7f800000u;
}

// An infinite value times a weight in words is a NaN, from the words that are 0 or negative.
// So where a sum of the part of a unit that keys j0 .. j1 - 1 make is NaN, it is taken again
// over the infinite and NaN values alone, with whole weights, as fp32 arithmetic has it; a
// sum that meets none stays NaN.  Rare and slow: not inlined, and nothing of it is on the way
// of finite values (inlined it costs the kernel registers: 64 ragged sequences 127 -> 130 us,
// 12 heads of 256 160 -> 265).
// The unit: of sequence b, query heads `out_row` .. + rows - 1 on key head h.  sums: the
// lane's, [d][n][4]; sc, minus: [n][2], as in the kernel.
template <class S>
__device__ __noinline__ void nonfinite_sums(const Args &a, int b, int h, int num_rows,
                                            int64_t out_row, int64_t j0, int64_t j1, float *sums,
                                            const float *sc, const float *minus) {
    constexpr int kD = S::kD, kN = S::kN, kSums = kD / 4 * kN;
    const int lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
    uint32_t was[(kSums + 31) / 32] = {};  // the sums that are NaN
#pragma unroll
    for (int e = 0; e < kSums; ++e)
        if (isnan(sums[e])) {
            was[e / 32] |= 1u << (e % 32);
            sums[e] = 0.f;
        }
    const __nv_bfloat16 *q = a.q + b * a.q_row_stride + (out_row - static_cast<int64_t>(b) * a.q_heads) * kD;
#pragma unroll 1
    for (; j0 < j1; j0 += 32) {
        // a lane looks through a key's values
        int64_t off = 0;
        bool hit = false;
        if (j0 + lane < j1) {
            uint32_t idx, r;
            a.cache.page.divmod(static_cast<uint32_t>(j0 + lane), idx, r);
            const int page = a.block_table[static_cast<int64_t>(b) * a.max_pages + idx];
            if (page >= 0 && page < a.cache.num_pages) {
                off = page * a.cache.page_stride + r * a.cache.token_stride + h * a.cache.head_stride;
                const uint4 *v = reinterpret_cast<const uint4 *>(a.cache.v + off);
#pragma unroll 4
                for (int c = 0; c < kD / 8; ++c) {
                    const uint4 x = v[c];
                    hit |= any_nonfinite(x.x) || any_nonfinite(x.y) || any_nonfinite(x.z) ||
                           any_nonfinite(x.w);
                }
            }
        }
#pragma unroll 1
        for (uint32_t hits = __ballot_sync(0xffffffffu, hit); hits != 0; hits &= hits - 1) {
            const int64_t at = __shfl_sync(0xffffffffu, off, __ffs(hits) - 1);
            const __nv_bfloat16 *k = reinterpret_cast<const __nv_bfloat16 *>(a.cache.k + at);
            const __nv_bfloat16 *v = reinterpret_cast<const __nv_bfloat16 *>(a.cache.v + at);
            float w[kN][2] = {};
#pragma unroll 1
            for (int row = 0; row < num_rows; ++row) {
                float dot = 0.f;
                for (int c = lane; c < kD; c += 32)
                    dot = fmaf(bf16_to_f32(q[row * kD + c]), bf16_to_f32(k[c]), dot);
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
                if (a.scale < 0.f) dot = -dot;
#pragma unroll
                for (int e = 0; e < 2 * kN; ++e)
                    if (row == 8 * (e / 2) + 2 * tq + e % 2) w[e / 2][e % 2] = ex2(fmaf(dot, sc[e], minus[e]));
            }
#pragma unroll
            for (int e = 0; e < kSums; ++e) {
                const float x = bf16_to_f32(v[16 * (e / (kN * 4)) + g + 8 * (e % 4 / 2)]);
                if (!isfinite(x) && (was[e / 32] >> (e % 32) & 1) != 0) sums[e] += w[e / 4 % kN][e % 2] * x;
            }
        }
    }
#pragma unroll
    for (int e = 0; e < kSums; ++e)
        if ((was[e / 32] >> (e % 32) & 1) != 0 && sums[e] == 0.f) sums[e] = NAN;
}

template <class S, bool kOnePage>
__global__ void __launch_bounds__(S::kWarps * 32, 1) paged_decode_kernel(const __grid_constant__ Args a) {
    constexpr int kD = S::kD, kN = S::kN, kHeads = S::kHeads;
    constexpr bool kFp8 = S::kFp8, kF16 = S::kFp8, kWide = S::kWide;
    constexpr bool kThird = kWide && !kF16;  // a third word of the weights
    constexpr int kWarps = S::kWarps, kThreads = kWarps * 32, kKeys = S::kKeys;
    constexpr int kBlocks = kKeys / 16;   // score blocks of 16 keys
    constexpr int kOT = kD / 16;          // output blocks of 16 channels
    constexpr int kParts = 2 * kWarps;
    // log2 of the most that a weight may be over 1 (see the reference below), and of what
    // the weights are multiplied by.  With it at most 1 over bf16, so that no sum leaves
    // fp32 that a sum of weights times values would not; just below fp16's 2^16 over 8 bits,
    // where values are small: what the words drop is then a fixed part of the largest weight
    // (see Precision), smaller the nearer the reference is (16 heads 184.0 us with 7, 184.8
    // with 3, 185.4 with 2, 187.1 with 1).
    constexpr float kSlack = !kF16 ? 7.f : kWide ? 3.f : 2.f, kUp = kF16 ? 15.f - kSlack : -kSlack;
    // what an fp32 output's second fp16 word is multiplied by: below 2^15 then, like the first
    constexpr float kLow = kF16 && kWide ? 4096.f : 1.f;
    static_assert(kParts <= 32, "a warp finds the runs");

    extern __shared__ __align__(1024) uint8_t s_ring[];
    __shared__ uint64_t s_valid[kWarps][4];
    __shared__ Part s_part[kParts];
    __shared__ float s_m[kParts][kHeads], s_l[kParts][kHeads], s_w[kParts][kHeads];
    __shared__ Run s_run[kParts];
    __shared__ PartAt s_at[kParts];
    __shared__ int s_runs, s_parts;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, tq = lane & 3;
    wait_for_kernel_before();

    const List<S> list(a, lane, gridDim.x);
    const int units = list.units, side_log = list.side_log();
    // this warp's head of those side by side, its place among the warps of that head, and
    // in the order that parts are joined in
    const int side = warp & ((1 << side_log) - 1), sub = warp >> side_log;
    const int place = side * list.warps() + sub;
    if (lane < 2) s_part[2 * place + lane].b = -1;
    __syncwarp();
    int64_t remaining = 0, begin = 0;  // this warp's tiles
    int64_t paced = 0;                 // fours of tiles that every warp of the CTA has
    if (blockIdx.x < list.ctas) {
        int64_t lo, hi;
        list.piece(a, blockIdx.x, lo, hi);
        const int64_t per = div64(hi - lo, list.warps()), more = hi - lo - per * list.warps();
        begin = lo + sub * per + min(static_cast<int64_t>(sub), more);
        remaining = per + (sub < more);
        paced = per / 4;
    }

    // ---- a warp's part of the piece --------------------------------------------------------
    if (remaining > 0) {
        const uint32_t ring = sm100::smem_addr(s_ring) + place * S::kRing;
        Cursor<kKeys> cur = list.find(a, begin);
        Copier<S, kOnePage> copier;
        copier.begin(a, cur, remaining, side_log, side, lane);
        int put = 0, copied = 0;  // the slot of the next half to copy; tiles begun
        auto next_slot = [&](int s) { return s == S::kSlots - 1 ? 0 : s + 1; };
        auto copy_keys = [&]() {
            copier.keys(a, units, lane, ring + put * S::kHalf, &s_valid[warp][copied++ & 3]);
            put = next_slot(put);
        };
        auto copy_values = [&]() {
            copier.values(a, lane, ring + put * S::kHalf);
            put = next_slot(put);
        };
        // kSlots - 1 halves ahead: with an odd number of slots the keys of a tile are
        // replaced by keys, with an even number by values
        constexpr bool kOdd = S::kSlots % 2 == 1;
#pragma unroll 1
        for (int i = 0; i < (S::kSlots - 1) / 2; ++i) {
            copy_keys();
            copy_values();
        }
        if (!kOdd) copy_keys();

        uint32_t qf[kOT][kN][2];
        uint2 *q_here = reinterpret_cast<uint2 *>(s_ring + kWarps * S::kRing + place * S::kQ) + lane;
        float acc[kOT][kN][4], m[kN][2], minus[kN][2], l[kN][2], sc[kN][2];
        int begun = cur.t;  // the part's first tile
        int slot = 0, tile = 0;
        bool fresh = true;
        while (true) {
            const int unit = (cur.u << side_log) + side;
            const UnitRows rows(a, cur.b, unit, kHeads);
            if (fresh) {
                // the unit's queries as the right operand (head 8 n + g); heads past the
                // group are zero
                fresh = false;
                const __nv_bfloat16 *q = a.q + cur.b * a.q_row_stride +
                                         (rows.out_row - static_cast<int64_t>(cur.b) * a.q_heads) * kD;
                const float factor = a.scale * kLog2e *
                                     (a.cache.k_scale == nullptr ? 1.f : a.cache.k_scale[rows.h]);
                // a negative factor's sign goes to the queries; zero times a left-out key's
                // -inf would be NaN
                const float base = at_least_normal(fabsf(factor));
                const uint32_t sign = factor < 0.f ? 0x80008000u : 0u;
#pragma unroll
                for (int n = 0; n < kN; ++n) {
                    const bool real = 8 * n + g < rows.rows;
                    const __nv_bfloat16 *x = q + (8 * n + g) * kD;
                    if constexpr (kFp8) {
                        // channels 16 c + 4 tq .. + 3, as the widened keys have them
                        float top = 0.f;
#pragma unroll
                        for (int c = 0; c < kOT; ++c) {
                            uint2 z = make_uint2(0, 0);
                            if (real) z = *reinterpret_cast<const uint2 *>(x + 16 * c + 4 * tq);
                            qf[c][n][0] = z.x;
                            qf[c][n][1] = z.y;
                            const float2 u0 = unpack2<false>(z.x), u1 = unpack2<false>(z.y);
                            top = fmaxf(fmaxf(top, fmaxf(fabsf(u0.x), fabsf(u0.y))),
                                        fmaxf(fabsf(u1.x), fabsf(u1.y)));
                        }
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                        // 2^e puts the head's largest value in [2^13, 2^14); an infinite or
                        // zero head is left as it is.  In two steps: 2^e itself may not be a
                        // float.
                        int e = 13 - (static_cast<int>((__float_as_uint(top) >> 23) & 0xff) - 127);
                        if (!(top > 0.f) || isinf(top)) e = 0;
                        const float f1 = exp2f(static_cast<float>(e / 2));
                        const float f2 = exp2f(static_cast<float>(e - e / 2));
#pragma unroll
                        for (int c = 0; c < kOT; ++c)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float2 u = unpack2<false>(qf[c][n][i]);
                                qf[c][n][i] = pack2<true>(u.x * f1 * f2, u.y * f1 * f2) ^ sign;
                            }
                        // the scores' columns are heads 2 tq, 2 tq + 1
                        const float mine_sc = at_least_normal(base / f1 / f2);
                        sc[n][0] = __shfl_sync(0xffffffffu, mine_sc, 8 * tq);
                        sc[n][1] = __shfl_sync(0xffffffffu, mine_sc, 8 * tq + 4);
                    } else {
                        sc[n][0] = sc[n][1] = base;
#pragma unroll
                        for (int c = 0; c < kOT; ++c)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                qf[c][n][i] = real ? *reinterpret_cast<const uint32_t *>(
                                                         x + 16 * c + 8 * i + 2 * tq) ^ sign
                                                   : 0;
                    }
                    if constexpr (S::kQShared) {
#pragma unroll
                        for (int c = 0; c < kOT; ++c)
                            q_here[(c * kN + n) * 32] = make_uint2(qf[c][n][0], qf[c][n][1]);
                    }
                    m[n][0] = m[n][1] = -INFINITY;
                    minus[n][0] = minus[n][1] = 0.f;
                    l[n][0] = l[n][1] = 0.f;
#pragma unroll
                    for (int d = 0; d < kOT; ++d)
                        acc[d][n][0] = acc[d][n][1] = acc[d][n][2] = acc[d][n][3] = 0.f;
                }
                begun = cur.t;
            }

            // the warps of a CTA keep pace, four tiles at a time, as far as all have tiles:
            // otherwise the last ends some 8 % after the first
            if ((tile & 3) == 3 && --paced >= 0)
                asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");

            // ---- scores: keys 16 k + g, + 8; heads 8 n + 2 tq, + 1
            asm volatile("cp.async.wait_group %0;" ::"n"(S::kSlots - 2) : "memory");
            __syncwarp();  // the keys are in, and the half before them is read by every lane
            if (kOdd) copy_keys();
            else copy_values();
            const uint32_t kt = ring + slot * S::kHalf;
            slot = next_slot(slot);
            auto query = [&](int c, int n) {
                return S::kQShared ? q_here[(c * kN + n) * 32] : make_uint2(qf[c][n][0], qf[c][n][1]);
            };
            float s[kBlocks][kN][4];
#pragma unroll
            for (int k = 0; k < kBlocks; ++k)
#pragma unroll
                for (int n = 0; n < kN; ++n) s[k][n][0] = s[k][n][1] = s[k][n][2] = s[k][n][3] = 0.f;
#pragma unroll
            for (int c = 0; c < kOT; c += kFp8 ? 2 : 1) {
#pragma unroll
                for (int k = 0; k < kBlocks; ++k) {
                    uint32_t r[4];
                    // rows 0-7 and 8-15 of a piece of 16 bytes, then of the next
                    ldsm4(r, kt + piece<S::kRowBytes>(16 * k + (lane & 15),
                                                      (kFp8 ? c : 2 * c) + (lane >> 4)));
                    if constexpr (kFp8) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t f[4] = {e4m3x2_to_f16x2(r[2 * i]), e4m3x2_to_f16x2(r[2 * i + 1]),
                                                   e4m3x2_to_f16x2(r[2 * i] >> 16),
                                                   e4m3x2_to_f16x2(r[2 * i + 1] >> 16)};
#pragma unroll
                            for (int n = 0; n < kN; ++n) {
                                const uint2 q = query(c + i, n);
                                mma<kF16>(s[k][n], f, q.x, q.y);
                            }
                        }
                    } else {
#pragma unroll
                        for (int n = 0; n < kN; ++n) {
                            const uint2 q = query(c, n);
                            mma<kF16>(s[k][n], r, q.x, q.y);
                        }
                    }
                }
            }
            const uint64_t valid = s_valid[warp][tile & 3];
            ++tile;
            constexpr uint64_t kAll = kKeys == 64 ? ~uint64_t{0} : (uint64_t{1} << (kKeys & 63)) - 1;
            if (valid != kAll) {
#pragma unroll
                for (int k = 0; k < kBlocks; ++k)
#pragma unroll
                    for (int n = 0; n < kN; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (!(valid >> (16 * k + g + 8 * (i >> 1)) & 1)) s[k][n][i] = -INFINITY;
            }
            // A weight is 2^(s sc - m + kUp).  m need not be the largest score so far, only
            // near it: it is moved when a score passes it by kSlack, which after the first
            // tiles is rare, and only then is the tile's maximum wanted (12 shuffles at 16
            // heads) and are the sums rescaled.
            bool high = false;
            float mt[kN][2];
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mt[n][i] = -INFINITY;
#pragma unroll
                    for (int k = 0; k < kBlocks; ++k)
                        mt[n][i] = fmaxf(mt[n][i], fmaxf(s[k][n][i], s[k][n][i + 2]));
                    high |= mt[n][i] * sc[n][i] > m[n][i] + kSlack;
                }
            if (__any_sync(0xffffffffu, high)) {
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float x = mt[n][i];
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        const float mn = fmaxf(m[n][i], x * sc[n][i]);
                        const float shrink = mn == m[n][i] ? 1.f : ex2(m[n][i] - mn);
                        m[n][i] = mn;
                        minus[n][i] = mn == -INFINITY ? 0.f : kUp - mn;
                        l[n][i] *= shrink;
#pragma unroll
                        for (int d = 0; d < kOT; ++d) {
                            acc[d][n][i] *= shrink;
                            acc[d][n][i + 2] *= shrink;
                        }
                    }
            }
            // ---- weights, in two or three words, as the right operand
            uint32_t p[kBlocks][kN][2], p2[kBlocks][kN][2], p3[kBlocks][kN][2];
#pragma unroll
            for (int k = 0; k < kBlocks; ++k)
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float x = ex2(fmaf(s[k][n][2 * j], sc[n][0], minus[n][0]));
                        const float y = ex2(fmaf(s[k][n][2 * j + 1], sc[n][1], minus[n][1]));
                        l[n][0] += x;
                        l[n][1] += y;
                        const uint32_t w = pack2<kF16>(x, y);
                        const float2 first = unpack2<kF16>(w);
                        p[k][n][j] = transpose8(w);
                        const uint32_t w2 = pack2<kF16>((x - first.x) * kLow, (y - first.y) * kLow);
                        p2[k][n][j] = transpose8(w2);
                        if constexpr (kThird) {
                            const float2 second = unpack2<kF16>(w2);
                            p3[k][n][j] = transpose8(pack2<kF16>(x - first.x - second.x,
                                                                 y - first.y - second.y));
                        }
                    }

            // ---- outputs: channels g, g + 8 of 16 d (8-bit: 2 g, 2 g + 1)
            asm volatile("cp.async.wait_group %0;" ::"n"(S::kSlots - 2) : "memory");
            __syncwarp();  // the values are in, and the keys are read by every lane
            if (kOdd) copy_values();
            else copy_keys();
            const uint32_t vt = ring + slot * S::kHalf;
            slot = next_slot(slot);
            constexpr int kStep = kFp8 ? 2 : 1;   // blocks of 16 channels to a load
            // channels 16 d .. of the 16 keys k: to[i], block d + i, += their products with the
            // weights' first words, and second[i] (may be to[i]) with the others
            auto products = [&](int k, int d, float(*to)[kN][4], float(*second)[kN][4]) {
                uint32_t r[4];
                auto product = [&](int i, const uint32_t (&f)[4]) {
#pragma unroll
                    for (int n = 0; n < kN; ++n) {
                        mma<kF16>(to[i][n], f, p[k][n][0], p[k][n][1]);
                        mma<kF16>(second[i][n], f, p2[k][n][0], p2[k][n][1]);
                        if constexpr (kThird) mma<kF16>(second[i][n], f, p3[k][n][0], p3[k][n][1]);
                    }
                };
                if constexpr (kFp8) {
                    ldsm4_trans(r, vt + piece<S::kRowBytes>(16 * k + (lane & 15), d + (lane >> 4)));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        // bytes: channels 2 g, 2 g + 1 of key 2 tq, then of key 2 tq + 1
                        const uint32_t x = __byte_perm(r[2 * i], 0, 0x3120);
                        const uint32_t y = __byte_perm(r[2 * i + 1], 0, 0x3120);
                        const uint32_t f[4] = {e4m3x2_to_f16x2(x), e4m3x2_to_f16x2(x >> 16),
                                               e4m3x2_to_f16x2(y), e4m3x2_to_f16x2(y >> 16)};
                        product(i, f);
                    }
                } else {
                    // pieces 2 d and 2 d + 1 of keys 0-7, then of keys 8-15
                    ldsm4_trans(r, vt + piece<S::kRowBytes>(16 * k + (lane & 7) + ((lane >> 4) << 3),
                                                            2 * d + ((lane >> 3) & 1)));
                    product(0, r);
                }
            };
            if constexpr (S::kApart) {
#pragma unroll
                for (int d = 0; d < kOT; d += kStep) {
                    // this tile's products in a sum of their own; scaled words' in another
                    float own[kStep][kN][4], low[kStep][kN][4];
#pragma unroll
                    for (int i = 0; i < kStep; ++i)
#pragma unroll
                        for (int n = 0; n < kN; ++n)
#pragma unroll
                            for (int j = 0; j < 4; ++j) own[i][n][j] = low[i][n][j] = 0.f;
#pragma unroll
                    for (int k = 0; k < kBlocks; ++k) products(k, d, own, kLow != 1.f ? low : own);
#pragma unroll
                    for (int i = 0; i < kStep; ++i)
#pragma unroll
                        for (int n = 0; n < kN; ++n)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                float &sum = acc[d + i][n][j];
                                sum += own[i][n][j];
                                if constexpr (kLow != 1.f) sum = fmaf(low[i][n][j], 1.f / kLow, sum);
                            }
                }
            } else {
#pragma unroll
                for (int k = 0; k < kBlocks; ++k)
#pragma unroll
                    for (int d = 0; d < kOT; d += kStep) products(k, d, acc + d, acc + d);
            }

            // ---- the end of a unit, or of the warp's part
            --remaining;
            const bool ends = cur.t == cur.tiles - 1;
            if (ends || remaining == 0) {
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], 4);
                        l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], 8);
                        l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], 16);
                        m[n][i] -= kUp;  // the sums carry 2^kUp
                    }
                if constexpr (!kFp8) {  // (8 bits hold no infinity)
                    bool nan = false;
#pragma unroll
                    for (int n = 0; n < kN; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float t[2] = {l[n][i], l[n][i]};
#pragma unroll
                            for (int d = 0; d < kOT; ++d) t[d & 1] = max3_nan(t[d & 1], acc[d][n][i], acc[d][n][i + 2]);
                            nan |= isnan(t[0] + t[1]) && !isnan(l[n][i]);
                        }
                    if (__any_sync(0xffffffffu, nan)) {
                        float sums[kOT * kN * 4], of_heads[2][kN * 2];
#pragma unroll
                        for (int e = 0; e < kOT * kN * 4; ++e) sums[e] = acc[e / (kN * 4)][e / 4 % kN][e % 4];
#pragma unroll
                        for (int e = 0; e < kN * 2; ++e) {
                            of_heads[0][e] = sc[e / 2][e % 2];
                            of_heads[1][e] = minus[e / 2][e % 2];
                        }
                        nonfinite_sums<S>(a, cur.b, rows.h, rows.rows, rows.out_row, begun * kKeys,
                                          min(int64_t{cur.len}, (cur.t + int64_t{1}) * kKeys), sums,
                                          of_heads[0], of_heads[1]);
#pragma unroll
                        for (int e = 0; e < kOT * kN * 4; ++e) acc[e / (kN * 4)][e / 4 % kN][e % 4] = sums[e];
                    }
                }
                const bool whole = ends && begun == 0;
                float *part = nullptr;
                int pitch = kD;
                if (!whole) {
                    const int at = 2 * place + (remaining == 0 ? 1 : 0);
                    if (remaining == 0) {
                        asm volatile("cp.async.wait_all;" ::: "memory");
                        __syncwarp();  // the ring is free: the part goes there
                        part = reinterpret_cast<float *>(s_ring + place * S::kRing);
                        pitch = S::kPitch;
                    } else {
                        part = a.ws.head + (static_cast<int64_t>(blockIdx.x) * kWarps + place) * kHeads * kD;
                    }
                    if (g == 0) {
#pragma unroll
                        for (int n = 0; n < kN; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                s_m[at][8 * n + 2 * tq + i] = m[n][i];
                                s_l[at][8 * n + 2 * tq + i] = l[n][i];
                            }
                    }
                    if (lane == 0) {
                        s_part[at].b = cur.b;
                        s_part[at].u = unit;
                        s_part[at].starts = begun == 0;
                        s_part[at].ends = ends;
                        s_part[at].in_global = remaining != 0;
                    }
                }
                const float vs = a.cache.v_scale == nullptr ? 1.f : a.cache.v_scale[rows.h];
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int row = 8 * n + 2 * tq + i;
                        if (row >= rows.rows) continue;
                        const float f = whole ? (l[n][i] == 0.f ? 0.f : vs / l[n][i]) : vs;
                        if (whole && g == 0) write_lse(a, rows.out_row + row, m[n][i], l[n][i]);
#pragma unroll
                        for (int d = 0; d < kOT; ++d) {
                            const float x = acc[d][n][i] * f, y = acc[d][n][i + 2] * f;
                            const int dx = 16 * d + (kFp8 ? 2 * g : g), dy = kFp8 ? dx + 1 : dx + 8;
                            if (!whole) {
                                part[row * pitch + dx] = x;
                                part[row * pitch + dy] = y;
                            } else if constexpr (!kWide) {
                                __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) + (rows.out_row + row) * kD;
                                o[dx] = __float2bfloat16_rn(x);
                                o[dy] = __float2bfloat16_rn(y);
                            } else {
                                float *o = static_cast<float *>(a.o) + (rows.out_row + row) * kD;
                                o[dx] = x;
                                o[dy] = y;
                            }
                        }
                    }
                fresh = true;
                if (remaining == 0) break;
            }
            cur.next(a, units);
        }
    }
    __syncthreads();

    // ---- joining the CTA's parts: the parts there are, and the runs of one unit among
    // them, in the list's order
    if (warp == 0) {
        Part part;
        part.b = -1;
        if (lane < kParts) part = s_part[lane];
        const uint32_t valid = __ballot_sync(0xffffffffu, part.b >= 0);
        const uint32_t below = valid & ((1u << lane) - 1);
        const int src = below == 0 ? 0 : 31 - __clz(below);
        const int prev_b = __shfl_sync(0xffffffffu, part.b, src);
        const int prev_u = __shfl_sync(0xffffffffu, part.u, src);
        const bool first = part.b >= 0 && (below == 0 || prev_b != part.b || prev_u != part.u);
        const uint32_t firsts = __ballot_sync(0xffffffffu, first);
        const uint32_t later = lane == 31 ? 0 : firsts >> (lane + 1) << (lane + 1);
        const uint32_t run = later == 0 ? valid : valid & ((later & -later) - 1);  // up to its end
        const int ends = __shfl_sync(0xffffffffu, part.ends, run == 0 ? 0 : 31 - __clz(run));
        const int at = __popc(below), r = __popc(firsts & (0xffffffffu >> (31 - lane))) - 1;
        if (part.b >= 0) {
            PartAt &x = s_at[at];
            x.part = lane;
            x.run = r;
            x.pitch = part.in_global ? kD : S::kPitch;
            x.sums = part.in_global
                         ? a.ws.head + (static_cast<int64_t>(blockIdx.x) * kWarps + (lane >> 1)) * kHeads * kD
                         : reinterpret_cast<const float *>(s_ring + (lane >> 1) * S::kRing);
        }
        if (first) {
            const UnitRows rows(a, part.b, part.u, kHeads);
            Run &x = s_run[r];
            x.begin = at;
            x.end = __popc(run);
            x.rows = rows.rows;
            x.whole = part.starts && ends;
            x.out_row = rows.out_row;
            x.slot = ((static_cast<int64_t>(blockIdx.x) * 2 + (part.starts ? 1 : 0)) << side_log) +
                     (part.u & ((1 << side_log) - 1));
        }
        if (lane == 0) {
            s_runs = __popc(firsts);
            s_parts = __popc(valid);
        }
    }
    __syncthreads();
    // the parts' weights, for each head; a whole unit's hold 1 / l too
    for (int i = tid; i < s_parts * kHeads; i += kThreads) {
        const int e = i / kHeads, row = i % kHeads;
        const Run run = s_run[s_at[e].run];
        if (row >= run.rows) continue;
        float mm = -INFINITY, ll = 0.f;
#pragma unroll 4
        for (int j = run.begin; j < run.end; ++j) mm = fmaxf(mm, s_m[s_at[j].part][row]);
        const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll 4
        for (int j = run.begin; j < run.end; ++j)
            ll += ex2(s_m[s_at[j].part][row] - ref) * s_l[s_at[j].part][row];
        float w = ex2(s_m[s_at[e].part][row] - ref);
        if (run.whole) w = ll == 0.f ? 0.f : w / ll;
        s_w[e][row] = w;
        if (e != run.begin) continue;
        if (run.whole) write_lse(a, run.out_row + row, mm, ll);
        else *reinterpret_cast<float2 *>(a.ws.ml + (run.slot * kHeads + row) * 2) = make_float2(mm, ll);
    }
    __syncthreads();
    constexpr int kPer = kHeads * (kD / 4);
    for (int i = tid; i < s_runs * kPer; i += kThreads) {
        const Run run = s_run[i / kPer];
        const int row = i % kPer / (kD / 4), d = i % (kD / 4) * 4;
        if (row >= run.rows) continue;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int e = run.begin; e < run.end; ++e) {
            const float w = s_w[e][row];
            const float4 y = *reinterpret_cast<const float4 *>(s_at[e].sums + row * s_at[e].pitch + d);
            x.x += w * y.x;
            x.y += w * y.y;
            x.z += w * y.z;
            x.w += w * y.w;
        }
        if (run.whole) write_out<S::kWide>(a, (run.out_row + row) * kD + d, x);
        else *reinterpret_cast<float4 *>(a.ws.cut + (run.slot * kHeads + row) * kD + d) = x;
    }

    // ---- sequences without keys ----------------------------------------------------------
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (valid_len(a, b) > 0) continue;
        if (tid == 0 && a.seq_lens[b] != 0) record_device_error(a.err, kDevInvalidArg);
        for (int i = tid; i < a.q_heads * (kD / 4); i += kThreads)
            write_out<S::kWide>(a, static_cast<int64_t>(b) * a.q_heads * kD + i * 4, make_float4(0.f, 0.f, 0.f, 0.f));
        if (a.lse != nullptr)
            for (int i = tid; i < a.q_heads; i += kThreads)
                a.lse[static_cast<int64_t>(b) * a.q_heads + i] = -INFINITY;
    }
}

// Joins the parts of the unit that CTA blockIdx.x of the first kernel began and
// did not finish: its slot 1 and slot 0 of the CTAs after it, up to the last.
// blockIdx.y: 64 channels; .z: of the heads side by side.  Which parts those are follows from the lengths, so it
// is known before the wait; after it there is one trip to memory, for the parts'
// maxima and sums together with the first of their products.
constexpr int kJoinThreads = 256;

template <class S>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Args a) {
    constexpr int kD = S::kD, kHeads = S::kHeads;
    constexpr int kQuads = 16;                                       // float4s of 64 channels
    constexpr int kItems = kHeads * kQuads;
    constexpr int kGroups = max_of(1, kJoinThreads / kItems);        // share the parts
    constexpr int kTurns = (kItems + kJoinThreads - 1) / kJoinThreads;  // items of a thread; the
    // last turn may do items again
    constexpr int kAhead = 8 / kTurns;                               // parts read ahead, each
    constexpr int kRowsOfWarp = kHeads / (kJoinThreads / 32);
    __shared__ float s_w[kMaxCtas][kHeads];
    __shared__ float4 s_sum[kGroups][kItems];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c0 = blockIdx.x;
    // (this kernel is set up once the first one's blocks have all waited for what was before
    // them, so the lengths, which the first one does not write, may be read here)
    const List<S> list(a, lane, gridDim.x);
    const int64_t hi = list.even_begin(c0 + int64_t{1});
    bool mine = !list.whole && c0 < static_cast<int>(list.ctas) && hi < list.total;
    Cursor<S::kKeys> cut = {};
    if (blockIdx.z >> list.side_log() != 0) mine = false;
    if (mine) cut = list.find(a, hi);
    if (cut.t == 0 || hi - cut.t < list.even_begin(c0)) mine = false;  // not cut, or begun before
    if (!mine) {
        // the kernels after this one count on the first having ended when this one has
        wait_for_kernel_before();
        return;
    }
    const int parts = list.even_piece_of(hi - cut.t + cut.tiles - 1) - c0 + 1;
    const UnitRows rows(a, cut.b, (cut.u << list.side_log()) + blockIdx.z, kHeads);
    // part i's sums: slot 1 of CTA c0, slot 0 of CTA c0 + i
    auto slot = [&](int i) {
        return ((static_cast<int64_t>(c0 + i) * 2 + (i == 0 ? 1 : 0)) << list.side_log()) + blockIdx.z;
    };
    auto ml_at = [&](int i, int row) {
        return *reinterpret_cast<const float2 *>(a.ws.ml + (slot(i) * kHeads + row) * 2);
    };
    const int group = tid / kItems;                                  // 0 where a thread has turns
    auto sums_at = [&](int i, int turn) {
        const int item = (tid + turn * kJoinThreads) % kItems;
        return *reinterpret_cast<const float4 *>(
            a.ws.cut + (slot(i) * kHeads + item / kQuads) * kD + blockIdx.y * 64 + item % kQuads * 4);
    };

    wait_for_kernel_before();
    float2 ml[kRowsOfWarp];
#pragma unroll
    for (int k = 0; k < kRowsOfWarp; ++k)
        if (lane < parts) ml[k] = ml_at(lane, warp + k * (kJoinThreads / 32));
    // (rows past the group's heads are read like the others and not written)
    float4 y[kTurns][kAhead];
#pragma unroll
    for (int k = 0; k < kTurns; ++k)
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (group + j * kGroups < parts) y[k][j] = sums_at(group + j * kGroups, k);
#pragma unroll
    for (int k = 0; k < kRowsOfWarp; ++k) {
        const int row = warp + k * (kJoinThreads / 32);
        if (row >= rows.rows) break;
        float mm = lane < parts ? ml[k].x : -INFINITY, ll = 0.f;
        for (int i = lane + 32; i < parts; i += 32) mm = fmaxf(mm, ml_at(i, row).x);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
        const float ref = mm == -INFINITY ? 0.f : mm;
        for (int i = lane; i < parts; i += 32) {
            const float2 x = i == lane ? ml[k] : ml_at(i, row);
            const float w = ex2(x.x - ref);
            s_w[i][row] = w;
            ll += w * x.y;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, d);
        const float f = ll == 0.f ? 0.f : 1.f / ll;
        for (int i = lane; i < parts; i += 32) s_w[i][row] *= f;
        if (lane == 0 && blockIdx.y == 0) write_lse(a, rows.out_row + row, mm, ll);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        const int item = (tid + k * kJoinThreads) % kItems, row = item / kQuads;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](int i, float4 v) {
            const float w = s_w[i][row];
            x.x += w * v.x;
            x.y += w * v.y;
            x.z += w * v.z;
            x.w += w * v.w;
        };
        if (row < rows.rows) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (group + j * kGroups < parts) add(group + j * kGroups, y[k][j]);
#pragma unroll 8
            for (int i = group + kAhead * kGroups; i < parts; i += kGroups) add(i, sums_at(i, k));
        }
        if constexpr (kGroups > 1) {
            s_sum[group][item] = x;
            __syncthreads();
            if (group > 0) return;
#pragma unroll
            for (int i = 1; i < kGroups; ++i) {
                const float4 v = s_sum[i][item];
                x.x += v.x;
                x.y += v.y;
                x.z += v.z;
                x.w += v.w;
            }
        }
        if (row < rows.rows)
            write_out<S::kWide>(a, (rows.out_row + row) * kD + blockIdx.y * 64 + item % kQuads * 4, x);
    }
}

template <class S>
cudaError_t launch_shape(Args a, int ctas, cudaStream_t s) {
    const int page_size = static_cast<int>(a.cache.page.d);
    auto kern = page_size % S::kKeys == 0 ? paged_decode_kernel<S, true> : paged_decode_kernel<S, false>;
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kern), S::kSmem);
    if (e != cudaSuccess) return e;
    // heads side by side: a token's, next to each other, where a row is less than 256 bytes
    // (64 channels, 8 bits: 134 us without, 80 with; bf16: 159 and 145; 128 channels, bf16:
    // 145 and 146)
    a.side_log = 0;
    if (S::kSide && a.head_tiles == 1 && a.cache.head_stride == S::kRowBytes)
        while (2 << a.side_log <= kMaxSide && a.cache.heads % (2 << a.side_log) == 0) ++a.side_log;
    // a table without room for longer units: the kernel cuts none (see List)
    const bool whole = static_cast<int64_t>(a.max_pages) * page_size <= 2 * (S::kWarps >> a.side_log) * S::kKeys;
    const cudaError_t e1 = launch_early(kern, dim3(ctas), S::kWarps * 32, S::kSmem, s, a);
    if (e1 != cudaSuccess || whole) return e1;
    return launch_early(join_kernel<S>, dim3(ctas, S::kD / 64, 1 << a.side_log), kJoinThreads, 0, s, a);
}

template <int kD, bool kFp8, bool kWide>
cudaError_t launch_heads(const Args &a, int heads, int ctas, cudaStream_t s) {
    if (heads == 8) return launch_shape<Shape<kD, kFp8, 1, kWide>>(a, ctas, s);
    if constexpr (kD <= 128) {
        if (heads == 24) return launch_shape<Shape<kD, kFp8, 3, kWide>>(a, ctas, s);
        if (heads == 32) return launch_shape<Shape<kD, kFp8, 4, kWide>>(a, ctas, s);
    }
    return launch_shape<Shape<kD, kFp8, 2, kWide>>(a, ctas, s);
}

}  // namespace

// Instantiated for each head_dim in a file of its own: they compile side by side.
template <int kD>
cudaError_t launch_paged_decode_dim(const Args &a, bool o_bf16, int heads, int ctas, cudaStream_t s) {
    if (a.cache.fp8)
        return o_bf16 ? launch_heads<kD, true, false>(a, heads, ctas, s)
                      : launch_heads<kD, true, true>(a, heads, ctas, s);
    return o_bf16 ? launch_heads<kD, false, false>(a, heads, ctas, s)
                  : launch_heads<kD, false, true>(a, heads, ctas, s);
}

}  // namespace paged
}  // namespace kda
