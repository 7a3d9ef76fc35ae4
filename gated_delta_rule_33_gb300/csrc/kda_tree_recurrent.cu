// kda_tree_recurrent.cu -- the KDA recurrence over a tree of drafted tokens: outputs for every
// node from the state that its request holds (which stays as it is), and the state after the
// path that is accepted.
//
// With a_i = exp(g_i), path(i) the ancestors of node i and i itself, E_ij the product of a_l
// over the nodes l of path(i) behind j, and E_i that over all of path(i), the state that node
// i's update meets, applied to a vector x, is
//
//   S'^T x = S_0^T (E_i x) + sum_{j above i} ((E_ij k_j) . x) u_j
//   u_i = beta_i (v_i - S'^T k_i),   o_i = S'^T (scale q_i) + (k_i . scale q_i) u_i
//
// and after the path of node e the state is Diag(E_e) S_0 + sum_{j in path(e)} (E_ej k_j) u_j^T.
// E_ij is formed by products along the path, from node i upwards: no decay is divided out, so
// none is too strong.
//
// Decode.  Bound: the state is read once (64 KB of fp32 a head, 32 KB of bf16) and meets 2 n
// vectors, 4 n 128^2 flops: HBM.  On the fp32 pipe that product alone takes as long (337 us where
// the bytes take 82); so it runs on the matrix instructions, every operand as three bf16 words, 24
// bits together, and the six products that reach 2^-24 (u becomes state; two tf32 words and
// three products hold less and took twice as long).  A block walks over units, each a
// (request, head); up to 16 nodes three blocks share an SM, so that some compute while others wait.
// The state comes by 16-byte copies (bulk copies of a row each took 5 us to issue), to rows 8 words
// apart in the banks.  An fp32 state of a call with up to 32 nodes comes in quarters of which two are there
// at a time: one meets the vectors while the next arrives, and the next unit's first two come while
// this one's updates run.  A bf16 state, and that of a call with more nodes, comes whole, while the updates
// of the unit before run.  A warp a node
// walks its path for E_i k_i, E_i q_i and the products (E_ij k_j) . k_i and . q_i.  Then a warp has
// 16 columns of the product for all rows; then each thread solves its column of the updates, 8
// nodes in registers, and the outputs follow.
//
// Measured, 64 requests of 7 to 16 nodes, 96 heads, fp32 state: 192 us (82 at a copy's rate).  337
// with the product on the fp32 pipe, 280 as two tf32 words, 226 with 16-byte copies, 213 with
// paths in packed pairs (219 as three bf16 words, which hold more), 211 walking over units, 207 with
// a unit's place loaded ahead, 197 with the state in halves and a third block, 188 in quarters.
// (512 threads a block: 244.)  Over a bf16 state 145 us (52).  64 requests of 24 nodes 427 us (105), of 64
// nodes 1548 us (180), over a bf16 state 343 and 1385.  What bounds it: some 2300 instructions a warp and unit, which fill
// half of the issue slots; a unit's phases (decays, paths, product, updates, outputs) are chains
// with barriers between them, and three blocks do not fill all of their gaps.
//
// What is not finite.  In the tables of products a node that is not above another has a 0, and 0 times
// an update that is not finite is NaN; an infinite operand has no second word either (inf - inf).  So
// a block that met an output that is not finite goes over its units again in the end and solves what
// is not finite in them in fp32 arithmetic, the nodes chosen by their words (solve_again).  To look for
// it costs 1 to 2 % (192 us where there were 189).
#include <cfloat>
#include <type_traits>

#include "kda_f32x2.cuh"
#include "kda_sm100.cuh"
#include "kda_tree.cuh"

namespace kda {
namespace {

constexpr int kD = 128;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <bool kBf16>
__device__ __forceinline__ void write_out(void *o, int64_t i, float x) {
    if constexpr (kBf16) static_cast<__nv_bfloat16 *>(o)[i] = __float2bfloat16_rn(x);
    else static_cast<float *>(o)[i] = x;
}

// The state of request b, or -1 (inactive, or a bad slot: an error).
__device__ __forceinline__ int64_t slot_of(const TreeStep &a, int b) {
    if (a.slots == nullptr) return b;
    const int s = a.slots[b];
    if (s >= a.num_slots && threadIdx.x == 0) record_device_error(a.err, kDevInvalidArg);
    return s < 0 || s >= a.num_slots ? -1 : s;
}

__device__ __forceinline__ float4 widen4(uint2 x) {
    return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
                       __uint_as_float(x.y & 0xffff0000u));
}

// ---- decode --------------------------------------------------------------------------------

constexpr int kPitch = 132;  // floats of a state's or product's row: eight banks between every second

// Left operands of 16 rows x 16 k's, for eight nodes: rows g are E_i k_i, rows 8 + g their E_i q_i.
// Up to 16 nodes they lie as bf16 words, a block of 32 lanes' registers and a gap for the banks;
// more of them as fp32, which each warp splits.
template <int kEights>
struct LeftOperands {
    static constexpr bool kWords = kEights <= 2;
    static constexpr int kBlock = kWords ? 3 * 512 + 32 : 32 * 32 + 32;  // bytes at 16 k's
    static constexpr int kEight = kD / 16 * kBlock;                      // and at all
    static_assert(kEight >= 16 * kPitch * 4, "the products take their place");
};

// Shared memory: nodes in eights, as many as nc nodes fill.
template <int kEights, bool kStateBf16>
struct TreeSmem {
    // The state comes in parts of kPartRows rows, two at a time, where that lets another block
    // share the SM.  (A bf16 row's pitch: 8 banks between every second, as of an fp32 one.)
    static constexpr int kParts = kEights <= 4 && !kStateBf16 ? 4 : 1, kSlots = kParts < 2 ? 1 : 2;
    static constexpr int kPartRows = kD / kParts, kStatePitch = kStateBf16 ? kD * 2 + 16 : kPitch * 4;
    static constexpr int kPart = kPartRows * kStatePitch, kState = kSlots * kPart;
    int nc;
    uint8_t *state;   // [kSlots][kPartRows][kStatePitch]
    uint8_t *rows;    // [eight][k / 16]: LeftOperands; then the products [eight][16][kPitch] of the
                      // eight's E_i k_i with the state, and of its E_i scale q_i
    float *ak, *aq;   // [j][i]: (E_ij k_j) . k_i (0 where j is not above i), (E_ij k_j) . scale q_i
    float *decay;     // [n][128] a_i; then u_i
    float *beta;
    __nv_bfloat16 *k; // [n][128]; then v_i

    __host__ __device__ static int nodes(int max_nodes) { return (max_nodes + 7) / 8 * 8; }
    __host__ __device__ static int bytes(int nc) {
        return kState + nc / 8 * LeftOperands<kEights>::kEight + 2 * nc * nc * 4 + nc * kD * (4 + 2) + nc * 4;
    }
    __device__ TreeSmem(uint8_t *base, int max_nodes) {
        nc = nodes(max_nodes);
        state = base;
        rows = base + kState;
        ak = reinterpret_cast<float *>(rows + nc / 8 * LeftOperands<kEights>::kEight);
        aq = ak + nc * nc;
        decay = aq + nc * nc;
        k = reinterpret_cast<__nv_bfloat16 *>(decay + nc * kD);
        beta = reinterpret_cast<float *>(k + nc * kD);
    }
};

// c (16 x 8) += a (16 x 16) b (16 x 8), bf16 operands.
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// Two values as sums of three bf16 words each.
__device__ __forceinline__ void split3(float a, float b, uint32_t &h, uint32_t &m, uint32_t &l) {
    auto pack = [](float x, float y) {
        const __nv_bfloat162 w = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&w);
    };
    h = pack(a, b);
    a -= __uint_as_float(h << 16);
    b -= __uint_as_float(h & 0xffff0000u);
    m = pack(a, b);
    a -= __uint_as_float(m << 16);
    b -= __uint_as_float(m & 0xffff0000u);
    l = pack(a, b);
}

struct Pairs {  // four channels
    uint64_t x, y;
};
__device__ __forceinline__ Pairs pairs(uint2 v) {
    const float4 f = widen4(v);
    return {f2(f.x, f.y), f2(f.z, f.w)};
}

__device__ __forceinline__ int count_leading(uint32_t x) { return __clz(static_cast<int>(x)); }
__device__ __forceinline__ int count_leading(uint64_t x) { return __clzll(static_cast<long long>(x)); }

// Eight values of each lane summed over the warp: lane l returns the sum of value (l >> 2) & 7.
__device__ __forceinline__ float sum_eight(float (&x)[8]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int step = 4, bit = 16; step >= 1; step >>= 1, bit >>= 1) {
        const bool up = lane & bit;
#pragma unroll
        for (int i = 0; i < step; ++i) {
            const float send = up ? x[i] : x[i + step], keep = up ? x[i + step] : x[i];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
        }
    }
    x[0] += __shfl_xor_sync(0xffffffffu, x[0], 2);
    x[0] += __shfl_xor_sync(0xffffffffu, x[0], 1);
    return x[0];
}

// What says where a (request, head) lies: loaded early, looked at when it is needed.
struct TreePlace {
    int h, lo, hi, slot;

    __device__ __forceinline__ TreePlace(const TreeStep &a, uint32_t unit) {
        const uint32_t b = unit / static_cast<uint32_t>(a.H);
        h = static_cast<int>(unit - b * static_cast<uint32_t>(a.H));
        lo = a.cu[b];
        hi = a.cu[b + 1];
        slot = a.slots != nullptr ? a.slots[b] : static_cast<int>(b);
    }
};

// A (request, head) of a block.
struct TreeUnit {
    int64_t first;
    int slot, n, rows, h;

    __device__ __forceinline__ TreeUnit(const TreeStep &a, const TreePlace &p) {
        h = p.h;
        const TreeRows t = tree_rows_between(p.lo, p.hi, a.N, a.max_nodes);
        const bool outside = a.slots != nullptr && p.slot >= a.num_slots;
        if ((t.bad || outside) && threadIdx.x == 0) record_device_error(a.err, kDevInvalidArg);
        slot = outside ? -1 : p.slot;
        first = t.first;
        rows = t.rows;
        n = slot < 0 ? 0 : t.n;
    }
    __device__ __forceinline__ int64_t at(const TreeStep &a, int i) const { return ((first + i) * a.H + h) * kD; }
};

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= FLT_MAX; }

// What of a unit's updates and outputs is not finite, once more, in fp32 arithmetic and with the
// nodes chosen by their words.  What is finite stays as it is.  By the whole block, which has nothing
// else to do and nothing on its way to shared memory.  (Inlined: as a function it took the kernel
// registers that the loop needs, 193 us.)
template <bool kStateBf16, bool kOutBf16, int kEights>
__device__ __forceinline__ void solve_again(const TreeStep &a, uint32_t which, uint8_t *smem) {
    const TreeUnit unit(a, TreePlace(a, which));
    if (unit.n == 0) return;
    const TreeSmem<kEights, kStateBf16> s(smem, a.max_nodes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = unit.n, nc = s.nc;
    float *rows = reinterpret_cast<float *>(s.rows), *u = s.decay;  // [n][2][kD]: E_i k_i, E_i scale q_i
    auto output = [&](int64_t at) {
        if constexpr (kOutBf16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(a.o)[at]);
        else return static_cast<const float *>(a.o)[at];
    };
    bool all = true;
    for (int i = tid; i < n * kD; i += kThreads) {
        const int64_t at = unit.at(a, i / kD) + i % kD;
        all &= finite(output(at)) && (a.u == nullptr || finite(a.u[at]));
        s.decay[i] = expf(a.g[at]);
        s.k[i] = a.k[at];
    }
    if (!__syncthreads_or(!all)) return;
    for (int i = warp; i < n; i += kWarps) {  // a warp a node, up its path
        const int64_t at = unit.at(a, i) + lane * 4;
        const float4 k = widen4(*reinterpret_cast<const uint2 *>(s.k + i * kD + lane * 4));
        float4 q = widen4(*reinterpret_cast<const uint2 *>(a.q + at)), e = make_float4(1.f, 1.f, 1.f, 1.f);
        q = make_float4(q.x * a.scale, q.y * a.scale, q.z * a.scale, q.w * a.scale);
        for (uint64_t path = path_of(a.ancestors[unit.first + i], i); path != 0;) {
            const int j = top_bit(path);
            path ^= uint64_t{1} << j;
            const float4 kj = widen4(*reinterpret_cast<const uint2 *>(s.k + j * kD + lane * 4));
            const float4 d = *reinterpret_cast<const float4 *>(s.decay + j * kD + lane * 4);
            const float4 y = make_float4(e.x * kj.x, e.y * kj.y, e.z * kj.z, e.w * kj.w);
            float dk = y.x * k.x + y.y * k.y + y.z * k.z + y.w * k.w;
            float dq = y.x * q.x + y.y * q.y + y.z * q.z + y.w * q.w;
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) {
                dk += __shfl_xor_sync(0xffffffffu, dk, m);
                dq += __shfl_xor_sync(0xffffffffu, dq, m);
            }
            if (lane == 0) {
                s.ak[j * nc + i] = dk;
                s.aq[j * nc + i] = dq;
            }
            e = make_float4(e.x * d.x, e.y * d.y, e.z * d.z, e.w * d.w);
        }
        float4 *row = reinterpret_cast<float4 *>(rows + i * 2 * kD) + lane;
        row[0] = make_float4(e.x * k.x, e.y * k.y, e.z * k.z, e.w * k.w);
        row[kD / 4] = make_float4(e.x * q.x, e.y * q.y, e.z * q.z, e.w * q.w);
    }
    __syncthreads();
    if (tid < kD) {  // a thread a column
        const int64_t state = (static_cast<int64_t>(unit.slot) * a.H + unit.h) * (kD * kD) + tid;
        for (int i = 0; i < n; ++i) {
            const int64_t at = unit.at(a, i) + tid;
            const float *row = rows + i * 2 * kD;
            float w = 0.f, z = 0.f;
#pragma unroll 8
            for (int k = 0; k < kD; ++k) {
                float x;
                if constexpr (kStateBf16) x = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.pool)[state + k * kD]);
                else x = static_cast<const float *>(a.pool)[state + k * kD];
                w += row[k] * x;
                z += row[kD + k] * x;
            }
            for (uint64_t p = a.ancestors[unit.first + i] & bits_below(i); p != 0; p &= p - 1) {
                const int j = __ffsll(static_cast<long long>(p)) - 1;
                w += s.ak[j * nc + i] * u[j * kD + tid];
                z += s.aq[j * nc + i] * u[j * kD + tid];
            }
            float x = a.beta[(unit.first + i) * a.H + unit.h] * (__bfloat162float(a.v[at]) - w);
            if (a.u != nullptr) {
                if (finite(a.u[at])) x = a.u[at];
                else a.u[at] = x;
            }
            u[i * kD + tid] = x;
            if (!finite(output(at))) write_out<kOutBf16>(a.o, at, z + s.aq[i * nc + i] * x);
        }
    }
    __syncthreads();
}

// By registers (the accumulators of a warp are 16 an eight) and shared memory.
constexpr int blocks_an_sm(int eights) { return eights <= 2 ? 3 : eights <= 4 ? 2 : 1; }

// kEights: eights of nodes that the accumulators hold.  A block walks over units, gridDim.x apart.
template <bool kStateBf16, bool kOutBf16, int kEights>
__global__ void __launch_bounds__(kThreads, blocks_an_sm(kEights)) tree_decode_kernel(const TreeStep a) {
    using Left = LeftOperands<kEights>;
    using Smem = TreeSmem<kEights, kStateBf16>;
    using Word = std::conditional_t<kEights <= 4, uint32_t, uint64_t>;
    constexpr int kBits = 8 * sizeof(Word);
    constexpr uint32_t kRow = kD * (kStateBf16 ? 2 : 4);
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_again;  // some unit of the block's has an output that is not finite
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Smem s(smem, a.max_nodes);
    const uint32_t units = static_cast<uint32_t>(a.B) * static_cast<uint32_t>(a.H);

    // What a unit brings from memory, ahead of its turn: the state and the keys to shared memory,
    // and in registers the gates (four channels of nodes warp, warp + 8, ..), the queries of the
    // same nodes, their words and (of the first threads) beta.
    float4 g4[kEights];
    uint2 q2[kEights];
    uint64_t words[kEights];
    float beta = 0.f;
    auto fetch_inputs = [&](const TreeUnit &u) {
        if (u.n == 0) return;
#pragma unroll
        for (int i = 0; i < kEights; ++i) {
            const int node = warp + kWarps * i;
            if (node < u.n) {
                g4[i] = *reinterpret_cast<const float4 *>(a.g + u.at(a, node) + lane * 4);
                q2[i] = *reinterpret_cast<const uint2 *>(a.q + u.at(a, node) + lane * 4);
                words[i] = a.ancestors[u.first + node];
            }
        }
        if (tid < u.n) beta = a.beta[(u.first + tid) * a.H + u.h];
    };
    auto fetch_part = [&](const TreeUnit &u, int part) {
        if (u.n == 0) return;
        const uint8_t *src = static_cast<const uint8_t *>(a.pool) +
                             (static_cast<int64_t>(u.slot) * a.H + u.h) * (kD * kRow) + part * (Smem::kPartRows * kRow);
        constexpr int kPieces = kRow / 16;
#pragma unroll
        for (int i = 0; i < Smem::kPartRows * kPieces / kThreads; ++i) {
            const int k = (tid + i * kThreads) / kPieces, c = (tid + i * kThreads) % kPieces;
            sm100::cp_async_16(s.state + part % Smem::kSlots * Smem::kPart + k * Smem::kStatePitch + c * 16, src + k * kRow + c * 16, true);
        }
    };
    auto fetch_first_parts = [&](const TreeUnit &u) {
        fetch_part(u, 0);
        if constexpr (Smem::kSlots == 2) fetch_part(u, 1);
    };
    auto fetch_rows = [&](const TreeUnit &u, const __nv_bfloat16 *x) {  // keys, or values in their place
        for (int i = tid; i < u.n * 16; i += kThreads)
            sm100::cp_async_16(s.k + i * 8, x + u.at(a, i >> 4) + (i & 15) * 8, true);
    };

    if (tid == 0) s_again = 0;  // (the first unit's barriers come before it is written again)
    TreeUnit u(a, TreePlace(a, blockIdx.x));
    fetch_inputs(u);
    fetch_first_parts(u);
    fetch_rows(u, a.k);
    for (uint32_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const bool more = unit + gridDim.x < units;
        const TreePlace place(a, more ? unit + gridDim.x : unit);
        const int n = u.n;
        if (n == 0) {
            for (int64_t i = tid; i < static_cast<int64_t>(u.rows) * kD; i += kThreads) {
                const int64_t at = ((u.first + i / kD) * a.H + u.h) * kD + i % kD;
                write_out<kOutBf16>(a.o, at, 0.f);
                if (a.u != nullptr) a.u[at] = 0.f;
            }
            u = TreeUnit(a, place);
            if (more) {
                fetch_inputs(u);
                fetch_first_parts(u);
                fetch_rows(u, a.k);
            }
            continue;
        }
        const int eights = (n + 7) / 8;
#pragma unroll
        for (int i = 0; i < kEights; ++i) {
            const int node = warp + kWarps * i;
            if (node < n)
                *reinterpret_cast<float4 *>(s.decay + node * kD + lane * 4) =
                    make_float4(expf(g4[i].x), expf(g4[i].y), expf(g4[i].z), expf(g4[i].w));
        }
        for (int i = tid; i < n * s.nc / 4; i += kThreads)
            reinterpret_cast<float4 *>(s.ak)[i] = reinterpret_cast<float4 *>(s.aq)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (tid < n) s.beta[tid] = beta;
        sm100::cp_async_wait_all();
        __syncthreads();

        // A warp a node: four channels a lane, four nodes of the path at a time.
#pragma unroll
        for (int eight = 0; eight < kEights; ++eight) {
            if (eight >= eights) break;
            const int i = warp + kWarps * eight;
            // this lane's k's, 4 lane ..: for lane lane0 and the next of the operand at lane / 4, their
            // first or second pair
            const int lane0 = (i & 7) * 4 + 2 * (lane & 1), pair = (lane >> 1) & 1;
            uint8_t *rows = s.rows + eight * Left::kEight + (lane >> 2) * Left::kBlock;
            auto write = [&](float2 k0, float2 k1, float2 q0, float2 q1) {
                if constexpr (Left::kWords) {
                    uint32_t k[2][3], q[2][3];
                    split3(k0.x, k0.y, k[0][0], k[0][1], k[0][2]);
                    split3(k1.x, k1.y, k[1][0], k[1][1], k[1][2]);
                    split3(q0.x, q0.y, q[0][0], q[0][1], q[0][2]);
                    split3(q1.x, q1.y, q[1][0], q[1][1], q[1][2]);
#pragma unroll
                    for (int w = 0; w < 3; ++w) {
                        uint2 *to = reinterpret_cast<uint2 *>(rows + w * 512) + lane0 * 2 + pair;
                        to[0] = make_uint2(k[0][w], q[0][w]);
                        to[2] = make_uint2(k[1][w], q[1][w]);
                    }
                } else {
                    float4 *to = reinterpret_cast<float4 *>(rows) + lane0 * 2 + pair;
                    to[0] = make_float4(k0.x, k0.y, q0.x, q0.y);
                    to[2] = make_float4(k1.x, k1.y, q1.x, q1.y);
                }
            };
            if (i >= n) {  // rows of the last eight that are no node
                const float2 zero = make_float2(0.f, 0.f);
                write(zero, zero, zero, zero);
                continue;
            }
            Word path = static_cast<Word>(path_of(words[eight], i));
            const Pairs k = pairs(*reinterpret_cast<const uint2 *>(s.k + i * kD + 4 * lane));
            Pairs q = pairs(q2[eight]);
            const uint64_t scale = f2(a.scale, a.scale), one = f2(1.f, 1.f);
            q = {f2_mul(q.x, scale), f2_mul(q.y, scale)};
            Pairs e = {one, one};
            while (path != 0) {
                float x[8];
                int js[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const bool some = path != 0;
                    const int j = some ? kBits - 1 - count_leading(path) : 0;
                    js[m] = some ? j : -1;
                    path &= (Word{1} << j) - 1;  // (nothing is left of none)
                    const Pairs kj = pairs(*reinterpret_cast<const uint2 *>(s.k + j * kD + 4 * lane));
                    const float4 d = *reinterpret_cast<const float4 *>(s.decay + j * kD + 4 * lane);
                    const Pairs y = {f2_mul(e.x, kj.x), f2_mul(e.y, kj.y)};
                    const float2 dk = f2_split(f2_fma(y.y, k.y, f2_mul(y.x, k.x)));
                    const float2 dq = f2_split(f2_fma(y.y, q.y, f2_mul(y.x, q.x)));
                    x[2 * m] = dk.x + dk.y;
                    x[2 * m + 1] = dq.x + dq.y;
                    if (some) e = {f2_mul(e.x, f2(d.x, d.y)), f2_mul(e.y, f2(d.z, d.w))};
                }
                const float sum = sum_eight(x);
                const int m = lane >> 3, j = m == 0 ? js[0] : m == 1 ? js[1] : m == 2 ? js[2] : js[3];
                if ((lane & 3) == 0 && j >= 0) {
                    if (lane & 4) s.aq[j * s.nc + i] = sum;
                    else if (j != i) s.ak[j * s.nc + i] = sum;
                }
            }
            write(f2_split(f2_mul(e.x, k.x)), f2_split(f2_mul(e.y, k.y)), f2_split(f2_mul(e.x, q.x)),
                  f2_split(f2_mul(e.y, q.y)));
        }
        __syncthreads();
        if constexpr (Smem::kParts == 1) fetch_rows(u, a.v);

        // The product: a warp has columns 16 warp .. + 15 of all rows.
        const int g = lane >> 2, tq = lane & 3;
        float acc[kEights][2][4], low[kEights][2][4];  // (the lower words' products apart: shorter chains)
#pragma unroll
        for (int m = 0; m < kEights; ++m)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[m][i >> 2][i & 3] = low[m][i >> 2][i & 3] = 0.f;
        auto product_of = [&](int ks, const uint8_t *state) {  // 16 k's; where the first k's row would lie
            uint32_t b[3][2][2];  // word, tile, pair of k's
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int k = 16 * ks + 2 * tq + 8 * i, col = 16 * warp + 8 * c + g;
                    if constexpr (kStateBf16) {
                        const uint16_t *x = reinterpret_cast<const uint16_t *>(state + k * Smem::kStatePitch) + col;
                        b[0][c][i] = x[0] | static_cast<uint32_t>(x[Smem::kStatePitch / 2]) << 16;
                    } else {
                        const float *x = reinterpret_cast<const float *>(state + k * Smem::kStatePitch) + col;
                        split3(x[0], x[kPitch], b[0][c][i], b[1][c][i], b[2][c][i]);
                    }
                }
            // two eights at a time, their products in turn
#pragma unroll
            for (int m0 = 0; m0 < kEights; m0 += 2) {
                if (m0 >= eights) break;
                uint32_t w[2][3][4];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const uint8_t *rows = s.rows + (m0 + m) * Left::kEight + ks * Left::kBlock;
                    if (m0 + m >= eights) break;
                    if constexpr (Left::kWords) {
#pragma unroll
                        for (int i = 0; i < 3; ++i) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(rows + i * 512 + lane * 16);
                            w[m][i][0] = x.x;
                            w[m][i][1] = x.y;
                            w[m][i][2] = x.z;
                            w[m][i][3] = x.w;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float4 x = reinterpret_cast<const float4 *>(rows)[lane * 2 + i];
                            split3(x.x, x.y, w[m][0][2 * i], w[m][1][2 * i], w[m][2][2 * i]);
                            split3(x.z, x.w, w[m][0][2 * i + 1], w[m][1][2 * i + 1], w[m][2][2 * i + 1]);
                        }
                    }
                }
                // words (i, k) of the two operands, i + k <= 2; a bf16 state is one word
#pragma unroll
                for (int i = 0; i < 3; ++i)
#pragma unroll
                    for (int k = 0; k < (kStateBf16 ? 1 : 3 - i); ++k)
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            if (m0 + m >= eights) break;
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                mma_bf16(i + k == 0 ? acc[m0 + m][c] : low[m0 + m][c], w[m][i], b[k][c]);
                        }
            }
        };
        for (int part = 0;; ++part) {
            const uint8_t *state = s.state + part % Smem::kSlots * Smem::kPart - part * Smem::kPart;
#pragma unroll 2
            for (int ks = part * Smem::kPartRows / 16; ks < (part + 1) * Smem::kPartRows / 16; ++ks)
                product_of(ks, state);
            if (part + 1 == Smem::kParts) break;
            sm100::cp_async_wait_all();
            __syncthreads();  // the next part is there, and this one's place is free
            if (part + 2 < Smem::kParts) fetch_part(u, part + 2);
            if (part == 0) fetch_rows(u, a.v);
        }
        sm100::cp_async_wait_all();
        __syncthreads();
        // nobody reads the state or the left operands any more: the next unit's state may come, and
        // the products go where the operands were
        const TreeUnit next(a, place);
        if (more) {
            fetch_inputs(next);
            fetch_first_parts(next);
        }
        float *products = reinterpret_cast<float *>(s.rows);
#pragma unroll
        for (int m = 0; m < kEights; ++m) {
            if (m >= eights) break;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float *to = products + (m * 16 + g) * kPitch + 16 * warp + 8 * c + 2 * tq;
                *reinterpret_cast<float2 *>(to) = make_float2(acc[m][c][0] + low[m][c][0], acc[m][c][1] + low[m][c][1]);
                *reinterpret_cast<float2 *>(to + 8 * kPitch) =
                    make_float2(acc[m][c][2] + low[m][c][2], acc[m][c][3] + low[m][c][3]);
            }
        }
        __syncthreads();
        auto product = [&](int m, int r, int c) { return products[(m * 16 + r) * kPitch + c]; };

        // The updates: a thread a column, eight nodes in registers.
        const int c = tid & (kD - 1);
        if (tid < kD) {
            for (int m = 0; m < eights; ++m) {
                float w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = product(m, i, c);
#pragma unroll 4
                for (int j = 0; j < 8 * m; ++j) {
                    const float x = s.decay[j * kD + c];
                    const float4 y = *reinterpret_cast<const float4 *>(s.ak + j * s.nc + 8 * m);
                    const float4 z = *reinterpret_cast<const float4 *>(s.ak + j * s.nc + 8 * m + 4);
                    w[0] += y.x * x;
                    w[1] += y.y * x;
                    w[2] += y.z * x;
                    w[3] += y.w * x;
                    w[4] += z.x * x;
                    w[5] += z.y * x;
                    w[6] += z.z * x;
                    w[7] += z.w * x;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int node = 8 * m + i;
                    if (node >= n) break;
                    const float x = s.beta[node] * (__bfloat162float(s.k[node * kD + c]) - w[i]);
                    s.decay[node * kD + c] = x;
                    if (a.u != nullptr) a.u[u.at(a, node) + c] = x;
#pragma unroll
                    for (int l = i + 1; l < 8; ++l) w[l] += s.ak[node * s.nc + 8 * m + l] * x;
                }
            }
        }
        __syncthreads();
        if (more) fetch_rows(next, a.k);
        // The outputs: half of an eight's nodes for each half of the threads.
        for (int m = 0; m < eights; ++m) {
            float w[4];
            const int i0 = 8 * m + 4 * (tid / kD);
            if (i0 >= n) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = product(m, 8 + (i0 & 7) + i, c);
            const int end = min(i0 + 4, n);
#pragma unroll 4
            for (int j = 0; j < end; ++j) {
                const float x = s.decay[j * kD + c];
                const float4 y = *reinterpret_cast<const float4 *>(s.aq + j * s.nc + i0);
                w[0] += y.x * x;
                w[1] += y.y * x;
                w[2] += y.z * x;
                w[3] += y.w * x;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i0 + i < n) write_out<kOutBf16>(a.o, u.at(a, i0 + i) + c, w[i]);
            // (an update that is not finite shows in its own node's output)
            if (!finite((w[0] + w[1]) + (w[2] + w[3]))) s_again = 1;
        }
        __syncthreads();
        u = next;
    }
    __syncthreads();  // (there may have been no unit with nodes)
    if (s_again == 0) return;
    for (uint32_t unit = blockIdx.x; unit < units; unit += gridDim.x)
        solve_again<kStateBf16, kOutBf16, kEights>(a, unit, smem);
}

// ---- commit --------------------------------------------------------------------------------

// One block a (request, head); the state stays in registers between its read and its write: warp
// w owns rows w, w + 8, .., lane l the columns 4 l .. 4 l + 3, so a warp moves whole rows.  The
// path's nodes act sixteen at a time: S <- Diag(E) S + sum_j (E_j k_j) u_j^T, E and E_j the decays
// of the sixteen, and of those behind j.  Bound: the state is read and written once, 121 us for
// 6144 heads of fp32 at a copy's rate.  With the two other memories' commits 137 us; 161 with the
// path's rows loaded one after another, which waited behind the state each time (165 at two
// blocks an SM).
constexpr int kCommitNodes = 16;
constexpr int kRows = kD / kWarps;

template <bool kStateBf16>
__global__ void __launch_bounds__(kThreads, 3) tree_commit_kernel(const TreeStep a) {
    __shared__ __align__(16) float s_w[kCommitNodes][kD], s_u[kCommitNodes][kD], s_g[kCommitNodes][kD];
    __shared__ __align__(16) __nv_bfloat16 s_k[kCommitNodes][kD];
    __shared__ float s_decay[kD];
    const int b = blockIdx.x / a.H, h = blockIdx.x % a.H, tid = threadIdx.x;
    const int warp = tid >> 5, lane = tid & 31;
    const TreeRows t = tree_rows(a.cu, b, a.N, a.max_nodes);
    const int end = a.last[b];
    const int64_t slot = slot_of(a, b);
    if ((t.bad || end >= t.n) && tid == 0) record_device_error(a.err, kDevInvalidArg);
    if (end < 0 || end >= t.n || slot < 0) return;
    // the whole state in flight first
    const int64_t base = (slot * a.H + h) * (kD * kD) + warp * kD + 4 * lane;
    float4 x[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int64_t i = base + r * kWarps * kD;
        if constexpr (kStateBf16) {
            // four bf16 in the first two floats: one set of registers for both forms
            const float2 raw = __ldcs(reinterpret_cast<const float2 *>(static_cast<const __nv_bfloat16 *>(a.pool) + i));
            x[r].x = raw.x;
            x[r].y = raw.y;
        } else {
            x[r] = __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(a.pool) + i));
        }
    }
    uint64_t path = path_of(a.ancestors[t.first + end], end);
    auto at = [&](int i) { return ((t.first + i) * a.H + h) * kD; };
    bool first = true;
    while (path != 0) {
        // the next sixteen nodes from the root, and their last
        uint64_t some = 0, rest = path;
        int m = 0;
        for (; m < kCommitNodes && rest != 0; ++m) {
            some |= rest & (~rest + 1);
            rest &= rest - 1;
        }
        path = rest;
        if (!first) __syncthreads();
        // their rows, all on their way at once, from the last node up
        int r = 0;
        for (uint64_t p = some; p != 0; ++r) {
            const int j = top_bit(p);
            p ^= uint64_t{1} << j;
            if (r % kWarps != warp) continue;
            if (lane < 16) sm100::cp_async_16(&s_k[r][8 * lane], a.k + at(j) + 8 * lane, true);
            sm100::cp_async_16(&s_g[r][4 * lane], a.g + at(j) + 4 * lane, true);
            sm100::cp_async_16(&s_u[r][4 * lane], a.u + at(j) + 4 * lane, true);
        }
        sm100::cp_async_wait_all();
        __syncthreads();
        if (tid < kD) {
            float e = 1.f;
            for (r = 0; r < m; ++r) {
                s_w[r][tid] = e * __bfloat162float(s_k[r][tid]);
                e *= expf(s_g[r][tid]);
            }
            s_decay[tid] = e;
        }
        __syncthreads();
        if constexpr (kStateBf16)
            if (first)
#pragma unroll
                for (int r = 0; r < kRows; ++r)
                    x[r] = widen4(make_uint2(__float_as_uint(x[r].x), __float_as_uint(x[r].y)));
        first = false;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const float d = s_decay[warp + kWarps * r];
            x[r] = make_float4(x[r].x * d, x[r].y * d, x[r].z * d, x[r].w * d);
        }
        for (int j = 0; j < m; ++j) {
            const float4 u = *reinterpret_cast<const float4 *>(&s_u[j][4 * lane]);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float w = s_w[j][warp + kWarps * r];
                x[r].x += w * u.x;
                x[r].y += w * u.y;
                x[r].z += w * u.z;
                x[r].w += w * u.w;
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int64_t i = base + r * kWarps * kD;
        if constexpr (kStateBf16) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(x[r].x, x[r].y), hi = __floats2bfloat162_rn(x[r].z, x[r].w);
            __stcs(reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.pool) + i),
                   make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi)));
        } else {
            __stcs(reinterpret_cast<float4 *>(static_cast<float *>(a.pool) + i), x[r]);
        }
    }
}

template <bool kStateBf16, bool kOutBf16, int kEights>
cudaError_t decode_n(const TreeStep &a, int num_sms, cudaStream_t s) {
    using Smem = TreeSmem<kEights, kStateBf16>;
    const auto kernel = &tree_decode_kernel<kStateBf16, kOutBf16, kEights>;
    const cudaError_t e =
        ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), Smem::bytes(8 * kEights));
    if (e != cudaSuccess) return e;
    const int64_t units = static_cast<int64_t>(a.B) * a.H, most = static_cast<int64_t>(num_sms) * blocks_an_sm(kEights);
    kernel<<<static_cast<unsigned>(units < most ? units : most), kThreads,
             Smem::bytes(Smem::nodes(a.max_nodes)), s>>>(a);
    return cudaGetLastError();
}

template <bool kStateBf16, bool kOutBf16>
cudaError_t decode_t(const TreeStep &a, int num_sms, cudaStream_t s) {
    // (64 requests of 24 nodes, 96 heads: 444 us in the form of up to 32 nodes, 645 in that of 64; of 12
    // nodes 190, 260 and 374 us in the three)
    return a.max_nodes <= 16   ? decode_n<kStateBf16, kOutBf16, 2>(a, num_sms, s)
           : a.max_nodes <= 32 ? decode_n<kStateBf16, kOutBf16, 4>(a, num_sms, s)
                               : decode_n<kStateBf16, kOutBf16, 8>(a, num_sms, s);
}

template <bool kStateBf16>
cudaError_t commit_t(const TreeStep &a, cudaStream_t s) {
    tree_commit_kernel<kStateBf16><<<static_cast<unsigned>(a.B * a.H), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_decode(const TreeStep &a, bool state_bf16, bool o_bf16, int num_sms, cudaStream_t s) {
    if (state_bf16) return o_bf16 ? decode_t<true, true>(a, num_sms, s) : decode_t<true, false>(a, num_sms, s);
    return o_bf16 ? decode_t<false, true>(a, num_sms, s) : decode_t<false, false>(a, num_sms, s);
}

cudaError_t launch_tree_commit(const TreeStep &a, bool state_bf16, cudaStream_t s) {
    return state_bf16 ? commit_t<true>(a, s) : commit_t<false>(a, s);
}

}  // namespace kda
