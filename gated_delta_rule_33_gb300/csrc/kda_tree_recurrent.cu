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
#include "kda_sm100.cuh"
#include "kda_tree.cuh"

namespace kda {
namespace {

constexpr int kD = 128;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <bool kBf16>
__device__ __forceinline__ float state_at(const void *pool, int64_t i) {
    if constexpr (kBf16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(pool)[i]);
    else return static_cast<const float *>(pool)[i];
}

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

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// One block a (request, head).
template <bool kStateBf16, bool kOutBf16>
__global__ void __launch_bounds__(kThreads) tree_decode_kernel(const TreeStep a) {
    extern __shared__ float smem[];
    const int b = blockIdx.x / a.H, h = blockIdx.x % a.H, tid = threadIdx.x;
    const int warp = tid >> 5, lane = tid & 31;
    const TreeRows t = tree_rows(a.cu, b, a.N, a.max_nodes);
    if (t.bad && tid == 0) record_device_error(a.err, kDevInvalidArg);
    const int64_t slot = slot_of(a, b);
    const int n = t.n;
    if (n == 0 || slot < 0) {
        for (int64_t i = tid; i < static_cast<int64_t>(t.rows) * kD; i += kThreads) {
            const int64_t at = ((t.first + i / kD) * a.H + h) * kD + i % kD;
            write_out<kOutBf16>(a.o, at, 0.f);
            if (a.u != nullptr) a.u[at] = 0.f;
        }
        return;
    }
    float *s_kb = smem;                      // [n][128] E_i k_i
    float *s_qb = s_kb + a.max_nodes * kD;   // [n][128] scale E_i q_i
    float *s_u = s_qb + a.max_nodes * kD;    // [n][128]
    float *s_ak = s_u + a.max_nodes * kD;    // [n][n] (E_ij k_j) . k_i
    float *s_aq = s_ak + a.max_nodes * a.max_nodes;
    auto at = [&](int i) { return ((t.first + i) * a.H + h) * kD; };

    for (int i = warp; i < n; i += kWarps) {
        uint64_t path = path_of(a.ancestors[t.first + i], i);
        float e[4] = {1.f, 1.f, 1.f, 1.f}, k[4], q[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            k[c] = __bfloat162float(a.k[at(i) + lane + 32 * c]);
            q[c] = a.scale * __bfloat162float(a.q[at(i) + lane + 32 * c]);
        }
        while (path != 0) {
            const int j = top_bit(path);
            path ^= uint64_t{1} << j;
            float dk = 0.f, dq = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float x = e[c] * __bfloat162float(a.k[at(j) + lane + 32 * c]);
                dk += x * k[c];
                dq += x * q[c];
                e[c] *= expf(a.g[at(j) + lane + 32 * c]);
            }
            dk = warp_sum(dk);
            dq = warp_sum(dq);
            if (lane == 0) {
                s_ak[i * a.max_nodes + j] = dk;
                s_aq[i * a.max_nodes + j] = dq;
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            s_kb[i * kD + lane + 32 * c] = e[c] * k[c];
            s_qb[i * kD + lane + 32 * c] = e[c] * q[c];
        }
    }
    __syncthreads();
    // threads 0 .. 127 the k products and the updates, the others the q products
    const int c = tid & (kD - 1);
    const bool is_q = tid >= kD;
    const int64_t S = (slot * a.H + h) * (kD * kD) + c;
    for (int i = 0; i < n; ++i) {
        const float *row = (is_q ? s_qb : s_kb) + i * kD;
        float acc = 0.f;
        for (int r = 0; r < kD; ++r) acc += row[r] * state_at<kStateBf16>(a.pool, S + r * kD);
        uint64_t path = a.ancestors[t.first + i] & bits_below(i);
        while (path != 0) {
            const int j = top_bit(path);
            path ^= uint64_t{1} << j;
            acc += (is_q ? s_aq : s_ak)[i * a.max_nodes + j] * s_u[j * kD + c];
        }
        if (!is_q) {
            const float u = a.beta[(t.first + i) * a.H + h] * (__bfloat162float(a.v[at(i) + c]) - acc);
            s_u[i * kD + c] = u;
            if (a.u != nullptr) a.u[at(i) + c] = u;
        }
        __syncthreads();
        if (is_q)
            write_out<kOutBf16>(a.o, at(i) + c, acc + s_aq[i * a.max_nodes + i] * s_u[i * kD + c]);
    }
}

// One block a (request, head): warp w owns rows w, w + 8, .. of the state, lane l the columns
// 4 l .. 4 l + 3, so a warp moves whole 512-byte rows.
template <bool kStateBf16>
__global__ void __launch_bounds__(kThreads) tree_commit_kernel(const TreeStep a) {
    extern __shared__ float smem[];
    const int b = blockIdx.x / a.H, h = blockIdx.x % a.H, tid = threadIdx.x;
    const int warp = tid >> 5, lane = tid & 31;
    const TreeRows t = tree_rows(a.cu, b, a.N, a.max_nodes);
    const int end = a.last[b];
    if ((t.bad || end >= t.n) && tid == 0) record_device_error(a.err, kDevInvalidArg);
    const int64_t slot = slot_of(a, b);
    if (end < 0 || end >= t.n || slot < 0) return;
    float *s_w = smem;                             // [nodes of the path][128] E_ej k_j
    float *s_u = smem + a.max_nodes * kD;          // [nodes of the path][128]
    __shared__ float s_decay[kD];
    uint64_t path = path_of(a.ancestors[t.first + end], end);
    const int m = __popcll(path);
    auto at = [&](int i) { return ((t.first + i) * a.H + h) * kD; };
    if (tid < kD) {
        float e = 1.f;
        for (int r = 0; r < m; ++r) {
            const int j = top_bit(path);
            path ^= uint64_t{1} << j;
            s_w[r * kD + tid] = e * __bfloat162float(a.k[at(j) + tid]);
            e *= expf(a.g[at(j) + tid]);
        }
        s_decay[tid] = e;
    } else {
        for (int r = 0; r < m; ++r) {
            const int j = top_bit(path);
            path ^= uint64_t{1} << j;
            s_u[r * kD + tid - kD] = a.u[at(j) + tid - kD];
        }
    }
    __syncthreads();
    const int64_t S = (slot * a.H + h) * (kD * kD);
    for (int r = warp; r < kD; r += kWarps) {
        const int64_t i = S + r * kD + 4 * lane;
        float x[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = s_decay[r] * state_at<kStateBf16>(a.pool, i + c);
        for (int j = 0; j < m; ++j) {
            const float w = s_w[j * kD + r];
#pragma unroll
            for (int c = 0; c < 4; ++c) x[c] += w * s_u[j * kD + 4 * lane + c];
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) write_out<kStateBf16>(a.pool, i + c, x[c]);
    }
}

int decode_smem(int n) { return (3 * n * kD + 2 * n * n) * 4; }
int commit_smem(int n) { return 2 * n * kD * 4; }

template <bool kStateBf16, bool kOutBf16>
cudaError_t decode_t(const TreeStep &a, cudaStream_t s) {
    const auto kernel = &tree_decode_kernel<kStateBf16, kOutBf16>;
    const cudaError_t e =
        ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), decode_smem(kTreeNodes));
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(a.B * a.H), kThreads, decode_smem(a.max_nodes), s>>>(a);
    return cudaGetLastError();
}

template <bool kStateBf16>
cudaError_t commit_t(const TreeStep &a, cudaStream_t s) {
    const auto kernel = &tree_commit_kernel<kStateBf16>;
    const cudaError_t e =
        ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), commit_smem(kTreeNodes));
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(a.B * a.H), kThreads, commit_smem(a.max_nodes), s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_decode(const TreeStep &a, bool state_bf16, bool o_bf16, cudaStream_t s) {
    if (state_bf16) return o_bf16 ? decode_t<true, true>(a, s) : decode_t<true, false>(a, s);
    return o_bf16 ? decode_t<false, true>(a, s) : decode_t<false, false>(a, s);
}

cudaError_t launch_tree_commit(const TreeStep &a, bool state_bf16, cudaStream_t s) {
    return state_bf16 ? commit_t<true>(a, s) : commit_t<false>(a, s);
}

}  // namespace kda
