// distill.cu -- a drafter's rows held to a teacher's top tokens: the divergence
// of the two and the gradient of the drafter's logits.
//
// With q = softmax(x / T) over the row and the teacher's K listed tokens:
//   p_k = exp(value_k) / sum of them,              L = sum_k p_k (log p_k - log q_k)
//     dL/dt_v = q_v - p_v
//   or, with the rest of the vocabulary as one more class,
//   p_k = exp(value_k), p_rest = 1 - sum of them,  L = the same + p_rest (log p_rest - log q_rest)
//     dL/dt_v = q_v M - p_v (listed),  q_v M - p_rest q_v / q_rest (not listed),  M = sum p_k + p_rest
// q_rest is summed over the tokens that are not listed, with a maximum of its own
// (as 1 - sum q_k it would be lost where the drafter is sure of a listed token): a
// bit per element says which are listed, and these are left out of the pass and
// joined at the end.
//
// The gradient needs the row twice: the pass leaves it in shared memory, spread
// over the CTAs of a cluster, so that it is read from memory once, and the
// gradient may take the row's place.  (A row too long for that is read again.)
#include <algorithm>

#include "kernels.cuh"
#include "rows.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;

struct Shared {
    SoftSum part[kWarps];
    SoftSum rest;            // this CTA's part of the tokens that are not listed
    int32_t ids[DSPARK_TOP_MAX];
    float4 red[kWarps];
    uint32_t bad;            // a bad teacher of this row, as this CTA sees it
};

// The CTA's largest a and b, and its sums of a, b and c; every thread gets them.
__device__ __forceinline__ void block_max(Shared& sh, float& a, float& b) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a = fmaxf(a, shfl_xor(a, o));
        b = fmaxf(b, shfl_xor(b, o));
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.red[threadIdx.x >> 5] = make_float4(a, b, 0.0f, 0.0f);
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) {
        const float4 o = sh.red[w];
        a = fmaxf(a, o.x);
        b = fmaxf(b, o.y);
    }
}
__device__ __forceinline__ void block_sum3(Shared& sh, float& a, float& b, float& c) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += shfl_xor(a, o);
        b += shfl_xor(b, o);
        c += shfl_xor(c, o);
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.red[threadIdx.x >> 5] = make_float4(a, b, c, 0.0f);
    __syncthreads();
    a = b = c = 0.0f;
    for (int w = 0; w < kWarps; ++w) {
        const float4 o = sh.red[w];
        a += o.x;
        b += o.y;
        c += o.z;
    }
}

template <typename G>
__device__ __forceinline__ G grad_of(float x);
template <>
__device__ __forceinline__ float grad_of<float>(float x) { return x; }
template <>
__device__ __forceinline__ uint16_t grad_of<uint16_t>(float x) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// One CTA's part of a gradient row, all of it one value.
template <typename G>
__device__ __forceinline__ void fill_grad(G* g, int V, uint32_t rank, uint32_t size, float x) {
    const G y = grad_of<G>(x);
    const int64_t a = (int64_t)V * rank / size, b = (int64_t)V * (rank + 1) / size;
    for (int64_t v = a + threadIdx.x; v < b; v += kThreads) g[v] = y;
}

// T: the logits' elements, G: the gradient's, kGrad: there is one.
template <typename T, typename G, bool kGrad>
__global__ void __launch_bounds__(kThreads) distill_kernel(const DistillParams p) {
    constexpr int kVec = Elem<T>::kVec;
    extern __shared__ uint4 dyn[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int64_t n = blockIdx.x / size;
    const T* row = reinterpret_cast<const T*>(p.student) + n * p.stride;
    G* grad = kGrad ? reinterpret_cast<G*>(p.grad) + n * p.grad_stride : nullptr;
    const float weight = p.weight ? p.weight[n] : 1.0f;
    if (weight == 0.0f) {
        if (kGrad) fill_grad(grad, p.V, rank, size, 0.0f);
        if (rank == 0 && tid == 0) p.loss[n] = 0.0f;
        return;
    }
    const RowView<T> view(row, p.V);
    const int first = (int)((int64_t)view.pieces * rank / size), end = (int)((int64_t)view.pieces * (rank + 1) / size);
    const int n_pieces = end - first;
    const bool staged = kGrad && p.staged;
    uint4* stage = dyn;                                                          // [n_pieces] if staged
    uint32_t* bits = reinterpret_cast<uint32_t*>(dyn + (staged ? n_pieces : 0));  // a bit per element of them
    const int n_words = (n_pieces * kVec + 31) / 32;

    // ---- the teacher's tokens: one to a thread
    const int id = tid < p.top_k ? p.ids[n * p.top_k + tid] : -1;
    const float value = id >= 0 ? p.teacher[n * p.top_k + tid] : -INFINITY;
    const bool listed = id >= 0 && id < p.V;
    const float x_mine = listed ? view.at(id) : -INFINITY;
    for (int i = tid; i < n_words; i += kThreads) bits[i] = 0;
    if (tid < DSPARK_TOP_MAX) sh.ids[tid] = id;
    if (tid == 0) sh.bad = 0;
    __syncthreads();
    if (id >= p.V || value != value || value == INFINITY || !(fabsf(weight) < INFINITY)) sh.bad = 1;
    const int mine = id - view.head - first * kVec;  // this CTA's element
    const bool here = listed && id >= view.head && mine >= 0 && mine < n_pieces * kVec;
    if (here && (atomicOr(&bits[mine >> 5], 1u << (mine & 31)) >> (mine & 31) & 1u)) sh.bad = 1;  // listed twice
    const int v_edge = view.edge(tid, rank == 0, rank == size - 1);
    int edge_count = 0;
    if (v_edge >= 0)
        for (int k = 0; k < p.top_k; ++k) edge_count += sh.ids[k] == v_edge;
    if (edge_count > 1) sh.bad = 1;
    const float x_edge = v_edge >= 0 ? view.at(v_edge) : -INFINITY;
    __syncthreads();

    // ---- one pass over the tokens that are not listed
    SoftSum t;
    for (int i0 = tid; i0 - tid < n_pieces; i0 += kUnroll * kThreads) {
        uint4 w[kUnroll];
#pragma unroll
        for (int q = 0; q < kUnroll; ++q) w[q] = load_piece<T>(view.base + first, i0 + q * kThreads, n_pieces);
        float x[kUnroll * kVec];
#pragma unroll
        for (int q = 0; q < kUnroll; ++q) {
            const int i = i0 + q * kThreads;
            Elem<T>::unpack(w[q], x + q * kVec);
            if (i < n_pieces) {
                if (staged) stage[i] = w[q];
                const uint32_t m = bits[i * kVec >> 5] >> (i * kVec & 31) & ((1u << kVec) - 1u);
                if (m)
#pragma unroll
                    for (int e = 0; e < kVec; ++e)
                        if (m >> e & 1u) x[q * kVec + e] = -INFINITY;
            }
        }
        soft_add<false>(t, x, p.c2);
    }
    const float edge[2] = {edge_count ? -INFINITY : x_edge, -INFINITY};
    soft_add<false>(t, edge, p.c2);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        SoftSum b;
        b.m = shfl_xor(t.m, o);
        b.s = shfl_xor(t.s, o);
        soft_merge<false>(t, b, p.c2);
    }
    if (lane == 0) sh.part[warp] = t;
    __syncthreads();
    if (tid == 0) {
        SoftSum a = sh.part[0];
        for (int w = 1; w < kWarps; ++w) soft_merge<false>(a, sh.part[w], p.c2);
        sh.rest = a;
    }
    cluster_sync();
    // ---- joined over the cluster, by every CTA
    SoftSum rest;
    bool bad = false;
    for (uint32_t c = 0; c < size; ++c) {
        const uint32_t a = cluster_map(&sh.rest, c);
        SoftSum b;
        b.m = cluster_ld_f32(a + offsetof(SoftSum, m));
        b.s = cluster_ld_f32(a + offsetof(SoftSum, s));
        soft_merge<false>(rest, b, p.c2);
        bad |= cluster_ld_u32(cluster_map(&sh.bad, c)) != 0;
    }
    // the teacher's classes, and the row's maximum and sum over listed tokens and rest
    float top = x_mine, v_top = value;
    block_max(sh, top, v_top);
    const float v_ref = p.rest ? 0.0f : v_top;  // (a list of -inf alone has no mass)
    const float p_raw = value > -INFINITY ? expf(value - v_ref) : 0.0f;
    const float m_all = fmaxf(top, rest.m);
    const float f_rest = rest.m > -INFINITY ? exp2_approx(fmaxf((rest.m - m_all) * p.c2, -200.0f)) : 0.0f;
    float mass = p_raw, e_sum = x_mine > -INFINITY ? exp2_approx(fmaxf((x_mine - m_all) * p.c2, -200.0f)) : 0.0f;
    float bad_listed = x_mine != x_mine ? 1.0f : 0.0f;
    block_sum3(sh, mass, e_sum, bad_listed);
    const float total = e_sum + rest.s * f_rest;
    bad |= bad_listed > 0.0f || !(total > 0.0f && total < INFINITY) || m_all == INFINITY || rest.s != rest.s ||
           !(mass < INFINITY);
    const float log_total = logf(total);
    float p_rest = 0.0f, scale = 1.0f, log_scale = 0.0f, all_mass;
    if (p.rest) {
        // (no class of the rest where the drafter has no token left for it)
        if (rest.m > -INFINITY) p_rest = fmaxf(1.0f - mass, 0.0f);
        all_mass = mass + p_rest;
    } else {
        all_mass = mass > 0.0f ? 1.0f : 0.0f;  // nothing listed: nothing to learn from
        if (mass > 0.0f) {
            scale = 1.0f / mass;
            log_scale = -v_ref - logf(mass);
        }
    }
    const float p_mine = p_raw * scale;
    float term = 0.0f;
    if (p_mine > 0.0f) term = p_mine * ((value + log_scale) - ((x_mine - m_all) * p.invT - log_total));
    float none = 0.0f, zero = 0.0f;
    block_sum3(sh, term, none, zero);
    if (p_rest > 0.0f) term += p_rest * (logf(p_rest) - ((rest.m - m_all) * p.invT + logf(rest.s) - log_total));
    if (rank == 0 && tid == 0) {
        p.loss[n] = bad ? NAN : weight * term;
        if (bad) report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
    }
    if (size > 1) cluster_sync();  // (no CTA ends, or writes over the row, while another reads)
    if (!kGrad) return;
    if (bad) {
        fill_grad(grad, p.V, rank, size, NAN);
        return;
    }
    // ---- the gradient: e^(t - t_rest max) times one factor where a token is not listed
    const float w = weight * p.invT;
    const float m_ref = rest.m;
    const float factor = m_ref > -INFINITY ? w * (all_mass * f_rest / total - (p_rest > 0.0f ? p_rest / rest.s : 0.0f)) : 0.0f;
    auto gradient = [&](float x) {
        return m_ref > -INFINITY ? factor * exp2_approx(fmaxf((x - m_ref) * p.c2, -200.0f)) : 0.0f;
    };
    for (int i = tid; i < n_pieces; i += kThreads) {
        float x[kVec];
        Elem<T>::unpack(staged ? stage[i] : __ldcs(view.base + first + i), x);
#pragma unroll
        for (int e = 0; e < kVec; ++e) grad[(int64_t)view.head + ((int64_t)first + i) * kVec + e] = grad_of<G>(gradient(x[e]));
    }
    if (v_edge >= 0 && !edge_count) grad[v_edge] = grad_of<G>(gradient(x_edge));
    __syncthreads();
    const bool edge_mine = listed && (id < view.head ? rank == 0 : id >= view.head + view.pieces * kVec && rank == size - 1);
    if (here || edge_mine) {
        const float q = x_mine > -INFINITY ? exp2_approx(fmaxf((x_mine - m_all) * p.c2, -200.0f)) / total : 0.0f;
        grad[id] = grad_of<G>(w * (all_mass * q - p_mine));
    }
}

template <typename T>
const void* kernel_of(bool grad, int grad_dtype) {
    if (!grad) return (const void*)distill_kernel<T, float, false>;
    return grad_dtype == DSPARK_F32 ? (const void*)distill_kernel<T, float, true>
                                    : (const void*)distill_kernel<T, uint16_t, true>;
}

}  // namespace

cudaError_t launch_distill(DistillParams p, cudaStream_t stream) {
    const int vec = p.dtype == DSPARK_F32 ? 4 : 8;
    const int64_t pieces = p.V / vec;
    int ctas = 1;
    auto smem_of = [&](int c, bool staged) {
        const int64_t per = (pieces + c - 1) / c;
        return (size_t)(staged ? per * 16 : 0) + (size_t)((per * vec + 31) / 32) * 4;
    };
    while (ctas < 8 && smem_of(ctas, p.grad != nullptr) > 72 * 1024) ctas *= 2;
    p.staged = p.grad && smem_of(ctas, true) <= 200 * 1024;
    const size_t smem = smem_of(ctas, p.staged);
    const void* fn = p.dtype == DSPARK_F32 ? kernel_of<float>(p.grad != nullptr, p.grad_dtype)
                                           : kernel_of<uint16_t>(p.grad != nullptr, p.grad_dtype);
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.rows * (int64_t)ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {&p};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace dspark
