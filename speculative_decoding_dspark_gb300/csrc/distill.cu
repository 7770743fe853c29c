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
// The gradient of a token that is not listed is one factor times exp(t - t_max of
// the rest), so it takes a second pass over the row once the sums are known.  Rows
// stay in shared memory for it, each spread over the CTAs of a cluster, so that
// they are read from memory once, and the gradient may take the row's place.
// Clusters walk down the rows; a thread's pieces of the next row are on their way, by
// asynchronous copies into the places that the second pass has just emptied (each
// thread fills and empties places of its own: no barrier).  What a place cannot be
// found for (rows longer than the cluster's shared memory) is read twice.  One warp
// keeps the listed tokens and does all that is done once per row.
#include <algorithm>

#include "kernels.cuh"
#include "rows.cuh"
#include "tc_ptx.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;     // pieces of a batch
constexpr int kMaxCtas = 8;    // of a cluster
constexpr int kPerLane = DSPARK_TOP_MAX / 32;

struct Part {  // the tokens that are not listed, as one CTA sees them
    float m, s, bad;
};

struct Shared {
    SoftSum warp_sum[kWarps];
    Part parts[2][kMaxCtas];  // of all CTAs, by the row's parity
    float factor, m_ref;      // the gradient of a token that is not listed: factor 2^((x - m_ref) c2)
    int bad;
};

__device__ __forceinline__ float warp_max(float a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, shfl_xor(a, o));
    return a;
}
__device__ __forceinline__ float warp_sum(float a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += shfl_xor(a, o);
    return a;
}

template <typename G>
__device__ __forceinline__ G grad_of(float x);
template <>
__device__ __forceinline__ float grad_of<float>(float x) { return x; }
template <>
__device__ __forceinline__ uint16_t grad_of<uint16_t>(float x) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// N neighbours of a gradient row, whose address is a multiple of their size (or of 16).
template <int N>
__device__ __forceinline__ void store_piece(float* p, const float (&x)[N]) {
#pragma unroll
    for (int e = 0; e < N; e += 4) __stcs(reinterpret_cast<float4*>(p + e), make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]));
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    const __nv_bfloat162 y = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ void store_piece(uint16_t* p, const float (&x)[4]) {
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3])));
}
__device__ __forceinline__ void store_piece(uint16_t* p, const float (&x)[8]) {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]),
                                                   bf16_pair(x[6], x[7])));
}

// One CTA's part of a gradient row, all of it one value.
template <typename G>
__device__ __forceinline__ void fill_grad(G* g, int V, uint32_t rank, uint32_t size, float x) {
    const G y = grad_of<G>(x);
    const int64_t a = (int64_t)V * rank / size, b = (int64_t)V * (rank + 1) / size;
    for (int64_t v = a + threadIdx.x; v < b; v += kThreads) g[v] = y;
}

// At most `left` (or 7) of this thread's groups of copies still on their way.
__device__ __forceinline__ void copies_left(int left) {
    switch (left) {
        case 0: tc::cp_async_wait<0>(); break;
        case 1: tc::cp_async_wait<1>(); break;
        case 2: tc::cp_async_wait<2>(); break;
        case 3: tc::cp_async_wait<3>(); break;
        case 4: tc::cp_async_wait<4>(); break;
        case 5: tc::cp_async_wait<5>(); break;
        case 6: tc::cp_async_wait<6>(); break;
        default: tc::cp_async_wait<7>(); break;
    }
}

// This CTA's share of a row.
template <typename T>
struct Share {
    RowView<T> view;
    int first, n;      // its pieces
    int v0, v1;        // its elements, the row's edges among them
    __device__ __forceinline__ Share(const DistillParams& p, int64_t row, uint32_t rank, uint32_t size)
        : view(reinterpret_cast<const T*>(p.student) + row * p.stride, p.V) {
        first = (int)((int64_t)view.pieces * rank / size);
        const int end = (int)((int64_t)view.pieces * (rank + 1) / size);
        n = end - first;
        v0 = rank == 0 ? 0 : view.head + first * Elem<T>::kVec;
        v1 = rank == size - 1 ? p.V : view.head + end * Elem<T>::kVec;
    }
    __device__ __forceinline__ const uint4* pieces() const { return view.base + first; }
    // The bit of its element v (a word is kept for the edges on either side).
    __device__ __forceinline__ int bit(int v) const { return v - view.head - first * Elem<T>::kVec + 32; }
    __device__ __forceinline__ int batches() const { return (n + kUnroll * kThreads - 1) / (kUnroll * kThreads); }
};

// A row's listed tokens, four to a lane of the first warp.
struct Listed {
    int id[kPerLane];    // -1: none
    float x[kPerLane];   // the drafter's logit
    float value[kPerLane];
};

// T: the logits' elements, G: the gradient's, kGrad: there is one.
template <typename T, typename G, bool kGrad>
__global__ void __launch_bounds__(kThreads) distill_kernel(const DistillParams p) {
    constexpr int kVec = Elem<T>::kVec;
    extern __shared__ uint4 dyn[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int clusters = gridDim.x / size;
    uint4* stage = dyn + tid;                                                     // [p.staged batches][kUnroll][kThreads]
    uint32_t* bits = reinterpret_cast<uint32_t*>(dyn + p.staged * kUnroll * kThreads);
    for (int i = tid; i < p.bit_words; i += kThreads) bits[i] = 0;

    auto weight_of = [&](int64_t n) { return p.weight ? __ldg(p.weight + n) : 1.0f; };
    // The next row from n on that has a weight; those that have none are done with.
    auto active = [&](int64_t n, float& w) {
        while (n < p.rows && w == 0.0f) {
            if (kGrad) fill_grad(reinterpret_cast<G*>(p.grad) + n * p.grad_stride, p.V, rank, size, 0.0f);
            if (rank == 0 && tid == 0) p.loss[n] = 0.0f;
            n += clusters;
            if (n < p.rows) w = weight_of(n);
        }
        return n;
    };
    auto copy_batch = [&](const Share<T>& s, int b) {
#pragma unroll
        for (int q = 0; q < kUnroll; ++q) {
            const int i = (b * kUnroll + q) * kThreads + tid;
            if (i < s.n) tc::cp_async_16(tc::smem_u32(stage + (b * kUnroll + q) * kThreads), s.pieces() + i, 16);
        }
        tc::cp_async_commit();
    };
    // (first warp) a row's listed tokens
    auto fetch = [&](int64_t n, Listed& t) {
        const RowView<T> view(reinterpret_cast<const T*>(p.student) + n * p.stride, p.V);
#pragma unroll
        for (int q = 0; q < kPerLane; ++q) {
            const int k = lane + 32 * q;
            t.id[q] = k < p.top_k ? __ldg(p.ids + n * p.top_k + k) : -1;
            t.value[q] = k < p.top_k ? __ldg(p.teacher + n * p.top_k + k) : -INFINITY;
        }
#pragma unroll
        for (int q = 0; q < kPerLane; ++q) {
            if (t.id[q] < 0) t.value[q] = -INFINITY;
            t.x[q] = t.id[q] >= 0 && t.id[q] < p.V ? view.at(t.id[q]) : -INFINITY;
        }
    };
    // (first warp) marks a row's listed tokens; whether something is wrong with them
    auto mark = [&](const Share<T>& s, const Listed& t) {
        bool bad = false;
#pragma unroll
        for (int q = 0; q < kPerLane; ++q) {
            bad |= t.id[q] >= p.V || t.value[q] != t.value[q] || t.value[q] == INFINITY || t.x[q] != t.x[q];
            if (t.id[q] >= s.v0 && t.id[q] < s.v1) {
                const int b = s.bit(t.id[q]);
                bad |= (atomicOr(&bits[b >> 5], 1u << (b & 31)) >> (b & 31) & 1u) != 0;  // listed twice
            }
        }
        return __any_sync(0xFFFFFFFFu, bad);
    };

    int64_t row = blockIdx.x / size;
    if (row >= p.rows) return;  // (the whole cluster)
    float weight = weight_of(row);
    row = active(row, weight);
    Listed now;
    bool bad_list = false;
    __syncthreads();
    if (row < p.rows) {
        const Share<T> s(p, row, rank, size);
        if (kGrad)
            for (int b = 0; b < p.staged; ++b) copy_batch(s, b);
        if (warp == 0) {
            fetch(row, now);
            bad_list = mark(s, now);
        }
    }
    __syncthreads();

    for (int parity = 0; row < p.rows; parity ^= 1) {
        const Share<T> s(p, row, rank, size);
        const int n_batches = s.batches();
        const int v_edge = warp == 1 ? s.view.edge(lane, rank == 0, rank == size - 1) : -1;
        const float x_edge = v_edge >= 0 ? s.view.at(v_edge) : -INFINITY;
        int64_t next = row + clusters;
        float next_weight = next < p.rows ? weight_of(next) : 0.0f;

        // ---- first pass: the tokens that are not listed
        SoftSum t;
        for (int b = 0; b < n_batches; ++b) {
            uint4 w[kUnroll];
            if (kGrad && b < p.staged) {
                copies_left(p.staged - 1 - b);
#pragma unroll
                for (int q = 0; q < kUnroll; ++q) {
                    constexpr uint32_t k = Elem<T>::kMinusInf;
                    const int i = (b * kUnroll + q) * kThreads + tid;
                    w[q] = i < s.n ? stage[(b * kUnroll + q) * kThreads] : make_uint4(k, k, k, k);
                }
            } else {
#pragma unroll
                for (int q = 0; q < kUnroll; ++q) w[q] = load_piece<T>(s.pieces(), (b * kUnroll + q) * kThreads + tid, s.n);
            }
            float x[kUnroll * kVec];
#pragma unroll
            for (int q = 0; q < kUnroll; ++q) {
                const int i = (b * kUnroll + q) * kThreads + tid;
                Elem<T>::unpack(w[q], x + q * kVec);
                if (i < s.n) {
                    const uint32_t m = bits[1 + (i * kVec >> 5)] >> (i * kVec & 31) & ((1u << kVec) - 1u);
                    if (m)
#pragma unroll
                        for (int e = 0; e < kVec; ++e)
                            if (m >> e & 1u) x[q * kVec + e] = -INFINITY;
                }
            }
            soft_add<false>(t, x, p.c2);
        }
        if (warp == 1) {
            const int b = v_edge >= 0 ? s.bit(v_edge) : 0;
            const float edge[2] = {v_edge >= 0 && !(bits[b >> 5] >> (b & 31) & 1u) ? x_edge : -INFINITY, -INFINITY};
            soft_add<false>(t, edge, p.c2);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            SoftSum b;
            b.m = shfl_xor(t.m, o);
            b.s = shfl_xor(t.s, o);
            soft_merge<false>(t, b, p.c2);
        }
        if (lane == 0) sh.warp_sum[warp] = t;
        __syncthreads();
        // ---- the CTA's sums to all CTAs of the cluster
        if (warp == 0) {
            SoftSum a;
            if (lane < kWarps) a = sh.warp_sum[lane];
#pragma unroll
            for (int o = kWarps / 2; o > 0; o >>= 1) {
                SoftSum b;
                b.m = shfl_xor(a.m, o);
                b.s = shfl_xor(a.s, o);
                soft_merge<false>(a, b, p.c2);
            }
            a.m = __shfl_sync(0xFFFFFFFFu, a.m, 0);
            a.s = __shfl_sync(0xFFFFFFFFu, a.s, 0);
            if (lane < (int)size) {
                const uint32_t to = cluster_map(&sh.parts[parity][rank], lane);
                cluster_st_f32(to + offsetof(Part, m), a.m);
                cluster_st_f32(to + offsetof(Part, s), a.s);
                cluster_st_f32(to + offsetof(Part, bad), bad_list ? 1.0f : 0.0f);
            }
            __syncwarp();
        }
        cluster_arrive();
        next = active(next, next_weight);
        Listed then;
        if (warp == 0) {
            // this row's marks go
#pragma unroll
            for (int q = 0; q < kPerLane; ++q)
                if (now.id[q] >= s.v0 && now.id[q] < s.v1) bits[s.bit(now.id[q]) >> 5] = 0;
            if (next < p.rows) fetch(next, then);
            cluster_wait();
            SoftSum rest;
            float bad_f = 0.0f;
            if (lane < (int)size) {
                const Part a = sh.parts[parity][lane];
                rest.m = a.m;
                rest.s = a.s;
                bad_f = a.bad;
            }
#pragma unroll
            for (int o = kMaxCtas / 2; o > 0; o >>= 1) {
                SoftSum b;
                b.m = shfl_xor(rest.m, o);
                b.s = shfl_xor(rest.s, o);
                soft_merge<false>(rest, b, p.c2);
            }
            rest.m = __shfl_sync(0xFFFFFFFFu, rest.m, 0);
            rest.s = __shfl_sync(0xFFFFFFFFu, rest.s, 0);
            bool bad = __any_sync(0xFFFFFFFFu, bad_f != 0.0f) || !(fabsf(weight) < INFINITY);
            // the teacher's classes, and the row's maximum and sum over listed tokens and rest
            float x_top = -INFINITY, v_top = -INFINITY;
#pragma unroll
            for (int q = 0; q < kPerLane; ++q) {
                x_top = fmaxf(x_top, now.x[q]);
                v_top = fmaxf(v_top, now.value[q]);
            }
            const float m_all = fmaxf(warp_max(x_top), rest.m);
            v_top = p.rest ? 0.0f : warp_max(v_top);  // (a list of -inf alone has no mass)
            float prob[kPerLane], e_listed[kPerLane], mass = 0.0f, e_sum = 0.0f;
#pragma unroll
            for (int q = 0; q < kPerLane; ++q) {
                prob[q] = now.value[q] > -INFINITY ? expf(now.value[q] - v_top) : 0.0f;
                e_listed[q] = now.x[q] > -INFINITY ? exp2_approx((now.x[q] - m_all) * p.c2) : 0.0f;
                mass += prob[q];
                e_sum += e_listed[q];
            }
            mass = warp_sum(mass);
            const float f_rest = rest.m > -INFINITY ? exp2_approx((rest.m - m_all) * p.c2) : 0.0f;
            const float total = warp_sum(e_sum) + rest.s * f_rest;
            bad |= !(total > 0.0f && total < INFINITY) || m_all == INFINITY || rest.s != rest.s || !(mass < INFINITY);
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
                    log_scale = -v_top - logf(mass);
                }
            }
            const float w = weight * p.invT;
            if (rank == 0) {
                float term = 0.0f;
#pragma unroll
                for (int q = 0; q < kPerLane; ++q)
                    if (prob[q] > 0.0f)
                        term += prob[q] * scale * ((now.value[q] + log_scale) - ((now.x[q] - m_all) * p.invT - log_total));
                term = warp_sum(term);
                if (p_rest > 0.0f) term += p_rest * (logf(p_rest) - ((rest.m - m_all) * p.invT + logf(rest.s) - log_total));
                if (lane == 0) {
                    p.loss[row] = bad ? NAN : weight * term;
                    if (bad) report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
                }
            }
            if (lane == 0) {
                sh.bad = bad;
                sh.m_ref = rest.m;
                sh.factor = rest.m > -INFINITY ? w * (all_mass * f_rest / total - (p_rest > 0.0f ? p_rest / rest.s : 0.0f)) : 0.0f;
            }
            // the listed tokens' gradients, to be written over those of the second pass
            if (kGrad)
#pragma unroll
                for (int q = 0; q < kPerLane; ++q) now.x[q] = w * (all_mass * (e_listed[q] / total) - prob[q] * scale);
        } else {
            cluster_wait();
        }
        __syncthreads();
        // ---- second pass: the gradient; the next row's pieces follow this one's
        if (kGrad) {
            G* grad = reinterpret_cast<G*>(p.grad) + row * p.grad_stride;
            const Share<T> after(p, next < p.rows ? next : row, rank, size);
            const bool bad = sh.bad, more = next < p.rows;
            const float m_ref = bad ? NAN : sh.m_ref, factor = sh.factor;
            const bool none = !bad && m_ref == -INFINITY;  // (-inf alone is not listed)
            const float2 minus = make_float2(-m_ref, -m_ref), c2 = make_float2(p.c2, p.c2), f2 = make_float2(factor, factor);
            G* out = grad + s.view.head + (int64_t)s.first * kVec;
            const bool wide = reinterpret_cast<uintptr_t>(out) % (kVec * sizeof(G) < 16 ? kVec * sizeof(G) : 16) == 0;
            const int all_batches = more ? max(n_batches, p.staged) : n_batches;
            for (int b = 0; b < all_batches; ++b) {
                uint4 w[kUnroll];
#pragma unroll
                for (int q = 0; q < kUnroll; ++q) {
                    const int i = (b * kUnroll + q) * kThreads + tid;
                    if (i < s.n) w[q] = b < p.staged ? stage[(b * kUnroll + q) * kThreads] : __ldcs(s.pieces() + i);
                }
#pragma unroll
                for (int q = 0; q < kUnroll; ++q) {
                    const int i = (b * kUnroll + q) * kThreads + tid;
                    if (i >= s.n) continue;
                    float x[kVec];
                    Elem<T>::unpack(w[q], x);
#pragma unroll
                    for (int e = 0; e < kVec; e += 2) {
                        const float2 a = mul2(add2(make_float2(x[e], x[e + 1]), minus), c2);
                        const float2 y = mul2(make_float2(exp2_approx(a.x), exp2_approx(a.y)), f2);
                        x[e] = none ? 0.0f : y.x;
                        x[e + 1] = none ? 0.0f : y.y;
                    }
                    if (wide) {
                        store_piece(out + (int64_t)i * kVec, x);
                    } else {
#pragma unroll
                        for (int e = 0; e < kVec; ++e) out[(int64_t)i * kVec + e] = grad_of<G>(x[e]);
                    }
                }
                if (more && b < p.staged) copy_batch(after, b);
            }
            if (v_edge >= 0) grad[v_edge] = grad_of<G>(none ? 0.0f : factor * exp2_approx((x_edge - m_ref) * p.c2));
            if (warp == 0 && more) bad_list = mark(after, then);
            __syncthreads();
            if (warp == 0 && !bad)
#pragma unroll
                for (int q = 0; q < kPerLane; ++q)
                    if (now.id[q] >= s.v0 && now.id[q] < s.v1) grad[now.id[q]] = grad_of<G>(now.x[q]);
        } else {
            if (warp == 0 && next < p.rows) bad_list = mark(Share<T>(p, next, rank, size), then);
            __syncthreads();
        }
        now = then;
        row = next;
        weight = next_weight;
    }
    cluster_sync();  // (no CTA ends while another may still write to its shared memory)
}

template <typename T>
const void* kernel_of(bool grad, int grad_dtype) {
    if (!grad) return (const void*)distill_kernel<T, float, false>;
    return grad_dtype == DSPARK_F32 ? (const void*)distill_kernel<T, float, true>
                                    : (const void*)distill_kernel<T, uint16_t, true>;
}

}  // namespace

cudaError_t launch_distill(DistillParams p, cudaStream_t stream) {
    constexpr size_t kShare = 104 * 1024;  // shared memory of a CTA, so that two fit on an SM
    const int vec = p.dtype == DSPARK_F32 ? 4 : 8;
    const int64_t pieces = p.V / vec;
    int ctas = 1;
    auto batches_of = [&](int c) { return (int)(((pieces + c - 1) / c + kUnroll * kThreads - 1) / (kUnroll * kThreads)); };
    auto bits_of = [&](int c) { return (int)(((pieces + c - 1) / c * vec + 31) / 32 + 2); };
    auto smem_of = [&](int c, int batches) { return (size_t)batches * kUnroll * kThreads * 16 + (size_t)bits_of(c) * 4; };
    auto larger = [&](int c) {
        return smem_of(c, p.grad ? batches_of(c) : 0) > kShare || ((int64_t)p.rows * c < 152 && pieces / c > 2 * kThreads);
    };
    while (ctas < kMaxCtas && larger(ctas)) ctas *= 2;
    p.staged = p.grad ? std::min<int64_t>(batches_of(ctas), (int64_t)((kShare - std::min(kShare, smem_of(ctas, 0))) / (kUnroll * kThreads * 16))) : 0;
    p.bit_words = bits_of(ctas);
    const size_t smem = smem_of(ctas, p.staged);
    const void* fn = p.dtype == DSPARK_F32 ? kernel_of<float>(p.grad != nullptr, p.grad_dtype)
                                           : kernel_of<uint16_t>(p.grad != nullptr, p.grad_dtype);
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = p.rows;
    if (p.grad) {  // as many as there is room for at a time: they walk down the rows
        cfg.gridDim = dim3((unsigned)ctas);
        int room = 0;
        if ((e = cudaOccupancyMaxActiveClusters(&room, fn, &cfg)) != cudaSuccess) return e;
        clusters = std::min(clusters, std::max(1, room));
    }
    cfg.gridDim = dim3((unsigned)(clusters * (int64_t)ctas));
    void* args[] = {&p};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace dspark
