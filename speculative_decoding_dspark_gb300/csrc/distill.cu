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
// of its own keeps the listed tokens and does all that is done once per row.
#include <algorithm>

#include "kernels.cuh"
#include "rows.cuh"
#include "tc_ptx.cuh"

namespace dspark {
namespace {

// kThreads walk through the rows, and a warp more keeps the listed tokens: the large CTA,
// or the small one where a row has few pieces and what is done once per row counts.
constexpr int kLarge = 256, kSmall = 64;
constexpr int kUnroll = 4;     // pieces of a batch
constexpr int kMaxCtas = 8;    // of a cluster
constexpr int kPerLane = DSPARK_TOP_MAX / 32;
// Rows of at most this many pieces take the small CTA, of which nine fit on an SM.  4096 rows, 64 tokens, bf16 gradient, large
// and small, us: of 500, 4096, 8192 and 16384 fp32 43 and 20, 46 and 30, 54 and 57, 77 and 133; of 4096, 16384 and 32000
// bf16 50 and 27, 69 and 75, 105 and 174.
constexpr int kSmallPieces = 1792;

// What is known of a row's listed tokens before its sums are.  (Sixteen bytes, one load: with a fifth word 896 rows of
// 151936 fp32 took 183 us instead of 170.)
struct Kept {
    float x_top, e_sum;  // the largest logit, the sum of 2^((x - x_top) c2)
    float mass;          // the teacher's: the sum of p, or, as a negative number, what that leaves to the rest as a class
    float bad;
};

// A row's listed tokens.  (In shared memory: held by the lanes, 24 registers, they kept every
// thread of the kernel above 72, at which three CTAs fit on an SM.)
struct Listed {
    int id[DSPARK_TOP_MAX];      // -1: none
    float x[DSPARK_TOP_MAX];     // the drafter's logit
    float value[DSPARK_TOP_MAX];
    float p[DSPARK_TOP_MAX];     // exp(value - its reference)
};

template <int kThreads>
struct Shared {
    Listed list[2];                    // by the row's parity
    float2 sums[2][kMaxCtas][kThreads / 32];  // (m, s) of all warps of the cluster, by the row's parity
    float bad[2][kMaxCtas];            // whether a CTA found fault with the listed tokens
    Kept kept[2];
    uint32_t marked[kThreads];         // which batches of a thread hold listed tokens (bit 31: the 32nd or a later one)
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

// (a warp) What the listed tokens leave of a teacher's probability.  What its surest token leaves is 1 - p of it, whose
// bits 1 - (a sum in 32 bits) would lose where that token has nearly all; from that the sum of the others.  In 32 bits
// the difference is off by 13 u of what the surest token leaves (u = 2^-24: expm1f and expf 2 u each, eight sums, the
// difference itself): up to 1e-3 of itself where it is not below kLittle of that; below, it is taken in 64 bits.  (In
// 64 bits always, with 64 tokens, us: 4096 rows of 500 fp32 28 instead of 20, 2000 of 32000 82 instead of 72, 896 of
// 151936 174 instead of 170.)
constexpr float kLittle = 1.0f / 1024;
__device__ __noinline__ float little_left(const float* value, int n) {
    double s = 0.0;
    for (int k = threadIdx.x & 31; k < n; k += 32)
        if (value[k] > -INFINITY) s += exp((double)value[k]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    return (float)fmax(1.0 - s, 0.0);
}
__device__ __forceinline__ float left_of(float top, float others, const float* value, int n) {
    const float beside = -expm1f(top), left = beside - others;
    if (fabsf(left) < kLittle * beside) return little_left(value, n);
    return fmaxf(left, 0.0f);
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

// This CTA's share of a gradient row of weight 0.
template <typename G, int kAllThreads>
__device__ __forceinline__ void clear_grad(G* g, int V, int rank, int size) {
    constexpr int kVec = 16 / sizeof(G);
    const int head = min(V, (int)(((16 - (reinterpret_cast<uintptr_t>(g) & 15)) & 15) / sizeof(G)));
    const int pieces = (V - head) / kVec, first = pieces * rank / size, end = pieces * (rank + 1) / size;
    uint4* wide = reinterpret_cast<uint4*>(g + head);
    for (int i = first + threadIdx.x; i < end; i += kAllThreads) __stcs(wide + i, make_uint4(0, 0, 0, 0));
    if (rank == 0 && (int)threadIdx.x < head) g[threadIdx.x] = G(0);
    const int tail = head + pieces * kVec + (int)threadIdx.x;
    if (rank == size - 1 && tail < V) g[tail] = G(0);
}

__device__ __forceinline__ void copy_word(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
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
    __device__ __forceinline__ Share(const DistillParams& p, int64_t row, int rank)
        : view(reinterpret_cast<const T*>(p.student) + row * p.stride, p.V) {
        first = view.pieces * rank >> p.log_ctas;
        const int end = view.pieces * (rank + 1) >> p.log_ctas;
        n = end - first;
        v0 = rank == 0 ? 0 : view.head + first * Elem<T>::kVec;
        v1 = rank + 1 == 1 << p.log_ctas ? p.V : view.head + end * Elem<T>::kVec;
    }
    __device__ __forceinline__ const uint4* pieces() const { return view.base + first; }
    // The bit of its element v (a word is kept for the edges on either side).
    __device__ __forceinline__ int bit(int v) const { return v - view.head - first * Elem<T>::kVec + 32; }
};

// T: the logits' elements, G: the gradient's, kGrad: there is one.
template <typename T, typename G, bool kGrad, int kThreads>
__global__ void __launch_bounds__(kThreads + 32, kThreads == kLarge ? 3 : 9) distill_kernel(const DistillParams p) {
    constexpr int kVec = Elem<T>::kVec, kWarps = kThreads / 32, kAllThreads = kThreads + 32;
    constexpr int kBatch = kUnroll * kThreads;  // pieces
    extern __shared__ uint4 dyn[];
    __shared__ Shared<kThreads> sh;
    static_assert(sizeof(Shared<kThreads>) + kSharedAnyway <= 48 * 1024, "what a launch may have without asking");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool keeper = warp == kWarps;
    const int rank = (int)cluster_rank(), size = 1 << p.log_ctas;
    const int clusters = gridDim.x >> p.log_ctas;
    cluster_arrive();  // (this CTA has started: the others may write to its shared memory once all have)
    uint4* stage = dyn + tid;  // [p.staged batches][kUnroll][kThreads]
    uint32_t* bits = reinterpret_cast<uint32_t*>(dyn + p.staged * kBatch);
    for (int i = tid; i < p.bit_words; i += kAllThreads) bits[i] = 0;
    if (tid < kThreads) sh.marked[tid] = 0;

    auto weight_of = [&](int64_t n) { return p.weight && n < p.rows ? __ldg(p.weight + n) : 1.0f; };
    // The next row from n on that has a weight; those that have none are done with.
    auto active = [&](int64_t n, float& w) {
        while (n < p.rows && w == 0.0f) {
            if (kGrad) clear_grad<G, kAllThreads>(reinterpret_cast<G*>(p.grad) + n * p.grad_stride, p.V, rank, size);
            if (rank == 0 && tid == 0) p.loss[n] = 0.0f;
            n += clusters;
            w = weight_of(n);
        }
        return n;
    };
    auto copy_batch = [&](const uint4* from, int n, int b) {  // of a row's n pieces from `from` on
        const uint32_t to = tc::smem_u32(stage + b * kBatch);
        const int left = n - b * kBatch - tid;
        from += b * kBatch + tid;
        if (left > (kUnroll - 1) * kThreads) {
#pragma unroll
            for (int q = 0; q < kUnroll; ++q) tc::cp_async_16(to + q * kThreads * 16, from + q * kThreads, 16);
        } else {
#pragma unroll
            for (int q = 0; q < kUnroll; ++q)
                if (q * kThreads < left) tc::cp_async_16(to + q * kThreads * 16, from + q * kThreads, 16);
        }
        tc::cp_async_commit();
    };
    // (keeper) a row's listed tokens and their values on their way
    const int n_list = (p.top_k + 31) / 32 * 32;
    auto fetch = [&](int64_t n, Listed& t) {
        for (int k = lane; k < p.top_k; k += 32) {
            copy_word(&t.id[k], p.ids + n * p.top_k + k);
            copy_word(&t.value[k], p.teacher + n * p.top_k + k);
        }
        tc::cp_async_commit();
    };
    auto fetched = [&](Listed& t) {
        tc::cp_async_wait<0>();
        for (int k = lane; k < n_list; k += 32) {
            if (k >= p.top_k) t.id[k] = -1;
            if (t.id[k] < 0) t.value[k] = -INFINITY;
        }
        __syncwarp();
    };
    // (keeper) marks a row's listed tokens; whether something is wrong with them
    auto mark = [&](const Share<T>& s, const Listed& t) {
        bool bad = false;
        for (int k = lane; k < n_list; k += 32) {
            const int id = t.id[k];
            bad |= id >= p.V || t.value[k] != t.value[k] || t.value[k] == INFINITY;
            if (id >= s.v0 && id < s.v1) {
                const int b = s.bit(id), piece = (b - 32) / kVec;
                if (!IN_BOUNDS(b >= 0 && b >> 5 < p.bit_words, p.dev_status)) continue;
                bad |= (atomicOr(&bits[b >> 5], 1u << (b & 31)) >> (b & 31) & 1u) != 0;  // listed twice
                if (b >= 32 && piece < s.n) atomicOr(&sh.marked[piece % kThreads], 1u << min(piece / kBatch, 31));
            }
        }
        return __any_sync(0xFFFFFFFFu, bad);
    };
    auto unmark = [&](const Share<T>& s, const Listed& t) {
        for (int k = lane; k < n_list; k += 32)
            if (t.id[k] >= s.v0 && t.id[k] < s.v1) {
                const int b = s.bit(t.id[k]), piece = (b - 32) / kVec;
                if (!IN_BOUNDS(b >= 0 && b >> 5 < p.bit_words, p.dev_status)) continue;
                bits[b >> 5] = 0;
                if (b >= 32 && piece < s.n) sh.marked[piece % kThreads] = 0;
            }
        __syncwarp();
    };

    // The row's sums over the cluster (every warp by itself; the lanes agree).
    struct Joined {
        SoftSum rest;              // the tokens that are not listed
        float m_all, f_rest, f_listed, total, p_rest, all_mass;
        float m_ref, factor;       // the gradient of a token that is not listed: factor 2^((x - m_ref) c2)
        bool bad;
    };
    auto joined = [&](int parity, float weight) {
        Joined j;
        const Kept kept = sh.kept[parity];
        constexpr int kEach = (kMaxCtas * kWarps + 31) / 32;
        SoftSum each[kEach], t;
        const int n_sums = size * kWarps;
#pragma unroll
        for (int q = 0; q < kEach; ++q) {
            const int at = lane + 32 * q;
            if (at < n_sums) {
                const float2 a = sh.sums[parity][at / kWarps][at % kWarps];
                each[q].m = a.x;
                each[q].s = a.y;
            }
            t.m = fmaxf(t.m, each[q].m);
        }
#pragma unroll
        for (int q = 0; q < kEach; ++q)
            t.s += each[q].m == -INFINITY ? each[q].s : each[q].s * exp2_approx((each[q].m - t.m) * p.c2);
        j.rest = soft_join<false, 32>(t, p.c2);
        const float bad_there = lane < size ? sh.bad[parity][lane] : 0.0f;
        j.m_all = fmaxf(kept.x_top, j.rest.m);
        j.f_rest = j.rest.m > -INFINITY ? exp2_approx((j.rest.m - j.m_all) * p.c2) : 0.0f;
        j.f_listed = kept.x_top > -INFINITY ? exp2_approx((kept.x_top - j.m_all) * p.c2) : 0.0f;
        j.total = kept.e_sum * j.f_listed + j.rest.s * j.f_rest;
        j.bad = __any_sync(0xFFFFFFFFu, bad_there != 0.0f) || kept.bad != 0.0f || !(j.total > 0.0f && j.total < INFINITY) ||
                j.m_all == INFINITY || j.rest.s != j.rest.s;
        const bool none = j.rest.m == -INFINITY;  // (what is not listed is -inf alone: no class of the rest)
        j.p_rest = none ? 0.0f : fmaxf(-kept.mass, 0.0f);
        j.all_mass = kept.mass < 0.0f ? (none ? 1.0f + kept.mass : 1.0f) : kept.mass;
        j.m_ref = none ? 0.0f : j.rest.m;
        j.factor = j.bad ? NAN
                   : none ? 0.0f
                          : weight * p.invT * (__fdividef(j.all_mass * j.f_rest, j.total) - (j.p_rest > 0.0f ? __fdividef(j.p_rest, j.rest.s) : 0.0f));
        return j;
    };

    int64_t row = blockIdx.x >> p.log_ctas;
    float weight = weight_of(row);
    row = active(row, weight);
    float ahead = weight_of(row + clusters);
    bool bad_list = false;
    __syncthreads();
    if (row < p.rows) {
        const Share<T> s(p, row, rank);
        if (keeper) {
            fetch(row, sh.list[0]);
            fetched(sh.list[0]);
            bad_list = mark(s, sh.list[0]);
        } else if (kGrad) {
            for (int b = 0; b < p.staged; ++b) copy_batch(s.pieces(), s.n, b);
        }
    }
    __syncthreads();
    cluster_wait();  // (over by now: the first row's copies are on their way)

    Share<T> s(p, min(row, (int64_t)p.rows - 1), rank);
    for (int parity = 0; row < p.rows; parity ^= 1) {
        float next_weight = ahead;
        const int64_t next = active(row + clusters, next_weight);
        ahead = weight_of(next + clusters);
        const bool more = next < p.rows;
        const Share<T> after(p, more ? next : row, rank);
        if (!keeper) {
            const int n_batches = (s.n + kBatch - 1) / kBatch;
            const int v_edge = warp == 0 ? s.view.edge(lane, rank == 0, rank == size - 1) : -1;
            const float x_edge = v_edge >= 0 ? s.view.at(v_edge) : -INFINITY;
            const uint32_t marked = sh.marked[tid];
            // ---- first pass: the tokens that are not listed
            SoftSum t;
            auto add_batch = [&](uint4 (&w)[kUnroll], int b) {
                if (marked >> min(b, 31) & 1u) {
#pragma unroll
                    for (int q = 0; q < kUnroll; ++q) {
                        const int at = (b * kBatch + q * kThreads + tid) * kVec;
                        if (at < s.n * kVec) w[q] = Elem<T>::without(w[q], bits[1 + (at >> 5)] >> (at & 31));
                    }
                }
                soft_add<T, false>(t, w, p.c2);
            };
            const int half = p.staged / 2;  // (two waits a row: one for each batch cost 2 %)
            for (int b = 0; b < n_batches; ++b) {
                constexpr uint32_t k = Elem<T>::kMinusInf;
                const int left = s.n - b * kBatch - tid;
                uint4 w[kUnroll];
                if (kGrad && b < p.staged) {
                    if (b == 0)
                        copies_left(half);
                    else if (b == p.staged - half)
                        copies_left(0);
                    if (left > (kUnroll - 1) * kThreads) {
#pragma unroll
                        for (int q = 0; q < kUnroll; ++q) w[q] = stage[b * kBatch + q * kThreads];
                    } else {
#pragma unroll
                        for (int q = 0; q < kUnroll; ++q)
                            w[q] = q * kThreads < left ? stage[b * kBatch + q * kThreads] : make_uint4(k, k, k, k);
                    }
                } else {
                    const uint4* from = s.pieces() + b * kBatch + tid;
#pragma unroll
                    for (int q = 0; q < kUnroll; ++q)
                        w[q] = q * kThreads < left ? __ldcs(from + q * kThreads) : make_uint4(k, k, k, k);
                }
                add_batch(w, b);
            }
            if (v_edge >= 0) {
                const int b = s.bit(v_edge);
                if (!(bits[b >> 5] >> (b & 31) & 1u)) soft_add_one<false>(t, x_edge, p.c2);
            }
            __syncwarp();
            // ---- to all CTAs of the cluster
            t = soft_join<false, 32>(t, p.c2);
            if (lane < size) cluster_st_f32x2(cluster_map(&sh.sums[parity][rank][warp], lane), t.m, t.s);
            __syncwarp();
            cluster_arrive();
            cluster_wait();
            // ---- second pass: the gradient; the next row's pieces follow this one's
            if (kGrad) {
                G* grad = reinterpret_cast<G*>(p.grad) + row * p.grad_stride;
                const Joined j = joined(parity, weight);
                const float m_ref = j.m_ref, factor = j.factor;
                const Two scale = two(p.c2, p.c2), f2 = two(factor, factor), minus = two(-m_ref, -m_ref);
                G* out = grad + s.view.head + (int64_t)s.first * kVec;
                const uint4* next_pieces = after.pieces();
                const bool wide = reinterpret_cast<uintptr_t>(out) % (kVec * sizeof(G) < 16 ? kVec * sizeof(G) : 16) == 0;
                const int all_batches = more ? max(n_batches, p.staged) : n_batches;
                auto write = [&](const uint4& w, G* to, bool whole) {
                    float x[kVec];
#pragma unroll
                    for (int e = 0; e < kVec; e += 2) {
                        const float2 a = split(mul_two(add_two(Elem<T>::pair(w, e / 2), minus), scale));
                        const float2 g = split(mul_two(two(exp2_approx(a.x), exp2_approx(a.y)), f2));
                        x[e] = g.x;
                        x[e + 1] = g.y;
                    }
                    if (whole) {
                        store_piece(to, x);
                    } else {
#pragma unroll
                        for (int e = 0; e < kVec; ++e) to[e] = grad_of<G>(x[e]);
                    }
                };
                for (int b = 0; b < all_batches; ++b) {
                    const int i0 = b * kBatch + tid, left = s.n - i0;
                    G* to = out + (int64_t)i0 * kVec;
                    uint4 w[kUnroll];
                    if (wide && left > (kUnroll - 1) * kThreads && b < p.staged) {
#pragma unroll
                        for (int q = 0; q < kUnroll; ++q) w[q] = stage[b * kBatch + q * kThreads];
#pragma unroll
                        for (int q = 0; q < kUnroll; ++q) write(w[q], to + q * kThreads * kVec, true);
                    } else {
#pragma unroll
                        for (int q = 0; q < kUnroll; ++q)
                            if (q * kThreads < left)
                                w[q] = b < p.staged ? stage[b * kBatch + q * kThreads] : __ldcs(s.pieces() + i0 + q * kThreads);
#pragma unroll
                        for (int q = 0; q < kUnroll; ++q)
                            if (q * kThreads < left) write(w[q], to + q * kThreads * kVec, wide);
                    }
                    if (more && b < p.staged) copy_batch(next_pieces, after.n, b);
                }
                if (v_edge >= 0) grad[v_edge] = grad_of<G>(factor * exp2_approx((x_edge - m_ref) * p.c2));
            }
            __syncthreads();  // the gradient is written, the next row's tokens are marked
        } else {
            // ---- the keeper: what does not wait for this row's sums
            Listed &now = sh.list[parity], &then = sh.list[parity ^ 1];
            if (more) fetch(next, then);
            const T* student = reinterpret_cast<const T*>(p.student) + row * p.stride;
            float x[kPerLane], x_top = -INFINITY, v_top = -INFINITY;
#pragma unroll
            for (int q = 0; q < kPerLane; ++q) {
                const int id = 32 * q < n_list ? now.id[lane + 32 * q] : -1;
                x[q] = id >= 0 && id < p.V ? Elem<T>::to_float(student[id]) : -INFINITY;
            }
#pragma unroll
            for (int q = 0; q < kPerLane; ++q) {
                now.x[lane + 32 * q] = x[q];
                bad_list |= x[q] != x[q];
                x_top = fmaxf(x_top, x[q]);
                if (32 * q < n_list) v_top = fmaxf(v_top, now.value[lane + 32 * q]);
            }
            bad_list = __any_sync(0xFFFFFFFFu, bad_list);
            x_top = warp_max(x_top);
            const float v_lane = v_top;
            v_top = warp_max(v_top);  // (a list of -inf alone has no mass)
            const bool surest = lane == __ffs(__ballot_sync(0xFFFFFFFFu, v_lane == v_top)) - 1;
            const float ref = p.rest ? 0.0f : v_top;
            float others = 0.0f, e_sum = 0.0f;
            bool skip = surest;  // (of equal ones, one)
            for (int k = lane; k < n_list; k += 32) {
                const float value = now.value[k], prob = value > -INFINITY ? expf(value - ref) : 0.0f;
                now.p[k] = prob;
                if (skip && value == v_top)
                    skip = false;
                else
                    others += prob;
                if (now.x[k] > -INFINITY) e_sum += exp2_approx((now.x[k] - x_top) * p.c2);
            }
            others = warp_sum(others);
            e_sum = warp_sum(e_sum);
            float mass = others + (v_top > -INFINITY ? expf(v_top - ref) : 0.0f);
            float scale = 1.0f, log_scale = 0.0f;
            const float left = p.rest ? left_of(v_top, others, now.value, n_list) : 0.0f;
            const bool bad_row = !(fabsf(weight) < INFINITY) || !(mass < INFINITY);
            if (!p.rest && mass > 0.0f) {
                scale = 1.0f / mass;
                log_scale = -ref - logf(mass);
                mass = 1.0f;  // (nothing listed: nothing to learn from)
            }
            if (lane == 0) {
                Kept k;
                k.x_top = x_top;
                k.e_sum = e_sum;
                k.mass = left > 0.0f ? -left : mass;
                k.bad = bad_row ? 1.0f : 0.0f;
                sh.kept[parity] = k;
            }
            if (lane < size) cluster_st_f32(cluster_map(&sh.bad[parity][rank], lane), bad_list ? 1.0f : 0.0f);
            __syncwarp();
            cluster_arrive();
            cluster_wait();
            const Joined j = joined(parity, weight);
            const float w = weight * p.invT;
            unmark(s, now);
            if (more) {
                fetched(then);
                bad_list = mark(after, then);
            }
            __syncthreads();
            if (rank == 0) {
                const float log_total = logf(j.total);
                float term = 0.0f;
                for (int k = lane; k < n_list; k += 32)
                    if (now.p[k] > 0.0f)
                        term += now.p[k] * scale *
                                ((now.value[k] + log_scale) - ((now.x[k] - j.m_all) * p.invT - log_total));
                term = warp_sum(term);
                if (j.p_rest > 0.0f)
                    term += j.p_rest * (logf(j.p_rest) - ((j.rest.m - j.m_all) * p.invT + logf(j.rest.s) - log_total));
                if (lane == 0) {
                    p.loss[row] = j.bad ? NAN : weight * term;
                    if (j.bad) report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
                }
            }
            // the listed tokens' own gradients over those of the second pass
            if (kGrad && !j.bad) {
                G* grad = reinterpret_cast<G*>(p.grad) + row * p.grad_stride;
                const float of_x = j.all_mass * j.f_listed / j.total;
                for (int k = lane; k < n_list; k += 32) {
                    const int id = now.id[k];
                    if (id < s.v0 || id >= s.v1) continue;
                    const float e = now.x[k] > -INFINITY ? exp2_approx((now.x[k] - x_top) * p.c2) : 0.0f;
                    grad[id] = grad_of<G>(w * (of_x * e - now.p[k] * scale));
                }
                __syncwarp();
            }
        }
        row = next;
        weight = next_weight;
        s = after;
    }
    cluster_sync();  // (no CTA ends while another may still write to its shared memory)
}

template <typename T, int kThreads>
const void* kernel_of(bool grad, int grad_dtype) {
    if (!grad) return (const void*)distill_kernel<T, float, false, kThreads>;
    return grad_dtype == DSPARK_F32 ? (const void*)distill_kernel<T, float, true, kThreads>
                                    : (const void*)distill_kernel<T, uint16_t, true, kThreads>;
}
template <typename T>
const void* kernel_of(bool grad, int grad_dtype, bool small) {
    return small ? kernel_of<T, kSmall>(grad, grad_dtype) : kernel_of<T, kLarge>(grad, grad_dtype);
}

}  // namespace

cudaError_t launch_distill(DistillParams p, cudaStream_t stream) {
    const int vec = p.dtype == DSPARK_F32 ? 4 : 8;
    const int64_t pieces = p.V / vec;
    const bool small = pieces <= kSmallPieces;
    const int threads = small ? kSmall : kLarge;
    // Shared memory of a CTA, so that three large ones fit on an SM (a row's last batch is read again then, of 151936 fp32
    // over eight CTAs the fifth).  Three with all but that, two with all of it: 170 and 174 us for 896 rows of 151936 fp32.
    constexpr size_t kShare = 68 * 1024;
    int ctas = 1;
    auto batches_of = [&](int c) { return (int)(((pieces + c - 1) / c + kUnroll * threads - 1) / (kUnroll * threads)); };
    auto bits_of = [&](int c) { return (int)(((pieces + c - 1) / c * vec + 31) / 32 + 2); };
    auto smem_of = [&](int c, int batches) { return (size_t)batches * kUnroll * threads * 16 + (size_t)bits_of(c) * 4; };
    auto larger = [&](int c) {
        return smem_of(c, p.grad ? batches_of(c) : 0) > kShare || ((int64_t)p.rows * c < 152 && pieces / c > 2 * kLarge);
    };
    while (ctas < kMaxCtas && larger(ctas)) ctas *= 2;
    p.staged = p.grad ? std::min<int64_t>(batches_of(ctas), (int64_t)((kShare - std::min(kShare, smem_of(ctas, 0))) / (kUnroll * threads * 16))) : 0;
    p.bit_words = bits_of(ctas);
    p.log_ctas = ctas == 1 ? 0 : ctas == 2 ? 1 : ctas == 4 ? 2 : 3;
    const size_t smem = smem_of(ctas, p.staged);
    const void* fn = p.dtype == DSPARK_F32 ? kernel_of<float>(p.grad != nullptr, p.grad_dtype, small)
                                           : kernel_of<uint16_t>(p.grad != nullptr, p.grad_dtype, small);
    // (the same limit in every call that sets it: two host threads may call at once)
    cudaError_t e = cudaSuccess;
    if (smem > kSharedAnyway) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kShare);
    static_assert(DSPARK_ROWS_MAX_V / 8 / 8 + 64 <= kShare, "the longest row's bits");
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(threads + 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // As many clusters as there is room for at a time: they walk down the rows.  Few rows need no asking (0.2 us).
    cfg.gridDim = dim3((unsigned)ctas);
    int room = p.rows;
    if (p.rows > 8 && (e = cudaOccupancyMaxActiveClusters(&room, fn, &cfg)) != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(std::min(p.rows, std::max(1, room)) * ctas));
    void* args[] = {&p};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace dspark
