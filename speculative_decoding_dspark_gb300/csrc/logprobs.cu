// logprobs.cu -- log probabilities of given tokens, entropy and top alternatives
// of the target's rows.
//
// With t = x / T over the row's V logits x, m its largest x and s = sum exp(t - t_m):
//   lse = t_m + log s,  logprob = t_token - lse,  entropy = log s - sum (t - t_m) exp(t - t_m) / s
// in one pass with the running maximum and sums of each thread, joined at the end.
//
// The K best: a thread's largest value is one of the row's values, so whatever K
// of the threads' maxima reach, at least K values reach: a bound found by bisecting
// the values' bits until K maxima or few more reach it (one warp, the maxima in its
// registers).  In a cluster of C CTAs each finds the bounds that K / C and that K of its
// own maxima reach; the lowest of the former serves, or the highest of the latter
// if that is higher (a mask may leave a CTA nothing).  The pass leaves the maximum of every batch
// of 32 elements in shared memory; only batches whose maximum reaches the bound are
// read again (from L2, by as many threads as there are pieces), and the values that
// reach it, the candidates, are ranked by counting: the value falls, then the place
// rises.  A row with more candidates than the list holds (equal values in their
// hundreds) has its bound found by counting the values' bits from the top, and
// equal values taken in the order of their places.
#include <algorithm>

#include "kernels.cuh"
#include "rows.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 32;       // elements of a batch (a thread's, of as many pieces)
constexpr int kCandidates = 1024;
constexpr int kHits = 1024;
constexpr int kSms = 152;
constexpr int kMaxShared = 64 * 1024;

__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);  // (-0 is 0)
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float of_order(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ uint64_t rank_key(float x, int v) {
    return ((uint64_t)order_of(x) << 32) | (0xFFFFFFFFu - (uint32_t)v);
}

struct Shared {
    uint64_t cand[kCandidates];
    float maxima[kThreads];
    SoftSum part[kWarps];
    SoftSum row;      // this CTA's part of the row
    float bound;      // what at least K / C of its threads' maxima reach
    float own_bound;  // what at least K of them reach (C > 1)
    uint32_t n_cand;  // leader: candidates of all CTAs
    uint32_t n_hits;  // batches whose maximum reaches the bound
    uint32_t hits[kHits];
    uint32_t hist[256];
    uint32_t found;
    uint32_t count[kWarps];
    uint32_t prefix, need;
};

// (one warp) A value that at least `want` of the CTA's maxima reach, and not many
// more: found when at most a quarter more do, or when no bit is left.
__device__ __forceinline__ float bound_of(const float* maxima, int want) {
    uint32_t k[kWarps], low = 0xFFFFFFFFu, high = 0;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) {
        k[q] = order_of(maxima[q * 32 + (threadIdx.x & 31)]);
        low = min(low, k[q]);
        high = max(high, k[q]);
    }
    low = __reduce_min_sync(0xFFFFFFFFu, low);    // (all reach it)
    high = __reduce_max_sync(0xFFFFFFFFu, high) + 1;  // (none does)
    while (high - low > 1) {
        const uint32_t mid = low + (high - low) / 2;
        int n = 0;
#pragma unroll
        for (int q = 0; q < kWarps; ++q) n += k[q] >= mid;
        n = __reduce_add_sync(0xFFFFFFFFu, n);
        if (n >= want) {
            low = mid;
            if (n <= want + 1 + want / 4) break;
        } else {
            high = mid;
        }
    }
    return of_order(low);
}

// Leaves of a long list those that reach a bound which K of them do, and not many
// more (as bound_of, by all threads): ranking costs the square of the list's length.
__device__ __noinline__ void shorten(Shared& sh, int K) {
    constexpr int kEach = kCandidates / kThreads;
    const int tid = threadIdx.x, found = (int)sh.n_cand;
    uint64_t mine[kEach];
    uint32_t low = 0xFFFFFFFFu, high = 0;
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
        const int c = tid + q * kThreads;
        mine[q] = c < found ? sh.cand[c] : 0;  // (0: below every candidate)
        if (c < found) {
            low = min(low, (uint32_t)(mine[q] >> 32));
            high = max(high, (uint32_t)(mine[q] >> 32));
        }
    }
    low = __reduce_min_sync(0xFFFFFFFFu, low);
    high = __reduce_max_sync(0xFFFFFFFFu, high);
    if ((tid & 31) == 0) {
        sh.hist[tid >> 5] = low;
        sh.hist[kWarps + (tid >> 5)] = high;
    }
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) {
        low = min(low, sh.hist[w]);
        high = max(high, sh.hist[kWarps + w]);
    }
    ++high;
    while (high - low > 1) {
        const uint32_t mid = low + (high - low) / 2;
        int n = 0;
#pragma unroll
        for (int q = 0; q < kEach; ++q) n += (uint32_t)(mine[q] >> 32) >= mid;
        n = __reduce_add_sync(0xFFFFFFFFu, n);
        __syncthreads();
        if ((tid & 31) == 0) sh.count[tid >> 5] = (uint32_t)n;
        __syncthreads();
        n = 0;
        for (int w = 0; w < kWarps; ++w) n += (int)sh.count[w];
        if (n >= K) {
            low = mid;
            if (n <= K + 1 + K / 4) break;
        } else {
            high = mid;
        }
    }
    __syncthreads();
    if (tid == 0) sh.n_cand = 0;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kEach; ++q)
        if (mine[q] != 0 && (uint32_t)(mine[q] >> 32) >= low) sh.cand[atomicAdd(&sh.n_cand, 1u)] = mine[q];
    __syncthreads();
}

// The K best when the list was too short; leaves exactly K of them in sh.cand.
template <typename T>
__device__ __noinline__ void select_by_bits(const T* row, int V, int K, Shared& sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t prefix = 0, mask = 0, need = (uint32_t)K;
    for (int shift = 24; shift >= 0; shift -= 8) {
        sh.hist[tid] = 0;
        __syncthreads();
        uint32_t bin = 0, run = 0;  // equal neighbours are counted together
        for (int64_t v = tid; v < V; v += kThreads) {
            const float x = Elem<T>::to_float(row[v]);
            const uint32_t k = order_of(x);
            if (x == -INFINITY || (k & mask) != prefix) continue;
            const uint32_t b = (k >> shift) & 255u;
            if (run && b != bin) {
                atomicAdd(&sh.hist[bin], run);
                run = 0;
            }
            bin = b;
            ++run;
        }
        if (run) atomicAdd(&sh.hist[bin], run);
        __syncthreads();
        if (tid == 0) {
            uint32_t above = 0;
            int b = 255;
            while (b > 0 && above + sh.hist[b] < need) above += sh.hist[b--];
            sh.prefix = prefix | ((uint32_t)b << shift);
            sh.need = need - above;
        }
        __syncthreads();
        prefix = sh.prefix;
        need = sh.need;
        mask |= 255u << shift;
    }
    if (tid == 0) sh.n_cand = 0;
    __syncthreads();
    for (int64_t v = tid; v < V; v += kThreads) {
        const float x = Elem<T>::to_float(row[v]);
        if (order_of(x) > prefix) {
            const uint32_t at = atomicAdd(&sh.n_cand, 1u);
            if (at < (uint32_t)kCandidates) sh.cand[at] = rank_key(x, (int)v);
        }
    }
    __syncthreads();
    uint32_t taken = 0;
    for (int64_t v0 = 0; v0 < V && taken < need; v0 += kThreads) {
        const int64_t v = v0 + tid;
        const float x = v < V ? Elem<T>::to_float(row[v]) : -INFINITY;
        const bool here = v < V && order_of(x) == prefix;
        const uint32_t votes = __ballot_sync(0xFFFFFFFFu, here);
        if (lane == 0) sh.count[warp] = __popc(votes);
        __syncthreads();
        uint32_t before = taken, all = taken;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += sh.count[w];
            all += sh.count[w];
        }
        before += __popc(votes & ((1u << lane) - 1u));
        if (here && before < need) sh.cand[(uint32_t)K - need + before] = rank_key(x, (int)v);
        taken = all;
        __syncthreads();
    }
    if (tid == 0) sh.n_cand = (uint32_t)K;
    __syncthreads();
}

// One row's outputs, all of them the same value.
__device__ __forceinline__ void fill_row(const LogprobsParams& p, int64_t n, float value, float top_value) {
    if (threadIdx.x == 0) {
        if (p.logprob) p.logprob[n] = value;
        if (p.lse) p.lse[n] = value;
        if (p.entropy) p.entropy[n] = value;
    }
    for (int k = threadIdx.x; k < p.top_k; k += kThreads) {
        p.top_ids[n * p.top_k + k] = -1;
        p.top_logprobs[n * p.top_k + k] = top_value;
    }
}

template <typename T, bool kEntropy, bool kTop>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobsParams p) {
    constexpr int kVec = Elem<T>::kVec, kUnroll = kBatch / kVec;
    extern __shared__ float batch_max[];  // [batches of this CTA][thread]
    __shared__ Shared sh;
    static_assert(sizeof(Shared) + kSharedAnyway <= 48 * 1024, "what a launch may have without asking");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    // ---- which row, which token (the same for all CTAs of the cluster)
    const int64_t at = blockIdx.x / size;
    int64_t n = at;
    int token = p.tokens ? __ldg(p.tokens + at) : 0;
    if (p.cu) {
        const int r = (int)(at / p.width), j = (int)(at % p.width);
        const int a = p.cu[r], b = p.cu[r + 1];
        if (a < 0 || b < a || b > p.rows || (r == 0 && a != 0)) {
            if (tid == 0) report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
            return;
        }
        if (rank == 0 && j == p.width - 1)  // rows that no token can stand beside
            for (int64_t rest = (int64_t)a + p.width; rest < b; ++rest) fill_row(p, rest, 0.0f, -INFINITY);
        if (j >= b - a) return;
        n = a + j;
    }
    if (token < 0) {
        if (rank == 0) fill_row(p, n, 0.0f, -INFINITY);
        return;
    }
    if (token >= p.V) {
        if (rank == 0) {
            fill_row(p, n, NAN, NAN);
            if (tid == 0) report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
        }
        return;
    }
    if (!IN_BOUNDS(n >= 0 && n < p.rows, p.dev_status)) return;  // (the same for all CTAs of the cluster)
    const T* row = reinterpret_cast<const T*>(p.logits) + n * p.stride;
    const float x_token = Elem<T>::to_float(row[token]);
    const RowView<T> view(row, p.V);
    const int first = (int)(view.pieces * rank / size), end = (int)(view.pieces * (rank + 1) / size);
    if (kTop && tid == 0) sh.n_cand = sh.n_hits = 0;

    // ---- one pass over this CTA's pieces
    SoftSum t;
    int batch = 0;
    for (int i0 = first + tid; i0 - tid < end; i0 += kUnroll * kThreads, ++batch) {
        uint4 w[kUnroll];
#pragma unroll
        for (int q = 0; q < kUnroll; ++q) {
            const int i = i0 + q * kThreads;
            w[q] = load_piece<T>(view.base, i, end);
        }
        const float top = soft_add<T, kEntropy>(t, w, p.c2);
        if (kTop) batch_max[batch * kThreads + tid] = top;
    }
    const int v_edge = view.edge(tid, rank == 0, rank == size - 1);
    const float x_edge = v_edge >= 0 ? view.at(v_edge) : -INFINITY;
    soft_add_one<kEntropy>(t, x_edge, p.c2);
    if (kTop) sh.maxima[tid] = t.m;
    // ---- joined over the CTA
    {
        const SoftSum a = soft_join<kEntropy, 32>(t, p.c2);
        if (lane == 0) sh.part[warp] = a;
    }
    __syncthreads();
    if (warp == 0) {
        const SoftSum a = soft_join<kEntropy, kWarps>(lane < kWarps ? sh.part[lane] : SoftSum(), p.c2);
        if (lane == 0) sh.row = a;
    }
    if (kTop && warp == 1) {
        const float bound = bound_of(sh.maxima, (p.top_k + size - 1) / size);
        if (lane == 0) sh.bound = bound;
    }
    if (kTop && warp == 2 && size > 1) {
        const float bound = bound_of(sh.maxima, p.top_k);
        if (lane == 0) sh.own_bound = bound;
    }
    if (size > 1)
        cluster_sync();
    else
        __syncthreads();
    // ---- joined over the cluster, by its first CTA; the bound by all
    SoftSum all;
    if (rank == 0) {
        if ((uint32_t)lane < size) {
            const uint32_t a = cluster_map(&sh.row, lane);
            all.m = cluster_ld_f32(a + offsetof(SoftSum, m));
            all.s = cluster_ld_f32(a + offsetof(SoftSum, s));
            all.u = cluster_ld_f32(a + offsetof(SoftSum, u));
        }
        all = soft_join<kEntropy, 32>(all, p.c2);
    }
    if (kTop) {
        float bound = sh.bound;
        if (size > 1) {
            float own = -INFINITY;
            for (uint32_t c = 0; c < size; ++c) {
                bound = fminf(bound, cluster_ld_f32(cluster_map(&sh.bound, c)));
                own = fmaxf(own, cluster_ld_f32(cluster_map(&sh.own_bound, c)));
            }
            bound = fmaxf(bound, own);
        }
        const uint32_t list = cluster_map(sh.cand, 0), count = cluster_map(&sh.n_cand, 0);
        auto offer = [&](float x, int v) {
            const uint32_t c = size > 1 ? cluster_atomic_add(count, 1u) : atomicAdd(&sh.n_cand, 1u);
            if (c < (uint32_t)kCandidates) cluster_st_u64(list + 8 * c, rank_key(x, v));
        };
        if (x_edge >= bound && x_edge > -INFINITY) offer(x_edge, v_edge);
        if (t.m >= bound)
#pragma unroll 4
            for (int b = 0; b < batch; ++b) {
                const float top = batch_max[b * kThreads + tid];
                if (top >= bound && top > -INFINITY) {
                    const uint32_t h = atomicAdd(&sh.n_hits, 1u);
                    if (h < (uint32_t)kHits) sh.hits[h] = first + b * kUnroll * kThreads + tid;
                }
            }
        __syncthreads();
        const int n_hits = (int)sh.n_hits;
        if (n_hits > kHits) {  // (as many candidates, then)
            if (tid == 0) cluster_atomic_add(count, (uint32_t)kCandidates + 1);
        } else {
            for (int h = tid; h < n_hits * kUnroll; h += kThreads) {
                const int i = (int)sh.hits[h / kUnroll] + h % kUnroll * kThreads;
                if (i >= end || !IN_BOUNDS(i >= first, p.dev_status)) continue;
                const uint4 w = __ldcs(view.base + i);
                uint32_t reach = 0;
#pragma unroll
                for (int e = 0; e < kVec; e += 2) {
                    const float2 x = split(Elem<T>::pair(w, e / 2));
                    reach |= (x.x >= bound ? 1u << e : 0u) | (x.y >= bound ? 2u << e : 0u);
                }
                for (; reach; reach &= reach - 1) {
                    const int e = __ffs(reach) - 1;
                    const float x = Elem<T>::at(w, e);
                    if (x > -INFINITY) offer(x, view.head + i * kVec + e);
                }
            }
        }
        if (size > 1)
            cluster_sync();
        else
            __syncthreads();
    } else if (size > 1) {
        cluster_sync();
    }
    if (rank != 0) return;
    // ---- the row's outputs
    if (!(all.s > 0.0f && all.s < INFINITY) || all.m == INFINITY) {
        // a NaN or +inf in it, or nothing but -inf
        fill_row(p, n, NAN, NAN);
        if (tid == 0) report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
        return;
    }
    const float log_s = logf(all.s);
    if (tid == 0) {
        if (p.logprob) p.logprob[n] = p.tokens ? (x_token - all.m) * p.invT - log_s : 0.0f;
        if (p.lse) p.lse[n] = all.m * p.invT + log_s;
        if (kEntropy) p.entropy[n] = log_s - kLn2F * (all.u / all.s);
    }
    if (kTop) {
        if (sh.n_cand > (uint32_t)kCandidates)
            select_by_bits<T>(row, p.V, p.top_k, sh);
        else if (sh.n_cand > (uint32_t)(2 * p.top_k + 64))
            shorten(sh, p.top_k);
        const int found = (int)sh.n_cand;
        // four threads to a candidate, each against a quarter of the others
        for (int c0 = 0; c0 < found; c0 += kThreads / 4) {
            const int c = c0 + tid / 4;
            const uint64_t mine = c < found ? sh.cand[c] : 0;
            int place = 0;
#pragma unroll 4
            for (int o = tid & 3; o < found; o += 4) place += sh.cand[o] > mine;
            place += shfl_xor(place, 1);
            place += shfl_xor(place, 2);
            if ((tid & 3) == 0 && c < found && place < p.top_k) {
                p.top_ids[n * p.top_k + place] = (int32_t)(0xFFFFFFFFu - (uint32_t)mine);
                p.top_logprobs[n * p.top_k + place] = (of_order((uint32_t)(mine >> 32)) - all.m) * p.invT - log_s;
            }
        }
        for (int k = found + tid; k < p.top_k; k += kThreads) {
            p.top_ids[n * p.top_k + k] = -1;
            p.top_logprobs[n * p.top_k + k] = -INFINITY;
        }
    }
}

template <typename T>
const void* kernel_of(bool entropy, bool top) {
    return entropy ? (top ? (const void*)logprobs_kernel<T, true, true> : (const void*)logprobs_kernel<T, true, false>)
                   : (top ? (const void*)logprobs_kernel<T, false, true> : (const void*)logprobs_kernel<T, false, false>);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsParams& p, cudaStream_t stream) {
    const int vec = p.dtype == DSPARK_F32 ? 4 : 8;
    const int64_t places = p.cu ? (int64_t)p.R * p.width : p.rows;
    int ctas = 1;
    const int64_t pieces = p.V / vec;
    auto smem_of = [&](int c) {
        const int64_t per = (pieces + c - 1) / c;
        return (size_t)(p.top_k ? (per * vec + kBatch * kThreads - 1) / (kBatch * kThreads) * kThreads * sizeof(float) : 0);
    };
    // Rows are shared by more CTAs until there are eight to an SM, as long as a CTA keeps 4096 pieces, or 1024 where an SM
    // would have none.  One, two, four and eight CTAs to a row, us: 15.5, 10.7, 7.6 and 6.9 for one row of 151936 fp32; 128, 143, 172
    // and 257 for 2560 rows of 129280 bf16; 15.4, 16.5, 21.4 and 35 for 333 rows of 50001 bf16.  Beside cu_seqlens the
    // places count, of which the kernel alone knows how many have a row and are asked for: 41.6, 48.3, 48.4 and 63.6 for 349 rows of 151936
    // fp32 in 1024 places (two by this rule; with the places held to the 544 rows there are it would be four), 36.9, 24.9, 27.1 and
    // 32.9 for those of 512 places (four), 27.0, 20.0, 15.9 and 17.3 for those of 256 (eight).
    auto larger = [&](int c) {
        return smem_of(c) > 48 * 1024 || (places * c < 8 * kSms && pieces / (2 * c) >= (places * c < kSms ? 1024 : 4096));
    };
    while (ctas < 8 && larger(ctas)) ctas *= 2;
    const size_t smem = smem_of(ctas);
    const void* fn = p.dtype == DSPARK_F32 ? kernel_of<float>(p.entropy, p.top_k > 0)
                                           : kernel_of<uint16_t>(p.entropy, p.top_k > 0);
    // (the same limit in every call that sets it: two host threads may call at once)
    cudaError_t e = cudaSuccess;
    if (smem > kSharedAnyway) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared);
    static_assert(DSPARK_ROWS_MAX_V / 8 / (kBatch * kThreads) * kThreads * sizeof(float) <= kMaxShared, "the longest row's maxima");
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(places * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {const_cast<LogprobsParams*>(&p)};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace dspark
