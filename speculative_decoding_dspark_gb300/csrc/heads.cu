// heads.cu -- the query, key and value heads of packed rows on their way into
// attention: RMS norm of every head, position rotation, and the write into the
// paged KV cache.
//
// For one head x[0 .. d) of a row at position pos:
//   y_i = x_i * rsqrt(mean_j x_j^2 + eps) * w_i             (no weight: y = x)
//   (y_a, y_b) <- (y_a c_f - y_b s_f, y_b c_f + y_a s_f),  c_f + i s_f = e^{i pos inv_freq_f}
// over the pairs (f, f + rot/2) or (2f, 2f + 1), f < rot/2; the rest of the
// head is left as it is.  Queries go to q_out, keys to k_out or to page
// block_table[r][pos / P], slot pos % P of the cache, values (append only) to
// the cache unchanged.
//
// Everything is held in fp32 and rounded once at the store.  The angle is
// formed in fp64: at position 500000 an fp32 product is off by 0.03 rad.  It is
// counted in turns, pos * inv_freq / (2 pi), so that taking off whole turns is
// exact and the fp32 sine and cosine see an argument of half a turn at most.
//
// What bounds it: bytes (each input element read once, each output written
// once).  A head is read by d / 8 lanes, eight elements (16 or 32 bytes) each,
// and its pairs meet by a shuffle, so nothing passes through shared memory but
// the row's rot/2 cosines and sines, which all of its heads share (fp64 runs at
// a sixty-fourth of the fp32 rate: one angle per row and pair, not per head).
#include "kernels.cuh"

namespace dspark {
namespace {

constexpr int kHeadThreads = 512;  // most threads of a CTA
constexpr int kHeadUnroll = 2;     // heads a lane group holds in registers at once
constexpr int kHeadRows = 8;       // most rows of a CTA

struct RowPlace {     // where a row's keys and values go
    long long page;   // page id, -1: the row is bad or past the last request
    int slot;         // row of the page
    int state;        // 0 write, 1 leave untouched, 2 bad input: outputs are NaN
};

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
    __nv_bfloat162 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
}

template <typename TIn, typename TOut, bool kPairs, bool kAppend>
__global__ void __launch_bounds__(kHeadThreads) heads_kernel(const HeadsParams p, int rows_per_cta, int lanes) {
    extern __shared__ float2 turn_smem[];  // [rows_per_cta][rot / 2] cosine, sine
    __shared__ RowPlace place[kHeadRows];
    const int half = p.rot / 2;
    const int row0 = blockIdx.x * rows_per_cta;
    const int rows = min(rows_per_cta, p.rows - row0);
    const int n_heads = p.hq + (kAppend ? 2 : 1) * p.hkv;
    const int sub = threadIdx.x % lanes, group = threadIdx.x / lanes, n_groups = blockDim.x / lanes;
    const bool active = 8 * sub < p.d;
    const int items = rows * n_heads;

    auto source = [&](int item) -> const TIn* {
        const int row = row0 + item / n_heads, h = item % n_heads;
        if (h < p.hq) return static_cast<const TIn*>(p.q) + row * p.q_stride + (long long)h * p.d;
        if (h < p.hq + p.hkv) return static_cast<const TIn*>(p.k) + row * p.k_stride + (long long)(h - p.hq) * p.d;
        return static_cast<const TIn*>(p.v) + row * p.v_stride + (long long)(h - p.hq - p.hkv) * p.d;
    };
    float x[kHeadUnroll][8];
    auto fetch = [&](int base) {
#pragma unroll
        for (int u = 0; u < kHeadUnroll; ++u) {
            const int item = base + u * n_groups;
            if (active && item < items) {
                load8(source(item) + 8 * sub, x[u]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[u][e] = 0.0f;
            }
        }
    };
    fetch(group);  // in flight while the angles are formed

    // each warp takes rows in turn: where the row goes, and its angles
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n_warps = blockDim.x >> 5;
    for (int i = warp; i < rows; i += n_warps) {
        const int row = row0 + i;
        long long pos = 0;
        RowPlace at{-1, 0, 0};
        if (kAppend) {
            const int r = owner_of(p.cu, p.R, row);
            const int lo = p.cu[r], hi = p.cu[r + 1], len = p.kv_len[r];
            if (row == 0 && lane == 0 && (p.cu[0] != 0 || p.cu[p.R] > p.rows || p.cu[p.R] < 0))
                report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
            if (row < lo || row >= hi) {
                at.state = row >= p.cu[p.R] ? 1 : 2;
            } else {
                pos = (long long)len + (row - lo);
                const long long b = pos / p.page;
                at.slot = (int)(pos - b * p.page);
                if (len < 0 || lo < 0 || b >= p.max_blocks) at.state = 2;
                else at.page = p.block_table[(long long)r * p.max_blocks + b];
                if (at.page < 0 || at.page >= p.pool_pages) at.state = 2;
            }
            if (at.state == 2 && lane == 0) report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
        } else if (half > 0) {
            pos = p.positions[row];
            if (pos < 0) {
                at.state = 2;
                if (lane == 0) report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
            }
        }
        if (lane == 0) place[i] = at;
        for (int f = lane; f < half; f += 32) {
            const double turns = (double)pos * (double)p.inv_freq[f] * 0.15915494309189533577;  // 1 / (2 pi)
            float s, c;
            sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
            turn_smem[i * half + f] = make_float2(c, s);
        }
    }
    __syncthreads();

    for (int base = group;; base += kHeadUnroll * n_groups) {
#pragma unroll
        for (int u = 0; u < kHeadUnroll; ++u) {
            const int item = base + u * n_groups;  // (groups past the end take part in the shuffles)
            const int i = item < items ? item / n_heads : 0, h = item < items ? item % n_heads : 0;
            const bool is_q = h < p.hq, is_v = h >= p.hq + p.hkv;
            const void* weight = is_q ? p.wq : p.wk;
            const bool norm = !is_v && weight != nullptr;
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[u][e], x[u][e], ss);
            for (int o = lanes >> 1; o; o >>= 1) ss += shfl_xor(ss, o);
            if (norm && active) {
                const float r = rsqrtf(ss / (float)p.d + p.eps);
                float w[8];
                load8(static_cast<const TIn*>(weight) + 8 * sub, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[u][e] = x[u][e] * r * w[e];
            }
            const bool turned = !is_v && 8 * sub < p.rot;
            if (kPairs) {
                if (turned) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 cs = turn_smem[i * half + 4 * sub + e];
                        const float a = x[u][2 * e], b = x[u][2 * e + 1];
                        x[u][2 * e] = a * cs.x - b * cs.y;
                        x[u][2 * e + 1] = b * cs.x + a * cs.y;
                    }
                }
            } else if (half > 0) {
                // the other half's elements are half / 8 lanes away
                const bool low = 8 * sub < half;
                const int peer = (threadIdx.x & 31) + (turned ? (low ? half / 8 : -(half / 8)) : 0);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float other = __shfl_sync(0xFFFFFFFFu, x[u][e], peer);
                    if (turned) {
                        const float2 cs = turn_smem[i * half + (low ? 8 * sub : 8 * sub - half) + e];
                        x[u][e] = x[u][e] * cs.x + (low ? -other : other) * cs.y;
                    }
                }
            }
            const RowPlace at = place[i];
            const bool write = item < items && active && (at.state == 0 || (at.state == 2 && (is_q || !kAppend)));
            if (write) {
                if (at.state == 2) {  // (of a bad row nothing goes into the cache)
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[u][e] = __int_as_float(0x7FC00000);
                }
                const long long row = row0 + i;
                TOut* out;
                if (is_q) {
                    out = static_cast<TOut*>(p.q_out) + row * p.q_out_stride + (long long)h * p.d;
                } else if (!kAppend) {
                    out = static_cast<TOut*>(p.k_out) + row * p.k_out_stride + (long long)(h - p.hq) * p.d;
                } else {
                    const int kh = is_v ? h - p.hq - p.hkv : h - p.hq;
                    out = static_cast<TOut*>(is_v ? p.v_cache : p.k_cache) +
                          ((at.page * p.hkv + kh) * p.page + at.slot) * p.d;
                }
                store8(out + 8 * sub, x[u]);
            }
        }
        if (base - group + kHeadUnroll * n_groups >= items) break;  // the same for every group
        fetch(base + kHeadUnroll * n_groups);
    }
}

template <typename TIn, typename TOut>
cudaError_t launch_typed(const HeadsParams& p, cudaStream_t stream) {
    const int lanes = p.d <= 64 ? 8 : p.d <= 128 ? 16 : 32;
    const int n_heads = p.hq + (p.v ? 2 : 1) * p.hkv;
    // A CTA of about kHeadThreads / 2 threads, each group of lanes holding kHeadUnroll heads: a row of 40 heads
    // of 128 has one to itself, rows of few heads share one (up to kHeadRows).
    const int want = kHeadThreads / 2 / lanes * kHeadUnroll;  // heads of a CTA
    int rows_per_cta = want / n_heads;
    rows_per_cta = rows_per_cta < 1 ? 1 : rows_per_cta > kHeadRows ? kHeadRows : rows_per_cta;
    const int groups = (rows_per_cta * n_heads + kHeadUnroll - 1) / kHeadUnroll;
    int threads = (groups * lanes + 31) / 32 * 32;
    if (threads > kHeadThreads) threads = kHeadThreads;
    const unsigned grid = (unsigned)((p.rows + rows_per_cta - 1) / rows_per_cta);
    const size_t smem = sizeof(float2) * (size_t)rows_per_cta * (p.rot / 2);
    const bool append = p.v != nullptr;
    if (p.pairs) {
        if (append) heads_kernel<TIn, TOut, true, true><<<grid, threads, smem, stream>>>(p, rows_per_cta, lanes);
        else heads_kernel<TIn, TOut, true, false><<<grid, threads, smem, stream>>>(p, rows_per_cta, lanes);
    } else {
        if (append) heads_kernel<TIn, TOut, false, true><<<grid, threads, smem, stream>>>(p, rows_per_cta, lanes);
        else heads_kernel<TIn, TOut, false, false><<<grid, threads, smem, stream>>>(p, rows_per_cta, lanes);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_heads(const HeadsParams& p, cudaStream_t stream) {
    if (p.in_dtype == DSPARK_F32)
        return p.out_dtype == DSPARK_F32 ? launch_typed<float, float>(p, stream)
                                         : launch_typed<float, __nv_bfloat16>(p, stream);
    return p.out_dtype == DSPARK_F32 ? launch_typed<__nv_bfloat16, float>(p, stream)
                                     : launch_typed<__nv_bfloat16, __nv_bfloat16>(p, stream);
}

}  // namespace dspark
