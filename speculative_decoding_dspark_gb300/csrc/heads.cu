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
// Everything is held in fp32 and rounded once at the store.  An fp32 angle is
// off by 0.03 rad at position 500000, so the angle is counted in turns of 2^-64:
// a frequency is inv_freq / (2 pi) in 64-bit fixed point (rounded from fp64),
// pos times that wraps at whole turns by itself, and what is left is within
// pos * 2^-56 of a turn.  The fp32 sine and cosine see half a turn at most.
//
// What bounds it: bytes (each input element read once, each output written
// once).  A head is read by d / 8 lanes; a lane holds four pairs, two groups of
// four contiguous elements, so that pairs meet in its registers, and kHeadUnroll
// heads at once, whose loads are in flight together.  The angles of a row are
// formed once for all of its heads, those of a CTA's rows together.
#include "kernels.cuh"

namespace dspark {
namespace {

constexpr int kHeadThreads = 512;  // most threads of a CTA
constexpr int kHeadUnroll = 3;     // heads a lane group holds at once
constexpr int kHeadRows = 8;       // most rows of a CTA

struct RowPlace {     // where a row's keys and values go
    long long page;   // page id
    int slot;         // row of the page
    int state;        // 0 write, 1 leave untouched, 2 bad input: outputs are NaN
};

// Four elements as they lie in memory.
template <typename T> struct Quad;
template <> struct Quad<float> {
    float4 v;
    __device__ __forceinline__ void get(float* x) const { x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w; }
    __device__ __forceinline__ void set(const float* x) { v = make_float4(x[0], x[1], x[2], x[3]); }
};
template <> struct Quad<__nv_bfloat16> {
    uint2 v;
    __device__ __forceinline__ void get(float* x) const {
        x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xFFFF0000u);
        x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
    __device__ __forceinline__ void set(const float* x) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
        v = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
};

// n / d for n * d < 2^32, by a product with ceil(2^32 / d) (d > 1).
struct Divider {
    uint32_t d, m;
    __host__ explicit Divider(int x) : d((uint32_t)x), m(x > 1 ? (uint32_t)(((1ull << 32) + x - 1) / x) : 0) {}
    __device__ __forceinline__ int div(int n) const { return d == 1 ? n : (int)__umulhi((uint32_t)n, m); }
};

template <typename TIn, typename TOut, bool kPairs, bool kAppend>
__global__ void __launch_bounds__(kHeadThreads) heads_kernel(const HeadsParams p, int rows_per_cta, int log_lanes,
                                                             const Divider by_heads) {
    extern __shared__ __align__(16) float2 turn_smem[];  // [rows_per_cta][rot / 2] cosine, sine
    __shared__ RowPlace place[kHeadRows];
    const int half = p.rot / 2;
    const int row0 = blockIdx.x * rows_per_cta;
    const int rows = min(rows_per_cta, p.rows - row0);
    const int n_heads = p.hq + (kAppend ? 2 : 1) * p.hkv;
    const int sub = threadIdx.x & ((1 << log_lanes) - 1), group = threadIdx.x >> log_lanes;
    const int n_groups = blockDim.x >> log_lanes;
    const bool active = 8 * sub < p.d;
    const bool turned = 8 * sub < p.rot;
    const int items = rows * n_heads;
    // this lane's two quads of a head
    const int at0 = !kPairs && turned ? 4 * sub : 8 * sub, at1 = !kPairs && turned ? half + 4 * sub : 8 * sub + 4;

    Quad<TIn> raw[kHeadUnroll][2];
    auto fetch = [&](int base) {
#pragma unroll
        for (int u = 0; u < kHeadUnroll; ++u) {
            const int item = base + u * n_groups;
            if (!active || item >= items) continue;
            const int i = by_heads.div(item), h = item - i * n_heads;
            const long long row = row0 + i;
            const TIn* x = h < p.hq            ? static_cast<const TIn*>(p.q) + row * p.q_stride + h * p.d
                           : h < p.hq + p.hkv  ? static_cast<const TIn*>(p.k) + row * p.k_stride + (h - p.hq) * p.d
                                               : static_cast<const TIn*>(p.v) + row * p.v_stride + (h - p.hq - p.hkv) * p.d;
            raw[u][0] = *reinterpret_cast<const Quad<TIn>*>(x + at0);
            raw[u][1] = *reinterpret_cast<const Quad<TIn>*>(x + at1);
        }
    };
    fetch(group);  // in flight while the angles are formed

    // each warp takes rows in turn: where the row goes, and its angles
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n_warps = blockDim.x >> 5;
    for (int w = warp; w < rows * 2; w += n_warps) {  // two warps to a row: each has half of the angles
        const int i = w >> 1, row = row0 + i;
        long long pos = 0;
        RowPlace at{-1, 0, 0};
        if (kAppend) {
            const int r = owner_of(p.cu, p.R, row);
            const int lo = p.cu[r], hi = p.cu[r + 1], len = p.kv_len[r], live = p.cu[p.R];
            if (w == 0 && row == 0 && lane == 0 && (p.cu[0] != 0 || live > p.rows || live < 0))
                report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
            if (row < lo || row >= hi) {
                at.state = row >= live ? 1 : 2;
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
        if (lane == 0 && !(w & 1)) place[i] = at;
        for (int f = lane + 32 * (w & 1); f < half; f += 64) {
            const double turn = (double)p.inv_freq[f] * 0.15915494309189533577;  // 1 / (2 pi)
            const double part = turn - rint(turn);                                // whole turns leave no trace
            const long long step = __double2ll_rn(part * 18446744073709551616.0 * 0.5);  // of 2^-63 turns
            const int left = (int)(2 * (unsigned long long)pos * (unsigned long long)step >> 32);  // what is left of a turn, 2^-32
            float s, c;
            sincospif((float)left * 0x1p-31f, &s, &c);
            turn_smem[i * half + f] = make_float2(c, s);
        }
    }
    float wq[8], wk[8];  // the weights of this lane's elements
    auto weights = [&](const void* from, float (&w)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.0f;
        if (active && from) {
            reinterpret_cast<const Quad<TIn>*>(static_cast<const TIn*>(from) + at0)->get(w);
            reinterpret_cast<const Quad<TIn>*>(static_cast<const TIn*>(from) + at1)->get(w + 4);
        }
    };
    weights(p.wq, wq);
    weights(p.wk, wk);
    const float inv_d = 1.0f / (float)p.d;
    __syncthreads();

    for (int base = group;; base += kHeadUnroll * n_groups) {
#pragma unroll
        for (int u = 0; u < kHeadUnroll; ++u) {
            const int item = base + u * n_groups;  // (groups past the end take part in the shuffles)
            const bool there = active && item < items;
            const int i = item < items ? by_heads.div(item) : 0, h = item < items ? item - i * n_heads : 0;
            const bool is_q = h < p.hq, is_v = h >= p.hq + p.hkv;
            float x[8];
            raw[u][0].get(x);
            raw[u][1].get(x + 4);
            if (p.wq || p.wk) {
                float ss = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
                if (!there) ss = 0.0f;
                for (int o = 1 << log_lanes >> 1; o; o >>= 1) ss += shfl_xor(ss, o);
                if (!is_v && (is_q ? p.wq : p.wk)) {
                    const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = x[e] * r * (is_q ? wq[e] : wk[e]);
                }
            }
            if (!is_v && turned) {
                const float4* cs = reinterpret_cast<const float4*>(turn_smem + i * half + 4 * sub);
                const float4 t0 = cs[0], t1 = cs[1];
                const float c[4] = {t0.x, t0.z, t1.x, t1.z}, s[4] = {t0.y, t0.w, t1.y, t1.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int ia = kPairs ? 2 * e : e, ib = kPairs ? 2 * e + 1 : e + 4;
                    const float a = x[ia], b = x[ib];
                    x[ia] = a * c[e] - b * s[e];
                    x[ib] = b * c[e] + a * s[e];
                }
            }
            const RowPlace at = place[i];
            if (there && (at.state == 0 || (at.state == 2 && (is_q || !kAppend)))) {
                if (at.state == 2) {  // (of a bad row nothing goes into the cache)
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = __int_as_float(0x7FC00000);
                }
                const long long row = row0 + i;
                TOut* out;
                if (is_q) {
                    out = static_cast<TOut*>(p.q_out) + row * p.q_out_stride + h * p.d;
                } else if (!kAppend) {
                    out = static_cast<TOut*>(p.k_out) + row * p.k_out_stride + (h - p.hq) * p.d;
                } else {
                    const int kh = is_v ? h - p.hq - p.hkv : h - p.hq;
                    out = static_cast<TOut*>(is_v ? p.v_cache : p.k_cache) +
                          ((at.page * p.hkv + kh) * p.page + at.slot) * p.d;
                }
                Quad<TOut> y;
                y.set(x);
                *reinterpret_cast<Quad<TOut>*>(out + at0) = y;
                y.set(x + 4);
                *reinterpret_cast<Quad<TOut>*>(out + at1) = y;
            }
        }
        if (base - group + kHeadUnroll * n_groups >= items) break;  // the same for every group
        fetch(base + kHeadUnroll * n_groups);
    }
}

template <typename TIn, typename TOut>
cudaError_t launch_typed(const HeadsParams& p, cudaStream_t stream) {
    const int log_lanes = p.d <= 64 ? 3 : p.d <= 128 ? 4 : 5;
    const int n_heads = p.hq + (p.v ? 2 : 1) * p.hkv;
    // A CTA's groups of lanes hold all heads of its rows at once where about 256 threads can (a row of 40 heads of
    // 128: 224), and it has as many rows as leave four CTAs to an SM (152 of them), so that their angles are formed
    // together.
    const int want = (256 >> log_lanes) * kHeadUnroll;  // heads of a pass
    int rows_per_cta = p.rows / (4 * 152);
    rows_per_cta = rows_per_cta < 1 ? 1 : rows_per_cta > kHeadRows ? kHeadRows : rows_per_cta;
    const int pass = n_heads * rows_per_cta < want ? n_heads * rows_per_cta : n_heads > want ? want : n_heads * (want / n_heads);
    const int threads = (((pass + kHeadUnroll - 1) / kHeadUnroll << log_lanes) + 31) / 32 * 32;
    const unsigned grid = (unsigned)((p.rows + rows_per_cta - 1) / rows_per_cta);
    const size_t smem = sizeof(float2) * (size_t)rows_per_cta * (p.rot / 2);
    const Divider by_heads(n_heads);
    const bool append = p.v != nullptr;
    if (p.pairs) {
        if (append) heads_kernel<TIn, TOut, true, true><<<grid, threads, smem, stream>>>(p, rows_per_cta, log_lanes, by_heads);
        else heads_kernel<TIn, TOut, true, false><<<grid, threads, smem, stream>>>(p, rows_per_cta, log_lanes, by_heads);
    } else {
        if (append) heads_kernel<TIn, TOut, false, true><<<grid, threads, smem, stream>>>(p, rows_per_cta, log_lanes, by_heads);
        else heads_kernel<TIn, TOut, false, false><<<grid, threads, smem, stream>>>(p, rows_per_cta, log_lanes, by_heads);
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
