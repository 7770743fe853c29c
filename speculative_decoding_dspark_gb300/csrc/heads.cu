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
// once), and before that instructions and latency.  A head of a row is d / 16
// lanes, each with eight pairs in its registers (two groups of eight elements, of
// a half-rotated head half of the rotated part apart); a group of lanes keeps its
// head and goes down the CTA's rows, whose next three are on their way by 16-byte
// copies into places of the group's own, so that no register waits for memory.
// The places and angles of the rows are worked out once for all heads.
// 16384 rows of 32 + 8 heads of 128 in bf16 (336 MB): a head at a time with eight
// elements to a lane took 191 us, 104 with its next in registers, this 58 us, 85 %
// of the copy rate.  10200 rows of 24 + 8 + 8 heads of 64 from fp32 into pages of
// 12 (157 MB): 44 us, 53 %: there a CTA's start, four loads that wait for each
// other until it knows its pages, is a third of its life.
#include "kernels.cuh"
#include "tc_ptx.cuh"

namespace dspark {
namespace {

constexpr int kHeadThreads = 256;  // most threads of a CTA
constexpr int kHeadRows = 8;       // most rows of a CTA
constexpr int kHeadAhead = 3;      // rows a thread has on their way

struct RowPlace {
    long long at;     // where the row's keys and values go: elements from the cache's first head to the slot
    int state;        // 0 write, 1 leave untouched, 2 bad input: outputs are NaN
    int pad;
};

// Shared memory of a CTA besides the rows' turns and the places for rows on their way.
struct HeadsShared {
    RowPlace place[kHeadRows];
    long long pos[kHeadRows];
    long long steps[DSPARK_HEADS_MAX_D / 2];  // a pair's turn from one position to the next, in 2^-63 (LLONG_MIN: it has none)
};

// Eight elements as they lie in memory.
template <typename T> struct Octet;
template <> struct Octet<float> {
    float4 v[2];
    __device__ __forceinline__ void get(float2* x) const {
        x[0] = make_float2(v[0].x, v[0].y); x[1] = make_float2(v[0].z, v[0].w);
        x[2] = make_float2(v[1].x, v[1].y); x[3] = make_float2(v[1].z, v[1].w);
    }
    __device__ __forceinline__ void set(const float2* x) {
        v[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
        v[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
    }
    static constexpr int kParts = 2;  // of 16 bytes
    __device__ __forceinline__ void load(const float* p) { v[0] = reinterpret_cast<const float4*>(p)[0]; v[1] = reinterpret_cast<const float4*>(p)[1]; }
    __device__ __forceinline__ void store(float* p) const { reinterpret_cast<float4*>(p)[0] = v[0]; reinterpret_cast<float4*>(p)[1] = v[1]; }
};
template <> struct Octet<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void get(float2* x) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
    __device__ __forceinline__ void set(const float2* x) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 a = __floats2bfloat162_rn(x[i].x, x[i].y);
            w[i] = *reinterpret_cast<const uint32_t*>(&a);
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    static constexpr int kParts = 1;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
};

template <typename TIn, typename TOut, bool kPairs, bool kAppend>
__global__ void __launch_bounds__(kHeadThreads, 4) heads_kernel(const HeadsParams p, int rows_per_cta, int log_lanes) {
    // [rows_per_cta][2][rot / 2] cosines and sines, then each thread's places for the rows on their way:
    // [kHeadAhead][octet][16-byte part][thread]
    extern __shared__ __align__(16) float turn_smem[];
    constexpr int kParts = Octet<TIn>::kParts;
    __shared__ HeadsShared sh;
    const int half = p.rot / 2;
    const int row0 = blockIdx.x * rows_per_cta;
    const int rows = min(rows_per_cta, p.rows - row0);
    const int n_heads = p.hq + (kAppend ? 2 : 1) * p.hkv;
    const int sub = threadIdx.x & ((1 << log_lanes) - 1), n_groups = blockDim.x >> log_lanes;
    const bool turned = 16 * sub < p.rot;
    // this lane's two octets of a head: of a half-rotated head eight pairs' first elements, then their second ones
    const int at0 = !kPairs && turned ? 8 * sub : 16 * sub, at1 = !kPairs && turned ? half + 8 * sub : 16 * sub + 8;
    const bool have0 = at0 < p.d, have1 = at1 < p.d && have0;

    float4* const ring = reinterpret_cast<float4*>(turn_smem + rows_per_cta * p.rot);
    // Of a head in memory a lane copies every (lanes)th 16 bytes, so that a group's copies are contiguous, each to the
    // place of the lane that has these elements.
    constexpr int kChunk = 8 / kParts;
    int copy_to[2 * kParts], copy_from[2 * kParts];
#pragma unroll
    for (int q = 0; q < 2 * kParts; ++q) {
        const int e = (sub + (q << log_lanes)) * kChunk;  // its first element
        const bool halves = !kPairs && e < p.rot;
        const int in = halves && e >= half ? e - half : e;
        const int lane = halves ? in / 8 : e / 16, octet = halves ? (e >= half) : (e / 8) & 1;
        copy_from[q] = e < p.d ? e : -1;
        copy_to[q] = (octet * kParts + e % 8 / kChunk) * blockDim.x + threadIdx.x - sub + lane;
    }

    // The rows of the group's first head, then of its next, ...
    const int first_head = blockIdx.y * n_groups + (threadIdx.x >> log_lanes), head_step = gridDim.y * n_groups;
    const int n_rows = (n_heads + head_step - 1) / head_step * rows;  // of all the group's heads
    int next_h = first_head, next_i = 0;
    const TIn* from = nullptr;
    int64_t from_stride = 0;
    auto fetch = [&](int stage) {
        if (next_i == 0) {
            const bool is_q = next_h < p.hq, is_v = next_h >= p.hq + p.hkv;
            from_stride = is_q ? p.q_stride : is_v ? p.v_stride : p.k_stride;
            from = static_cast<const TIn*>(is_q ? p.q : is_v ? p.v : p.k) + row0 * from_stride +
                   (is_q ? next_h : is_v ? next_h - p.hq - p.hkv : next_h - p.hq) * p.d;
        }
        if (next_h < n_heads) {
#pragma unroll
            for (int q = 0; q < 2 * kParts; ++q)
                if (copy_from[q] >= 0) tc::cp_async_16(tc::smem_u32(ring + stage * 2 * kParts * blockDim.x + copy_to[q]), from + copy_from[q], 16);
        }
        tc::cp_async_commit();
        from += from_stride;
        if (++next_i == rows) {
            next_i = 0;
            next_h += head_step;
        }
    };
#pragma unroll
    for (int i = 0; i < kHeadAhead; ++i) fetch(i);  // in flight while the angles are formed

    // where the rows go: the first row's request by the first warp together, from there on a lane to a row
    if (threadIdx.x < 32) {
        const int i = threadIdx.x, row = row0 + i;
        int r = kAppend ? owner_of(p.cu, p.R, row0) : 0;
        if (i < rows) {
            long long at_pos = 0;
            RowPlace at{0, 0, 0};
            if (kAppend) {
                const int live = p.cu[p.R];
                while (r + 1 < p.R && p.cu[r + 1] <= row) ++r;
                const int lo = p.cu[r], hi = p.cu[r + 1], len = p.kv_len[r];
                if (row == 0 && (p.cu[0] != 0 || live > p.rows || live < 0)) report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
                if (row < lo || row >= hi) {
                    at.state = row >= live ? 1 : 2;
                } else {
                    at_pos = (long long)len + (row - lo);
                    const int b = len < 0 || at_pos > INT_MAX ? p.max_blocks : (int)at_pos / p.page;
                    const int id = lo < 0 || b >= p.max_blocks ? -1 : p.block_table[(long long)r * p.max_blocks + b];
                    if (id < 0 || id >= p.pool_pages) at.state = 2;
                    else at.at = ((long long)id * p.hkv * p.page + ((int)at_pos - b * p.page)) * p.d;
                }
            } else if (half > 0) {
                at_pos = p.positions[row];
                if (at_pos < 0) at.state = 2;
            }
            if (at.state == 2) report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
            sh.place[i] = at;
            sh.pos[i] = at_pos;
        }
    }
    for (int f = threadIdx.x; f < half; f += blockDim.x) {
        const double turn = (double)p.inv_freq[f] * 0.15915494309189533577;  // 1 / (2 pi)
        const double part = turn - rint(turn);                                // whole turns leave no trace
        sh.steps[f] = isnan(part) ? LLONG_MIN : __double2ll_rn(part * 18446744073709551616.0 * 0.5);
    }
    __syncthreads();
    for (int j = threadIdx.x; j < rows * half; j += blockDim.x) {
        const int i = j / half, f = j - i * half;
        const int left = (int)(2 * (unsigned long long)sh.pos[i] * (unsigned long long)sh.steps[f] >> 32);  // of a turn, in 2^-32
        float s, c;
        sincospif((float)left * 0x1p-31f, &s, &c);
        if (sh.steps[f] == LLONG_MIN) s = c = __int_as_float(0x7FC00000);
        turn_smem[2 * i * half + f] = c;
        turn_smem[2 * i * half + half + f] = s;
    }
    const float inv_d = 1.0f / (float)p.d;
    __syncthreads();

    float2 wt[8];  // the weights of this lane's elements
    int h = first_head, i = 0;
    bool is_q = false, norm = false, turn = false, there = false, cached = false;
    TOut* out = nullptr;
    int64_t out_stride = 0;
#pragma unroll 1
    for (int n = 0; n < n_rows; ++n) {  // (groups without a head take part in the shuffles)
        if (i == 0) {  // a new head
            const bool is_v = h >= p.hq + p.hkv;
            is_q = h < p.hq;
            there = h < n_heads;
            norm = there && !is_v && (is_q ? p.wq : p.wk) != nullptr;
            turn = !is_v && turned;
            cached = kAppend && !is_q;
            const int kh = is_q ? h : is_v ? h - p.hq - p.hkv : h - p.hq;
            out_stride = cached ? 0 : is_q ? p.q_out_stride : p.k_out_stride;
            out = static_cast<TOut*>(is_q ? p.q_out : kAppend ? (is_v ? p.v_cache : p.k_cache) : p.k_out) + row0 * out_stride +
                  (long long)kh * p.d * (cached ? p.page : 1);
            if (norm && have0) {
                const TIn* const w = static_cast<const TIn*>(is_q ? p.wq : p.wk);
                Octet<TIn> o;
                o.load(w + at0);
                o.get(wt);
                if (have1) o.load(w + at1);
                o.get(wt + 4);
            }
        }
        {
            const int stage = n % kHeadAhead;
            tc::cp_async_wait<kHeadAhead - 1>();
            __syncwarp();
            Octet<TIn> raw[2];
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int e = 0; e < kParts; ++e)
                    reinterpret_cast<float4*>(&raw[o])[e] = ring[((stage * 2 + o) * kParts + e) * blockDim.x + threadIdx.x];
            __syncwarp();
            fetch(stage);
            float2 x[8];  // this lane's elements: the first octet's, then the second's
            raw[0].get(x);
            raw[1].get(x + 4);
            if (p.wq || p.wk) {
                float2 sq = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < 4 ? have0 : have1) sq = fma2(x[e], x[e], sq);
                float ss = there ? sq.x + sq.y : 0.0f;
                ss += shfl_xor(ss, 1);
                ss += shfl_xor(ss, 2);
                if (log_lanes >= 3) ss += shfl_xor(ss, 4);
                if (log_lanes >= 4) ss += shfl_xor(ss, 8);
                if (norm) {
                    const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = mul2(mul2(x[e], make_float2(r, r)), wt[e]);
                }
            }
            if (turn) {
                // cosines and sines of this lane's eight pairs
                const float* const cs = turn_smem + 2 * i * half + 8 * sub;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float4 c = reinterpret_cast<const float4*>(cs)[q], s = reinterpret_cast<const float4*>(cs + half)[q];
                    if (kPairs) {
                        float2* const y = x + 4 * q;
                        y[0] = make_float2(y[0].x * c.x - y[0].y * s.x, y[0].y * c.x + y[0].x * s.x);
                        y[1] = make_float2(y[1].x * c.y - y[1].y * s.y, y[1].y * c.y + y[1].x * s.y);
                        y[2] = make_float2(y[2].x * c.z - y[2].y * s.z, y[2].y * c.z + y[2].x * s.z);
                        y[3] = make_float2(y[3].x * c.w - y[3].y * s.w, y[3].y * c.w + y[3].x * s.w);
                    } else {
                        const float2 a0 = x[2 * q], a1 = x[2 * q + 1], b0 = x[2 * q + 4], b1 = x[2 * q + 5];
                        const float2 c0 = make_float2(c.x, c.y), c1 = make_float2(c.z, c.w);
                        x[2 * q] = fma2(a0, c0, mul2(b0, make_float2(-s.x, -s.y)));
                        x[2 * q + 1] = fma2(a1, c1, mul2(b1, make_float2(-s.z, -s.w)));
                        x[2 * q + 4] = fma2(b0, c0, mul2(a0, make_float2(s.x, s.y)));
                        x[2 * q + 5] = fma2(b1, c1, mul2(a1, make_float2(s.z, s.w)));
                    }
                }
            }
            const RowPlace at = sh.place[i];
            const bool inside = IN_BOUNDS(row0 + i < p.rows && (!cached || at.state != 0 ||
                                                                (at.at >= 0 && at.at < ((p.pool_pages - 1LL) * p.hkv + 1) * p.page * p.d)),
                                          p.dev_status);
            if (inside && there && (at.state == 0 || (at.state == 2 && !cached))) {  // (of a bad row nothing goes into the cache)
                if (at.state == 2) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = make_float2(__int_as_float(0x7FC00000), __int_as_float(0x7FC00000));
                }
                TOut* const to = cached ? out + at.at : out;
                Octet<TOut> y;
                y.set(x);
                if (have0) y.store(to + at0);
                y.set(x + 4);
                if (have1) y.store(to + at1);
            }
            out += out_stride;
        }
        if (++i == rows) {
            i = 0;
            h += head_step;
        }
    }
}

template <typename TIn, typename TOut>
cudaError_t launch_typed(const HeadsParams& p, cudaStream_t stream) {
    const int log_lanes = p.d <= 64 ? 2 : p.d <= 128 ? 3 : 4;
    const int n_heads = p.hq + (p.v ? 2 : 1) * p.hkv;
    // A group of lanes to every k-th head, k the least that keeps a CTA within 256 threads.  Few rows: a head to a
    // group, spread over CTAs of 128 threads, each forming the angles anew.  Many: kHeadRows of them to a CTA, which
    // leaves four CTAs and more to an SM.
    int rows_per_cta = p.rows / (4 * 152);
    rows_per_cta = rows_per_cta < 1 ? 1 : rows_per_cta > kHeadRows ? kHeadRows : rows_per_cta;
    const int k = (n_heads * (1 << log_lanes) + kHeadThreads - 1) / kHeadThreads, split = p.rows <= 152 ? (n_heads * (1 << log_lanes) + 127) / 128 : 1;
    const int groups = split > 1 ? (n_heads + split - 1) / split : (n_heads + k - 1) / k;
    const int threads = ((groups << log_lanes) + 31) / 32 * 32;
    const dim3 grid((unsigned)((p.rows + rows_per_cta - 1) / rows_per_cta), split);
    const size_t smem = sizeof(float) * (size_t)rows_per_cta * p.rot + sizeof(float4) * kHeadAhead * 2 * Octet<TIn>::kParts * threads;
    const bool append = p.v != nullptr;
    void (*const kernel)(const HeadsParams, int, int) =
        p.pairs ? (append ? heads_kernel<TIn, TOut, true, true> : heads_kernel<TIn, TOut, true, false>)
                : (append ? heads_kernel<TIn, TOut, false, true> : heads_kernel<TIn, TOut, false, false>);
    if (smem + sizeof(HeadsShared) > 48 * 1024) {  // (more than a launch has unasked)
        const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (err != cudaSuccess) return err;
    }
    kernel<<<grid, threads, smem, stream>>>(p, rows_per_cta, log_lanes);
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
