// attention.cu -- attention of packed verify rows over the paged KV cache.
//
// Row i of request r (row cu[r] + i of q) stands at position kv_len[r] + i.
// With g = hq / hkv query heads to a key head, s_j = scale * q . K[j] over the
// keys j it sees (j <= kv_len + i, or every j < kv_len + n in a full block):
//   out = sum_j e^{s_j - lse} V[j],   lse = log sum_j e^{s_j}
//
// One warp per (row, query head), one pass over the keys with the running
// maximum and sum of the softmax in fp32.
#include "kernels.cuh"

namespace dspark {
namespace {

constexpr int kAttnThreads = 256;

// The group of request r: the last g with group_start[g] <= r.
__device__ __forceinline__ int group_of(const AttnParams& p, int r) {
    int g = 0;
    while (g + 1 < p.n_groups && p.group_start[g + 1] <= r) ++g;
    return g;
}

template <int kD>
__global__ void __launch_bounds__(kAttnThreads) attention_kernel(const AttnParams p) {
    constexpr int kPer = kD / 32;
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * (kAttnThreads / 32) + (threadIdx.x >> 5);
    if (item >= (long long)p.rows * p.hq) return;
    const int row = (int)(item / p.hq), hq = (int)(item % p.hq), h = hq / (p.hq / p.hkv);
    // offsets that are not 0 .. rows spoil the whole batch, and so do groups that are not 0 .. R
    bool ok = p.cu[0] == 0 && p.cu[p.R] <= p.rows;
    for (int r = lane; r < p.R; r += 32) ok = ok && p.cu[r] <= p.cu[r + 1];
    if (p.n_groups > 0) {
        ok = ok && p.group_start[0] == 0 && p.group_start[p.n_groups] == p.R;
        for (int g = lane; g < p.n_groups; g += 32) ok = ok && p.group_start[g] <= p.group_start[g + 1];
    }
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (ok && row >= p.cu[p.R]) return;
    int r = 0;
    while (ok && r + 1 < p.R && p.cu[r + 1] <= row) ++r;
    const int lo = p.cu[r], hi = p.cu[r + 1], len = p.kv_len[r];
    ok = ok && row >= lo && row < hi && len >= 0;
    const long long total = (long long)len + (hi - lo);
    ok = ok && total <= (long long)p.max_blocks * p.page;
    int shared = 0, first = 0;
    if (p.n_groups > 0) {
        const int g = ok ? group_of(p, r) : 0;
        shared = p.shared_len[g];
        first = p.group_start[g];
        ok = ok && shared >= 0 && shared <= len && shared % p.page == 0 && first >= 0 && first <= r;
    }
    float q[kPer], o[kPer], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        q[e] = __bfloat162float(p.q[item * kD + lane + 32 * e]);
        o[e] = 0.0f;
    }
    const int last = p.full_block ? (int)total - 1 : len + (row - lo);
    for (int j = 0; ok && j <= last; ++j) {
        const int b = j / p.page;
        const int page = p.block_table[(long long)(j < shared ? first : r) * p.max_blocks + b];
        if (page < 0 || page >= p.pool_pages) { ok = false; break; }
        const long long at = (((long long)page * p.hkv + h) * p.page + (j - b * p.page)) * kD + lane;
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) s = fmaf(q[e], __bfloat162float(p.k_cache[at + 32 * e]), s);
#pragma unroll
        for (int x = 16; x; x >>= 1) s += shfl_xor(s, x);
        s *= p.scale;
        const float top = fmaxf(m, s);
        const float ref = top == -INFINITY ? 0.0f : top;
        const float keep = expf(m - ref), w = expf(s - ref);
        l = l * keep + w;
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] = fmaf(w, __bfloat162float(p.v_cache[at + 32 * e]), o[e] * keep);
        m = top;
    }
    if (!ok && lane == 0) report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
    const float inv = ok ? 1.0f / l : __int_as_float(0x7FC00000);
#pragma unroll
    for (int e = 0; e < kPer; ++e) p.out[item * kD + lane + 32 * e] = __float2bfloat16(ok ? o[e] * inv : inv);
    if (p.lse && lane == 0) p.lse[item] = ok ? m + logf(l) : inv;
}

}  // namespace

size_t attention_workspace(int, int, int, int, int, int) { return 256; }

cudaError_t launch_attention(const AttnParams& p, cudaStream_t stream) {
    const unsigned grid = (unsigned)(((long long)p.rows * p.hq + kAttnThreads / 32 - 1) / (kAttnThreads / 32));
    if (p.d == 64) attention_kernel<64><<<grid, kAttnThreads, 0, stream>>>(p);
    else attention_kernel<128><<<grid, kAttnThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dspark
