// markov_grad.cu -- gradients of the Markov factors from the gradient of the
// drafter's logits.
//
// The drafter's logits of row n are U[n] + W2 . W1[prev[n]], so with g = dL/dlogits
//   grad_prev[n] = sum_v g[n][v] W2[v]            (dL / d W1[prev[n]], of this row)
//   dW1[a]       = sum of grad_prev[n] over the rows with prev[n] = a
//   dW2[v]       = sum_n g[n][v] W1[prev[n]]
// Both products are sums of exact products of bf16 values in fp32.
#include <algorithm>

#include "kernels.cuh"

namespace dspark {
namespace {

constexpr int kTile = 64, kStep = 16, kThreads = 256;
constexpr int kSplitKeys = 8192;

int splits_of(int V) { return (V + kSplitKeys - 1) / kSplitKeys; }

// ---- W1 rows of the previous tokens, zeros where there is none
__global__ void __launch_bounds__(128) gather_kernel(const MarkovGradParams p, uint16_t* E) {
    const int n = blockIdx.x;
    const int a = p.prev[n];
    if (a >= p.V && threadIdx.x == 0) report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
    const bool there = a >= 0 && a < p.V;
    for (int i = threadIdx.x; i < p.rank; i += 128)
        E[(size_t)n * p.rank + i] = there ? p.W1[(size_t)a * p.rank + i] : (uint16_t)0;
}

// C[m][r] = sum_k A[m][k] B[k][r] over k in [z * per, ...): a tile of 64 x 64 per CTA.
__global__ void __launch_bounds__(kThreads) product_kernel(const uint16_t* A, int64_t sm, int64_t sk, const uint16_t* B,
                                                           int M, int K, int rank, int per, float* C, int accumulate) {
    __shared__ float a[kStep][kTile + 1], b[kStep][kTile + 1];
    const int m0 = blockIdx.x * kTile, r0 = blockIdx.y * kTile, z = blockIdx.z;
    const int k_begin = z * per, k_end = min(K, k_begin + per);
    const int tm = threadIdx.x / 16 * 4, tr = threadIdx.x % 16 * 4;
    float acc[4][4] = {};
    for (int k0 = k_begin; k0 < k_end; k0 += kStep) {
        for (int i = threadIdx.x; i < kStep * kTile; i += kThreads) {
            // neighbouring threads along the contiguous direction
            const int ka = sk == 1 ? i % kStep : i / kTile, ma = sk == 1 ? i / kStep : i % kTile;
            a[ka][ma] = k0 + ka < k_end && m0 + ma < M ? bf16_bits_to_float(A[(m0 + ma) * sm + (k0 + ka) * sk]) : 0.0f;
            const int kb = i / kTile, rb = i % kTile;
            b[kb][rb] = k0 + kb < k_end ? bf16_bits_to_float(B[(size_t)(k0 + kb) * rank + r0 + rb]) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kStep; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += a[k][tm + i] * b[k][tr + j];
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j)
            if (m0 + tm + i < M) {
                float* c = C + ((size_t)z * M + m0 + tm + i) * rank + r0 + tr + j;
                *c = accumulate ? *c + acc[i][j] : acc[i][j];
            }
}

// ---- the splits of grad_prev, in order
__global__ void __launch_bounds__(128) join_kernel(const MarkovGradParams p, const float* part, int splits) {
    const int n = blockIdx.x;
    const int a = p.prev[n];
    for (int i = threadIdx.x; i < p.rank; i += 128) {
        float s = 0.0f;
        for (int z = 0; z < splits; ++z) s += part[((size_t)z * p.rows + n) * p.rank + i];
        p.grad_prev[(size_t)n * p.rank + i] = a < 0 ? 0.0f : a >= p.V ? NAN : s;
    }
}

// ---- dW1: the first row of each previous token adds up all of them, in order
__global__ void __launch_bounds__(128) scatter_kernel(const MarkovGradParams p) {
    const int n = blockIdx.x;
    const int a = p.prev[n];
    if (a < 0 || a >= p.V) return;
    int seen = 0;
    for (int m = threadIdx.x; m < n; m += 128) seen |= p.prev[m] == a;
    if (__syncthreads_or(seen)) return;
    constexpr int kMost = 4;  // rank <= 512
    float s[kMost] = {};
    for (int m0 = n; m0 < p.rows; m0 += 32) {
        const int m = m0 + (threadIdx.x & 31);
        unsigned same = __ballot_sync(0xFFFFFFFFu, m < p.rows && p.prev[m] == a);
        for (; same; same &= same - 1) {
            const float* g = p.grad_prev + (size_t)(m0 + __ffs(same) - 1) * p.rank;
#pragma unroll
            for (int i = 0; i < kMost; ++i)
                if (threadIdx.x + 128 * i < p.rank) s[i] += g[threadIdx.x + 128 * i];
        }
    }
    float* d = p.dW1 + (size_t)a * p.rank;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        const int r = threadIdx.x + 128 * i;
        if (r < p.rank) d[r] = p.accumulate ? d[r] + s[i] : s[i];
    }
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t markov_grad_workspace(int rows, int V, int rank) {
    return 256 + align256((size_t)rows * rank * 2) + (size_t)splits_of(V) * rows * rank * 4;
}

cudaError_t launch_markov_grad(const MarkovGradParams& p, cudaStream_t stream) {
    if (p.rows == 0) {
        if (!p.dW2 || p.accumulate) return cudaSuccess;
        return cudaMemsetAsync(p.dW2, 0, (size_t)p.V * p.rank * sizeof(float), stream);
    }
    uint16_t* E = static_cast<uint16_t*>(p.ws);
    float* part = reinterpret_cast<float*>(static_cast<unsigned char*>(p.ws) + align256((size_t)p.rows * p.rank * 2));
    const int splits = splits_of(p.V);
    gather_kernel<<<p.rows, 128, 0, stream>>>(p, E);
    product_kernel<<<dim3((p.rows + kTile - 1) / kTile, p.rank / kTile, splits), kThreads, 0, stream>>>(
        p.grad, p.stride, 1, p.W2, p.rows, p.V, p.rank, kSplitKeys, part, 0);
    join_kernel<<<p.rows, 128, 0, stream>>>(p, part, splits);
    if (p.dW1) scatter_kernel<<<p.rows, 128, 0, stream>>>(p);
    if (p.dW2)
        product_kernel<<<dim3((p.V + kTile - 1) / kTile, p.rank / kTile, 1), kThreads, 0, stream>>>(
            p.grad, 1, p.stride, E, p.V, p.rows, p.rank, p.rows, p.dW2, p.accumulate);
    return cudaGetLastError();
}

}  // namespace dspark
