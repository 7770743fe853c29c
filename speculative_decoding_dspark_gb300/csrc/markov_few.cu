// markov_few.cu -- gradients of the Markov factors (markov_grad.cu) for a few rows: a block of one
// request, or of a few.
//
// W2 has to come and dW2 to go once each, and there is little to compute: one kernel makes both products in
// one pass over V, two launches in all instead of four.  A warp has 64 columns of the factors and walks down V, 16
// elements at a time: W2's 16 x 64 arrive in shared memory by asynchronous copies, three of these ahead, and g's 16 x rows
// stand there for all warps.  Sixteen rows are one operand of mma.sync in either direction:
//   grad_prev += g (rows x 16) . W2 (16 x 64),  sums in registers for 512 terms at a time;
//   dW2        = g^T (16 x rows) . E (rows x 64),  E, the rows' W1 rows, in registers.
// (The tensor cores' 128-row tiles would be empty but for these, and the sums over V in parts need more steps; the bytes bound
// it as it is.)  The CTAs of a cluster join their sums through distributed shared memory, few_join_kernel adds
// those of the clusters in order, for dW1 too.
//
// Against the two products of markov_grad.cu: 12.9 and 22.9 us for 7 rows of 32000 at rank 256 (7.4 us of bytes), 18.9 and
// 24.5 for 32 of these, 83.9 and 97.5 for 7 rows of 151936 at rank 512 (70 us of bytes), 7.3 and 12.6 for 7 rows of 8000
// at rank 64.  On the CUDA cores, two rows to a multiply-add, the first took 17.5 us and 16 rows of 151936
// at rank 512 145: there the multiply-adds bound it.  A cluster of two CTAs, one by itself, four: 14.0, 14.5 and
// 14.6 us for the first with nothing in L2; two CTAs of 256 threads on an SM, one of 512: 13.9 and 14.7.
#include <algorithm>

#include "kernels.cuh"
#include "rows.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kChunk = 128;    // elements of g's rows that stand in shared memory at a time
// Stages of W2 to a warp.  Four and two: 12.9 and 14.5 us for 7 rows of 32000 at rank 256 (three or four stages in all, which are
// best on their way at once), 82.8 and 79.8 for 7 rows of 151936 at rank 512.
constexpr int kStages = 4;
constexpr int kStage = 16 * 64 * 2;  // bytes of W2
constexpr int kCluster = 2;
template <int kRows> constexpr int clusters() { return kRows == 16 ? 152 : 76; }  // at most: two CTAs to an SM, or one
template <int kRows> constexpr int g_bytes() { return kChunk * kRows * 2; }
template <int kRows> constexpr int shared_bytes() { return kWarps * kStages * kStage + 2 * g_bytes<kRows>(); }
// A chain of products ends after 512 terms, as in markov_grad.cu, and is added up in fp32; the sums of a warp that has more
// stand in shared memory of its own.  (One chain to a warp: grad_prev of 32 rows of 2^22 elements at rank 512, all terms of one sign,
// was off by 1.4e-4 of itself, 8e-7 with these; 151936 elements 1.9e-6 and 8e-7.)
constexpr int kChain = 32;  // steps of 16 terms
template <int kRows> constexpr int chain_bytes() { return kWarps * kRows * 64 * 4; }
static_assert(kWarps * 32 * 64 * 4 <= shared_bytes<32>(), "the sums take the stages' place");

__device__ __forceinline__ float4 cluster_ld_f32x4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void add_to(float4* p, float4 v) {
    asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ float4 plus(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }

// 16 bytes to shared memory; zeros instead where `there` is false.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }

// Four blocks of 8 x 8, the rows' addresses from the lanes 8 k to 8 k + 7 for block k.
__device__ __forceinline__ void load_blocks(uint32_t (&x)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void load_blocks_turned(uint32_t (&x)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
}
// d += a (16 x 16) . b (16 x 8)
__device__ __forceinline__ void multiply(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// CTA b has the elements from b * per on; `part` is [cluster][row][column].
template <int kRows>
__global__ void __launch_bounds__(kThreads, kRows == 16 ? 2 : 1) few_kernel(const MarkovGradParams p, int per, float* part) {
    constexpr int kTiles = kRows / 16, kPieces = kChunk / 8 * kRows / kThreads;
    extern __shared__ __align__(128) unsigned char memory[];  // W2 [warp][stage][16][64], g twice [oct][row][8]; then the sums
    __shared__ int32_t token[kRows];                          // -1: the row gives nothing
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slices = p.rank / 64, groups = kWarps / slices;
    const int slice = warp % slices, group = warp / slices;   // the warp's columns, and which of the elements
    const bool active = group < groups;
    const int begin = min((int)blockIdx.x * per, p.V), n = min(per, p.V - begin);  // the CTA's elements
    wait_prior_grid();

    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(memory) + warp * kStages * kStage;
    const uint16_t* W2 = p.W2 + (int64_t)begin * p.rank + slice * 64;
    // (a row's eight pieces stand in another order in each of eight rows, so that the reads of eight rows meet in no bank)
    auto fetch = [&](int k) {
        const int v0 = 16 * (group + k * groups);
        const uint32_t to = ring + k % kStages * kStage;
        if (active && v0 < n)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = lane / 8 + 4 * q, piece = lane % 8;
                const bool there = v0 + row < n;
                copy16(to + row * 128 + ((piece ^ (row & 7)) << 4), W2 + (there ? (v0 + row) * p.rank + piece * 8 : 0), there);
            }
        copies_commit();
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(k);

    // eight elements of a row to a piece
    auto load_g = [&](uint4 (&x)[kPieces], int base) {
#pragma unroll
        for (int q = 0; q < kPieces; ++q) {
            const int at = tid + q * kThreads, row = at % kRows, v = base + at / kRows * 8;
            x[q] = row < p.rows && v < n ? __ldcs(reinterpret_cast<const uint4*>(p.grad + (int64_t)row * p.stride + begin + v))
                                         : make_uint4(0, 0, 0, 0);
        }
    };
    uint4 x[kPieces];
    load_g(x, 0);
    if (tid < kRows) {
        const int a = tid < p.rows ? p.prev[tid] : -1;
        token[tid] = a < p.V ? a : -1;
        if (a >= p.V && blockIdx.x == 0) report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
    }
    __syncthreads();
    // Of 16 columns the first product by E takes the even ones, the second the odd ones: a load brings both products', and a
    // thread then has four columns of dW2 side by side.
    const int t = lane & 3, o = lane >> 2;
    uint32_t e[kTiles][8][2];
#pragma unroll
    for (int z = 0; z < kTiles; ++z)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int a0 = token[16 * z + 8 * h + 2 * t], a1 = token[16 * z + 8 * h + 2 * t + 1];
            const uint32_t* w0 = reinterpret_cast<const uint32_t*>(p.W1 + (int64_t)max(a0, 0) * p.rank + slice * 64) + o;
            const uint32_t* w1 = reinterpret_cast<const uint32_t*>(p.W1 + (int64_t)max(a1, 0) * p.rank + slice * 64) + o;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const uint32_t x0 = a0 >= 0 && active ? __ldg(w0 + 8 * m) : 0, x1 = a1 >= 0 && active ? __ldg(w1 + 8 * m) : 0;
                e[z][2 * m][h] = __byte_perm(x0, x1, 0x5410);
                e[z][2 * m + 1][h] = __byte_perm(x0, x1, 0x7632);
            }
        }
    float acc[kTiles][8][4];
#pragma unroll
    for (int z = 0; z < kTiles; ++z)
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[z][j][q] = 0.0f;

    float4* const chains = reinterpret_cast<float4*>(memory + shared_bytes<kRows>()) + warp * kTiles * 8 * 32 + lane;
    auto end_chain = [&](bool first) {
#pragma unroll
        for (int z = 0; z < kTiles; ++z)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float4 s = make_float4(acc[z][j][0], acc[z][j][1], acc[z][j][2], acc[z][j][3]);
                if (!first) s = plus(chains[(z * 8 + j) * 32], s);
                chains[(z * 8 + j) * 32] = s;
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[z][j][q] = 0.0f;
            }
    };
    unsigned char* const g_at = memory + kWarps * kStages * kStage;
    float* dW2 = p.dW2 + (int64_t)begin * p.rank + slice * 64 + 4 * t;
    const int block = lane >> 3, in_block = lane & 7;
    int k = 0, half = 0;
    for (int base = 0; base < n; base += kChunk, half ^= 1) {
        uint4* g = reinterpret_cast<uint4*>(g_at + half * g_bytes<kRows>());
#pragma unroll
        for (int q = 0; q < kPieces; ++q) {
            const int at = tid + q * kThreads;
            g[at] = token[at % kRows] >= 0 ? x[q] : make_uint4(0, 0, 0, 0);
        }
        load_g(x, base + kChunk);
        __syncthreads();  // (the other half is free: its readers are past it)
        const uint32_t g_s = (uint32_t)__cvta_generic_to_shared(g);
        if (active)
            for (int v0 = 16 * group; v0 < min(kChunk, n - base); v0 += 16 * groups, ++k) {
                if (k > 0 && k % kChain == 0) end_chain(k == kChain);
                copies_wait<kStages - 2>();
                __syncwarp();  // (every lane's copies; and every lane has read the stage that is filled next)
                fetch(k + kStages - 1);
                uint32_t g_rows[kTiles][4], g_cols[kTiles][4];
#pragma unroll
                for (int z = 0; z < kTiles; ++z) {
                    const int row = 16 * z + in_block, oct = v0 / 8;
                    load_blocks(g_rows[z], g_s + (((oct + (block >> 1)) * kRows + row + 8 * (block & 1)) << 4));
                    load_blocks_turned(g_cols[z], g_s + (((oct + (block & 1)) * kRows + row + 8 * (block >> 1)) << 4));
                }
                const uint32_t w = ring + k % kStages * kStage + (in_block + 8 * (block & 1)) * 128;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    uint32_t b[4];
                    load_blocks_turned(b, w + (((2 * m + (block >> 1)) ^ in_block) << 4));
#pragma unroll
                    for (int z = 0; z < kTiles; ++z) {
                        multiply(acc[z][2 * m], g_rows[z], b[0], b[1]);
                        multiply(acc[z][2 * m + 1], g_rows[z], b[2], b[3]);
                    }
                    if (p.dW2) {
                        float d[2][4] = {};
#pragma unroll
                        for (int z = 0; z < kTiles; ++z)
#pragma unroll
                            for (int j = 0; j < 2; ++j) multiply(d[j], g_cols[z], e[z][2 * m + j][0], e[z][2 * m + j][1]);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int v = base + v0 + o + 8 * h;
                            const float4 y = make_float4(d[0][2 * h], d[1][2 * h], d[0][2 * h + 1], d[1][2 * h + 1]);
                            float4* to = reinterpret_cast<float4*>(dW2 + v * p.rank + 16 * m);
                            if (v < n) {
                                if (p.accumulate)
                                    add_to(to, y);
                                else
                                    __stcs(to, y);
                            }
                        }
                    }
                }
            }
    }

    if (k > kChain)
#pragma unroll
        for (int z = 0; z < kTiles; ++z)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float4 s = chains[(z * 8 + j) * 32];
                acc[z][j][0] += s.x;
                acc[z][j][1] += s.y;
                acc[z][j][2] += s.z;
                acc[z][j][3] += s.w;
            }
    // the groups' sums in order, and those of the cluster's CTAs: a half of the columns to each
    copies_wait<0>();
    __syncthreads();  // (W2 and g have been read)
    float* sums = reinterpret_cast<float*>(memory);  // [group][row][column]
    if (active)
#pragma unroll
        for (int z = 0; z < kTiles; ++z)
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<float2*>(sums + (group * kRows + 16 * z + 8 * h + o) * p.rank + slice * 64 + 8 * j + 2 * t) =
                        make_float2(acc[z][j][2 * h], acc[z][j][2 * h + 1]);
    cluster_sync();
    const int rank = (int)cluster_rank(), cluster = blockIdx.x / kCluster, quads = p.rank / 4;
    for (int at = rank * kThreads + tid; at < p.rows * quads; at += kCluster * kThreads) {
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int c = 0; c < kCluster; ++c) {
            const uint32_t from = cluster_map(memory, c) + at * 16;
            for (int i = 0; i < groups; ++i) s = plus(s, cluster_ld_f32x4(from + i * kRows * quads * 16));
        }
        reinterpret_cast<float4*>(part)[(int64_t)cluster * p.rows * quads + at] = s;
    }
    launch_dependents();  // (earlier, and few_join_kernel's CTAs take room on the SMs: 16.9 instead of 15.6 us for 16 rows)
    cluster_sync();  // (no CTA's memory goes while another reads it)
}

// The parts' sums of 64 columns of a row, the same for every row that has its token, which the first of them adds
// to dW1.  A half of a warp to a part, 32 at a time; then the warps' sums in order.
constexpr int kJoinThreads = 512;
__global__ void __launch_bounds__(kJoinThreads) few_join_kernel(const MarkovGradParams p, const float* part, int parts) {
    __shared__ float4 sums[kJoinThreads / 32][16];
    __shared__ int32_t token[kMarkovFewRows];
    const int tid = threadIdx.x, n = blockIdx.y, col = blockIdx.x * 64;
    const int i = tid % 16, group = tid / 16;
    wait_prior_grid();
    if (tid < p.rows) token[tid] = p.prev[tid];
    // (threads 0 to 63: a column each)
    auto sum_of = [&](int m) {
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        constexpr int kGroups = kJoinThreads / 16, kEach = (clusters<16>() + kGroups - 1) / kGroups;
        float4 x[kEach];
#pragma unroll
        for (int q = 0; q < kEach; ++q) {
            const int z = group + q * kGroups;
            x[q] = z < parts ? __ldcg(reinterpret_cast<const float4*>(part + ((int64_t)z * p.rows + m) * p.rank + col) + i)
                             : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int q = 0; q < kEach; ++q) s = plus(s, x[q]);
        const float4 y = make_float4(__shfl_down_sync(~0u, s.x, 16), __shfl_down_sync(~0u, s.y, 16),
                                     __shfl_down_sync(~0u, s.z, 16), __shfl_down_sync(~0u, s.w, 16));
        if ((tid & 31) < 16) sums[tid / 32][i] = plus(s, y);
        __syncthreads();
        float t = 0.0f;
        if (tid < 64)
#pragma unroll
            for (int k = 0; k < kJoinThreads / 32; ++k) t += reinterpret_cast<const float*>(sums[k])[tid];
        __syncthreads();
        return t;
    };
    float s = sum_of(n);
    const int a = token[n];
    if (tid < 64) p.grad_prev[(int64_t)n * p.rank + col + tid] = a < 0 ? 0.0f : a >= p.V ? NAN : s;
    if (!p.dW1 || a < 0 || a >= p.V) return;
    for (int m = 0; m < n; ++m)
        if (token[m] == a) return;
    for (int m = n + 1; m < p.rows; ++m)
        if (token[m] == a) s += sum_of(m);
    if (tid < 64) {
        float* d = p.dW1 + (int64_t)a * p.rank + col + tid;
        *d = p.accumulate ? *d + s : s;
    }
}

int up(int a, int b) { return (a + b - 1) / b; }

template <int kRows>
cudaError_t launch_few(const MarkovGradParams& p, cudaStream_t stream) {
    const int groups = kWarps / (p.rank / 64);  // (a stage for each warp at least)
    const int per = std::max(up(up(p.V, 16), clusters<kRows>() * kCluster), groups) * 16, parts = up(up(p.V, per), kCluster);
    float* part = static_cast<float*>(p.ws);
    const auto kernel = few_kernel<kRows>;
    constexpr int most = shared_bytes<kRows>() + chain_bytes<kRows>();  // (two CTAs of 16 rows still have room on an SM)
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = kCluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(parts * kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = up(per / 16, groups) > kChain ? most : shared_bytes<kRows>();
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    if ((e = cudaLaunchKernelEx(&cfg, kernel, p, per, part)) != cudaSuccess) return e;
    return launch_after(few_join_kernel, dim3(p.rank / 64, p.rows), kJoinThreads, 0, stream, p, part, parts);
}

}  // namespace

size_t markov_few_workspace(int rows, int rank) {
    return (size_t)std::max(clusters<16>() * std::min(rows, 16), clusters<32>() * rows) * rank * sizeof(float);
}

cudaError_t launch_markov_few(const MarkovGradParams& p, cudaStream_t stream) {
    return p.rows <= 16 ? launch_few<16>(p, stream) : launch_few<32>(p, stream);
}

}  // namespace dspark
