// markov_grad.cu -- gradients of the Markov factors from the gradient of the
// drafter's logits.
//
// The drafter's logits of row n are U[n] + W2 . W1[prev[n]], so with g = dL/dlogits
//   grad_prev[n] = sum_v g[n][v] W2[v]            (dL / d W1[prev[n]], of this row)
//   dW1[a]       = sum of grad_prev[n] over the rows with prev[n] = a
//   dW2[v]       = sum_n g[n][v] W1[prev[n]]
// Two products of the same gradient, both on the tensor cores (exact products of
// bf16 values, fp32 sums).  One kernel computes both, tiles of 128 x 256:
//   grad_prev: rows x rank, summed over V.  Few tiles and a long sum, so it is cut
//              into parts; the parts of all tiles go through the same stretch of V at the same
//              time (g and W2 are read from memory about once, then from L2), and
//              join_kernel adds them in order.
//   dW2:       V x rank, summed over the rows: many tiles, each written once.  g's tile
//              is read with V, the contiguous direction, as the product's rows.
// The tensor cores may cut off what lies below the accumulator's last bit, so a
// chain of products ends after 32 of them (512 terms); the epilogue's threads
// hold the tile in registers and add the chains in fp32.  (dW2 of 896 rows against
// 64 bits, relative: 1.2e-6 with chains of 1024 terms, 7e-7 with these, at 1 % of the time.)
// Up to 32 rows, which would leave most of a tile empty, have a kernel of their own (markov_few.cu).
#include <algorithm>

#include "kernels.cuh"
#include "tc_ptx.cuh"

namespace dspark {
namespace {

constexpr int kTileM = 128, kTileN = 256;
constexpr int kBlockK = 64;            // terms of a pipeline stage
constexpr int kChain = 8;              // stages of a chain
constexpr int kGroup = 64 * 64 * 2;    // 64 rows of 128 bytes
constexpr int kABytes = kTileM * kBlockK * 2;
constexpr int kEpilogueWarps = 8;
constexpr int kThreads = 32 * (kEpilogueWarps + 2);
constexpr int kPiece = 32 * 32 * 4;    // 32 rows of 32 sums: what a warp hands to one store
constexpr uint32_t kIdescATransposed = 1u << 15;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kMaxRows = 1 << 19;
constexpr int kGridSms = 152;          // what the parts of a sum are counted for

// A tile of kCtas x 128 rows and 256 columns by kCtas CTAs: each holds its rows of A and
// its part of B's columns.  A CTA of a pair takes 32 KB to a stage where one by itself takes 48
// (512 cycles of products either way, and the way into an SM gives about 62 bytes a cycle).
template <int kCtas>
struct Ring {
    static constexpr int kBBytes = kTileN / kCtas * kBlockK * 2;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kStages = kCtas == 1 ? 4 : 6;
    static constexpr size_t kSmem = kStages * kStageBytes + kEpilogueWarps * kPiece + 1024;
};

struct Product {
    int M, rank;           // rows and columns of the result
    int blocks;            // stages of the whole sum
    int tiles_n, tiles;    // tiles along the columns, in all
    int parts, per;        // parts of a sum, stages in each
    int accumulate;
    const uint8_t* drop;   // rows of g that are to be cleared (dW2)
    int rows;              // of g (dW2)
    int inject;            // 1 (tests): no stage is ever complete
    int32_t* dev_status;
};

struct Barriers {
    uint64_t full[6], empty[6], land[6], tfull[2], tempty[2], drain;
    uint32_t tmem;
    int abort_flag;
    uint32_t has_drop[kMaxRows / kBlockK / 32];  // a bit per stage: some of its rows are to be cleared
};

// ---- what a pair of CTAs does together (a pair's first CTA issues the products of both)
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(dst)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}
// As tc::tma_load_2d into this CTA's memory, counted on a barrier of either CTA (a cluster address).
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
// (nothing is published by it; as a release in the cluster it took 700 cycles)
__device__ __forceinline__ void expect_at(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void arrive_at(uint32_t bar) {  // (what this thread has written is visible to either CTA)
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void arrive_read(uint32_t bar) {  // (for what it has read alone)
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t cluster_address(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ uint32_t pair_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void pair_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void umma_pair_elect(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// As tc::umma_commit_elect, on the barrier at this place in both CTAs.
__device__ __forceinline__ void commit_pair_elect(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            tc::smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// 32 x 32 sums from shared memory to (or added to) columns x.., rows y.. of part z.
__device__ __forceinline__ void store_piece(const CUtensorMap* map, const void* src, int x, int y, int z, int add) {
    if (add)
        asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                         reinterpret_cast<uint64_t>(map)),
                     "r"(tc::smem_u32(src)), "r"(x), "r"(y), "r"(z)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                         reinterpret_cast<uint64_t>(map)),
                     "r"(tc::smem_u32(src)), "r"(x), "r"(y), "r"(z)
                     : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Until the stores of this thread have read their shared memory; until they are done.
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// (acquires what either CTA of a pair has released)
__device__ __forceinline__ bool try_wait(uint64_t* bar, uint32_t parity, uint32_t hint_ns) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity), "r"(hint_ns)
        : "memory");
    return ok != 0;
}
// At most 2 s, or until another thread of the CTA has given up.
static __device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    const uint64_t t0 = global_ns();
    for (;;) {
        if (try_wait(bar, parity, 20000)) return true;
        if (*abort_flag) return false;
        if (global_ns() - t0 > kWaitNs) {
            *abort_flag = 1;
            return false;
        }
    }
}
// (the slow part out of line: in line it took the issue of the products from 100 to 370 cycles each)
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    if (__builtin_expect(try_wait(bar, parity, 0), 1)) return true;
    return wait_slow(bar, parity, abort_flag);
}
// The same for threads whose registers are full (in line: all 128 sums of an epilogue's
// thread were spilled around the call).
__device__ __forceinline__ bool wait_held(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    if (try_wait(bar, parity, 0)) return true;
    const uint64_t t0 = global_ns();
    for (;;) {
        if (try_wait(bar, parity, 20000)) return true;
        if (*abort_flag) return false;
        if (global_ns() - t0 > kWaitNs) {
            *abort_flag = 1;
            return false;
        }
    }
}

// kSumRows: the sum runs over g's rows (dW2), else over V (grad_prev).
template <bool kSumRows, int kCtas>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const Product p, const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ CUtensorMap map_c) {
    using R = Ring<kCtas>;
    constexpr int kStages = R::kStages;
    extern __shared__ unsigned char dyn[];
    __shared__ Barriers sh;
    unsigned char* ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cta = kCtas == 1 ? 0 : (int)pair_rank();
    volatile int* abort_flag = &sh.abort_flag;
    if (warp == kEpilogueWarps + 1) {
        if (kCtas == 1) {
            tc::tmem_alloc(&sh.tmem, 512);
            tc::tmem_relinquish();
        } else {
            tmem_alloc_pair(&sh.tmem, 512);
        }
    } else if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(&sh.full[s], kCtas + p.inject);
            tc::mbar_init(&sh.empty[s], 1);
            tc::mbar_init(&sh.land[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            tc::mbar_init(&sh.tfull[a], 1);
            tc::mbar_init(&sh.tempty[a], kEpilogueWarps * kCtas);
        }
        tc::mbar_init(&sh.drain, 1);
        sh.abort_flag = 0;
        tc::fence_barrier_init();
    }
    tc::tc_fence_before();
    __syncthreads();
    if (kCtas > 1) pair_sync();
    tc::tc_fence_after();
    const uint32_t tmem = sh.tmem;
    wait_prior_grid();
    launch_dependents();
    auto marked = [&](int n) { return n < p.rows && __ldcg(p.drop + n) != 0; };
    if (kSumRows) {
        for (int w = warp; 32 * w < p.blocks; w += kThreads / 32) {
            uint32_t any = 0;
#pragma unroll 8
            for (int k = 32 * w; k < min(32 * w + 32, p.blocks); ++k)
                if (__any_sync(0xFFFFFFFFu, marked(kBlockK * k + lane) || marked(kBlockK * k + 32 + lane))) any |= 1u << (k & 31);
            if (lane == 0) sh.has_drop[w] = any;
        }
        __syncthreads();
    }
    const int units = p.tiles * p.parts, stride = gridDim.x / kCtas;

    // a unit of work: one tile's sum over the stages [k0, k1)
    struct Unit {
        int m0, n0, cols, part, k0, k1;
    };
    auto unit_of = [&](int u) {
        Unit x;
        x.part = u / p.tiles;
        const int t = u - x.part * p.tiles;
        x.m0 = (t / p.tiles_n * kCtas + cta) * kTileM;
        x.n0 = t % p.tiles_n * kTileN;
        // (whole groups of 64 for each CTA; what lies past the rank is zeros, and not written)
        x.cols = min(kTileN, (p.rank - x.n0 + 64 * kCtas - 1) / (64 * kCtas) * (64 * kCtas));
        x.k0 = x.part * p.per;
        x.k1 = min(p.blocks, x.k0 + p.per);
        return x;
    };
    // rows that give nothing and hold a NaN or an infinity: cleared once they have landed.  (Clearing every row without a
    // token instead took dW2 of 2560 rows, 129280 tokens and rank 512 from 264 to 309 us.)
    auto dropped = [&](int k) { return kSumRows && (sh.has_drop[k >> 5] >> (k & 31) & 1u); };
    uint32_t landed = 0;  // parities
    auto clear = [&](int k, int s) {
        uint64_t drop = __ballot_sync(0xFFFFFFFFu, marked(kBlockK * k + lane));
        drop |= (uint64_t)__ballot_sync(0xFFFFFFFFu, marked(kBlockK * k + 32 + lane)) << 32;
        const bool go = __all_sync(0xFFFFFFFFu, wait_bounded(&sh.land[s], landed >> s & 1u, abort_flag));
        landed ^= 1u << s;
        if (go) {
            unsigned char* a = ring + s * R::kStageBytes;
            for (; drop; drop &= drop - 1) {
                const int r = __ffsll((long long)drop) - 1;
                if (lane < 16) *reinterpret_cast<uint4*>(a + (lane >> 3) * kGroup + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive_at(cluster_address(&sh.full[s], 0));
        }
        return go;
    };

    if (warp == kEpilogueWarps) {
        // ---------------------------------------------------------------- loads
        if (lane == 0) {
            tc::prefetch_tmap(&map_a);
            tc::prefetch_tmap(&map_b);
            int i = 0;
            bool go = true;
            for (int u = blockIdx.x / kCtas; go && u < units; u += stride) {
                const Unit x = unit_of(u);
                const int cols = x.cols / kCtas;  // this CTA's
                const uint32_t bytes = kABytes + cols / 64 * kGroup;
                for (int k = x.k0; k < x.k1; ++k, ++i) {
                    const int s = i % kStages;
                    const bool fix = dropped(k);
                    if (i >= kStages && !(go = wait_bounded(&sh.empty[s], (i / kStages - 1) & 1, abort_flag))) break;
                    unsigned char* a = ring + s * R::kStageBytes;
                    unsigned char* b = a + kABytes;
                    // (of a pair, both CTAs' loads are counted by the first, which issues the products)
                    const uint32_t bar = fix ? cluster_address(&sh.land[s], cta) : cluster_address(&sh.full[s], 0);
                    expect_at(bar, bytes);
                    auto load = [&](void* dst, const CUtensorMap* map, int c, int r) {
                        if (kCtas == 1)
                            tc::tma_load_2d(dst, map, fix ? &sh.land[s] : &sh.full[s], c, r);
                        else
                            tma_load_pair(dst, map, bar, c, r);
                    };
                    if (kSumRows) {
                        load(a, &map_a, x.m0, k * kBlockK);
                        load(a + kGroup, &map_a, x.m0 + 64, k * kBlockK);
                    } else {
                        load(a, &map_a, k * kBlockK, x.m0);
                    }
                    for (int c = 0; c < cols; c += 64) load(b + c / 64 * kGroup, &map_b, x.n0 + cta * cols + c, k * kBlockK);
                }
            }
        }
        __syncwarp();
    } else if (warp == kEpilogueWarps + 1) {
        // ---------------------------------------------------------------- products
        int i = 0, chain = 0;
        bool go = true;
        for (int u = blockIdx.x / kCtas; go && u < units; u += stride) {
            const Unit x = unit_of(u);
            if (cta != 0) {  // the other CTA of a pair has rows to clear, at most
                for (int k = x.k0; go && k < x.k1; ++k, ++i) {
                    if (dropped(k)) go = clear(k, i % kStages);
                }
                continue;
            }
            const uint32_t idesc =
                tc::idesc_bf16_f32(kTileM * kCtas, x.cols) | tc::kIdescBTransposed | (kSumRows ? kIdescATransposed : 0u);
            for (int c0 = x.k0; go && c0 < x.k1; c0 += kChain, ++chain) {
                const int buf = chain & 1;
                if (chain >= 2 && !(go = __all_sync(0xFFFFFFFFu, wait_bounded(&sh.tempty[buf], (chain / 2 - 1) & 1, abort_flag)))) break;
                tc::tc_fence_after();
                const uint32_t d = tmem + buf * kTileN;
                const int c1 = min(x.k1, c0 + kChain);
                for (int k = c0; k < c1; ++k, ++i) {
                    const int s = i % kStages;
                    if (dropped(k) && !(go = clear(k, s))) break;
                    if (!(go = __all_sync(0xFFFFFFFFu, wait_bounded(&sh.full[s], (i / kStages) & 1, abort_flag)))) break;
                    tc::tc_fence_after();
                    const uint32_t sa = tc::smem_u32(ring + s * R::kStageBytes);
                    const uint64_t ad = kSumRows ? tc::smem_desc_sw128_mn(sa, kGroup) : tc::smem_desc_sw128(sa);
                    const uint64_t bd = tc::smem_desc_sw128_mn(sa + kABytes, kGroup);
#pragma unroll
                    for (int j = 0; j < kBlockK / 16; ++j) {
                        const uint64_t aj = ad + (uint64_t)(j * ((kSumRows ? 2048 : 32) >> 4)), bj = bd + (uint64_t)(j * (2048 >> 4));
                        if (kCtas == 1)
                            tc::umma_bf16_elect(d, aj, bj, idesc, k > c0 || j > 0);
                        else
                            umma_pair_elect(d, aj, bj, idesc, k > c0 || j > 0);
                    }
                    if (kCtas == 1)
                        tc::umma_commit_elect(&sh.empty[s]);
                    else
                        commit_pair_elect(&sh.empty[s]);
                }
                if (go) {
                    if (kCtas == 1)
                        tc::umma_commit_elect(&sh.tfull[buf]);
                    else
                        commit_pair_elect(&sh.tfull[buf]);
                }
            }
        }
        __syncwarp();
        if (cta == 0) {
            // (whatever ended the loop, the products are done before tensor memory is given back)
            if (kCtas == 1)
                tc::umma_commit_elect(&sh.drain);
            else
                commit_pair_elect(&sh.drain);
        }
        int never = 0;
        wait_bounded(&sh.drain, 0, &never);
    } else {
        // ---------------------------------------------------------------- chains added up, tiles written
        const int quad = warp & 3, half = warp >> 2;
        unsigned char* piece = ring + kStages * R::kStageBytes + warp * kPiece;
        int chain = 0;
        bool go = true;
        for (int u = blockIdx.x / kCtas; go && u < units; u += stride) {
            const Unit x = unit_of(u);
            const int cols = min(128, min(x.cols, p.rank - x.n0) - half * 128);  // (none: only the barriers)
            float acc[128];
#pragma unroll
            for (int e = 0; e < 128; ++e) acc[e] = 0.0f;
            for (int c0 = x.k0; c0 < x.k1; c0 += kChain, ++chain) {
                const int buf = chain & 1;
                if (!(go = __all_sync(0xFFFFFFFFu, wait_held(&sh.tfull[buf], (chain / 2) & 1, abort_flag)))) break;
                tc::tc_fence_after();
                if (cols > 0) {
                    const uint32_t t = tmem + ((uint32_t)(quad * 32) << 16) + buf * kTileN + half * 128;
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        float v[16];
                        tc::tmem_ld_32x32b_x16<0>(t + 16 * q, v);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[16 * q + e] += v[e];
                    }
                }
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_read(cluster_address(&sh.tempty[buf], 0));
            }
            // 32 columns at a time through shared memory (16-byte pieces in the order the store's swizzle
            // undoes), then to memory by one store, which leaves out what lies past the result's rows.  Stores
            // from registers, a row to a thread: dW2 of 896 rows, 151936 tokens and rank 512 took 210 us where it took 136 with these.
            const int row = x.m0 + quad * 32;
            if (go && row < p.M) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (32 * q < cols) {
                        if (lane == 0) bulk_wait_read();
                        __syncwarp();
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *reinterpret_cast<float4*>(piece + lane * 128 + ((e ^ (lane & 7)) << 4)) =
                                make_float4(acc[32 * q + 4 * e], acc[32 * q + 4 * e + 1], acc[32 * q + 4 * e + 2], acc[32 * q + 4 * e + 3]);
                        tc::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) store_piece(&map_c, piece, x.n0 + half * 128 + 32 * q, row, x.part, p.accumulate);
                    }
                }
            }
        }
        if (lane == 0) bulk_wait();
        __syncwarp();
    }
    tc::tc_fence_before();
    __syncthreads();
    if (sh.abort_flag) {
        if (tid == 0) report(p.dev_status, DSPARK_ERR_TIMEOUT);
        const uint64_t t0 = global_ns();  // loads in flight end before their memory goes
        while (global_ns() - t0 < 1000000) {}
    }
    if (kCtas > 1) pair_sync();  // (neither CTA's memory goes while the other's products or arrivals use it)
    tc::tc_fence_after();
    if (warp == kEpilogueWarps + 1) {
        if (kCtas == 1)
            tc::tmem_dealloc(tmem, 512);
        else
            tmem_dealloc_pair(tmem, 512);
    }
}

// ---- the parts of grad_prev: every group of threads adds its own in order, then the groups in order.
// The row's W1 row goes to E, what dW2's products take of it: zeros for a row without a token, which gives
// nothing.  If a NaN or an infinity stands in such a row zeros do not do, and its sums are not all finite: it is
// marked, to be cleared on its way into the products.
constexpr int kJoinThreads = 512;  // at most
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const MarkovGradParams p, const float* part, int parts, uint16_t* E,
                                                            uint8_t* drop) {
    __shared__ float4 sums[kJoinThreads];
    const int n = blockIdx.x, quads = p.rank / 4, groups = blockDim.x / quads;
    const int i = threadIdx.x % quads, g = threadIdx.x / quads;
    wait_prior_grid();
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int z0 = g; z0 < parts; z0 += 4 * groups) {
        float4 x[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int z = z0 + q * groups;
            x[q] = z < parts ? __ldcs(reinterpret_cast<const float4*>(part + ((size_t)z * p.rows + n) * p.rank) + i)
                             : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) s = make_float4(s.x + x[q].x, s.y + x[q].y, s.z + x[q].z, s.w + x[q].w);
    }
    sums[threadIdx.x] = s;
    __syncthreads();
    const int a = p.prev[n];
    const bool there = a >= 0 && a < p.V;
    if (threadIdx.x < p.rank / 8)
        reinterpret_cast<uint4*>(E + (size_t)n * p.rank)[threadIdx.x] =
            there ? __ldg(reinterpret_cast<const uint4*>(p.W1 + (size_t)a * p.rank) + threadIdx.x) : make_uint4(0, 0, 0, 0);
    bool odd = false;
    if (g == 0) {
        for (int o = 1; o < groups; ++o) {
            const float4 x = sums[o * quads + i];
            s = make_float4(s.x + x.x, s.y + x.y, s.z + x.z, s.w + x.w);
        }
        odd = !there && !(fabsf(s.x) < INFINITY && fabsf(s.y) < INFINITY && fabsf(s.z) < INFINITY && fabsf(s.w) < INFINITY);
        if (a < 0) s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (a >= p.V) s = make_float4(NAN, NAN, NAN, NAN);
        reinterpret_cast<float4*>(p.grad_prev + (size_t)n * p.rank)[i] = s;
    }
    odd = __syncthreads_or(odd);
    if (threadIdx.x == 0) {
        drop[n] = odd;
        if (a >= p.V) report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
    }
    launch_dependents();
}

// s + x, and in c what s lacks: the error of a sum of any length stays near 2 u of its terms' magnitudes (u = 2^-24), where
// a plain one's grows with their number.  (An infinity or a NaN stays what it is.)
__device__ __forceinline__ void add_kept(float& s, float& c, float x) {
    const float y = x - c, t = s + y;
    c = fabsf(t) < INFINITY ? (t - s) - y : 0.0f;
    s = t;
}

// ---- dW1: the first row of each previous token adds up all of them, in order (20000 rows of one token, terms of one
// sign: off by 7e-6 of their sum with plain additions, 4e-8 with these).  A row to a warp, up to four of its token's
// rows on their way at once; the tokens are looked through in shared memory, 128 at a time.  Tokens that repeat cost the call
// of 2560 rows, 129280 tokens and rank 512, us: 471 if hardly any does, 517 with one before 5 % of the rows, 555 with a
// language's frequencies (the r-th commonest 1 / r), 1295 with one before all.  Launched after dW2's product, it runs on
// the SMs that the product has left: it may start once the product has itself waited for join_kernel, whose sums are
// all that this needs.  (What others wrote is read from L2: a kernel that has not waited may find older lines in L1.)
constexpr int kScatterRows = 8, kScatterTile = 2048;
__global__ void __launch_bounds__(32 * kScatterRows) scatter_kernel(const MarkovGradParams p) {
    __shared__ int32_t token[kScatterTile];
    const int lane = threadIdx.x & 31, n = blockIdx.x * kScatterRows + (threadIdx.x >> 5);
    if (!p.dW2) wait_prior_grid();
    const int a = n < p.rows ? __ldcg(p.prev + n) : -1;
    bool mine = a >= 0 && a < p.V;  // until an earlier row has the token
    constexpr int kQuads = 4;       // rank <= 512
    constexpr int kAtOnce = 4;      // rows
    float4 s[kQuads], c[kQuads];
#pragma unroll
    for (int q = 0; q < kQuads; ++q) s[q] = c[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int m0 = 0; m0 < p.rows; m0 += kScatterTile) {
        __syncthreads();
        for (int i = threadIdx.x; i < kScatterTile; i += 32 * kScatterRows) token[i] = i < p.rows - m0 ? __ldcg(p.prev + m0 + i) : -1;
        if (!__syncthreads_or(mine)) break;
        for (int i0 = 0; mine && i0 < min(kScatterTile, p.rows - m0); i0 += 128) {
            int t[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) t[z] = token[i0 + 32 * z + lane];
            if (!__any_sync(0xFFFFFFFFu, t[0] == a || t[1] == a || t[2] == a || t[3] == a)) continue;
#pragma unroll 1
            for (int z = 0; mine && z < 4; ++z) {
                const int from = m0 + i0 + 32 * z;
                unsigned same = __ballot_sync(0xFFFFFFFFu, token[i0 + 32 * z + lane] == a);
                if (same && from + __ffs(same) - 1 < n) mine = false;
                while (mine && same) {
                    float4 x[kAtOnce][kQuads];
                    const int rows = min(kAtOnce, __popc(same));
#pragma unroll
                    for (int j = 0; j < kAtOnce; ++j)
                        if (j < rows) {
                            const float4* row = reinterpret_cast<const float4*>(p.grad_prev + (size_t)(from + __ffs(same) - 1) * p.rank);
                            same &= same - 1;
#pragma unroll
                            for (int q = 0; q < kQuads; ++q)
                                if (4 * (lane + 32 * q) < p.rank) x[j][q] = __ldcg(row + lane + 32 * q);
                        }
#pragma unroll
                    for (int j = 0; j < kAtOnce; ++j)
                        if (j < rows)
#pragma unroll
                            for (int q = 0; q < kQuads; ++q)
                                if (4 * (lane + 32 * q) < p.rank) {
                                    add_kept(s[q].x, c[q].x, x[j][q].x);
                                    add_kept(s[q].y, c[q].y, x[j][q].y);
                                    add_kept(s[q].z, c[q].z, x[j][q].z);
                                    add_kept(s[q].w, c[q].w, x[j][q].w);
                                }
                }
            }
        }
    }
    if (mine) {
        float4* d = reinterpret_cast<float4*>(p.dW1 + (size_t)a * p.rank);
#pragma unroll
        for (int q = 0; q < kQuads; ++q)
            if (4 * (lane + 32 * q) < p.rank) {
                float4 y = s[q];
                if (p.accumulate) {
                    const float4 o = __ldcg(d + lane + 32 * q);
                    y = make_float4(o.x + y.x, o.y + y.y, o.z + y.z, o.w + y.w);
                }
                d[lane + 32 * q] = y;
            }
    }
    if (p.dW2) wait_prior_grid();  // (it ends after the product, as what follows it expects)
}

// ------------------------------------------------------------------------------- host
size_t align256(size_t x) { return (x + 255) / 256 * 256; }
int up(int a, int b) { return (a + b - 1) / b; }

// CTAs to a tile of grad_prev: a pair where there are rows for both.
int ctas_of(int rows) { return rows > kTileM ? 2 : 1; }

// How many parts the sum over V is cut into: the fewest cycles of the busiest SM,
// a stage counted as 540 cycles (of a pair) or 775, and a part's way to memory and back
// as its bytes at 23 a cycle and SM.
int parts_of(int rows, int V, int rank) {
    const int ctas = ctas_of(rows), slots = kGridSms / ctas;
    const int tiles = up(rows, kTileM * ctas) * up(rank, kTileN), blocks = up(V, kBlockK);
    double best = 0;
    int parts = 1;
    for (int n = 1; n <= std::min(blocks, kGridSms); ++n) {
        const double steps = (double)up(tiles * n, slots) * (up(blocks, n) * (ctas == 2 ? 540.0 : 775.0) + 3000.0);
        const double moved = (double)n * rows * rank * 8.0 / (23.0 * kGridSms);
        if (n == 1 || steps + moved < best) {
            best = steps + moved;
            parts = n;
        }
    }
    return up(blocks, up(blocks, parts));
}

struct Layout {
    size_t E, drop, part, total;
    int parts;
};
Layout layout_of(int rows, int V, int rank) {
    Layout L;
    size_t off = 0;
    L.E = off; off += align256((size_t)rows * rank * 2);
    L.drop = off; off += align256((size_t)rows);
    L.parts = parts_of(rows, V, rank);
    L.part = off; off += align256((size_t)L.parts * rows * rank * 4);
    L.total = std::max<size_t>(off, 256);
    if (rows <= kMarkovFewRows) L.total = std::max(L.total, markov_few_workspace(rows, rank));
    return L;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
    static const EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<EncodeTiled>(f) : nullptr;
    }();
    return fn;
}

// Boxes of 64 columns and `box_rows` rows of a bf16 matrix; zeros outside it.
bool encode(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t stride, int box_rows) {
    const EncodeTiled enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    const cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Boxes of 32 columns and 32 rows of [parts][rows][cols] fp32.
bool encode_sums(CUtensorMap* m, const void* base, int cols, int rows, int parts) {
    const EncodeTiled enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)parts};
    const cuuint64_t strides[2] = {(cuuint64_t)cols * 4, (cuuint64_t)cols * 4 * rows};
    const cuuint32_t box[3] = {32, 32, 1};
    const cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kSumRows, int kCtas>
cudaError_t launch_product(Product p, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c, int n_sm,
                           cudaStream_t stream) {
    p.tiles_n = up(p.rank, kTileN);
    p.tiles = up(p.M, kTileM * kCtas) * p.tiles_n;
    p.per = up(p.blocks, p.parts);
    const auto kernel = product_kernel<kSumRows, kCtas>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Ring<kCtas>::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = kCtas;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(std::min(n_sm / kCtas, p.tiles * p.parts) * kCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Ring<kCtas>::kSmem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p, a, b, c);
}

}  // namespace

size_t markov_grad_workspace(int rows, int V, int rank) { return layout_of(rows, V, rank).total; }

// Fewer rows are cut into more parts, and may take more room than many.  Rows of as many tiles: the fewest have the most
// parts (a part's way to memory, which is what grows with them, counts against its number).
size_t markov_grad_workspace_up_to(int rows, int V, int rank) {
    size_t part = 0;
    for (int n = 1; n <= std::min(rows, kMarkovFewRows); ++n) part = std::max(part, (size_t)parts_of(n, V, rank) * n);
    for (int low = kMarkovFewRows + 1; low <= rows;) {
        const int tile = kTileM * ctas_of(low), high = std::min(rows, up(low, tile) * tile);
        part = std::max(part, (size_t)std::max(parts_of(low, V, rank), parts_of(high, V, rank)) * high);
        low = high + 1;
    }
    const size_t total = align256((size_t)rows * rank * 2) + align256((size_t)rows) + align256(part * rank * 4);
    return std::max({total, markov_few_workspace(std::min(rows, kMarkovFewRows), rank), (size_t)256});
}

cudaError_t launch_markov_grad(const MarkovGradParams& p, cudaStream_t stream) {
    if (p.rows == 0) {
        if (!p.dW2 || p.accumulate) return cudaSuccess;
        return cudaMemsetAsync(p.dW2, 0, (size_t)p.V * p.rank * sizeof(float), stream);
    }
    // (what a test injects is in the products' waits)
    if (p.rows <= kMarkovFewRows && !p.inject) return launch_markov_few(p, stream);
    int dev = 0, n_sm = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const Layout L = layout_of(p.rows, p.V, p.rank);
    unsigned char* w = static_cast<unsigned char*>(p.ws);
    uint16_t* E = reinterpret_cast<uint16_t*>(w + L.E);
    float* part = reinterpret_cast<float*>(w + L.part);
    const int parts = L.parts;
    const int64_t stride = p.rows > 1 ? p.stride : p.V;
    CUtensorMap g_rows, g_cols, w2, before, sums, dW2;
    if (!encode(&g_rows, p.grad, p.V, p.rows, stride, kTileM) || !encode(&g_cols, p.grad, p.V, p.rows, stride, kBlockK) ||
        !encode(&w2, p.W2, p.rank, p.V, p.rank, kBlockK) || !encode(&before, E, p.rank, p.rows, p.rank, kBlockK) ||
        !encode_sums(&sums, part, p.rank, p.rows, parts) || (p.dW2 && !encode_sums(&dW2, p.dW2, p.rank, p.V, 1)))
        return cudaErrorInvalidValue;
    Product q{};
    q.rank = p.rank;
    q.dev_status = p.dev_status;
    q.inject = p.inject;
    q.M = p.rows; q.blocks = up(p.V, kBlockK); q.parts = parts;
    e = ctas_of(p.rows) == 2 ? launch_product<false, 2>(q, g_rows, w2, sums, n_sm, stream)
                            : launch_product<false, 1>(q, g_rows, w2, sums, n_sm, stream);
    if (e != cudaSuccess) return e;
    // (groups of threads, four parts each)
    const int quads = p.rank / 4, groups = std::min(std::max(parts / 4, 1), kJoinThreads / quads);
    uint8_t* drop = w + L.drop;
    if ((e = launch_after(join_kernel, dim3(p.rows), quads * groups, 0, stream, p, part, parts, E, drop)) != cudaSuccess) return e;
    if (p.dW2) {
        q.M = p.V; q.blocks = up(p.rows, kBlockK); q.parts = 1; q.accumulate = p.accumulate;
        q.drop = drop; q.rows = p.rows;
        if ((e = launch_product<true, 2>(q, g_cols, before, dW2, n_sm, stream)) != cudaSuccess) return e;
    }
    if (p.dW1 && (e = launch_after(scatter_kernel, dim3(up(p.rows, kScatterRows)), 32 * kScatterRows, 0, stream, p)) != cudaSuccess) return e;
    return cudaSuccess;
}

}  // namespace dspark
