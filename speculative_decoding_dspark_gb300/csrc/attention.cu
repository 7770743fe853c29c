// attention.cu -- attention of packed verify rows over the paged KV cache, with
// or without leading pages that groups of requests share.
//
// Row i of request r (row cu[r] + i of q) stands at position kv_len[r] + i.
// With g = hq / hkv query heads to a key head, s_j = scale * q . K[j] over the
// keys j it sees (j <= kv_len + i, or every j < kv_len + n in a full block):
//   out = sum_j e^{s_j - lse} V[j],   lse = log sum_j e^{s_j}
// A sum over any part of the keys is a triple (m, l, O): a reference exponent,
// sum_j 2^{x_j - m} and sum_j 2^{x_j - m} V[j] with x = s log2(e); triples of
// disjoint parts add up after scaling each by 2^{m - max m}.
//
// An item is 128 rows of one key head: the rows of a request (of a group, over
// its shared pages) by query heads of that key head, so that a key read once
// serves them all.  Its keys go by in blocks of 128:
//   S = Q K^T     tcgen05, 128 x 128, fp32 in tensor memory
//   P = 2^(x - m) one thread a row: the row's maximum, 128 exponentials, the
//                 sum; P goes back to tensor memory in bf16 over S
//   O += P V      tcgen05 with P from tensor memory, 128 x d, fp32
// The reference m of a row moves only when the maximum has grown by more than
// 2^8 (O is rescaled then): P stays below 2^8 and fp32 sums lose nothing.
// P is the one rounding to fewer bits besides the output: 2^-8 of each weight
// at most, and l adds the weights before it.
//
// Splitting: the blocks of all items form one line, which is cut into equal
// pieces, one per CTA (two CTAs per SM; each item costs a block more, for its
// queries and output).  An item that is cut leaves (m, l, O) in the workspace
// and a second kernel joins its pieces in their order.  The cut depends on the
// lengths, which only the device knows: every CTA scans them itself.
#include "kernels.cuh"
#include "tc_ptx.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = 128;   // rows of an item
constexpr int kBlock = 128;  // keys of a block
constexpr int kItemCost = 1;
constexpr int kMaxCtas = 304;            // two per SM
constexpr uint32_t kNoSlot = 0xFFFFFFFFu;
constexpr float kGrowth = 8.0f;
constexpr uint64_t kWaitNs = 2000000000ull;  // of a CTA on its own tensor-core operations
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------- the plan
// Workspace of one launch: where each entry's (request's or group's) work
// begins on the line, and the pieces of items that were cut.
struct Plan {
    int* bad;            // cu or group_start is not what it has to be
    long long* start;    // [entries + 1]
    float* part;         // [2 * ctas][kTile][d]  slot 2c: the item cut before CTA c's piece, 2c + 1: after it
    float2* part_ml;     // [2 * ctas][kTile]
    float* whole;        // groups only, [rows, hq, d]: items that were not cut
    float2* whole_ml;    // [rows, hq]
};

struct Entry {     // a request's own keys, or a group's shared ones
    int row0, n;   // its rows of q (0: nothing to do)
    int begin;     // first key
    int end;       // past the last key any of its rows sees
    int len;       // causal: row i sees keys below len + i + 1
    int causal;
    int table;     // the block table's row
    int tiles, blocks;
    __device__ long long items(int hkv) const { return (long long)tiles * hkv; }
    __device__ long long cost(int hkv) const { return items(hkv) * (blocks + kItemCost); }
    // past the last key seen by row i of the entry
    __device__ int limit(int i) const { return causal ? len + i + 1 : end; }
};

__device__ __forceinline__ int group_of(const AttnParams& p, int r) {
    int lo = 0, hi = p.n_groups;  // the last group that starts at or before r
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.group_start[mid] <= r) lo = mid; else hi = mid;
    }
    return lo;
}

// Keys below which request r's are shared (0 without groups); -1: its group's length is bad.
__device__ __forceinline__ int shared_of(const AttnParams& p, int r) {
    if (p.n_groups == 0) return 0;
    const int s = p.shared_len[group_of(p, r)];
    return s >= 0 && s % p.page == 0 ? s : -1;
}

__device__ __forceinline__ bool request_ok(const AttnParams& p, int len, int n, int shared) {
    return len >= 0 && shared >= 0 && shared <= len && (long long)len + n <= (long long)p.max_blocks * p.page &&
           (long long)len + n < (1LL << 31) - kBlock;
}

template <bool kGroups>
__device__ __forceinline__ Entry entry_of(const AttnParams& p, int e) {
    Entry x;
    x.causal = 0;
    x.begin = 0;
    if (kGroups) {
        const int r0 = p.group_start[e], r1 = p.group_start[e + 1];
        const int s = p.shared_len[e];
        x.table = r0;
        x.row0 = p.cu[r0];
        x.n = p.cu[r1] - x.row0;
        x.len = x.end = s;
        if (s <= 0 || s % p.page || (long long)s > (long long)p.max_blocks * p.page || s >= INT_MAX - kBlock) x.n = 0;
    } else {
        const int lo = p.cu[e], n = p.cu[e + 1] - lo, len = p.kv_len[e];
        const int shared = shared_of(p, e);
        x.table = e;
        x.row0 = lo;
        x.n = request_ok(p, len, n, shared) ? n : 0;
        x.begin = shared;
        x.len = len;
        x.end = len + n;
        x.causal = !p.full_block;
    }
    if (x.n <= 0) {
        x.n = x.tiles = x.blocks = 0;
    } else {
        x.tiles = (int)(((long long)x.n * (p.hq / p.hkv) + kTile - 1) / kTile);
        x.blocks = (x.end - x.begin + kBlock - 1) / kBlock;
    }
    return x;
}

// Blocks of tile t of an entry that some row of it sees.
__device__ __forceinline__ int tile_blocks(const Entry& x, int t, int g) {
    const long long last = ((long long)t * kTile + kTile - 1) / g;
    const int i = last < x.n - 1 ? (int)last : x.n - 1;
    return (x.limit(i) - x.begin + kBlock - 1) / kBlock;
}

// Pieces the line is cut into: each has a unit at least.
__device__ __forceinline__ int pieces(long long total, int ctas) { return total < ctas ? (int)total : ctas; }

// The CTA whose piece of the line [total * c / ctas, total * (c + 1) / ctas) holds unit u.
__device__ __forceinline__ int cta_of(long long u, long long total, int ctas) {
    return (int)(((u + 1) * ctas - 1) / total);
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---------------------------------------------------------------- the kernel
template <int kD>
struct Smem {
    static constexpr int kHalf = kTile * 128;           // 128 rows of 64 elements, 128-byte swizzle
    static constexpr int kOperand = kD / 64 * kHalf;    // Q, K or V
    static constexpr int kTotal = 3 * kOperand + 1024;  // (the operands start on a 1024-byte boundary)
};

// 16-byte chunk c of row r of an operand tile.
__device__ __forceinline__ uint32_t chunk_offset(int r, int c) {
    return (uint32_t)((c >> 3) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

template <int kD, bool kGroups>
__global__ void __launch_bounds__(kThreads, 2) attention_kernel(const AttnParams p, const Plan plan, const int max_ctas,
                                                               const int entries) {
    constexpr int kChunks = kD / 8;
    constexpr uint32_t kTmemO = kBlock;  // columns: S (and P over it) 0 .. 127, O 128 .. 128 + d
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t bar_s, bar_o;
    __shared__ uint32_t tmem_base_smem;
    __shared__ volatile int abort_flag;
    __shared__ int bad_page[2];  // of this piece and the next
    __shared__ uint32_t slots[2][kBlock];   // cache rows of the keys of two blocks
    __shared__ uint32_t odd_keys[kBlock / 32];  // keys with a value that is not finite
    __shared__ long long scan_sum[kThreads / 32];
    __shared__ long long first_start;
    __shared__ int first_entry;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = p.hq / p.hkv;
    unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sQ = tc::smem_u32(base), sK = sQ + Smem<kD>::kOperand, sV = sK + Smem<kD>::kOperand;

    // ---- the line of all items' blocks, and this CTA's piece of it
    int bad = 0;
    if (tid == 0) {
        bad = p.cu[0] != 0 || p.cu[p.R] > p.rows;
        if (p.n_groups) bad |= p.group_start[0] != 0 || p.group_start[p.n_groups] != p.R;
    }
    for (int r = tid; r < p.R; r += kThreads) bad |= p.cu[r] > p.cu[r + 1];
    for (int e = tid; e < p.n_groups; e += kThreads) bad |= p.group_start[e] > p.group_start[e + 1];
    if (tid == 0) { abort_flag = 0; bad_page[0] = bad_page[1] = 0; first_entry = -1; }
    bad = __syncthreads_or(bad);
    if (blockIdx.x == 0 && tid == 0) *plan.bad = bad;
    if (bad) return;  // (the joining kernel marks the rows)
    const int per = (entries + kThreads - 1) / kThreads;
    const int e0 = min(entries, tid * per), e1 = min(entries, e0 + per);
    long long mine = 0;
    for (int e = e0; e < e1; ++e) mine += entry_of<kGroups>(p, e).cost(p.hkv);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) scan_sum[warp] = incl;
    __syncthreads();
    long long before = incl - mine, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += scan_sum[w];
        total += scan_sum[w];
    }
    const int ctas = pieces(total, max_ctas);
    long long x = total, x1 = total;
    if (blockIdx.x < ctas) {
        x = total * blockIdx.x / ctas;
        x1 = total * (blockIdx.x + 1) / ctas;
    }
    if (blockIdx.x == 0) {
        long long at = before;
        for (int e = e0; e < e1; ++e) {
            plan.start[e] = at;
            at += entry_of<kGroups>(p, e).cost(p.hkv);
        }
        if (tid == 0) plan.start[entries] = total;
    }
    if (x >= before && x < before + mine) {
        long long at = before;
        for (int e = e0; e < e1; ++e) {
            const long long c = entry_of<kGroups>(p, e).cost(p.hkv);
            if (x < at + c) {
                first_entry = e;
                first_start = at;
                break;
            }
            at += c;
        }
    }
    if (tid == 0) {
        tc::mbar_init(&bar_s, 1);
        tc::mbar_init(&bar_o, 1);
        tc::fence_barrier_init();
    }
    __syncthreads();
    if (x >= x1) return;  // (less work than CTAs)
    if (warp == 0) {
        tc::tmem_alloc(&tmem_base_smem, 256);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = tmem_base_smem;
    const uint32_t my_tmem = tmem + ((uint32_t)(warp * 32) << 16);
    uint32_t phase_s = 0, phase_o = 0;
    int turn = 0;
    const float sl2 = p.scale * kLog2e;

    int e = first_entry;
    long long e_start = first_start;
    Entry en = entry_of<kGroups>(p, e);
    while (x < x1) {
        while (x >= e_start + en.cost(p.hkv)) {  // (entries without work cost nothing)
            e_start += en.cost(p.hkv);
            en = entry_of<kGroups>(p, ++e);
        }
        const long long item_cost = en.blocks + kItemCost;
        const int item = (int)((x - e_start) / item_cost);
        const long long s0 = e_start + item * item_cost;
        const int h = item / en.tiles, t = item - h * en.tiles;
        const int n_blocks = tile_blocks(en, t, g);
        const int b0 = (int)max(x - s0 - kItemCost, 0LL);
        const int b1 = (int)min(min(x1, s0 + item_cost) - s0 - kItemCost, (long long)n_blocks);
        x = s0 + item_cost;
        if (b0 >= b1) continue;

        // ---- one piece: blocks [b0, b1) of tile t of key head h
        const long long r_tile = (long long)t * kTile;
        const int n_rows = (int)min((long long)en.n * g - r_tile, (long long)kTile);
        const bool live = tid < n_rows;
        const bool warp_live = warp * 32 < n_rows;
        const int my_i = live ? (int)((r_tile + tid) / g) : 0;
        const long long my_row = (long long)(en.row0 + my_i) * p.hq + h * g + (live ? (int)((r_tile + tid) - (long long)my_i * g) : 0);
        const int my_limit = live ? en.limit(my_i) : en.limit(0);
        const int low_limit = en.limit((int)(r_tile / g));  // of the tile's first row
        const int high_limit = en.limit((int)((r_tile + n_rows - 1) / g));

        // the cache row of key `tid` of block b
        auto slot_of = [&](int b) -> uint32_t {
            const int pos = en.begin + b * kBlock + tid;
            if (b >= b1 || pos >= high_limit) return kNoSlot;
            const int pb = pos / p.page;
            const int id = p.block_table[(long long)en.table * p.max_blocks + pb];
            if (id < 0 || id >= p.pool_pages) {
                bad_page[turn] = 1;
                return kNoSlot;
            }
            return ((uint32_t)id * p.hkv + h) * p.page + (pos - pb * p.page);
        };
        auto load_block = [&](uint32_t dst, const __nv_bfloat16* cache, const uint32_t* from) {
#pragma unroll 4
            for (int i = 0; i < kBlock * kChunks / kThreads; ++i) {
                const int idx = i * kThreads + tid, r = idx / kChunks, c = idx % kChunks;
                const uint32_t s = from[r];
                tc::cp_async_16(dst + chunk_offset(r, c), cache + (size_t)(s == kNoSlot ? 0 : s) * kD + c * 8,
                                s == kNoSlot ? 0 : 16);
            }
        };

        slots[b0 & 1][tid] = slot_of(b0);
        slots[(b0 + 1) & 1][tid] = slot_of(b0 + 1);
        for (int idx = tid; idx < n_rows * kChunks; idx += kThreads) {
            const int r = idx / kChunks, c = idx % kChunks;
            const int i = (int)((r_tile + r) / g);
            const size_t row = (size_t)(en.row0 + i) * p.hq + h * g + ((r_tile + r) - (long long)i * g);
            tc::cp_async_16(sQ + chunk_offset(r, c), p.q + row * kD + c * 8, 16);
        }
        __syncthreads();
        load_block(sK, p.k_cache, slots[b0 & 1]);
        tc::cp_async_commit();

        float m = -INFINITY, l = 0.0f;  // m in raw scores
        for (int b = b0; b < b1; ++b) {
            const int key0 = en.begin + b * kBlock;
            // K of this block has arrived; every thread is done with the last S
            tc::cp_async_wait<0>();
            tc::fence_proxy_async_smem();
            tc::tc_fence_before();
            __syncthreads();
            if (warp == 0) {
                tc::tc_fence_after();
                constexpr uint32_t idesc = tc::idesc_bf16_f32(kTile, kBlock);
                const uint64_t qd = tc::smem_desc_sw128(sQ), kd = tc::smem_desc_sw128(sK);
#pragma unroll
                for (int k = 0; k < kD / 16; ++k) {
                    const uint64_t step = (uint64_t)((k >> 2) * (Smem<kD>::kHalf >> 4) + (k & 3) * 2);
                    tc::umma_bf16_elect(tmem, qd + step, kd + step, idesc, k != 0);
                }
                tc::umma_commit_elect(&bar_s);
            }
            // V's buffer is free once the last block's product is done
            if (b > b0) {
                tc::mbar_wait(&bar_o, phase_o, &abort_flag, kWaitNs);
                phase_o ^= 1;
            }
            load_block(sV, p.v_cache, slots[b & 1]);
            tc::cp_async_commit();
            tc::mbar_wait(&bar_s, phase_s, &abort_flag, kWaitNs);
            phase_s ^= 1;
            tc::tc_fence_after();
            if (b + 1 < b1) load_block(sK, p.k_cache, slots[(b + 1) & 1]);
            tc::cp_async_commit();
            const uint32_t next_slot = slot_of(b + 2);

            __syncwarp();
            if (warp_live) {
                float s[kBlock];
                tc::tmem_ld_32x32b_x32<0>(my_tmem, s);
                tc::tmem_ld_32x32b_x32<32>(my_tmem + 32, s);
                tc::tmem_ld_32x32b_x32<64>(my_tmem + 64, s);
                tc::tmem_ld_32x32b_x32<96>(my_tmem + 96, s);
                tc::tmem_ld_wait();
                const int seen = my_limit - key0;  // keys of the block this row sees
                const bool whole = __all_sync(0xFFFFFFFFu, seen >= kBlock);
                if (!whole) {
#pragma unroll
                    for (int j = 0; j < kBlock; ++j) s[j] = j < seen ? s[j] : -INFINITY;
                }
                float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int j = 4; j < kBlock; ++j) top[j & 3] = fmaxf(top[j & 3], s[j]);
                const float mb = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                // move the reference when the maximum has grown by more than 2^kGrowth
                const bool move = mb > m && !((mb - m) * sl2 <= kGrowth);
                if (__any_sync(0xFFFFFFFFu, move)) {
                    const float f = !move ? 1.0f : m == -INFINITY ? 0.0f : exp2_approx((m - mb) * sl2);
                    if (move) m = mb;
                    l *= f;
                    if (b > b0) {
#pragma unroll 1
                        for (int c = 0; c < kD; c += 16) {
                            float o[16];
                            uint32_t u[16];
                            tc::tmem_ld_32x32b_x16<0>(my_tmem + kTmemO + c, o);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j) u[j] = __float_as_uint(o[j] * f);
                            tc::tmem_st_32x32b_x16<0>(my_tmem + kTmemO + c, u);
                        }
                    }
                }
                const float ref = m == -INFINITY ? 0.0f : m * sl2;
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < kBlock; c += 32) {
                    uint32_t u[16];
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        float a = exp2_approx(fmaf(s[c + j], sl2, -ref)), d = exp2_approx(fmaf(s[c + j + 1], sl2, -ref));
                        if (!whole) {
                            a = c + j < seen ? a : 0.0f;
                            d = c + j + 1 < seen ? d : 0.0f;
                        }
                        sum[(j >> 1) & 1] += a;
                        sum[2 + ((j >> 1) & 1)] += d;
                        const __nv_bfloat162 w = __floats2bfloat162_rn(a, d);
                        u[j >> 1] = *reinterpret_cast<const uint32_t*>(&w);
                    }
                    tc::tmem_st_32x32b_x16<0>(my_tmem + c / 2, u);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tc::tmem_st_wait();
            }
            // V of this block has arrived (the next K may be on its way)
            tc::cp_async_wait<1>();
            int odd = 0;
            if (low_limit < high_limit && key0 + kBlock > low_limit) {
                // some row does not see all of these keys: a value that is not finite must not reach
                // it through a zero weight.  Such keys are taken out here and added by hand below.
                if (tid < kBlock / 32) odd_keys[tid] = 0;
                __syncthreads();
                const int key = tid;
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    const uint4 w = *reinterpret_cast<const uint4*>(base + 2 * Smem<kD>::kOperand + chunk_offset(key, c));
                    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        odd |= (v[j] & 0x7F80u) == 0x7F80u || (v[j] & 0x7F800000u) == 0x7F800000u;
                }
                if (odd) {
                    atomicOr(&odd_keys[key >> 5], 1u << (key & 31));
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        *reinterpret_cast<uint4*>(base + 2 * Smem<kD>::kOperand + chunk_offset(key, c)) = make_uint4(0, 0, 0, 0);
                }
                odd = __syncthreads_or(odd);
            }
            tc::fence_proxy_async_smem();
            tc::tc_fence_before();
            __syncthreads();
            if (warp == 0) {
                tc::tc_fence_after();
                constexpr uint32_t idesc = tc::idesc_bf16_f32(kTile, kD) | tc::kIdescBTransposed;
                const uint64_t vd = tc::smem_desc_sw128_mn(sV, Smem<kD>::kHalf);
#pragma unroll
                for (int k = 0; k < kBlock / 16; ++k)
                    tc::umma_bf16_ta_elect(tmem + kTmemO, tmem + 8 * k, vd + (uint64_t)(k * (2048 >> 4)), idesc,
                                           b != b0 || k != 0);
                tc::umma_commit_elect(&bar_o);
            }
            if (odd) {
                tc::mbar_wait(&bar_o, phase_o, &abort_flag, kWaitNs);  // (waited for again: the phase stays)
                tc::tc_fence_after();
                __syncwarp();
                if (warp_live) {
                    for (int key = 0; key < kBlock; ++key) {
                        if (!(odd_keys[key >> 5] >> (key & 31) & 1)) continue;
                        const uint32_t pair = tc::tmem_ld_32x32b_x1(my_tmem + key / 2);
                        tc::tmem_ld_wait();
                        const float w = __uint_as_float(key & 1 ? pair & 0xFFFF0000u : pair << 16);
                        const __nv_bfloat16* v = p.v_cache + (size_t)slots[b & 1][key] * kD;
                        for (int c = 0; c < kD; c += 16) {
                            float o[16];
                            uint32_t u[16];
                            tc::tmem_ld_32x32b_x16<0>(my_tmem + kTmemO + c, o);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                u[j] = __float_as_uint(key0 + key < my_limit ? fmaf(w, __bfloat162float(v[c + j]), o[j]) : o[j]);
                            tc::tmem_st_32x32b_x16<0>(my_tmem + kTmemO + c, u);
                        }
                    }
                    tc::tmem_st_wait();
                }
                tc::tc_fence_before();
            }
            if (odd) __syncthreads();  // (the slots were read)
            slots[b & 1][tid] = next_slot;
        }
        tc::mbar_wait(&bar_o, phase_o, &abort_flag, kWaitNs);
        phase_o ^= 1;
        tc::tc_fence_after();
        __syncthreads();  // (bad_page, slots)
        if (tid == 0) bad_page[turn ^ 1] = 0;

        // ---- the piece's triple
        const bool spoiled = bad_page[turn] != 0 || abort_flag != 0;
        if (spoiled && tid == 0) report(p.dev_status, abort_flag ? DSPARK_ERR_TIMEOUT : DSPARK_ERR_DEVICE_INPUT);
        if (spoiled) l = __int_as_float(0x7FC00000);
        const bool uncut = b0 == 0 && b1 == n_blocks;
        if (warp_live) {
            const float m2 = m == -INFINITY ? -INFINITY : m * sl2;
            const int slot = 2 * blockIdx.x + (b0 == 0);
            const bool final = !kGroups && uncut && p.n_groups == 0;
            float* to = uncut ? plan.whole + my_row * kD : plan.part + ((size_t)slot * kTile + tid) * kD;
            const float inv = 1.0f / l;
#pragma unroll 1
            for (int c = 0; c < kD; c += 32) {
                float o[32];
                tc::tmem_ld_32x32b_x32<0>(my_tmem + kTmemO + c, o);
                tc::tmem_ld_wait();
                if (live && final) {
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        __nv_bfloat162 w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            w[i] = __floats2bfloat162_rn(o[j + 2 * i] * inv, o[j + 2 * i + 1] * inv);
                        *reinterpret_cast<uint4*>(p.out + my_row * kD + c + j) = *reinterpret_cast<const uint4*>(w);
                    }
                } else if (live) {
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        *reinterpret_cast<float4*>(to + c + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                }
                __syncwarp();
            }
            if (live) {
                if (!final) (uncut ? plan.whole_ml[my_row] : plan.part_ml[(size_t)slot * kTile + tid]) = make_float2(m2, l);
                else if (p.lse) p.lse[my_row] = (m2 + log2f(l)) * kLn2;
            }
        }
        tc::tc_fence_before();
        __syncthreads();
        tc::tc_fence_after();
        turn ^= 1;
    }
    __syncthreads();
    if (warp == 0) tc::tmem_dealloc(tmem, 256);
}

// ---------------------------------------------------------------- joining the pieces
constexpr int kJoinThreads = 256;

struct Joined {
    float m, l;
    float o[4];
};

// Adds the pieces of the row's item over one entry's keys, in their order.  Lane i holds d / 32 elements.
template <int kD, bool kGroups>
__device__ __forceinline__ void join_entry(const AttnParams& p, const Plan& plan, int max_ctas, int entries, int e, int row,
                                           int head, Joined& a) {
    constexpr int kPer = kD / 32;
    const int lane = threadIdx.x & 31, g = p.hq / p.hkv;
    const Entry x = entry_of<kGroups>(p, e);
    if (x.n == 0) return;
    const int h = head / g;
    const long long at = (long long)(row - x.row0) * g + (head - h * g);
    const int t = (int)(at / kTile), r = (int)(at % kTile);
    const long long s0 = plan.start[e] + ((long long)h * x.tiles + t) * (x.blocks + kItemCost) + kItemCost;
    const int n_blocks = tile_blocks(x, t, g);
    const long long total = plan.start[entries];
    const int ctas = pieces(total, max_ctas);
    const int c0 = cta_of(s0, total, ctas), c1 = cta_of(s0 + n_blocks - 1, total, ctas);
    for (int c = c0; c <= c1; ++c) {
        const long long item = (long long)row * p.hq + head;
        const long long slot = (long long)(2 * c + (c == c0)) * kTile + r;
        const float2 ml = c0 == c1 ? plan.whole_ml[item] : plan.part_ml[slot];
        const float* from = (c0 == c1 ? plan.whole + item * kD : plan.part + slot * kD) + lane * kPer;
        float o[4];
        if (kPer == 4) *reinterpret_cast<float4*>(o) = *reinterpret_cast<const float4*>(from);
        else *reinterpret_cast<float2*>(o) = *reinterpret_cast<const float2*>(from);
        const float top = fmaxf(a.m, ml.x);
        const float fa = a.m == -INFINITY ? 0.0f : exp2f(a.m - top);
        const float fb = ml.x == -INFINITY && ml.y == 0.0f ? 0.0f : exp2f(ml.x - top);
        a.m = top;
        a.l = a.l * fa + ml.y * fb;
#pragma unroll
        for (int i = 0; i < kPer; ++i) a.o[i] = a.o[i] * fa + o[i] * fb;
    }
}

// One warp per (row, query head): rows whose item was cut, or that have a
// shared part, get their sums; rows of requests that cannot be right get NaN.
template <int kD>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const AttnParams p, const Plan plan, const Plan shared_plan,
                                                           const int max_ctas) {
    constexpr int kPer = kD / 32;
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
    if (item >= (long long)p.rows * p.hq) return;
    const int row = (int)(item / p.hq), head = (int)(item % p.hq), g = p.hq / p.hkv;
    bool ok = *plan.bad == 0;
    if (!ok && item == 0 && lane == 0) report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
    Joined a{-INFINITY, 0.0f, {0.0f, 0.0f, 0.0f, 0.0f}};
    if (ok) {
        if (row >= p.cu[p.R]) return;
        const int r = owner_of(p.cu, p.R, row);
        const Entry x = entry_of<false>(p, r);
        if (x.n == 0) {  // a length, or its group, is bad
            ok = false;
            if (lane == 0) report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
        } else {
            if (p.n_groups == 0) {
                const long long at = (long long)(row - x.row0) * g + head % g;
                const int t = (int)(at / kTile);
                const long long s0 = plan.start[r] + ((long long)(head / g) * x.tiles + t) * (x.blocks + kItemCost) + kItemCost;
                const long long total = plan.start[p.R];
                const int ctas = pieces(total, max_ctas);
                if (cta_of(s0, total, ctas) == cta_of(s0 + tile_blocks(x, t, g) - 1, total, ctas)) return;  // not cut
            } else {
                join_entry<kD, true>(p, shared_plan, max_ctas, p.n_groups, group_of(p, r), row, head, a);
            }
            join_entry<kD, false>(p, plan, max_ctas, p.R, r, row, head, a);
        }
    }
    const float inv = ok ? 1.0f / a.l : __int_as_float(0x7FC00000);
    __nv_bfloat16 w[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) w[i] = __float2bfloat16(ok ? a.o[i] * inv : inv);
    if (kPer == 4) *reinterpret_cast<uint2*>(p.out + item * kD + lane * kPer) = *reinterpret_cast<const uint2*>(w);
    else *reinterpret_cast<uint32_t*>(p.out + item * kD + lane * kPer) = *reinterpret_cast<const uint32_t*>(w);
    if (p.lse && lane == 0) p.lse[item] = ok ? (a.m + log2f(a.l)) * kLn2 : inv;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

// One launch's plan in the workspace at `off` (which moves on).
Plan plan_at(void* ws, size_t& off, int entries, long long items, int d, bool whole) {
    unsigned char* b = static_cast<unsigned char*>(ws);
    Plan p;
    p.bad = reinterpret_cast<int*>(b + off); off += 256;
    p.start = reinterpret_cast<long long*>(b + off); off += up(sizeof(long long) * ((size_t)entries + 1));
    p.part = reinterpret_cast<float*>(b + off); off += sizeof(float) * 2 * kMaxCtas * kTile * (size_t)d;
    p.part_ml = reinterpret_cast<float2*>(b + off); off += sizeof(float2) * 2 * kMaxCtas * kTile;
    p.whole = reinterpret_cast<float*>(b + off); off += whole ? up(sizeof(float) * (size_t)items * d) : 0;
    p.whole_ml = reinterpret_cast<float2*>(b + off); off += whole ? up(sizeof(float2) * (size_t)items) : 0;
    return p;
}

template <int kD>
cudaError_t launch_d(const AttnParams& p, cudaStream_t stream) {
    int dev = 0, n_sm = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if ((err = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return err;
    const int ctas = 2 * n_sm < kMaxCtas ? 2 * n_sm : kMaxCtas;
    const long long items = (long long)p.rows * p.hq;
    size_t off = 0;
    const Plan plan = plan_at(p.ws, off, p.R, items, kD, p.n_groups > 0);
    Plan shared_plan = plan;
    const int smem = Smem<kD>::kTotal;
    if (p.n_groups > 0) {
        shared_plan = plan_at(p.ws, off, p.n_groups, items, kD, true);
        if ((err = cudaFuncSetAttribute(attention_kernel<kD, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
            return err;
        attention_kernel<kD, true><<<ctas, kThreads, smem, stream>>>(p, shared_plan, ctas, p.n_groups);
        if ((err = cudaGetLastError()) != cudaSuccess) return err;
    }
    if ((err = cudaFuncSetAttribute(attention_kernel<kD, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
        return err;
    attention_kernel<kD, false><<<ctas, kThreads, smem, stream>>>(p, plan, ctas, p.R);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
    const unsigned grid = (unsigned)((items + kJoinThreads / 32 - 1) / (kJoinThreads / 32));
    join_kernel<kD><<<grid, kJoinThreads, 0, stream>>>(p, plan, shared_plan, ctas);
    return cudaGetLastError();
}

}  // namespace

size_t attention_workspace(int R, int n_groups, int rows, int hq, int, int d) {
    size_t off = 0;
    plan_at(nullptr, off, R, (long long)rows * hq, d, n_groups > 0);
    if (n_groups > 0) plan_at(nullptr, off, n_groups, (long long)rows * hq, d, true);
    return off;
}

cudaError_t launch_attention(const AttnParams& p, cudaStream_t stream) {
    return p.d == 64 ? launch_d<64>(p, stream) : launch_d<128>(p, stream);
}

}  // namespace dspark
