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
// An item is up to 256 rows of one key head: the rows of a request (of a group,
// over its shared pages) by query heads of that key head, so that a key read
// once serves them all.  Its keys go by in blocks of 128, and a step is one
// block against one tile of 128 rows:
//   S = Q K^T     tcgen05, 128 x 128, fp32 in tensor memory
//   P = 2^(x - m) one thread a row: the row's maximum, 128 exponentials, the
//                 sum; P goes back to tensor memory in bf16 over S
//   O += P V      tcgen05 with P from tensor memory, 128 x d, fp32
// Two tiles are in work at a time, so that the tensor cores have the one's
// products while the other's exponentials are formed: of an item of more than
// 128 rows its two halves over the same block, else the same rows over
// alternating blocks, whose two triples are added at the end (both lie in the
// same lanes of tensor memory).
//
// The reference m of a row moves only when the maximum has grown by more than
// 2^8 (O is rescaled then): P stays below 2^8 and fp32 sums lose nothing.
// P is the one rounding to fewer bits besides the output: 2^-8 of each weight
// at most, and l adds the weights before it.
//
// One CTA per SM, sixteen warps: 0-3 and 4-7 form the exponentials of the two
// tiles and write the sums out, 8-11 load keys and values, 15 queries, 12 issues
// the products, 13 finds the CTA's pieces of items and posts them to the others,
// 14 looks at blocks of values that not every row sees whole.  Keys and values come
// through a ring of 160 KB, queries through two buffers, so that the next item's
// first product does not wait for the last one's output.  Pages of a multiple of
// 8 slots come by TMA, each lane of a loading warp having a box of up to 128 rows
// by 64 elements inside one page.  Other pages may end anywhere in a block: their rows
// are gathered by 16-byte copies (a row to a lane, the queries' too), which have about
// 64 KB in flight per SM where TMA has the whole ring.  949 MB of keys and values
// (2 requests of 115000 keys): 150 us by TMA, 93 % of the copy rate, 200 us gathered;
// four rows to a TMA gather moved 6.4 bytes a cycle (500 us).
//
// Up to 32 rows (a few drafted tokens of one key head) lie in the tile four times
// and each copy takes a quarter of a block's keys: all four warps form exponentials
// then, 720 cycles for a block instead of 1350.  The product with V of a quarter's keys
// leaves the other copies' lanes alone.
//
// Values that are not finite: a weight of zero times one of them would be a NaN in rows
// that do not see it.  In a block that not all rows see whole such keys are taken out
// before the product and added by hand, by the weights in tensor memory, to the rows
// that see them; until then the issuing warp does not let the tile's next scores lie
// over the weights.
//
// Splitting: the steps of all items form one line, which is cut into equal
// pieces, one per CTA (each item costs some steps more, for its queries and
// output).  Each is charged its request's keys, so a prompt's early items, which see
// fewer, are less than their share: 8192 rows without history take 853 us (floor 290).
// An item that is cut leaves its triples in the workspace and a second kernel joins
// them in a fixed order.  With shared pages the groups' items (their
// keys, the rows of all their requests) and the requests' own go into the same line,
// and the second kernel adds each row's parts.  The cut depends on the lengths, which
// only the device knows: every CTA scans them itself.
//
// What bounds it: bytes, where few rows read many keys (128 requests of up to 5000,
// 1296 MB: 207 us, 92 % of the copy rate).  Many rows over the same keys: the way of
// a tile from its scores to its next ones, 1350 cycles of exponentials and 1950 of
// products and their hand-over, in which the other tile's go by too: 1024 of 1665
// cycles of a step the tensor cores are at work.  Short items: some 9000 cycles from
// the last product to the output and the next item's first weights.  Small calls:
// 14000 cycles until the first product, most of them code that comes into the
// instruction cache while every warp waits for it (95 KB of it; at 180 KB a third of
// the issue slots waited throughout, and waits that took 10 KB more made 128 short
// requests behind a shared prefix a fifth slower), and the second launch.
#include <type_traits>

#include "kernels.cuh"
#include "tc_ptx.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 512;
constexpr int kLoaders = 128;
constexpr int kTile = 128;   // rows of a tile
constexpr int kRows = 256;   // rows of an item
constexpr int kBlock = 128;  // keys of a block
// Steps that an item costs besides its own.  At 2, 3, 4, 5: 205, 206, 208, 210 us for 128 long ragged requests, 143, 141,
// 146, 151 for 128 short ones behind a shared prefix of 8192 keys, 74, 77, 81, 86 behind one of 2048, 59.2, 58.5, 59.2, 60.3
// for 48 blocks of 17 rows: 2 and 3 are within 4 % of each other either way.
constexpr int kItemCost = 3;
constexpr int kMaxCtas = 152;            // one per SM
constexpr int kMaxKeys = INT_MAX - 4 * kBlock;  // (loads look up to two blocks past the last key)
constexpr float kGrowth = 8.0f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------- the plan
// A cut item, by the CTA that has its first blocks.
struct Job {
    int n_rows;         // of the item (0: this CTA began none that it did not finish)
    int first, last;    // CTAs that have a piece
    int row0, tile_row; // rows of q of the entry, and the item's first (row, query head) of it
    int head;           // key head
    int pad[2];
};

// Workspace.  Of a query row and head, lin = row * g + (its place among the key head's).
struct Plan {
    float* part;      // [2 * ctas][d / 4][kRows][4]  sums of slot 2c: the item cut before CTA c's piece, 2c + 1: after it
    float2* part_ml;  // [2 * ctas][kRows]
    Job* jobs;        // [ctas]; with shared parts instead, of each row's own and shared part:
    float* whole;     // [2][hkv][d / 4][rows * g][4]  its sums, if the item was not cut
    float2* whole_ml; // [2][hkv][rows * g]
    int* where;       // [2][hkv][rows * g]  a Where
};

// Where the sums of a row's part lie.
struct Where {
    static constexpr int kSkip = -1, kCut = 1 << 24, kShared = 1 << 25;  // (of the own part: there is a shared one)
    static __device__ __forceinline__ int of(int first, int last, int row) { return kCut | first << 16 | last << 8 | row; }
};
static_assert(kMaxCtas <= 256 && kRows <= 256, "bytes of a Where");

struct Entry {     // a request's own keys, or a group's shared ones
    int row0, n;   // its rows of q (0: nothing to do)
    int begin;     // first key
    int end;       // past the last key any of its rows sees
    int len;       // row i sees keys below len + i + 1 (-1: all rows see the same keys)
    int table;     // the block table's row
    int tiles, blocks;
    bool shared;   // a group's
    bool last_pair; // its last item has more than kTile rows (as all others)
    // A block of an item takes 2^log_steps(t) steps; what the item costs, and all of a key head.
    __device__ int log_steps(int t) const { return t < tiles - 1 || last_pair; }
    __device__ int units(int t) const { return (blocks << log_steps(t)) + kItemCost; }
    __device__ long long per_head() const { return tiles ? (long long)(tiles - 1) * units(0) + units(tiles - 1) : 0; }
    // past the last key seen by row i of the entry
    __device__ int limit(int i) const { return len < 0 ? end : len + i + 1; }
};

__device__ __forceinline__ int group_of(const AttnParams& p, int r) {
    int lo = 0, hi = p.n_groups;  // the last group that starts at or before r
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.group_start[mid] <= r) lo = mid; else hi = mid;
    }
    return lo;
}

// Keys below which request r's are shared; -1: its group's length is bad.
__device__ __forceinline__ int shared_of(const AttnParams& p, int r) {
    const int s = p.shared_len[group_of(p, r)];
    return s >= 0 && s % p.page == 0 ? s : -1;
}

__device__ __forceinline__ bool request_ok(const AttnParams& p, int len, int n, int shared) {
    return len >= 0 && shared >= 0 && shared <= len && (long long)len + n <= (long long)p.max_blocks * p.page &&
           (long long)len + n <= kMaxKeys;
}

// Entry e: with kPrefix the groups' come first.
template <bool kPrefix>
__device__ __forceinline__ Entry entry_of(const AttnParams& p, int e) {
    Entry x;
    x.begin = 0;
    x.shared = kPrefix && e < p.n_groups;
    if (x.shared) {
        const int r0 = p.group_start[e], r1 = p.group_start[e + 1];
        const int s = p.shared_len[e];
        const bool ok = r0 >= 0 && r0 <= r1 && r1 <= p.R && s > 0 && s <= kMaxKeys && s % p.page == 0 && s / p.page <= p.max_blocks;
        x.table = r0;
        x.row0 = ok ? p.cu[r0] : 0;
        x.n = ok ? p.cu[r1] - x.row0 : 0;
        x.len = -1;
        x.end = s;
    } else {
        const int r = kPrefix ? e - p.n_groups : e;
        const int lo = p.cu[r], n = p.cu[r + 1] - lo, len = p.kv_len[r];
        const int shared = kPrefix ? shared_of(p, r) : 0;
        x.table = r;
        x.row0 = lo;
        x.n = request_ok(p, len, n, shared) ? n : 0;
        x.begin = shared;
        x.len = p.full_block ? -1 : len;
        x.end = len + n;
    }
    const int rows = x.n * (p.hq / p.hkv);
    x.last_pair = (rows - 1) % kRows >= kTile;
    if (x.n <= 0) {
        x.n = x.tiles = x.blocks = 0;
    } else {
        x.tiles = (rows - 1) / kRows + 1;
        x.blocks = (x.end - x.begin + kBlock - 1) / kBlock;
    }
    return x;
}

// a / b for a >= 0, b > 0.  Both fit 32 bits but for more units than the GPU does in half a minute; then bit by bit, which is
// 3 KB less code than the compiler's 64-bit divisions (code is what short items pay for: see above).
__device__ __forceinline__ long long divide(long long a, long long b) {
    if (!((a | b) >> 32)) return (long long)((uint32_t)a / (uint32_t)b);
    long long q = 0, rest = 0;
#pragma unroll 1
    for (int i = 62; i >= 0; --i) {
        rest = rest << 1 | (a >> i & 1);
        if (rest >= b) {
            rest -= b;
            q |= 1LL << i;
        }
    }
    return q;
}

// Units of the line to a CTA (two at least, so that a block begins in each piece of an item; at 3, 4, 6 a request
// of 777 keys took 15.9, 16.7, 17.7 us, at 2 15.2).
__device__ __forceinline__ long long piece_length(long long total, int ctas) { return max(divide(total + ctas - 1, ctas), 2LL); }

// What a CTA does of one item: blocks [b0, b1) of it.
struct Piece {
    int steps;            // 0: there are no more
    int pair;             // two tiles over each block
    int b0, uncut;        // the piece is the whole item
    int row0, tile_row;   // rows of q of the entry, and the item's first (row, query head) of it
    int n_rows, head;     // rows of the item, key head
    int begin, end, len;  // as in the entry
    int table;
    int low, high;        // past the last key that the item's first and last row see
    int g0;               // steps of the pieces before
    int last_cta;         // that has a piece of the item
    int shared;           // of a group's keys
    int spoiled;          // a page is missing: the rows are NaN
    int edge, look;       // first block, from b0 on, that some row does not see whole; that a box may overrun
    int log_copies;       // the rows lie in a tile so many times
    int n_q;              // query buffers used before
    __device__ __forceinline__ int limit(int i) const { return len < 0 ? end : len + i + 1; }
};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
// Waits until the phase of `parity` completes, at most *limit ns (0 once the CTA is to stop).
constexpr uint32_t kWaitNs = 2000000000;
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, const volatile uint32_t* limit) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 from, now, most;\n\tmov.u32 from, %%globaltimer_lo;\n"
        "again:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
        "@p bra done;\n\t"
        "ld.volatile.shared.u32 most, [%3];\n\t"
        "mov.u32 now, %%globaltimer_lo;\n\t"
        "sub.u32 now, now, from;\n\t"
        "setp.lt.u32 q, now, most;\n\t"
        "@q bra again;\n"
        "done:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity), "r"(tc::smem_u32(const_cast<const uint32_t*>(limit)))
        : "memory");
    return ok != 0;
}

// The same for the warps that run ahead of the products (pieces, queries, values that are looked at): they wait as long as
// the work on the items before takes, whose own waits have the limit, and give up when one of those has.  (At most 2^24
// suspensions, a minute or so.)
__device__ __forceinline__ bool wait_ahead_bounded(uint64_t* bar, uint32_t parity, const volatile uint32_t* limit) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 n, most;\n\tmov.u32 n, 16777216;\n"
        "again:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
        "@p bra done;\n\t"
        "ld.volatile.shared.u32 most, [%3];\n\t"
        "sub.u32 n, n, 1;\n\t"
        "setp.ne.u32 q, n, 0;\n\t"
        "setp.ne.and.u32 q, most, 0, q;\n\t"
        "@q bra again;\n"
        "done:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity), "r"(tc::smem_u32(const_cast<const uint32_t*>(limit)))
        : "memory");
    return ok != 0;
}

// The compiler is to know nothing of x: loops whose first rounds leave out a part
// would else be written out for each of them, and all the warps' code has to stay
// in the instruction cache.
__device__ __forceinline__ int opaque(int x) {
    asm volatile("" : "+r"(x));
    return x;
}

// ---------------------------------------------------------------- the kernel
// 16-byte chunk c of row r of an operand.
__device__ __forceinline__ uint32_t chunk_offset(int r, int c) {
    return (uint32_t)((c >> 3) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

constexpr int kPieces = 4;    // ahead of the products
constexpr int kReaders = 15;  // warps that read them

// kSteps: more than the loads can be ahead.
template <int kSlots, int kSteps>
struct Shared {
    uint64_t full[kSlots], empty[kSlots];  // ring slots
    uint64_t landed[kSlots];               // values that are looked at before they are full
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], p_full[2];         // per tile: scores formed, weights written
    uint64_t o_done[2], o_free[2];         // a product with V is done; the output was read
    uint64_t odd_done[2];                  // values that are not finite were added: the weights may be written over
    uint64_t merge;                        // the second tile's sums are ready
    uint64_t drain;
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    Piece pieces[kPieces];
    float2 ml[2][kTile];                   // each tile's m and l of its rows, for the other tile or its own copies
    alignas(16) uint32_t odd[kSteps][4];   // by step: keys of a block whose values are not finite
    volatile uint32_t limit, last_limit;   // of the waits, ns (0: one ran out); of the last one
    uint32_t tmem_base;
    long long scan[kThreads / 32];
};

template <int kD>
struct Layout {
    static constexpr int kHalf = kTile * 128;           // 128 rows of 64 elements, 128-byte swizzle
    static constexpr int kOperand = kD / 64 * kHalf;    // a tile of Q, a block of K or V
    static constexpr int kSlots = 5 * 128 / kD;         // of the ring
    static constexpr int kSteps = 8 * 128 / kD;
    static constexpr int kTotal = (2 + kSlots) * kOperand + (int)sizeof(Shared<kSlots, kSteps>);
    static_assert(kTotal <= 227 * 1024, "shared memory of a CTA");
};

// Arrives on `bar` when this thread's copies so far are done.
__device__ __forceinline__ void cp_async_arrive_noinc(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}
// `n` arrivals by one thread.
__device__ __forceinline__ void arrive_n(uint64_t* bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(tc::smem_u32(bar)), "r"(n) : "memory");
}

struct Maps {
    CUtensorMap k, v;  // [pages * hkv * page, d] in boxes of box_rows x 64
    int box_rows;      // 0: rows are gathered one by one
};

template <int kD, bool kPrefix>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const AttnParams p, const Plan plan, const int max_ctas,
                                                               const int entries, const __grid_constant__ Maps maps) {
    using L = Layout<kD>;
    constexpr int kChunks = kD / 8;
    constexpr int kSlots = L::kSlots;
    constexpr uint32_t kTmemO = 2 * kBlock;  // columns: S of the tiles (P over it) 0 and 128, O 256 and 256 + 128
    constexpr int kOddRing = L::kSteps;
    extern __shared__ __align__(1024) unsigned char base[];
    auto& sh = *reinterpret_cast<Shared<kSlots, kOddRing>*>(base + (2 + kSlots) * L::kOperand);

    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
    const int g = p.hq / p.hkv;
    const uint32_t sQ = tc::smem_u32(base), sRing = sQ + 2 * L::kOperand;
    const __nv_bfloat16 kNan = __ushort_as_bfloat16(0x7FFF);

    const uint32_t loaders = maps.box_rows > 0 ? 1 : kLoaders;  // arrivals that fill a slot
    // ---- the line of all items' blocks, and this CTA's piece of it
    if (warp == 12) {
        tc::tmem_alloc(&sh.tmem_base, 512);
        tc::tmem_relinquish();
    }
    if (warp == 13) {
        if (lane < kSlots) {
            tc::mbar_init(&sh.full[lane], loaders);
            tc::mbar_init(&sh.landed[lane], loaders);
            tc::mbar_init(&sh.empty[lane], 1);
        }
        if (lane < 2) {
            tc::mbar_init(&sh.q_full[lane], 32 + p.inject);
            tc::mbar_init(&sh.q_empty[lane], 2);
            tc::mbar_init(&sh.s_full[lane], 1);
            tc::mbar_init(&sh.p_full[lane], 4);
            tc::mbar_init(&sh.o_done[lane], 1);
            tc::mbar_init(&sh.o_free[lane], 4);
            tc::mbar_init(&sh.odd_done[lane], 4);
        }
        if (lane < kPieces) {
            tc::mbar_init(&sh.piece_full[lane], 1);
            tc::mbar_init(&sh.piece_empty[lane], kReaders);
        }
        if (lane == 0) {
            tc::mbar_init(&sh.merge, 4);
            tc::mbar_init(&sh.drain, 1);
            sh.limit = sh.last_limit = kWaitNs;
        }
        tc::fence_barrier_init();
    }
    wait_prior_grid();  // (nothing before this depends on what earlier kernels wrote)
    launch_dependents();
    if (!kPrefix && tid == 0) plan.jobs[blockIdx.x].n_rows = 0;
    // every thread has `per` entries
    const int per = (entries + kThreads - 1) / kThreads;
    auto cost_of = [&](int t) {
        long long c = 0;
#pragma unroll 1
        for (int e = t * per; e < min(entries, (t + 1) * per); ++e) c += entry_of<kPrefix>(p, e).per_head() * p.hkv;
        return c;
    };
    auto scanned = [&](long long c) {  // over the warp, each lane's included
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xFFFFFFFFu, c, o);
            if (lane >= o) c += up;
        }
        return c;
    };
    int bad = p.cu[0] != 0 || p.cu[p.R] > p.rows;
    if (kPrefix) bad |= p.group_start[0] != 0 || p.group_start[p.n_groups] != p.R;
#pragma unroll 1
    for (int r = tid; r < p.R; r += kThreads) bad |= p.cu[r] > p.cu[r + 1];
    if (kPrefix)
#pragma unroll 1
        for (int e = tid; e < p.n_groups; e += kThreads) bad |= p.group_start[e] > p.group_start[e + 1];
    const long long mine = scanned(cost_of(tid));
    if (lane == 31) sh.scan[warp] = mine;
    long long* const scans = reinterpret_cast<long long*>(base + 2 * L::kOperand);  // each thread's, over its warp (in the ring)
    scans[tid] = mine;
    tc::fence_proxy_async_smem();
    tc::tc_fence_before();
    bad = __syncthreads_or(bad);
    tc::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sh.tmem_base, 0);
    if (bad) {  // nothing can be said of any row
        if (warp == 12) tc::tmem_dealloc(tmem, 512);
        const long long n = (long long)p.rows * p.hq;
#pragma unroll 1
        for (long long i = (long long)blockIdx.x * kThreads + tid; i < n * kD; i += (long long)gridDim.x * kThreads) p.out[i] = kNan;
        if (p.lse)
#pragma unroll 1
            for (long long i = (long long)blockIdx.x * kThreads + tid; i < n; i += (long long)gridDim.x * kThreads)
                p.lse[i] = __int_as_float(0x7FC00000);
        if (kPrefix)
#pragma unroll 1
            for (long long i = (long long)blockIdx.x * kThreads + tid; i < n; i += (long long)gridDim.x * kThreads)
                plan.where[i] = Where::kSkip;
        if (blockIdx.x == 0 && tid == 0) report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
        return;
    }
    const float sl2 = fmaxf(p.scale * kLog2e, 1e-37f);  // (a masked score, -inf, weighs nothing at a scale of 0 too)
    // Waits for the phase of that parity; false (and the CTA stops) when the limit passes, and from then on at once.  What
    // is waited for may then be missing: nothing goes out of bounds by it, and what the call writes is not valid.
    // (No function is called: the register split below leaves none for a call's frame.)
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool ok = wait_bounded(bar, parity & 1, &sh.limit);
        if (!ok) sh.limit = 0;
        return ok;
    };
    auto wait_ahead = [&](uint64_t* bar, uint32_t parity) {
        const bool ok = wait_ahead_bounded(bar, parity & 1, &sh.limit);
        if (!ok) sh.limit = 0;
        return ok;
    };
    // The same, one answer for the warp.
    auto held = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(bar, parity)) != 0; };

    // Whether the phase is there already.
    auto test = [&](uint64_t* bar, uint32_t parity) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(tc::smem_u32(bar)), "r"(parity & 1)
            : "memory");
        return __all_sync(0xFFFFFFFFu, ok) != 0;
    };

    // A warp's place in the sequence of pieces: piece `i` and step `u` of it.
    struct Cursor {
        int i = 0, u = 0, steps = 0, pair = 0, edge = 0, copies = 0;
        const Piece* at = nullptr;
        __device__ __forceinline__ int block() const { return pair ? u >> 1 : u; }     // from the piece's first on
        __device__ __forceinline__ bool leads() const { return !(u & pair); }          // the step brings a block
    };
    // A place in the ring.
    struct Ring {
        uint32_t s = 0, phase = 0;
        __device__ __forceinline__ void next() {
            if (++s == kSlots) {
                s = 0;
                phase ^= 1;
            }
        }
    };
    auto read = [&](Cursor& c, bool ok) {  // false: there are no more
        c.at = &sh.pieces[c.i % kPieces];
        // (what a shuffle gives is the same for all lanes, and the compiler keeps it in uniform registers)
        c.steps = __shfl_sync(0xFFFFFFFFu, ok ? c.at->steps : 0, 0);
        c.pair = __shfl_sync(0xFFFFFFFFu, c.at->pair, 0);
        c.edge = __shfl_sync(0xFFFFFFFFu, c.at->edge, 0);
        c.copies = __shfl_sync(0xFFFFFFFFu, c.at->log_copies, 0);
        c.u = 0;
        return c.steps > 0;
    };
    auto open = [&](Cursor& c) { return read(c, wait(&sh.piece_full[c.i % kPieces], c.i / kPieces)); };
    auto open_ahead = [&](Cursor& c) { return read(c, wait_ahead(&sh.piece_full[c.i % kPieces], c.i / kPieces)); };
    auto stopped = [&]() { return __any_sync(0xFFFFFFFFu, sh.limit == 0); };
    auto close = [&](Cursor& c) {  // done with the piece; on to the next
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.piece_empty[c.i % kPieces]);
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    }

    if (warp < 8) {
        // ================================================================ exponentials
        const int X = warp >> 2, t128 = tid & (kTile - 1);
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lanes + X * kBlock, tO = tmem + lanes + kTmemO + X * kBlock;
        const uint32_t tO2 = tmem + lanes + kTmemO + (X ^ 1) * kBlock;
        // The warp's arrival (32 of them on one barrier take some 4 cycles each: 2000 cycles of a step).
        auto arrive = [&](uint64_t* bar) {
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar);
        };
        auto tile_sync = [&]() {
            __syncwarp();  // (the barrier counts warps: their lanes have to come together)
            asm volatile("bar.sync %0, 128;" ::"r"(1 + X) : "memory");
        };
        // Whether all four warps of the tile go on: they meet in tile_sync, which has no limit, the same number of times.
        auto all_go = [&](bool go) {
            uint32_t all;
            __syncwarp();
            asm volatile(
                "{\n\t.reg .pred p, q;\n\t"
                "setp.ne.u32 p, %1, 0;\n\t"
                "bar.red.and.pred q, %2, 128, p;\n\t"
                "selp.u32 %0, 1, 0, q;\n\t}"
                : "=r"(all)
                : "r"((uint32_t)go), "r"(1 + X)
                : "memory");
            return all != 0;
        };
        int n_step = 0;     // steps of this tile so far
        int n_done = 0;     // of them, the ones whose product is waited for
        int n_merge = 0;
        Cursor at;
        for (; all_go(open(at) && !stopped()); close(at), ++at.i) {
            const Piece& w = *at.at;
            const int g0 = w.g0, steps = at.steps;
            const int u0 = X ^ (g0 & 1);
            if (u0 >= steps) continue;  // (one step, the other tile's)
            const int sub = at.pair ? u0 : 0;
            // Up to 32 rows lie in the tile four times, each copy takes a quarter of a block's keys: all four warps
            // form exponentials then, and each 32 of a row instead of 128.
            const int log_copies = w.log_copies, log_rows = 7 - log_copies;
            const int n_rows = min(w.n_rows - sub * kTile, kTile), t_row = t128 & ((1 << log_rows) - 1);
            const int col0 = (t128 >> log_rows) << log_rows;  // this copy's first key of a block
            const bool live = t_row < n_rows, warp_live = (t_row & ~31) < n_rows;
            const int my_r = w.tile_row + (live ? sub * kTile + t_row : 0), my_i = my_r / g;
            const int my_limit = w.limit(my_i);
            const int first_key = w.begin + w.b0 * kBlock;
            float m = -INFINITY, l = 0.0f;  // m in raw scores
#pragma unroll 1
            for (int u = u0; u < steps; u += 2) {
                const int key0 = first_key + (at.pair ? u >> 1 : u) * kBlock;
                // N scores of this row from column col0 on: maximum, weights, their sum
                auto weigh = [&](auto n_) {
                    constexpr int N = decltype(n_)::value;
                    float s[N];
                    tc::tmem_ld_32x32b_x32<0>(tS + col0, s);
                    if constexpr (N == kBlock) {
                        tc::tmem_ld_32x32b_x32<32>(tS + 32, s);
                        tc::tmem_ld_32x32b_x32<64>(tS + 64, s);
                        tc::tmem_ld_32x32b_x32<96>(tS + 96, s);
                    }
                    tc::tmem_ld_wait();
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int j = 0; j < N; j += 8) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) top[i] = max3(top[i], s[j + 2 * i], s[j + 2 * i + 1]);
                    }
                    const float mb = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                    // move the reference when the maximum has grown by more than 2^kGrowth
                    const bool move = live && mb > m && !((mb - m) * sl2 <= kGrowth);
                    if (__any_sync(0xFFFFFFFFu, move)) {
                        const float f = !move ? 1.0f : m == -INFINITY ? 0.0f : exp2_approx((m - mb) * sl2);
                        if (move) m = mb;
                        l *= f;
                        if (u > u0) {
#pragma unroll 1
                            for (int c = 0; c < kD; c += 16) {
                                float o[16];
                                uint32_t v[16];
                                tc::tmem_ld_32x32b_x16<0>(tO + c, o);
                                tc::tmem_ld_wait();
#pragma unroll
                                for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(o[j] * f);
                                tc::tmem_st_32x32b_x16<0>(tO + c, v);
                            }
                        }
                    }
                    const float ref = m == -INFINITY ? 0.0f : -m * sl2;
                    float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                    for (int c = 0; c < N; c += 32) {
                        uint32_t v[16];
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            const float2 x = fma2(make_float2(s[c + j], s[c + j + 1]), make_float2(sl2, sl2), make_float2(ref, ref));
                            const float2 y = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                            sum[(j >> 1) & 1] = add2(sum[(j >> 1) & 1], y);
                            const __nv_bfloat162 both = __floats2bfloat162_rn(y.x, y.y);
                            v[j >> 1] = *reinterpret_cast<const uint32_t*>(&both);
                        }
                        tc::tmem_st_32x32b_x16<0>(tS + (col0 + c) / 2, v);
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    tc::tmem_st_wait();
                };
                // (the scores are formed after the last product with V of this tile: that one is done too)
                if (!held(&sh.s_full[X], n_step)) break;
                tc::tc_fence_after();
                if (warp_live) {
                    const int seen = my_limit - key0;  // keys of the block this row sees
                    if (!__all_sync(0xFFFFFFFFu, seen >= kBlock)) {
#pragma unroll 1
                        for (int c = col0; c < col0 + (1 << log_rows); c += 16) {
                            float x[16];
                            uint32_t v[16];
                            tc::tmem_ld_32x32b_x16<0>(tS + c, x);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[j] = j < seen - c ? __float_as_uint(x[j]) : 0xFF800000u;
                            tc::tmem_st_32x32b_x16<0>(tS + c, v);
                        }
                        tc::tmem_st_wait();
                    }
                    if (log_copies) weigh(std::integral_constant<int, 32>{});
                    else weigh(std::integral_constant<int, kBlock>{});
                }
                tc::tc_fence_before();
                arrive(&sh.p_full[X]);
                ++n_step;
                if ((at.pair ? u >> 1 : u) >= at.edge) {
                    // Some row does not see all of these keys.  Values that are not finite were taken out of the
                    // block, so that they reach no row through a zero weight; here the rows that do see them get them,
                    // by the weights in tensor memory; until odd_done the tile's next scores are not formed over them.
                    wait(&sh.o_done[X], n_done);
                    if (u + 2 < steps) ++n_done;
                    tc::tc_fence_after();
                    __syncwarp();
                    const uint32_t* odd = sh.odd[(g0 + (at.pair ? u & ~1 : u)) % kOddRing];
                    const bool some = (odd[0] | odd[1] | odd[2] | odd[3]) != 0;
                    if (warp_live && some) {
#pragma unroll 1
                        for (int key = col0; key < col0 + (1 << log_rows); ++key) {
                            if (!(odd[key >> 5] >> (key & 31) & 1)) continue;
                            const int pos = key0 + key, pb = pos / p.page;
                            const int id = IN_BOUNDS(pb < p.max_blocks, p.dev_status) ? p.block_table[(long long)w.table * p.max_blocks + pb] : 0;
                            if (!IN_BOUNDS(id >= 0 && id < p.pool_pages, p.dev_status)) continue;
                            const __nv_bfloat16* v = p.v_cache + (((size_t)id * p.hkv + w.head) * p.page + (pos - pb * p.page)) * kD;
                            const uint32_t both = tc::tmem_ld_32x32b_x1(tS + key / 2);
                            tc::tmem_ld_wait();
                            const float weight = __uint_as_float(key & 1 ? both & 0xFFFF0000u : both << 16);
#pragma unroll 1
                            for (int c = 0; c < kD; c += 16) {
                                float o[16];
                                uint32_t q[16];
                                tc::tmem_ld_32x32b_x16<0>(tO + c, o);
                                tc::tmem_ld_wait();
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    q[j] = __float_as_uint(pos < my_limit ? fmaf(weight, __bfloat162float(v[c + j]), o[j]) : o[j]);
                                tc::tmem_st_32x32b_x16<0>(tO + c, q);
                            }
                            tc::tmem_st_wait();
                        }
                    }
                    tc::tc_fence_before();
                    if (some) arrive(&sh.odd_done[X]);
                }
            }
            // ---- the triple of this tile's rows
            // The other tile may have a part of the same rows: the one with the last step waits the least for it, and
            // the next item begins with the other.
            const bool two = !at.pair && steps > 1, last = at.pair || ((steps - 1 - u0) & 1) == 0;
            // (without copies the query buffer is not needed below)
            if (last && !log_copies && t128 == 0) tc::mbar_arrive(&sh.q_empty[(w.n_q + sub) & 1]);
            wait(&sh.o_done[X], n_done);
            ++n_done;
            tc::tc_fence_after();
            __syncwarp();
            if (two && !last) {
                sh.ml[X][t128] = make_float2(m, l);
                tc::tc_fence_before();
                arrive(&sh.merge);
                ++n_merge;
                continue;
            }
            // adds another part's (m, l) to (m0, l0): their common reference, and both scales.  (A sum that is not a
            // number stays one, whatever its scale.)
            auto add = [](float& m0, float& l0, float m1, float l1, float& f0, float& f1) {
                const float top = fmaxf(m0, m1);
                f0 = m0 == -INFINITY ? 0.0f : exp2_approx(m0 - top);
                f1 = m1 == -INFINITY ? 0.0f : exp2_approx(m1 - top);
                l0 = (m0 == -INFINITY ? l0 : l0 * f0) + (m1 == -INFINITY ? l1 : l1 * f1);
                m0 = top;
            };
            m = m == -INFINITY ? -INFINITY : m * sl2;  // base-2 from here on
            float f1 = 1.0f, f2 = 0.0f;                // scales of this tile's, the other tile's sums
            if (two) {
                wait(&sh.merge, n_merge);
                tc::tc_fence_after();
                __syncwarp();
                ++n_merge;
                const float2 other = sh.ml[X ^ 1][t128];
                add(m, l, other.x == -INFINITY ? -INFINITY : other.x * sl2, other.y, f1, f2);
            }
            if (log_copies) {
                sh.ml[X][t128] = make_float2(m, l);
                tile_sync();
                const float own = m;
                m = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < 1 << log_copies; ++c) m = fmaxf(m, sh.ml[X][(c << log_rows) + t_row].x);
                l = 0.0f;
#pragma unroll 1
                for (int c = 0; c < 1 << log_copies; ++c) {
                    const float2 ml = sh.ml[X][(c << log_rows) + t_row];
                    l += ml.x == -INFINITY ? ml.y : ml.y * exp2_approx(ml.x - m);
                }
                const float f = own == -INFINITY ? 0.0f : exp2_approx(own - m);
                f1 *= f;
                f2 *= f;
                tile_sync();  // (the places are used again)
            }
            if (w.spoiled) l = __int_as_float(0x7FC00000);
            const bool uncut = w.uncut != 0;
            const bool final = !kPrefix && uncut;
            const size_t slot = (size_t)(2 * blockIdx.x + (w.b0 == 0)) * kRows;  // its first row
            if (final) {
                const float inv = 1.0f / l;
                f1 *= inv;
                f2 *= inv;
            }
            // partial sums lie by four columns, then rows, so that a warp's stores are contiguous
            const bool whole = kPrefix && uncut;
            const size_t lin_step = (size_t)p.rows * g, lin0 = (size_t)w.row0 * g + w.tile_row + sub * kTile;
            const size_t part_of = (size_t)(w.shared * p.hkv + w.head) * lin_step;  // in the rows' own or shared parts
            float4* const to = reinterpret_cast<float4*>(whole ? plan.whole + part_of * kD : plan.part + slot * kD);
            const size_t to0 = whole ? lin0 : sub * kTile, to_step = whole ? lin_step : kRows;
            const size_t out_row = (size_t)(w.row0 + my_i) * p.hq + w.head * g + (my_r - my_i * g);
            const bool writes = live && IN_BOUNDS(w.row0 >= 0 && my_i >= 0 && w.head < p.hkv && out_row < (size_t)p.rows * p.hq, p.dev_status);
            auto sums = [&](int c, float (&o)[16]) {  // 16 columns of this lane's row, of both tiles
                float o2[16];
                tc::tmem_ld_32x32b_x16<0>(tO + c, o);
                if (two) tc::tmem_ld_32x32b_x16<0>(tO2 + c, o2);
                tc::tmem_ld_wait();
                if (c + 16 == kD) {  // the next item's products may have the place
                    tc::tc_fence_before();
                    arrive(&sh.o_free[X]);
                    if (two) arrive(&sh.o_free[X ^ 1]);
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = two ? o[j] * f1 + o2[j] * f2 : o[j] * f1;
            };
            auto pack = [](float4 y) {
                const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y), hi = __floats2bfloat162_rn(y.z, y.w);
                return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
            };
            if (!log_copies) {
                // A row to a lane: a column of a warp's sums lies in one piece, and of the output each lane writes whole
                // sectors.
                __nv_bfloat16* const out = p.out + out_row * kD;
#pragma unroll 1
                for (int c = 0; c < kD; c += 16) {
                    float o[16];
                    sums(c, o);
                    if (writes) {
                        uint2 b[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 y = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                            b[j] = pack(y);
                            if (!final) to[(size_t)(c / 4 + j) * to_step + to0 + t_row] = y;
                        }
                        if (final) {
                            reinterpret_cast<uint4*>(out + c)[0] = make_uint4(b[0].x, b[0].y, b[1].x, b[1].y);
                            reinterpret_cast<uint4*>(out + c)[1] = make_uint4(b[2].x, b[2].y, b[3].x, b[3].y);
                        }
                    }
                }
            } else {
                // The copies' sums meet in the item's query buffer, half of the columns at a time.
                float4* const stage = reinterpret_cast<float4*>(base + (w.n_q & 1) * L::kOperand);  // [c / 4][128 lanes]
                if (final) sh.ml[X][t128].x = __int_as_float((int)out_row);
                constexpr int kQuads = kD / 8, kApart = kTile / kQuads, kBatch = 32 / kApart;
                const int my_q = opaque(t128) % kQuads, my_r0 = opaque(t128) / kQuads;  // of the output: four columns of every kApart-th row
#pragma unroll 1
                for (int c0 = 0; c0 < kD; c0 += kD / 2) {
#pragma unroll 1
                    for (int c = 0; c < kD / 2; c += 16) {
                        float o[16];
                        sums(c0 + c, o);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int q = c / 4 + j;
                            stage[q * kTile + (t128 ^ (q & 15))] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                        }
                    }
                    tile_sync();
                    auto sum_of = [&](int q, int r) {  // over the copies
                        float4 y = stage[q * kTile + (r ^ (q & 15))];
#pragma unroll
                        for (int c = 32; c < kTile; c += 32) {
                            const float4 v = stage[q * kTile + ((c + r) ^ (q & 15))];
                            y.x += v.x; y.y += v.y; y.z += v.z; y.w += v.w;
                        }
                        return y;
                    };
                    if (final) {  // a row's columns side by side
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) {
                            const int r = my_r0 + i * kApart;
                            if (r < n_rows) {
                                const int at_row = __float_as_int(sh.ml[X][r].x);
                                if (!IN_BOUNDS(at_row >= 0 && at_row / p.hq < p.rows, p.dev_status)) continue;
                                *reinterpret_cast<uint2*>(p.out + (size_t)at_row * kD + c0 + 4 * my_q) = pack(sum_of(my_q, r));
                            }
                        }
                    } else {  // a column's rows
#pragma unroll 1
                        for (int q = t128 >> log_rows; q < kQuads && writes; q += 1 << log_copies)
                            to[(size_t)(c0 / 4 + q) * to_step + to0 + t_row] = sum_of(q, t_row);
                    }
                    tile_sync();
                }
                if (t128 == 0) tc::mbar_arrive(&sh.q_empty[w.n_q & 1]);
            }
            if (writes && t128 == t_row) {
                if (!final) (whole ? plan.whole_ml + part_of : plan.part_ml + slot)[to0 + t_row] = make_float2(m, l);
                else if (p.lse) p.lse[out_row] = (m + log2f(l)) * kLn2;
                if (kPrefix && w.b0 == 0)
                    plan.where[part_of + lin0 + t_row] = (uncut ? 0 : Where::of(blockIdx.x, w.last_cta, sub * kTile + t_row)) |
                                                         (w.begin > 0 ? Where::kShared : 0);
            }
            if (!kPrefix && t128 == 0 && !uncut && w.b0 == 0 && sub == 0) {
                Job j;
                j.n_rows = w.n_rows;
                j.first = blockIdx.x;
                j.last = w.last_cta;
                j.row0 = w.row0;
                j.tile_row = w.tile_row;
                j.head = w.head;
                j.pad[0] = j.pad[1] = 0;
                plan.jobs[blockIdx.x] = j;
            }
        }
    } else if (warp < 12 && maps.box_rows > 0) {
        // ================================================================ loads by TMA
        // A lane has one box of a block, its first key and 64 of its columns; each of the four warps has slots of its
        // own (one takes it about 1500 cycles, of pages of 16).  All uses of a slot are one warp's: its wait for the
        // slot to be empty again is then never for another phase of the same parity.
        const int none = p.pool_pages * p.hkv * p.page;  // past the matrices: zeros
        const int boxes = kBlock / maps.box_rows, box_key = lane % boxes * maps.box_rows, half = lane / boxes;
        const int pages_on = kBlock / p.page, slots_on = kBlock - pages_on * p.page;  // from a block to the next
        const uint32_t dst = half * L::kHalf + box_key * 128;
        Ring ring;
        uint32_t filled = 0;
        // this lane's box of the next block of keys: its position, page and slot of it, and the page's id
        int pos = 0, page = 0, slot = 0, id = 0;
        const int32_t* table = nullptr;
        int high = 0, head = 0;
        Cursor k, v;
        bool more;
        auto open_k = [&]() {
            more = open(k);
            if (!more) return;
            const Piece& w = *k.at;
            pos = w.begin + w.b0 * kBlock + box_key;
            page = pos / p.page;
            slot = pos - page * p.page;
            table = p.block_table + (long long)w.table * p.max_blocks;
            high = w.high;
            head = w.head;
            if (pos < high) id = IN_BOUNDS(page < p.max_blocks, p.dev_status) ? __ldg(table + page) : -1;
        };
        open_k();
        open(v);
        int kept0 = 0, kept1 = 0, n_kept = 0;
#pragma unroll 1
        for (int i = opaque(-4); v.steps > 0 && !stopped(); ++i) {  // values of a step, keys of the step after the next
            const bool is_k = i & 1;
            if (is_k ? !more : i < 0) continue;
            const Cursor& c = is_k ? k : v;
            if (c.leads()) {
                int row = kept0;
                uint64_t* bar = &sh.full[ring.s];
                if (is_k) {
                    row = none;
                    if (pos < high) {
                        if (id >= 0 && id < p.pool_pages && IN_BOUNDS(head < p.hkv && slot >= 0 && slot < p.page, p.dev_status)) {
                            row = (id * p.hkv + head) * p.page + slot;
                        } else {
                            sh.pieces[k.i % kPieces].spoiled = 1;
                            report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
                        }
                    }
                    (n_kept == 0 ? kept0 : kept1) = row;
                    ++n_kept;
                    // on to the next block: its page's id is there when it is wanted
                    pos += kBlock;
                    page += pages_on;
                    slot += slots_on;
                    if (slot >= p.page) {
                        slot -= p.page;
                        ++page;
                    }
                    if (pos < high) id = IN_BOUNDS(page < p.max_blocks, p.dev_status) ? __ldg(table + page) : -1;
                } else {
                    kept0 = kept1;
                    --n_kept;
                    if (c.block() >= c.at->look) bar = &sh.landed[ring.s];
                }
                if ((int)(ring.s & 3) == (warp & 3)) {
                    if (filled == kSlots && !held(&sh.empty[ring.s], ring.phase ^ 1)) break;  // (its last fill may be on its way)
                    __syncwarp();  // (what a lane noted of a missing page goes before the arrival)
                    if (lane == 0) tc::mbar_arrive_expect_tx(bar, L::kOperand);
                    __syncwarp();
                    if (half < kD / 64)
                        tc::tma_load_2d(base + (2 + ring.s) * L::kOperand + dst, is_k ? &maps.k : &maps.v, bar, half * 64, row);
                }
                if (filled < kSlots) ++filled;
                ring.next();
            }
            if (is_k) {
                if (++k.u == k.steps) {
                    ++k.i;
                    open_k();
                }
            } else if (++v.u == v.steps) {
                close(v);
                ++v.i;
                open(v);
            }
        }
    } else if (warp < 12 || warp == 15) {
        // ================================================================ rows copied one by one
        // (the queries' by warp 15; with TMA no others)
        constexpr int kNone = -1, kMissing = -2, kPerPass = 32 / kChunks;  // (rows that 32 chunks make up)
        const int part = warp & 3;
        auto first_key = [](const Cursor& c) { return c.at->begin + (c.at->b0 + c.block()) * kBlock; };
        // the cache row of this lane's key of the cursor's block
        auto row_of = [&](const Cursor& c) -> int {
            const Piece& w = *c.at;
            const int pos = first_key(c) + part * 32 + lane;
            if (pos >= w.high) return kNone;
            const int pb = pos / p.page;
            if (!IN_BOUNDS(w.table < p.R && pb < p.max_blocks && w.head < p.hkv, p.dev_status)) return kMissing;
            const int id = __ldg(p.block_table + (long long)w.table * p.max_blocks + pb);
            if (id < 0 || id >= p.pool_pages) return kMissing;
            return (id * p.hkv + w.head) * p.page + (pos - pb * p.page);
        };
        // This lane's row and those of its warp (row < 0: zeros) to their places of an operand.
        auto copy = [&](uint32_t dst, int part, const __nv_bfloat16* rows, int row) {
            const int c = lane % kChunks;
            const char* const from = reinterpret_cast<const char*>(rows) + c * 16;
            dst += part * 32 * 128;
#pragma unroll 4
            for (int i = 0; i < kChunks; ++i) {
                const int r = i * kPerPass + lane / kChunks, from_row = __shfl_sync(0xFFFFFFFFu, row, r);
                tc::cp_async_16(dst + chunk_offset(r, c), from + (size_t)max(from_row, 0) * (kD * 2), from_row < 0 ? 0 : 16);
            }
        };
        Cursor k;
        if (warp == 15) {
            uint32_t n_q = 0;
#pragma unroll 1
            for (; open_ahead(k) && !stopped(); close(k), ++k.i) {
                const Piece& w = *k.at;
#pragma unroll 1
                for (int sub = 0; sub <= k.pair; ++sub, ++n_q) {
                    const int q = n_q & 1;
                    if (n_q >= 2) wait_ahead(&sh.q_empty[q], (n_q >> 1) - 1);
                    // Only rows that there are (the others' scores are their own), each to all its copies.
                    const int at0 = w.tile_row + sub * kTile, n_rows = min(w.n_rows - sub * kTile, kTile);
                    const bool copies = w.log_copies != 0;
#pragma unroll 1
                    for (int r0 = 0; r0 < n_rows; r0 += 32) {
                        const int at = at0 + min(r0 + lane, n_rows - 1), qi = at / g;
                        int row = (w.row0 + qi) * p.hq + w.head * g + (at - qi * g);
                        if (!IN_BOUNDS(row >= 0 && row / p.hq < p.rows, p.dev_status)) row = 0;
                        if (!copies) {
                            copy(sQ + q * L::kOperand, r0 / 32, p.q, row);
                            continue;
                        }
                        const int c = lane % kChunks;
                        const char* const from = reinterpret_cast<const char*>(p.q) + c * 16;
#pragma unroll 1
                        for (int i = 0; i < n_rows; i += kPerPass) {
                            const int r = i + lane / kChunks, from_row = __shfl_sync(0xFFFFFFFFu, row, r);
                            const uint32_t to = sQ + q * L::kOperand + chunk_offset(r, c);
#pragma unroll
                            for (int k = 0; k < 4; ++k)  // (rows 32 apart have a chunk in the same place)
                                tc::cp_async_16(to + k * 32 * 128, from + (size_t)from_row * (kD * 2), 16);
                        }
                    }
                    cp_async_arrive_noinc(&sh.q_full[q]);
                }
            }
        } else {
            bool more = open(k);
            // Keys two steps ahead of the values, as the products take them.  A block's rows are looked up once, a
            // step before its keys are loaded, and kept until its values are.
            Cursor v;
            open(v);
            int next = 0, kept0 = 0, kept1 = 0, n_kept = 0;
            Ring ring;
            uint32_t filled = 0;
            if (more) next = row_of(k);
#pragma unroll 1
            for (int i = opaque(-4); v.steps > 0 && !stopped(); ++i) {  // values of a step, keys of the step after the next
                const bool is_k = i & 1;
                if (is_k ? !more : i < 0) continue;
                const Cursor& c = is_k ? k : v;
                if (c.leads()) {
                    const int row = is_k ? next : kept0;
                    if (is_k) {
                        if (next == kMissing) {
                            sh.pieces[k.i % kPieces].spoiled = 1;
                            report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
                        }
                        (n_kept == 0 ? kept0 : kept1) = next;
                        ++n_kept;
                    } else {
                        kept0 = kept1;
                        --n_kept;
                    }
                    uint64_t* const bar = !is_k && c.block() >= c.at->look ? &sh.landed[ring.s] : &sh.full[ring.s];
                    if (filled == kSlots) wait(&sh.empty[ring.s], ring.phase ^ 1);
                    else ++filled;
                    copy(sRing + ring.s * L::kOperand, part, is_k ? p.k_cache : p.v_cache, row);
                    if (__any_sync(0xFFFFFFFFu, row == kMissing)) {  // (what the warp noted of it goes before the arrival)
                        asm volatile("cp.async.wait_all;" ::: "memory");
                        tc::mbar_arrive(bar);
                    } else {
                        cp_async_arrive_noinc(bar);
                    }
                    ring.next();
                }
                if (is_k) {
                    if (++k.u == k.steps) {
                        ++k.i;
                        more = open(k);
                    }
                    if (more && k.leads()) next = row_of(k);
                } else if (++v.u == v.steps) {
                    close(v);
                    ++v.i;
                    open(v);
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == 14) {
        // ================================================================ values that not every row may see
        // The slots go by as in the loading warp.  In a block that some row does not see whole, values that are
        // not finite must not reach that row through a zero weight: their keys are taken out of the block and
        // noted for the warps that add them by hand.
        Ring ring;
        uint32_t gv = 0, parity = 0;
        Cursor k, v;
        bool more = open_ahead(k);
        open_ahead(v);
#pragma unroll 1
        for (int i = opaque(-2); v.steps > 0 && !stopped(); ++i) {
            if (i >= 0 && v.leads()) {
                const Piece& w = *v.at;
                if (v.block() >= w.look) {
                    const uint32_t s = ring.s;
                    const int key0 = w.begin + (w.b0 + v.block()) * kBlock;
                    const bool edge = v.block() >= v.edge, past = key0 + kBlock > w.high && maps.box_rows > 0;
                    wait_ahead(&sh.landed[s], parity >> s);
                    parity ^= 1u << s;
                    unsigned char* const at = base + (2 + s) * L::kOperand;
                    if (lane < 4) sh.odd[gv % kOddRing][lane] = 0;
                    __syncwarp();
                    const int from = max(w.low - key0, 0), to = min(w.high - key0, kBlock);
                    if (past)  // a box holds what lies past the last key
#pragma unroll 1
                        for (int i = to * kChunks + lane; i < (to + maps.box_rows - 1) / maps.box_rows * maps.box_rows * kChunks; i += 32)
                            *reinterpret_cast<uint4*>(at + chunk_offset(i / kChunks, i % kChunks)) = make_uint4(0, 0, 0, 0);
#pragma unroll 1
                    for (int i = from * kChunks + lane; edge && i < to * kChunks; i += 32) {
                        const int r = i / kChunks;
                        const uint4 q = *reinterpret_cast<const uint4*>(at + chunk_offset(r, i % kChunks));
                        const uint32_t x[4] = {q.x, q.y, q.z, q.w};
                        int odd = 0;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            odd |= (x[j] & 0x7F80u) == 0x7F80u || (x[j] & 0x7F800000u) == 0x7F800000u;
                        if (odd) atomicOr(&sh.odd[gv % kOddRing][r >> 5], 1u << (r & 31));
                    }
                    __syncwarp();
#pragma unroll 1
                    for (int r = from; edge && r < to; ++r) {
                        if (!(sh.odd[gv % kOddRing][r >> 5] >> (r & 31) & 1)) continue;
                        if (lane < kChunks) *reinterpret_cast<uint4*>(at + chunk_offset(r, lane)) = make_uint4(0, 0, 0, 0);
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive_n(&sh.full[s], loaders);
                }
                ring.next();
            }
            if (more) {
                if (k.leads()) ring.next();
                if (++k.u == k.steps) {
                    ++k.i;
                    more = open_ahead(k);
                }
            }
            if (i >= 0) {
                ++gv;
                if (++v.u == v.steps) {
                    close(v);
                    ++v.i;
                    open_ahead(v);
                }
            }
        }
    } else if (warp == 12) {
        // ================================================================ products
        constexpr uint32_t idesc_s = tc::idesc_bf16_f32(kTile, kBlock);
        constexpr uint32_t idesc_o = tc::idesc_bf16_f32(kTile, kD) | tc::kIdescBTransposed;
        const bool copied = maps.box_rows == 0;  // (not by the async proxy)
        Ring ring;
        uint32_t n_q = 0, k_slot = 0, k_phase = 0, v_slot = 0;
        int gk = 0, gv = 0;                 // steps of the two walks
        uint32_t used[2] = {0, 0};          // items that used each tile's output
        Cursor k, v;
        bool more = open(k);
        open(v);
        uint32_t odd_phase = 0;              // of odd_done, a bit to a tile
        int owed = 0;             // scores that may be formed
        bool slot_known = false;  // of the next ones' keys
#pragma unroll 1
        for (int i = opaque(-2);; ++i) {  // values of a step, then scores of the step after the next
            if (i >= 0) {
                const int X = gv & 1, sub = v.u & v.pair;
                wait(&sh.p_full[X], gv >> 1);
                if (sub == 0) {
                    v_slot = ring.s;
                    wait(&sh.full[v_slot], ring.phase);
                    ring.next();
                }
                if (v.u < 2) {
                    if (used[X]) wait(&sh.o_free[X], used[X] - 1);
                    ++used[X];
                }
                if (copied) tc::fence_proxy_async_smem();
                tc::tc_fence_after();
                __syncwarp();
                const uint64_t vd = tc::smem_desc_sw128_mn(sRing + v_slot * L::kOperand, L::kHalf);
                // Copies of the rows (32 lanes each) take a quarter of the keys each: the other lanes stay as they are.
                // (Weights of zero for the other quarters would make an infinite value a NaN.)
                const uint32_t off = v.copies ? 0xFFFFFFFFu : 0u;
#pragma unroll
                for (int j = 0; j < kBlock / 16; ++j)
                    tc::umma_bf16_ta_lanes_elect(tmem + kTmemO + X * kBlock, tmem + X * kBlock + 8 * j,
                                                 vd + (uint64_t)(j * (2048 >> 4)), idesc_o,
                                                 v.u >= 2 || (j & 1) || (j != 0 && !off), j >> 1, off);
                if (sub == v.pair) tc::umma_commit_elect(&sh.empty[v_slot]);
                if (v.u + 2 >= v.steps || v.block() >= v.edge) tc::umma_commit_elect(&sh.o_done[X]);
                if (v.block() >= v.edge) {
                    // Weights that values are still to be added by must not be written over by the tile's next scores.
                    const uint32_t* odd = sh.odd[(gv - sub) % kOddRing];
                    if (odd[0] | odd[1] | odd[2] | odd[3]) {
                        wait(&sh.odd_done[X], odd_phase >> X);
                        odd_phase ^= 1u << X;
                    }
                }
                ++gv;
                if (++v.u == v.steps) {
                    close(v);
                    ++v.i;
                    open(v);
                }
            }
            if (v.steps == 0 || stopped()) break;
            ++owed;
#pragma unroll 1
            for (; owed > 0 && more; --owed) {
                const int X = gk & 1, sub = k.u & k.pair;
                const uint32_t q = n_q + sub;
                if (!slot_known && sub == 0) {
                    k_slot = ring.s;
                    k_phase = ring.phase;
                    ring.next();
                }
                slot_known = true;
                // An item's first scores wait for its queries, these for the output of the item before the last, and the
                // product that comes next for neither: it goes first.
                if (k.u == 0 && n_q >= 2 && gk > gv && !test(&sh.q_full[q & 1], q >> 1)) break;
                slot_known = false;
                if (k.u <= k.pair) wait(&sh.q_full[q & 1], q >> 1);
                if (sub == 0) wait(&sh.full[k_slot], k_phase);
                if (copied || k.u <= k.pair) tc::fence_proxy_async_smem();
                tc::tc_fence_after();
                __syncwarp();
                const uint64_t qd = tc::smem_desc_sw128(sQ + (q & 1) * L::kOperand);
                const uint64_t kd = tc::smem_desc_sw128(sRing + k_slot * L::kOperand);
#pragma unroll
                for (int j = 0; j < kD / 16; ++j) {
                    const uint64_t at = (uint64_t)((j >> 2) * (L::kHalf >> 4) + (j & 3) * 2);
                    tc::umma_bf16_elect(tmem + X * kBlock, qd + at, kd + at, idesc_s, j != 0);
                }
                tc::umma_commit_elect(&sh.s_full[X]);
                if (sub == k.pair) tc::umma_commit_elect(&sh.empty[k_slot]);
                if (k.u + k.pair + 1 >= k.steps) tc::umma_commit_elect(&sh.q_empty[q & 1]);
                ++gk;
                if (++k.u == k.steps) {
                    n_q += 1 + k.pair;
                    ++k.i;
                    more = open(k);
                }
            }
        }
        __syncwarp();
        tc::umma_commit_elect(&sh.drain);
        wait_bounded(&sh.drain, 0, &sh.last_limit);  // (whatever made the CTA stop, its products are done before tensor memory is given back)
    } else if (warp == 13) {
        // ================================================================ the pieces, one after the other
        int i = 0;
        auto post = [&](const Piece& x) {
            if (i >= kPieces && !__all_sync(0xFFFFFFFFu, wait_ahead(&sh.piece_empty[i % kPieces], i / kPieces - 1)))
                return;  // (others may still read the one before)
            if (lane == 0) {
                sh.pieces[i % kPieces] = x;
                tc::mbar_arrive(&sh.piece_full[i % kPieces]);
            }
            __syncwarp();
            ++i;
        };
        // this CTA's piece of the line, and the thread whose entries it begins in
        const long long sums = lane < kThreads / 32 ? sh.scan[lane] : 0, upto = scanned(sums);
        const long long total = __shfl_sync(0xFFFFFFFFu, upto, 31), length = piece_length(total, max_ctas);
        const long long x0 = min(blockIdx.x * length, total), x1 = min(x0 + length, total);
        Piece x;
        x.g0 = x.n_q = 0;
        if (x0 < x1) {
            const int w = __ffs(__ballot_sync(0xFFFFFFFFu, x0 < upto)) - 1;
            const long long before = __shfl_sync(0xFFFFFFFFu, upto - sums, w), end = before + scans[32 * w + lane];
            const int l = __ffs(__ballot_sync(0xFFFFFFFFu, x0 < end)) - 1;
            long long start = l ? __shfl_sync(0xFFFFFFFFu, end, max(l - 1, 0)) : before;  // the item's first unit
            __syncwarp();
#pragma unroll 1
            for (int e = (32 * w + l) * per; start < x1 && e < entries && !stopped(); ++e) {
                const Entry en = entry_of<kPrefix>(p, e);
                const long long per_head = en.per_head();
                if (per_head == 0) continue;
                int h = (int)min(divide(max(x0 - start, 0LL), per_head), (long long)p.hkv);
                start += h * per_head;
                int t = h < p.hkv ? (int)min(divide(max(x0 - start, 0LL), en.units(0)), en.tiles - 1LL) : 0;
                start += (long long)t * en.units(0);
#pragma unroll 1
                while (h < p.hkv && start < x1 && !stopped()) {
                    const int log_steps = en.log_steps(t), round = (1 << log_steps) - 1;
                    const int tile_row = t * kRows, n_rows = min(en.n * g - tile_row, kRows);
                    const int high = en.limit((tile_row + n_rows - 1) / g), n_blocks = (high - en.begin + kBlock - 1) / kBlock;
                    const long long first = start + kItemCost;
                    // block b begins at unit first + (b << log_steps)
                    const int b0 = x0 > first ? (int)((x0 - first + round) >> log_steps) : 0;
                    const int b1 = (int)min(max(x1 - first + round, 0LL) >> log_steps, (long long)n_blocks);
                    if (b0 < b1) {
                        x.b0 = b0;
                        x.uncut = b0 == 0 && b1 == n_blocks;
                        x.row0 = en.row0;
                        x.tile_row = tile_row;
                        x.n_rows = n_rows;
                        x.head = h;
                        x.begin = en.begin;
                        x.end = en.end;
                        x.len = en.len;
                        x.table = en.table;
                        x.shared = en.shared;
                        x.low = en.limit(t ? tile_row / g : 0);
                        x.high = high;
                        x.edge = x.low < high ? max((x.low - en.begin) / kBlock - b0, 0) : INT_MAX;
                        x.look = maps.box_rows > 0 && (high - en.begin) % kBlock ? min(x.edge, n_blocks - 1 - b0) : x.edge;
                        x.pair = n_rows > kTile;
                        x.steps = (b1 - b0) << x.pair;
                        x.log_copies = n_rows <= 32 ? 2 : 0;
                        x.last_cta = 0;
                        if (b0 == 0 && !x.uncut)  // (the last CTA with a piece: every one has `length` units)
                            x.last_cta = blockIdx.x + 1 + (int)divide(first + ((n_blocks - 1) << log_steps) - x1, length);
                        // A page that only later rows of the request see spoils these rows too.  (One piece of an item does.)
                        x.spoiled = 0;
                        if (b0 == 0 && high < en.end) {
                            bool missing = false;
#pragma unroll 1
                            for (int pb = (high - 1) / p.page + 1 + lane; (long long)pb * p.page < en.end; pb += 32) {
                                const int id = __ldg(p.block_table + (long long)en.table * p.max_blocks + pb);
                                missing |= id < 0 || id >= p.pool_pages;
                            }
                            x.spoiled = __any_sync(0xFFFFFFFFu, missing);
                            if (x.spoiled) report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
                        }
                        post(x);
                        x.g0 += x.steps;
                        x.n_q += 1 + x.pair;
                    }
                    start += en.units(t);
                    if (++t == en.tiles) {
                        t = 0;
                        ++h;
                    }
                }
            }
        }
        x.steps = 0;
        post(x);
        // requests that cannot be right
#pragma unroll 1
        for (int r = blockIdx.x; r < p.R; r += gridDim.x) {
            const int n = p.cu[r + 1] - p.cu[r];
            if (n == 0 || entry_of<kPrefix>(p, kPrefix ? p.n_groups + r : r).n > 0) continue;
            const long long from = (long long)p.cu[r] * p.hq, to = (long long)p.cu[r + 1] * p.hq;
#pragma unroll 1
            for (long long j = from * kD + lane; j < to * kD; j += 32) p.out[j] = kNan;
            if (p.lse)
#pragma unroll 1
                for (long long j = from + lane; j < to; j += 32) p.lse[j] = __int_as_float(0x7FC00000);
            if (kPrefix)
#pragma unroll 1
                for (int h = 0; h < p.hkv; ++h)
                    for (long long j = (long long)p.cu[r] * g + lane; j < (long long)p.cu[r + 1] * g; j += 32)
                        plan.where[(long long)h * p.rows * g + j] = Where::kSkip;
            if (lane == 0) report(p.dev_status, DSPARK_ERR_DEVICE_INPUT);
        }
    }
    __syncwarp();
    __syncthreads();
    if (sh.limit == 0) {
        if (tid == 0) report(p.dev_status, DSPARK_ERR_TIMEOUT);
        for (const uint64_t t0 = global_ns(); global_ns() - t0 < 1000000;) {}  // (copies in flight land before the CTA ends)
    }
    if (warp == 12) tc::tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- joining the pieces
constexpr int kJoinCols = 16;  // of a CTA

// A row's sums over 16 columns, from col (in fours) on.
struct RowSum {
    static constexpr int kQuads = kJoinCols / 4;
    float m = -INFINITY, l = 0.0f;
    float4 o[kQuads] = {};

    __device__ __forceinline__ void add(float2 ml, const float4* from, size_t step) {
        const float top = fmaxf(m, ml.x);
        const float fa = m == -INFINITY ? 0.0f : exp2_approx(m - top), fb = ml.x == -INFINITY ? 0.0f : exp2_approx(ml.x - top);
        l = (m == -INFINITY ? l : l * fa) + (ml.x == -INFINITY ? ml.y : ml.y * fb);
        m = top;
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
            const float4 v = from[q * step];
            o[q].x = o[q].x * fa + v.x * fb; o[q].y = o[q].y * fa + v.y * fb;
            o[q].z = o[q].z * fa + v.z * fb; o[q].w = o[q].w * fa + v.w * fb;
        }
    }
    // Row r of the item that CTAs first .. last have pieces of: the k-th of them and every n-th from there on.
    template <int kD>
    __device__ __forceinline__ void add_pieces(const Plan& plan, int first, int last, int k, int n, int r, int col, int32_t* dev_status) {
#pragma unroll 4
        for (int c = first + k; c <= last && IN_BOUNDS(c >= 0 && c < kMaxCtas && r >= 0 && r < kRows, dev_status); c += n) {
            const size_t slot = (size_t)(2 * c + (c == first)) * kRows;
            add(plan.part_ml[slot + r], reinterpret_cast<const float4*>(plan.part + slot * kD) + col * kRows + r, kRows);
        }
    }
    // Adds the sums of the threads `apart` from each other to those of the first of them.  (Called by the whole CTA.)
    __device__ __forceinline__ void gather(int apart) {
        __shared__ float2 all_ml[kRows];
        __shared__ float4 all[kQuads][kRows];
        all_ml[threadIdx.x] = make_float2(m, l);
#pragma unroll
        for (int q = 0; q < kQuads; ++q) all[q][threadIdx.x] = o[q];
        __syncthreads();
        if (threadIdx.x < apart)
#pragma unroll 1
            for (int t = threadIdx.x + apart; t < kRows; t += apart) add(all_ml[t], &all[0][t], kRows);
    }
    template <int kD>
    __device__ __forceinline__ void write(const AttnParams& p, size_t row, int col) const {
        if (!IN_BOUNDS(row < (size_t)p.rows * p.hq && col * 4 < p.d, p.dev_status)) return;
        const float inv = 1.0f / l;
        alignas(16) __nv_bfloat162 w[2 * kQuads];
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
            w[2 * q] = __floats2bfloat162_rn(o[q].x * inv, o[q].y * inv);
            w[2 * q + 1] = __floats2bfloat162_rn(o[q].z * inv, o[q].w * inv);
        }
        uint4* to = reinterpret_cast<uint4*>(p.out + row * kD + col * 4);
#pragma unroll
        for (int q = 0; q < kQuads / 2; ++q) to[q] = reinterpret_cast<const uint4*>(w)[q];
        if (p.lse && col == 0) p.lse[row] = (m + log2f(l)) * kLn2;
    }
};

// CTA (c, i): columns [16 i, 16 i + 16) of the item that CTA c of the attention
// kernel began and did not finish.  A thread to a row; where there are many pieces
// and few rows, up to 32 threads that share the pieces (a request of 13000 keys in 50
// of them: 16 us instead of 38; where there are few it costs 0.6 us).
constexpr int kManyPieces = 8;
template <int kD>
__global__ void __launch_bounds__(kRows) join_kernel(const AttnParams p, const Plan plan) {
    launch_dependents();
    wait_prior_grid();
    const Job job = plan.jobs[blockIdx.x];
    const bool share = job.last - job.first >= kManyPieces;
    if (!share && (int)threadIdx.x >= job.n_rows) return;
    int log_rows = share ? 3 : 8;
    while (1 << log_rows < job.n_rows) ++log_rows;
    const int r = threadIdx.x & ((1 << log_rows) - 1), g = p.hq / p.hkv, col = blockIdx.y * RowSum::kQuads;
    RowSum sum;
    if (r < job.n_rows) sum.add_pieces<kD>(plan, job.first, job.last, threadIdx.x >> log_rows, kRows >> log_rows, r, col, p.dev_status);
    if (share) sum.gather(1 << log_rows);
    if ((int)threadIdx.x >= job.n_rows) return;
    const int i = (job.tile_row + r) / g;
    sum.write<kD>(p, (size_t)(job.row0 + i) * p.hq + job.head * g + (job.tile_row + r - i * g), col);
}

// CTA (i, j): columns [16 j, 16 j + 16) of 2^log_rows rows of a key head: their
// shared parts, then their own.  (256 / 2^log_rows threads to a row share the pieces.)
template <int kD>
__global__ void __launch_bounds__(kRows) prefix_join_kernel(const AttnParams p, const Plan plan, const int log_rows) {
    launch_dependents();
    wait_prior_grid();
    const int g = p.hq / p.hkv, col = blockIdx.y * RowSum::kQuads, k = threadIdx.x >> log_rows;
    const long long lins = (long long)p.rows * g, blocks = (lins + (1 << log_rows) - 1) >> log_rows;
    const int head = (int)(blockIdx.x / blocks);
    const long long lin = ((blockIdx.x - head * blocks) << log_rows) + threadIdx.x - (k << log_rows), row = lin / g;
    const int own = row < min(p.cu[p.R], p.rows) ? plan.where[head * lins + lin] : Where::kSkip;
    RowSum sum;
#pragma unroll
    for (int side = 1; side >= 0; --side) {
        if (own == Where::kSkip || (side && !(own & Where::kShared))) continue;
        const long long at = (side * p.hkv + head) * lins + lin;
        const int w = side ? plan.where[at] : own;
        if (w & Where::kCut) sum.add_pieces<kD>(plan, w >> 16 & 255, min(w >> 8 & 255, kMaxCtas - 1), k, kRows >> log_rows, w & 255, col, p.dev_status);
        else if (k == 0) sum.add(plan.whole_ml[at], reinterpret_cast<const float4*>(plan.whole) + (at - lin) * (kD / 4) + col * lins + lin, lins);
    }
    if (kRows >> log_rows > 1) sum.gather(1 << log_rows);
    if (k == 0 && own != Where::kSkip) sum.write<kD>(p, row * p.hq + head * g + (lin - row * g), col);
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

// The plan in the workspace; its size.
size_t plan_at(void* ws, Plan& p, long long items, int d, bool prefix) {
    unsigned char* b = static_cast<unsigned char*>(ws);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        void* at = b + off;
        off += up(bytes);
        return at;
    };
    p.part = static_cast<float*>(take(sizeof(float) * 2 * kMaxCtas * kRows * (size_t)d));
    p.part_ml = static_cast<float2*>(take(sizeof(float2) * 2 * kMaxCtas * kRows));
    p.jobs = static_cast<Job*>(take(prefix ? 0 : sizeof(Job) * kMaxCtas));
    p.whole = static_cast<float*>(take(prefix ? sizeof(float) * 2 * (size_t)items * d : 0));
    p.whole_ml = static_cast<float2*>(take(prefix ? sizeof(float2) * 2 * (size_t)items : 0));
    p.where = static_cast<int*>(take(prefix ? sizeof(int) * 2 * (size_t)items : 0));
    return off;
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

// A [rows, d] matrix of bf16 in boxes of box_rows x 64.
bool encode_boxes(CUtensorMap* m, const void* base, long long rows, int d, int box_rows) {
    const EncodeTiled enc = encoder();
    const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)d * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    const cuuint32_t es[2] = {1, 1};
    return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kD, bool kPrefix>
cudaError_t launch_as(const AttnParams& p, cudaStream_t stream) {
    Maps maps{};
    int box_rows = 128;  // the largest power of two that every page is a multiple of
    while (p.page % box_rows) box_rows /= 2;
    if (box_rows >= 8 && p.pool_pages > 0) {
        const long long rows = (long long)p.pool_pages * p.hkv * p.page;
        if (!encode_boxes(&maps.k, p.k_cache, rows, kD, box_rows) || !encode_boxes(&maps.v, p.v_cache, rows, kD, box_rows))
            return cudaErrorInvalidValue;
        maps.box_rows = box_rows;
    }
    int dev = 0, n_sm = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if ((err = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return err;
    const int ctas = n_sm < kMaxCtas ? n_sm : kMaxCtas;
    Plan plan;
    plan_at(p.ws, plan, (long long)p.rows * p.hq, kD, kPrefix);
    const int smem = Layout<kD>::kTotal;
    if ((err = cudaFuncSetAttribute(attention_kernel<kD, kPrefix>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
        return err;
    if ((err = launch_after(attention_kernel<kD, kPrefix>, dim3(ctas), kThreads, smem, stream, p, plan, ctas,
                            kPrefix ? p.n_groups + p.R : p.R, maps)) != cudaSuccess)
        return err;
    if (!kPrefix) return launch_after(join_kernel<kD>, dim3(ctas, kD / kJoinCols), kRows, 0, stream, p, plan);
    // Few rows are few items in many pieces: eight threads to a row up to 4096 rows of all heads.  Eight threads, one: 27 and
    // 33 us at 1900 rows (of 32 query heads behind a prefix of 4096), 36.8 and 38.1 at 3500, 42.4 and 42.7 at 4700, 56 and 54
    // at 7800, 79 and 71 at 11600.
    const long long lins = (long long)p.rows * (p.hq / p.hkv);
    const int log_rows = lins * p.hkv <= 16 * kRows ? 5 : 8;
    const long long blocks = ((lins + (1 << log_rows) - 1) >> log_rows) * p.hkv;
    return launch_after(prefix_join_kernel<kD>, dim3((unsigned)blocks, kD / kJoinCols), kRows, 0, stream, p, plan, log_rows);
}

template <int kD>
cudaError_t launch_d(const AttnParams& p, cudaStream_t stream) {
    return p.n_groups > 0 ? launch_as<kD, true>(p, stream) : launch_as<kD, false>(p, stream);
}

}  // namespace

size_t attention_workspace(int, int n_groups, int rows, int hq, int, int d) {
    Plan plan;
    return plan_at(nullptr, plan, (long long)rows * hq, d, n_groups > 0);
}

cudaError_t launch_attention(const AttnParams& p, cudaStream_t stream) {
    return p.d == 64 ? launch_d<64>(p, stream) : launch_d<128>(p, stream);
}

}  // namespace dspark
