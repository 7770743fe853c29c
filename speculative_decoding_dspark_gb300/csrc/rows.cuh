// rows.cuh -- device helpers of the kernels that stream vocabulary rows of any
// length, stride and alignment (logprobs.cu, distill.cu).
//
// A row is walked in 16-byte pieces from its first 16-byte boundary on; the few
// elements before and after these are read one by one.  A row is shared by the CTAs of a cluster, each taking a
// contiguous range of pieces, which join their results through distributed
// shared memory: no workspace, and nothing to clear between calls.
#pragma once

#include "common.cuh"

namespace dspark {

// Shared memory that every kernel may have beside its own static arrays without asking for it
// (which takes 0.4 us of a call's 3.7).
constexpr size_t kSharedAnyway = 32 * 1024;

constexpr float kLog2eF = 1.4426950408889634f;
constexpr float kLn2F = 0.6931471805599453f;

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The larger one; a NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// Two floats in one 64-bit register, and the operations on both at once.
using Two = unsigned long long;
__device__ __forceinline__ Two two(float lo, float hi) {
    Two y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(lo), "f"(hi));
    return y;
}
__device__ __forceinline__ float2 split(Two x) {
    float2 y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(y.x), "=f"(y.y) : "l"(x));
    return y;
}
__device__ __forceinline__ Two add_two(Two a, Two b) {
    Two y;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}
__device__ __forceinline__ Two mul_two(Two a, Two b) {
    Two y;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}
__device__ __forceinline__ Two fma_two(Two a, Two b, Two c) {
    Two y;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(a), "l"(b), "l"(c));
    return y;
}

// ---- clusters ---------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// The two halves of it; a thread waits before it arrives again.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// All threads of the cluster meet; shared-memory writes before it are visible after it.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The address of `p` (this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_map(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float cluster_ld_f32(uint32_t a) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t cluster_ld_u32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t cluster_atomic_add(uint32_t a, uint32_t x) {
    uint32_t v;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(v) : "r"(a), "r"(x) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_st_f32(uint32_t a, float x) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(x) : "memory");
}
__device__ __forceinline__ void cluster_st_f32x2(uint32_t a, float x, float y) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ void cluster_st_u64(uint32_t a, uint64_t x) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(x) : "memory");
}

// ---- rows ---------------------------------------------------------------------
template <typename T> struct Elem;  // T: float, or uint16_t for the bits of a bf16
template <> struct Elem<float> {
    static constexpr int kVec = 4;
    static constexpr uint32_t kMinusInf = 0xFF800000u;  // a 32-bit word of them
    static __device__ __forceinline__ float to_float(float x) { return x; }
    // Elements 2 i and 2 i + 1 of a piece.
    static __device__ __forceinline__ Two pair(const uint4& w, int i) {
        return i == 0 ? two(__uint_as_float(w.x), __uint_as_float(w.y)) : two(__uint_as_float(w.z), __uint_as_float(w.w));
    }
    static __device__ __forceinline__ float at(const uint4& w, int e) {
        return __uint_as_float(e == 0 ? w.x : e == 1 ? w.y : e == 2 ? w.z : w.w);
    }
    static __device__ __forceinline__ uint4 without(const uint4& w, uint32_t mask) {  // -inf where mask has a bit
        return make_uint4(mask & 1 ? kMinusInf : w.x, mask & 2 ? kMinusInf : w.y, mask & 4 ? kMinusInf : w.z,
                          mask & 8 ? kMinusInf : w.w);
    }
    template <int N>
    static __device__ __forceinline__ float largest(const uint4 (&w)[N]) {
        float m = __uint_as_float(w[0].x);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            m = max3_nan(m, __uint_as_float(w[i].x), __uint_as_float(w[i].y));
            m = max3_nan(m, __uint_as_float(w[i].z), __uint_as_float(w[i].w));
        }
        return m;
    }
};
template <> struct Elem<uint16_t> {
    static constexpr int kVec = 8;
    static constexpr uint32_t kMinusInf = 0xFF80FF80u;
    static __device__ __forceinline__ float to_float(uint16_t x) { return bf16_bits_to_float(x); }
    static __device__ __forceinline__ Two pair(const uint4& w, int i) {
        const uint32_t u = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
        return two(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
    }
    static __device__ __forceinline__ float at(const uint4& w, int e) {
        const uint32_t u = e < 2 ? w.x : e < 4 ? w.y : e < 6 ? w.z : w.w;
        return __uint_as_float(e & 1 ? u & 0xFFFF0000u : u << 16);
    }
    static __device__ __forceinline__ uint32_t without(uint32_t u, uint32_t mask) {
        const uint32_t off = (mask & 1 ? 0xFFFFu : 0u) | (mask & 2 ? 0xFFFF0000u : 0u);
        return (u & ~off) | (kMinusInf & off);
    }
    static __device__ __forceinline__ uint4 without(const uint4& w, uint32_t mask) {
        return make_uint4(without(w.x, mask), without(w.y, mask >> 2), without(w.z, mask >> 4), without(w.w, mask >> 6));
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t y;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
        return y;
    }
    template <int N>
    static __device__ __forceinline__ float largest(const uint4 (&w)[N]) {
        uint32_t m = max2(max2(w[0].x, w[0].y), max2(w[0].z, w[0].w));
#pragma unroll
        for (int i = 1; i < N; ++i) m = max2(m, max2(max2(w[i].x, w[i].y), max2(w[i].z, w[i].w)));
        return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    }
};

// A row's 16-byte pieces, from the first 16-byte boundary within it, and the few
// elements before and after them (the edges).
template <typename T>
struct RowView {
    const T* row;
    const uint4* base;
    int V, head, pieces;  // elements before the first piece, whole pieces
    __device__ __forceinline__ RowView(const T* p, int V_) : row(p), V(V_) {
        constexpr int kVec = Elem<T>::kVec;
        head = min(V, (int)(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T)));
        base = reinterpret_cast<const uint4*>(p + head);
        pieces = (V - head) / kVec;
    }
    // The edge element of thread `tid` in a CTA whose first and last pieces are the row's
    // (-1: none): the elements before the pieces, then those after them.
    __device__ __forceinline__ int edge(int tid, bool first, bool last) const {
        constexpr int kVec = Elem<T>::kVec;
        if (tid < kVec) return first && tid < head ? tid : -1;
        const int v = head + pieces * kVec + tid - kVec;
        return last && v < V ? v : -1;
    }
    __device__ __forceinline__ float at(int v) const { return Elem<T>::to_float(row[v]); }
};

// The row's piece i if i < end, else -inf everywhere.
template <typename T>
__device__ __forceinline__ uint4 load_piece(const uint4* base, int i, int end) {
    constexpr uint32_t k = Elem<T>::kMinusInf;
    return i < end ? __ldcs(base + i) : make_uint4(k, k, k, k);
}

// ---- the running softmax sums of a row --------------------------------------------
// m the largest x, s = sum 2^a and u = sum a 2^a over the x seen, a = (x - m) c2.
// The difference comes first: the largest value's a is 0, and rows whose values are
// all near the type's lowest keep their sums (x c2 alone would overflow).  A NaN
// makes s a NaN.
struct SoftSum {
    float m = -INFINITY, s = 0.0f, u = 0.0f;
};

// The sums of kWidth neighbouring lanes, in each of them: the maximum first, then
// each lane's sums brought to it.
template <bool kEntropy, int kWidth>
__device__ __forceinline__ SoftSum soft_join(const SoftSum& t, float c2) {
    SoftSum a;
    a.m = t.m;
#pragma unroll
    for (int o = kWidth / 2; o > 0; o >>= 1) a.m = fmaxf(a.m, shfl_xor(a.m, o));
    const bool none = t.m == -INFINITY;  // (s is 0, or a NaN)
    const float d = none ? 0.0f : fmaxf((t.m - a.m) * c2, -200.0f), f = exp2_approx(d);
    a.s = f * t.s;
    if (kEntropy) a.u = f * (t.u + d * t.s);
#pragma unroll
    for (int o = kWidth / 2; o > 0; o >>= 1) {
        a.s += shfl_xor(a.s, o);
        if (kEntropy) a.u += shfl_xor(a.u, o);
    }
    return a;
}

// `top`, a new value or the largest of several, may be the new maximum.
template <bool kEntropy>
__device__ __forceinline__ void soft_raise(SoftSum& t, float top, float c2) {
    if (top <= t.m) return;
    if (top != top) {
        t.s = top;
        return;
    }
    if (t.m != -INFINITY) {
        const float d = fmaxf((t.m - top) * c2, -200.0f), f = exp2_approx(d);
        if (kEntropy) t.u = f * (t.u + d * t.s);
        t.s *= f;
    }
    t.m = top;
}

// N more pieces; returns their largest value.  It comes first, so that one rescaling serves all.
template <typename T, bool kEntropy, int N>
__device__ __forceinline__ float soft_add(SoftSum& t, const uint4 (&w)[N], float c2) {
    const float top = Elem<T>::largest(w);
    soft_raise<kEntropy>(t, top, c2);
    if (t.m == -INFINITY) return top;
    Two s0 = two(0.0f, 0.0f), s1 = s0, u0 = s0;
    const Two scale = two(c2, c2), minus = two(-t.m, -t.m);
#pragma unroll
    for (int q = 0; q < N; ++q)
#pragma unroll
        for (int i = 0; i < Elem<T>::kVec / 2; ++i) {
            float2 a = split(mul_two(add_two(Elem<T>::pair(w[q], i), minus), scale));
            if (kEntropy) {  // (2^-200 is zero, and so is its product)
                a.x = fmaxf(a.x, -200.0f);
                a.y = fmaxf(a.y, -200.0f);
            }
            const Two e = two(exp2_approx(a.x), exp2_approx(a.y));
            if (i & 1) s1 = add_two(s1, e);
            else s0 = add_two(s0, e);
            if (kEntropy) u0 = fma_two(e, two(a.x, a.y), u0);
        }
    const float2 s = split(add_two(s0, s1));
    t.s += s.x + s.y;
    if (kEntropy) {
        const float2 u = split(u0);
        t.u += u.x + u.y;
    }
    return top;
}

// One more value.
template <bool kEntropy>
__device__ __forceinline__ void soft_add_one(SoftSum& t, float x, float c2) {
    soft_raise<kEntropy>(t, x, c2);
    if (t.m == -INFINITY) return;
    const float a = fmaxf((x - t.m) * c2, -200.0f), e = exp2_approx(a);
    t.s += e;
    if (kEntropy) t.u += e * a;
}

}  // namespace dspark
