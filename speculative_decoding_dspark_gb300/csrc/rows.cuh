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
__device__ __forceinline__ void cluster_st_u64(uint32_t a, uint64_t x) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(x) : "memory");
}

// ---- rows ---------------------------------------------------------------------
template <typename T> struct Elem;  // T: float, or uint16_t for the bits of a bf16
template <> struct Elem<float> {
    static constexpr int kVec = 4;
    static constexpr uint32_t kMinusInf = 0xFF800000u;  // a 32-bit word of them
    static __device__ __forceinline__ float to_float(float x) { return x; }
    static __device__ __forceinline__ void unpack(const uint4& w, float* f) {
        f[0] = __uint_as_float(w.x); f[1] = __uint_as_float(w.y);
        f[2] = __uint_as_float(w.z); f[3] = __uint_as_float(w.w);
    }
};
template <> struct Elem<uint16_t> {
    static constexpr int kVec = 8;
    static constexpr uint32_t kMinusInf = 0xFF80FF80u;
    static __device__ __forceinline__ float to_float(uint16_t x) { return bf16_bits_to_float(x); }
    static __device__ __forceinline__ void unpack(const uint4& w, float* f) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
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
// The difference comes first: rows whose values are all near the type's lowest
// keep their sums (x c2 alone would overflow).  A NaN makes s a NaN.
struct SoftSum {
    float m = -INFINITY, s = 0.0f, u = 0.0f;
};

template <bool kEntropy>
__device__ __forceinline__ void soft_merge(SoftSum& a, const SoftSum& b, float c2) {
    if (b.m == -INFINITY) {
        a.s += b.s;  // nothing, or a NaN
        return;
    }
    if (a.m == -INFINITY) {
        const float s = a.s;
        a = b;
        a.s += s;
        return;
    }
    const float m = fmaxf(a.m, b.m);
    const float da = fmaxf((a.m - m) * c2, -200.0f), db = fmaxf((b.m - m) * c2, -200.0f);
    const float fa = exp2_approx(da), fb = exp2_approx(db);
    if (kEntropy) a.u = fa * (a.u + da * a.s) + fb * (b.u + db * b.s);
    a.s = fa * a.s + fb * b.s;
    a.m = m;
}

// N more values.  Their largest comes first, so that one rescaling serves all.
template <bool kEntropy, int N>
__device__ __forceinline__ float soft_add(SoftSum& t, const float (&x)[N], float c2) {
    float g[N];
#pragma unroll
    for (int i = 0; i < N; ++i) g[i] = x[i];
#pragma unroll
    for (int o = N / 2; o > 0; o /= 2)
#pragma unroll
        for (int i = 0; i < o; ++i) g[i] = max_nan(g[i], g[i + o]);
    const float top = g[0];
    if (!(top <= t.m)) {
        if (top != top) {
            t.s = top;
        } else {
            if (t.m != -INFINITY) {
                const float d = fmaxf((t.m - top) * c2, -200.0f), f = exp2_approx(d);
                if (kEntropy) t.u = f * (t.u + d * t.s);
                t.s *= f;
            }
            t.m = top;
        }
    }
    if (t.m == -INFINITY) return top;
    const float2 minus = make_float2(-t.m, -t.m), scale = make_float2(c2, c2);
    float2 s = make_float2(0.0f, 0.0f), u = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        float2 a = mul2(add2(make_float2(x[i], x[i + 1]), minus), scale);
        if (kEntropy) {  // (2^-200 is zero, and so is its product)
            a.x = fmaxf(a.x, -200.0f);
            a.y = fmaxf(a.y, -200.0f);
        }
        const float2 e = make_float2(exp2_approx(a.x), exp2_approx(a.y));
        s = add2(s, e);
        if (kEntropy) u = fma2(e, a, u);
    }
    t.s += s.x + s.y;
    if (kEntropy) t.u += u.x + u.y;
    return top;
}

}  // namespace dspark
