// Shared by the kernels of what stands around a recurrence: vectors of elements, and the slots of decode steps.
#pragma once
#include <type_traits>

#include "kda_common.cuh"

namespace kda {
namespace layer {

// at most 16-byte aligned: eight fp32 beside eight bf16 move as two pieces
template <typename T, int V> struct alignas(sizeof(T) * V < 16 ? sizeof(T) * V : 16) vec {
    T x[V];
};
template <typename T, int V> __device__ __forceinline__ vec<T, V> load(const T *p) { return *reinterpret_cast<const vec<T, V> *>(p); }
// written once: evicted first
template <typename T, int V> __device__ __forceinline__ void store_once(T *p, const vec<T, V> &v) {
    if constexpr (sizeof(v) == 16) __stcs(reinterpret_cast<uint4 *>(p), *reinterpret_cast<const uint4 *>(&v));
    else if constexpr (sizeof(v) == 8) __stcs(reinterpret_cast<uint2 *>(p), *reinterpret_cast<const uint2 *>(&v));
    else *reinterpret_cast<vec<T, V> *>(p) = v;
}
template <typename T, int V> __device__ __forceinline__ void store(T *p, const vec<T, V> &v) { *reinterpret_cast<vec<T, V> *>(p) = v; }

// V values as fp32 and back, two bf16 at a time
template <typename T, int V> __device__ __forceinline__ void unpack(const vec<T, V> &v, float *f) {
    if constexpr (sizeof(T) == 2 && V > 1) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&v);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = ld(&v.x[i]);
    }
}
template <typename T, int V> __device__ __forceinline__ vec<T, V> pack(const float *f) {
    vec<T, V> v;
    if constexpr (sizeof(T) == 2 && V > 1) {
        __nv_bfloat162 *w = reinterpret_cast<__nv_bfloat162 *>(&v);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) w[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) st(&v.x[i], f[i]);
    }
    return v;
}

// Arithmetic on one fp32 or on two at a time (one instruction for both)
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 add(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
template <typename F> __device__ __forceinline__ F splat(float x);
template <> __device__ __forceinline__ float splat<float>(float x) { return x; }
template <> __device__ __forceinline__ float2 splat<float2>(float x) { return make_float2(x, x); }
// f of each
template <typename Fn> __device__ __forceinline__ float each(Fn f, float a) { return f(a); }
template <typename Fn> __device__ __forceinline__ float2 each(Fn f, float2 a) { return make_float2(f(a.x), f(a.y)); }
template <typename Fn> __device__ __forceinline__ float each(Fn f, float a, float b) { return f(a, b); }
template <typename Fn> __device__ __forceinline__ float2 each(Fn f, float2 a, float2 b) { return make_float2(f(a.x, b.x), f(a.y, b.y)); }
template <typename Fn> __device__ __forceinline__ float each(Fn f, float a, float b, float c) { return f(a, b, c); }
template <typename Fn> __device__ __forceinline__ float2 each(Fn f, float2 a, float2 b, float2 c) {
    return make_float2(f(a.x, b.x, c.x), f(a.y, b.y, c.y));
}
// 2^x, 1 / x and 1 / sqrt(x) by the special function unit, each to about 2^-22 of itself; results (and arguments) below the
// normal range count as 0
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rsq(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 ex2(float2 x) { return make_float2(ex2(x.x), ex2(x.y)); }
__device__ __forceinline__ float2 rcp(float2 x) { return make_float2(rcp(x.x), rcp(x.y)); }
__device__ __forceinline__ float2 rsq(float2 x) { return make_float2(rsq(x.x), rsq(x.y)); }

constexpr float LOG2E = 1.4426950408889634f;

// Sigmoid(y); 2^-y overflows to infinity and the quotient is 0
template <typename F> __device__ __forceinline__ F sigmoid(F y) { return rcp(add(ex2(mul(y, splat<F>(-LOG2E))), splat<F>(1.f))); }
// Sigmoid(y) and 1 - Sigmoid(y), each to a few units of 2^-23 of itself; both 0 where Sigmoid(y) is below 2^-126
template <typename F> struct sig {
    F s, n;
};
template <typename F> __device__ __forceinline__ sig<F> sigmoids(F y) {
    // (at most 2^127, whose quotient counts as 0, so that no infinity meets it; min.NaN keeps a NaN)
    const F e = ex2(each([](float v) {
        float t;
        asm("min.NaN.f32 %0, %1, 0f42FE0000;" : "=f"(t) : "f"(v));
        return t;
    }, mul(y, splat<F>(-LOG2E))));
    const F s = rcp(add(e, splat<F>(1.f)));
    return {s, mul(e, s)};
}

// V values as V / K pairs or single ones
template <int V> struct lanes {
    static constexpr int K = V % 2 == 0 ? 2 : 1, N = V / K;
    using F = typename std::conditional<K == 2, float2, float>::type;
};
template <typename T, int V, typename F> __device__ __forceinline__ void unpack(const vec<T, V> &v, F *f) {
    unpack<T, V>(v, reinterpret_cast<float *>(f));
}
template <typename T, int V, typename F> __device__ __forceinline__ vec<T, V> pack(const F *f) {
    return pack<T, V>(reinterpret_cast<const float *>(f));
}

// The slot of row n of a step: -1 for a row of a padded batch and for a slot outside the pool (which sets the device error).  Whether an
// earlier row has the slot, so that nothing of this one is written (an error as well), every thread of the block of NT asks
// when it has its loads on their way: the answer takes a trip to memory for every NT rows.
__device__ __forceinline__ int64_t slot_of(const int32_t *idx, int64_t slots, int64_t n, int *err) {
    if (!idx) return n;
    const int32_t s = idx[n];
    if (s >= 0 && s < slots) return s;
    if (s != -1 && threadIdx.x == 0) set_error(err, KDA_ERR_BAD_STATE_INDEX);
    return -1;
}
template <int NT> __device__ __forceinline__ bool taken(const int32_t *idx, int64_t n, int64_t slot, int *err) {
    if (!idx) return false;
    bool bad = false;
    for (int64_t m = threadIdx.x; m < n; m += NT) bad |= idx[m] == (int32_t)slot;
    if (!__syncthreads_or(bad)) return false;
    if (threadIdx.x == 0) set_error(err, KDA_ERR_BAD_STATE_INDEX);
    return true;
}

}  // namespace layer
}  // namespace kda
