// Shared by the kernels of what stands around a recurrence: vectors of elements, and the slots of decode steps.
#pragma once
#include "kda_common.cuh"

namespace kda {
namespace layer {

// at most 16-byte aligned: eight fp32 beside eight bf16 move as two pieces
template <typename T, int V> struct alignas(sizeof(T) * V < 16 ? sizeof(T) * V : 16) vec {
    T x[V];
};
template <typename T, int V> __device__ __forceinline__ vec<T, V> load(const T *p) { return *reinterpret_cast<const vec<T, V> *>(p); }
// read once, written once: evicted first
template <typename T, int V> __device__ __forceinline__ vec<T, V> load_once(const T *p) {
    vec<T, V> v;
    if constexpr (sizeof(v) == 16) *reinterpret_cast<uint4 *>(&v) = __ldcs(reinterpret_cast<const uint4 *>(p));
    else if constexpr (sizeof(v) == 8) *reinterpret_cast<uint2 *>(&v) = __ldcs(reinterpret_cast<const uint2 *>(p));
    else v = load<T, V>(p);
    return v;
}
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

// The slot of row n of a step.  False for a row of a padded batch (-1), for a slot outside the pool, and for one
// that an earlier row has (both set the device error); every thread of the block of NT gets the same answer.
template <int NT>
__device__ __forceinline__ bool find_slot(const int32_t *idx, int64_t slots, int64_t n, int64_t *slot, int *err) {
    *slot = n;
    if (!idx) return true;
    const int32_t s = idx[n];
    if (s == -1) return false;
    bool bad = s < 0 || s >= slots;
    if (!bad)
        for (int64_t m = threadIdx.x; m < n; m += NT) bad |= idx[m] == s;
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) set_error(err, KDA_ERR_BAD_STATE_INDEX);
        return false;
    }
    *slot = s;
    return true;
}

}  // namespace layer
}  // namespace kda
