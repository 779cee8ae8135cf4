// Shared by the two directions of kda_block_norm: a row's place in a block of threads, its sums, and which variant a
// call takes.
#pragma once
#include "kda_internal.h"
#include "kda_layer.cuh"

namespace kda {
namespace norm {

// NT threads on a row (a warp, with four rows to a block, or a whole block), each with E vectors of V elements: vector
// e begins at column (e * NT + thread) * V.
template <int NT> struct place {
    static constexpr int BLOCK = NT < 128 ? 128 : NT;
    static constexpr int ROWS = BLOCK / NT;
};

// N sums over the NT threads of a row.  `at` alternates between two places of shared memory, so that one barrier
// separates a sum's parts from the sum after the next.
template <int NT, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float *shared, int &at) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    if constexpr (NT > 32) {
        constexpr int W = NT / 32;
        float *s = shared + at * (2 * W);
        at ^= 1;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) s[i * W + (threadIdx.x >> 5)] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) v[i] += s[i * W + w];
        }
    }
}

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

template <int V> __device__ __forceinline__ void load_weight(const float *w, int c, float *f) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = 1.f;
        return;
    }
    layer::unpack<float, V>(layer::load<float, V>(w + c), f);
}

// Calls go(T, RT, V, E, NT as a tag) for a call's types and sizes: 16-byte vectors of dtype where every row's address allows
// them, the fewest threads that hold a row at 8 (D up to 2048) or 16 elements each.
template <typename T, typename RT, int V, int E, int NT> struct tag {
    using t = T;
    using rt = RT;
    static constexpr int v = V, e = E, nt = NT;
};
template <typename T, typename RT, typename F>
void choose_size(int D, bool wide, F &&go) {
    constexpr int V = 16 / (int)sizeof(T);
    if (wide) {
        if (D <= 256) go(tag<T, RT, V, 8 / V, 32>{});
        else if (D <= 512) go(tag<T, RT, V, 16 / V, 32>{});
        else if (D <= 1024) go(tag<T, RT, V, 8 / V, 128>{});
        else if (D <= 2048) go(tag<T, RT, V, 8 / V, 256>{});
        else if (D <= 4096) go(tag<T, RT, V, 16 / V, 256>{});
        else go(tag<T, RT, V, 16 / V, 512>{});
    } else {
        if (D <= 512) go(tag<T, RT, 1, 16, 32>{});
        else if (D <= 2048) go(tag<T, RT, 1, 16, 128>{});
        else go(tag<T, RT, 1, 16, 512>{});
    }
}
template <typename F>
void choose(kda_dtype_t dtype, kda_dtype_t residual, int D, bool wide, F &&go) {
    if (dtype == KDA_F32) choose_size<float, float>(D, wide, go);
    else if (residual == KDA_F32) choose_size<bf16, float>(D, wide, go);
    else choose_size<bf16, bf16>(D, wide, go);
}
// whether all of these (NULL: absent) may be read and written as 16-byte vectors
template <int N> bool all_wide(int D, kda_dtype_t dtype, const void *const (&p)[N]) {
    if (D % (dtype == KDA_BF16 ? 8 : 4)) return false;
    uintptr_t any = 0;
    for (const void *x : p) any |= (uintptr_t)x;
    return (any & 15) == 0;
}

}  // namespace norm
}  // namespace kda
