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

// N (one or two) sums over the NT threads of a row.  `at` alternates between two places of shared memory (16-byte aligned), so that one barrier
// separates a sum's parts from the sum after the next.  Two sums go over the lanes as one, each half of a warp with its own.
template <int NT, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float *shared, int &at) {
    static_assert(N <= 2 && (NT == 32 || NT % 128 == 0), "shapes");
    constexpr int H = 32 / N;  // lanes to a sum
    const int lane = threadIdx.x & 31;
    float x = v[0];
    if constexpr (N == 2) x = (lane & 16 ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, lane & 16 ? v[0] : v[1], 16);
#pragma unroll
    for (int off = H / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    if constexpr (NT == 32) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = N == 1 ? x : __shfl_sync(0xffffffffu, x, i * H);
    } else {
        constexpr int W = NT / 32;
        float *s = shared + at * (2 * W);
        at ^= 1;
        if (lane % H == 0) s[lane / H * W + (threadIdx.x >> 5)] = x;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = 0.f;
#pragma unroll
            for (int w = 0; w < W; w += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(s + i * W + w);
                v[i] += (f.x + f.y) + (f.z + f.w);
            }
        }
    }
}

__device__ __forceinline__ float total(float v) { return v; }
__device__ __forceinline__ float total(float2 v) { return v.x + v.y; }

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
