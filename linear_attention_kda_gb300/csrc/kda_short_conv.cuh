// Shared by the kernels of the short convolution.
#pragma once
#include "kda_internal.h"
#include "kda_layer.cuh"
#include "kda_linear.cuh"
#include "kda_row_map.h"
#include "tc_util.cuh"

namespace kda {
namespace conv {

using layer::add;
using layer::fma;
using layer::mul;
using layer::splat;
using layer::vec;

struct spec {
    int64_t T, N;
    int D, K, act, norm;
    float eps;
    const float *w, *b;
    const int32_t *cu;
    int64_t stride;  // of x
};
template <typename A> inline spec spec_of(const A *a, int64_t T, const int32_t *cu) {
    return {T, a->N, a->D, a->K, a->activation, a->norm_dim, a->norm_eps, a->weight, a->bias, cu, a->x_stride};
}

// V channels from p on, of which `have` exist: as 16-byte (8-byte) vectors where every row allows them (WIDE), else one by one
template <typename T, int V, bool WIDE> __device__ __forceinline__ vec<T, V> load(const T *p, int have) {
    vec<T, V> v;
    if constexpr (WIDE) {
        if (have > 0) v = layer::load<T, V>(p);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < have) v.x[i] = p[i];
    }
    return v;
}
template <typename T, int V, bool WIDE> __device__ __forceinline__ void store(T *p, const vec<T, V> &v, int have) {
    if constexpr (WIDE) {
        if (have > 0) layer::store_once(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < have) p[i] = v.x[i];
    }
}
template <typename T, int V> __device__ __forceinline__ vec<T, V> zeros() {
    vec<T, V> v;
#pragma unroll
    for (int i = 0; i < V; ++i) st(&v.x[i], 0.f);
    return v;
}

// Taps and bias of V channels
template <int V, int K> struct taps {
    float2 w[K][V / 2], b[V / 2];
    __device__ __forceinline__ taps(const spec &S, int c, int have) {
        float t[K][V], u[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            u[v] = S.b && v < have ? S.b[c + v] : 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) t[k][v] = v < have ? S.w[(int64_t)(c + v) * K + k] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            b[i] = make_float2(u[2 * i], u[2 * i + 1]);
#pragma unroll
            for (int k = 0; k < K; ++k) w[k][i] = make_float2(t[k][2 * i], t[k][2 * i + 1]);
        }
    }
};

// Sums over the lanes that hold a head (norm / V of them, V channels each)
template <int V> __device__ __forceinline__ float head_sum(float v, int norm) {
#pragma unroll
    for (int off = 1; off < 32; off *= 2)
        if (off * V < norm) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Both sums at once: each half of the lanes takes one of them after the first step (six shuffles for ten)
template <int V> __device__ __forceinline__ void head_sums(float &a, float &b, int norm) {
    const int half = norm / V / 2;
    const bool upper = (threadIdx.x & half) != 0;
    float v = upper ? b : a;
    v += __shfl_xor_sync(0xffffffffu, upper ? a : b, half);
#pragma unroll
    for (int off = 1; off < 16; off *= 2)
        if (off < half) v += __shfl_xor_sync(0xffffffffu, v, off);
    const float w = __shfl_xor_sync(0xffffffffu, v, half);
    a = upper ? w : v;
    b = upper ? v : w;
}

// Four sums: a quarter of the lanes takes each of them after two steps (heads over eight lanes or more; ten shuffles for 24)
template <int V> __device__ __forceinline__ void head_sums(float (&a)[4], int norm) {
    const int lane = threadIdx.x & 31, half = norm / V / 2, quarter = half / 2;
    const bool upper = (lane & half) != 0, second = (lane & quarter) != 0;
    float v[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) v[j] = (upper ? a[2 + j] : a[j]) + __shfl_xor_sync(0xffffffffu, upper ? a[j] : a[2 + j], half);
    float s = (second ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, second ? v[0] : v[1], quarter);
#pragma unroll
    for (int off = 1; off < 8; off *= 2)
        if (off < quarter) s += __shfl_xor_sync(0xffffffffu, s, off);
    const int base = lane & ~(2 * half - 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = __shfl_sync(0xffffffffu, s, base + j * quarter);
}
template <int V> __device__ __forceinline__ void head_sums(float (&a)[2], int norm) { head_sums<V>(a[0], a[1], norm); }

// Where rows of a sequence come from: its history and then its tokens
template <typename T, int V, bool WIDE> struct rows {
    const T *x, *hist;  // the sequence's first token and history (NULL: zeros), at this lane's channels
    int64_t stride;
    int D, K, have;
    __device__ __forceinline__ vec<T, V> at(int i) const {  // token i, from -(K - 1) on
        if (i >= 0) return load<T, V, WIDE>(x + i * stride, have);
        return hist ? load<T, V, WIDE>(hist + (int64_t)(i + K - 1) * D, have) : zeros<T, V>();
    }
};

// The sequence of a slot and the run of L of its tokens, [first, last).  False: none; an empty sequence has a run of no tokens.
struct run {
    int64_t n, a;          // sequence, its first token
    int len, first, last;  // its tokens, the run's
};
__device__ __forceinline__ bool find_run(const spec &S, int64_t slot, int L, run *r) {
    int64_t i;
    lin::span s;
    if (!lin::find_slot(S.cu, S.T, S.N, L, slot, &r->n, &i, &s)) return false;
    r->a = s.a;
    r->len = (int)(s.b - s.a);
    if (i > 0 && i * L >= r->len) return false;
    r->first = (int)(i * L);
    r->last = r->first + L < r->len ? r->first + L : r->len;
    return true;
}

// A warp's next rows, 2 KB of them (or half as many) at a time and up to NS times as many, on their way by TMA: the registers that as many loads
// would take are those of four more warps.
template <typename T, int V> constexpr int some_rows = 2048 / (32 * V * (int)sizeof(T));
constexpr int NS = 3;
template <typename T, int V, int NI, int ROWS> struct alignas(128) ring {
    T x[NS][NI][ROWS][32 * V];
    uint64_t full[NS];
};
struct row_maps {
    CUtensorMap x, dy;
};

// Tokens of a run: what a block takes is about L of them and 16 more (those that two runs share, and its beginning), and the
// blocks come in rounds of as many as the GPU holds (`at_once`).  `runs` to a block, `blocks` of channels.  (Powers of two alone: 6 sequences
// of 512 to 8192 tokens forwards 100 us for 98, gradients of 8 of 300 to 5000 216 for 193.)
inline int run_length(int64_t T, int64_t N, int blocks, int runs, int at_once) {
    int best = 16;
    int64_t least = INT64_MAX;
    for (int L : {16, 32, 48, 64, 96, 128, 192, 256}) {
        const int64_t grid = (lin::chunk_slots(T, N, L) + runs - 1) / runs * blocks, cost = (grid + at_once - 1) / at_once * (L + 16);
        if (cost < least) least = cost, best = L;
    }
    return best;
}

__device__ __forceinline__ void check_all(const spec &S, int *err) {
    if (blockIdx.x > 0 || blockIdx.y > 0) return;
    for (int64_t n = threadIdx.x; n < S.N; n += blockDim.x) {
        lin::span s;
        if (!lin::seq_span(S.cu, S.T, S.N, n, &s)) set_error(err, KDA_ERR_BAD_SEQLENS);
    }
}

}  // namespace conv
}  // namespace kda
