// Shared by the linear-attention kernels (a decay per head): where the chunks of a packed batch lie, and the
// cumulative log-decays of one chunk.
#pragma once
#include <atomic>

#include "kda_common.cuh"

namespace kda {
namespace lin {

// Allows a kernel its dynamic shared memory, once for each device.  `done`: a bit per device, one such word per kernel.
template <typename K>
inline cudaError_t allow_smem(K *kernel, int bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// Sequence n's tokens, [a, b).  False (and the device error set by one caller) where cu_seqlens is not
// 0 = c_0 <= ... <= c_N = T around it: nothing out of range is ever formed from it.
struct span {
    int64_t a, b;
};
__device__ __forceinline__ int64_t seq_start(const int32_t *cu, int64_t T, int64_t N, int64_t n) {
    return cu ? (int64_t)cu[n] : n * (T / N);
}
__device__ __forceinline__ bool seq_span(const int32_t *cu, int64_t T, int64_t N, int64_t n, span *s) {
    s->a = seq_start(cu, T, N, n);
    s->b = seq_start(cu, T, N, n + 1);
    return s->a >= 0 && s->a <= s->b && s->b <= T && (n > 0 || s->a == 0) && (n < N - 1 || s->b == T);
}

// Chunks need no plan kernel: sequence n's first chunk has slot a / C + n, and since
// ceil((b - a) / C) <= b / C - a / C + 1, its chunks end before the next sequence's begin.  A batch has
// T / C + N slots, a few of which stay empty.
__host__ __device__ __forceinline__ int64_t chunk_slots(int64_t T, int64_t N, int C) { return T / C + N; }

// The sequence and index of the run of W tokens in a slot (false: a slot that lies in no sequence with a good
// range; the caller compares the index with the sequence's length).  Every lane of a warp calls it: the 32 lanes
// search the sequences 32 ways at once.
__device__ __forceinline__ bool find_slot(const int32_t *cu, int64_t T, int64_t N, int64_t W, int64_t slot, int64_t *n,
                                          int64_t *index, span *s) {
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, hi = N;
    while (hi - lo > 1) {
        const int64_t step = (hi - lo + 31) / 32, i = lo + lane * step;
        const bool at_or_before = i < hi && seq_start(cu, T, N, i) / W + i <= slot;
        const unsigned m = __ballot_sync(0xffffffffu, at_or_before);
        lo += (m ? 31 - __clz(m) : 0) * step;
        hi = hi < lo + step ? hi : lo + step;
    }
    *n = lo;
    if (!seq_span(cu, T, N, lo, s)) return false;
    *index = slot - (s->a / W + lo);
    return *index >= 0;
}

struct chunk {
    int64_t tok0;  // first token
    int len;       // tokens, 1 .. C
    bool first, last;  // of its sequence
};
template <int C>
__device__ __forceinline__ bool find_chunk(const int32_t *cu, int64_t T, int64_t N, int64_t slot, chunk *c) {
    int64_t n, i;
    span s;
    if (!find_slot(cu, T, N, C, slot, &n, &i, &s) || s.a + i * C >= s.b) return false;
    c->tok0 = s.a + i * C;
    c->len = (int)(s.b - c->tok0 < C ? s.b - c->tok0 : C);
    c->first = i == 0;
    c->last = s.b - c->tok0 <= C;
    return true;
}

// Sums of two floats each (48 bits): the fp64 pipe of this GPU would take three times as long for a chunk's sums.
struct ff {
    float h, l;
};
__device__ __forceinline__ ff ff_add(const ff &a, const ff &b) {
    const float s = a.h + b.h, t = s - a.h, e = ((a.h - (s - t)) + (b.h - t)) + (a.l + b.l), h = s + e;
    return {h, e - (h - s)};
}
__device__ __forceinline__ float ff_diff(const ff &a, const ff &b) { return (a.h - b.h) + (a.l - b.l); }
__device__ __forceinline__ ff ff_shfl(const ff &a, int lane) {
    return {__shfl_sync(0xffffffffu, a.h, lane), __shfl_sync(0xffffffffu, a.l, lane)};
}

// A log-decay below -104 counts as -104 (exp of it is 0 in fp32); a NaN stays one.
__device__ __forceinline__ float clamp_decay(float g) { return g < -104.f ? -104.f : g; }

// To be called on values that decay by the factor f: where f is 0 nothing of them is left, infinities and NaN included.
template <int N> __device__ __forceinline__ void erase(float (&x)[N], float f) {
    if (f == 0.f) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = 0.f;
    }
}

// Cumulative log-decays G of one chunk, by one warp, kept as fp32 pairs hi + lo: the difference of two of them, (hi_r -
// hi_j) + (lo_r - lo_j), is then good to an fp32 rounding of itself even where many erasing decays have made both
// large.  x: this lane's log-decays, tokens lane * C / 32 on.
template <int C>
__device__ __forceinline__ void load_decays(const float *g, int g_stride, int len, float *x) {
    constexpr int P = C / 32;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int r = lane * P + i;
        x[i] = g && r < len ? g[(int64_t)r * g_stride] : 0.f;
    }
}
template <int C>
__device__ __forceinline__ void chunk_decays(const float *x, float *hi, float *lo) {
    static_assert(C % 32 == 0, "lanes");
    constexpr int P = C / 32;
    const int lane = threadIdx.x & 31;
    ff G[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const ff y{clamp_decay(x[i]), 0.f};
        G[i] = i ? ff_add(G[i - 1], y) : y;
    }
    ff pre = G[P - 1];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const ff y = ff_shfl(pre, lane - off);
        if (lane >= off) pre = ff_add(y, pre);
    }
    ff before = ff_shfl(pre, lane - 1);
    if (lane == 0) before = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const ff y = ff_add(before, G[i]);
        hi[lane * P + i] = y.h;
        lo[lane * P + i] = y.l;
    }
}

}  // namespace lin
}  // namespace kda
