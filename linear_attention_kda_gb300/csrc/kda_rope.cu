// kda_rope: pairs of the first `rot` channels of every head of q and k turned by positions[t] * freqs[i].
//
// Angles.  An angle matters modulo one turn, and positions are integers, so a frequency is kept as turns per
// position in 64-bit fixed point, F = round(freq / 2 pi * 2^64) mod 2^64, and the angle of position p is p * F mod
// 2^64: one integer product, wrong by at most |p| / 2 units of 2^-64 turns (2^-34 turns at the largest int32), where
// an fp32 product p * freq would be wrong by half a radian at a position of 2^23.  The high 32 bits, as a signed
// fraction of a turn, go to sincospif.
//
// A CTA takes TB tokens: it first writes their sines and cosines (shared by all heads) to shared memory, then
// streams the heads' rows through 16-byte vectors.  Bound by HBM: q and k read once and written once; channels behind
// `rot` are copied, or left alone when the output is the input.
#include <math.h>

#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace rope {

struct turns {
    uint64_t f[128];
};
struct tensor {
    const void *in;
    void *out;
    int64_t si, so;  // elements between tokens
    int H;
};

template <typename T, int V> struct alignas(sizeof(T) * V) vec {
    T x[V];
};

// One item: V elements of each half of a pair group (half layout), or V elements holding V / 2 pairs (interleaved;
// one pair by its elements where V is 1), or V elements behind `rot`.
template <typename T, int V>
__device__ __forceinline__ void rows(const tensor &t, int64_t tok0, int ntok, int d, int rot, int layout,
                                     const float2 *cs) {
    const int half = rot >> 1;
    const int turn = layout == KDA_ROPE_HALF ? half / V : (V > 1 ? rot / V : half);  // items that turn
    const int rest = t.in == t.out && t.si == t.so ? 0 : (d - rot) / V;     // items that are copied
    const int per = turn + rest;
    const int total = ntok * t.H * per;
    using VT = vec<T, V>;
    for (int e = threadIdx.x; e < total; e += blockDim.x) {
        const int r = e / per, i = e - r * per;
        const int tk = r / t.H, h = r - tk * t.H;
        const T *in = (const T *)t.in + (tok0 + tk) * t.si + (int64_t)h * d;
        T *out = (T *)t.out + (tok0 + tk) * t.so + (int64_t)h * d;
        if (i >= turn) {
            const int c = rot + (i - turn) * V;
            *reinterpret_cast<VT *>(out + c) = *reinterpret_cast<const VT *>(in + c);
        } else if (layout == KDA_ROPE_HALF) {
            const int c = i * V;
            VT a = *reinterpret_cast<const VT *>(in + c), b = *reinterpret_cast<const VT *>(in + half + c);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float2 w = cs[tk * half + c + j];
                const float x = ld(&a.x[j]), y = ld(&b.x[j]);
                st(&a.x[j], x * w.x - y * w.y);
                st(&b.x[j], y * w.x + x * w.y);
            }
            *reinterpret_cast<VT *>(out + c) = a;
            *reinterpret_cast<VT *>(out + half + c) = b;
        } else if (V == 1) {
            const float2 w = cs[tk * half + i];
            const float x = ld(in + 2 * i), y = ld(in + 2 * i + 1);
            st(out + 2 * i, x * w.x - y * w.y);
            st(out + 2 * i + 1, y * w.x + x * w.y);
        } else {
            const int c = i * V;
            VT a = *reinterpret_cast<const VT *>(in + c);
#pragma unroll
            for (int j = 0; j + 1 < V; j += 2) {
                const float2 w = cs[tk * half + ((c + j) >> 1)];
                const float x = ld(&a.x[j]), y = ld(&a.x[j + 1]);
                st(&a.x[j], x * w.x - y * w.y);
                st(&a.x[j + 1], y * w.x + x * w.y);
            }
            *reinterpret_cast<VT *>(out + c) = a;
        }
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ turns F, tensor q, tensor k, int64_t tokens,
                                                   int TB, const int32_t *__restrict__ pos, int d, int rot, int layout,
                                                   int inverse, float scale) {
    extern __shared__ float2 cs[];  // [TB][rot / 2] cosine and sine, times scale
    const int half = rot >> 1;
    const int64_t tok0 = (int64_t)blockIdx.x * TB;
    const int ntok = (int)(tokens - tok0 < TB ? tokens - tok0 : TB);
    for (int e = threadIdx.x; e < ntok * half; e += 256) {
        const int tk = e / half, i = e - tk * half;
        const uint64_t turn = (uint64_t)(int64_t)pos[tok0 + tk] * F.f[i];
        float s, c;
        sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);  // half turns: 2^-31 each
        cs[e] = make_float2(scale * c, scale * (inverse ? -s : s));
    }
    __syncthreads();
    if (q.H) rows<T, V>(q, tok0, ntok, d, rot, layout, cs);
    if (k.H) rows<T, V>(k, tok0, ntok, d, rot, layout, cs);
}

template <typename T, int V>
static void launch(const kda_rope_args *a, const turns &F, cudaStream_t stream) {
    const tensor q{a->q, a->q_out, a->q_stride, a->q_out_stride, a->Hq};
    const tensor k{a->k, a->k_out, a->k_stride, a->k_out_stride, a->Hk};
    const int TB = 1;
    const unsigned grid = (unsigned)((a->T + TB - 1) / TB);
    rope_kernel<T, V><<<grid, 256, (size_t)TB * (a->rot / 2) * sizeof(float2), stream>>>(
        F, q, k, a->T, TB, a->positions, a->d, a->rot, a->layout, a->inverse, a->scale);
}

template <typename T>
static void launch_t(const kda_rope_args *a, const turns &F, cudaStream_t stream) {
    // The widest vector (up to 16 bytes) that divides what a lane moves and that every row's address is a multiple
    // of; single elements (pairs of them, interleaved) otherwise.
    auto fits = [&](int w) {
        const int64_t part = a->layout == KDA_ROPE_HALF ? a->rot / 2 : a->rot;
        if (part % w || (a->d - a->rot) % w || a->d % w) return false;
        const uintptr_t bytes = (uintptr_t)w * sizeof(T);
        const bool q = !a->Hq || (!(((uintptr_t)a->q | (uintptr_t)a->q_out) % bytes) && a->q_stride % w == 0 &&
                                  a->q_out_stride % w == 0);
        const bool k = !a->Hk || (!(((uintptr_t)a->k | (uintptr_t)a->k_out) % bytes) && a->k_stride % w == 0 &&
                                  a->k_out_stride % w == 0);
        return q && k;
    };
    constexpr int V16 = 16 / (int)sizeof(T);
    if (fits(V16)) launch<T, V16>(a, F, stream);
    else if (fits(4)) launch<T, 4>(a, F, stream);
    else launch<T, 1>(a, F, stream);
}

}  // namespace rope
}  // namespace kda

kda_status_t kda_launch_rope(const kda_rope_args *a, cudaStream_t stream) {
    kda::rope::turns F{};
    for (int i = 0; i < a->rot / 2; ++i) {
        // Turns per position, freq / 2 pi, as a sum of two doubles: one alone is off by 2^-53 of itself, which the
        // largest positions would make 2^-22 turns.  Whole turns change nothing for whole positions.
        const double f = fabs(a->freqs[i]), t = f * 0.15915494309189535;
        const double rest = fma(f, 0.15915494309189535, -t) + f * -9.839338337591243e-18;
        const double part = t - floor(t);
        // 2^64 part in two halves of 32 bits, both exact (part < 1 has 53 bits)
        const double hi = floor(part * 4294967296.0), lo = (part * 4294967296.0 - hi) * 4294967296.0;
        F.f[i] = ((uint64_t)hi << 32) + (uint64_t)lo + (uint64_t)(int64_t)llrint(rest * 18446744073709551616.0);
        if (a->freqs[i] < 0) F.f[i] = 0 - F.f[i];
    }
    if (a->dtype == KDA_BF16) kda::rope::launch_t<kda::bf16>(a, F, stream);
    else kda::rope::launch_t<float>(a, F, stream);
    return kda_cuda_status(cudaGetLastError());
}
