// kda_rope: pairs of the first `rot` channels of every head of q and k turned by positions[t] * freqs[i].
//
// Angles.  An angle matters modulo one turn, and positions are integers, so a frequency is kept as turns per
// position in 64-bit fixed point, F = round(freq / 2 pi * 2^64) mod 2^64, and the angle of position p is p * F mod
// 2^64: one integer product, wrong by at most |p| / 2 units of 2^-64 turns (2^-34 turns at the largest int32), where
// an fp32 product p * freq would be wrong by half a radian at a position of 2^23.  The high 32 bits, a signed fraction of
// a turn, are rounded to an fp32 (2^-26 turns at most, next to half a turn: 1e-7 radians, about what an fp32 sine is good
// to) and go to sincospif.
//
// A CTA takes TB tokens: it first writes their sines and cosines (shared by all heads) to shared memory, then
// streams the heads' rows in 16-byte pieces, four in flight per thread.  Bound by HBM: q and k read once and written
// once; channels behind `rot` are copied, or left alone when the output is the input.  131071 tokens, 32 + 8 heads of
// 128 bf16 channels, 64 of them turned, into other tensors: 395 us, 6.8 TB/s (one token and piece at a time: 601 us; with
// conversions and index divisions element by element: 1065 us, bound by instructions); in place 225 us.
#include <math.h>

#include <type_traits>

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

// x / d for x * d < 2^32, by a product with ceil(2^32 / d)
struct divisor {
    uint32_t d, m;
};
static divisor make_divisor(uint32_t d) { return {d, d > 1 ? (uint32_t)((((uint64_t)1 << 32) + d - 1) / d) : 0}; }
__device__ __forceinline__ uint32_t quotient(uint32_t x, const divisor &v) { return v.d > 1 ? __umulhi(x, v.m) : x; }

struct job {
    tensor t;
    divisor heads, per;   // per: pieces of a head's row, those that turn, then those that are copied
};

// V values as fp32 and back, packed conversions where they are 16 bytes or pairs
template <typename T, int V>
__device__ __forceinline__ void unpack(const vec<T, V> &v, float *f) {
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
template <typename T, int V>
__device__ __forceinline__ void pack(vec<T, V> &v, const float *f) {
    if constexpr (sizeof(T) == 2 && V > 1) {
        __nv_bfloat162 *w = reinterpret_cast<__nv_bfloat162 *>(&v);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) w[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) st(&v.x[i], f[i]);
    }
}

constexpr int FLIGHT = 4;  // pieces a thread has in flight

// A piece: V elements of each half of a pair group (half layout), or V elements holding V / 2 pairs (interleaved; one
// pair by its elements where V is 1), or V elements behind `rot`.
template <typename T, int V, bool HALVES>
__device__ __forceinline__ void rows(const job &J, int64_t tok0, int ntok, int d, int half, int turn, const float2 *cs) {
    using VT = vec<T, V>;
    constexpr bool TWO = HALVES || V == 1;  // a turning piece is two vectors
    const uint32_t per = J.per.d, total = (uint32_t)ntok * J.heads.d * per;
    const T *base = (const T *)J.t.in + tok0 * J.t.si;
    T *dest = (T *)J.t.out + tok0 * J.t.so;
    for (uint32_t e0 = threadIdx.x; e0 < total; e0 += 256 * FLIGHT) {
        VT a[FLIGHT], b[FLIGHT];
        uint32_t tk[FLIGHT], h[FLIGHT], i[FLIGHT];
#pragma unroll
        for (int j = 0; j < FLIGHT; ++j) {
            const uint32_t e = e0 + 256 * j, r = quotient(e, J.per);
            i[j] = e - r * per;
            tk[j] = quotient(r, J.heads);
            h[j] = r - tk[j] * J.heads.d;
            if (e >= total) continue;
            const bool turned = (int)i[j] < turn;
            const uint32_t at = h[j] * d + (turned ? (TWO && !HALVES ? 2 : V) * i[j] : 2 * half + (i[j] - turn) * V);
            const T *p = base + tk[j] * J.t.si + at;
            a[j] = *reinterpret_cast<const VT *>(p);
            if (TWO && turned) b[j] = *reinterpret_cast<const VT *>(p + (HALVES ? half : 1));
        }
#pragma unroll
        for (int j = 0; j < FLIGHT; ++j) {
            if (e0 + 256 * j >= total) continue;
            const bool turned = (int)i[j] < turn;
            const uint32_t at = h[j] * d + (turned ? (TWO && !HALVES ? 2 : V) * i[j] : 2 * half + (i[j] - turn) * V);
            T *p = dest + tk[j] * J.t.so + at;
            if (turned) {
                float x[V], y[V];
                unpack<T, V>(a[j], x);
                if constexpr (TWO) {
                    const float2 *w = cs + tk[j] * half + V * i[j];
                    unpack<T, V>(b[j], y);
#pragma unroll
                    for (int n = 0; n < V; ++n) {
                        const float2 c = w[n];
                        const float u = x[n] * c.x - y[n] * c.y;
                        y[n] = y[n] * c.x + x[n] * c.y;
                        x[n] = u;
                    }
                    pack<T, V>(b[j], y);
                    *reinterpret_cast<VT *>(p + (HALVES ? half : 1)) = b[j];
                } else {
                    const float2 *w = cs + tk[j] * half + V / 2 * i[j];
#pragma unroll
                    for (int n = 0; n + 1 < V; n += 2) {
                        const float2 c = w[n / 2];
                        const float u = x[n] * c.x - x[n + 1] * c.y;
                        x[n + 1] = x[n + 1] * c.x + x[n] * c.y;
                        x[n] = u;
                    }
                }
                pack<T, V>(a[j], x);
            }
            *reinterpret_cast<VT *>(p) = a[j];
        }
    }
}

template <typename T, int V, bool HALVES>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ turns F, const __grid_constant__ job q,
                                                   const __grid_constant__ job k, int64_t tokens, int TB,
                                                   const int32_t *__restrict__ pos, int d, int half, int turn, int inverse,
                                                   float scale) {
    extern __shared__ __align__(16) float2 cs[];  // [TB][rot / 2] cosine and sine, times scale
    const int64_t tok0 = (int64_t)blockIdx.x * TB;
    const int ntok = (int)(tokens - tok0 < TB ? tokens - tok0 : TB);
    for (int e = threadIdx.x; e < ntok * half; e += 256) {
        const int tk = e / half, i = e - tk * half;
        const uint64_t turn64 = (uint64_t)(int64_t)pos[tok0 + tk] * F.f[i];
        float s, c;
        sincospif((float)(int32_t)(turn64 >> 32) * 4.656612873077393e-10f, &s, &c);  // half turns: 2^-31 each
        cs[e] = make_float2(scale * c, scale * (inverse ? -s : s));
    }
    __syncthreads();
    if (q.t.H) rows<T, V, HALVES>(q, tok0, ntok, d, half, turn, cs);
    if (k.t.H) rows<T, V, HALVES>(k, tok0, ntok, d, half, turn, cs);
}

template <typename T, int V, bool HALVES>
static void launch(const kda_rope_args *a, const turns &F, cudaStream_t stream) {
    const int half = a->rot / 2, turn = HALVES ? half / V : (V > 1 ? a->rot / V : half);
    auto job_of = [&](const void *in, void *out, int64_t si, int64_t so, int H) {
        const bool copied = !(in == out && si == so);
        return job{{in, out, si, so, H}, make_divisor((uint32_t)H),
                   make_divisor((uint32_t)(turn + (copied ? (a->d - a->rot) / V : 0)))};
    };
    // Enough tokens to a CTA for a few rounds of its pieces, as long as every SM still has three CTAs.  bf16, 32 + 8
    // heads of 128, 64 channels turned, into other tensors, by 1, 2, 4, 8 and 16 tokens: 131071 tokens 573, 432, 403, 394
    // and 405 us, 4096 tokens 16.8, 14.0, 13.3, 14.4 and 18.1, 256 tokens 3.1, 3.3, 4.5, 7.0 and 12.1.  (At most 2048 rows, or one token:
    // quotient()'s range.)
    int64_t TB = 2048 / (a->Hq + a->Hk);
    if (TB > a->T / (3 * 152)) TB = a->T / (3 * 152);
    if (TB > 8) TB = 8;
    if (TB < 1) TB = 1;
    rope_kernel<T, V, HALVES><<<(unsigned)((a->T + TB - 1) / TB), 256, (size_t)TB * half * sizeof(float2), stream>>>(
        F, job_of(a->q, a->q_out, a->q_stride, a->q_out_stride, a->Hq),
        job_of(a->k, a->k_out, a->k_stride, a->k_out_stride, a->Hk), a->T, (int)TB, a->positions, a->d, half, turn,
        a->inverse, a->scale);
}

template <typename T>
static void launch_t(const kda_rope_args *a, const turns &F, cudaStream_t stream) {
    // The widest vector (up to 16 bytes) that divides what a lane moves and that every row's address is a multiple
    // of; single elements (pairs of them, interleaved) otherwise.  The same 131071 tokens by 8, 4 and 1 elements: 395, 498
    // and 1111 us.
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
    auto go = [&](auto halves) {
        constexpr bool H = decltype(halves)::value;
        if (fits(V16)) launch<T, V16, H>(a, F, stream);
        else if (fits(4)) launch<T, 4, H>(a, F, stream);
        else launch<T, 1, H>(a, F, stream);
    };
    if (a->layout == KDA_ROPE_HALF) go(std::true_type{});
    else go(std::false_type{});
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
