// Arithmetic of the gated recurrence over channels, h <- a h + c(a) Sigmoid(i) x with a = exp(g), shared by its
// kernels: the gates, the step and its derivative.
//
// The decay a is kept as one fp32 `d`: d < 0 stands for a = 1 + d (a in [3/4, 1)), d >= 0 for a = d.  Near 1 an fp32 a
// is good to 2^-25, which a state that remembers 1 / (1 - a) tokens takes in as many times; a - 1 is good to 2^-24 of
// itself, which it takes in once (4096 tokens at g = -1e-4: final states off by 9e-6 with a, 1e-7 with a - 1).  A run of
// tokens is described by the sum of its log-decays and the state that it leaves from zero.
#pragma once
#include "kda_common.cuh"

namespace kda {
namespace scan {

struct spec {  // how a call forms a and c(a)
    int gate, input;
    float g_min;
};
struct channel {  // a channel's parameters
    float b, rate;  // dt_bias and exp(A_log)
};

// Sigmoid(y) and 1 - Sigmoid(y), each to a few units of 2^-24 of itself
struct sig {
    float s, n;
};
__device__ __forceinline__ sig sigmoid(float y) {
    const float e = __expf(-fabsf(y)), r = __fdividef(1.f, 1.f + e), q = e * r;
    return {y >= 0.f ? r : q, y >= 0.f ? q : r};
}
// Softplus(y) = max(y, 0) + ln(1 + e), e = exp(-|y|): ln(1 + e) / e by the polynomial of degree 8 that meets it in the
// Chebyshev points of [0, 1] (2e-7 with its roundings)
__device__ __forceinline__ float softplus(float y) {
    const float e = __expf(-fabsf(y));
    float p = 0.005126102361828089f;
    p = fmaf(p, e, -0.029074065387248993f);
    p = fmaf(p, e, 0.0775160863995552f);
    p = fmaf(p, e, -0.13602247834205627f);
    p = fmaf(p, e, 0.19076880812644958f);
    p = fmaf(p, e, -0.2483539879322052f);
    p = fmaf(p, e, 0.3331812024116516f);
    p = fmaf(p, e, -0.4999944567680359f);
    p = fmaf(p, e, 0.9999999403953552f);
    return fmaf(p, e, fmaxf(y, 0.f));
}
// exp(g) - 1 to a few units of 2^-24 of itself: its series to g^7 / 7! where |g| < 1/4 (the rest is below 2e-9 of it), else by exp(g),
// which is at least 2/9 away from 1 there
__device__ __forceinline__ float small_expm1(float g) {
    float p = 1.f / 5040.f;
    p = fmaf(p, g, 1.f / 720.f);
    p = fmaf(p, g, 1.f / 120.f);
    p = fmaf(p, g, 1.f / 24.f);
    p = fmaf(p, g, 1.f / 6.f);
    p = fmaf(p, g, 0.5f);
    return fmaf(p * g, g, g);
}

// d of a log-decay, and exp(g) - 1
struct decay {
    float d, m;
};
__device__ __forceinline__ decay decay_of(float g) {
    const float e = __expf(g), m = small_expm1(g);
    const bool near = fabsf(g) < 0.25f;
    // (g = 0 and the small g > 0 that KDA_SCAN_LOG may bring: a = 1 + m)
    return {near ? (m < 0.f ? m : 1.f + m) : e, near ? m : e - 1.f};
}
__device__ __forceinline__ float factor(float d) { return d < 0.f ? 1.f + d : d; }
// a h, where nothing is left of h if a is 0, an infinity or a NaN in h included
__device__ __forceinline__ float decayed(float d, float h) {
    const float k = d == 0.f ? 0.f : h;
    return fmaf(d, k, d < 0.f ? k : 0.f);
}

// g, and for the gradients dg/dz and dg/dA_log
__device__ __forceinline__ float log_decay(const spec &S, const channel &C, float z) {
    if (S.gate == KDA_SCAN_LOG) return z;
    const float y = z + C.b;
    if (S.gate == KDA_SCAN_SOFTPLUS) return -C.rate * softplus(y);
    if (S.gate == KDA_SCAN_SIGMOID) return -C.rate * sigmoid(y).s;
    return S.g_min * sigmoid(C.rate * y).s;
}
__device__ __forceinline__ float log_decay(const spec &S, const channel &C, float z, float *dz, float *dA) {
    if (S.gate == KDA_SCAN_LOG) {
        *dz = 1.f;
        *dA = 0.f;
        return z;
    }
    const float y = z + C.b;
    if (S.gate == KDA_SCAN_LOWER_BOUND) {
        const sig w = sigmoid(C.rate * y);
        const float g = S.g_min * w.s;
        *dz = g * w.n * C.rate;
        *dA = *dz * y;
        return g;
    }
    const sig w = sigmoid(y);
    const float g = -C.rate * (S.gate == KDA_SCAN_SOFTPLUS ? softplus(y) : w.s);
    *dz = S.gate == KDA_SCAN_SOFTPLUS ? -C.rate * w.s : g * w.n;
    *dA = g;
    return g;
}

// c(a) from m = a - 1: 1 - a^2 = -m (2 + m) has no cancellation.  Where it is not above 0, c = sqrt(1 - a^2) and its derivative count as 0.
__device__ __forceinline__ float input_factor(const spec &S, float m) {
    if (S.input == KDA_SCAN_INPUT_PLAIN) return 1.f;
    if (S.input == KDA_SCAN_INPUT_COMPLEMENT) return -m;
    const float q = -m * (2.f + m);
    return q > 0.f ? q * rsqrtf(q) : (q <= 0.f ? 0.f : q);
}
// dc/dg: -a of 1 - a, -a^2 / c of sqrt(1 - a^2)
__device__ __forceinline__ float input_slope(const spec &S, float a, float c) {
    if (S.input == KDA_SCAN_INPUT_PLAIN) return 0.f;
    if (S.input == KDA_SCAN_INPUT_COMPLEMENT) return -a;
    return c > 0.f ? -a * __fdividef(a, c) : (c <= 0.f ? 0.f : c);
}

// What enters at a token, c(a) Sigmoid(i) x
__device__ __forceinline__ float entering(const spec &S, float m, float x, bool gated, float i) {
    const float u = gated ? x * sigmoid(i).s : x;
    return S.input == KDA_SCAN_INPUT_PLAIN ? u : u * input_factor(S, m);
}

__device__ __forceinline__ channel load_channel(const float *A_log, const float *dt_bias, int c) {
    return {dt_bias ? dt_bias[c] : 0.f, A_log ? expf(A_log[c]) : 1.f};
}

}  // namespace scan
}  // namespace kda
