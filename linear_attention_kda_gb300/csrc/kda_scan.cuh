// Arithmetic of the gated recurrence over channels, h <- a h + c(a) Sigmoid(i) x with a = exp(g), shared by its
// kernels: the gates, the step and their derivatives.  F is one fp32 or a pair of them.
//
// The decay a is kept as one fp32 `d`: d < 0 stands for a = 1 + d (a in [0.778, 1)), d >= 0 for a = d.  Near 1 an fp32 a
// is good to 2^-25, which a state that remembers 1 / (1 - a) tokens takes in as many times; a - 1 is good to 2^-23 of
// itself, which it takes in once.  A run of tokens is described by the sum of its log-decays and the state that it
// leaves from zero.
//
// Bound by instructions before it is bound by HBM (8 bytes an element in bf16 leave about 42 of them an element at the copy
// rate): everything that can be is done on two channels at a time, exponentials and quotients by the special function
// unit (2^-22, so far below what the recurrence itself rounds).
#pragma once
#include "kda_layer.cuh"

namespace kda {
namespace scan {

using layer::add;
using layer::each;
using layer::ex2;
using layer::fma;
using layer::mul;
using layer::rcp;
using layer::rsq;
using layer::LOG2E;
using layer::sig;
using layer::sigmoid;
using layer::sigmoids;
using layer::splat;

struct spec {  // how a call forms a and c(a)
    int gate, input;
    float g_min;
};
template <typename F> struct channel {  // a channel's parameters: dt_bias and exp(A_log)
    F b, rate;
};

// Softplus(y) = max(y, 0) + ln(1 + e), e = exp(-|y|): ln(1 + e) / e by the polynomial of degree 8 that meets it in the
// Chebyshev points of [0, 1] (2e-7 with its roundings)
template <typename F> __device__ __forceinline__ F softplus(F y) {
    const F e = ex2(each([](float v) { return fabsf(v) * -LOG2E; }, y));
    F p = fma(splat<F>(0.005126102361828089f), e, splat<F>(-0.029074065387248993f));
    p = fma(p, e, splat<F>(0.0775160863995552f));
    p = fma(p, e, splat<F>(-0.13602247834205627f));
    p = fma(p, e, splat<F>(0.19076880812644958f));
    p = fma(p, e, splat<F>(-0.2483539879322052f));
    p = fma(p, e, splat<F>(0.3331812024116516f));
    p = fma(p, e, splat<F>(-0.4999944567680359f));
    p = fma(p, e, splat<F>(0.9999999403953552f));
    return fma(p, e, each([](float v) { return fmaxf(v, 0.f); }, y));
}

// Log-decays are moved by this much, which changes nothing but 0 and -0 to a decay below 1 (d < 0)
constexpr float NUDGE = -1e-37f;

// d of a log-decay (nudged), and m = exp(g) - 1: by its series to g^6 / 6! where -1/4 < g < 0 (the rest is below 5e-8 of it), else from
// exp(g), which is at least 2/9 away from 1 there (what g > 0 KDA_SCAN_LOG may bring is computed as given, a = exp(g))
template <typename F> struct decay {
    F d, m;
};
template <typename F> __device__ __forceinline__ decay<F> decay_of(F g) {
    const F e = ex2(mul(g, splat<F>(LOG2E)));
    F p = fma(splat<F>(1.f / 720.f), g, splat<F>(1.f / 120.f));
    p = fma(p, g, splat<F>(1.f / 24.f));
    p = fma(p, g, splat<F>(1.f / 6.f));
    p = fma(p, g, splat<F>(0.5f));
    p = fma(mul(p, g), g, g);
    // as integers, the negative floats above -1/4 lie below the bits of -1/4
    const auto near = [](float v) { return __float_as_int(v) < (int)0xBE800000; };
    return {each([&](float v, float s, float f) { return near(v) ? s : f; }, g, p, e),
            each([&](float v, float s, float f) { return near(v) ? s : f; }, g, p, add(e, splat<F>(-1.f)))};
}
template <typename F> __device__ __forceinline__ F factor(F d) {
    return each([](float v) { return v < 0.f ? 1.f + v : v; }, d);
}
// a - 1
template <typename F> __device__ __forceinline__ F below_one(F d) {
    return each([](float v) { return v < 0.f ? v : v - 1.f; }, d);
}
// a h + u for finite h.  An infinity or a NaN leaves one of the two behind, whatever follows, so that a run of steps is looked at in its end
// and, where it has to be, taken again by step_any().
template <typename F> __device__ __forceinline__ F step(F d, F h, F u) {
    return fma(d, h, fma(each([](float v) { return v < 0.f ? 1.f : 0.f; }, d), h, u));
}
// a h + u for every h: nothing is left of it where a is 0, an infinity or a NaN included, and an infinity stays one under other decays (step()
// would take it from itself)
__device__ __forceinline__ float step_any(float d, float h, float u) {
    const float finite = step(d, h, u), other = d == 0.f ? u : fma(fabsf(d), h, u);
    return d == 0.f || fabsf(h) == __int_as_float(0x7F800000) ? other : finite;
}
__device__ __forceinline__ float2 step_any(float2 d, float2 h, float2 u) {
    return make_float2(step_any(d.x, h.x, u.x), step_any(d.y, h.y, u.y));
}
__device__ __forceinline__ bool finite(float h) { return fabsf(h) <= 3.402823466e38f; }
__device__ __forceinline__ bool finite(float2 h) { return finite(h.x) && finite(h.y); }

// For the gradients: N tokens' dg/dz, in the place of z, and dg/dA_log
template <int N, typename F>
__device__ __forceinline__ void decay_slopes(const spec &S, const channel<F> &C, F (&z)[N], F (&dA)[N]) {
    const F k = mul(C.rate, splat<F>(-1.f));
    if (S.gate == KDA_SCAN_LOG) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            z[i] = splat<F>(1.f);
            dA[i] = splat<F>(0.f);
        }
    } else if (S.gate == KDA_SCAN_LOWER_BOUND) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const F y = add(z[i], C.b);
            const sig<F> w = sigmoids(mul(C.rate, y));
            z[i] = mul(mul(mul(splat<F>(S.g_min), C.rate), w.s), w.n);
            dA[i] = mul(z[i], y);
        }
    } else if (S.gate == KDA_SCAN_SIGMOID) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const sig<F> w = sigmoids(add(z[i], C.b));
            dA[i] = mul(k, w.s);
            z[i] = mul(dA[i], w.n);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const F y = add(z[i], C.b);
            dA[i] = mul(k, softplus(y));
            z[i] = mul(k, sigmoid(y));
        }
    }
}

// c(a) = sqrt(1 - a^2) from m = a - 1: 1 - a^2 = -m (2 + m) has no cancellation.  Where it is not above 1e-30, c and its derivative
// count as 0.  (A NaN's c is 0, but its decay is a NaN, too.)  inverse: 1 / c
template <typename F> __device__ __forceinline__ F norm_factor(F m, F *inverse) {
    const F q = each([](float v) { return fmaxf(v, 0.f); }, fma(mul(m, splat<F>(-1.f)), add(m, splat<F>(2.f)), splat<F>(-1e-30f)));
    *inverse = rsq(add(q, splat<F>(1e-37f)));
    return mul(q, *inverse);
}

// N tokens' log-decays from their logits, in place, and what enters at them, x -> c(a) Sigmoid(i) x with m = a - 1.  The
// kinds are told apart outside the loops, so that a polynomial's constants are set up once for all tokens.
template <int N, typename F> __device__ __forceinline__ void log_decays(const spec &S, const channel<F> &C, F (&z)[N]) {
    const F k = mul(C.rate, splat<F>(-1.f)), nudge = splat<F>(NUDGE);
    if (S.gate == KDA_SCAN_LOG) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = add(z[i], nudge);
    } else if (S.gate == KDA_SCAN_SOFTPLUS) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = fma(k, softplus(add(z[i], C.b)), nudge);
    } else if (S.gate == KDA_SCAN_SIGMOID) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = fma(k, sigmoid(add(z[i], C.b)), nudge);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = fma(splat<F>(S.g_min), sigmoid(mul(C.rate, add(z[i], C.b))), nudge);
    }
}
template <int N, typename F> __device__ __forceinline__ void scale_inputs(const spec &S, const F (&m)[N], F (&x)[N]) {
    if (S.input == KDA_SCAN_INPUT_PLAIN) return;
    if (S.input == KDA_SCAN_INPUT_COMPLEMENT) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = mul(x[i], mul(m[i], splat<F>(-1.f)));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            F inverse;
            x[i] = mul(x[i], norm_factor(m[i], &inverse));
        }
    }
}
template <int N, typename F> __device__ __forceinline__ void gate_inputs(const F (&i)[N], F (&x)[N]) {
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = mul(x[k], sigmoid(i[k]));
}

// For the gradients: with d the decays, x what enters but for c(a), and e = a h: e += dc/dg x, and x's factor s *= c.  dc/dg is -a of
// c = 1 - a and -a^2 / c of sqrt(1 - a^2).
template <int N, typename F>
__device__ __forceinline__ void input_slopes(const spec &S, const F *d, const F (&x)[N], F (&e)[N], F (&s)[N]) {
    const F minus = splat<F>(-1.f);
    if (S.input == KDA_SCAN_INPUT_COMPLEMENT) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            e[i] = fma(mul(factor(d[i]), minus), x[i], e[i]);
            s[i] = mul(s[i], mul(below_one(d[i]), minus));
        }
    } else if (S.input == KDA_SCAN_INPUT_NORM) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            F inverse;
            const F c = norm_factor(below_one(d[i]), &inverse), a = factor(d[i]);
            // (c / c is 0 where c is)
            e[i] = fma(mul(mul(mul(a, a), inverse), mul(mul(c, inverse), minus)), x[i], e[i]);
            s[i] = mul(s[i], c);
        }
    }
}

template <int V, typename F>
__device__ __forceinline__ void load_channels(const float *A_log, const float *dt_bias, int c, bool some, channel<F> *C) {
    float b[V], r[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        b[v] = some && dt_bias ? dt_bias[c + v] : 0.f;
        r[v] = some && A_log ? expf(A_log[c + v]) : 1.f;
    }
#pragma unroll
    for (int i = 0; i < layer::lanes<V>::N; ++i) {
        if constexpr (std::is_same<F, float2>::value) C[i] = {make_float2(b[2 * i], b[2 * i + 1]), make_float2(r[2 * i], r[2 * i + 1])};
        else C[i] = {b[i], r[i]};
    }
}

}  // namespace scan
}  // namespace kda
