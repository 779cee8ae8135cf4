// kda_block_norm_fwd: r' = r + scale * Sigmoid(gate) * P(y), P an RMSNorm or nothing, and n = RMSNorm(r').
//
// Bound by HBM traffic: y, the gate and r are read once, r' and n written once (10 bytes per channel in bf16, 14 with
// an fp32 residual).  A row stays in the registers of its threads between the two sums that its norms need; the
// weights come from L1 and L2.  65535 rows of 4096: with an fp32 residual 536 us, 7.0 TB/s,
// in bf16 437 us, 6.1 TB/s (one channel at a time 481; 512 threads a row were no faster than 256).
#include "kda_block_norm.cuh"

namespace kda {
namespace norm {

// Blocks that run on an SM.  More of them cover a row's two trips through its sums, but registers have to suffice: rows of 4096 in bf16 with a
// bf16 residual 438 us by five of 256 threads (48 registers; 463 by four), of 7168 955 by three of 512 (995 by two); with an fp32
// residual or in fp32 552 for 538 and worse, so that the compiler has its way there.
template <typename RT, int V, int E, int NT> constexpr int blocks_at_once = sizeof(RT) == 2 && V > 1 && E > 1 ? (NT == 256 ? 5 : NT == 512 ? 3 : 0) : 0;

template <typename T, typename RT, int V, int E, int NT>
__global__ void __launch_bounds__(place<NT>::BLOCK, (blocks_at_once<RT, V, E, NT>)) block_norm_fwd_kernel(const __grid_constant__ kda_block_norm_args A) {
    __shared__ __align__(16) float parts[2 * 2 * (NT > 32 ? NT / 32 : 1)];
    const int tid = threadIdx.x % NT;
    const int64_t row = (int64_t)blockIdx.x * place<NT>::ROWS + threadIdx.x / NT;
    if (row >= A.T) return;  // a whole warp where a block has several rows, else never
    int at = 0;
    const int64_t base = row * A.D;
    using F = typename layer::lanes<V>::F;
    constexpr int P = layer::lanes<V>::N;  // values of a vector, one or two at a time
    F r[E][P];
    layer::vec<T, V> y[E], g[E];
    const bool block = A.y != nullptr, channel = A.gate_kind == KDA_NORM_GATE_CHANNEL;
    const float inv = 1.f / A.D;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = (e * NT + tid) * V;
        if (c >= A.D) continue;
        layer::unpack<RT, V>(layer::load<RT, V>((const RT *)A.residual + base + c), r[e]);
        if (block) y[e] = layer::load<T, V>((const T *)A.y + base + c);
        if (channel) g[e] = layer::load<T, V>((const T *)A.gate + base + c);
    }
    if (block) {
        float k = 1.f;
        if (A.post_norm) {
            F q = layer::splat<F>(0.f);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if ((e * NT + tid) * V >= A.D) continue;
                F f[P];
                layer::unpack<T, V>(y[e], f);
#pragma unroll
                for (int i = 0; i < P; ++i) q = layer::fma(f[i], f[i], q);
            }
            float ss[1] = {total(q)};
            row_sum<NT>(ss, parts, at);
            k = rsqrtf(ss[0] * inv + A.eps);
        }
        if (A.gate_kind == KDA_NORM_GATE_TOKEN) k *= layer::sigmoid(ld((const T *)A.gate + row));
        if (!A.scale_vec) k *= A.scale;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = (e * NT + tid) * V;
            if (c >= A.D) continue;
            F f[P], w[P];
            layer::unpack<T, V>(y[e], f);
#pragma unroll
            for (int i = 0; i < P; ++i) f[i] = layer::mul(f[i], layer::splat<F>(k));
            for (const float *p : {A.scale_vec, A.post_weight}) {
                if (!p) continue;
                layer::unpack<float, V>(layer::load<float, V>(p + c), w);
#pragma unroll
                for (int i = 0; i < P; ++i) f[i] = layer::mul(f[i], w[i]);
            }
            if (channel) {
                layer::unpack<T, V>(g[e], w);
#pragma unroll
                for (int i = 0; i < P; ++i) r[e][i] = layer::fma(f[i], layer::sigmoid(w[i]), r[e][i]);
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i) r[e][i] = layer::add(f[i], r[e][i]);
            }
            layer::store((RT *)A.residual_out + base + c, layer::pack<RT, V>(r[e]));
        }
    }
    if (!A.pre_norm) return;
    F q = layer::splat<F>(0.f);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if ((e * NT + tid) * V >= A.D) continue;
#pragma unroll
        for (int i = 0; i < P; ++i) q = layer::fma(r[e][i], r[e][i], q);
    }
    float ss[1] = {total(q)};
    row_sum<NT>(ss, parts, at);
    const F k = layer::splat<F>(rsqrtf(ss[0] * inv + A.eps));
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = (e * NT + tid) * V;
        if (c >= A.D) continue;
        if (A.pre_weight) {
            F w[P];
            layer::unpack<float, V>(layer::load<float, V>(A.pre_weight + c), w);
#pragma unroll
            for (int i = 0; i < P; ++i) r[e][i] = layer::mul(r[e][i], w[i]);
        }
#pragma unroll
        for (int i = 0; i < P; ++i) r[e][i] = layer::mul(r[e][i], k);
        layer::store((T *)A.normed + base + c, layer::pack<T, V>(r[e]));
    }
}

}  // namespace norm
}  // namespace kda

kda_status_t kda_launch_block_norm_fwd(const kda_block_norm_args *a, cudaStream_t stream) {
    using namespace kda::norm;
    const bool wide = all_wide(a->D, a->dtype, {a->residual, a->y, a->gate_kind == KDA_NORM_GATE_CHANNEL ? a->gate : nullptr, a->scale_vec,
                                                a->post_weight, a->pre_weight, a->residual_out, a->normed});
    choose(a->dtype, a->residual_dtype, a->D, wide, [&](auto t) {
        using K = decltype(t);
        using P = place<K::nt>;
        block_norm_fwd_kernel<typename K::t, typename K::rt, K::v, K::e, K::nt>
            <<<(unsigned)((a->T + P::ROWS - 1) / P::ROWS), P::BLOCK, 0, stream>>>(*a);
    });
    return kda_cuda_status(cudaGetLastError());
}
