// kda_block_norm_fwd: r' = r + scale * Sigmoid(gate) * P(y), P an RMSNorm or nothing, and n = RMSNorm(r').
//
// Bound by HBM traffic: y, the gate and r are read once, r' and n written once (10 bytes per channel in bf16, 14 with
// an fp32 residual).  A row stays in the registers of its threads between the two sums that its norms need; the
// weights come from L1 and L2.  65535 rows of 4096, fp32 residual: 531 us, 7.1 TB/s (512 threads a row were no faster than 256).
#include "kda_block_norm.cuh"

namespace kda {
namespace norm {

template <typename T, typename RT, int V, int E, int NT>
__global__ void __launch_bounds__(place<NT>::BLOCK) block_norm_fwd_kernel(const __grid_constant__ kda_block_norm_args A) {
    __shared__ float parts[2 * 2 * (NT > 32 ? NT / 32 : 1)];
    const int tid = threadIdx.x % NT;
    const int64_t row = (int64_t)blockIdx.x * place<NT>::ROWS + threadIdx.x / NT;
    if (row >= A.T) return;  // a whole warp where a block has several rows, else never
    int at = 0;
    const int64_t base = row * A.D;
    float r[E * V], ss[1] = {0.f};
    layer::vec<T, V> y[E], g[E];
    const bool block = A.y != nullptr, channel = A.gate_kind == KDA_NORM_GATE_CHANNEL;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = (e * NT + tid) * V;
        if (c >= A.D) continue;
        layer::unpack<RT, V>(layer::load<RT, V>((const RT *)A.residual + base + c), r + e * V);
        if (block) y[e] = layer::load<T, V>((const T *)A.y + base + c);
        if (channel) g[e] = layer::load<T, V>((const T *)A.gate + base + c);
    }
    if (block) {
        float k = 1.f;
        if (A.post_norm) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if ((e * NT + tid) * V >= A.D) continue;
                float f[V];
                layer::unpack<T, V>(y[e], f);
#pragma unroll
                for (int i = 0; i < V; ++i) ss[0] = fmaf(f[i], f[i], ss[0]);
            }
            row_sum<NT>(ss, parts, at);
            k = rsqrtf(ss[0] / A.D + A.eps);
        }
        if (A.gate_kind == KDA_NORM_GATE_TOKEN) k *= sigmoid(ld((const T *)A.gate + row));
        if (!A.scale_vec) k *= A.scale;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = (e * NT + tid) * V;
            if (c >= A.D) continue;
            float f[V], s[V], w[V], gf[V];
            layer::unpack<T, V>(y[e], f);
            load_weight<V>(A.scale_vec, c, s);
            load_weight<V>(A.post_weight, c, w);
            if (channel) layer::unpack<T, V>(g[e], gf);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float p = k * f[i] * w[i] * s[i];
                r[e * V + i] = fmaf(p, channel ? sigmoid(gf[i]) : 1.f, r[e * V + i]);
            }
            layer::store((RT *)A.residual_out + base + c, layer::pack<RT, V>(r + e * V));
        }
    }
    if (!A.pre_norm) return;
    ss[0] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if ((e * NT + tid) * V >= A.D) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) ss[0] = fmaf(r[e * V + i], r[e * V + i], ss[0]);
    }
    row_sum<NT>(ss, parts, at);
    const float k = rsqrtf(ss[0] / A.D + A.eps);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = (e * NT + tid) * V;
        if (c >= A.D) continue;
        float w[V];
        load_weight<V>(A.pre_weight, c, w);
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] *= k * r[e * V + i];
        layer::store((T *)A.normed + base + c, layer::pack<T, V>(w));
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
