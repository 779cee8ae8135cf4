// kda_block_norm_bwd.  With yh = y / rms(y), p = post_weight * yh (or y), s = Sigmoid(gate), rh = r' / rms(r'):
//     d   = dL/dr' + (pre_weight dn - rh mean(pre_weight dn rh)) / rms(r')          all of the gradient of r', and of r
//     dgate = d scale p s (1 - s),   dscale = sum d s p,   dp = d scale s
//     dy  = (post_weight dp - yh mean(post_weight dp yh)) / rms(y)
//     dpre_weight = sum dn rh,   dpost_weight = sum dp yh                            sums over tokens
//
// Bound by HBM traffic: y, gate, r, dr' and dn read once, dr, dy and dgate written once (16 bytes per channel in bf16).  A
// row stays in registers between its three sums; a block takes every G-th row and keeps the tokens' sums of its columns in
// registers, the blocks' sums meet in a second kernel in a fixed order.
#include "kda_block_norm.cuh"

namespace kda {
namespace norm {

// rows of sums that the blocks leave: at most this many blocks
constexpr int MAX_BLOCKS = 152 * 4;

template <typename T, typename RT, int V, int E, int NT>
__global__ void __launch_bounds__(place<NT>::BLOCK) block_norm_bwd_kernel(const __grid_constant__ kda_block_norm_bwd_args A, float *sums) {
    __shared__ float parts[2 * 2 * (NT > 32 ? NT / 32 : 1)];
    const int tid = threadIdx.x % NT;
    const int64_t first = (int64_t)blockIdx.x * place<NT>::ROWS + threadIdx.x / NT, each = (int64_t)gridDim.x * place<NT>::ROWS;
    int at = 0;
    const bool block = A.y != nullptr, channel = A.gate_kind == KDA_NORM_GATE_CHANNEL, pre = A.pre_norm && A.grad_normed;
    float sw[E * V] = {}, sp[E * V] = {}, sc[E * V] = {};  // sums for post_weight, pre_weight and scale
    for (int64_t row = first; row < A.T; row += each) {
        const int64_t base = row * A.D;
        layer::vec<T, V> y[E], g[E], dn[E];
        float r[E * V], d[E * V];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = (e * NT + tid) * V;
            if (c >= A.D) continue;
            layer::unpack<RT, V>(layer::load<RT, V>((const RT *)A.residual + base + c), r + e * V);
            if (block) y[e] = layer::load<T, V>((const T *)A.y + base + c);
            if (channel) g[e] = layer::load<T, V>((const T *)A.gate + base + c);
            if (pre) dn[e] = layer::load<T, V>((const T *)A.grad_normed + base + c);
            if (A.grad_residual_out) layer::unpack<RT, V>(layer::load<RT, V>((const RT *)A.grad_residual_out + base + c), d + e * V);
            else
#pragma unroll
                for (int i = 0; i < V; ++i) d[e * V + i] = 0.f;
        }
        float ky = 1.f, kt = 1.f;  // 1 / rms(y), and the gate of a token
        if (A.post_norm) {
            float ss[1] = {0.f};
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if ((e * NT + tid) * V >= A.D) continue;
                float f[V];
                layer::unpack<T, V>(y[e], f);
#pragma unroll
                for (int i = 0; i < V; ++i) ss[0] = fmaf(f[i], f[i], ss[0]);
            }
            row_sum<NT>(ss, parts, at);
            ky = rsqrtf(ss[0] / A.D + A.eps);
        }
        if (A.gate_kind == KDA_NORM_GATE_TOKEN) kt = sigmoid(ld((const T *)A.gate + row));
        if (pre) {
            float ss[2] = {0.f, 0.f};
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int c = (e * NT + tid) * V;
                if (c >= A.D) continue;
                float f[V], s[V], w[V], gf[V], nf[V];
                if (block) {
                    layer::unpack<T, V>(y[e], f);
                    load_weight<V>(A.scale_vec, c, s);
                    load_weight<V>(A.post_weight, c, w);
                    if (channel) layer::unpack<T, V>(g[e], gf);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float p = ky * f[i] * w[i] * (A.scale_vec ? s[i] : A.scale);
                        r[e * V + i] = fmaf(p, channel ? sigmoid(gf[i]) : kt, r[e * V + i]);
                    }
                }
                layer::unpack<T, V>(dn[e], nf);
                load_weight<V>(A.pre_weight, c, w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    ss[0] = fmaf(r[e * V + i], r[e * V + i], ss[0]);
                    ss[1] = fmaf(w[i] * nf[i], r[e * V + i], ss[1]);
                }
            }
            row_sum<NT>(ss, parts, at);
            const float k = rsqrtf(ss[0] / A.D + A.eps), m = ss[1] * k * k / A.D;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int c = (e * NT + tid) * V;
                if (c >= A.D) continue;
                float w[V], nf[V];
                layer::unpack<T, V>(dn[e], nf);
                load_weight<V>(A.pre_weight, c, w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    sp[e * V + i] = fmaf(nf[i], k * r[e * V + i], sp[e * V + i]);
                    d[e * V + i] = fmaf(k, w[i] * nf[i] - r[e * V + i] * m, d[e * V + i]);
                }
            }
        }
        // d is complete
        float ss[2] = {0.f, 0.f};  // post_weight dp yh, and d scale p of a token's gate
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = (e * NT + tid) * V;
            if (c >= A.D) continue;
            layer::store((RT *)A.grad_residual + base + c, layer::pack<RT, V>(d + e * V));
            if (!block) continue;
            float f[V], s[V], w[V], gf[V], dg[V];
            layer::unpack<T, V>(y[e], f);
            load_weight<V>(A.scale_vec, c, s);
            load_weight<V>(A.post_weight, c, w);
            if (channel) layer::unpack<T, V>(g[e], gf);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int j = e * V + i;
                const float yh = ky * f[i], p = w[i] * yh, k = channel ? sigmoid(gf[i]) : kt;
                sc[j] = fmaf(d[j] * k, p, sc[j]);
                const float ds = d[j] * (A.scale_vec ? s[i] : A.scale);
                dg[i] = ds * p * k * (1.f - k);
                ss[1] = fmaf(ds, p, ss[1]);
                const float dp = ds * k;
                sw[j] = fmaf(dp, yh, sw[j]);
                d[j] = dp * w[i];
                ss[0] = fmaf(d[j], yh, ss[0]);
            }
            if (channel) layer::store((T *)A.grad_gate + base + c, layer::pack<T, V>(dg));
        }
        if (!block) continue;
        if (A.post_norm || A.gate_kind == KDA_NORM_GATE_TOKEN) row_sum<NT>(ss, parts, at);
        if (A.gate_kind == KDA_NORM_GATE_TOKEN && tid == 0) st((T *)A.grad_gate + row, ss[1] * kt * (1.f - kt));
        const float m = A.post_norm ? ss[0] / A.D : 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = (e * NT + tid) * V;
            if (c >= A.D) continue;
            float f[V];
            layer::unpack<T, V>(y[e], f);
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = ky * (d[e * V + i] - ky * f[i] * m);
            layer::store((T *)A.grad_y + base + c, layer::pack<T, V>(f));
        }
    }
    if (!sums) return;
    // [row of the grid][3][D]
    float *out = sums + first * 3 * A.D;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = (e * NT + tid) * V;
        if (c >= A.D) continue;
        layer::store(out + c, layer::pack<float, V>(sw + e * V));
        layer::store(out + A.D + c, layer::pack<float, V>(sp + e * V));
        layer::store(out + 2 * A.D + c, layer::pack<float, V>(sc + e * V));
    }
}

// Column sums of the blocks' rows: 8 rows at a time by the warps of a block, 32 columns to a block.
__global__ void __launch_bounds__(256) block_norm_sums_kernel(const float *sums, int rows, int D, float *post, float *pre, float *scale) {
    __shared__ float part[8][32];
    float *out = blockIdx.y == 0 ? post : blockIdx.y == 1 ? pre : scale;
    if (!out) return;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < D)
        for (int r = w; r < rows; r += 8) v += sums[((int64_t)r * 3 + blockIdx.y) * D + c];
    part[w][lane] = v;
    __syncthreads();
    if (w == 0 && c < D) {
        v = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v += part[i][lane];
        out[c] = v;
    }
}

}  // namespace norm
}  // namespace kda

size_t kda_block_norm_bwd_bytes(int64_t T, int D) {
    const int64_t rows = T < kda::norm::MAX_BLOCKS ? T : kda::norm::MAX_BLOCKS;
    return (size_t)((rows + 3) / 4 * 4) * 3 * D * 4;
}

kda_status_t kda_launch_block_norm_bwd(const kda_block_norm_bwd_args *a, void *ws, cudaStream_t stream) {
    using namespace kda::norm;
    const bool want = a->grad_post_weight || a->grad_pre_weight || a->grad_scale;
    int rows = 0;
    if (a->T > 0) {
        const bool wide = all_wide(a->D, a->dtype, {a->residual, a->y, a->gate_kind == KDA_NORM_GATE_CHANNEL ? a->gate : nullptr, a->scale_vec,
                                                    a->post_weight, a->pre_weight, a->grad_residual_out, a->grad_normed, a->grad_y,
                                                    a->gate_kind == KDA_NORM_GATE_CHANNEL ? a->grad_gate : nullptr, a->grad_residual});
        choose(a->dtype, a->residual_dtype, a->D, wide, [&](auto t) {
            using K = decltype(t);
            using P = place<K::nt>;
            int64_t blocks = (a->T + P::ROWS - 1) / P::ROWS;
            if (blocks > MAX_BLOCKS / P::ROWS) blocks = MAX_BLOCKS / P::ROWS;
            rows = (int)blocks * P::ROWS;
            block_norm_bwd_kernel<typename K::t, typename K::rt, K::v, K::e, K::nt>
                <<<(unsigned)blocks, P::BLOCK, 0, stream>>>(*a, want ? (float *)ws : nullptr);
        });
    }
    if (want)
        block_norm_sums_kernel<<<dim3((a->D + 31) / 32, 3), 256, 0, stream>>>((const float *)ws, rows, a->D, a->grad_post_weight,
                                                                            a->grad_pre_weight, a->grad_scale);
    return kda_cuda_status(cudaGetLastError());
}
