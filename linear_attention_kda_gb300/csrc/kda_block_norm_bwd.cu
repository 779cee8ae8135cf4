// kda_block_norm_bwd.  With yh = y / rms(y), p = post_weight * yh (or y), s = Sigmoid(gate), rh = r' / rms(r'):
//     d   = dL/dr' + (pre_weight dn - rh mean(pre_weight dn rh)) / rms(r')          all of the gradient of r', and of r
//     dgate = d scale p s (1 - s),   dp = d scale s
//     dy  = (post_weight dp - yh mean(post_weight dp yh)) / rms(y)
//     dpre_weight = sum dn rh,   dpost_weight = scale sum d s yh,   dscale = post_weight sum d s yh      over tokens
//
// Bound by HBM traffic: y, gate, r, dr' and dn read once, dr, dy and dgate written once (16 bytes per channel in bf16).  A
// row stays in registers between its three sums, all arithmetic is on two channels at a time (about thirty instructions a channel; one at
// a time and with gates formed twice 98, 570 us for 16384 rows of 4096).  A block takes every G-th row, the next one on its way to
// shared memory meanwhile, and keeps the tokens' sums of its columns in registers; the blocks' sums meet in a second kernel in a
// fixed order.
#include <atomic>

#include "kda_block_norm.cuh"
#include "kda_linear.cuh"
#include "tc_util.cuh"

namespace kda {
namespace norm {

using layer::add;
using layer::fma;
using layer::mul;
using layer::splat;

// A row on its way: r, dr', y, gate and dn one after the other, those that the call has
template <typename T, typename RT> __host__ __device__ __forceinline__ int row_bytes(const kda_block_norm_bwd_args &A) {
    const int rt = A.D * (int)sizeof(RT), t = A.D * (int)sizeof(T);
    return rt + (A.grad_residual_out ? rt : 0) + (A.y ? t : 0) + (A.gate_kind == KDA_NORM_GATE_CHANNEL ? t : 0) + (A.grad_normed ? t : 0);
}

__device__ __forceinline__ float total(float v) { return v; }
__device__ __forceinline__ float total(float2 v) { return v.x + v.y; }

// BULK: rows come by bulk copies into two places of shared memory in turn
template <typename T, typename RT, int V, int E, int NT, bool BULK>
__global__ void __launch_bounds__(place<NT>::BLOCK, NT <= 256 ? 512 / place<NT>::BLOCK : 1)
block_norm_bwd_kernel(const __grid_constant__ kda_block_norm_bwd_args A, float *sums, int *err) {
    using F = typename layer::lanes<V>::F;
    constexpr int P = layer::lanes<V>::N;  // values of a vector, one or two at a time
    __shared__ float parts[2 * 2 * (NT > 32 ? NT / 32 : 1)];
    __shared__ uint64_t full[2];
    extern __shared__ __align__(128) char memory[];
    const int tid = threadIdx.x % NT;
    const int64_t first = (int64_t)blockIdx.x * place<NT>::ROWS + threadIdx.x / NT, each = (int64_t)gridDim.x * place<NT>::ROWS;
    const bool block = A.y != nullptr, channel = A.gate_kind == KDA_NORM_GATE_CHANNEL, pre = A.grad_normed != nullptr;
    const int stage_bytes = BULK ? row_bytes<T, RT>(A) : 0, rt = A.D * (int)sizeof(RT), tt = A.D * (int)sizeof(T);
    auto ask = [&](int64_t row, int stage) {
        if (!BULK || threadIdx.x != 0 || row >= A.T) return;
        char *to = memory + stage * stage_bytes;
        tc::mbar_arrive_expect_tx(&full[stage], stage_bytes);
        auto copy = [&](const void *p, int bytes) {
            if (!p) return;
            tc::bulk_g2s(to, (const char *)p + row * bytes, bytes, &full[stage]);
            to += bytes;
        };
        copy(A.residual, rt);
        copy(A.grad_residual_out, rt);
        copy(A.y, tt);
        copy(channel ? A.gate : nullptr, tt);
        copy(A.grad_normed, tt);
    };
    if (BULK) {
        if (threadIdx.x == 0) {
            tc::mbar_init(&full[0], 1);
            tc::mbar_init(&full[1], 1);
            tc::fence_proxy_async();
        }
        __syncthreads();
        ask(first, 0);
        ask(first + each, 1);
    }
    int at = 0, stage = 0, phase = 0;
    F sq[E][P], sp[E][P];  // sums of d s yh and of dn rh
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
        for (int i = 0; i < P; ++i) sq[e][i] = sp[e][i] = splat<F>(0.f);
    const float inv = 1.f / A.D;
    for (int64_t row = first; row < A.T; row += each) {
        const int64_t base = row * A.D;
        F r[E][P], d[E][P], y[E][P], s[E][P], dn[E][P];
        if (BULK && !tc::mbar_wait(&full[stage], phase)) set_error(err, KDA_ERR_DEVICE_TIMEOUT);
        const char *here = memory + stage * stage_bytes;
        auto rows = [&](const void *p, auto kind, int bytes, F (&f)[E][P]) {
            using K = decltype(kind);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int c = (e * NT + tid) * V;
                if (p && c < A.D) layer::unpack<K, V>(layer::load<K, V>((BULK ? (const K *)here : (const K *)p + base) + c), f[e]);
                else
#pragma unroll
                    for (int i = 0; i < P; ++i) f[e][i] = splat<F>(0.f);
            }
            if (p) here += bytes;
        };
        rows(A.residual, RT{}, rt, r);
        rows(A.grad_residual_out, RT{}, rt, d);
        rows(A.y, T{}, tt, y);
        rows(channel ? A.gate : nullptr, T{}, tt, s);
        rows(A.grad_normed, T{}, tt, dn);
        const float kt = A.gate_kind == KDA_NORM_GATE_TOKEN ? layer::sigmoid(ld((const T *)A.gate + row)) : 1.f;
        if (BULK) {
            __syncthreads();
            ask(row + 2 * each, stage);
            if (++stage == 2) stage = 0, phase ^= 1;
        }
        float ky = 1.f;
        if (A.post_norm) {
            F q = splat<F>(0.f);
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
                for (int i = 0; i < P; ++i) q = fma(y[e][i], y[e][i], q);
            float ss[1] = {total(q)};
            row_sum<NT>(ss, parts, at);
            ky = rsqrtf(ss[0] * inv + A.eps);
        }
        // weights of a vector's channels: 1 where there are none, and behind the last channel
        auto weights = [&](const float *w, int e, F (&f)[P], float none) {
            const int c = (e * NT + tid) * V;
            if (w && c < A.D) layer::unpack<float, V>(layer::load<float, V>(w + c), f);
            else
#pragma unroll
                for (int i = 0; i < P; ++i) f[i] = splat<F>(none);
        };
        float sr[2] = {0.f, 0.f};
        {
            F q = splat<F>(0.f), t = q;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                F w[P], c[P], v[P];
                weights(A.post_weight, e, w, 1.f);
                weights(A.scale_vec, e, c, A.scale);
                weights(A.pre_weight, e, v, 1.f);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    if (block) {
                        s[e][i] = channel ? layer::sigmoid(s[e][i]) : splat<F>(kt);
                        y[e][i] = mul(y[e][i], splat<F>(ky));  // yh
                        r[e][i] = fma(mul(y[e][i], w[i]), mul(c[i], s[e][i]), r[e][i]);
                    }
                    q = fma(r[e][i], r[e][i], q);
                    t = fma(mul(v[i], dn[e][i]), r[e][i], t);
                }
            }
            sr[0] = total(q);
            sr[1] = total(t);
        }
        if (pre) {
            row_sum<NT>(sr, parts, at);
            const float k = rsqrtf(sr[0] * inv + A.eps), m = -sr[1] * k * k * inv;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                F v[P];
                weights(A.pre_weight, e, v, 1.f);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    sp[e][i] = fma(mul(dn[e][i], splat<F>(k)), r[e][i], sp[e][i]);
                    d[e][i] = fma(splat<F>(k), fma(r[e][i], splat<F>(m), mul(v[i], dn[e][i])), d[e][i]);
                }
            }
        }
        // d is complete
        F sy = splat<F>(0.f), sg = sy;  // sums of post_weight dp yh, and of d scale p for a token's gate
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = (e * NT + tid) * V;
            if (c < A.D) layer::store_once((RT *)A.grad_residual + base + c, layer::pack<RT, V>(d[e]));
            if (!block) continue;
            F w[P], cs[P], dg[P];
            weights(A.post_weight, e, w, 1.f);
            weights(A.scale_vec, e, cs, A.scale);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const F ds = mul(d[e][i], s[e][i]);
                sq[e][i] = fma(ds, y[e][i], sq[e][i]);
                const F g = mul(mul(cs[i], w[i]), y[e][i]);  // scale p
                dg[i] = mul(mul(g, ds), fma(s[e][i], splat<F>(-1.f), splat<F>(1.f)));
                sg = fma(d[e][i], g, sg);
                sy = fma(ds, g, sy);
                d[e][i] = mul(ds, mul(cs[i], w[i]));
            }
            if (channel && c < A.D) layer::store_once((T *)A.grad_gate + base + c, layer::pack<T, V>(dg));
        }
        if (!block) continue;
        float ss[2] = {total(sy), total(sg)};
        if (A.post_norm || A.gate_kind == KDA_NORM_GATE_TOKEN) row_sum<NT>(ss, parts, at);
        if (A.gate_kind == KDA_NORM_GATE_TOKEN && tid == 0) st((T *)A.grad_gate + row, ss[1] * kt * (1.f - kt));
        const float m = A.post_norm ? -ss[0] * inv : 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = (e * NT + tid) * V;
            if (c >= A.D) continue;
#pragma unroll
            for (int i = 0; i < P; ++i) d[e][i] = mul(fma(y[e][i], splat<F>(m), d[e][i]), splat<F>(ky));
            layer::store_once((T *)A.grad_y + base + c, layer::pack<T, V>(d[e]));
        }
    }
    if (!sums) return;
    // [row of the grid][2][D]
    float *out = sums + first * 2 * A.D;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = (e * NT + tid) * V;
        if (c >= A.D) continue;
        layer::store(out + c, layer::pack<float, V>(sq[e]));
        layer::store(out + A.D + c, layer::pack<float, V>(sp[e]));
    }
}

// Column sums of the blocks' rows: 8 rows at a time by the warps of a block, 32 columns to a block.
__global__ void __launch_bounds__(256) block_norm_sums_kernel(const float *sums, int rows, const __grid_constant__ kda_block_norm_bwd_args A) {
    __shared__ float part[8][32];
    const bool pre = blockIdx.y == 1;
    if (pre ? !A.grad_pre_weight : !A.grad_post_weight && !A.grad_scale) return;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < A.D)
        for (int r = w; r < rows; r += 8) v += sums[((int64_t)r * 2 + blockIdx.y) * A.D + c];
    part[w][lane] = v;
    __syncthreads();
    if (w > 0 || c >= A.D) return;
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += part[i][lane];
    if (pre) {
        A.grad_pre_weight[c] = v;
    } else {
        if (A.grad_post_weight) A.grad_post_weight[c] = v * (A.scale_vec ? A.scale_vec[c] : A.scale);
        if (A.grad_scale) A.grad_scale[c] = v * (A.post_weight ? A.post_weight[c] : 1.f);
    }
}

template <typename K, bool BULK>
static cudaError_t launch(const kda_block_norm_bwd_args *a, float *sums, int smem, cudaStream_t stream, int *rows, int *err) {
    using P = place<K::nt>;
    auto *kernel = block_norm_bwd_kernel<typename K::t, typename K::rt, K::v, K::e, K::nt, BULK>;
    if (smem > 48 * 1024) {
        static std::atomic<uint64_t> done{0};
        const cudaError_t e = lin::allow_smem(kernel, 227 * 1024 - 1024, done);
        if (e != cudaSuccess) return e;
    }
    // as many blocks as run at once: 512 threads to an SM
    const int64_t most = 152 * (K::nt <= 256 ? 512 / P::BLOCK : 1);
    int64_t blocks = (a->T + P::ROWS - 1) / P::ROWS;
    if (blocks > most) blocks = most;
    *rows = (int)blocks * P::ROWS;
    kernel<<<(unsigned)blocks, P::BLOCK, smem, stream>>>(*a, sums, err);
    return cudaGetLastError();
}

}  // namespace norm
}  // namespace kda

size_t kda_block_norm_bwd_bytes(int64_t T, int D) {
    // rows: four for each block of warps, one for each other block
    const int64_t most = 152 * 16, rows = (T + 3) / 4 * 4;
    return (size_t)(rows < most ? rows : most) * 2 * D * 4;
}

kda_status_t kda_launch_block_norm_bwd(const kda_block_norm_bwd_args *a, void *ws, cudaStream_t stream) {
    int *err = kda_device_error_ptr();
    if (!err) return KDA_ERR_CUDA;
    using namespace kda::norm;
    const bool want = a->grad_post_weight || a->grad_pre_weight || a->grad_scale;
    int rows = 0;
    cudaError_t e = cudaSuccess;
    if (a->T > 0) {
        const bool wide = all_wide(a->D, a->dtype, {a->residual, a->y, a->gate_kind == KDA_NORM_GATE_CHANNEL ? a->gate : nullptr, a->scale_vec,
                                                    a->post_weight, a->pre_weight, a->grad_residual_out, a->grad_normed, a->grad_y,
                                                    a->gate_kind == KDA_NORM_GATE_CHANNEL ? a->grad_gate : nullptr, a->grad_residual});
        choose(a->dtype, a->residual_dtype, a->D, wide, [&](auto t) {
            using K = decltype(t);
            float *sums = want ? (float *)ws : nullptr;
            if constexpr (K::nt >= 128 && K::v > 1) {
                // two rows ahead, where as many blocks still fit into an SM
                const int smem = 2 * row_bytes<typename K::t, typename K::rt>(*a);
                if (smem <= (K::nt <= 256 ? 112 * place<K::nt>::BLOCK / 256 : 224) * 1024) {
                    e = launch<K, true>(a, sums, smem, stream, &rows, err);
                    return;
                }
            }
            e = launch<K, false>(a, sums, 0, stream, &rows, err);
        });
    }
    if (e == cudaSuccess && want) {
        block_norm_sums_kernel<<<dim3((a->D + 31) / 32, 2), 256, 0, stream>>>((const float *)ws, rows, *a);
        e = cudaGetLastError();
    }
    return kda_cuda_status(e);
}
