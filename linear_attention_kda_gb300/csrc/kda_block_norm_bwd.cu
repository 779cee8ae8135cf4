// kda_block_norm_bwd.  With yh = y / rms(y), p = post_weight * yh (or y), s = Sigmoid(gate), rh = r' / rms(r'):
//     d   = dL/dr' + (pre_weight dn - rh mean(pre_weight dn rh)) / rms(r')          all of the gradient of r', and of r
//     dgate = d scale p s (1 - s),   dp = d scale s
//     dy  = (post_weight dp - yh mean(post_weight dp yh)) / rms(y)
//     dpre_weight = sum dn rh,   dpost_weight = scale sum d s yh,   dscale = post_weight sum d s yh      over tokens
//
// Bound by HBM traffic: y, gate, r, dr' and dn read once, dr, dy and dgate written once (16 bytes per channel in bf16).  A
// row stays in registers between its three sums, all arithmetic is on two channels at a time (45 instructions a channel, half of
// the issue slots).  16384 rows of 4096 in bf16: 185 us, 5.8 TB/s (588 at first); fp32 345 us, 6.2 TB/s.  A block takes every G-th row, the next one on its way to
// shared memory meanwhile, and keeps the tokens' sums of its columns in registers; the blocks' sums meet in a second kernel in a
// fixed order.  Rows of up to 512 channels, a warp to a row, have no next row on its way and wait for their loads: 262144 of 256 424 us, 2.5 TB/s,
// 131072 of 512 445 us.
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

template <typename K, bool BULK> __device__ __forceinline__ const void *at_row(const void *p, int64_t base, const char *near) {
    if constexpr (BULK) return near;
    return (const K *)p + base;
}
template <typename K, int V, typename F, int P> __device__ __forceinline__ void row_part(const void *p, int c, F (&f)[P]) {
    layer::unpack<K, V>(layer::load<K, V>((const K *)p + c), f);
}

// BULK: rows come by bulk copies into one or two places (`stages`) of shared memory in turn, and are read from there when they are needed.
// Behind them lie scale * post_weight and pre_weight.  FULL: the call has every part.
template <typename T, typename RT, int V, int E, int NT, bool BULK, bool FULL>
__global__ void __launch_bounds__(place<NT>::BLOCK, NT <= 256 ? 512 / place<NT>::BLOCK : 1)
block_norm_bwd_kernel(const __grid_constant__ kda_block_norm_bwd_args A, float *sums, int stages, int *err) {
    using F = typename layer::lanes<V>::F;
    constexpr int P = layer::lanes<V>::N;  // values of a vector, one or two at a time
    __shared__ __align__(16) float parts[2 * 2 * (NT > 32 ? NT / 32 : 1)];
    __shared__ uint64_t full[2];
    extern __shared__ __align__(128) char memory[];
    const int tid = threadIdx.x % NT;
    const int64_t first = (int64_t)blockIdx.x * place<NT>::ROWS + threadIdx.x / NT, each = (int64_t)gridDim.x * place<NT>::ROWS;
    const bool block = FULL || A.y != nullptr, channel = FULL || A.gate_kind == KDA_NORM_GATE_CHANNEL, pre = FULL || A.grad_normed != nullptr,
               post = FULL || A.post_norm, behind = FULL || A.grad_residual_out != nullptr, token = !FULL && A.gate_kind == KDA_NORM_GATE_TOKEN;
    const int stage_bytes = BULK ? row_bytes<T, RT>(A) : 0, rt = A.D * (int)sizeof(RT), tt = A.D * (int)sizeof(T);
    // where the parts of a row begin in its place
    const int at_d = rt, at_y = at_d + (behind ? rt : 0), at_g = at_y + (block ? tt : 0), at_n = at_g + (channel ? tt : 0);
    auto ask = [&](int64_t row, int stage) {
        if (!BULK || threadIdx.x != 0 || row >= A.T) return;
        char *to = memory + stage * stage_bytes;
        tc::mbar_arrive_expect_tx(&full[stage], stage_bytes);
        auto copy = [&](const void *p, int at, int bytes) {
            if (p) tc::bulk_g2s(to + at, (const char *)p + row * bytes, bytes, &full[stage]);
        };
        copy(A.residual, 0, rt);
        copy(A.grad_residual_out, at_d, rt);
        copy(A.y, at_y, tt);
        copy(channel ? A.gate : nullptr, at_g, tt);
        copy(A.grad_normed, at_n, tt);
    };
    float *const near = reinterpret_cast<float *>(memory + stages * stage_bytes);
    if (BULK) {
        if (threadIdx.x == 0) {
            tc::mbar_init(&full[0], 1);
            tc::mbar_init(&full[1], 1);
            tc::fence_proxy_async();
        }
        for (int c = threadIdx.x; c < A.D; c += NT) {
            near[c] = (A.scale_vec ? A.scale_vec[c] : A.scale) * (A.post_weight ? A.post_weight[c] : 1.f);
            near[A.D + c] = A.pre_weight ? A.pre_weight[c] : 1.f;
        }
        __syncthreads();
        ask(first, 0);
        if (stages == 2) ask(first + each, 1);
    }
    int at = 0, stage = 0, phase = 0;
    F sq[E][P], sp[E][P];  // sums of d s yh and of dn rh
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
        for (int i = 0; i < P; ++i) sq[e][i] = sp[e][i] = splat<F>(0.f);
    auto column = [&](int e) { return (e * NT + tid) * V; };
    // weights of a vector's channels
    auto from = [&](const float *w, int c, F (&f)[P], float none) {
        if (w) layer::unpack<float, V>(layer::load<float, V>(w + c), f);
        else
#pragma unroll
            for (int i = 0; i < P; ++i) f[i] = splat<F>(none);
    };
    auto scaled = [&](int c, F (&f)[P]) {  // scale * post_weight
        if constexpr (BULK) {
            layer::unpack<float, V>(layer::load<float, V>(near + c), f);
        } else {
            F w[P];
            from(A.scale_vec, c, f, A.scale);
            from(A.post_weight, c, w, 1.f);
#pragma unroll
            for (int i = 0; i < P; ++i) f[i] = mul(f[i], w[i]);
        }
    };
    auto normal = [&](int c, F (&f)[P]) {
        if constexpr (BULK) layer::unpack<float, V>(layer::load<float, V>(near + A.D + c), f);
        else from(A.pre_weight, c, f, 1.f);
    };
    const float inv = 1.f / A.D;
    for (int64_t row = first; row < A.T; row += each) {
        const int64_t base = row * A.D;
        const char *here = memory + stage * stage_bytes;
        if (BULK && !tc::mbar_wait(&full[stage], phase)) set_error(err, KDA_ERR_DEVICE_TIMEOUT);
        F r[E][P], d[E][P], y[E][P], s[E][P];
        const float kt = token ? layer::sigmoid(ld((const T *)A.gate + row)) : 1.f;
        float ky = 1.f;
        if (block) {
            F q = splat<F>(0.f);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (column(e) >= A.D) continue;
                row_part<T, V>(at_row<T, BULK>(A.y, base, here + at_y), column(e), y[e]);
#pragma unroll
                for (int i = 0; i < P; ++i) q = fma(y[e][i], y[e][i], q);
            }
            if (post) {
                float ss[1] = {total(q)};
                row_sum<NT>(ss, parts, at);
                ky = rsqrtf(ss[0] * inv + A.eps);
            }
        }
        F q = splat<F>(0.f), t = q;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = column(e);
            if (c >= A.D) continue;
            row_part<RT, V>(at_row<RT, BULK>(A.residual, base, here), c, r[e]);
            if (block) {
                F w[P];
                scaled(c, w);
                if (channel) {
                    row_part<T, V>(at_row<T, BULK>(A.gate, base, here + at_g), c, s[e]);
#pragma unroll
                    for (int i = 0; i < P; ++i) s[e][i] = layer::sigmoid(s[e][i]);
                } else {
#pragma unroll
                    for (int i = 0; i < P; ++i) s[e][i] = splat<F>(kt);
                }
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    y[e][i] = mul(y[e][i], splat<F>(ky));  // yh
                    r[e][i] = fma(mul(y[e][i], w[i]), s[e][i], r[e][i]);
                }
            }
            if (pre) {
                F n[P], v[P];
                row_part<T, V>(at_row<T, BULK>(A.grad_normed, base, here + at_n), c, n);
                normal(c, v);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    q = fma(r[e][i], r[e][i], q);
                    t = fma(mul(v[i], n[i]), r[e][i], t);
                }
            }
        }
        float k = 0.f, m = 0.f;
        if (pre) {
            float sr[2] = {total(q), total(t)};
            row_sum<NT>(sr, parts, at);
            k = rsqrtf(sr[0] * inv + A.eps);
            m = -sr[1] * k * k * inv;
        }
        F sy = splat<F>(0.f), sg = sy;  // sums of post_weight dp yh, and of d scale p for a token's gate
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = column(e);
            if (c >= A.D) continue;
            if (behind) row_part<RT, V>(at_row<RT, BULK>(A.grad_residual_out, base, here + at_d), c, d[e]);
            else
#pragma unroll
                for (int i = 0; i < P; ++i) d[e][i] = splat<F>(0.f);
            if (pre) {
                F n[P], v[P];
                row_part<T, V>(at_row<T, BULK>(A.grad_normed, base, here + at_n), c, n);
                normal(c, v);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    sp[e][i] = fma(mul(n[i], splat<F>(k)), r[e][i], sp[e][i]);
                    d[e][i] = fma(splat<F>(k), fma(r[e][i], splat<F>(m), mul(v[i], n[i])), d[e][i]);
                }
            }
            layer::store_once((RT *)A.grad_residual + base + c, layer::pack<RT, V>(d[e]));
            if (!block) continue;
            F w[P], dg[P];
            scaled(c, w);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const F ds = mul(d[e][i], s[e][i]), g = mul(w[i], y[e][i]);  // d s, scale p
                sq[e][i] = fma(ds, y[e][i], sq[e][i]);
                dg[i] = mul(mul(g, ds), fma(s[e][i], splat<F>(-1.f), splat<F>(1.f)));
                sg = fma(d[e][i], g, sg);
                sy = fma(ds, g, sy);
                d[e][i] = mul(ds, w[i]);
            }
            if (channel) layer::store_once((T *)A.grad_gate + base + c, layer::pack<T, V>(dg));
        }
        if (BULK) {
            __syncthreads();
            ask(row + stages * each, stage);
            if (++stage == stages) stage = 0, phase ^= 1;
        }
        if (!block) continue;
        float ss[2] = {total(sy), total(sg)};
        if (post || token) row_sum<NT>(ss, parts, at);
        if (token && tid == 0) st((T *)A.grad_gate + row, ss[1] * kt * (1.f - kt));
        m = -ss[0] * inv;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = column(e);
            if (c >= A.D) continue;
            if (post) {  // (without a norm nothing of y, which may be an infinity, is in its gradient)
#pragma unroll
                for (int i = 0; i < P; ++i) d[e][i] = mul(fma(y[e][i], splat<F>(m), d[e][i]), splat<F>(ky));
            }
            layer::store_once((T *)A.grad_y + base + c, layer::pack<T, V>(d[e]));
        }
    }
    if (!sums) return;
    // [row of the grid][2][D]
    float *out = sums + first * 2 * A.D;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = column(e);
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

struct share {
    int smem, stages, per_sm;  // of a block
};
template <typename K, bool BULK, bool FULL>
static cudaError_t launch(const kda_block_norm_bwd_args *a, float *sums, const share &S, cudaStream_t stream, int *rows, int *err) {
    using P = place<K::nt>;
    auto *kernel = block_norm_bwd_kernel<typename K::t, typename K::rt, K::v, K::e, K::nt, BULK, FULL>;
    if (S.smem > 46 * 1024) {  // (with what the kernel declares, above 48 KB)
        static std::atomic<uint64_t> done{0};
        const cudaError_t e = lin::allow_smem(kernel, 226 * 1024 + 512, done);
        if (e != cudaSuccess) return e;
    }
    int64_t blocks = (a->T + P::ROWS - 1) / P::ROWS;
    if (blocks > 152 * S.per_sm) blocks = 152 * S.per_sm;
    *rows = (int)blocks * P::ROWS;
    kernel<<<(unsigned)blocks, P::BLOCK, S.smem, stream>>>(*a, sums, S.stages, err);
    return cudaGetLastError();
}

// The weights and two rows on their way where as many blocks as registers allow (512 threads) still fit into an SM, else the weights and one
// row, else one block with two or one.  The largest row and its weights, fp32 of 8192, take 224 KB.  (bf16, 16384 rows of 4096 with an fp32
// residual: one row 247 us, two without the weights 338, one block with two rows and weights 274.  fp32 of 5120: one row 462 us, two
// without the weights 647.)  An SM has 228 KB, of which a block takes 1 KB and some bytes beside its rows.
static share share_of(int row, int weights, int per_sm) {
    for (int n : {per_sm, 1})
        for (int stages : {2, 1})
            if (stages * row + weights <= 228 * 1024 / n - 1024 - 512) return {stages * row + weights, stages, n};
    return {0, 0, 0};
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
        // a block, its norm and gate, and what comes behind them: the kernel that need not ask (16384 rows of 4096 185 us, 196;
        // fp32 346 for 336, so bf16 alone)
        const bool full = a->y && a->gate_kind == KDA_NORM_GATE_CHANNEL && a->post_norm && a->grad_normed && a->grad_residual_out;
        choose(a->dtype, a->residual_dtype, a->D, wide, [&](auto t) {
            using K = decltype(t);
            float *sums = want ? (float *)ws : nullptr;
            const int per_sm = K::nt <= 256 ? 512 / place<K::nt>::BLOCK : 1;
            if constexpr (K::nt >= 128 && K::v > 1) {
                const share S = share_of(row_bytes<typename K::t, typename K::rt>(*a), 8 * a->D, per_sm);
                if (S.smem == 0) e = cudaErrorInvalidConfiguration;
                else if (sizeof(typename K::t) == 2 && full) e = launch<K, true, sizeof(typename K::t) == 2>(a, sums, S, stream, &rows, err);
                else e = launch<K, true, false>(a, sums, S, stream, &rows, err);
            } else {
                e = launch<K, false, false>(a, sums, {0, 0, per_sm}, stream, &rows, err);
            }
        });
    }
    if (e == cudaSuccess && want) {
        block_norm_sums_kernel<<<dim3((a->D + 31) / 32, 2), 256, 0, stream>>>((const float *)ws, rows, *a);
        e = cudaGetLastError();
    }
    return kda_cuda_status(e);
}
