// kda_short_conv_fwd, _bwd, _step: a thread per (token, channel).
#include "kda_internal.h"
#include "kda_layer.cuh"
#include "kda_linear.cuh"

namespace kda {
namespace conv {

struct spec {
    int64_t T, N;
    int D, K, act, norm;
    float eps;
    const float *w, *b;
    const int32_t *cu;
};

// element e of a sequence's history and tokens, one after the other
template <typename T>
__device__ __forceinline__ float row(const spec &S, const T *x, int64_t stride, const T *hist, int64_t n, int64_t a, int64_t e, int c) {
    if (e < S.K - 1) return hist ? ld(hist + (n * (S.K - 1) + e) * S.D + c) : 0.f;
    return ld(x + (a + e - (S.K - 1)) * stride + c);
}

__device__ __forceinline__ float head_sum(float v, int norm) {
    __shared__ float part[8];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    const int w = norm / 32, first = (threadIdx.x >> 5) / w * w;
    v = 0.f;
    for (int i = 0; i < w; ++i) v += part[first + i];
    return v;
}

template <typename T>
__global__ void __launch_bounds__(256) conv_fwd_kernel(spec S, const T *x, int64_t stride, const T *hist, T *y) {
    const int64_t t = blockIdx.x;
    const int c = blockIdx.y * 256 + threadIdx.x;
    const int64_t n = S.cu ? find_seq(S.cu, (int)S.N, t) : t / (S.T / S.N);
    lin::span s;
    if (!lin::seq_span(S.cu, S.T, S.N, n, &s) || t < s.a || t >= s.b) return;
    float p = 0.f;
    if (c < S.D) {
        p = S.b ? S.b[c] : 0.f;
        for (int j = 0; j < S.K; ++j) p = fmaf(S.w[(int64_t)c * S.K + j], row(S, x, stride, hist, n, s.a, t - s.a + j, c), p);
        if (S.act) p = p / (1.f + expf(-p));
    }
    if (S.norm) p *= rsqrtf(head_sum(p * p, S.norm) + S.eps);
    if (c < S.D) st(y + t * S.D + c, p);
}

template <typename T>
__global__ void __launch_bounds__(256) conv_tail_kernel(spec S, const T *x, int64_t stride, const T *hist, T *out, int *err) {
    const int64_t n = blockIdx.x;
    const int c = blockIdx.y * 256 + threadIdx.x;
    lin::span s;
    if (!lin::seq_span(S.cu, S.T, S.N, n, &s)) {
        if (threadIdx.x == 0) set_error(err, KDA_ERR_BAD_SEQLENS);
        return;
    }
    if (c >= S.D || !out) return;
    float v[3];
    for (int r = 0; r < S.K - 1; ++r) v[r] = row(S, x, stride, hist, n, s.a, s.b - s.a + r, c);
    for (int r = 0; r < S.K - 1; ++r) st(out + (n * (S.K - 1) + r) * S.D + c, v[r]);
}

// dL/dp of every token
template <typename T>
__global__ void __launch_bounds__(256) conv_dp_kernel(spec S, const T *x, int64_t stride, const T *hist, const T *dy, float *dp) {
    const int64_t t = blockIdx.x;
    const int c = blockIdx.y * 256 + threadIdx.x;
    const int64_t n = S.cu ? find_seq(S.cu, (int)S.N, t) : t / (S.T / S.N);
    lin::span s;
    if (!lin::seq_span(S.cu, S.T, S.N, n, &s) || t < s.a || t >= s.b) return;
    float p = 0.f, d = 0.f, v = 0.f, sg = 1.f;
    if (c < S.D) {
        p = S.b ? S.b[c] : 0.f;
        for (int j = 0; j < S.K; ++j) p = fmaf(S.w[(int64_t)c * S.K + j], row(S, x, stride, hist, n, s.a, t - s.a + j, c), p);
        if (S.act) sg = 1.f / (1.f + expf(-p));
        v = p * sg;
        d = ld(dy + t * S.D + c);
    }
    if (S.norm) {
        const float r = rsqrtf(head_sum(v * v, S.norm) + S.eps);
        d = r * (d - v * r * (head_sum(d * v, S.norm) * r));
    }
    if (S.act) d *= sg * (1.f + p * (1.f - sg));
    if (c < S.D) dp[t * S.D + c] = d;
}

// dL/d(element e of history and tokens)
template <typename T>
__device__ __forceinline__ float row_grad(const spec &S, const float *dp, const T *dtail, int64_t n, const lin::span &s, int64_t e, int c) {
    const int64_t len = s.b - s.a;
    float d = 0.f;
    for (int j = 0; j < S.K; ++j) {
        const int64_t t = e - j;
        if (t >= 0 && t < len) d = fmaf(S.w[(int64_t)c * S.K + j], dp[(s.a + t) * S.D + c], d);
    }
    if (dtail && e >= len) d += ld(dtail + (n * (S.K - 1) + e - len) * S.D + c);
    return d;
}

template <typename T>
__global__ void __launch_bounds__(256) conv_dx_kernel(spec S, const float *dp, const T *dtail, T *dx) {
    const int64_t t = blockIdx.x;
    const int c = blockIdx.y * 256 + threadIdx.x;
    const int64_t n = S.cu ? find_seq(S.cu, (int)S.N, t) : t / (S.T / S.N);
    lin::span s;
    if (!lin::seq_span(S.cu, S.T, S.N, n, &s) || t < s.a || t >= s.b || c >= S.D) return;
    st(dx + t * S.D + c, row_grad(S, dp, dtail, n, s, t - s.a + S.K - 1, c));
}

// per sequence: the history's gradient and the sums for weight and bias
template <typename T>
__global__ void __launch_bounds__(256) conv_sums_kernel(spec S, const T *x, int64_t stride, const T *hist, const float *dp, const T *dtail,
                                                        T *dhist, float *part, int *err) {
    const int64_t n = blockIdx.x;
    const int c = blockIdx.y * 256 + threadIdx.x;
    lin::span s;
    const bool good = lin::seq_span(S.cu, S.T, S.N, n, &s);
    if (!good && threadIdx.x == 0) set_error(err, KDA_ERR_BAD_SEQLENS);
    if (c >= S.D) return;
    float sum[5] = {};
    if (good) {
        for (int r = 0; dhist && r < S.K - 1; ++r) st(dhist + (n * (S.K - 1) + r) * S.D + c, row_grad(S, dp, dtail, n, s, r, c));
        for (int64_t t = s.a; t < s.b; ++t) {
            const float d = dp[t * S.D + c];
            for (int j = 0; j < S.K; ++j) sum[j] = fmaf(d, row(S, x, stride, hist, n, s.a, t - s.a + j, c), sum[j]);
            sum[4] += d;
        }
    }
    for (int j = 0; j < 5; ++j) part[(n * 5 + j) * S.D + c] = sum[j];
}

__global__ void __launch_bounds__(256) conv_params_kernel(const float *part, int64_t N, int D, int K, float *dw, float *db) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= D) return;
    for (int j = 0; j < 5; ++j) {
        float v = 0.f;
        for (int64_t n = 0; n < N; ++n) v += part[(n * 5 + j) * D + c];
        if (j < K && dw) dw[(int64_t)c * K + j] = v;
        if (j == 4 && db) db[c] = v;
    }
}

template <typename T>
__global__ void __launch_bounds__(256) conv_step_kernel(spec S, const T *x, int64_t stride, T *state, const int32_t *idx, int64_t slots,
                                                        T *y, int *err) {
    const int64_t n = blockIdx.x;
    const int c = blockIdx.y * 256 + threadIdx.x;
    int64_t slot;
    if (!layer::find_slot<256>(idx, slots, n, &slot, err)) return;
    float p = 0.f, v[4];
    if (c < S.D) {
        p = S.b ? S.b[c] : 0.f;
        for (int j = 0; j < S.K; ++j) {
            v[j] = row(S, x + n * stride, stride, (const T *)state, slot, 0, j, c);
            p = fmaf(S.w[(int64_t)c * S.K + j], v[j], p);
        }
        for (int j = 1; j < S.K; ++j) st(state + (slot * (S.K - 1) + j - 1) * S.D + c, v[j]);
        if (S.act) p = p / (1.f + expf(-p));
    }
    if (S.norm) p *= rsqrtf(head_sum(p * p, S.norm) + S.eps);
    if (c < S.D) st(y + n * S.D + c, p);
}

template <typename A>
static spec spec_of(const A *a) {
    return {a->T, a->N, a->D, a->K, a->activation, a->norm_dim, a->norm_eps, a->weight, a->bias, a->cu_seqlens};
}

template <typename T>
static void fwd(const kda_short_conv_args *a, cudaStream_t stream, int *err) {
    const spec S = spec_of(a);
    const unsigned by = (a->D + 255) / 256;
    if (a->T > 0) conv_fwd_kernel<T><<<dim3((unsigned)a->T, by), 256, 0, stream>>>(S, (const T *)a->x, a->x_stride, (const T *)a->initial_state, (T *)a->y);
    conv_tail_kernel<T><<<dim3((unsigned)a->N, by), 256, 0, stream>>>(S, (const T *)a->x, a->x_stride, (const T *)a->initial_state, (T *)a->final_state, err);
}

template <typename T>
static void bwd(const kda_short_conv_bwd_args *a, void *ws, cudaStream_t stream, int *err) {
    const spec S = spec_of(a);
    const unsigned by = (a->D + 255) / 256;
    float *dp = (float *)ws, *part = dp + a->T * a->D;
    const T *x = (const T *)a->x, *hist = (const T *)a->initial_state, *dtail = (const T *)a->grad_final_state;
    if (a->T > 0) {
        conv_dp_kernel<T><<<dim3((unsigned)a->T, by), 256, 0, stream>>>(S, x, a->x_stride, hist, (const T *)a->grad_y, dp);
        conv_dx_kernel<T><<<dim3((unsigned)a->T, by), 256, 0, stream>>>(S, dp, dtail, (T *)a->grad_x);
    }
    conv_sums_kernel<T><<<dim3((unsigned)a->N, by), 256, 0, stream>>>(S, x, a->x_stride, hist, dp, dtail, (T *)a->grad_initial_state, part, err);
    if (a->grad_weight || a->grad_bias) conv_params_kernel<<<by, 256, 0, stream>>>(part, a->N, a->D, a->K, a->grad_weight, a->grad_bias);
}

}  // namespace conv
}  // namespace kda

size_t kda_short_conv_bwd_bytes(int64_t T, int64_t N, int D, int) { return (size_t)(T + 5 * N) * D * 4; }

kda_status_t kda_launch_short_conv_fwd(const kda_short_conv_args *a, cudaStream_t stream) {
    int *err = kda_device_error_ptr();
    if (!err) return KDA_ERR_CUDA;
    if (a->dtype == KDA_BF16) kda::conv::fwd<kda::bf16>(a, stream, err);
    else kda::conv::fwd<float>(a, stream, err);
    return kda_cuda_status(cudaGetLastError());
}

kda_status_t kda_launch_short_conv_bwd(const kda_short_conv_bwd_args *a, void *ws, cudaStream_t stream) {
    int *err = kda_device_error_ptr();
    if (!err) return KDA_ERR_CUDA;
    if (a->dtype == KDA_BF16) kda::conv::bwd<kda::bf16>(a, ws, stream, err);
    else kda::conv::bwd<float>(a, ws, stream, err);
    return kda_cuda_status(cudaGetLastError());
}

kda_status_t kda_launch_short_conv_step(const kda_short_conv_step_args *a, cudaStream_t stream) {
    int *err = kda_device_error_ptr();
    if (!err) return KDA_ERR_CUDA;
    const kda::conv::spec S{a->N, a->N, a->D, a->K, a->activation, a->norm_dim, a->norm_eps, a->weight, a->bias, nullptr};
    const dim3 grid((unsigned)a->N, (a->D + 255) / 256);
    using kda::bf16;
    if (a->dtype == KDA_BF16)
        kda::conv::conv_step_kernel<bf16><<<grid, 256, 0, stream>>>(S, (const bf16 *)a->x, a->x_stride, (bf16 *)a->state, a->state_indices, a->num_slots, (bf16 *)a->y, err);
    else
        kda::conv::conv_step_kernel<float><<<grid, 256, 0, stream>>>(S, (const float *)a->x, a->x_stride, (float *)a->state, a->state_indices, a->num_slots, (float *)a->y, err);
    return kda_cuda_status(cudaGetLastError());
}
