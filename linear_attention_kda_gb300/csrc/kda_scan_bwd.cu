// kda_scan_bwd: a thread per (sequence, channel) goes through the tokens.
#include "kda_internal.h"
#include "kda_linear.cuh"
#include "kda_scan.cuh"

namespace kda {
namespace scan {

constexpr int CK = KDA_SCAN_CHECKPOINT;

template <typename T>
__global__ void __launch_bounds__(128) scan_bwd_kernel(kda_scan_bwd_args A, spec S, float *part, int *err) {
    const int c = blockIdx.x * 128 + threadIdx.x;
    const int64_t n = blockIdx.y;
    lin::span s;
    const bool good = lin::seq_span(A.cu_seqlens, A.T, A.N, n, &s);
    if (!good && threadIdx.x == 0) set_error(err, KDA_ERR_BAD_SEQLENS);
    if (c >= A.D) return;
    float sA = 0.f, sb = 0.f;
    if (good) {
        channel<float> C[1];
        load_channels<1>(A.A_log, A.dt_bias, c, true, C);
        float lam = A.grad_final_state ? A.grad_final_state[n * A.D + c] : 0.f, before[CK];
        for (int64_t k = (s.b - s.a + CK - 1) / CK - 1; k >= 0; --k) {
            const int64_t t0 = s.a + k * CK;
            const int len = (int)(s.b - t0 < CK ? s.b - t0 : CK);
            float h = A.checkpoints[(s.a / CK + n + k) * A.D + c];
            for (int r = 0; r < len; ++r) {
                const int64_t t = t0 + r;
                before[r] = h;
                float dz, dA;
                const decay<float> d = decay_of(log_decay(S, C[0], ld((const T *)A.z + t * A.z_stride + c), &dz, &dA));
                const float m[1] = {d.m};
                float x[1] = {ld((const T *)A.x + t * A.x_stride + c)}, i[1];
                scale_inputs(S, m, x);
                if (A.input_gate) {
                    i[0] = ld((const T *)A.input_gate + t * A.i_stride + c);
                    gate_inputs(i, x);
                }
                h = step_or_erase(d.d, h, x[0]);
            }
            for (int r = len - 1; r >= 0; --r) {
                const int64_t t = t0 + r;
                float dz, dA;
                const decay<float> d = decay_of(log_decay(S, C[0], ld((const T *)A.z + t * A.z_stride + c), &dz, &dA));
                const float x = ld((const T *)A.x + t * A.x_stride + c), cf = S.input == KDA_SCAN_INPUT_PLAIN ? 1.f : input_factor(S, d.m);
                sig<float> w{1.f, 0.f};
                if (A.input_gate) w = sigmoids(ld((const T *)A.input_gate + t * A.i_stride + c));
                lam += ld((const T *)A.grad_h + t * A.D + c);
                st((T *)A.grad_x + t * A.D + c, cf * w.s * lam);
                if (A.input_gate) st((T *)A.grad_input_gate + t * A.D + c, cf * x * w.s * w.n * lam);
                const float dg = step_or_erase(d.d, before[r], S.input == KDA_SCAN_INPUT_PLAIN ? 0.f : input_slope(S, factor(d.d), cf) * w.s * x) * lam;
                st((T *)A.grad_z + t * A.D + c, dg * dz);
                sA += dg * dA;
                sb += dg * dz;
                lam = step_or_erase(d.d, lam, 0.f);
            }
        }
        if (A.grad_initial_state) A.grad_initial_state[n * A.D + c] = lam;
    }
    part[(2 * n) * A.D + c] = sA;
    part[(2 * n + 1) * A.D + c] = sb;
}

__global__ void __launch_bounds__(128) scan_params_kernel(const float *part, int64_t N, int D, float *dA, float *db) {
    const int c = blockIdx.x * 128 + threadIdx.x;
    if (c >= D) return;
    float sA = 0.f, sb = 0.f;
    for (int64_t n = 0; n < N; ++n) {
        sA += part[2 * n * D + c];
        sb += part[(2 * n + 1) * D + c];
    }
    if (dA) dA[c] = sA;
    if (db) db[c] = sb;
}

}  // namespace scan
}  // namespace kda

size_t kda_scan_bwd_bytes(int64_t, int64_t N, int D, kda_dtype_t) { return (size_t)N * D * 8; }

kda_status_t kda_launch_scan_bwd(const kda_scan_bwd_args *a, void *ws, cudaStream_t stream) {
    int *err = kda_device_error_ptr();
    if (!err) return KDA_ERR_CUDA;
    using namespace kda::scan;
    const spec S{a->gate_kind, a->input_scale, a->g_min};
    const dim3 grid((a->D + 127) / 128, (unsigned)a->N);
    if (a->dtype == KDA_BF16) scan_bwd_kernel<kda::bf16><<<grid, 128, 0, stream>>>(*a, S, (float *)ws, err);
    else scan_bwd_kernel<float><<<grid, 128, 0, stream>>>(*a, S, (float *)ws, err);
    if (a->grad_A_log || a->grad_dt_bias)
        scan_params_kernel<<<grid.x, 128, 0, stream>>>((const float *)ws, a->N, a->D, a->grad_A_log, a->grad_dt_bias);
    return kda_cuda_status(cudaGetLastError());
}
