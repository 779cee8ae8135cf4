// kda_scan_step: one decode token per sequence of the gated recurrence over channels, states updated in place.
//
// Bound by HBM traffic (bf16 with an input gate: 8 bytes of tokens and 8 of state per channel), for few sequences by the
// launch.  A thread takes V channels of one sequence: its slot, then the state, then the block's vote on whether an earlier row has the slot, which is
// looked up while the loads are on their way.  256 sequences of 4096 channels, bf16, gated: 4.4 us replayed one after the other, 8.1 us with
// caches cold (16.8 MB, whose copy takes 2.5 us).
#include "kda_internal.h"
#include "kda_layer.cuh"
#include "kda_scan.cuh"

namespace kda {
namespace scan {

template <typename T, int V>
__global__ void __launch_bounds__(128) scan_step_kernel(const __grid_constant__ kda_scan_step_args A, int *err) {
    const int c = (blockIdx.y * 128 + threadIdx.x) * V;
    const int64_t n = blockIdx.x, slot = layer::slot_of(A.state_indices, A.num_slots, n, err);
    if (slot < 0) return;
    const spec S{A.gate_kind, A.input_scale, A.g_min};
    constexpr int P = layer::lanes<V>::N;
    using F = typename layer::lanes<V>::F;
    float *state = A.state + slot * A.D + c;
    const bool mine = c < A.D;
    layer::vec<T, V> rx, rz, ri;
    layer::vec<float, V> rs;
    if (mine) {
        rx = layer::load<T, V>((const T *)A.x + n * A.x_stride + c);
        rz = layer::load<T, V>((const T *)A.z + n * A.z_stride + c);
        if (A.input_gate) ri = layer::load<T, V>((const T *)A.input_gate + n * A.i_stride + c);
        rs = layer::load<float, V>(state);
    }
    channel<F> C[P];
    load_channels<V>(A.A_log, A.dt_bias, c, mine, C);
    if (layer::taken<128>(A.state_indices, n, slot, err) || !mine) return;
    F x[P], z[P], i[P], h[P];
    layer::unpack<T, V>(rx, x);
    layer::unpack<T, V>(rz, z);
    if (A.input_gate) layer::unpack<T, V>(ri, i);
    layer::unpack<float, V>(rs, h);
#pragma unroll
    for (int k = 0; k < P; ++k) {
        F zk[1] = {z[k]}, xk[1] = {x[k]}, ik[1] = {i[k]};
        log_decays(S, C[k], zk);
        const decay<F> d = decay_of(zk[0]);
        const F m[1] = {d.m};
        scale_inputs(S, m, xk);
        if (A.input_gate) gate_inputs(ik, xk);
        h[k] = step_any(d.d, h[k], xk[0]);
    }
    layer::store(state, layer::pack<float, V>(h));
    layer::store((T *)A.h + n * A.D + c, layer::pack<T, V>(h));
}

template <typename T, int V>
static void launch(const kda_scan_step_args *a, cudaStream_t stream, int *err) {
    const int per = 128 * V;
    scan_step_kernel<T, V><<<dim3((unsigned)a->N, (a->D + per - 1) / per), 128, 0, stream>>>(*a, err);
}

template <typename T>
static void launch_t(const kda_scan_step_args *a, cudaStream_t stream, int *err) {
    // Four channels a thread where every row's address allows vectors of them (256 sequences of 4096 channels, bf16: two
    // thirds of the time one by one)
    const uintptr_t tok = (uintptr_t)a->x | (uintptr_t)a->z | (uintptr_t)a->input_gate | (uintptr_t)a->h;
    const bool wide = a->D % 4 == 0 && a->x_stride % 4 == 0 && a->z_stride % 4 == 0 && a->i_stride % 4 == 0 && tok % (4 * sizeof(T)) == 0 &&
                      (uintptr_t)a->state % 16 == 0;
    if (wide) launch<T, 4>(a, stream, err);
    else launch<T, 1>(a, stream, err);
}

}  // namespace scan
}  // namespace kda

kda_status_t kda_launch_scan_step(const kda_scan_step_args *a, cudaStream_t stream) {
    int *err = kda_device_error_ptr();
    if (!err) return KDA_ERR_CUDA;
    if (a->dtype == KDA_BF16) kda::scan::launch_t<kda::bf16>(a, stream, err);
    else kda::scan::launch_t<float>(a, stream, err);
    return kda_cuda_status(cudaGetLastError());
}
