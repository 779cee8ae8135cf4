// kda_scan_step: one decode token per sequence of the gated recurrence over channels, states updated in place.
//
// Bound by HBM traffic (bf16 with an input gate: 8 bytes of tokens and 8 of state per channel), for few sequences by the
// launch.  A thread takes V channels of one sequence.
#include "kda_internal.h"
#include "kda_layer.cuh"
#include "kda_scan.cuh"

namespace kda {
namespace scan {

template <typename T, int V>
__global__ void __launch_bounds__(128) scan_step_kernel(const __grid_constant__ kda_scan_step_args A, int *err) {
    const int c = (blockIdx.x * 128 + threadIdx.x) * V;
    const int64_t n = blockIdx.y;
    int64_t slot;
    if (!layer::find_slot<128>(A.state_indices, A.num_slots, n, &slot, err) || c >= A.D) return;
    const spec S{A.gate_kind, A.input_scale, A.g_min};
    layer::vec<T, V> x, z, i, h;
    layer::vec<float, V> s;
    float *state = A.state + slot * A.D + c;
    x = layer::load<T, V>((const T *)A.x + n * A.x_stride + c);
    z = layer::load<T, V>((const T *)A.z + n * A.z_stride + c);
    if (A.input_gate) i = layer::load<T, V>((const T *)A.input_gate + n * A.i_stride + c);
    s = layer::load<float, V>(state);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const channel C = load_channel(A.A_log, A.dt_bias, c + e);
        const decay d = decay_of(log_decay(S, C, ld(&z.x[e])));
        s.x[e] = decayed(d.d, s.x[e]) + entering(S, d.m, ld(&x.x[e]), A.input_gate != nullptr, A.input_gate ? ld(&i.x[e]) : 0.f);
        st(&h.x[e], s.x[e]);
    }
    layer::store(state, s);
    layer::store((T *)A.h + n * A.D + c, h);
}

template <typename T, int V>
static void launch(const kda_scan_step_args *a, cudaStream_t stream, int *err) {
    const int per = 128 * V;
    scan_step_kernel<T, V><<<dim3((a->D + per - 1) / per, (unsigned)a->N), 128, 0, stream>>>(*a, err);
}

template <typename T>
static void launch_t(const kda_scan_step_args *a, cudaStream_t stream, int *err) {
    launch<T, 1>(a, stream, err);
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
