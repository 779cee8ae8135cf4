// kda_scan_fwd: a block takes a tile of 64 tokens by 32 V channels (kda_scan_tiles.cuh), each of its eight warps 8
// tokens, each lane V channels.  A thread forms the decay and the input of its elements once, keeps both in registers,
// runs them from zero for the tile's sums, and, when it knows what enters them, runs them again for h.
#include "kda_internal.h"
#include "kda_layer.cuh"
#include "kda_scan_tiles.cuh"

namespace kda {
namespace scan {

template <typename T, int V>
__global__ void __launch_bounds__(NT, 2) scan_fwd_kernel(const __grid_constant__ kda_scan_args A, const __grid_constant__ board B, bool joined,
                                                         int blocks, int *err) {
    constexpr int W = 32 * V;
    __shared__ tile_memory<W> M;
    if (!take_tile(B, joined, A.cu_seqlens, A.T, A.N, blocks, M, err)) return;
    tile t = M.t;
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32, c0 = t.block * W, c = c0 + lane * V;
    const bool mine = c < A.D;
    const spec S{A.gate_kind, A.input_scale, A.g_min};
    channel C[V];
#pragma unroll
    for (int v = 0; v < V; ++v) C[v] = mine ? load_channel(A.A_log, A.dt_bias, c + v) : channel{0.f, 0.f};
    for (;; ++t.p) {
        const int64_t tok = t.s.a + t.p * L + w * R;
        const int len = (int)(t.s.b - tok < R ? t.s.b - tok : R);  // of this warp; below 1 where it has none
        layer::vec<T, V> x[R], z[R], i[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (mine && r < len) {
                z[r] = layer::load_once<T, V>((const T *)A.z + (tok + r) * A.z_stride + c);
                x[r] = layer::load_once<T, V>((const T *)A.x + (tok + r) * A.x_stride + c);
                if (A.input_gate) i[r] = layer::load_once<T, V>((const T *)A.input_gate + (tok + r) * A.i_stride + c);
            }
        float d[R][V], u[R][V], sum[V] = {}, h[V] = {};
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                d[r][v] = 1.f;
                u[r][v] = 0.f;
            }
            if (mine && r < len) {
                float fz[V], fx[V], fi[V];
                layer::unpack<T, V>(z[r], fz);
                layer::unpack<T, V>(x[r], fx);
                if (A.input_gate) layer::unpack<T, V>(i[r], fi);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float g = log_decay(S, C[v], fz[v]);
                    const decay e = decay_of(g);
                    sum[v] += g;
                    d[r][v] = e.d;
                    u[r][v] = entering(S, e.m, fx[v], A.input_gate != nullptr, fi[v]);
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = decayed(d[r][v], h[v]) + u[r][v];
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            M.g[w][lane * V + v] = sum[v];
            M.d[w][lane * V + v] = decay_of(sum[v]).d;
            M.b[w][lane * V + v] = h[v];
        }
        join<W>(B, joined, t, c0, A.D, A.initial_state, M, err);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int ch = lane * V + v;
            h[v] = decayed(M.run_d[ch], M.from[ch]) + M.run_b[ch];
        }
        if (A.checkpoints && w == 0 && mine && t.count > 0)
#pragma unroll
            for (int v = 0; v < V; ++v) A.checkpoints[(t.first + t.p) * A.D + c + v] = h[v];
#pragma unroll
        for (int k = 0; k < NW - 1; ++k)
            if (k < w)
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = decayed(M.d[k][lane * V + v], h[v]) + M.b[k][lane * V + v];
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = decayed(d[r][v], h[v]) + u[r][v];
            if (mine && r < len) layer::store_once((T *)A.h + (tok + r) * A.D + c, layer::pack<T, V>(h));
        }
        if (t.serial) __syncthreads();  // M.from has been read
        if (w == NW - 1) {
            if (A.final_state && mine && t.p + 1 >= t.count)
#pragma unroll
                for (int v = 0; v < V; ++v) A.final_state[t.n * A.D + c + v] = h[v];
            leave<W, V>(B, joined, t, c0, A.D, h, M);
        }
        if (!t.serial || t.p + 1 >= t.count) return;
        __syncthreads();
    }
}

template <typename T, int V>
static void launch(const kda_scan_args *a, void *ws, cudaStream_t stream, int *err) {
    const int W = 32 * V, blocks = (a->D + W - 1) / W;
    const int64_t slots = lin::chunk_slots(a->T, a->N, L);
    board B{};
    const bool joined = board_layout(a->T, a->N, a->D, W, ws, &B) > 0;
    if (joined)
        scan_clear_kernel<<<(unsigned)((B.control_words + 2047) / 2048), 256, 0, stream>>>(B.control, B.control_words, a->cu_seqlens, a->T, a->N, err);
    scan_fwd_kernel<T, V><<<(unsigned)(slots * blocks), NT, 0, stream>>>(*a, B, joined, blocks, err);
}

}  // namespace scan
}  // namespace kda

size_t kda_scan_fwd_bytes(int64_t T, int64_t N, int D) { return kda::scan::board_layout(T, N, D, 32, nullptr, nullptr); }

kda_status_t kda_launch_scan_fwd(const kda_scan_args *a, void *ws, cudaStream_t stream) {
    int *err = kda_device_error_ptr();
    if (!err) return KDA_ERR_CUDA;
    using namespace kda::scan;
    // 8 bytes a lane where every row's address allows it
    auto wide = [&](int V) {
        const uintptr_t bytes = V * (a->dtype == KDA_BF16 ? 2 : 4);
        return a->D % V == 0 && a->x_stride % V == 0 && a->z_stride % V == 0 && a->i_stride % V == 0 &&
               (((uintptr_t)a->x | (uintptr_t)a->z | (uintptr_t)a->input_gate | (uintptr_t)a->h) % bytes) == 0;
    };
    if (a->dtype == KDA_BF16) wide(4) ? launch<kda::bf16, 4>(a, ws, stream, err) : launch<kda::bf16, 1>(a, ws, stream, err);
    else wide(2) ? launch<float, 2>(a, ws, stream, err) : launch<float, 1>(a, ws, stream, err);
    return kda_cuda_status(cudaGetLastError());
}
