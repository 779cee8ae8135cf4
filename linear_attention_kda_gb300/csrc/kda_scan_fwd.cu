// kda_scan_fwd: a block takes tiles of 64 tokens by 32 V channels (kda_scan_tiles.cuh), each of its eight warps 8
// tokens, each lane V channels.  A thread forms the decay and the input of its elements once, keeps both in registers,
// runs them from zero for the tile's sums, asks for its elements of the next tile, and, when it knows what enters, runs
// them again for h.
#include "kda_scan_tiles.cuh"

namespace kda {
namespace scan {

template <typename T, int V>
__global__ void __launch_bounds__(NT, 2) scan_fwd_kernel(const __grid_constant__ kda_scan_args A, const __grid_constant__ board B, int joined,
                                                         int blocks, int *err) {
    constexpr int W = 32 * V, P = layer::lanes<V>::N;
    using F = typename layer::lanes<V>::F;
    extern __shared__ __align__(16) char memory[];
    tile_memory<W> &M = *reinterpret_cast<tile_memory<W> *>(memory);
    ahead<T, V, 3> &next = *reinterpret_cast<ahead<T, V, 3> *>(memory + sizeof(tile_memory<W>));
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const spec S{A.gate_kind, A.input_scale, A.g_min};
    const bool gated = A.input_gate != nullptr;
    const bool serial = joined && __ldcg(B.bad) != 0;
    const int64_t items = serial ? A.N * blocks : lin::chunk_slots(A.T, A.N, L) * blocks;

    // the tile of an item; p = -1: none
    auto take = [&](int64_t item) {
        tile t{0, -1, 0, 0, 0, 0};
        if (item >= items) return t;
        t.block = (int)(item % blocks);
        const int64_t i = item / blocks;
        if (joined && !serial) {
            const int4 q = __ldg(B.plan + i);
            t.n = q.x, t.p = q.y, t.a = q.z, t.b = q.w;
        } else {
            int64_t n = i, p = 0;
            lin::span s;
            if (serial ? lin::seq_span(A.cu_seqlens, A.T, A.N, n, &s) : lin::find_slot(A.cu_seqlens, A.T, A.N, L, i, &n, &p, &s)) {
                if (p == 0 || p < (s.b - s.a + L - 1) / L) t.p = (int)p;
                t.n = (int)n, t.a = (int)s.a, t.b = (int)s.b;
            }
        }
        t.count = (t.b - t.a + L - 1) / L;
        return t;
    };
    auto ask = [&](const tile &t) {
        const int64_t tok = t.a + (int64_t)t.p * L + w * R;
        const int c = t.block * W + lane * V;
        if (t.p < 0 || c >= A.D) return;
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (tok + r < t.b) {
                next.ask(r, 0, (const T *)A.z + (tok + r) * A.z_stride + c);
                next.ask(r, 1, (const T *)A.x + (tok + r) * A.x_stride + c);
                if (gated) next.ask(r, 2, (const T *)A.input_gate + (tok + r) * A.i_stride + c);
            }
    };

    int64_t item = blockIdx.x;
    tile t = take(item);
    ask(t);
    channel<F> C[P];
    int of = -1;  // the block of channels whose parameters C holds
    while (item < items) {
        if (t.p < 0) {
            t = take(item += gridDim.x);
            ask(t);
            continue;
        }
        const int64_t tok = t.a + (int64_t)t.p * L + w * R;
        const int len = (int)(t.b - tok < R ? t.b - tok : R), c = t.block * W + lane * V;  // tokens of this warp, below 1 where it has none
        const bool mine = c < A.D;
        if (of != t.block) load_channels<V>(A.A_log, A.dt_bias, c, mine, C);
        of = t.block;
        tile then = t;  // the tile after this one
        int64_t after = item;
        if (serial && t.p + 1 < t.count) ++then.p;
        else then = take(after += gridDim.x);
        cp_async_wait_all();
        F d[R][P], u[R][P], sum[P], h[P], whole[P];
#pragma unroll
        for (int i = 0; i < P; ++i) sum[i] = h[i] = splat<F>(0.f);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (mine && r < len) {
                F z[P], x[P], g[P];
                layer::unpack<T, V>(next.x[r][0][threadIdx.x], z);
                layer::unpack<T, V>(next.x[r][1][threadIdx.x], x);
                if (gated) layer::unpack<T, V>(next.x[r][2][threadIdx.x], g);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const F k = log_decay(S, C[i], z[i]);
                    const decay<F> e = decay_of(k);
                    sum[i] = add(sum[i], k);
                    d[r][i] = e.d;
                    u[r][i] = entering(S, e.m, x[i], gated, g[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    d[r][i] = splat<F>(1.f);
                    u[r][i] = splat<F>(0.f);
                }
            }
#pragma unroll
            for (int i = 0; i < P; ++i) h[i] = step(d[r][i], h[i], u[r][i]);
        }
        ask(then);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int at = lane * V + i * layer::lanes<V>::K;
            *reinterpret_cast<F *>(&M.g[w][at]) = sum[i];
            *reinterpret_cast<F *>(&M.d[w][at]) = decay_of(sum[i]).d;
            *reinterpret_cast<F *>(&M.b[w][at]) = h[i];
        }
        join<W>(B, joined && !serial, serial && t.p > 0, t, A.D, A.initial_state, M, err);
        enter<W, V>(M, w, lane, h, whole);
        if (A.checkpoints && w == 0 && mine && t.count > 0)
#pragma unroll
            for (int v = 0; v < V; ++v) A.checkpoints[((int64_t)t.first() + t.p) * A.D + c + v] = reinterpret_cast<const float *>(whole)[v];
        // what enters may be an infinity or a NaN, which a decay of 0 erases
        bool odd = false;
#pragma unroll
        for (int i = 0; i < P; ++i) odd |= !finite(h[i]);
        odd = __any_sync(0xffffffffu, odd);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (odd) {
#pragma unroll
                for (int i = 0; i < P; ++i) h[i] = each([](float v, float s) { return v == 0.f ? 0.f : s; }, d[r][i], h[i]);
            }
#pragma unroll
            for (int i = 0; i < P; ++i) h[i] = step(d[r][i], h[i], u[r][i]);
            if (mine && r < len) layer::store_once((T *)A.h + (tok + r) * A.D + c, layer::pack<T, V>(h));
        }
        if (serial) __syncthreads();  // M.from has been read
        if (w == NW - 1) {
            const float *last = reinterpret_cast<const float *>(h);
            if (A.final_state && mine && t.p + 1 >= t.count)
#pragma unroll
                for (int v = 0; v < V; ++v) A.final_state[(int64_t)t.n * A.D + c + v] = last[v];
            if (serial)
#pragma unroll
                for (int v = 0; v < V; ++v) M.from[lane * V + v] = last[v];
            else if (joined)
                leave<W, V>(B, t, lane, A.D, h);
        }
        t = then;
        item = after;
    }
    if (!joined && blockIdx.x == 0)
        for (int64_t n = threadIdx.x; n < A.N; n += NT) {
            lin::span s;
            if (!lin::seq_span(A.cu_seqlens, A.T, A.N, n, &s)) set_error(err, KDA_ERR_BAD_SEQLENS);
        }
}

template <typename T, int V>
static cudaError_t launch(const kda_scan_args *a, void *ws, cudaStream_t stream, int *err) {
    static std::atomic<int> running[64];
    constexpr size_t smem = sizeof(tile_memory<32 * V>) + sizeof(ahead<T, V, 3>);
    int blocks = (a->D + 32 * V - 1) / (32 * V), grid = 0;
    const int64_t tiles = lin::chunk_slots(a->T, a->N, L) * blocks;
    board B{};
    int joined = board_layout(a->T, a->N, a->D, 32 * V, ws, &B) > 0;
    const cudaError_t e = running_blocks(scan_fwd_kernel<T, V>, smem, running, tiles, &grid);
    if (e != cudaSuccess) return e;
    if (!joined) {
        scan_fwd_kernel<T, V><<<grid, NT, smem, stream>>>(*a, B, 0, blocks, err);
        return cudaGetLastError();
    }
    launch_plan(B, a->cu_seqlens, a->T, a->N, stream, err);
    kda_scan_args args = *a;
    void *p[] = {&args, &B, &joined, &blocks, &err};
    return cudaLaunchCooperativeKernel((const void *)scan_fwd_kernel<T, V>, dim3(grid), dim3(NT), p, smem, stream);
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
    if (a->dtype == KDA_BF16) return kda_cuda_status(wide(4) ? launch<kda::bf16, 4>(a, ws, stream, err) : launch<kda::bf16, 1>(a, ws, stream, err));
    return kda_cuda_status(wide(2) ? launch<float, 2>(a, ws, stream, err) : launch<float, 1>(a, ws, stream, err));
}
