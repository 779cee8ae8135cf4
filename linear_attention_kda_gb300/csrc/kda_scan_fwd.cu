// kda_scan_fwd: a block takes tiles of L tokens by 64 channels (kda_scan_tiles.cuh), each of its eight warps L / 8 tokens,
// each lane two channels.  Tiles come by TMA two ahead.  A thread forms the decay and the input of its elements once,
// keeps both in registers, runs them from zero for the tile's sums, and, when it knows what enters, runs them again for h.
#include "kda_scan_tiles.cuh"

namespace kda {
namespace scan {

// Tokens of a tile: a long one shares the cost of joining, its inputs twice and d and u have to fit.
template <typename T> constexpr int fwd_tile = sizeof(T) == 2 ? 128 : 64;

template <typename T> struct fwd_memory {
    ring<T, 3, fwd_tile<T>> next;
    tile_memory M;
};

// TMA: rows are 16-byte aligned.  Else a thread reads its elements when it needs them.
template <typename T, bool TMA>
__global__ void __launch_bounds__(NT, 2)
scan_fwd_kernel(const __grid_constant__ kda_scan_args A, const __grid_constant__ board B, const __grid_constant__ row_maps<3> maps, int joined,
                int blocks, int *err) {
    constexpr int L = fwd_tile<T>, R = L / NW;
    extern __shared__ __align__(128) char memory[];
    fwd_memory<T> &S = *reinterpret_cast<fwd_memory<T> *>(memory);
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const spec K{A.gate_kind, A.input_scale, A.g_min};
    const bool gated = A.input_gate != nullptr;
    if (joined) make_plan(B, A.cu_seqlens, A.T, A.N, blocks, err);
    const bool chains = joined && __ldcg(B.mode) != 0, loader = w == NW - 1;
    course<L> way(B, A.cu_seqlens, A.T, A.N, blocks, joined, false);
    // the next tile of the course, its boxes asked for
    auto ask = [&](int stage) {
        way.next();
        if (lane != 0) return;
        S.next.t[stage] = way.t;
        if (!TMA || way.t.p < 0) return;
        const int tok = way.t.a + way.t.p * L, n = gated ? 3 : 2;
        tc::fence_proxy_async();  // (join() has written to the stage)
        tc::mbar_arrive_expect_tx(&S.next.full[stage], (uint32_t)(n * L * W * sizeof(T)));
        for (int i = 0; i < n; ++i) tc::tma_load_3d(&S.next.x[stage][i][0][0], &maps.m[i], way.t.block * W, 0, tok, &S.next.full[stage]);
    };
    if (TMA && threadIdx.x == 0) {
        tc::mbar_init(&S.next.full[0], 1);
        tc::mbar_init(&S.next.full[1], 1);
        tc::fence_proxy_async();
    }
    __syncthreads();
    if (loader) {
        ask(0);
        ask(1);
    }
    __syncthreads();
    channel<float2> C{};
    int of = -1;  // the block of channels whose parameters C holds
    for (int turn = 0;; ++turn) {
        const tile t = S.next.t[turn & 1];
        if (t.p < 0) break;
        const int tok = t.a + t.p * L + w * R, len = t.b - tok < R ? t.b - tok : R;  // tokens of this warp, below 1 where it has none
        const int c = t.block * W + lane * 2, have = A.D - c;
        if (of != t.block) C = load_channel(A.A_log, A.dt_bias, c, have);
        of = t.block;
        const int stage = turn & 1;
        if (TMA && !tc::mbar_wait(&S.next.full[stage], (turn >> 1) & 1)) set_error(err, KDA_ERR_DEVICE_TIMEOUT);
        float2 u[R], d[R], sum = make_float2(0.f, 0.f), h = sum;
        // PART tokens at a time, so that their logits fit beside d and u
        constexpr int PART = 8;
#pragma unroll
        for (int r0 = 0; r0 < R; r0 += PART) {
            auto get = [&](int k, const void *p, int64_t stride, float2 (&f)[PART]) {
#pragma unroll
                for (int r = 0; r < PART; ++r)  // (by TMA there are rows of other sequences behind the last token)
                    f[r] = TMA ? load_pair<T, true>(&S.next.x[stage][k][w * R + r0 + r][lane * 2], 2)
                               : load_pair<T, false>((const T *)p + (int64_t)(tok + r0 + r) * stride + c, r0 + r < len ? have : 0);
            };
            float2 z[PART], x[PART];
            get(0, A.z, A.z_stride, z);
            log_decays(K, C, z);
            if (len < r0 + PART) {
#pragma unroll
                for (int r = 0; r < PART; ++r)
                    if (r0 + r >= len) z[r] = make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int r = 0; r < PART; ++r) {
                const decay<float2> e = decay_of(z[r]);
                sum = add(sum, z[r]);
                d[r0 + r] = e.d;
                z[r] = e.m;
            }
            get(1, A.x, A.x_stride, x);
            scale_inputs(K, z, x);
            if (gated) {
                get(2, A.input_gate, A.i_stride, z);
                gate_inputs(z, x);
            }
#pragma unroll
            for (int r = 0; r < PART; ++r) u[r0 + r] = x[r];
        }
        if (len < R) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r >= len) u[r] = make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) h = step(d[r], h, u[r]);
        *reinterpret_cast<float2 *>(&S.M.g[w][lane * 2]) = sum;
        *reinterpret_cast<float2 *>(&S.M.d[w][lane * 2]) = decay_of(sum).d;
        *reinterpret_cast<float2 *>(&S.M.b[w][lane * 2]) = h;
        join<R, false>(B, joined && !chains, t, A.D, A.initial_state, A.final_state,
                A.checkpoints ? A.checkpoints + ((int64_t)t.a / CK + t.n + t.p * (L / CK)) * A.D : nullptr, (t.b - t.a - t.p * L + CK - 1) / CK, S.M,
                *reinterpret_cast<entries *>(&S.next.x[stage]), err, [](int, int) {});
        if (loader) ask(stage);  // every warp is done with this stage
        h = *reinterpret_cast<const float2 *>(&S.M.g[w][lane * 2]);
        // what enters may be an infinity or a NaN, which a decay of 0 erases
        const bool odd = __any_sync(0xffffffffu, !finite(h));
        T *out = (T *)A.h + (int64_t)tok * A.D + c;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (odd) h = each([](float v, float s) { return v == 0.f ? 0.f : s; }, d[r], h);
            h = step(d[r], h, u[r]);
            if (r < len && have > 0) store_pair<T, TMA>(out, h, have);
            out += A.D;
        }
    }
    if (!joined) check_all(A.cu_seqlens, A.T, A.N, err);
}

template <typename T, bool TMA>
static cudaError_t launch(const kda_scan_args *a, const row_maps<3> &maps, void *ws, cudaStream_t stream, int *err) {
    static std::atomic<int> running[64];
    constexpr size_t smem = sizeof(fwd_memory<T>);
    int blocks = (a->D + W - 1) / W, grid = 0;
    const int64_t tiles = lin::chunk_slots(a->T, a->N, fwd_tile<T>) * blocks;
    board B{};
    int joined = a->T > fwd_tile<T>;  // else no sequence has a second tile
    if (joined) board_layout(a->T, a->N, a->D, fwd_tile<T>, ws, &B);
    const cudaError_t e = running_blocks(scan_fwd_kernel<T, TMA>, smem, running, tiles, &grid);
    if (e != cudaSuccess) return e;
    if (!joined) {
        scan_fwd_kernel<T, TMA><<<grid, NT, smem, stream>>>(*a, B, maps, 0, blocks, err);
        return cudaGetLastError();
    }
    kda_scan_args args = *a;
    row_maps<3> m = maps;
    void *p[] = {&args, &B, &m, &joined, &blocks, &err};
    return cudaLaunchCooperativeKernel((const void *)scan_fwd_kernel<T, TMA>, dim3(grid), dim3(NT), p, smem, stream);
}

}  // namespace scan
}  // namespace kda

size_t kda_scan_fwd_bytes(int64_t T, int64_t N, int D, kda_dtype_t dtype) {
    using namespace kda::scan;
    const int L = dtype == KDA_BF16 ? fwd_tile<kda::bf16> : fwd_tile<float>;
    return T > L ? board_layout(T, N, D, L, nullptr, nullptr) : 0;
}

kda_status_t kda_launch_scan_fwd(const kda_scan_args *a, void *ws, cudaStream_t stream) {
    int *err = kda_device_error_ptr();
    if (!err) return KDA_ERR_CUDA;
    using namespace kda::scan;
    row_maps<3> maps{};
    const int64_t es = a->dtype == KDA_BF16 ? 2 : 4, per = 16 / es;
    const int L = a->dtype == KDA_BF16 ? fwd_tile<kda::bf16> : fwd_tile<float>;
    const bool tma = a->T > 0 && a->D % 2 == 0 && (uintptr_t)a->h % (2 * es) == 0 &&
                     (((uintptr_t)a->x | (uintptr_t)a->z | (uintptr_t)a->input_gate) & 15) == 0 && a->x_stride % per == 0 &&
                     a->z_stride % per == 0 && (!a->input_gate || a->i_stride % per == 0);
    if (tma && (!make_row_map(&maps.m[0], a->z, a->T, a->D, a->z_stride, a->dtype, L) || !make_row_map(&maps.m[1], a->x, a->T, a->D, a->x_stride, a->dtype, L) ||
                (a->input_gate && !make_row_map(&maps.m[2], a->input_gate, a->T, a->D, a->i_stride, a->dtype, L))))
        return KDA_ERR_CUDA;
    if (a->dtype == KDA_BF16)
        return kda_cuda_status(tma ? launch<kda::bf16, true>(a, maps, ws, stream, err) : launch<kda::bf16, false>(a, maps, ws, stream, err));
    return kda_cuda_status(tma ? launch<float, true>(a, maps, ws, stream, err) : launch<float, false>(a, maps, ws, stream, err));
}
