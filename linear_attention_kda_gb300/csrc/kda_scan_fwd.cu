// kda_scan_fwd: a block takes tiles of L tokens by W channels (kda_scan_tiles.cuh), each of its eight warps L / 8 tokens,
// each lane two channels and R of them.  Tiles come by TMA two ahead.  A thread forms the decay and the input of its elements once,
// keeps both in registers, runs them from zero for the tile's sums, and, when it knows what enters, runs them again for h.
//
// Bound by instructions and by the two barriers of a tile: 45 instructions an element (softplus, c of the norm, gated; 5 of the special function
// unit, 12 of the integer and selecting pipe, 21 multiply-adds), issued in 59 % of the cycles, where all cycles at HBM's rate would hold
// 42.  bf16, gated, D = 4096: 32 sequences of 512 to 8192 tokens 1003 us, 4.3 TB/s (a thread to a channel of a sequence, a token at a time,
// 9110); 16 such sequences in fp32 763 us, 6.4 TB/s; one sequence of 4096 tokens 47 us.  131072 tokens of 256 channels 104 us, bound by tiles that
// wait for one another (issued in 33 % of the cycles).
#include "kda_scan_tiles.cuh"

namespace kda {
namespace scan {

// Many tokens a thread share the cost of joining; the tile's inputs twice (in shared memory) and d and u have to fit.
template <typename T, int W> using fwd_shape = shape<W, sizeof(T) == 2 ? 16 : 8>;

template <typename T, int W> struct fwd_memory {
    ring<T, 3, fwd_shape<T, W>> next;
    tile_memory<W> M;
};

// The tokens of a thread by step_any() from h on, read again from memory: what a tile does in which infinities or NaN are found, out of the
// way of the others, whose decays and inputs stay in registers.  *sum: of the log-decays; STORE: leaves the states.
template <typename T, bool STORE>
static __device__ __noinline__ float2 run_any(const kda_scan_args &A, int tok, int len, int c, float2 h, float2 *sum) {
    const int have = A.D - c;
    const spec K{A.gate_kind, A.input_scale, A.g_min};
    const channel<float2> C = load_channel(A.A_log, A.dt_bias, c, have);
    *sum = make_float2(0.f, 0.f);
    for (int64_t t = tok; t < tok + len; ++t) {
        float2 z[1] = {load_pair<T, false>((const T *)A.z + t * A.z_stride + c, have)}, x[1] = {load_pair<T, false>((const T *)A.x + t * A.x_stride + c, have)};
        log_decays(K, C, z);
        const decay<float2> e = decay_of(z[0]);
        *sum = add(*sum, z[0]);
        z[0] = e.m;
        scale_inputs(K, z, x);
        if (A.input_gate) {
            z[0] = load_pair<T, false>((const T *)A.input_gate + t * A.i_stride + c, have);
            gate_inputs(z, x);
        }
        h = step_any(e.d, h, x[0]);
        if (STORE) store_pair<T, false>((T *)A.h + t * A.D + c, h, have);
    }
    return h;
}

// TMA: rows are 16-byte aligned.  Else a thread reads its elements when it needs them.  PLAN: make_plan() says what the tiles are (a
// kernel of its own for the others: one for all was 2 to 8 % slower where tiles join).
template <typename T, int W, bool TMA, bool PLAN>
__global__ void __launch_bounds__(NT, 2)
scan_fwd_kernel(const __grid_constant__ kda_scan_args A, const __grid_constant__ board B, const __grid_constant__ row_maps<3> maps, layout how,
                int blocks, int *err) {
    using X = fwd_shape<T, W>;
    constexpr int L = X::L, R = X::R;
    extern __shared__ __align__(128) char memory[];
    fwd_memory<T, W> &S = *reinterpret_cast<fwd_memory<T, W> *>(memory);
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32, pair = lane % X::LPR * 2, row0 = w * X::RW + lane / X::LPR * R;
    const spec K{A.gate_kind, A.input_scale, A.g_min};
    const bool gated = A.input_gate != nullptr;
    if (PLAN) make_plan(B, A.cu_seqlens, A.T, A.N, A.D, blocks, err);
    const bool links = PLAN && !planned_chains(B), loader = w == NW - 1;
    course<L, PLAN> way(B, S.next.way, A.cu_seqlens, A.T, A.N, blocks, how, false);
    // the next tile of the course, its boxes asked for
    auto ask = [&](int stage) {
        const tile t = way.next();
        if (lane != 0) return;
        S.next.t[stage] = t;
        if (!TMA || t.p < 0) return;
        const int tok = t.a + t.p * L, n = gated ? 3 : 2;
        tc::fence_proxy_async();  // (join() has written to the stage)
        tc::mbar_arrive_expect_tx(&S.next.full[stage], (uint32_t)(n * L * W * sizeof(T)));
        for (int i = 0; i < n; ++i) load_rows<X>(&S.next.x[stage][i][0][0], maps.m[i], t.block, tok, &S.next.full[stage]);
    };
    if (threadIdx.x == 0) S.M.odd = 0;
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
        const int tok = t.a + t.p * L + row0, len = t.b - tok < R ? t.b - tok : R;  // tokens of this thread, below 1 where it has none
        const int c = t.block * W + pair, have = A.D - c;
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
                    f[r] = TMA ? load_pair<T, true>(&S.next.x[stage][k][row0 + r0 + r][pair], 2)
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
        if (!finite(h)) S.M.odd = turn + 1;
        float2 before_sum, before;
        over_groups<X, false, false>(sum, h, before_sum, before);
        if (lane >= 32 - X::LPR) {
            *reinterpret_cast<float2 *>(&S.M.g[w][pair]) = sum;
            *reinterpret_cast<float2 *>(&S.M.d[w][pair]) = decay_of(sum).d;
            *reinterpret_cast<float2 *>(&S.M.b[w][pair]) = h;
        }
        const bool odd = join<X, false>(
            B, links, t, A.D, A.initial_state, A.final_state,
            A.checkpoints ? A.checkpoints + ((int64_t)t.a / CK + t.n + t.p * (L / CK)) * A.D : nullptr,
            (t.b - t.a - t.p * L + CK - 1) / CK, S.M, *reinterpret_cast<entries<W> *>(&S.next.x[stage]), turn + 1, err, [](int, int) {},
            [&] {
                float2 s, v = run_any<T, false>(A, tok, len, c, make_float2(0.f, 0.f), &s);
                over_groups<X, false, true>(s, v, before_sum, before);
                if (lane >= 32 - X::LPR) *reinterpret_cast<float2 *>(&S.M.b[w][pair]) = v;
            });
        if (loader) ask(stage);  // every warp is done with this stage
        const float2 enters = *reinterpret_cast<const float2 *>(&S.M.g[w][pair]);
        h = group_entry<X, false>(enters, before_sum, before);
        if (__any_sync(0xffffffffu, odd || !finite(h))) {
            float2 s;
            run_any<T, true>(A, tok, len, c, group_entry<X, true>(enters, before_sum, before), &s);
            continue;
        }
        // (what the first pass made of the decays is not kept for the second: registers)
#pragma unroll
        for (int r = 0; r < R; ++r) asm("" : "+f"(d[r].x), "+f"(d[r].y));
        T *out = (T *)A.h + (int64_t)tok * A.D + c;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            h = step(d[r], h, u[r]);
            if (r < len && have > 0) store_pair<T, TMA>(out, h, have);
            out += A.D;
        }
    }
    if (!PLAN) check_all(A.cu_seqlens, A.T, A.N, err);
}

template <typename T, int W, bool TMA>
static cudaError_t launch(const kda_scan_args *a, void *ws, cudaStream_t stream, int *err) {
    using X = fwd_shape<T, W>;
    static std::atomic<int> running[2][64];
    constexpr size_t smem = sizeof(fwd_memory<T, W>);
    row_maps<3> maps{};
    if (TMA && (!make_row_map<X>(&maps.m[0], a->z, a->T, a->D, a->z_stride, a->dtype) ||
                !make_row_map<X>(&maps.m[1], a->x, a->T, a->D, a->x_stride, a->dtype) ||
                (a->input_gate && !make_row_map<X>(&maps.m[2], a->input_gate, a->T, a->D, a->i_stride, a->dtype))))
        return cudaErrorUnknown;
    int blocks = (a->D + W - 1) / W, grid = 0;
    board B{};
    layout how = SINGLE;
    kda_scan_args args = *a;
    void *p[] = {&args, &B, &maps, &how, &blocks, &err};
    cudaError_t e = running_blocks(scan_fwd_kernel<T, W, TMA, false>, smem, running[0], lin::chunk_slots(a->T, a->N, X::L) * blocks, &grid);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (a->T / a->N + X::L - 1) / X::L;  // of a sequence, where they are alike
    if (a->T > X::L) how = (!a->cu_seqlens || a->N == 1) && rather_whole(tiles, tiles * a->N, blocks, grid) ? EQUAL : PLANNED;
    if (how != PLANNED) return cudaLaunchKernel((const void *)scan_fwd_kernel<T, W, TMA, false>, dim3(grid), dim3(NT), p, smem, stream);
    e = running_blocks(scan_fwd_kernel<T, W, TMA, true>, smem, running[1], lin::chunk_slots(a->T, a->N, X::L) * blocks, &grid);
    if (e != cudaSuccess) return e;
    board_layout(a->T, a->N, a->D, X::L, ws, &B);
    return cudaLaunchCooperativeKernel((const void *)scan_fwd_kernel<T, W, TMA, true>, dim3(grid), dim3(NT), p, smem, stream);
}

template <typename T> static cudaError_t choose(const kda_scan_args *a, void *ws, cudaStream_t stream, int *err) {
    const int64_t es = sizeof(T), per = 16 / es;
    const bool tma = a->T > 0 && a->D % 2 == 0 && (uintptr_t)a->h % (2 * es) == 0 &&
                     (((uintptr_t)a->x | (uintptr_t)a->z | (uintptr_t)a->input_gate) & 15) == 0 && a->x_stride % per == 0 &&
                     a->z_stride % per == 0 && (!a->input_gate || a->i_stride % per == 0);
    // (by element alignment alone the same tiles are taken, so that the results are the same)
    switch (tile_width(a->N, a->D)) {
        case 16: return tma ? launch<T, 16, true>(a, ws, stream, err) : launch<T, 16, false>(a, ws, stream, err);
        case 32: return tma ? launch<T, 32, true>(a, ws, stream, err) : launch<T, 32, false>(a, ws, stream, err);
        default: return tma ? launch<T, 64, true>(a, ws, stream, err) : launch<T, 64, false>(a, ws, stream, err);
    }
}

}  // namespace scan
}  // namespace kda

size_t kda_scan_fwd_bytes(int64_t T, int64_t N, int D, kda_dtype_t dtype) {
    using namespace kda::scan;
    // (the shortest tile's, which holds all)
    const int L = dtype == KDA_BF16 ? fwd_shape<kda::bf16, 64>::L : fwd_shape<float, 64>::L;
    return T > L ? board_layout(T, N, D, L, nullptr, nullptr) : 0;
}

kda_status_t kda_launch_scan_fwd(const kda_scan_args *a, void *ws, cudaStream_t stream) {
    int *err = kda_device_error_ptr();
    if (!err) return KDA_ERR_CUDA;
    using namespace kda::scan;
    return kda_cuda_status(a->dtype == KDA_BF16 ? choose<kda::bf16>(a, ws, stream, err) : choose<float>(a, ws, stream, err));
}
