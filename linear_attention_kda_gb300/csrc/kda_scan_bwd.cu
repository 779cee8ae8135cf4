// kda_scan_bwd: tiles of L tokens by W channels as in kda_scan_fwd, taken from a sequence's last to its first.  With the
// adjoint lambda_t = dh_t + m_{t+1}, m_t = a_t lambda_t is what goes on to the token before.
//
// A thread forms decays and inputs of its eight tokens, runs the state forwards and the adjoint backwards from zero for the
// tile's sums, and, when it knows what enters from both sides (the state from the tile's checkpoint, the adjoint from the
// tiles behind it), runs them again: the states are kept in the place of the inputs, and the gates are formed once
// more, with their slopes, as the adjoint passes.  Sums over tokens for A_log and dt_bias leave a row for each tile, which
// a second kernel adds up.  Bound by instructions: 106 an element for 14 bytes in bf16 (gated, c of the norm), issued in
// 61 % of the cycles.  12 sequences of 700 to 5000 tokens, 4096 channels, bf16: 677 us, 3.0 TB/s (a thread to a channel of a sequence 9055); one of
// 8192 tokens 209 us; the 12 in fp32, one block to an SM, 957 us, 4.3 TB/s.  Eight tokens a thread, as many as keep their states, decays and gradients in 128 registers, two blocks to an SM.
#include "kda_scan_tiles.cuh"

namespace kda {
namespace scan {

// a tile begins at a checkpoint: L = 64, 128 or 256 tokens
template <int W> using bwd_shape = shape<W, 8>;
static_assert(bwd_shape<64>::L % CK == 0, "checkpoints");

template <typename T, int W> struct bwd_memory {
    ring<T, 4, bwd_shape<W>> next;
    tile_memory<W> M;
    entries<W> E;
    float f[NW][W];               // the warps' values of the state, then the states that enter their tokens
    float sA[NW][W], sb[NW][W];   // the warps' sums for A_log and dt_bias
};

struct sums_of {
    float *rows;  // [slots][2][D], or NULL
};

// The tokens of a thread (up to 8) by step_any(), read again from memory, as in kda_scan_fwd: h and m, the state and the adjoint that enter them from
// either side, become those that they leave; *sum: of the log-decays.  GRADS: leaves the tokens' gradients, and their sums for A_log and dt_bias,
// in the order of the others.
template <typename T, bool GRADS>
static __device__ __noinline__ void run_any(const kda_scan_bwd_args &A, int tok, int len, int c, float2 *h, float2 *m, float2 *sum, float2 *sA, float2 *sb) {
    constexpr int R = bwd_shape<64>::R;
    const int have = A.D - c;
    const spec K{A.gate_kind, A.input_scale, A.g_min};
    const channel<float2> C = load_channel(A.A_log, A.dt_bias, c, have);
    const float2 zero = make_float2(0.f, 0.f);
    const bool gated = A.input_gate != nullptr;
    auto get = [&](const void *p, int64_t stride, int r) { return load_pair<T, false>((const T *)p + (int64_t)(tok + r) * stride + c, have); };
    float2 d[R], u[R];  // u: a h before each token
    *sum = *sA = *sb = zero;
    for (int r = 0; r < len; ++r) {
        float2 z[1] = {get(A.z, A.z_stride, r)}, x[1] = {get(A.x, A.x_stride, r)};
        log_decays(K, C, z);
        const decay<float2> e = decay_of(z[0]);
        *sum = add(*sum, z[0]);
        d[r] = e.d;
        z[0] = e.m;
        scale_inputs(K, z, x);
        if (gated) {
            z[0] = get(A.input_gate, A.i_stride, r);
            gate_inputs(z, x);
        }
        u[r] = step_any(d[r], *h, zero);
        *h = GRADS ? add(u[r], x[0]) : step_any(d[r], *h, x[0]);
    }
    float2 lam[R];
    for (int r = len - 1; r >= 0; --r) {
        lam[r] = add(*m, get(A.grad_h, A.D, r));
        *m = step_any(d[r], lam[r], zero);
    }
    if (!GRADS) return;
    for (int i = 0; i < R; ++i) {  // two at a time from the last on
        const int r = R - 2 - i / 2 * 2 + i % 2;
        if (r >= len) continue;
        float2 z[1] = {get(A.z, A.z_stride, r)}, kA[1], x[1] = {get(A.x, A.x_stride, r)}, s[1] = {make_float2(1.f, 1.f)}, e[1] = {u[r]}, g = zero;
        decay_slopes(K, C, z, kA);
        if (gated) {
            const sig<float2> v = sigmoids(get(A.input_gate, A.i_stride, r));
            s[0] = v.s;
            g = mul(v.n, x[0]);
            x[0] = mul(x[0], v.s);
        }
        input_slopes(K, &d[r], x, e, s);
        const float2 dg = mul(e[0], lam[r]);
        *sA = fma(dg, kA[0], *sA);
        z[0] = mul(dg, z[0]);
        *sb = add(*sb, z[0]);
        s[0] = mul(s[0], lam[r]);
        const int64_t o = (int64_t)(tok + r) * A.D + c;
        store_pair<T, false>((T *)A.grad_x + o, s[0], have);
        store_pair<T, false>((T *)A.grad_z + o, z[0], have);
        if (gated) store_pair<T, false>((T *)A.grad_input_gate + o, mul(s[0], g), have);
    }
}

// PLAN: as for scan_fwd_kernel; the rows of slots without a tile are zeros then
template <typename T, int W, bool TMA, bool PLAN>
__global__ void __launch_bounds__(NT, sizeof(T) == 2 ? 2 : 1)
scan_bwd_kernel(const __grid_constant__ kda_scan_bwd_args A, const __grid_constant__ board B, const __grid_constant__ row_maps<4> maps,
                const __grid_constant__ sums_of out, layout how, int blocks, int *err) {
    using X = bwd_shape<W>;
    constexpr int L = X::L, R = X::R;
    extern __shared__ __align__(128) char memory[];
    bwd_memory<T, W> &S = *reinterpret_cast<bwd_memory<T, W> *>(memory);
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32, pair = lane % X::LPR * 2, row0 = w * X::RW + lane / X::LPR * R;
    const spec K{A.gate_kind, A.input_scale, A.g_min};
    const bool gated = A.input_gate != nullptr;
    if (PLAN && out.rows)
        for (int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x; i < B.slots * 2 * A.D; i += (int64_t)gridDim.x * NT) out.rows[i] = 0.f;
    if (PLAN) make_plan(B, A.cu_seqlens, A.T, A.N, A.D, blocks, err);
    const bool links = PLAN && !planned_chains(B), loader = w == NW - 1;
    course<L, PLAN> way(B, S.next.way, A.cu_seqlens, A.T, A.N, blocks, how, true);
    // the first token of a tile
    auto begin = [](const tile &t) { return t.a + (t.count > 0 ? t.count - 1 - t.p : 0) * L; };
    auto ask = [&](int turn) {
        if (!TMA || lane != 0) return;
        const tile &t = S.next.t[turn & 3];
        if (t.p < 0) return;
        const int stage = turn & 1, tok = begin(t), n = gated ? 4 : 3;
        tc::mbar_arrive_expect_tx(&S.next.full[stage], (uint32_t)(n * L * W * sizeof(T)));
        for (int i = 0; i < n; ++i) load_rows<X>(&S.next.x[stage][i][0][0], maps.m[i], t.block, tok, &S.next.full[stage]);
    };
    auto advance = [&](int turn) {
        const tile t = way.next();
        if (lane == 0) S.next.t[turn & 3] = t;
        __syncwarp();
    };
    if (threadIdx.x == 0) S.M.odd = 0;
    if (TMA && threadIdx.x == 0) {
        tc::mbar_init(&S.next.full[0], 1);
        tc::mbar_init(&S.next.full[1], 1);
        tc::fence_proxy_async();
    }
    __syncthreads();
    if (loader) {
        advance(0);
        advance(1);
        ask(0);
    }
    __syncthreads();
    constexpr int WARPS = W > 32 ? W / 32 : 1;     // of a role in join(), and
    const int mine = threadIdx.x % (32 * WARPS);  // this thread's channel in it
    channel<float2> C{};
    int of = -1;      // the block of channels whose parameters C holds
    tile last{0, -1, 0, 0, 0, 0, 0};  // the tile before, whose sums are in place
    auto add_up = [&](int ch) {
        if (!out.rows || last.p < 0 || last.count == 0 || last.block * W + ch >= A.D) return;
        float sA = 0.f, sb = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            sA += S.sA[i][ch];
            sb += S.sb[i][ch];
        }
        float *row = out.rows + (int64_t)(last.first + last.p) * 2 * A.D + last.block * W + ch;
        row[0] = sA;
        row[A.D] = sb;
    };
    for (int turn = 0;; ++turn) {
        const tile t = S.next.t[turn & 3];
        if (t.p < 0) break;
        const int stage = turn & 1, first = begin(t), tok = first + row0, len = t.b - tok < R ? t.b - tok : R;
        const int c = t.block * W + pair, have = A.D - c;
        if (of != t.block) C = load_channel(A.A_log, A.dt_bias, c, have);
        of = t.block;
        // the state that enters the tile, asked for early by those who will run it over the warps
        float checkpoint = 0.f;
        if (w / WARPS == 2 && mine < W && t.count > 0 && t.block * W + mine < A.D)
            checkpoint = A.checkpoints[((int64_t)t.a / CK + t.n + (first - t.a) / CK) * A.D + t.block * W + mine];
        if (TMA && !tc::mbar_wait(&S.next.full[stage], (turn >> 1) & 1)) set_error(err, KDA_ERR_DEVICE_TIMEOUT);
        // some tokens from r0 on of input k (z, x, grad_h, input_gate)
        auto get = [&](int k, int r0, const void *p, int64_t stride, auto &f) {
            constexpr int N = sizeof(f) / sizeof(f[0]);
#pragma unroll
            for (int r = 0; r < N; ++r)  // (by TMA there are rows of other sequences behind the last token)
                f[r] = TMA ? load_pair<T, true>(&S.next.x[stage][k][row0 + r0 + r][pair], 2)
                           : load_pair<T, false>((const T *)p + (int64_t)(tok + r0 + r) * stride + c, r0 + r < len ? have : 0);
        };
        float2 u[R], d[R], sum = make_float2(0.f, 0.f), h = sum, m = sum;
        constexpr int P1 = 8, P2 = 2;  // tokens whose gates are formed at a time, before the join and after it
#pragma unroll
        for (int r0 = 0; r0 < R; r0 += P1) {
            float2 z[P1], x[P1];
            get(0, r0, A.z, A.z_stride, z);
            log_decays(K, C, z);
            if (len < r0 + P1) {
#pragma unroll
                for (int r = 0; r < P1; ++r)
                    if (r0 + r >= len) z[r] = make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int r = 0; r < P1; ++r) {
                const decay<float2> e = decay_of(z[r]);
                sum = add(sum, z[r]);
                d[r0 + r] = e.d;
                z[r] = e.m;
            }
            get(1, r0, A.x, A.x_stride, x);
            scale_inputs(K, z, x);
            if (gated) {
                get(3, r0, A.input_gate, A.i_stride, z);
                gate_inputs(z, x);
            }
#pragma unroll
            for (int r = 0; r < P1; ++r) u[r0 + r] = x[r];
        }
        if (len < R) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r >= len) u[r] = make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) h = step(d[r], h, u[r]);
#pragma unroll
        for (int r0 = R - P1; r0 >= 0; r0 -= P1) {
            float2 g[P1];
            get(2, r0, A.grad_h, A.D, g);
#pragma unroll
            for (int r = P1 - 1; r >= 0; --r) {
                if (r0 + r >= len) g[r] = make_float2(0.f, 0.f);
                m = step(d[r0 + r], add(m, g[r]), make_float2(0.f, 0.f));
            }
        }
        if (!finite(h) || !finite(m)) S.M.odd = turn + 1;
        float2 before_sum, before, behind_sum, behind, all = sum;
        over_groups<X, false, false>(all, h, before_sum, before);
        if (lane >= 32 - X::LPR) *reinterpret_cast<float2 *>(&S.f[w][pair]) = h;
        over_groups<X, true, false>(sum, m, behind_sum, behind);
        if (lane < X::LPR) {
            *reinterpret_cast<float2 *>(&S.M.g[w][pair]) = sum;
            *reinterpret_cast<float2 *>(&S.M.d[w][pair]) = decay_of(sum).d;
            *reinterpret_cast<float2 *>(&S.M.b[w][pair]) = m;
        }
        const bool odd = join<X, true>(B, links, t, A.D, A.grad_final_state, A.grad_initial_state, nullptr, 0, S.M, S.E, turn + 1, err, [&](int role, int ch) {
            if (role == 2) {
                float v = checkpoint, b[NW];
#pragma unroll
                for (int i = 0; i < NW; ++i) {
                    b[i] = S.f[i][ch];
                    S.f[i][ch] = v;
                    v = step(S.M.d[i][ch], v, b[i]);
                }
                if (!finite(v)) {
                    v = checkpoint;
#pragma unroll
                    for (int i = 0; i < NW; ++i) {
                        S.f[i][ch] = v;
                        v = step_any(S.M.d[i][ch], v, b[i]);
                    }
                }
            } else {
                add_up(ch);
            }
        }, [&] {
            float2 s, f = make_float2(0.f, 0.f), b = f, none;
            run_any<T, false>(A, tok, len, c, &f, &b, &s, &none, &none);
            float2 up_to = s;
            over_groups<X, false, true>(up_to, f, before_sum, before);
            if (lane >= 32 - X::LPR) *reinterpret_cast<float2 *>(&S.f[w][pair]) = f;
            over_groups<X, true, true>(s, b, behind_sum, behind);
            if (lane < X::LPR) *reinterpret_cast<float2 *>(&S.M.b[w][pair]) = b;
        });
        if (loader) {
            // every warp is done with the tile before, whose stage the next one takes
            ask(turn + 1);
            advance(turn + 2);
        }
        const float2 h_in = *reinterpret_cast<const float2 *>(&S.f[w][pair]), m_in = *reinterpret_cast<const float2 *>(&S.M.g[w][pair]);
        h = group_entry<X, false>(h_in, before_sum, before);
        m = group_entry<X, false>(m_in, behind_sum, behind);
        float2 sA = make_float2(0.f, 0.f), sb = sA;
        if (__any_sync(0xffffffffu, odd || !finite(h) || !finite(m))) {
            float2 hs = group_entry<X, true>(h_in, before_sum, before), ms = group_entry<X, true>(m_in, behind_sum, behind), none, A2, b2;
            run_any<T, true>(A, tok, len, c, &hs, &ms, &none, &A2, &b2);
            sA = A2, sb = b2;
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) {  // u: a h before each token
                const float2 v = u[r];
                u[r] = step(d[r], h, make_float2(0.f, 0.f));
                h = add(u[r], v);
            }
            const int64_t at = (int64_t)tok * A.D + c;
#pragma unroll
            for (int r0 = R - P2; r0 >= 0; r0 -= P2) {
                float2 z[P2], kA[P2], x[P2], s[P2], e[P2], g[P2], lam[P2];
                get(0, r0, A.z, A.z_stride, z);
                decay_slopes(K, C, z, kA);
                get(1, r0, A.x, A.x_stride, x);
                get(2, r0, A.grad_h, A.D, g);
                if (len < r0 + P2) {
#pragma unroll
                    for (int r = 0; r < P2; ++r)
                        if (r0 + r >= len) z[r] = kA[r] = g[r] = make_float2(0.f, 0.f);
                }
#pragma unroll
                for (int r = P2 - 1; r >= 0; --r) {
                    lam[r] = m = add(m, g[r]);
                    m = step(d[r0 + r], m, make_float2(0.f, 0.f));
                }
                // g: what x is multiplied by but for c(a) and the gate's slope, s (1 - s)
                if (gated) {
                    get(3, r0, A.input_gate, A.i_stride, g);
#pragma unroll
                    for (int r = 0; r < P2; ++r) {
                        const sig<float2> v = sigmoids(g[r]);
                        s[r] = v.s;
                        g[r] = mul(v.n, x[r]);
                        x[r] = mul(x[r], v.s);
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < P2; ++r) s[r] = make_float2(1.f, 1.f);
                }
#pragma unroll
                for (int r = 0; r < P2; ++r) e[r] = u[r0 + r];
                input_slopes(K, &d[r0], x, e, s);
#pragma unroll
                for (int r = 0; r < P2; ++r) {
                    const float2 dg = mul(e[r], lam[r]);
                    sA = fma(dg, kA[r], sA);
                    z[r] = mul(dg, z[r]);
                    sb = add(sb, z[r]);
                    s[r] = mul(s[r], lam[r]);
                    if (r0 + r < len && have > 0) {
                        const int64_t o = at + (int64_t)(r0 + r) * A.D;
                        store_pair<T, TMA>((T *)A.grad_x + o, s[r], have);
                        store_pair<T, TMA>((T *)A.grad_z + o, z[r], have);
                        if (gated) store_pair<T, TMA>((T *)A.grad_input_gate + o, mul(s[r], g[r]), have);
                    }
                }
            }
        }
#pragma unroll
        for (int off = X::LPR; off < 32; off *= 2) {
            sA = add(sA, make_float2(__shfl_xor_sync(0xffffffffu, sA.x, off), __shfl_xor_sync(0xffffffffu, sA.y, off)));
            sb = add(sb, make_float2(__shfl_xor_sync(0xffffffffu, sb.x, off), __shfl_xor_sync(0xffffffffu, sb.y, off)));
        }
        if (lane < X::LPR) {
            *reinterpret_cast<float2 *>(&S.sA[w][pair]) = sA;
            *reinterpret_cast<float2 *>(&S.sb[w][pair]) = sb;
        }
        last = t;
    }
    __syncthreads();
    if (w / WARPS == 3 && mine < W) add_up(mine);
    if (!PLAN) check_all(A.cu_seqlens, A.T, A.N, err);
}

// The rows of a call without a plan: those of slots without a tile were not written, nor was any of one sequence that is bad.
struct alike {
    const int32_t *cu;
    int64_t T, N;
    int L;  // 0: a call with a plan
    __device__ __forceinline__ bool has(int64_t slot) const {
        if (L == 0) return true;
        const int64_t each = T / N, n = ((slot + 1) * L - 1) / (each + L);  // the last sequence whose first slot, n each / L + n, is not behind
        lin::span s;
        return n < N && lin::seq_span(cu, T, N, n, &s) && slot - (s.a / L + n) < (each + L - 1) / L;
    }
};

// Column sums of the tiles' rows: 32 columns to a block, its eight warps every eighth row.
__global__ void __launch_bounds__(256) scan_sums_kernel(const float *rows, int64_t slots, const __grid_constant__ alike some, int D, float *dA, float *db) {
    __shared__ float part[8][32];
    float *to = blockIdx.y == 0 ? dA : db;
    if (!to) return;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v[4] = {};
    if (c < D) {
        const float *p = rows + (int64_t)blockIdx.y * D + c;
        int64_t r = w;
        for (; r + 24 < slots; r += 32)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (some.has(r + 8 * i)) v[i] += p[(r + 8 * i) * 2 * D];
        for (; r < slots; r += 8)
            if (some.has(r)) v[0] += p[r * 2 * D];
    }
    part[w][lane] = (v[0] + v[1]) + (v[2] + v[3]);
    __syncthreads();
    if (w == 0 && c < D) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += part[i][lane];
        to[c] = s;
    }
}

template <typename T, int W, bool TMA>
static cudaError_t launch(const kda_scan_bwd_args *a, void *ws, cudaStream_t stream, int *err) {
    using X = bwd_shape<W>;
    static std::atomic<int> running[2][64];
    constexpr size_t smem = sizeof(bwd_memory<T, W>);
    row_maps<4> maps{};
    if (TMA && (!make_row_map<X>(&maps.m[0], a->z, a->T, a->D, a->z_stride, a->dtype) ||
                !make_row_map<X>(&maps.m[1], a->x, a->T, a->D, a->x_stride, a->dtype) ||
                !make_row_map<X>(&maps.m[2], a->grad_h, a->T, a->D, a->D, a->dtype) ||
                (a->input_gate && !make_row_map<X>(&maps.m[3], a->input_gate, a->T, a->D, a->i_stride, a->dtype))))
        return cudaErrorUnknown;
    int blocks = (a->D + W - 1) / W, grid = 0;
    board B{};
    const size_t rows = board_layout(a->T, a->N, a->D, X::L, ws, &B);
    sums_of out{a->grad_A_log || a->grad_dt_bias ? (float *)((char *)ws + rows) : nullptr};
    layout how = PLANNED;
    kda_scan_bwd_args args = *a;
    void *p[] = {&args, &B, &maps, &out, &how, &blocks, &err};
    cudaError_t e = running_blocks(scan_bwd_kernel<T, W, TMA, false>, smem, running[0], B.slots * blocks, &grid);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (a->T / a->N + X::L - 1) / X::L;  // of a sequence, where they are alike
    if ((!a->cu_seqlens || a->N == 1) && rather_whole(tiles, tiles * a->N, blocks, grid)) {
        how = EQUAL;
        e = cudaLaunchKernel((const void *)scan_bwd_kernel<T, W, TMA, false>, dim3(grid), dim3(NT), p, smem, stream);
    } else {
        e = running_blocks(scan_bwd_kernel<T, W, TMA, true>, smem, running[1], B.slots * blocks, &grid);
        if (e != cudaSuccess) return e;
        e = cudaLaunchCooperativeKernel((const void *)scan_bwd_kernel<T, W, TMA, true>, dim3(grid), dim3(NT), p, smem, stream);
    }
    if (e != cudaSuccess || !out.rows) return e;
    const alike some{a->cu_seqlens, a->T, a->N, how == EQUAL ? X::L : 0};
    scan_sums_kernel<<<dim3((a->D + 31) / 32, 2), 256, 0, stream>>>(out.rows, B.slots, some, a->D, a->grad_A_log, a->grad_dt_bias);
    return cudaGetLastError();
}

template <typename T> static cudaError_t choose(const kda_scan_bwd_args *a, void *ws, cudaStream_t stream, int *err) {
    const int64_t es = sizeof(T), per = 16 / es;
    const bool tma = a->T > 0 && a->D % per == 0 &&
                     (((uintptr_t)a->x | (uintptr_t)a->z | (uintptr_t)a->input_gate | (uintptr_t)a->grad_h) & 15) == 0 &&
                     (((uintptr_t)a->grad_x | (uintptr_t)a->grad_z | (uintptr_t)a->grad_input_gate) % (2 * es)) == 0 && a->x_stride % per == 0 &&
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

size_t kda_scan_bwd_bytes(int64_t T, int64_t N, int D, kda_dtype_t) {
    using namespace kda::scan;
    // (the shortest tile's, which holds all)
    constexpr int L = bwd_shape<64>::L;
    return board_layout(T, N, D, L, nullptr, nullptr) + (size_t)kda::lin::chunk_slots(T, N, L) * 2 * D * 4;
}

kda_status_t kda_launch_scan_bwd(const kda_scan_bwd_args *a, void *ws, cudaStream_t stream) {
    int *err = kda_device_error_ptr();
    if (!err) return KDA_ERR_CUDA;
    using namespace kda::scan;
    return kda_cuda_status(a->dtype == KDA_BF16 ? choose<kda::bf16>(a, ws, stream, err) : choose<float>(a, ws, stream, err));
}
