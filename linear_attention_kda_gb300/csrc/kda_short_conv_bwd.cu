// kda_short_conv_bwd: a warp takes a run of L tokens of one sequence by 32 V channels.  At token t it forms p, s and y once
// more, from the last K rows in registers, and with them
//     ds = (dy - y sum(dy y)) / |s|  (or dy),      dp_t = ds dSwish(p)  (or ds),
// whose last K - 1 are in registers too: dx_{t-K+1} = sum_j weight_j dp_{t-j} is then complete, for K - 1 tokens behind
// the run as well, whose dp is formed a second time by the next one.  weight and bias gather their sums over tokens in
// registers; the four warps of a block, which have four runs of the same channels, add theirs up in shared memory, and
// a second kernel adds up the blocks' rows, all in a fixed order.  Bound by instructions: 48 an element with the norm
// over heads of 128, for 6 bytes in bf16, issued in 59 % of the cycles.  65536 tokens of 4096 channels 567 us, 2.8 TB/s (without the norm 381 us), 4096
// tokens 52 us; 32768 tokens in fp32 304 us, 5.3 TB/s.  Two tokens' sums at once
// and a second copy of the loop without questions about a run's ends cost more registers or instructions fetched than they saved.
#include <atomic>

#include "kda_short_conv.cuh"

namespace kda {
namespace conv {

// Four warps, four blocks to an SM: 65536 tokens 560 us, 584 with eight and two
constexpr int NW = 4;
// Rows at a time, which is how far the loop over tokens is unrolled: bf16 by fours (8 sequences of 300 to 5000 tokens, runs of 64: 215 us, 234 by eights; fp32 gained
// nothing by twos, heads of 256 lost)
template <typename T, int V> constexpr int bwd_rows = sizeof(T) == 2 && V == 4 ? some_rows<T, V> / 2 : some_rows<T, V>;

template <typename T, int K, int V, bool WIDE>
__global__ void __launch_bounds__(32 * NW, V == 4 ? 4 : 2)
conv_bwd_kernel(const __grid_constant__ spec S, const __grid_constant__ row_maps maps, const T *x, const T *hist, const T *dy, const T *dtail, T *dx, T *dhist, float *sums, int L,
                int64_t slots, int *err) {
    constexpr int U = bwd_rows<T, V>;
    extern __shared__ __align__(128) char memory[];
    float (*part)[32 * V] = reinterpret_cast<float(*)[32 * V]>(memory + (WIDE ? NW * sizeof(ring<T, V, 2, bwd_rows<T, V>>) : 0));
    check_all(S, err);
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t slot = (int64_t)blockIdx.x * NW + w;
    const int c0 = (int)blockIdx.y * 32 * V, c = c0 + lane * V, have = S.D - c;
    float2 dw[K][V / 2], db[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        db[i] = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < K; ++k) dw[k][i] = db[i];
    }
    run r;
    if (slot < slots && find_run(S, slot, L, &r)) {
        const rows<T, V, WIDE> X{x + r.a * S.stride + c, hist ? hist + r.n * (K - 1) * S.D + c : nullptr, S.stride, S.D, K, have};
        const taps<V, K> P(S, c, have);
        // tokens behind the run's end that its gradients need; those behind the sequence have dp = 0
        const int stop = r.last + K - 1, turns = (stop - r.first + U - 1) / U;
        ring<T, V, 2, bwd_rows<T, V>> &Q = reinterpret_cast<ring<T, V, 2, bwd_rows<T, V>> *>(memory)[w];
        auto ask = [&](int turn) {
            if (!WIDE || lane != 0 || turn >= turns) return;
            const int stage = turn % NS, tok = (int)r.a + r.first + turn * U;
            tc::mbar_arrive_expect_tx(&Q.full[stage], sizeof(Q.x[0]));
            tc::tma_load_3d(&Q.x[stage][0], &maps.x, c0, 0, tok, &Q.full[stage]);
            tc::tma_load_3d(&Q.x[stage][1], &maps.dy, c0, 0, tok, &Q.full[stage]);
        };
        if (WIDE) {
            if (lane == 0) {
#pragma unroll
                for (int i = 0; i < NS; ++i) tc::mbar_init(&Q.full[i], 1);
                tc::fence_proxy_async();
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < NS; ++i) ask(i);
        }
        float2 row[K - 1 + U][V / 2], dp[K - 1 + U][V / 2];
#pragma unroll
        for (int k = 0; k < K - 1; ++k) {
            layer::unpack<T, V>(X.at(r.first - (K - 1) + k), row[k]);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) dp[k][i] = make_float2(0.f, 0.f);
        }
        const T *px = X.x + r.first * S.stride, *pg = dy + (r.a + r.first) * S.D + c;
        T *out = dx + (r.a + r.first - (K - 1)) * S.D + c;
        int t = r.first;
        for (int turn = 0, stage = 0, phase = 0; turn < turns; ++turn) {
            if (WIDE && !tc::mbar_wait(&Q.full[stage], phase)) set_error(err, KDA_ERR_DEVICE_TIMEOUT);
#pragma unroll
            for (int u = 0; u < U; ++u, ++t, out += S.D) {
                float2 d[V / 2], p[V / 2], ds[V / 2], q = make_float2(0.f, 0.f), e = q;
                if constexpr (WIDE) {  // (rows of the next sequence, or what a box beyond the last one is filled with, are left out below)
                    layer::unpack<T, V>(layer::load<T, V>(&Q.x[stage][0][u][lane * V]), row[K - 1 + u]);
                    layer::unpack<T, V>(layer::load<T, V>(&Q.x[stage][1][u][lane * V]), d);
                } else {
                    if (t < r.len) {
                        layer::unpack<T, V>(load<T, V, false>(px, have), row[K - 1 + u]);
                        layer::unpack<T, V>(load<T, V, false>(pg, have), d);
                    }
                    px += S.stride;
                    pg += S.D;
                }
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    p[i] = P.b[i];
#pragma unroll
                    for (int k = 0; k < K; ++k) p[i] = fma(P.w[k][i], row[u + k][i], p[i]);
                }
                if (S.act) {
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        const layer::sig<float2> v = layer::sigmoids(p[i]);
                        ds[i] = fma(mul(p[i], v.n), v.s, v.s);
                        p[i] = mul(p[i], v.s);
                    }
                }
                if (S.norm) {
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        q = fma(p[i], p[i], q);
                        e = fma(d[i], p[i], e);
                    }
                    float k = q.x + q.y, dot = e.x + e.y;
                    head_sums<V>(k, dot, S.norm);
                    k = rsqrtf(k + S.eps);
                    dot *= -k * k;
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) d[i] = mul(fma(p[i], make_float2(dot, dot), d[i]), make_float2(k, k));
                }
                if (S.act) {
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) d[i] = mul(d[i], ds[i]);
                }
                if (t >= r.len) {
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) d[i] = make_float2(0.f, 0.f);
                }
#pragma unroll
                for (int i = 0; i < V / 2; ++i) dp[K - 1 + u][i] = d[i];
                if (t < r.last) {
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        db[i] = add(db[i], d[i]);
#pragma unroll
                        for (int k = 0; k < K; ++k) dw[k][i] = fma(d[i], row[u + k][i], dw[k][i]);
                    }
                }
                // row t - K + 1 of the sequence, its history's where that is below 0
                const int at = t - (K - 1);
                if (at < r.last && (at >= r.first || (r.first == 0 && dhist))) {
                    float2 v[V / 2];
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        v[i] = mul(P.w[0][i], d[i]);
#pragma unroll
                        for (int k = 1; k < K; ++k) v[i] = fma(P.w[k][i], dp[K - 1 + u - k][i], v[i]);
                    }
                    if (dtail && at >= r.len - (K - 1)) {
                        float2 f[V / 2];
                        layer::unpack<T, V>(load<T, V, WIDE>(dtail + (r.n * (K - 1) + at - r.len + K - 1) * S.D + c, have), f);
#pragma unroll
                        for (int i = 0; i < V / 2; ++i) v[i] = add(v[i], f[i]);
                    }
                    store<T, V, WIDE>(at >= 0 ? out : dhist + (r.n * (K - 1) + at + K - 1) * S.D + c, layer::pack<T, V>(v), have);
                }
            }
            __syncwarp();
            ask(turn + NS);
            if (++stage == NS) stage = 0, phase ^= 1;
#pragma unroll
            for (int k = 0; k < K - 1; ++k)
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    row[k][i] = row[U + k][i];
                    dp[k][i] = dp[U + k][i];
                }
        }
    }
    if (!sums) return;
    // [block of runs][K + 1][D]
#pragma unroll
    for (int k = 0; k <= K; ++k) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V / 2; ++i) *reinterpret_cast<float2 *>(&part[w][lane * V + 2 * i]) = k < K ? dw[k < K ? k : 0][i] : db[i];
        __syncthreads();
        for (int ch = threadIdx.x; ch < 32 * V; ch += 32 * NW) {
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < NW; ++i) v += part[i][ch];
            const int at = (int)blockIdx.y * 32 * V + ch;
            if (at < S.D) sums[((int64_t)blockIdx.x * (K + 1) + k) * S.D + at] = v;
        }
    }
}

// Column sums of the blocks' rows: 32 columns of one tap (or the bias) to a block, its eight warps every eighth row.
__global__ void __launch_bounds__(256) conv_sums_kernel(const float *sums, int64_t rows, int D, int K, float *dw, float *db) {
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, k = blockIdx.y;
    if (!(k < K ? dw : db)) return;
    float v = 0.f;
    if (c < D)
        for (int64_t r = w; r < rows; r += 8) v += sums[(r * (K + 1) + k) * D + c];
    part[w][lane] = v;
    __syncthreads();
    if (w == 0 && c < D) {
        v = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v += part[i][lane];
        if (k < K) dw[(int64_t)c * K + k] = v;
        else db[c] = v;
    }
}

// (4096 channels by runs of 32, 48, 64, 96 and 128: 4096 tokens 58, 73, 55, 66 and 76 us, 65536 tokens 687,
// 627, -, 568 and 557)
static int run_length(int64_t T, int64_t N, int D) { return run_length(T, N, (D + 127) / 128, NW, 4 * 152); }

template <typename T, int K, int V, bool WIDE>
static cudaError_t launch(const kda_short_conv_bwd_args *a, float *sums, cudaStream_t stream, int *err) {
    const int L = run_length(a->T, a->N, a->D);
    const int64_t slots = lin::chunk_slots(a->T, a->N, L), rows = (slots + NW - 1) / NW;
    row_maps maps{};
    if (WIDE && (!layer::make_row_map(&maps.x, a->x, a->T, a->D, a->x_stride, a->dtype, 32 * V, bwd_rows<T, V>) ||
                 !layer::make_row_map(&maps.dy, a->grad_y, a->T, a->D, a->D, a->dtype, 32 * V, bwd_rows<T, V>)))
        return cudaErrorUnknown;
    constexpr int smem = (WIDE ? NW * (int)sizeof(ring<T, V, 2, bwd_rows<T, V>>) : 0) + NW * 32 * V * 4;
    if (smem > 48 * 1024) {
        static std::atomic<uint64_t> done{0};
        const cudaError_t e = lin::allow_smem(conv_bwd_kernel<T, K, V, WIDE>, smem, done);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)rows, (a->D + 32 * V - 1) / (32 * V));
    conv_bwd_kernel<T, K, V, WIDE><<<grid, 32 * NW, smem, stream>>>(
        spec_of(a, a->T, a->cu_seqlens), maps, (const T *)a->x, (const T *)a->initial_state, (const T *)a->grad_y, (const T *)a->grad_final_state,
        (T *)a->grad_x, (T *)a->grad_initial_state, sums, L, slots, err);
    if (sums) conv_sums_kernel<<<dim3((a->D + 31) / 32, K + 1), 256, 0, stream>>>(sums, rows, a->D, K, a->grad_weight, a->grad_bias);
    return cudaGetLastError();
}

template <typename T, int K>
static cudaError_t choose(const kda_short_conv_bwd_args *a, float *sums, bool wide, cudaStream_t stream, int *err) {
    // four channels a lane, eight where a head is 256 wide and has to lie in a warp
    if (a->norm_dim == 256) return wide ? launch<T, K, 8, true>(a, sums, stream, err) : launch<T, K, 8, false>(a, sums, stream, err);
    return wide ? launch<T, K, 4, true>(a, sums, stream, err) : launch<T, K, 4, false>(a, sums, stream, err);
}

}  // namespace conv
}  // namespace kda

size_t kda_short_conv_bwd_bytes(int64_t T, int64_t N, int D, int K) {
    using namespace kda::conv;
    return (size_t)((kda::lin::chunk_slots(T, N, run_length(T, N, D)) + NW - 1) / NW) * (K + 1) * D * 4;
}

kda_status_t kda_launch_short_conv_bwd(const kda_short_conv_bwd_args *a, void *ws, cudaStream_t stream) {
    int *err = kda_device_error_ptr();
    if (!err) return KDA_ERR_CUDA;
    using namespace kda::conv;
    // vectors of V channels, and x and grad_y by TMA, where rows allow both
    const int V = a->norm_dim == 256 ? 8 : 4, per = a->dtype == KDA_BF16 ? 8 : 4;
    const uintptr_t bytes = V == 4 && per == 8 ? 8 : 16;
    const bool wide = a->T > 0 && a->D % (V > per ? V : per) == 0 && a->x_stride % per == 0 && (((uintptr_t)a->x | (uintptr_t)a->grad_y) & 15) == 0 &&
                      (((uintptr_t)a->grad_x | (uintptr_t)a->initial_state | (uintptr_t)a->grad_final_state | (uintptr_t)a->grad_initial_state) % bytes) == 0;
    float *sums = a->grad_weight || a->grad_bias ? (float *)ws : nullptr;
    auto go = [&](auto t) {
        using T = decltype(t);
        return a->K == 2 ? choose<T, 2>(a, sums, wide, stream, err) : a->K == 3 ? choose<T, 3>(a, sums, wide, stream, err)
                                                                              : choose<T, 4>(a, sums, wide, stream, err);
    };
    return kda_cuda_status(a->dtype == KDA_BF16 ? go(kda::bf16{}) : go(float{}));
}
