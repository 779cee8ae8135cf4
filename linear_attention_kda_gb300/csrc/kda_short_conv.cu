// kda_short_conv_fwd: a warp takes a run of L tokens of one sequence by 32 V channels, V to a lane, and goes through the
// tokens with the last K - 1 of them in registers; the sums of a head's squares meet by shuffles between the lanes that
// hold it.  Rows come by TMA, up to 24 tokens ahead.  Bound by HBM traffic, x read once (but for the K - 1 tokens before each
// run) and y written once, and close to that by instructions: 20 an element with the norm.  bf16, 32 sequences of 512 to 8192
// tokens, 4096 channels, four taps: 337 us, 6.4 TB/s; with the norm over heads of 128 409 us, 5.3 TB/s; 16 of them in fp32 371 us, 6.6 TB/s (four tokens' sums at once; 427 two
// and 479 one at a time).  V = 8 was no faster where 4 will do.
//
// kda_short_conv_step: the same for one token, whose history is a slot of a pool.
#include <atomic>

#include "kda_short_conv.cuh"

namespace kda {
namespace conv {

// One token from its K rows: s's V values, and the sum of their squares
template <int K, int V>
__device__ __forceinline__ float one(const spec &S, const taps<V, K> &P, const float2 (*row)[V / 2], float2 (&y)[V / 2]) {
    float2 q = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        y[i] = P.b[i];
#pragma unroll
        for (int k = 0; k < K; ++k) y[i] = fma(P.w[k][i], row[k][i], y[i]);
    }
    if (S.act) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) y[i] = mul(y[i], layer::sigmoid(y[i]));
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) q = fma(y[i], y[i], q);
    return q.x + q.y;
}
template <int V> __device__ __forceinline__ void scale(float2 (&y)[V / 2], float squares, float eps) {
    const float r = rsqrtf(squares + eps);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) y[i] = mul(y[i], make_float2(r, r));
}

template <typename T, int K, int V, bool WIDE>
__global__ void __launch_bounds__(128) conv_fwd_kernel(const __grid_constant__ spec S, const __grid_constant__ row_maps maps, const T *x,
                                                       const T *hist, T *tail, T *y, int L, int blocks, int64_t items, int *err) {
    constexpr int U = some_rows<T, V>, J = V == 4 ? 4 : 2;  // (four at V = 8 454 us for 440, registers)
    extern __shared__ __align__(128) char memory[];
    check_all(S, err);
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t item = (int64_t)blockIdx.x * 4 + w;
    if (item >= items) return;
    run r;
    if (!find_run(S, item / blocks, L, &r)) return;
    const int c0 = (int)(item % blocks) * 32 * V, c = c0 + lane * V, have = S.D - c;
    const rows<T, V, WIDE> X{x + r.a * S.stride + c, hist ? hist + r.n * (K - 1) * S.D + c : nullptr, S.stride, S.D, K, have};
    if (r.first < r.last) {
        ring<T, V, 1, some_rows<T, V>> &Q = reinterpret_cast<ring<T, V, 1, some_rows<T, V>> *>(memory)[w];
        const int turns = (r.last - r.first + U - 1) / U;
        auto ask = [&](int turn) {
            if (!WIDE || lane != 0 || turn >= turns) return;
            tc::mbar_arrive_expect_tx(&Q.full[turn % NS], sizeof(Q.x[0]));
            tc::tma_load_3d(&Q.x[turn % NS], &maps.x, c0, 0, (int)r.a + r.first + turn * U, &Q.full[turn % NS]);
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
        const taps<V, K> P(S, c, have);
        float2 row[K - 1 + U][V / 2];
#pragma unroll
        for (int k = 0; k < K - 1; ++k) layer::unpack<T, V>(X.at(r.first - (K - 1) + k), row[k]);
        const T *from = X.x + r.first * S.stride;
        T *out = y + (r.a + r.first) * S.D + c;
        for (int turn = 0, stage = 0, phase = 0; turn < turns; ++turn) {
            const int left = r.last - r.first - turn * U;
            if (WIDE && !tc::mbar_wait(&Q.full[stage], phase)) set_error(err, KDA_ERR_DEVICE_TIMEOUT);
#pragma unroll
            for (int u0 = 0; u0 < U; u0 += J) {  // J tokens, whose sums go over the lanes together
                float2 v[J][V / 2];
                float ss[J];
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int u = u0 + j;
                    if constexpr (WIDE) {
                        layer::unpack<T, V>(layer::load<T, V>(&Q.x[stage][0][u][lane * V]), row[K - 1 + u]);
                    } else {
                        if (u < left) layer::unpack<T, V>(load<T, V, false>(from, have), row[K - 1 + u]);
                        from += S.stride;
                    }
                    ss[j] = one<K, V>(S, P, &row[u], v[j]);
                }
                if (S.norm) {
                    head_sums<V>(ss, S.norm);
#pragma unroll
                    for (int j = 0; j < J; ++j) scale<V>(v[j], ss[j], S.eps);
                }
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    if (u0 + j < left) store<T, V, WIDE>(out, layer::pack<T, V>(v[j]), have);
                    out += S.D;
                }
            }
            __syncwarp();
            ask(turn + NS);
            if (++stage == NS) stage = 0, phase ^= 1;
#pragma unroll
            for (int k = 0; k < K - 1; ++k)
#pragma unroll
                for (int i = 0; i < V / 2; ++i) row[k][i] = row[U + k][i];
        }
    }
    // The history behind the sequence, by the lanes that alone read the one before it: the two may be the same
    if (tail && r.first == 0) {
        vec<T, V> v[K - 1];
#pragma unroll
        for (int k = 0; k < K - 1; ++k) v[k] = X.at(r.len - (K - 1) + k);
#pragma unroll
        for (int k = 0; k < K - 1; ++k) store<T, V, WIDE>(tail + (r.n * (K - 1) + k) * S.D + c, v[k], have);
    }
}

template <typename T, int K, int V, bool WIDE>
__global__ void __launch_bounds__(128) conv_step_kernel(const __grid_constant__ spec S, const T *x, T *state, const int32_t *idx, int64_t slots, T *y,
                                                        int *err) {
    const int64_t n = blockIdx.x;
    const int64_t slot = layer::slot_of(idx, slots, n, err);
    if (slot < 0) return;
    const int c = (blockIdx.y * 128 + threadIdx.x) * V, have = S.D - c;
    T *hist = state + slot * (K - 1) * S.D + c;
    const rows<T, V, WIDE> X{x + n * S.stride + c, hist, S.stride, S.D, K, have};
    vec<T, V> v[K];
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = X.at(k - (K - 1));
    const taps<V, K> P(S, c, have);
    if (layer::taken<128>(idx, n, slot, err)) return;
    float2 row[K][V / 2], out[V / 2];
#pragma unroll
    for (int k = 0; k < K; ++k) layer::unpack<T, V>(v[k], row[k]);
    const float ss = one<K, V>(S, P, row, out);
    if (S.norm) scale<V>(out, head_sum<V>(ss, S.norm), S.eps);
#pragma unroll
    for (int k = 0; k + 1 < K; ++k) store<T, V, WIDE>(hist + k * S.D, v[k + 1], have);
    store<T, V, WIDE>(y + n * S.D + c, layer::pack<T, V>(out), have);
}

template <typename T, int K, int V, bool WIDE>
static cudaError_t fwd(const kda_short_conv_args *a, cudaStream_t stream, int *err) {
    const int blocks = (a->D + 32 * V - 1) / (32 * V);
    // (five blocks an SM: 96 registers, in bf16 with the norm)
    const int L = run_length(a->T, a->N, (blocks + 3) / 4, 1, 5 * 152);
    const int64_t items = lin::chunk_slots(a->T, a->N, L) * blocks;
    row_maps maps{};
    if (WIDE && !layer::make_row_map(&maps.x, a->x, a->T, a->D, a->x_stride, a->dtype, 32 * V, some_rows<T, V>)) return cudaErrorUnknown;
    constexpr int smem = WIDE ? 4 * (int)sizeof(ring<T, V, 1, some_rows<T, V>>) : 0;
    if (smem > 48 * 1024) {
        static std::atomic<uint64_t> done{0};
        const cudaError_t e = lin::allow_smem(conv_fwd_kernel<T, K, V, WIDE>, smem, done);
        if (e != cudaSuccess) return e;
    }
    conv_fwd_kernel<T, K, V, WIDE><<<(unsigned)((items + 3) / 4), 128, smem, stream>>>(spec_of(a, a->T, a->cu_seqlens), maps, (const T *)a->x,
                                                                                      (const T *)a->initial_state, (T *)a->final_state,
                                                                                      (T *)a->y, L, blocks, items, err);
    return cudaGetLastError();
}

template <typename T, int K, int V, bool WIDE>
static void step(const kda_short_conv_step_args *a, cudaStream_t stream, int *err) {
    const int per = 128 * V;
    conv_step_kernel<T, K, V, WIDE><<<dim3((unsigned)a->N, (a->D + per - 1) / per), 128, 0, stream>>>(
        spec_of(a, a->N, nullptr), (const T *)a->x, (T *)a->state, a->state_indices, a->num_slots, (T *)a->y, err);
}

// Calls go(type, taps, channels to a lane, wide): four channels, eight where a head is 256 wide and has to lie in a warp.
template <int I> using number = std::integral_constant<int, I>;
template <typename A, typename F>
static void choose(const A *a, const void *first, const void *second, bool wide, F &&go) {
    const int V = a->norm_dim == 256 ? 8 : 4;
    const uintptr_t bytes = V == 4 && a->dtype == KDA_BF16 ? 8 : 16;
    wide = wide && a->D % V == 0 && a->x_stride % V == 0 &&
                      ((uintptr_t)a->x | (uintptr_t)a->y | (uintptr_t)first | (uintptr_t)second) % bytes == 0;
    auto width = [&](auto t, auto k, auto v) {
        if (wide) go(t, k, v, std::true_type{});
        else go(t, k, v, std::false_type{});
    };
    auto channels = [&](auto t, auto k) {
        if (V == 8) width(t, k, number<8>{});
        else width(t, k, number<4>{});
    };
    auto taps_of = [&](auto t) {
        if (a->K == 2) channels(t, number<2>{});
        else if (a->K == 3) channels(t, number<3>{});
        else channels(t, number<4>{});
    };
    if (a->dtype == KDA_BF16) taps_of(bf16{});
    else taps_of(float{});
}

}  // namespace conv
}  // namespace kda

kda_status_t kda_launch_short_conv_fwd(const kda_short_conv_args *a, cudaStream_t stream) {
    int *err = kda_device_error_ptr();
    if (!err) return KDA_ERR_CUDA;
    using namespace kda::conv;
    cudaError_t e = cudaSuccess;
    // (by TMA, where x's rows are multiples of 16 bytes)
    const int64_t per = a->dtype == KDA_BF16 ? 8 : 4;
    const bool rows = a->T > 0 && a->x_stride % per == 0 && ((uintptr_t)a->x & 15) == 0;
    choose(a, a->initial_state, a->final_state, rows, [&](auto t, auto k, auto v, auto w) {
        e = fwd<decltype(t), decltype(k)::value, decltype(v)::value, decltype(w)::value>(a, stream, err);
    });
    return kda_cuda_status(e);
}

kda_status_t kda_launch_short_conv_step(const kda_short_conv_step_args *a, cudaStream_t stream) {
    int *err = kda_device_error_ptr();
    if (!err) return KDA_ERR_CUDA;
    using namespace kda::conv;
    choose(a, a->state, nullptr, true, [&](auto t, auto k, auto v, auto w) {
        step<decltype(t), decltype(k)::value, decltype(v)::value, decltype(w)::value>(a, stream, err);
    });
    return kda_cuda_status(cudaGetLastError());
}
