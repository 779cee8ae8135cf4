// kda_linear_recurrent_step: one decode token per sequence of linear attention with a decay per head,
//     S <- a S + k v^T,  o = scale * S^T q,   a = exp(g),
// the state [dk, dv] of every (sequence, head) updated in place.
//
// Bound by HBM traffic on the fp32 state, read once and written once.  A CTA owns CW columns of one state:
// 256 threads, CW / 4 of them on a row with four columns each, so that a row's piece moves as 16-byte vectors
// (CW = 128: one 512-byte row per warp; CW = 32: whole 128-byte lines, four rows per warp).  A thread keeps its
// rows in registers between the read and the write and forms its part of S^T q on the way; the parts of the rows
// meet by shuffles and through shared memory.  Columns are independent, so a small batch splits every state over
// dv / 32 CTAs (see launch_w).  256 sequences x 32 heads, bf16, dk = dv = 128: 160 us, 6.78 TB/s.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace lin {

template <int DK, int DV, int CW, typename T>
__global__ void __launch_bounds__(256)
linear_step_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                   const float *__restrict__ g, int g_stride, float scale, float *__restrict__ state,
                   const int32_t *__restrict__ idx, int64_t slots, int H, int rq, int rk, int rv, T *__restrict__ o,
                   int *err) {
    constexpr int LPR = CW / 4;           // lanes on a row
    constexpr int RPP = 256 / LPR;        // rows per pass of the CTA
    constexpr int PASSES = DK / RPP;
    constexpr int SPLIT = DV / CW;
    static_assert(DK % RPP == 0 && LPR <= 32, "row split");
    __shared__ float s_q[DK], s_k[DK];
    __shared__ float4 s_part[8][LPR];

    const int part = blockIdx.x % SPLIT;
    const int64_t unit = blockIdx.x / SPLIT;
    const int64_t n = unit / H;
    const int h = (int)(unit % H);
    const int tid = threadIdx.x, lane = tid & 31;
    int64_t slot = n;
    if (idx) {
        slot = idx[n];
        if (slot == -1) return;  // an unused row of a padded batch
        if (slot < 0 || slot >= slots) {
            if (tid == 0) set_error(err, KDA_ERR_BAD_STATE_INDEX);
            return;
        }
    }
    const int col = (tid % LPR) * 4, row0 = tid / LPR;
    float *S = state + (slot * H + h) * (int64_t)(DK * DV) + part * CW + col;
    float4 s[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
        s[i] = __ldcs(reinterpret_cast<const float4 *>(S + (int64_t)(row0 + i * RPP) * DV));
    // an earlier row with the same slot has it: nothing of this one is written
    bool taken = false;
    if (idx)
        for (int64_t m = tid; m < n; m += 256) taken |= idx[m] == (int32_t)slot;
    const int Hq = H / rq, Hk = H / rk, Hv = H / rv;
    for (int i = tid; i < DK; i += 256) {
        s_q[i] = ld(q + (n * Hq + h / rq) * DK + i);
        s_k[i] = ld(k + (n * Hk + h / rk) * DK + i);
    }
    const T *vr = v + (n * Hv + h / rv) * DV + part * CW + col;
    const float4 vc = make_float4(ld(vr), ld(vr + 1), ld(vr + 2), ld(vr + 3));
    const float a = g ? expf(g[n * g_stride + h]) : 1.f;
    if (__syncthreads_or(taken)) {
        if (tid == 0) set_error(err, KDA_ERR_BAD_STATE_INDEX);
        return;
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const float kr = s_k[row0 + i * RPP], qr = s_q[row0 + i * RPP];
        // a state that the decay erases takes nothing from what it held (infinities there included)
        s[i].x = fmaf(kr, vc.x, a == 0.f ? 0.f : a * s[i].x);
        s[i].y = fmaf(kr, vc.y, a == 0.f ? 0.f : a * s[i].y);
        s[i].z = fmaf(kr, vc.z, a == 0.f ? 0.f : a * s[i].z);
        s[i].w = fmaf(kr, vc.w, a == 0.f ? 0.f : a * s[i].w);
        __stcs(reinterpret_cast<float4 *>(S + (int64_t)(row0 + i * RPP) * DV), s[i]);
        acc.x = fmaf(qr, s[i].x, acc.x);
        acc.y = fmaf(qr, s[i].y, acc.y);
        acc.z = fmaf(qr, s[i].z, acc.z);
        acc.w = fmaf(qr, s[i].w, acc.w);
    }
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1) {  // the rows of one warp
        acc.x += __shfl_xor_sync(0xffffffffu, acc.x, off);
        acc.y += __shfl_xor_sync(0xffffffffu, acc.y, off);
        acc.z += __shfl_xor_sync(0xffffffffu, acc.z, off);
        acc.w += __shfl_xor_sync(0xffffffffu, acc.w, off);
    }
    if (lane < LPR) s_part[tid >> 5][lane] = acc;
    __syncthreads();
    if (tid < CW) {
        float r = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) r += reinterpret_cast<const float *>(&s_part[w][0])[tid];
        st(o + (n * H + h) * DV + part * CW + tid, scale * r);
    }
}

template <int DK, int DV, int CW, typename T>
static void launch(const kda_linear_step_args *a, cudaStream_t stream, int *err) {
    const int64_t slots = a->num_slots > 0 ? a->num_slots : a->N;
    linear_step_kernel<DK, DV, CW, T><<<(unsigned)(a->N * a->H * (DV / CW)), 256, 0, stream>>>(
        (const T *)a->q, (const T *)a->k, (const T *)a->v, a->g, a->g_per_token ? a->H : 0, a->scale, a->state,
        a->state_indices, slots, a->H, a->H / a->Hq, a->H / a->Hk, a->H / a->Hv, (T *)a->o, err);
}

template <int DK, int DV, typename T>
static void launch_w(const kda_linear_step_args *a, cudaStream_t stream, int *err) {
    // Fewer states than half of the SMs: each is split into columns.  Measured, dk = dv = 128, 32 heads, split and
    // whole: 1 sequence 2.26 / 3.07 us, 4 sequences 3.69 / 3.08, 16 sequences 8.6 / 8.0, 32 sequences 15.0 / 13.7.
    if (a->N * a->H <= 76) launch<DK, DV, 32, T>(a, stream, err);
    else launch<DK, DV, DV, T>(a, stream, err);
}

template <typename T>
static void launch_t(const kda_linear_step_args *a, cudaStream_t stream, int *err) {
    if (a->dk == 128) {
        if (a->dv == 128) launch_w<128, 128, T>(a, stream, err); else launch_w<128, 64, T>(a, stream, err);
    } else {
        if (a->dv == 128) launch_w<64, 128, T>(a, stream, err); else launch_w<64, 64, T>(a, stream, err);
    }
}

}  // namespace lin
}  // namespace kda

kda_status_t kda_launch_linear_step(const kda_linear_step_args *a, cudaStream_t stream) {
    int *err = kda_device_error_ptr();
    if (!err) return KDA_ERR_CUDA;
    if (a->dtype == KDA_BF16) kda::lin::launch_t<kda::bf16>(a, stream, err);
    else kda::lin::launch_t<float>(a, stream, err);
    return kda_cuda_status(cudaGetLastError());
}
