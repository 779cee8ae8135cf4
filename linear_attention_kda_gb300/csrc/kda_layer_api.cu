// C ABI of the gated recurrence over channels, the short convolution and the norms around a block: host-side
// validation and dispatch.  Failing validation launches nothing.
#include <math.h>
#include <stdint.h>

#include "kda_checks.h"
#include "kda_common.cuh"
#include "kda_internal.h"

using namespace kda;

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 30;

// Tokens of a call: positions some tiles behind the last one still fit in 32 bits.
constexpr int64_t kMaxTokens = INT32_MAX - 4095;

// Tokens and channels of a packed call.  Grids of (16 tokens x 32 channels) and the like stay below 2^31.
kda_status_t check_sizes(int64_t T, int64_t N, int32_t D, kda_dtype_t dtype) {
    if (T < 0 || N < 0 || D < 1) return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return KDA_ERR_UNSUPPORTED_DTYPE;
    if (T > kMaxTokens || N > kMaxTokens || D > (1 << 20)) return KDA_ERR_UNSUPPORTED_SHAPE;
    if ((T / 16 + N) * (int64_t)(D / 32 + 1) > INT32_MAX) return KDA_ERR_UNSUPPORTED_SHAPE;
    return KDA_OK;
}

// [rows, D] elements, rows a stride apart (0: D): its bytes, and whether the stride is one
bool strided(const void *p, int64_t rows, int64_t D, int64_t *stride, int64_t es, range *r) {
    if (*stride == 0) *stride = D;
    *r = {p, rows > 0 ? ((rows - 1) * *stride + D) * es : 0};
    return *stride >= D && *stride <= kMaxStride;
}

// no output may meet an input or another output; inputs[same[i]] may be output i itself
template <int NI, int NO>
bool apart(const range (&in)[NI], const range (&out)[NO], const int (&same)[NO]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (overlap(out[i], in[j]) && !(j == same[i] && out[i].p == in[j].p && out[i].bytes == in[j].bytes)) return false;
        for (int j = i + 1; j < NO; ++j)
            if (overlap(out[i], out[j])) return false;
    }
    return true;
}

kda_status_t check_scan(int32_t gate, int32_t input, float g_min, const float *A_log, const float *dt_bias) {
    if (gate < KDA_SCAN_LOWER_BOUND || gate > KDA_SCAN_LOG || input < KDA_SCAN_INPUT_PLAIN || input > KDA_SCAN_INPUT_NORM)
        return KDA_ERR_INVALID_ARG;
    if (gate == KDA_SCAN_LOWER_BOUND && !(g_min < 0.f && isfinite(g_min))) return KDA_ERR_INVALID_ARG;
    if (gate == KDA_SCAN_LOG && (A_log || dt_bias)) return KDA_ERR_INVALID_ARG;
    return aligned(A_log, 4) && aligned(dt_bias, 4) ? KDA_OK : KDA_ERR_MISALIGNED;
}

kda_status_t check_conv(int32_t D, int32_t K, int32_t activation, int32_t norm_dim, float eps, const float *weight, const float *bias) {
    if (K < 2 || K > 4) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (norm_dim != 0 && norm_dim != 32 && norm_dim != 64 && norm_dim != 128 && norm_dim != 256) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (activation != KDA_CONV_NONE && activation != KDA_CONV_SILU) return KDA_ERR_INVALID_ARG;
    if (norm_dim && (D % norm_dim != 0 || !(eps > 0.f) || !isfinite(eps))) return KDA_ERR_INVALID_ARG;
    if (!weight) return KDA_ERR_INVALID_ARG;
    return aligned(weight, 4) && aligned(bias, 4) ? KDA_OK : KDA_ERR_MISALIGNED;
}

kda_status_t finite(const void *p, int64_t n, kda_dtype_t t, struct CUstream_st *s) { return kda_check_finite(p, n, t, (cudaStream_t)s); }

}  // namespace

extern "C" {

size_t kda_scan_fwd_workspace_size(int64_t T, int64_t N, int32_t D, kda_dtype_t dtype) {
    return N < 1 || check_sizes(T, N, D, dtype) != KDA_OK ? 0 : kda_scan_fwd_bytes(T, N, D, dtype);
}

size_t kda_scan_bwd_workspace_size(int64_t T, int64_t N, int32_t D, kda_dtype_t dtype) {
    return N < 1 || check_sizes(T, N, D, dtype) != KDA_OK ? 0 : kda_scan_bwd_bytes(T, N, D, dtype);
}

kda_status_t kda_scan_fwd(const kda_scan_args *args, void *workspace, size_t workspace_bytes, struct CUstream_st *stream) {
    if (!args) return KDA_ERR_INVALID_ARG;
    kda_scan_args b = *args, *a = &b;
    kda_status_t st = check_sizes(a->T, a->N, a->D, a->dtype);
    if (st != KDA_OK) return st;
    if (a->N < 1 || (!a->cu_seqlens && a->T % a->N != 0)) return KDA_ERR_INVALID_ARG;
    st = check_scan(a->gate_kind, a->input_scale, a->g_min, a->A_log, a->dt_bias);
    if (st != KDA_OK) return st;
    if (a->T > 0 && (!a->x || !a->z || !a->h)) return KDA_ERR_INVALID_ARG;
    const int64_t es = dtype_size(a->dtype), state = a->N * a->D * 4, par = (int64_t)a->D * 4;
    range x, z, i;
    if (!strided(a->x, a->T, a->D, &a->x_stride, es, &x) || !strided(a->z, a->T, a->D, &a->z_stride, es, &z) ||
        !strided(a->input_gate, a->T, a->D, &a->i_stride, es, &i))
        return KDA_ERR_INVALID_ARG;
    const range in[] = {{a->initial_state, state}, x, z, i, {a->A_log, par}, {a->dt_bias, par}, {a->cu_seqlens, (a->N + 1) * 4}};
    const range out[] = {{a->final_state, state}, {a->h, a->T * a->D * es},
                         {a->checkpoints, (a->T / KDA_SCAN_CHECKPOINT + a->N) * a->D * 4}};
    if (!apart(in, out, {0, -1, -1})) return KDA_ERR_INVALID_ARG;
    if (!aligned(a->x, es) || !aligned(a->z, es) || !aligned(a->input_gate, es) || !aligned(a->h, es) ||
        !aligned(a->cu_seqlens, 4) || !aligned(a->initial_state, 4) || !aligned(a->final_state, 4) || !aligned(a->checkpoints, 4))
        return KDA_ERR_MISALIGNED;
    const size_t need = kda_scan_fwd_bytes(a->T, a->N, a->D, a->dtype);
    if (workspace_bytes < need || (need > 0 && !workspace)) return KDA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return KDA_ERR_MISALIGNED;
    st = kda_check_device();
    if (st != KDA_OK) return st;
    st = kda_launch_scan_fwd(a, workspace, (cudaStream_t)stream);
    if (st == KDA_OK && (kda_debug_flags() & KDA_CHECK_FINITE)) {
        st = finite(a->h, a->T * (int64_t)a->D, a->dtype, stream);
        if (st == KDA_OK) st = finite(a->final_state, state / 4, KDA_F32, stream);
    }
    return st;
}

kda_status_t kda_scan_bwd(const kda_scan_bwd_args *args, void *workspace, size_t workspace_bytes, struct CUstream_st *stream) {
    if (!args) return KDA_ERR_INVALID_ARG;
    kda_scan_bwd_args b = *args, *a = &b;
    kda_status_t st = check_sizes(a->T, a->N, a->D, a->dtype);
    if (st != KDA_OK) return st;
    if (a->N < 1 || (!a->cu_seqlens && a->T % a->N != 0)) return KDA_ERR_INVALID_ARG;
    st = check_scan(a->gate_kind, a->input_scale, a->g_min, a->A_log, a->dt_bias);
    if (st != KDA_OK) return st;
    if (a->gate_kind == KDA_SCAN_LOG && (a->grad_A_log || a->grad_dt_bias)) return KDA_ERR_INVALID_ARG;
    if (!a->input_gate != !a->grad_input_gate && a->T > 0) return KDA_ERR_INVALID_ARG;
    if (a->T > 0 && (!a->x || !a->z || !a->grad_h || !a->checkpoints || !a->grad_x || !a->grad_z)) return KDA_ERR_INVALID_ARG;
    const int64_t es = dtype_size(a->dtype), state = a->N * a->D * 4, par = (int64_t)a->D * 4, tok = a->T * a->D * es;
    range x, z, i;
    if (!strided(a->x, a->T, a->D, &a->x_stride, es, &x) || !strided(a->z, a->T, a->D, &a->z_stride, es, &z) ||
        !strided(a->input_gate, a->T, a->D, &a->i_stride, es, &i))
        return KDA_ERR_INVALID_ARG;
    const range in[] = {x, z, i, {a->A_log, par}, {a->dt_bias, par}, {a->cu_seqlens, (a->N + 1) * 4}, {a->grad_h, tok},
                        {a->checkpoints, (a->T / KDA_SCAN_CHECKPOINT + a->N) * a->D * 4}, {a->grad_final_state, state}};
    const range out[] = {{a->grad_x, tok}, {a->grad_z, tok}, {a->grad_input_gate, tok}, {a->grad_A_log, par},
                         {a->grad_dt_bias, par}, {a->grad_initial_state, state}};
    if (!apart(in, out, {-1, -1, -1, -1, -1, -1})) return KDA_ERR_INVALID_ARG;
    if (!aligned(a->x, es) || !aligned(a->z, es) || !aligned(a->input_gate, es)) return KDA_ERR_MISALIGNED;
    for (int k = 5; k < 9; ++k)
        if (!aligned(in[k].p, k == 6 ? es : 4)) return KDA_ERR_MISALIGNED;
    for (int k = 0; k < 6; ++k)
        if (!aligned(out[k].p, k < 3 ? es : 4)) return KDA_ERR_MISALIGNED;
    const size_t need = kda_scan_bwd_bytes(a->T, a->N, a->D, a->dtype);
    if (workspace_bytes < need || (need > 0 && !workspace)) return KDA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return KDA_ERR_MISALIGNED;
    st = kda_check_device();
    if (st != KDA_OK) return st;
    st = kda_launch_scan_bwd(a, workspace, (cudaStream_t)stream);
    if (kda_debug_flags() & KDA_CHECK_FINITE)
        for (int k = 0; k < 6 && st == KDA_OK; ++k)
            st = finite(out[k].p, out[k].bytes / (k < 3 ? es : 4), k < 3 ? a->dtype : KDA_F32, stream);
    return st;
}

kda_status_t kda_scan_step(const kda_scan_step_args *args, struct CUstream_st *stream) {
    if (!args) return KDA_ERR_INVALID_ARG;
    kda_scan_step_args b = *args, *a = &b;
    kda_status_t st = check_sizes(a->N, a->N, a->D, a->dtype);
    if (st != KDA_OK) return st;
    st = check_scan(a->gate_kind, a->input_scale, a->g_min, a->A_log, a->dt_bias);
    if (st != KDA_OK) return st;
    if (a->num_slots < 0) return KDA_ERR_INVALID_ARG;
    if (a->N == 0) return KDA_OK;
    if (!a->x || !a->z || !a->h || !a->state) return KDA_ERR_INVALID_ARG;
    if (!a->state_indices && a->num_slots != 0 && a->num_slots < a->N) return KDA_ERR_INVALID_ARG;
    if (a->num_slots == 0) a->num_slots = a->N;
    const int64_t es = dtype_size(a->dtype), par = (int64_t)a->D * 4;
    if (a->num_slots > INT32_MAX || !pool_ok(a->num_slots, par)) return KDA_ERR_UNSUPPORTED_SHAPE;
    range x, z, i;
    if (!strided(a->x, a->N, a->D, &a->x_stride, es, &x) || !strided(a->z, a->N, a->D, &a->z_stride, es, &z) ||
        !strided(a->input_gate, a->N, a->D, &a->i_stride, es, &i))
        return KDA_ERR_INVALID_ARG;
    const range in[] = {x, z, i, {a->A_log, par}, {a->dt_bias, par}, {a->state_indices, a->N * 4}};
    const range out[] = {{a->state, a->num_slots * par}, {a->h, a->N * a->D * es}};
    if (!apart(in, out, {-1, -1})) return KDA_ERR_INVALID_ARG;
    if (!aligned(a->x, es) || !aligned(a->z, es) || !aligned(a->input_gate, es) || !aligned(a->h, es) || !aligned(a->state, 4) ||
        !aligned(a->state_indices, 4))
        return KDA_ERR_MISALIGNED;
    st = kda_check_device();
    if (st != KDA_OK) return st;
    st = kda_launch_scan_step(a, (cudaStream_t)stream);
    if (st == KDA_OK && (kda_debug_flags() & KDA_CHECK_FINITE)) {
        st = kda_check_finite_rows(a->h, a->D, a->N, a->state_indices, nullptr, a->num_slots, a->dtype, (cudaStream_t)stream);
        if (st == KDA_OK)
            st = kda_check_finite_rows(a->state, a->D, a->N, a->state_indices, a->state_indices, a->num_slots, KDA_F32,
                                       (cudaStream_t)stream);
    }
    return st;
}

kda_status_t kda_short_conv_fwd(const kda_short_conv_args *args, struct CUstream_st *stream) {
    if (!args) return KDA_ERR_INVALID_ARG;
    kda_short_conv_args b = *args, *a = &b;
    kda_status_t st = check_sizes(a->T, a->N, a->D, a->dtype);
    if (st != KDA_OK) return st;
    if (a->N < 1 || (!a->cu_seqlens && a->T % a->N != 0)) return KDA_ERR_INVALID_ARG;
    st = check_conv(a->D, a->K, a->activation, a->norm_dim, a->norm_eps, a->weight, a->bias);
    if (st != KDA_OK) return st;
    if (a->T > 0 && (!a->x || !a->y)) return KDA_ERR_INVALID_ARG;
    const int64_t es = dtype_size(a->dtype), hist = a->N * (a->K - 1) * a->D * es, par = (int64_t)a->D * 4;
    range x;
    if (!strided(a->x, a->T, a->D, &a->x_stride, es, &x)) return KDA_ERR_INVALID_ARG;
    const range in[] = {{a->initial_state, hist}, x, {a->weight, par * a->K}, {a->bias, par}, {a->cu_seqlens, (a->N + 1) * 4}};
    const range out[] = {{a->final_state, hist}, {a->y, a->T * a->D * es}};
    if (!apart(in, out, {0, -1})) return KDA_ERR_INVALID_ARG;
    if (!aligned(a->x, es) || !aligned(a->y, es) || !aligned(a->initial_state, es) || !aligned(a->final_state, es) ||
        !aligned(a->cu_seqlens, 4))
        return KDA_ERR_MISALIGNED;
    st = kda_check_device();
    if (st != KDA_OK) return st;
    st = kda_launch_short_conv_fwd(a, (cudaStream_t)stream);
    if (st == KDA_OK && (kda_debug_flags() & KDA_CHECK_FINITE)) {
        st = finite(a->y, a->T * (int64_t)a->D, a->dtype, stream);
        if (st == KDA_OK) st = finite(a->final_state, hist / es, a->dtype, stream);
    }
    return st;
}

size_t kda_short_conv_bwd_workspace_size(int64_t T, int64_t N, int32_t D, int32_t K, kda_dtype_t dtype) {
    return N < 1 || K < 2 || K > 4 || check_sizes(T, N, D, dtype) != KDA_OK ? 0 : kda_short_conv_bwd_bytes(T, N, D, K);
}

kda_status_t kda_short_conv_bwd(const kda_short_conv_bwd_args *args, void *workspace, size_t workspace_bytes,
                                struct CUstream_st *stream) {
    if (!args) return KDA_ERR_INVALID_ARG;
    kda_short_conv_bwd_args b = *args, *a = &b;
    kda_status_t st = check_sizes(a->T, a->N, a->D, a->dtype);
    if (st != KDA_OK) return st;
    if (a->N < 1 || (!a->cu_seqlens && a->T % a->N != 0)) return KDA_ERR_INVALID_ARG;
    st = check_conv(a->D, a->K, a->activation, a->norm_dim, a->norm_eps, a->weight, a->bias);
    if (st != KDA_OK) return st;
    if (a->T > 0 && (!a->x || !a->grad_y || !a->grad_x)) return KDA_ERR_INVALID_ARG;
    const int64_t es = dtype_size(a->dtype), hist = a->N * (a->K - 1) * a->D * es, par = (int64_t)a->D * 4, tok = a->T * a->D * es;
    range x;
    if (!strided(a->x, a->T, a->D, &a->x_stride, es, &x)) return KDA_ERR_INVALID_ARG;
    const range in[] = {x, {a->weight, par * a->K}, {a->bias, par}, {a->cu_seqlens, (a->N + 1) * 4}, {a->initial_state, hist},
                        {a->grad_y, tok}, {a->grad_final_state, hist}};
    const range out[] = {{a->grad_x, tok}, {a->grad_initial_state, hist}, {a->grad_weight, par * a->K}, {a->grad_bias, par}};
    if (!apart(in, out, {-1, -1, -1, -1})) return KDA_ERR_INVALID_ARG;
    for (int k = 0; k < 7; ++k)
        if (!aligned(in[k].p, k >= 1 && k <= 3 ? 4 : es)) return KDA_ERR_MISALIGNED;
    for (int k = 0; k < 4; ++k)
        if (!aligned(out[k].p, k < 2 ? es : 4)) return KDA_ERR_MISALIGNED;
    const size_t need = kda_short_conv_bwd_bytes(a->T, a->N, a->D, a->K);
    if (workspace_bytes < need || (need > 0 && !workspace)) return KDA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return KDA_ERR_MISALIGNED;
    st = kda_check_device();
    if (st != KDA_OK) return st;
    st = kda_launch_short_conv_bwd(a, workspace, (cudaStream_t)stream);
    if (kda_debug_flags() & KDA_CHECK_FINITE)
        for (int k = 0; k < 4 && st == KDA_OK; ++k)
            st = finite(out[k].p, out[k].bytes / (k < 2 ? es : 4), k < 2 ? a->dtype : KDA_F32, stream);
    return st;
}

kda_status_t kda_short_conv_step(const kda_short_conv_step_args *args, struct CUstream_st *stream) {
    if (!args) return KDA_ERR_INVALID_ARG;
    kda_short_conv_step_args b = *args, *a = &b;
    kda_status_t st = check_sizes(a->N, a->N, a->D, a->dtype);
    if (st != KDA_OK) return st;
    st = check_conv(a->D, a->K, a->activation, a->norm_dim, a->norm_eps, a->weight, a->bias);
    if (st != KDA_OK) return st;
    if (a->num_slots < 0) return KDA_ERR_INVALID_ARG;
    if (a->N == 0) return KDA_OK;
    if (!a->x || !a->y || !a->state) return KDA_ERR_INVALID_ARG;
    if (!a->state_indices && a->num_slots != 0 && a->num_slots < a->N) return KDA_ERR_INVALID_ARG;
    if (a->num_slots == 0) a->num_slots = a->N;
    const int64_t es = dtype_size(a->dtype), par = (int64_t)a->D * 4, slot = (a->K - 1) * a->D * es;
    if (a->num_slots > INT32_MAX || !pool_ok(a->num_slots, slot)) return KDA_ERR_UNSUPPORTED_SHAPE;
    range x;
    if (!strided(a->x, a->N, a->D, &a->x_stride, es, &x)) return KDA_ERR_INVALID_ARG;
    const range in[] = {x, {a->weight, par * a->K}, {a->bias, par}, {a->state_indices, a->N * 4}};
    const range out[] = {{a->state, a->num_slots * slot}, {a->y, a->N * a->D * es}};
    if (!apart(in, out, {-1, -1})) return KDA_ERR_INVALID_ARG;
    if (!aligned(a->x, es) || !aligned(a->y, es) || !aligned(a->state, es) || !aligned(a->state_indices, 4)) return KDA_ERR_MISALIGNED;
    st = kda_check_device();
    if (st != KDA_OK) return st;
    st = kda_launch_short_conv_step(a, (cudaStream_t)stream);
    if (st == KDA_OK && (kda_debug_flags() & KDA_CHECK_FINITE)) {
        st = kda_check_finite_rows(a->y, a->D, a->N, a->state_indices, nullptr, a->num_slots, a->dtype, (cudaStream_t)stream);
        if (st == KDA_OK)
            st = kda_check_finite_rows(a->state, slot / es, a->N, a->state_indices, a->state_indices, a->num_slots, a->dtype,
                                       (cudaStream_t)stream);
    }
    return st;
}

static kda_status_t check_norm(int64_t T, int32_t D, kda_dtype_t dtype, kda_dtype_t residual_dtype) {
    if (T < 0 || D < 1) return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || (residual_dtype != dtype && residual_dtype != KDA_F32)) return KDA_ERR_UNSUPPORTED_DTYPE;
    return T > INT32_MAX || D > 8192 ? KDA_ERR_UNSUPPORTED_SHAPE : KDA_OK;
}

// the options of a call, as both directions take them
static kda_status_t check_norm_parts(int32_t gate_kind, int32_t post_norm, int32_t pre_norm, float eps, float scale, const float *scale_vec,
                                     bool block, bool gate, const float *post_weight, const float *pre_weight) {
    if (gate_kind < KDA_NORM_GATE_NONE || gate_kind > KDA_NORM_GATE_TOKEN || (post_norm != 0 && post_norm != 1) ||
        (pre_norm != 0 && pre_norm != 1) || !(eps > 0.f) || !isfinite(eps) || !isfinite(scale))
        return KDA_ERR_INVALID_ARG;
    if (gate != (gate_kind != KDA_NORM_GATE_NONE) || (post_weight && !post_norm) || (pre_weight && !pre_norm)) return KDA_ERR_INVALID_ARG;
    if (!block && (gate_kind != KDA_NORM_GATE_NONE || post_norm || scale_vec || !pre_norm)) return KDA_ERR_INVALID_ARG;
    return aligned(scale_vec, 4) && aligned(post_weight, 4) && aligned(pre_weight, 4) ? KDA_OK : KDA_ERR_MISALIGNED;
}

kda_status_t kda_block_norm_fwd(const kda_block_norm_args *a, struct CUstream_st *stream) {
    if (!a) return KDA_ERR_INVALID_ARG;
    kda_status_t st = check_norm(a->T, a->D, a->dtype, a->residual_dtype);
    if (st != KDA_OK) return st;
    // an empty call may leave every token tensor out
    const bool some = a->T > 0;
    st = check_norm_parts(a->gate_kind, a->post_norm, a->pre_norm, a->eps, a->scale, a->scale_vec, some ? a->y != nullptr : true,
                          some ? a->gate != nullptr : a->gate_kind != KDA_NORM_GATE_NONE, a->post_weight, a->pre_weight);
    if (st != KDA_OK) return st;
    if (!some) return KDA_OK;
    if (!a->residual || !a->y != !a->residual_out || !a->pre_norm != !a->normed) return KDA_ERR_INVALID_ARG;
    const int64_t es = dtype_size(a->dtype), rs = dtype_size(a->residual_dtype), n = a->T * a->D, par = (int64_t)a->D * 4;
    const range in[] = {{a->residual, n * rs}, {a->y, n * es}, {a->gate, (a->gate_kind == KDA_NORM_GATE_TOKEN ? a->T : n) * es},
                        {a->scale_vec, par}, {a->post_weight, par}, {a->pre_weight, par}};
    const range out[] = {{a->residual_out, n * rs}, {a->normed, n * es}};
    if (!apart(in, out, {0, 1})) return KDA_ERR_INVALID_ARG;
    if (!aligned(a->residual, rs) || !aligned(a->residual_out, rs) || !aligned(a->y, es) || !aligned(a->gate, es) || !aligned(a->normed, es))
        return KDA_ERR_MISALIGNED;
    st = kda_check_device();
    if (st != KDA_OK) return st;
    st = kda_launch_block_norm_fwd(a, (cudaStream_t)stream);
    if (st == KDA_OK && (kda_debug_flags() & KDA_CHECK_FINITE)) {
        st = finite(a->residual_out, n, a->residual_dtype, stream);
        if (st == KDA_OK) st = finite(a->normed, n, a->dtype, stream);
    }
    return st;
}

size_t kda_block_norm_bwd_workspace_size(int64_t T, int32_t D, kda_dtype_t dtype) {
    return check_norm(T, D, dtype, KDA_F32) != KDA_OK ? 0 : kda_block_norm_bwd_bytes(T, D);
}

kda_status_t kda_block_norm_bwd(const kda_block_norm_bwd_args *a, void *workspace, size_t workspace_bytes, struct CUstream_st *stream) {
    if (!a) return KDA_ERR_INVALID_ARG;
    kda_status_t st = check_norm(a->T, a->D, a->dtype, a->residual_dtype);
    if (st != KDA_OK) return st;
    const bool some = a->T > 0;
    st = check_norm_parts(a->gate_kind, a->post_norm, a->pre_norm, a->eps, a->scale, a->scale_vec, some ? a->y != nullptr : true,
                          some ? a->gate != nullptr : a->gate_kind != KDA_NORM_GATE_NONE, a->post_weight, a->pre_weight);
    if (st != KDA_OK) return st;
    if (some && (!a->residual || !a->grad_residual || !a->y != !a->grad_y || !a->gate != !a->grad_gate)) return KDA_ERR_INVALID_ARG;
    if ((a->grad_post_weight && !a->post_norm) || (a->grad_pre_weight && !a->pre_norm) || (a->grad_normed && !a->pre_norm) ||
        (a->grad_scale && some && !a->y))
        return KDA_ERR_INVALID_ARG;
    const int64_t es = dtype_size(a->dtype), rs = dtype_size(a->residual_dtype), n = a->T * a->D, par = (int64_t)a->D * 4;
    const int64_t gate = (a->gate_kind == KDA_NORM_GATE_TOKEN ? a->T : n) * es;
    // (grad_y may be y or grad_normed: two entries of the list of inputs, so it is looked at by itself)
    const range in[] = {{a->residual, n * rs}, {a->grad_residual_out, n * rs}, {a->y, n * es}, {a->grad_normed, n * es}, {a->gate, gate},
                        {a->scale_vec, par}, {a->post_weight, par}, {a->pre_weight, par}};
    const range out[] = {{a->grad_residual, n * rs}, {a->grad_gate, gate}, {a->grad_post_weight, par}, {a->grad_pre_weight, par},
                         {a->grad_scale, par}};
    if (!apart(in, out, {1, -1, -1, -1, -1})) return KDA_ERR_INVALID_ARG;
    const range gy{a->grad_y, n * es};
    for (const range &r : in)
        if (overlap(gy, r) && !((r.p == a->y || r.p == a->grad_normed) && r.p == a->grad_y && r.bytes == gy.bytes)) return KDA_ERR_INVALID_ARG;
    for (const range &r : out)
        if (overlap(gy, r)) return KDA_ERR_INVALID_ARG;
    if (!aligned(a->residual, rs) || !aligned(a->grad_residual_out, rs) || !aligned(a->grad_residual, rs) || !aligned(a->y, es) ||
        !aligned(a->grad_normed, es) || !aligned(a->gate, es) || !aligned(a->grad_y, es) || !aligned(a->grad_gate, es) ||
        !aligned(a->grad_post_weight, 4) || !aligned(a->grad_pre_weight, 4) || !aligned(a->grad_scale, 4))
        return KDA_ERR_MISALIGNED;
    const size_t need = kda_block_norm_bwd_bytes(a->T, a->D);
    if (workspace_bytes < need || (need > 0 && !workspace)) return KDA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return KDA_ERR_MISALIGNED;
    st = kda_check_device();
    if (st != KDA_OK) return st;
    st = kda_launch_block_norm_bwd(a, workspace, (cudaStream_t)stream);
    if (kda_debug_flags() & KDA_CHECK_FINITE) {
        if (st == KDA_OK) st = finite(a->grad_y, n, a->dtype, stream);
        for (int k = 0; k < 5 && st == KDA_OK; ++k)
            st = finite(out[k].p, out[k].bytes / (k == 0 ? rs : k == 1 ? es : 4), k == 0 ? a->residual_dtype : k == 1 ? a->dtype : KDA_F32,
                        stream);
    }
    return st;
}

}  // extern "C"
