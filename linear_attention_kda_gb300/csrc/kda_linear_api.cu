// C ABI of linear attention with a decay per head, state-slot copies and rotary positions: host-side
// validation and dispatch, as kda_api.cu does for the KDA calls.  Failing validation launches nothing.
#include <math.h>
#include <stdint.h>

#include "kda_checks.h"
#include "kda_common.cuh"
#include "kda_internal.h"

using namespace kda;

namespace {

bool dim_ok(int32_t d) { return d == 64 || d == 128; }

// sizes that every linear call checks; rows is T, or N for the step
kda_status_t check_sizes(int64_t rows, int64_t N, int32_t H, int32_t Hq, int32_t Hk, int32_t Hv, int32_t dk,
                         int32_t dv, kda_dtype_t dtype) {
    if (rows < 0 || N < 0 || H < 1 || Hq < 1 || Hk < 1 || Hv < 1) return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return KDA_ERR_UNSUPPORTED_DTYPE;
    if (H % Hq != 0 || H % Hk != 0 || H % Hv != 0 || (Hq != H && Hk != H && Hv != H)) return KDA_ERR_INVALID_ARG;
    if (!dim_ok(dk) || !dim_ok(dv)) return KDA_ERR_UNSUPPORTED_SHAPE;
    // slots of 64 tokens x heads (and every launch grid made of them) stay below 2^31
    if (rows > INT32_MAX || N > INT32_MAX || H > 65535) return KDA_ERR_UNSUPPORTED_SHAPE;
    if ((rows / 64 + N) * (int64_t)H > INT32_MAX / 4) return KDA_ERR_UNSUPPORTED_SHAPE;
    return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_linear_chunk_fwd_workspace_size(int64_t T, int64_t N, int32_t H, int32_t dk, int32_t dv,
                                           kda_dtype_t dtype) {
    if (N < 1 || check_sizes(T, N, H, H, H, H, dk, dv, dtype) != KDA_OK) return 0;
    return kda_linear_fwd_layout_bytes(T, N, H, dk, dv, dtype);
}

size_t kda_linear_chunk_bwd_workspace_size(int64_t T, int64_t N, int32_t H, int32_t Hq, int32_t Hk, int32_t Hv,
                                           int32_t dk, int32_t dv, kda_dtype_t dtype) {
    if (N < 1 || check_sizes(T, N, H, Hq, Hk, Hv, dk, dv, dtype) != KDA_OK) return 0;
    return kda_linear_bwd_layout_bytes(T, N, H, Hq, Hk, Hv, dk, dv, dtype);
}

kda_status_t kda_linear_chunk_fwd(const kda_linear_args *a, void *workspace, size_t workspace_bytes,
                                  struct CUstream_st *stream) {
    if (!a) return KDA_ERR_INVALID_ARG;
    kda_status_t st = check_sizes(a->T, a->N, a->H, a->Hq, a->Hk, a->Hv, a->dk, a->dv, a->dtype);
    if (st != KDA_OK) return st;
    if (a->N < 1 || !isfinite(a->scale) || (a->g_per_token != 0 && a->g_per_token != 1)) return KDA_ERR_INVALID_ARG;
    if (!a->cu_seqlens && a->T % a->N != 0) return KDA_ERR_INVALID_ARG;
    const int64_t es = dtype_size(a->dtype), state = a->N * a->H * (int64_t)a->dk * a->dv * 4;
    if (a->T > 0 && (!a->q || !a->k || !a->v || !a->o)) return KDA_ERR_INVALID_ARG;
    const range in[] = {{a->q, a->T * a->Hq * a->dk * es}, {a->k, a->T * a->Hk * a->dk * es},
                        {a->v, a->T * a->Hv * a->dv * es}, {a->g, (a->g_per_token ? a->T : 1) * a->H * 4},
                        {a->cu_seqlens, (a->N + 1) * 4}, {a->initial_state, state}};
    const range o{a->o, a->T * a->H * a->dv * es}, fs{a->final_state, state};
    for (int i = 0; i < 6; ++i) {
        if (overlap(o, in[i])) return KDA_ERR_INVALID_ARG;
        if (overlap(fs, in[i]) && !(i == 5 && a->final_state == a->initial_state)) return KDA_ERR_INVALID_ARG;
    }
    if (overlap(o, fs)) return KDA_ERR_INVALID_ARG;
    if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->o, 16) || !aligned(a->g, 4) ||
        !aligned(a->cu_seqlens, 4) || !aligned(a->initial_state, 16) || !aligned(a->final_state, 16))
        return KDA_ERR_MISALIGNED;
    const size_t need = kda_linear_fwd_layout_bytes(a->T, a->N, a->H, a->dk, a->dv, a->dtype);
    if (workspace_bytes < need || (need > 0 && !workspace)) return KDA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return KDA_ERR_MISALIGNED;
    st = kda_check_device();
    if (st != KDA_OK) return st;
    st = kda_launch_linear_fwd(a, workspace, (cudaStream_t)stream);
    if (st == KDA_OK && (kda_debug_flags() & KDA_CHECK_FINITE)) {
        st = kda_check_finite(a->o, a->T * a->H * (int64_t)a->dv, a->dtype, (cudaStream_t)stream);
        if (st == KDA_OK) st = kda_check_finite(a->final_state, state / 4, KDA_F32, (cudaStream_t)stream);
    }
    return st;
}

kda_status_t kda_linear_chunk_bwd(const kda_linear_bwd_args *a, void *workspace, size_t workspace_bytes,
                                  struct CUstream_st *stream) {
    if (!a) return KDA_ERR_INVALID_ARG;
    kda_status_t st = check_sizes(a->T, a->N, a->H, a->Hq, a->Hk, a->Hv, a->dk, a->dv, a->dtype);
    if (st != KDA_OK) return st;
    if (a->N < 1 || !isfinite(a->scale) || (a->g_per_token != 0 && a->g_per_token != 1)) return KDA_ERR_INVALID_ARG;
    if (!a->cu_seqlens && a->T % a->N != 0) return KDA_ERR_INVALID_ARG;
    if (a->grad_g && !a->g) return KDA_ERR_INVALID_ARG;
    const int64_t es = dtype_size(a->dtype), state = a->N * a->H * (int64_t)a->dk * a->dv * 4;
    const int64_t gb = (a->g_per_token ? a->T : 1) * (int64_t)a->H * 4;
    const int64_t qb = a->T * a->Hq * a->dk * es, kb = a->T * a->Hk * a->dk * es, vb = a->T * a->Hv * a->dv * es;
    const range in[] = {{a->q, qb}, {a->k, kb}, {a->v, vb}, {a->grad_o, a->T * a->H * a->dv * es}, {a->g, gb},
                        {a->cu_seqlens, (a->N + 1) * 4}, {a->initial_state, state}, {a->grad_final_state, state}};
    const range out[] = {{a->grad_q, qb}, {a->grad_k, kb}, {a->grad_v, vb}, {a->grad_g, gb},
                         {a->grad_initial_state, state}};
    if (a->T > 0)
        for (int i = 0; i < 4; ++i)
            if (!in[i].p || (i < 3 && !out[i].p)) return KDA_ERR_INVALID_ARG;
    for (int i = 0; i < 5; ++i) {
        for (const range &r : in)
            if (overlap(out[i], r)) return KDA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 5; ++j)
            if (overlap(out[i], out[j])) return KDA_ERR_INVALID_ARG;
    }
    for (int i = 0; i < 8; ++i)
        if (!aligned(in[i].p, i == 4 || i == 5 ? 4 : 16)) return KDA_ERR_MISALIGNED;
    for (int i = 0; i < 5; ++i)
        if (!aligned(out[i].p, i == 3 ? 4 : 16)) return KDA_ERR_MISALIGNED;
    const size_t need = kda_linear_bwd_layout_bytes(a->T, a->N, a->H, a->Hq, a->Hk, a->Hv, a->dk, a->dv, a->dtype);
    if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return KDA_ERR_MISALIGNED;
    st = kda_check_device();
    if (st != KDA_OK) return st;
    st = kda_launch_linear_bwd(a, workspace, (cudaStream_t)stream);
    if (st == KDA_OK && (kda_debug_flags() & KDA_CHECK_FINITE)) {
        for (int i = 0; i < 5 && st == KDA_OK; ++i) {
            const bool io = i < 3;
            if (aligned(out[i].p, 16))
                st = kda_check_finite(out[i].p, out[i].bytes / (io ? es : 4), io ? a->dtype : KDA_F32,
                                      (cudaStream_t)stream);
        }
    }
    return st;
}

kda_status_t kda_linear_recurrent_step(const kda_linear_step_args *a, struct CUstream_st *stream) {
    if (!a) return KDA_ERR_INVALID_ARG;
    kda_status_t st = check_sizes(a->N, a->N, a->H, a->Hq, a->Hk, a->Hv, a->dk, a->dv, a->dtype);
    if (st != KDA_OK) return st;
    if (!isfinite(a->scale) || (a->g_per_token != 0 && a->g_per_token != 1) || a->num_slots < 0)
        return KDA_ERR_INVALID_ARG;
    if (a->N == 0) return KDA_OK;
    if (!a->q || !a->k || !a->v || !a->o || !a->state) return KDA_ERR_INVALID_ARG;
    if (!a->state_indices && a->num_slots != 0 && a->num_slots < a->N) return KDA_ERR_INVALID_ARG;
    const int64_t slots = a->num_slots ? a->num_slots : a->N, es = dtype_size(a->dtype);
    const int64_t per_slot = (int64_t)a->H * a->dk * a->dv;
    if (slots > INT32_MAX || !pool_ok(slots, per_slot * 4)) return KDA_ERR_UNSUPPORTED_SHAPE;
    const range in[] = {{a->q, a->N * a->Hq * a->dk * es}, {a->k, a->N * a->Hk * a->dk * es},
                        {a->v, a->N * a->Hv * a->dv * es}, {a->g, (a->g_per_token ? a->N : 1) * a->H * 4},
                        {a->state_indices, a->N * 4}};
    const range o{a->o, a->N * a->H * a->dv * es}, state{a->state, slots * per_slot * 4};
    for (const range &r : in)
        if (overlap(o, r) || overlap(state, r)) return KDA_ERR_INVALID_ARG;
    if (overlap(o, state)) return KDA_ERR_INVALID_ARG;
    if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->o, 16) || !aligned(a->g, 4) ||
        !aligned(a->state, 16) || !aligned(a->state_indices, 4))
        return KDA_ERR_MISALIGNED;
    st = kda_check_device();
    if (st != KDA_OK) return st;
    st = kda_launch_linear_step(a, (cudaStream_t)stream);
    if (st == KDA_OK && (kda_debug_flags() & KDA_CHECK_FINITE)) {
        // (the rows and slots of this call: an unused row's output and other slots may hold anything)
        const int64_t row = (int64_t)a->H * a->dv;
        st = kda_check_finite_rows(a->o, row, a->N, a->state_indices, nullptr, slots, a->dtype, (cudaStream_t)stream);
        if (st == KDA_OK)
            st = kda_check_finite_rows(a->state, per_slot, a->N, a->state_indices, a->state_indices, slots, KDA_F32,
                                       (cudaStream_t)stream);
    }
    return st;
}

kda_status_t kda_state_copy(const kda_state_copy_args *a, struct CUstream_st *stream) {
    if (!a) return KDA_ERR_INVALID_ARG;
    if (a->P < 0 || a->src_slots < 0 || a->dst_slots < 0 || a->slot_bytes < 0) return KDA_ERR_INVALID_ARG;
    if (a->P > INT32_MAX || a->src_slots > INT32_MAX || a->dst_slots > INT32_MAX || a->slot_bytes % 16 != 0 ||
        !pool_ok(a->src_slots, a->slot_bytes) || !pool_ok(a->dst_slots, a->slot_bytes))
        return KDA_ERR_UNSUPPORTED_SHAPE;
    if (a->P == 0 || a->slot_bytes == 0) return KDA_OK;
    if (!a->src || !a->dst || !a->dst_pool || (!a->src_pool && a->src_slots > 0)) return KDA_ERR_INVALID_ARG;
    const range s{a->src_pool, a->src_slots * a->slot_bytes}, d{a->dst_pool, a->dst_slots * a->slot_bytes};
    if (a->src_pool == a->dst_pool && a->src_slots != a->dst_slots) return KDA_ERR_INVALID_ARG;
    if (a->src_pool != a->dst_pool && overlap(s, d)) return KDA_ERR_INVALID_ARG;
    if (overlap({a->src, a->P * 4}, d) || overlap({a->dst, a->P * 4}, d)) return KDA_ERR_INVALID_ARG;
    if (!aligned(a->src_pool, 16) || !aligned(a->dst_pool, 16) || !aligned(a->src, 4) || !aligned(a->dst, 4))
        return KDA_ERR_MISALIGNED;
    const kda_status_t st = kda_check_device();
    return st != KDA_OK ? st : kda_launch_state_copy(a, (cudaStream_t)stream);
}

kda_status_t kda_rope(const kda_rope_args *a, struct CUstream_st *stream) {
    if (!a) return KDA_ERR_INVALID_ARG;
    if (a->T < 0 || a->Hq < 0 || a->Hk < 0 || (a->Hq == 0 && a->Hk == 0)) return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(a->dtype)) return KDA_ERR_UNSUPPORTED_DTYPE;
    if (a->d < 2 || a->d > 1024 || a->rot < 2 || a->rot > 256 || a->rot > a->d || a->rot % 2 != 0 ||
        a->T > INT32_MAX || a->Hq > 1024 || a->Hk > 1024)
        return KDA_ERR_UNSUPPORTED_SHAPE;
    if ((a->layout != KDA_ROPE_HALF && a->layout != KDA_ROPE_INTERLEAVED) || (a->inverse != 0 && a->inverse != 1) ||
        !isfinite(a->scale) || !a->freqs)
        return KDA_ERR_INVALID_ARG;
    for (int i = 0; i < a->rot / 2; ++i)
        if (!(fabs(a->freqs[i]) <= 1e6)) return KDA_ERR_INVALID_ARG;
    if (a->T == 0) return KDA_OK;
    if (!a->positions) return KDA_ERR_INVALID_ARG;
    const int64_t es = dtype_size(a->dtype);
    const void *in[] = {a->q, a->k};
    void *out[] = {a->q_out, a->k_out};
    const int64_t row[] = {(int64_t)a->Hq * a->d, (int64_t)a->Hk * a->d};
    int64_t si[] = {a->q_stride, a->k_stride}, so[] = {a->q_out_stride, a->k_out_stride};
    for (int i = 0; i < 2; ++i) {
        if (row[i] == 0) continue;
        if (!in[i] || !out[i]) return KDA_ERR_INVALID_ARG;
        if (si[i] == 0) si[i] = row[i];
        if (so[i] == 0) so[i] = row[i];
        // rows may not overlap their neighbours; the largest offset stays far inside 64 bits
        if (si[i] < row[i] || so[i] < row[i] || si[i] > ((int64_t)1 << 30) || so[i] > ((int64_t)1 << 30))
            return KDA_ERR_INVALID_ARG;
        if (!aligned(in[i], es) || !aligned(out[i], es)) return KDA_ERR_MISALIGNED;
    }
    if (!aligned(a->positions, 4)) return KDA_ERR_MISALIGNED;
    // Two strided views overlap only where some row of one meets a row of the other.  Views of the same stride
    // (slices of one fused buffer) interleave without meeting when their offset, modulo the stride, leaves room.
    auto meet = [&](const void *p, int64_t sp, int64_t rp, const void *q, int64_t sq, int64_t rq) {
        const range x{p, ((a->T - 1) * sp + rp) * es}, y{q, ((a->T - 1) * sq + rq) * es};
        if (rp == 0 || rq == 0 || !overlap(x, y)) return false;
        if (sp != sq) return true;
        const int64_t stride = sp * es;
        int64_t off = ((int64_t)((uintptr_t)q - (uintptr_t)p)) % stride;
        if (off < 0) off += stride;
        return off < rp * es || off + rq * es > stride;
    };
    for (int i = 0; i < 2; ++i) {
        if (row[i] == 0) continue;
        for (int j = 0; j < 2; ++j) {
            const bool same = i == j && in[j] == out[i] && si[j] == so[i];
            if (row[j] && !same && meet(out[i], so[i], row[i], in[j], si[j], row[j])) return KDA_ERR_INVALID_ARG;
        }
        if (overlap({out[i], ((a->T - 1) * so[i] + row[i]) * es}, {a->positions, a->T * 4})) return KDA_ERR_INVALID_ARG;
    }
    if (row[0] && row[1] && meet(out[0], so[0], row[0], out[1], so[1], row[1])) return KDA_ERR_INVALID_ARG;
    kda_status_t st = kda_check_device();
    if (st != KDA_OK) return st;
    kda_rope_args b = *a;
    b.q_stride = si[0], b.k_stride = si[1], b.q_out_stride = so[0], b.k_out_stride = so[1];
    st = kda_launch_rope(&b, (cudaStream_t)stream);
    if (st == KDA_OK && (kda_debug_flags() & KDA_CHECK_FINITE))
        for (int i = 0; i < 2 && st == KDA_OK; ++i)
            if (row[i] && so[i] == row[i] && aligned(out[i], 16))
                st = kda_check_finite(out[i], a->T * row[i], a->dtype, (cudaStream_t)stream);
    return st;
}

}  // extern "C"
