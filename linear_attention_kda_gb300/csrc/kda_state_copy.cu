// kda_state_copy: dst_pool[dst[p]] <- src_pool[src[p]] for p = 0 .. P - 1, in this order (src -1: zeros).
//
// Bound by HBM traffic: every source read once, every target written once.  A thread owns one 16-byte place of a
// slot and applies the pairs to it in order, W at a time: it loads the W sources first, so that W copies are in
// flight, and where a source is the target of an earlier pair of the same W it takes that pair's value from its
// registers.  Earlier groups' stores are the thread's own, to the very addresses that it loads later, so program
// order alone makes the result that of one pair after the other: no workspace, no barrier between pairs, and chains,
// swaps through a spare slot and compactions onto slots that move themselves all come out right.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace slots {

constexpr int W = 8;

__global__ void __launch_bounds__(256) state_copy_kernel(const char *src_pool, char *dst_pool, int64_t slot_bytes,
                                                         int32_t src_slots, int32_t dst_slots, int64_t P,
                                                         const int32_t *__restrict__ src,
                                                         const int32_t *__restrict__ dst, int *err) {
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 16;
    const bool mine = at < slot_bytes, same = src_pool == dst_pool;
    for (int64_t p0 = 0; p0 < P; p0 += W) {
        int32_t s[W], d[W];
        uint4 x[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            s[i] = d[i] = -1;
            if (p0 + i < P) {
                s[i] = src[p0 + i];
                d[i] = dst[p0 + i];
            }
            if (s[i] < -1 || s[i] >= src_slots || d[i] < -1 || d[i] >= dst_slots) {
                if (at == 0) set_error(err, KDA_ERR_BAD_STATE_INDEX);
                d[i] = -1;
            }
        }
#pragma unroll
        for (int i = 0; i < W; ++i) {
            x[i] = make_uint4(0, 0, 0, 0);
            if (mine && d[i] >= 0 && s[i] >= 0)
                x[i] = *reinterpret_cast<const uint4 *>(src_pool + (int64_t)s[i] * slot_bytes + at);
        }
        if (same) {
#pragma unroll
            for (int i = 1; i < W; ++i)
#pragma unroll
                for (int j = 0; j < i; ++j)  // the last earlier writer wins
                    if (s[i] >= 0 && d[j] == s[i]) x[i] = x[j];
        }
        if (mine) {
#pragma unroll
            for (int i = 0; i < W; ++i)
                if (d[i] >= 0) *reinterpret_cast<uint4 *>(dst_pool + (int64_t)d[i] * slot_bytes + at) = x[i];
        }
    }
}

}  // namespace slots
}  // namespace kda

kda_status_t kda_launch_state_copy(const kda_state_copy_args *a, cudaStream_t stream) {
    int *err = kda_device_error_ptr();
    if (!err) return KDA_ERR_CUDA;
    const int64_t blocks = (a->slot_bytes / 16 + 255) / 256;
    if (blocks > INT32_MAX) return KDA_ERR_UNSUPPORTED_SHAPE;
    kda::slots::state_copy_kernel<<<(unsigned)blocks, 256, 0, stream>>>(
        (const char *)a->src_pool, (char *)a->dst_pool, a->slot_bytes, (int32_t)a->src_slots, (int32_t)a->dst_slots,
        a->P, a->src, a->dst, err);
    return kda_cuda_status(cudaGetLastError());
}
