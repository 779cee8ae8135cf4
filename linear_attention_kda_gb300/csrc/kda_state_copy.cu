// kda_state_copy: dst_pool[dst[p]] <- src_pool[src[p]] for p = 0 .. P - 1, in this order (src -1: zeros).
//
// Bound by HBM traffic: every source read once, every target written once.  A thread owns one 16-byte place of a
// slot and applies the pairs to it in order, W at a time: it loads the W sources first, so that W copies are in
// flight, and where a source is the target of an earlier pair of the same W it takes that pair's value from its
// registers.  Earlier groups' stores are the thread's own, to the very addresses that it loads later, so program
// order alone makes the result that of one pair after the other: no workspace, no barrier between pairs, and chains,
// swaps through a spare slot and compactions onto slots that move themselves all come out right.
//
// Slots too small to fill the GPU with their places alone also split the pairs over gridDim.y blocks.  That is the same
// only where the pairs do not touch one another, which every block finds out for itself from a bitmap of the targets;
// where they do, the blocks of the first row take all pairs.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace slots {

// 150 slots of 2 MB onto one another, one GB300: W = 4 in blocks of 64 threads 101 us (6.25 TB/s of traffic, 0.92 of a
// plain copy), 4 and 128: 104, 8 and 128: 110, 8 and 256: 114 (3.4 blocks for an SM), 16 and 128: 110.
constexpr int W = 4;
constexpr int NT = 64;
constexpr int MAP = 1 << 16;   // slots that the bitmap holds

__global__ void __launch_bounds__(NT) state_copy_kernel(const char *src_pool, char *dst_pool, int64_t slot_bytes,
                                                        int32_t src_slots, int32_t dst_slots, int64_t P,
                                                        const int32_t *__restrict__ src,
                                                        const int32_t *__restrict__ dst, int *err) {
    const int64_t at = ((int64_t)blockIdx.x * NT + threadIdx.x) * 16;
    const bool mine = at < slot_bytes, same = src_pool == dst_pool;
    int64_t first = 0, last = P;
    if (gridDim.y > 1) {
        __shared__ uint32_t targets[MAP / 32];
        for (int i = threadIdx.x; i < (dst_slots + 31) / 32; i += NT) targets[i] = 0;
        __syncthreads();
        bool meet = false;
        for (int64_t p = threadIdx.x; p < P; p += NT) {
            const int32_t s = src[p], d = dst[p];
            if (d < 0 || d >= dst_slots || s < -1 || s >= src_slots) continue;
            meet |= (atomicOr(&targets[d >> 5], 1u << (d & 31)) >> (d & 31)) & 1;
        }
        __syncthreads();
        for (int64_t p = threadIdx.x; p < P && same; p += NT) {
            const int32_t s = src[p], d = dst[p];
            meet |= s >= 0 && s < dst_slots && s != d && ((targets[s >> 5] >> (s & 31)) & 1);
        }
        if (__syncthreads_or(meet)) {
            if (blockIdx.y > 0) return;
        } else {
            const int64_t each = (P + gridDim.y - 1) / gridDim.y;
            first = blockIdx.y * each;
            last = first + each < P ? first + each : P;
        }
    }
    for (int64_t p0 = first; p0 < last; p0 += W) {
        int32_t s[W], d[W];
        uint4 x[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            s[i] = d[i] = -1;
            if (p0 + i < last) {
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
    using namespace kda::slots;
    const int64_t blocks = (a->slot_bytes / 16 + NT - 1) / NT;
    if (blocks > INT32_MAX) return KDA_ERR_UNSUPPORTED_SHAPE;
    // Pairs are split where the places of a slot make fewer than four blocks for an SM, W pairs to a block at least:
    // 150 slots of 32 KB moved take 4.1 us, one block for all pairs 25; of 256 KB 18 and 28, of 512 KB 50 either way.
    int64_t split = 608 / blocks, groups = (a->P + W - 1) / W;
    if (split > groups) split = groups;
    if (split < 1 || a->dst_slots > MAP) split = 1;
    state_copy_kernel<<<dim3((unsigned)blocks, (unsigned)split), NT, 0, stream>>>(
        (const char *)a->src_pool, (char *)a->dst_pool, a->slot_bytes, (int32_t)a->src_slots, (int32_t)a->dst_slots,
        a->P, a->src, a->dst, err);
    return kda_cuda_status(cudaGetLastError());
}
