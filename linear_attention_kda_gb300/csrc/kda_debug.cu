// Optional numeric checks (kda_set_debug_checks): after an entry point's kernels, one more pass over
// what it wrote sets KDA_ERR_NUMERIC in the device error word if any value is NaN or infinite.  Off
// by default; the checks read every output once more, so they cost one extra HBM pass.
#include <atomic>

#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {

// Whether 16 bytes hold a NaN or an infinity (exponent all ones).
template <typename T> __device__ __forceinline__ bool not_finite(const uint4 &u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (sizeof(T) == 4) bad |= (w[j] & 0x7F800000u) == 0x7F800000u;
        else bad |= ((w[j] & 0x7F80u) == 0x7F80u) || ((w[j] & 0x7F800000u) == 0x7F800000u);
    }
    return bad;
}

template <typename T> __device__ __forceinline__ bool not_finite(const T *p) {
    if (sizeof(T) == 4) return (*reinterpret_cast<const uint32_t *>(p) & 0x7F800000u) == 0x7F800000u;
    return (*reinterpret_cast<const uint16_t *>(p) & 0x7F80u) == 0x7F80u;
}

// Grid-stride scan for a non-finite value: 16-byte loads over the 16-byte-aligned body, scalars for
// the head and the tail.  bf16 is checked on its bit pattern (exponent all ones).
template <typename T>
__global__ void __launch_bounds__(256) check_finite_kernel(const T *__restrict__ p, int64_t n, int *err) {
    constexpr int PER = 16 / sizeof(T);
    int64_t head = (int64_t)((16 - ((uintptr_t)p & 15)) & 15) / sizeof(T);
    if (head > n) head = n;
    const int64_t nv = (n - head) / PER, first = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    bool bad = false;
    for (int64_t i = first; i < nv; i += stride) bad |= not_finite<T>(reinterpret_cast<const uint4 *>(p + head)[i]);
    for (int64_t i = first; i < head; i += stride) bad |= not_finite<T>(p + i);
    for (int64_t i = head + nv * PER + first; i < n; i += stride) bad |= not_finite<T>(p + i);
    if (__syncthreads_or(bad) && threadIdx.x == 0) set_error(err, KDA_ERR_NUMERIC);
}

// The rows that a call with state indices wrote, one after the other in every block.
template <typename T>
__global__ void __launch_bounds__(256) check_finite_rows_kernel(const T *__restrict__ p, int64_t len, int64_t N, const int32_t *used,
                                                                const int32_t *at, int64_t slots, int *err) {
    const bool wide = len % (16 / (int)sizeof(T)) == 0 && ((uintptr_t)p & 15) == 0;
    const int64_t per_row = len / (16 / (int)sizeof(T)), stride = (int64_t)gridDim.x * blockDim.x;
    bool bad = false;
    for (int64_t n = blockIdx.y; n < N; n += gridDim.y) {
        if (used && (used[n] < 0 || used[n] >= slots)) continue;
        const T *row = p + (at ? at[n] : n) * len;
        const int64_t first = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
        if (wide)
            for (int64_t i = first; i < per_row; i += stride) bad |= not_finite<T>(reinterpret_cast<const uint4 *>(row)[i]);
        else
            for (int64_t i = first; i < len; i += stride) bad |= not_finite<T>(row + i);
    }
    if (__syncthreads_or(bad) && threadIdx.x == 0) set_error(err, KDA_ERR_NUMERIC);
}

}  // namespace kda

namespace {
std::atomic<int32_t> g_debug_flags{0};
}

int32_t kda_debug_flags() { return g_debug_flags.load(std::memory_order_relaxed); }

kda_status_t kda_check_finite(const void *p, int64_t n, kda_dtype_t dtype, cudaStream_t stream) {
    if (!p || n <= 0) return KDA_OK;
    int *err = kda_device_error_ptr();
    if (!err) return KDA_ERR_CUDA;
    int dev = 0, sms = 152;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t per = dtype == KDA_BF16 ? 8 : 4;
    const int64_t want = (n / per + 255) / 256;
    const unsigned grid = (unsigned)(want < 4 * (int64_t)sms ? (want > 0 ? want : 1) : 4 * sms);
    if (dtype == KDA_BF16)
        kda::check_finite_kernel<kda::bf16><<<grid, 256, 0, stream>>>((const kda::bf16 *)p, n, err);
    else
        kda::check_finite_kernel<float><<<grid, 256, 0, stream>>>((const float *)p, n, err);
    return kda_cuda_status(cudaGetLastError());
}

kda_status_t kda_check_finite_rows(const void *p, int64_t len, int64_t N, const int32_t *used, const int32_t *at, int64_t slots,
                                   kda_dtype_t dtype, cudaStream_t stream) {
    if (!p || len <= 0 || N <= 0) return KDA_OK;
    int *err = kda_device_error_ptr();
    if (!err) return KDA_ERR_CUDA;
    const int64_t per_row = len / (dtype == KDA_BF16 ? 8 : 4), want = (per_row + 255) / 256;
    // (rows shorter than a vector have none of them, but a block)
    const dim3 grid((unsigned)(want < 1 ? 1 : want < 32 ? want : 32), (unsigned)(N < 1024 ? N : 1024));
    if (dtype == KDA_BF16)
        kda::check_finite_rows_kernel<kda::bf16><<<grid, 256, 0, stream>>>((const kda::bf16 *)p, len, N, used, at, slots, err);
    else
        kda::check_finite_rows_kernel<float><<<grid, 256, 0, stream>>>((const float *)p, len, N, used, at, slots, err);
    return kda_cuda_status(cudaGetLastError());
}

extern "C" kda_status_t kda_set_debug_checks(int32_t flags) {
    if (flags & ~KDA_CHECK_FINITE) return KDA_ERR_INVALID_ARG;
    g_debug_flags.store(flags, std::memory_order_relaxed);
    return KDA_OK;
}
