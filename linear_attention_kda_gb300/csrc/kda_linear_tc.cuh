// Shared by the tensor-core kernels of linear attention with a decay per head (bf16 tensors, chunks of 128 tokens):
// tile maps, the decays of a chunk as its kernels use them, and the roles that every chain of chunks has.
#pragma once
#include <cuda.h>

#include "kda_internal.h"
#include "kda_linear.cuh"
#include "tc_util.cuh"

namespace kda {
namespace lin {
namespace tcl {

using namespace kda::tc;

constexpr int C = 128;       // tokens of a chunk: M of every product over tokens
constexpr int BLK = 32;      // tokens of a decay block (one warp's rows)

// The decays of one chunk.  With G the cumulative log-decay and E_b its value at the end of 32-token block b,
//     rel_j = G_j - E_{b-1} (from the start of j's block),   w_j = e^{E_b - G_j},
//     e^{G_r - G_j} = e^{G_r - E_b} w_j for j's block b before r's,   e^{rel_r - rel_j} inside one block,
// so that 128 x 128 masked decays take 32 + 3 exponentials a row, and a factor never exceeds 1 (for decays).  Only
// inside a block is a difference of two rounded values formed, off by 2^-24 of the block's whole log-decay, and that
// goes into bf16 products alone.  A NaN reaches the tokens from its own on, through rel, and what follows its block.
struct decays {
    float rel[C];
    float w[C];
    float hi[4], lo[4];  // E_b as fp32 pairs
};
__device__ __forceinline__ float ends(const decays &d, int a, int b) {  // E_a - E_b; E_{-1} = 0
    if (a < 0) return b < 0 ? 0.f : -d.hi[b];
    return b < 0 ? d.hi[a] : (d.hi[a] - d.hi[b]) + (d.lo[a] - d.lo[b]);
}
// One warp computes a chunk's decays, four tokens a lane, from log-decays that it has loaded before.
__device__ __forceinline__ float4 load_log_decays(const float *g, int g_stride, int len) {
    const int r = (threadIdx.x & 31) * 4;
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = g && r + i < len ? __ldg(g + (int64_t)(r + i) * g_stride) : 0.f;
    return make_float4(x[0], x[1], x[2], x[3]);
}
// (rel_lo: what rel leaves out of G_j - E_{b-1}, where fp32 results are made from differences inside a block.)
__device__ __forceinline__ void make_decays(const float4 &g, decays &d, float *rel_lo = nullptr) {
    const int lane = threadIdx.x & 31;
    const float in[4] = {g.x, g.y, g.z, g.w};
    ff x[4], pre;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const ff y{clamp_decay(in[i]), 0.f};
        x[i] = i ? ff_add(x[i - 1], y) : y;
    }
    pre = x[3];  // up to and with this lane
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const ff y = ff_shfl(pre, lane - off);
        if (lane >= off) pre = ff_add(y, pre);
    }
    const ff end = ff_shfl(pre, lane | 7);  // at the block's last lane
    ff before = ff_shfl(pre, lane - 1);
    if (lane == 0) before = {0.f, 0.f};
    const ff start = ff_shfl(before, lane & 24);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const ff G = ff_add(before, x[i]);
        const ff R = ff_add(G, {-start.h, -start.l});
        d.rel[lane * 4 + i] = R.h;
        if (rel_lo) rel_lo[lane * 4 + i] = R.l;
        d.w[lane * 4 + i] = expf(ff_diff(end, G));
    }
    if ((lane & 7) == 7) {
        d.hi[lane >> 3] = end.h;
        d.lo[lane >> 3] = end.l;
    }
    __syncwarp();
}

// A bounded wait in a few instructions (a chain's roles together have to fit the instruction cache, and every wait is
// a copy): attempts of about a microsecond each, given up after a million of them.
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity) {
    if (mbar_test_wait(bar, parity)) return true;
    uint32_t done;
#pragma unroll 1
    for (int n = 0; n < (1 << 20); ++n) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(done) : "r"(smem_u32(bar)), "r"(parity), "r"(1000u) : "memory");
        if (done) return true;
    }
    return false;
}

// [T, heads, D] bf16 as (channel, head, token), boxes of 64 channels x 1 head x 128 tokens, 128-byte swizzle: a box
// lands as the [128 tokens][64 channels] half of an operand tile.  Tokens past T read as zeros.
bool make_token_map(CUtensorMap *m, const void *base, int64_t T, int heads, int D);

// Chunks j0 .. j0 + N - 1 (16 bytes each) of row `row` of a [128][*] K-major tile times f, in place as its bf16 part,
// the rest of it to `rest`, by packed bf16 arithmetic: with f = fh + fl in two bf16 parts, hi = bf16(k fh + k fl),
// lo = bf16(k fl + (k fh - hi)).  Lost: 2^-16 of the row at most, 3e-6 of it on average.
template <int N>
__device__ __forceinline__ void scale_chunks(unsigned char *tile, unsigned char *rest, int row, int j0, float f) {
    const bf16 fh = __float2bfloat16_rn(f), fl = __float2bfloat16_rn(f - __bfloat162float(fh));
    const __nv_bfloat162 h2 = __halves2bfloat162(fh, fh), l2 = __halves2bfloat162(fl, fl);
    union chunk16 {
        uint4 u;
        __nv_bfloat162 p[4];
    } x[N], lo;
#pragma unroll
    for (int j = 0; j < N; ++j) x[j].u = *reinterpret_cast<const uint4 *>(tile + img_chunk_off(C, row, j0 + j));
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if (f == 0.f) x[j].u = make_uint4(0, 0, 0, 0);  // erased, whatever the row holds
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 hi = __hfma2(x[j].p[i], h2, __hmul2(x[j].p[i], l2));
            lo.p[i] = __hfma2(x[j].p[i], l2, __hfma2(x[j].p[i], h2, __hneg2(hi)));
            x[j].p[i] = hi;
        }
        *reinterpret_cast<uint4 *>(tile + img_chunk_off(C, row, j0 + j)) = x[j].u;
        *reinterpret_cast<uint4 *>(rest + img_chunk_off(C, row, j0 + j)) = lo.u;
    }
}
// x = hi + lo of two bf16 each, packed: 2^-16 of x is lost at most
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(a, b);
    lo = pack_bf16(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xFFFF0000u));
}
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
// The i-th longest sequence of a batch; every thread of the block calls it.  Batches of up to SORTED sequences run
// longest first (32 sequences x 32 heads of 64 to 8192 tokens: 680 us, as they come 716; 96 x 8: 610 and 722); ranks cost
// a scan of the lengths in every CTA, and longer batches even out by themselves.
constexpr int SORTED = 128;
__device__ __forceinline__ int64_t longest_first(const int32_t *cu, int64_t N, int64_t i, int *n_smem) {
    if (!cu || N < 2 || N > SORTED) return i;
    if (threadIdx.x < N) {
        const int t = threadIdx.x, len = cu[t + 1] - cu[t];
        int rank = 0;
        for (int m = 0; m < (int)N; ++m) {
            const int l = cu[m + 1] - cu[m];
            rank += l > len || (l == len && m < t);
        }
        if (rank == (int)i) *n_smem = t;
    }
    __syncthreads();
    return *n_smem;
}
// The first block looks all of cu_seqlens over.
__device__ __forceinline__ void check_seqlens(const int32_t *cu, int64_t T, int64_t N, int *err) {
    for (int64_t n = threadIdx.x; n < N; n += blockDim.x) {
        span s;
        if (!seq_span(cu, T, N, n, &s)) set_error(err, KDA_ERR_BAD_SEQLENS);
    }
}

// A row's values multiplied by f, in three parts which together are the fp32 product.
template <int N>
__device__ __forceinline__ void split_chunks(const unsigned char *tile, int row, int j0, float f, uint4 *hi, uint4 *mid, uint4 *lo) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
        uint4 u = *reinterpret_cast<const uint4 *>(tile + img_chunk_off(C, row, j0 + j));
        if (f == 0.f) u = make_uint4(0, 0, 0, 0);  // erased, whatever the row holds
        const uint32_t *x = reinterpret_cast<const uint32_t *>(&u);
        uint32_t *h = reinterpret_cast<uint32_t *>(hi + j), *m = reinterpret_cast<uint32_t *>(mid + j),
                 *l = reinterpret_cast<uint32_t *>(lo + j);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a = bf_lo(x[i]) * f, b = bf_hi(x[i]) * f;
            h[i] = pack_bf16(a, b);
            a -= bf_lo(h[i]), b -= bf_hi(h[i]);
            m[i] = pack_bf16(a, b);
            l[i] = pack_bf16(a - bf_lo(m[i]), b - bf_hi(m[i]));
        }
    }
}
template <int N>
__device__ __forceinline__ void clear_chunks(unsigned char *tile, int row, int j0) {
#pragma unroll
    for (int j = 0; j < N; ++j)
        *reinterpret_cast<uint4 *>(tile + img_chunk_off(C, row, j0 + j)) = make_uint4(0, 0, 0, 0);
}

// True in one lane of a converged warp.  The products' descriptors stay in uniform registers under it, which under
// `lane == 0` they do not: a product then issues every 120 cycles instead of every 70.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
    return p != 0;
}
// Asks L2 for one box of a tile map ahead of its load.
__device__ __forceinline__ void tma_prefetch_3d(const void *tmap, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];"
                 :: "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2) : "memory");
}
template <int N> __device__ __forceinline__ void tmem_load(uint32_t taddr, float *v) {
    if constexpr (N == 32) tmem_ld32(taddr, v);
    else tmem_ld16(taddr, v);
}
// Two times 16 columns behind one wait.
__device__ __forceinline__ void tmem_load_pair(uint32_t ta, uint32_t tb, float *a, float *b) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(a[0]), "=f"(a[1]), "=f"(a[2]), "=f"(a[3]), "=f"(a[4]), "=f"(a[5]), "=f"(a[6]), "=f"(a[7]),
          "=f"(a[8]), "=f"(a[9]), "=f"(a[10]), "=f"(a[11]), "=f"(a[12]), "=f"(a[13]), "=f"(a[14]), "=f"(a[15]),
          "=f"(b[0]), "=f"(b[1]), "=f"(b[2]), "=f"(b[3]), "=f"(b[4]), "=f"(b[5]), "=f"(b[6]), "=f"(b[7]),
          "=f"(b[8]), "=f"(b[9]), "=f"(b[10]), "=f"(b[11]), "=f"(b[12]), "=f"(b[13]), "=f"(b[14]), "=f"(b[15])
        : "r"(ta), "r"(tb) : "memory");
}
template <int N> __device__ __forceinline__ void tmem_store(uint32_t taddr, const float *v) {
    if constexpr (N == 32) tmem_st32(taddr, v);
    else tmem_st16(taddr, v);
}
// Meeting of the `threads` threads that share named barrier `id` (1 .. 15).
__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory");
}

// 32 bytes of a row: one whole sector at a time where the tensor's address allows it (wide), else two halves of one.
__device__ __forceinline__ void st_row_32B(void *p, const uint32_t *v, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                     :: "l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

}  // namespace tcl
}  // namespace lin
}  // namespace kda
