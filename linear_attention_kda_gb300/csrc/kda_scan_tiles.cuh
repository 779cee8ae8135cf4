// How the two sequence-long directions of kda_scan split a batch and join it again.
//
// A tile is L tokens of one sequence by W = 64 channels, taken by one block of threads; it reads its inputs once and
// keeps what it made of them.  What a tile does to the state that enters it is two numbers per channel, its decay and the state that it
// leaves from zero, and tiles join at three levels, each in a fixed order, so that the result does not depend on which
// block ran first:
//   - a tile leaves its (decay, value) as soon as it has them, waiting for nothing;
//   - the last of 16 tiles folds them into the group's, waiting for the tiles alone;
//   - the last of 16 groups leaves the state behind it, from the last such state and the groups and tiles since.
// The state that enters a tile is the fold of what lies between, at most 1 + 15 + 15 entries, and the chain of waits
// grows by one per 256 tiles.  An entry is one 64-bit word, cleared to all ones before, so that reading it and seeing that it is
// there are one access: a flag beside the data took a fence, a barrier and a second trip to L2.  The blocks of a
// cooperative launch, all of them running, take every gridDim-th tile in the direction of the scan: the first tile that is not
// done waits for none that is not, so that every wait ends; they are limited all the same.
#pragma once
#include <cuda.h>

#include <atomic>

#include "kda_internal.h"
#include "kda_linear.cuh"
#include "kda_scan.cuh"
#include "tc_util.cuh"

namespace kda {
namespace scan {

constexpr int CK = KDA_SCAN_CHECKPOINT;
constexpr int W = 64;                   // channels of a tile, two a lane
constexpr int NW = 8;                   // warps of a block
constexpr int NT = 32 * NW;
constexpr int G = 16;                   // tiles of a group, groups of a supergroup

// The workspace.  A sequence whose first tile has slot f (lin::chunk_slots) has its groups from f / 16 + n on and its
// supergroups from f / 256 + n on, for the reason that keeps the slots apart.
struct board {
    int32_t *bad;              // whether any of cu_seqlens is
    int4 *plan;                // [slots] tiles: sequence, index in it (-1: none), first token and that behind the last
    unsigned long long *entry[3];  // per level [slots, D]: decay and value; of the third level a state
    int64_t slots, words;      // words: of all entries
    int L;                     // tokens of a tile
};
inline int64_t level_slots(int64_t slots, int64_t N, int level) {
    return level == 0 ? slots : level == 1 ? slots / G + N : slots / (G * G) + N;
}
// Bytes of the workspace (0 where no sequence can have a second tile); sets *b where it is given.
inline size_t board_layout(int64_t T, int64_t N, int D, int L, void *ws, board *b) {
    if (T <= L) return 0;
    board x{};
    x.L = L;
    x.slots = lin::chunk_slots(T, N, L);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char *p = ws ? (char *)ws + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    x.bad = (int32_t *)take(4);
    x.plan = (int4 *)take(x.slots * sizeof(int4));
    int64_t before[3];
    for (int i = 0; i < 3; ++i) {
        before[i] = x.words;
        x.words += level_slots(x.slots, N, i) * D;
    }
    unsigned long long *first = (unsigned long long *)take(x.words * 8);
    for (int i = 0; i < 3; ++i) x.entry[i] = first + before[i];
    if (b) *b = x;
    return at;
}

// Clears the entries, looks at all of cu_seqlens and says which tiles there are.  Where any part of cu_seqlens is
// bad no tile waits for another (the slots may not be those that the sequences think), and a block goes through each
// good sequence by itself.
__global__ void __launch_bounds__(256) scan_plan_kernel(const __grid_constant__ board B, const int32_t *cu, int64_t T, int64_t N, int *err) {
    const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x, each = (int64_t)gridDim.x * 256;
    const int L = B.L;
    // (the entries begin on a 256-byte boundary and end before a multiple of it)
    for (int64_t i = first; i < (B.words + 1) / 2; i += each) reinterpret_cast<uint4 *>(B.entry[0])[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
    // Where in the plan a tile stands: first tiles of all sequences first, then their second ones and so on, so that what a tile
    // waits for was begun long before it wherever there are several sequences (32 sequences of 4096 channels: XXX).  A tile's place is a sum over
    // all sequences, so this is for up to 1024 of them; more are short enough in the order of their slots.
    const bool rounds = N > 1 && N <= 1024;
    auto tiles = [&](int64_t n) {
        lin::span s;
        return lin::seq_span(cu, T, N, n, &s) ? s.b > s.a ? (s.b - s.a + L - 1) / L : 1 : 0;
    };
    for (int64_t i = first; i < B.slots; i += each) {
        int64_t lo = 0, hi = N;
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) / 2;
            if (lin::seq_start(cu, T, N, mid) / L + mid <= i) lo = mid;
            else hi = mid;
        }
        lin::span s;
        int4 q = make_int4((int)lo, -1, 0, 0);
        int64_t p = -1;
        if (lin::seq_span(cu, T, N, lo, &s)) {
            p = i - (s.a / L + lo);
            // (an empty sequence has a slot, too: its final state)
            if (p >= 0 && p < tiles(lo)) q = make_int4((int)lo, (int)p, (int)s.a, (int)s.b);
        }
        if (!rounds) {
            B.plan[i] = q;
        } else if (q.y >= 0) {
            int64_t at = 0;
            for (int64_t n = 0; n < N; ++n) {
                const int64_t k = tiles(n);
                at += k < p ? k : p;
                at += n < lo && k > p;
            }
            // (in range, and every place once, where all of cu_seqlens is good; else the plan is not looked at)
            if (at < B.slots) B.plan[at] = q;
        }
    }
    // places behind the last tile
    if (rounds && blockIdx.x == gridDim.x - 1) {
        int64_t all = 0;
        for (int64_t n = threadIdx.x; n < N; n += 256) all += tiles(n);
        __shared__ unsigned long long total;
        if (threadIdx.x == 0) total = 0;
        __syncthreads();
        atomicAdd(&total, (unsigned long long)all);
        __syncthreads();
        for (int64_t i = (int64_t)total + threadIdx.x; i < B.slots; i += 256) B.plan[i] = make_int4(0, -1, 0, 0);
    }
    if (blockIdx.x > 0) return;
    bool bad = false;
    for (int64_t n = threadIdx.x; n < N; n += 256) {
        lin::span s;
        bad |= !lin::seq_span(cu, T, N, n, &s);
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        *B.bad = bad;
        if (bad) set_error(err, KDA_ERR_BAD_SEQLENS);
    }
}
inline void launch_plan(const board &B, const int32_t *cu, int64_t T, int64_t N, cudaStream_t stream, int *err) {
    const int64_t words = B.words / 2 > B.slots ? B.words / 2 : B.slots;
    const int64_t want = (words + 1023) / 1024;
    scan_plan_kernel<<<(unsigned)(want < 1216 ? want : 1216), 256, 0, stream>>>(B, cu, T, N, err);
}

__device__ __forceinline__ void sync_some(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
__device__ __forceinline__ void arrive_some(int id, int threads) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// An entry; its upper half is never all ones
__device__ __forceinline__ void put(unsigned long long *p, float d, float b) {
    const uint32_t hi = b != b ? 0x7FC00000u : __float_as_uint(b);
    asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(p), "l"((unsigned long long)hi << 32 | __float_as_uint(d)) : "memory");
}
__device__ __forceinline__ unsigned long long get(const unsigned long long *p) {
    unsigned long long v;
    asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
constexpr int BATCH = 8;
// n (up to BATCH) entries, `pitch` apart, waited for about a second at most
__device__ __forceinline__ void get_batch(const unsigned long long *p, int64_t pitch, int n, unsigned long long (&e)[BATCH], int *err) {
    for (int tries = 0;; ++tries) {
        bool all = true;
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            if (i < n) e[i] = get(p + i * pitch);
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            if (i < n) all &= (uint32_t)(e[i] >> 32) != ~0u;
        if (all) return;
        if (tries > 1 << 20) {
            set_error(err, KDA_ERR_DEVICE_TIMEOUT);
            return;
        }
        if (tries > 16) __nanosleep(50);
    }
}
__device__ __forceinline__ float entry_d(unsigned long long e) { return __uint_as_float((uint32_t)e); }
__device__ __forceinline__ float entry_b(unsigned long long e) { return __uint_as_float((uint32_t)(e >> 32)); }
// the decay of one run and then another
__device__ __forceinline__ float compose(float d1, float d2) {
    if (d1 < 0.f && d2 < 0.f) {
        const float m = fma(d1, d2, d1) + d2;
        return m > -0.22f ? m : 1.f + m;
    }
    return factor(d1) * factor(d2);
}

struct tile {
    int n, p, count;   // sequence, position in the direction of the scan (-1: no tile), tiles of the sequence
    int a, b;          // the sequence's tokens
    int block;         // of channels
    int first;         // slot of the sequence's first tile
};

struct tile_memory {
    float g[NW][W], d[NW][W], b[NW][W];  // the warps' sums of log-decays, decays and values; after join() g is the state that enters each warp's tokens
    float from[W];                       // the state that enters the run of tiles before this one in its group
};

// With every warp's (g, d, b) of its R tokens in place: leaves the tile's sum for others and finds what enters each warp's tokens.  start, end:
// the state (or adjoint) before and behind the sequence, [N, D] or NULL; kept: where the checkpoints of this tile go (NULL: nowhere), `room` rows.  links: tiles of this sequence wait for one another; else `serial` may say that M.from is in place for all tiles but the
// first, and is left so for the next.
template <int R>
__device__ __forceinline__ void join(const board &B, bool links, bool serial, const tile &t, int D, const float *start, float *end, float *kept, int room,
                                     tile_memory &M, int *err) {
    static_assert(2 * W <= NT, "two halves");
    const int tid = threadIdx.x, half = tid / W, ch = tid % W, c = t.block * W + ch;
    __syncthreads();
    const int q = links ? t.p % G : 0, gq = links ? t.p / G % G : 0, super = t.p / (G * G);
    const int64_t slot = t.first + t.p;
    const bool more = links && t.p + 1 < t.count;
    unsigned long long e[BATCH];
    if (half == 0) {
        if (more) {
            float sum = 0.f, v = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                sum += M.g[w][ch];
                v = step_or_erase(M.d[w][ch], v, M.b[w][ch]);
            }
            float d = decay_of(sum).d;
            if (t.p == 0) {  // nothing enters the first tile: its value is the state behind it
                v = step_or_erase(d, start && c < D ? start[(int64_t)t.n * D + c] : 0.f, v);
                d = 0.f;
            }
            if (c < D) put(B.entry[0] + slot * D + c, d, v);
            if (q == G - 1 && c < D) {
                float gd = 1.f, gb = 0.f;
                for (int i0 = 0; i0 < G - 1; i0 += BATCH) {
                    const int n = G - 1 - i0 < BATCH ? G - 1 - i0 : BATCH;
                    get_batch(B.entry[0] + (slot - q + i0) * D + c, D, n, e, err);
#pragma unroll
                    for (int i = 0; i < BATCH; ++i)
                        if (i < n) {
                            gb = step_or_erase(entry_d(e[i]), gb, entry_b(e[i]));
                            gd = compose(gd, entry_d(e[i]));
                        }
                }
                put(B.entry[1] + ((int64_t)t.first / G + t.n + t.p / G) * D + c, compose(gd, d), step_or_erase(d, gb, v));
            }
        }
        if (q > 0 && c < D) get_batch(B.entry[0] + (slot - q) * D + c, D, q < BATCH ? q : BATCH, e, err);
        sync_some(1, 2 * W);
        float h = M.from[ch];
        if (c < D)
            for (int i0 = 0; i0 < q; i0 += BATCH) {
                if (i0 > 0) get_batch(B.entry[0] + (slot - q + i0) * D + c, D, q - i0 < BATCH ? q - i0 : BATCH, e, err);
#pragma unroll
                for (int i = 0; i < BATCH; ++i)
                    if (i0 + i < q) h = step_or_erase(entry_d(e[i]), h, entry_b(e[i]));
            }
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w * R % CK == 0 && kept && w * R / CK < room && c < D) kept[(int64_t)(w * R / CK) * D + c] = h;
            M.g[w][ch] = h;
            h = step_or_erase(M.d[w][ch], h, M.b[w][ch]);
        }
        if (more && t.p % (G * G) == G * G - 1 && c < D)
            put(B.entry[2] + ((int64_t)t.first / (G * G) + t.n + super) * D + c, h, 0.f);
        if (end && c < D && t.p + 1 >= t.count) end[(int64_t)t.n * D + c] = h;
        if (serial) M.from[ch] = h;
    } else if (half == 1) {
        if (!(serial && t.p > 0)) {
            float v = 0.f;
            if (t.p == 0) {
                if (start && c < D) v = start[(int64_t)t.n * D + c];
            } else if (c < D) {
                if (super > 0) {
                    get_batch(B.entry[2] + ((int64_t)t.first / (G * G) + t.n + super - 1) * D + c, D, 1, e, err);
                    v = entry_d(e[0]);
                }
                const unsigned long long *groups = B.entry[1] + ((int64_t)t.first / G + t.n + super * G) * D + c;
                for (int i0 = 0; i0 < gq; i0 += BATCH) {
                    get_batch(groups + (int64_t)i0 * D, D, gq - i0 < BATCH ? gq - i0 : BATCH, e, err);
#pragma unroll
                    for (int i = 0; i < BATCH; ++i)
                        if (i0 + i < gq) v = step_or_erase(entry_d(e[i]), v, entry_b(e[i]));
                }
            }
            M.from[ch] = v;
        }
        arrive_some(1, 2 * W);
    }
    __syncthreads();
}

// Which tiles a block goes through: every gridDim.x-th, channels innermost; in a batch whose cu_seqlens is bad, all tiles of
// every gridDim.x-th sequence and block of channels.
template <int L> struct course {
    const board &B;
    const int32_t *cu;
    int64_t T, N, items;
    int blocks, joined, serial;
    struct place {
        int64_t item;
        tile t;
    };
    __device__ __forceinline__ course(const board &b, const int32_t *cu_, int64_t T_, int64_t N_, int blocks_, int joined_)
        : B(b), cu(cu_), T(T_), N(N_), blocks(blocks_), joined(joined_) {
        serial = joined && __ldcg(B.bad) != 0;
        items = (serial ? N : lin::chunk_slots(T, N, L)) * blocks;
    }
    __device__ __forceinline__ tile at(int64_t item, bool back) const {
        tile t{0, -1, 0, 0, 0, 0, 0};
        if (item >= items) return t;
        const int64_t r = back ? items - 1 - item : item, i = r / blocks;
        t.block = (int)(r - i * blocks);
        if (joined && !serial) {
            const int4 q = __ldg(B.plan + i);
            t.n = q.x, t.p = q.y, t.a = q.z, t.b = q.w;
        } else {
            int64_t n = i, p = 0;
            lin::span s;
            if (serial ? lin::seq_span(cu, T, N, n, &s) : lin::find_slot(cu, T, N, L, i, &n, &p, &s)) {
                if (p == 0 || p < (s.b - s.a + L - 1) / L) t.p = (int)p;
                t.n = (int)n, t.a = (int)s.a, t.b = (int)s.b;
            }
        }
        t.count = (t.b - t.a + L - 1) / L;
        t.first = t.a / L + t.n;
        if (back && !serial && t.p >= 0 && t.count > 0) t.p = t.count - 1 - t.p;  // positions count from the end
        return t;
    }
    // Every lane of a warp calls these.
    __device__ __forceinline__ void skip(place &x, bool back) const {
        while (x.t.p < 0 && x.item < items) x.t = at(x.item += gridDim.x, back);
    }
    __device__ __forceinline__ place begin(bool back) const {
        place x{(int64_t)blockIdx.x, at(blockIdx.x, back)};
        skip(x, back);
        return x;
    }
    __device__ __forceinline__ place next(place x, bool back) const {
        if (x.item >= items) return x;
        if (serial && x.t.p + 1 < x.t.count) {
            ++x.t.p;
            return x;
        }
        x.t = at(x.item += gridDim.x, back);
        skip(x, back);
        return x;
    }
};

// Sets the error of a call whose tiles do not wait for one another (the plan kernel does it for the others).
__device__ __forceinline__ void check_all(const int32_t *cu, int64_t T, int64_t N, int *err) {
    if (blockIdx.x > 0) return;
    for (int64_t n = threadIdx.x; n < N; n += NT) {
        lin::span s;
        if (!lin::seq_span(cu, T, N, n, &s)) set_error(err, KDA_ERR_BAD_SEQLENS);
    }
}

// A tile's boxes of NI tensors, two tiles ahead of their use
template <typename T, int NI, int L> struct ring {
    T x[2][NI][L][W];
    uint64_t full[2];
};
template <int NI> struct row_maps {
    CUtensorMap m[NI];
};
// [T, D] rows a stride apart, boxes of L rows and W channels.  Needs 16-byte aligned rows.
inline bool make_row_map(CUtensorMap *m, const void *base, int64_t T, int D, int64_t stride, kda_dtype_t dtype, int L) {
    typedef CUresult (*encode_fn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                  const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);
    static const encode_fn encode = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (encode_fn)p;
    }();
    if (!encode) return false;
    const int64_t es = dtype == KDA_BF16 ? 2 : 4;
    const cuuint64_t dims[3] = {(cuuint64_t)D, 1, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)(stride * es), (cuuint64_t)(stride * es)};
    const cuuint32_t box[3] = {W, 1, (cuuint32_t)L}, estr[3] = {1, 1, 1};
    return encode(m, dtype == KDA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void *>(base), dims,
                  strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Two neighbouring channels of a row: by one access where rows are aligned for it, else by their elements
template <typename T, bool TMA> __device__ __forceinline__ float2 load_pair(const T *p, int have) {
    if constexpr (TMA) {
        float2 f;
        layer::unpack<T, 2>(layer::load<T, 2>(p), &f);
        return f;
    }
    return make_float2(have > 0 ? ld(p) : 0.f, have > 1 ? ld(p + 1) : 0.f);
}
template <typename T, bool TMA> __device__ __forceinline__ void store_pair(T *p, float2 f, int have) {
    if constexpr (TMA) layer::store_once(p, layer::pack<T, 2>(&f));
    else {
        if (have > 0) st(p, f.x);
        if (have > 1) st(p + 1, f.y);
    }
}
__device__ __forceinline__ channel<float2> load_channel(const float *A_log, const float *dt_bias, int c, int have) {
    auto two = [&](const float *p, float none) { return make_float2(p && have > 0 ? p[c] : none, p && have > 1 ? p[c + 1] : none); };
    const float2 A = two(A_log, 0.f);
    return {two(dt_bias, 0.f), make_float2(expf(A.x), expf(A.y))};
}

// Blocks of a cooperative launch: as many as run at once, at most one for each tile.
template <typename K>
inline cudaError_t running_blocks(K *kernel, size_t smem, std::atomic<int> *per_device, int64_t tiles, int *grid) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int n = dev < 64 ? per_device[dev].load(std::memory_order_acquire) : 0;
    if (n == 0) {
        int per = 0, sms = 0;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, NT, smem);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        if (per < 1) return cudaErrorInvalidConfiguration;
        n = per * sms;
        if (dev < 64) per_device[dev].store(n, std::memory_order_release);
    }
    *grid = (int)(tiles < n ? tiles : n);
    return cudaSuccess;
}

}  // namespace scan
}  // namespace kda
