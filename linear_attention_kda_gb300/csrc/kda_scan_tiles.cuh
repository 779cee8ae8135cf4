// How the two sequence-long directions of kda_scan split a batch and join it again.
//
// A tile is L = 64 tokens of one sequence by W channels, taken by one block of threads; it reads its inputs once and keeps
// what it made of them.  What a tile does to the state that enters it is two numbers per channel, the sum G of its log-decays and the
// state B that it leaves from zero, and tiles join at three levels, each in a fixed order, so that the result does not
// depend on which block ran first:
//   - a tile leaves (G, B) as soon as it has them, waiting for nothing;
//   - the last of 16 tiles folds them into the group's (G, B), waiting for the tiles alone;
//   - the last of 16 groups leaves the state behind it, from the last such state and the groups and tiles since.
// The state that enters a tile is the fold of what lies between, at most 1 + 15 + 15 entries, and the chain of waits grows
// by one per 16384 tokens.  The blocks of a cooperative launch, all of them running, take every G-th tile in the
// direction of the scan: the first tile that is not done waits for none that is not, so that every wait ends; they are limited all
// the same.
#pragma once
#include <atomic>

#include "kda_internal.h"
#include "kda_linear.cuh"
#include "kda_scan.cuh"

namespace kda {
namespace scan {

constexpr int L = KDA_SCAN_CHECKPOINT;  // tokens of a tile
constexpr int NW = 8, R = L / NW;       // warps of a block, tokens of a warp
constexpr int NT = 32 * NW;
constexpr int G = 16;                   // tiles of a group, groups of a supergroup

// The workspace.  A sequence whose first tile has slot f (lin::chunk_slots) has its groups from f / 16 + n on and its
// supergroups from f / 256 + n on, for the reason that keeps the slots apart.
struct board {
    int32_t *bad;          // whether any of cu_seqlens is
    int4 *plan;            // [slots]: sequence, index of the tile in it (-1: none), first and last token
    int32_t *flag[3];      // per level [slots, blocks of channels]
    float *decay[2], *value[3];
    int64_t slots, flags;
    int blocks;
};
inline int64_t level_slots(int64_t slots, int64_t N, int level) {
    return level == 0 ? slots : level == 1 ? slots / G + N : slots / (G * G) + N;
}
// Bytes of the workspace (0 where no sequence can have a second tile); sets *b where it is given.
inline size_t board_layout(int64_t T, int64_t N, int D, int width, void *ws, board *b) {
    if (T <= L) return 0;
    board x{};
    x.slots = lin::chunk_slots(T, N, L);
    x.blocks = (D + width - 1) / width;
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
        before[i] = x.flags;
        x.flags += level_slots(x.slots, N, i) * x.blocks;
    }
    int32_t *flags = (int32_t *)take(x.flags * 4);
    for (int i = 0; i < 3; ++i) {
        const size_t bytes = (size_t)level_slots(x.slots, N, i) * D * 4;
        x.flag[i] = flags + before[i];
        if (i < 2) x.decay[i] = (float *)take(bytes);
        x.value[i] = (float *)take(bytes);
    }
    if (b) *b = x;
    return at;
}

// Clears the flags, looks at all of cu_seqlens and says which tile lies in each slot.  Where any part of cu_seqlens is bad
// no tile waits for another (the slots may not be those that the sequences think), and a block goes through each
// good sequence by itself.
__global__ void __launch_bounds__(256) scan_plan_kernel(const __grid_constant__ board B, const int32_t *cu, int64_t T, int64_t N, int *err) {
    const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x, each = (int64_t)gridDim.x * 256;
    for (int64_t i = first; i < B.flags; i += each) B.flag[0][i] = 0;
    for (int64_t i = first; i < B.slots; i += each) {
        int64_t lo = 0, hi = N;
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) / 2;
            if (lin::seq_start(cu, T, N, mid) / L + mid <= i) lo = mid;
            else hi = mid;
        }
        lin::span s;
        int4 q = make_int4((int)lo, -1, 0, 0);
        if (lin::seq_span(cu, T, N, lo, &s)) {
            const int64_t p = i - (s.a / L + lo), count = (s.b - s.a + L - 1) / L;
            // (an empty sequence has a slot, too: its final state)
            if (p >= 0 && (p < count || p == 0)) q = make_int4((int)lo, (int)p, (int)s.a, (int)s.b);
        }
        B.plan[i] = q;
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
    const int64_t words = B.flags > B.slots ? B.flags : B.slots;
    const int64_t want = (words + 1023) / 1024;
    scan_plan_kernel<<<(unsigned)(want < 608 ? want : 608), 256, 0, stream>>>(B, cu, T, N, err);
}

__device__ __forceinline__ void release(int32_t *flag) {
    __threadfence();
    asm volatile("st.release.gpu.global.s32 [%0], 1;" ::"l"(flag) : "memory");
}
// Waits for a flag, for about a second at most.
__device__ __forceinline__ bool acquire(const int32_t *flag) {
    int32_t v;
    for (int i = 0; i < 1 << 21; ++i) {
        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
        if (v) return true;
        if (i > 32) __nanosleep(64);
    }
    return false;
}
__device__ __forceinline__ void sync_half(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

struct tile {
    int n, p, count;   // sequence, position in the direction of the scan, tiles of the sequence
    int a, b;          // the sequence's tokens
    int block;         // of channels
    __device__ __forceinline__ int first() const { return a / L + n; }  // slot of the sequence's first tile
};

template <int W> struct tile_memory {
    float g[NW][W], d[NW][W], b[NW][W];  // the warps' sums of log-decays, decays and values; after join() g and b are those of the warps before
    float from[W];                       // the state that enters the run of tiles before this one in its group
    float run_d[W], run_b[W];            // that run
};

// With every warp's (g, d, b) in place: leaves the tile's sum for others and finds what enters it.  start: the state (or adjoint)
// that enters the sequence, [N, D] or NULL.  links: whether tiles of this sequence wait for one another; `keep` leaves M.from as it is.
template <int W>
__device__ __forceinline__ void join(const board &B, bool links, bool keep, const tile &t, int D, const float *start, tile_memory<W> &M, int *err) {
    static_assert(2 * W <= NT, "two halves");
    const int tid = threadIdx.x, half = tid / W, ch = tid % W, c = t.block * W + ch;
    __syncthreads();
    const int q = links ? t.p % G : 0, gq = links ? t.p / G % G : 0, super = t.p / (G * G);
    const int64_t slot = t.first() + t.p;
    const bool more = links && t.p + 1 < t.count;
    constexpr int BATCH = 8;
    // state of `n` entries of a level from slot `at` on behind the state v; run: the sum of their log-decays
    auto fold = [&](int level, int64_t at, int n, float &v, float &run) {
        const float *pg = B.decay[level] + at * D + c, *pb = B.value[level] + at * D + c;
        for (int i0 = 0; i0 < n; i0 += BATCH) {
            float eg[BATCH], eb[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if (i0 + i < n) {
                    eg[i] = __ldcg(pg + (int64_t)(i0 + i) * D);
                    eb[i] = __ldcg(pb + (int64_t)(i0 + i) * D);
                }
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if (i0 + i < n) {
                    v = step_or_erase(decay_of(eg[i]).d, v, eb[i]);
                    run += eg[i];
                }
        }
    };
    if (half == 0) {
        float sum = 0.f, v = 0.f, run_g = 0.f, run_b = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float g = M.g[w][ch], b = M.b[w][ch];
            M.g[w][ch] = sum;
            M.b[w][ch] = v;
            sum += g;
            v = step_or_erase(M.d[w][ch], v, b);
        }
        if (more) {
            if (t.p == 0) {  // nothing enters the first tile: its value is the state behind it
                v = step_or_erase(decay_of(sum).d, start && c < D ? start[(int64_t)t.n * D + c] : 0.f, v);
                sum = -INFINITY;
            }
            if (c < D) {
                __stcg(B.decay[0] + slot * D + c, sum);
                __stcg(B.value[0] + slot * D + c, v);
            }
            sync_half(1, W);
            if (tid == 0) release(B.flag[0] + slot * B.blocks + t.block);
        }
        if (q > 0) {
            if (tid < q && !acquire(B.flag[0] + (slot - q + tid) * B.blocks + t.block)) set_error(err, KDA_ERR_DEVICE_TIMEOUT);
            sync_half(1, W);
            if (c < D) fold(0, slot - q, q, run_b, run_g);
            if (q == G - 1 && more) {
                const int64_t at = t.first() / G + t.n + t.p / G;
                if (c < D) {
                    __stcg(B.decay[1] + at * D + c, run_g + sum);
                    __stcg(B.value[1] + at * D + c, step_or_erase(decay_of(sum).d, run_b, v));
                }
                sync_half(1, W);
                if (tid == 0) release(B.flag[1] + at * B.blocks + t.block);
            }
        }
        M.run_d[ch] = decay_of(run_g).d;
        M.run_b[ch] = run_b;
    } else if (half == 1 && !keep) {
        float v = 0.f, unused = 0.f;
        if (t.p == 0) {
            if (start && c < D) v = start[(int64_t)t.n * D + c];
        } else if (gq > 0 || super > 0) {
            const int64_t g0 = t.first() / G + t.n + super * G, s0 = t.first() / (G * G) + t.n + super - 1;
            bool ok = true;
            if (ch < gq) ok = acquire(B.flag[1] + (g0 + ch) * B.blocks + t.block);
            else if (ch == G && super > 0) ok = acquire(B.flag[2] + s0 * B.blocks + t.block);
            if (!ok) set_error(err, KDA_ERR_DEVICE_TIMEOUT);
            sync_half(2, W);
            if (c < D) {
                if (super > 0) v = __ldcg(B.value[2] + s0 * D + c);
                fold(1, g0, gq, v, unused);
            }
        }
        M.from[ch] = v;
    }
    __syncthreads();
}

// The state that enters this thread's tokens, after join(); *whole: the one that enters the tile
template <int W, int V, typename F>
__device__ __forceinline__ void enter(const tile_memory<W> &M, int w, int lane, F *h, F *whole) {
    const int at = lane * V;
    auto get = [&](const float *p, int i) { return layer::unpack_one<F>(p + at + i * layer::lanes<V>::K); };
#pragma unroll
    for (int i = 0; i < layer::lanes<V>::N; ++i) {
        whole[i] = step_or_erase(get(M.run_d, i), get(M.from, i), get(M.run_b, i));
        h[i] = step_or_erase(decay_of(get(M.g[w], i)).d, whole[i], get(M.b[w], i));
    }
}

// The state behind a tile, as the last warp has it, for the supergroup after
template <int W, int V, typename F>
__device__ __forceinline__ void leave(const board &B, const tile &t, int lane, int D, const F *h) {
    if (t.p % (G * G) != G * G - 1 || t.p + 1 >= t.count) return;
    const int64_t at = t.first() / (G * G) + t.n + t.p / (G * G);
    const int c = t.block * W + lane * V;
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (c + v < D) __stcg(B.value[2] + at * D + c + v, reinterpret_cast<const float *>(h)[v]);
    __syncwarp();
    if (lane == 0) release(B.flag[2] + at * B.blocks + t.block);
}

// A thread's own elements of the next tile, on their way to shared memory while the block is busy with this one: V elements of each
// of NI tensors for each of R tokens.  No barrier: a thread reads what it has asked for.
template <typename T, int V, int NI> struct ahead {
    layer::vec<T, V> x[R][NI][NT];
    __device__ __forceinline__ void ask(int r, int k, const T *p) {
        void *to = &x[r][k][threadIdx.x];
        if constexpr (sizeof(layer::vec<T, V>) == 8)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(p) : "memory");
        else if constexpr (sizeof(layer::vec<T, V>) == 4) cp_async4(to, p);
        else x[r][k][threadIdx.x] = layer::load<T, V>(p);
    }
};

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
        n = per * sms;
        if (dev < 64) per_device[dev].store(n, std::memory_order_release);
    }
    *grid = (int)(tiles < n ? tiles : n);
    return cudaSuccess;
}

}  // namespace scan
}  // namespace kda
