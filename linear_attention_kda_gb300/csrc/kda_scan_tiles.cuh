// How the two sequence-long directions of kda_scan split a batch and join it again.
//
// A tile is L = 64 tokens of one sequence by W channels, one block of threads; it reads its inputs once and keeps them.  What a
// tile does to the state that enters it is two numbers per channel, the sum G of its log-decays and the state B that
// it leaves from zero, and tiles join at three levels, each in a fixed order, so that the result does not depend on
// which block ran first:
//   - a tile leaves (G, B) as soon as it has them, waiting for nothing;
//   - the last of 16 tiles folds them into the group's (G, B), waiting for the tiles alone;
//   - the last of 16 groups leaves the state behind it, from the last such state and the groups and tiles since.
// The state that enters a tile is the fold of what lies between, at most 1 + 15 + 15 entries, and the chain of waits grows by one per
// 16384 tokens.  Blocks take tiles by a ticket, earlier tiles first, so that whatever a block waits for has
// already begun on another one; waits are limited all the same.
#pragma once
#include "kda_linear.cuh"
#include "kda_scan.cuh"

namespace kda {
namespace scan {

constexpr int L = KDA_SCAN_CHECKPOINT;  // tokens of a tile
constexpr int NW = 8, R = L / NW;       // warps of a block, tokens of a warp
constexpr int NT = 32 * NW;
constexpr int G = 16;                   // tiles of a group, groups of a supergroup

// The workspace.  A sequence whose first tile has slot f (lin::chunk_slots) has its groups from f / 16 + n on and its
// supergroups from f / 256 + n on, for the reason that keeps the slots apart.  `control`: the ticket and whether
// cu_seqlens is good, then the flags of the three levels, all cleared before the tiles run.
struct board {
    int32_t *control;
    int32_t *flag[3];
    float *decay[2], *value[3];
    int64_t slots, control_words;
    int blocks;  // of channels
};
inline int64_t level_slots(int64_t slots, int64_t N, int level) {
    return level == 0 ? slots : level == 1 ? slots / G + N : slots / (G * G) + N;
}
// Bytes of the workspace (0 where no sequence can have a second tile); sets *b where it is given.  The flags allow for the
// narrowest blocks of channels.
inline size_t board_layout(int64_t T, int64_t N, int D, int width, void *ws, board *b) {
    if (T <= L) return 0;
    char *p = (char *)ws;
    const int64_t slots = lin::chunk_slots(T, N, L);
    const int blocks = (D + width - 1) / width;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return p ? p + here : nullptr;
    };
    int64_t words = 2;
    for (int i = 0; i < 3; ++i) words += level_slots(slots, N, i) * blocks;
    int32_t *control = (int32_t *)take(words * 4);
    float *decay[2], *value[3];
    for (int i = 0; i < 3; ++i) {
        const size_t bytes = (size_t)level_slots(slots, N, i) * D * 4;
        if (i < 2) decay[i] = (float *)take(bytes);
        value[i] = (float *)take(bytes);
    }
    if (b) {
        b->control = control;
        b->control_words = words;
        b->slots = slots;
        b->blocks = blocks;
        int32_t *f = control + 2;
        for (int i = 0; i < 3; ++i) {
            b->flag[i] = f;
            f += level_slots(slots, N, i) * blocks;
            if (i < 2) b->decay[i] = decay[i];
            b->value[i] = value[i];
        }
    }
    return at;
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

// Which tile a block has: of sequence n with tokens [a, b), the position p of `count` in the direction of the scan.
struct tile {
    int64_t n, p, count, first;  // first: slot of the sequence's first tile
    lin::span s;
    int block;
    bool serial;                 // one block goes through the whole sequence (a batch whose cu_seqlens is bad elsewhere)
};

template <int W> struct tile_memory {
    float g[NW][W], d[NW][W], b[NW][W];  // the warps' sums of log-decays, their decay and value
    float from[W];                       // the state that enters the run of tiles before this one in its group
    float run_d[W], run_b[W];            // that run
    tile t;
    bool some;
};

// Takes a tile; false where there is none for this block.
template <int W> __device__ __forceinline__ bool take_tile(const board &B, bool joined, const int32_t *cu, int64_t T, int64_t N, int blocks,
                                                           tile_memory<W> &M, int *err) {
    if (threadIdx.x < 32) {
        int64_t at = blockIdx.x;
        bool good = true;
        if (joined) {
            int ticket = 0;
            if (threadIdx.x == 0) ticket = atomicAdd(B.control, 1);
            at = __shfl_sync(0xffffffffu, ticket, 0);
            good = __ldcg(B.control + 1) == 0;
        }
        tile t;
        t.block = (int)(at % blocks);
        t.serial = !good;
        bool some;
        if (good) {
            some = lin::find_slot(cu, T, N, L, at / blocks, &t.n, &t.p, &t.s);
        } else {
            t.n = at / blocks;
            t.p = 0;
            some = t.n < N && lin::seq_span(cu, T, N, t.n, &t.s);
        }
        if (some) {
            t.count = (t.s.b - t.s.a + L - 1) / L;
            t.first = t.s.a / L + t.n;
            some = t.p < t.count || t.p == 0;  // (an empty sequence has a slot, too)
        }
        if (threadIdx.x == 0) {
            M.t = t;
            M.some = some;
        }
    }
    __syncthreads();
    if (!joined && blockIdx.x == 0)
        for (int64_t n = threadIdx.x; n < N; n += NT) {
            lin::span s;
            if (!lin::seq_span(cu, T, N, n, &s)) set_error(err, KDA_ERR_BAD_SEQLENS);
        }
    return M.some;
}

// With every warp's (g, d, b) in place: leaves the tile's sum for others and finds what enters it.  start: the state (or adjoint) that
// enters the sequence, [N, D] or NULL.  Ends with a barrier; the state that enters the tile is then d_run from + b_run.
template <int W>
__device__ __forceinline__ void join(const board &B, bool joined, const tile &t, int c0, int D, const float *start, tile_memory<W> &M, int *err) {
    static_assert(2 * W <= NT, "two halves");
    const int tid = threadIdx.x, half = tid / W, ch = tid % W, c = c0 + ch;
    __syncthreads();
    const bool links = joined && !t.serial && t.count > 1;
    const int q = links ? (int)(t.p % G) : 0, gq = links ? (int)(t.p / G % G) : 0;
    const int64_t super = t.p / (G * G), slot = t.first + t.p;
    if (half == 0) {
        float sum = 0.f, v = 0.f, run_g = 0.f, run_b = 0.f;
        if (links && t.p + 1 < t.count) {
            if (t.p == 0) {
                sum = -INFINITY;  // nothing enters the first tile: its value is the state behind it
                v = start && c < D ? start[t.n * D + c] : 0.f;
            }
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                sum += M.g[w][ch];
                v = decayed(M.d[w][ch], v) + M.b[w][ch];
            }
            if (c < D) {
                __stcg(B.decay[0] + slot * D + c, sum);
                __stcg(B.value[0] + slot * D + c, v);
            }
            sync_half(1, W);
            if (tid == 0) release(B.flag[0] + slot * B.blocks + t.block);
        }
        if (q > 0) {
            bool ok = true;
            if (tid < q) ok = acquire(B.flag[0] + (slot - q + tid) * B.blocks + t.block);
            if (!ok) set_error(err, KDA_ERR_DEVICE_TIMEOUT);
            sync_half(1, W);
            if (c < D) {
                float eg[G - 1], eb[G - 1];
#pragma unroll
                for (int i = 0; i < G - 1; ++i)
                    if (i < q) {
                        eg[i] = __ldcg(B.decay[0] + (slot - q + i) * D + c);
                        eb[i] = __ldcg(B.value[0] + (slot - q + i) * D + c);
                    }
#pragma unroll
                for (int i = 0; i < G - 1; ++i)
                    if (i < q) {
                        run_b = decayed(decay_of(eg[i]).d, run_b) + eb[i];
                        run_g += eg[i];
                    }
            }
            if (q == G - 1 && t.p + 1 < t.count) {
                const int64_t at = t.first / G + t.n + t.p / G;
                if (c < D) {
                    __stcg(B.decay[1] + at * D + c, run_g + sum);
                    __stcg(B.value[1] + at * D + c, decayed(decay_of(sum).d, run_b) + v);
                }
                sync_half(1, W);
                if (tid == 0) release(B.flag[1] + at * B.blocks + t.block);
            }
        }
        M.run_d[ch] = decay_of(run_g).d;
        M.run_b[ch] = run_b;
    } else if (half == 1 && !(t.serial && t.p > 0)) {
        float v = 0.f;
        if (t.p == 0) {
            if (start && c < D) v = start[t.n * D + c];
        } else if (gq > 0 || super > 0) {
            const int64_t g0 = t.first / G + t.n + super * G, s0 = t.first / (G * G) + t.n + super - 1;
            bool ok = true;
            if (ch < gq) ok = acquire(B.flag[1] + (g0 + ch) * B.blocks + t.block);
            else if (ch == G && super > 0) ok = acquire(B.flag[2] + s0 * B.blocks + t.block);
            if (!ok) set_error(err, KDA_ERR_DEVICE_TIMEOUT);
            sync_half(2, W);
            if (c < D) {
                if (super > 0) v = __ldcg(B.value[2] + s0 * D + c);
                float eg[G - 1], eb[G - 1];
#pragma unroll
                for (int i = 0; i < G - 1; ++i)
                    if (i < gq) {
                        eg[i] = __ldcg(B.decay[1] + (g0 + i) * D + c);
                        eb[i] = __ldcg(B.value[1] + (g0 + i) * D + c);
                    }
#pragma unroll
                for (int i = 0; i < G - 1; ++i)
                    if (i < gq) v = decayed(decay_of(eg[i]).d, v) + eb[i];
            }
        }
        M.from[ch] = v;
    }
    __syncthreads();
}

// The state behind a tile, as the last warp has it (V channels a lane): for the supergroup after, or the next tile of a
// serial run.
template <int W, int V>
__device__ __forceinline__ void leave(const board &B, bool joined, const tile &t, int c0, int D, const float (&h)[V], tile_memory<W> &M) {
    const int lane = threadIdx.x & 31;
    if (!joined || t.p + 1 >= t.count) return;
    if (t.serial) {
#pragma unroll
        for (int v = 0; v < V; ++v) M.from[lane * V + v] = h[v];
    } else if (t.p % (G * G) == G * G - 1) {
        const int64_t at = t.first / (G * G) + t.n + t.p / (G * G);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (c0 + lane * V + v < D) __stcg(B.value[2] + at * D + c0 + lane * V + v, h[v]);
        __syncwarp();
        if (lane == 0) release(B.flag[2] + at * B.blocks + t.block);
    }
}

// Clears the flags and the ticket and looks at all of cu_seqlens: where any part is bad, no tile waits for another (the
// slots of a bad cu_seqlens may not be those that its sequences think), and a block goes through each good sequence.
__global__ void __launch_bounds__(256) scan_clear_kernel(int32_t *control, int64_t words, const int32_t *cu, int64_t T, int64_t N, int *err) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += (int64_t)gridDim.x * 256)
        if (i != 1) control[i] = 0;
    if (blockIdx.x > 0) return;
    bool bad = false;
    for (int64_t n = threadIdx.x; n < N; n += 256) {
        lin::span s;
        bad |= !lin::seq_span(cu, T, N, n, &s);
    }
    if (__syncthreads_or(bad) && threadIdx.x == 0) set_error(err, KDA_ERR_BAD_SEQLENS);
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) control[1] = bad;
}

}  // namespace scan
}  // namespace kda
