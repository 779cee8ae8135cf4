// How the two sequence-long directions of kda_scan split a batch and join it again.
//
// A tile is L tokens of one sequence by W channels, taken by one block of threads; it reads its inputs once and keeps
// what it made of them.  The tiles of a sequence and its W channels are a chain.  Where the chains are many and none much longer than
// the rest, a block goes through whole chains, longest first, and hands the state on by shared memory.  Else the blocks take every
// gridDim-th tile, and tiles join through L2: what a tile does to the state that enters it is two numbers per channel, its decay
// and the state that it leaves from zero, and there are three levels of them, each folded in a fixed order, so that the
// result does not depend on which block ran first:
//   - a tile leaves its (decay, value) as soon as it has them, waiting for nothing;
//   - the last of 16 tiles folds them into the group's, waiting for the tiles alone;
//   - the last of 16 groups leaves the state behind it, from the last such state and the groups and tiles since.
// The state that enters a tile is the fold of what lies between, at most 1 + 15 + 15 entries, and the chain of waits grows
// by one per 256 tiles.  An entry is one 64-bit word, cleared to all ones before, so that reading it and seeing that it is there are
// one access: a flag beside the data took a fence, a barrier and a second trip to L2.  All blocks of a cooperative launch
// run, and the first tile that is not done waits for none that is not, so that every wait ends; they are limited all the same.
#pragma once
#include <cooperative_groups.h>

#include <atomic>

#include "kda_internal.h"
#include "kda_linear.cuh"
#include "kda_row_map.h"
#include "kda_scan.cuh"
#include "kda_scan_course.h"
#include "tc_util.cuh"

namespace kda {
namespace scan {

constexpr int CK = KDA_SCAN_CHECKPOINT;
constexpr int NW = 8;                   // warps of a block
constexpr int NT = 32 * NW;

// A tile's shape: W channels, two a lane; a warp holds GW groups of R tokens one after the other.  64 channels are one group of 32
// lanes; 32 or 16 make two or four times as many chains, each of a half or a quarter of the tiles (tile_width()).
template <int W_, int R_> struct shape {
    static constexpr int W = W_, R = R_, LPR = W / 2, GW = 32 / LPR, RW = R * GW, L = NW * RW;
    static constexpr int BOX = L < 256 ? L : 256;  // rows of a TMA box
};
constexpr int G = 16;                   // tiles of a group, groups of a supergroup

// The workspace.  A sequence whose first tile has slot f (lin::chunk_slots) has its groups from f / 16 + n on and its
// supergroups from f / 256 + n on, for the reason that keeps the slots apart.
struct board {
    int32_t *mode;             // [2]: whether blocks take whole chains; how many chains are taken
    int4 *order;               // [N] sequences as chains are taken: sequence, 0 (-1: none), first token and that behind the last
    int4 *plan;                // [slots] tiles: sequence, index in it (-1: none), first token and that behind the last
    unsigned long long *entry[3];  // per level [slots, D]: decay and value; of the third level a state
    int64_t slots, words;      // words: of all entries
    int L;                     // tokens of a tile
};
inline int64_t level_slots(int64_t slots, int64_t N, int level) {
    return level == 0 ? slots : level == 1 ? slots / G + N : slots / (G * G) + N;
}
// Bytes of the workspace; sets *b where it is given.
inline size_t board_layout(int64_t T, int64_t N, int D, int L, void *ws, board *b) {
    board x{};
    x.L = L;
    x.slots = lin::chunk_slots(T, N, L);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char *p = ws ? (char *)ws + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    x.mode = (int32_t *)take(8);
    x.order = (int4 *)take(N * sizeof(int4));
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

// What a call's tiles are.  SINGLE: no sequence has a second one.  EQUAL: whole chains of sequences of one length, as the host can tell
// where there are no cu_seqlens or there is one sequence (one of 4096 tokens and channels 50 us, 60 with a plan).  PLANNED: make_plan() says.
enum layout : int { SINGLE, EQUAL, PLANNED };
__device__ __forceinline__ bool planned_chains(const board &B) { return __ldcg(B.mode) != 0; }
// whether chains, the longest of which has `longest` tiles of `total` in 1 / blocks of the channels, are taken whole by g blocks
__host__ __device__ __forceinline__ bool rather_whole(int64_t longest, int64_t total, int64_t blocks, int64_t g) {
    return longest * g * 5 <= total * blocks * 7;
}

// Clears the entries, looks at all of cu_seqlens, lists the tiles and the chains and chooses between the two ways: whole chains where
// the longest one is no more than 1.4 times a block's share of all tiles (a tile of a chain takes less than one that joins others; where both were tried,
// 16384 tokens of one sequence 193 us by chains and 213, 4 sequences of 512 to 8192 194 and 252), and where any part of cu_seqlens is bad (the slots may not be
// those that the sequences think, so that no tile may wait for another).
// Every thread of a cooperative launch calls it; behind it all blocks see all of it.  (As a kernel of its own it took 2 us more.)
static __device__ __noinline__ void make_plan(const board &B, const int32_t *cu, int64_t T, int64_t N, int64_t D, int blocks, int *err) {
    const int64_t first = (int64_t)blockIdx.x * NT + threadIdx.x, each = (int64_t)gridDim.x * NT;
    const int L = B.L;
    // (the entries begin on a 256-byte boundary and end before a multiple of it)
    for (int64_t i = first; i < (B.words + 1) / 2; i += each) reinterpret_cast<uint4 *>(B.entry[0])[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
    // the tiles of a sequence (an empty one has one, too: its final state; 0: a bad range)
    auto tiles = [&](int64_t n) {
        lin::span s;
        return lin::seq_span(cu, T, N, n, &s) ? s.b > s.a ? (s.b - s.a + L - 1) / L : 1 : 0;
    };
    // Tiles and chains in order of length are worth a look at all sequences for each of them (0.7 us a sequence in all) where sequences are few for
    // the call's size: the longest chain's end is about T D / N elements' work.  In order / as they come, bf16, us: 32 sequences of 512 to 8192 tokens
    // of 4096 channels 1005 / 1073, gradients of 12 of 700 to 5000 684 / 777, 16 of 1 to 2000 168 / 173 and 64, near the border, 577 / 562; of 256 channels
    // 8 of 1 to 2000 34 / 27, 512 of them 559 / 329, 1000 of 64 to 128 tokens 716 / 100.
    const bool sorted = T * D / N >= N << 16;
    // Where in the plan a tile stands: first tiles of all sequences first, then their second ones and so on, so that what a tile
    // waits for was begun long before it wherever there are several sequences.
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
            if (p >= 0 && p < tiles(lo)) q = make_int4((int)lo, (int)p, (int)s.a, (int)s.b);
        }
        if (!sorted || N == 1) {
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
    for (int64_t n = first; n < N; n += each) {
        lin::span s;
        const bool good = lin::seq_span(cu, T, N, n, &s);
        int64_t at = n;
        if (sorted) {
            const int64_t mine = tiles(n);
            at = 0;
            for (int64_t m = 0; m < N; ++m) {
                const int64_t k = tiles(m);
                at += k > mine || (k == mine && m < n);
            }
        }
        B.order[at] = good ? make_int4((int)n, 0, (int)s.a, (int)s.b) : make_int4((int)n, -1, 0, 0);
    }
    if (blockIdx.x == 0) {
        __shared__ unsigned long long total, longest;
        if (threadIdx.x == 0) total = longest = 0;
        __syncthreads();
        unsigned long long all = 0, most = 0;
        bool bad = false;
        for (int64_t n = threadIdx.x; n < N; n += NT) {
            const unsigned long long k = tiles(n);
            all += k;
            most = most > k ? most : k;
            bad |= k == 0;
        }
        atomicAdd(&total, all);
        atomicMax(&longest, most);
        bad = __syncthreads_or(bad);
        if (sorted && N > 1)  // places behind the last tile
            for (int64_t i = (int64_t)total + threadIdx.x; i < B.slots; i += NT) B.plan[i] = make_int4(0, -1, 0, 0);
        if (threadIdx.x == 0) {
            B.mode[0] = bad || rather_whole(longest, total, blocks, gridDim.x);
            B.mode[1] = 0;
            if (bad) set_error(err, KDA_ERR_BAD_SEQLENS);
        }
    }
    cooperative_groups::this_grid().sync();
}

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
// The state behind a supergroup
__device__ __forceinline__ float get_state(const unsigned long long *p, int *err) {
    unsigned long long e = get(p);
    for (int tries = 0; (uint32_t)(e >> 32) == ~0u; ++tries, e = get(p)) {
        if (tries > 1 << 20) {
            set_error(err, KDA_ERR_DEVICE_TIMEOUT);
            break;
        }
        __nanosleep(50);
    }
    return __uint_as_float((uint32_t)e);
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

template <int W> struct tile_memory {
    float g[NW][W], d[NW][W], b[NW][W];  // the warps' sums of log-decays, decays and values; after join() g is the state that enters each warp's tokens
    float from[W];                       // the state behind the last tile, where a block takes whole chains
    int odd;                             // the last turn in which a thread's tokens left an infinity or a NaN, counted from 1
};
// entries on their way through a block: those of the groups (at 1) and of the tiles (at G) before a tile
template <int W> using entries = unsigned long long[1 + 2 * (G - 1)][W];

// Over the groups of a warp, in the direction of the scan: sum and value become those up to and with each group's, before_* those up to it.
// ANY: with infinities and NaN.
template <typename X, bool BACK, bool ANY>
__device__ __forceinline__ void over_groups(float2 &sum, float2 &value, float2 &before_sum, float2 &before) {
    before_sum = before = make_float2(0.f, 0.f);
    if constexpr (X::GW > 1) {
        const int lane = threadIdx.x & 31, grp = lane / X::LPR;
        auto of = [&](float2 v, int groups) {
            const int from = lane + (BACK ? groups : -groups) * X::LPR;
            return make_float2(__shfl_sync(0xffffffffu, v.x, from), __shfl_sync(0xffffffffu, v.y, from));
        };
#pragma unroll
        for (int off = 1; off < X::GW; off *= 2) {
            const float2 s = of(sum, off), v = of(value, off);
            if (BACK ? grp + off < X::GW : grp >= off) {
                const float2 d = decay_of(sum).d;
                value = ANY ? step_any(d, v, value) : step(d, v, value);
                sum = add(sum, s);
            }
        }
        const float2 s = of(sum, 1), v = of(value, 1);
        if (BACK ? grp < X::GW - 1 : grp > 0) before_sum = s, before = v;
    }
}
// The state that enters a group's tokens from the one that enters the warp's
template <typename X, bool ANY> __device__ __forceinline__ float2 group_entry(float2 warp, float2 before_sum, float2 before) {
    if constexpr (X::GW > 1) {
        const float2 d = decay_of(before_sum).d;
        return ANY ? step_any(d, warp, before) : step(d, warp, before);
    }
    return warp;
}
// step_any() over n decays and values from h on, `pitch` apart; enters (or NULL): the state before each.  For what step() finds no longer
// finite in the end, and out of the way of the rest.
static __device__ __noinline__ float fold_any(float h, const float *d, const float *b, float *enters, int pitch, int n) {
    for (int i = 0; i < n; ++i, d += pitch, b += pitch) {
        if (enters) enters[i * pitch] = h;
        h = step_any(*d, h, *b);
    }
    return h;
}

// With every warp's (g, d, b) in place: leaves the tile's sum for others and finds what enters each warp's tokens.  start, end:
// the state (or adjoint) before and behind the sequence, [N, D] or NULL; kept: where the checkpoints of this tile go (NULL: nowhere), `room` rows.
// links: tiles of this sequence wait for one another; E: memory that every warp is done with at the first barrier.
// BACK: the direction is from the last token to the first, so from the last warp to the first.  more_work(role, channel): what
// two otherwise idle roles (2 and 3) do meanwhile.  again(): forms the warps' values again, with the infinities and NaN that one of them
// is found to have in this turn (returned).
template <typename X, bool BACK, typename F, typename Again>
__device__ __forceinline__ bool join(const board &B, bool links, const tile &t, int D, const float *start, float *end, float *kept, int room,
                                     tile_memory<X::W> &M, entries<X::W> &E, int turn, int *err, F &&more_work, Again &&again) {
    // four roles, each of as many warps as its W threads need
    constexpr int W = X::W, WARPS = W > 32 ? W / 32 : 1;
    static_assert(4 * WARPS <= NW, "four roles");
    const int ch = threadIdx.x % (32 * WARPS), role = ch < W ? (int)threadIdx.x / (32 * WARPS) : NW, c = t.block * W + ch;
    const bool more = t.p + 1 < t.count;
    __syncthreads();
    const bool odd = M.odd == turn;
    if (odd) {
        again();
        __syncthreads();
    }
    const int q = links ? t.p % G : 0, gq = links ? t.p / G % G : 0, super = links ? t.p / (G * G) : 0;
    const int64_t slot = t.first + t.p;
    float sum = 0.f, v = 0.f, h = 0.f;
    auto warp_at = [](int i) { return BACK ? NW - 1 - i : i; };  // the warps in the direction of the scan
    constexpr int PITCH = BACK ? -W : W;
    if (role == 0) {
        if (t.p == 0) h = start && c < D ? start[(int64_t)t.n * D + c] : 0.f;
        else if (!links) h = M.from[ch];
    }
    if (links) {
        const unsigned long long *tiles = B.entry[0] + (slot - q) * D,
                                 *groups = B.entry[1] + ((int64_t)t.first / G + t.n + super * G) * D;
        if (role == 0) {
            if (more) {
#pragma unroll
                for (int i = 0; i < NW; ++i) {
                    const int w = warp_at(i);
                    sum += M.g[w][ch];
                    v = step(M.d[w][ch], v, M.b[w][ch]);
                }
                if (!finite(v)) v = fold_any(0.f, &M.d[warp_at(0)][ch], &M.b[warp_at(0)][ch], nullptr, PITCH, NW);
                sum = decay_of(sum).d;
                if (t.p == 0) {  // nothing enters the first tile: its value is the state behind it
                    v = step_any(sum, h, v);
                    sum = 0.f;
                }
                if (c < D) put(B.entry[0] + slot * D + c, sum, v);
            }
        }
        // A role's entries: the first groups (1), tiles (2) and more tiles (3), and, when its own is on its way, more groups (0).  One
        // piece of code for all of them: instructions that do not fit beside the rest of a tile's are fetched anew for each tile.
        {
            const int from = role == 0 || role == 3 ? BATCH : 0, all = role > 1 ? q : gq, n = all - from < BATCH ? all - from : BATCH;
            if (role < 4 && n > 0 && c < D) {
                unsigned long long e[BATCH];
                get_batch((role > 1 ? tiles : groups) + (int64_t)from * D + c, D, n, e, err);
#pragma unroll
                for (int i = 0; i < BATCH; ++i)
                    if (i < n) E[(role > 1 ? G : 1) + from + i][ch] = e[i];
            }
        }
        if (role == 0 && super > 0 && c < D) h = get_state(B.entry[2] + ((int64_t)t.first / (G * G) + t.n + super - 1) * D + c, err);
        __syncthreads();
    }
    if (role == 0) {
        if (links && c < D) {
            // the state behind `all` entries from the i-th one on
            auto over = [&](float h, int i, int all, float to) {
                const float *e = reinterpret_cast<const float *>(&E[i][ch]);
                return finite(to) ? to : fold_any(h, e, e + 1, nullptr, 2 * W, all);
            };
            if (q == G - 1 && more) {
                // (from the first tile's, so that decays near 1 are joined as a - 1)
                float gd = entry_d(E[G][ch]), gb = entry_b(E[G][ch]);
#pragma unroll
                for (int i = 1; i < G - 1; ++i) {
                    const unsigned long long x = E[G + i][ch];
                    gb = step(entry_d(x), gb, entry_b(x));
                    gd = compose(gd, entry_d(x));
                }
                gb = over(entry_b(E[G][ch]), G + 1, G - 2, gb);
                put(B.entry[1] + ((int64_t)t.first / G + t.n + t.p / G) * D + c, compose(gd, sum), step_any(sum, gb, v));
            }
            const float before = h;
            for (int i = 0; i < gq; ++i) h = step(entry_d(E[1 + i][ch]), h, entry_b(E[1 + i][ch]));
            h = over(before, 1, gq, h);
            const float behind = h;
            for (int i = 0; i < q; ++i) h = step(entry_d(E[G + i][ch]), h, entry_b(E[G + i][ch]));
            h = over(behind, G, q, h);
        }
        const float from = h;
        auto keep = [&](int w, float v) {
            if (!BACK && w * X::RW % CK == 0 && kept && w * X::RW / CK < room && c < D) kept[(int64_t)(w * X::RW / CK) * D + c] = v;
        };
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const int w = warp_at(i);
            keep(w, h);
            M.g[w][ch] = h;
            h = step(M.d[w][ch], h, M.b[w][ch]);
        }
        if (!finite(h)) {
            h = fold_any(from, &M.d[warp_at(0)][ch], &M.b[warp_at(0)][ch], &M.g[warp_at(0)][ch], PITCH, NW);
#pragma unroll 1
            for (int w = 0; w < NW; ++w) keep(w, M.g[w][ch]);
        }
        if (links && more && t.p % (G * G) == G * G - 1 && c < D)
            put(B.entry[2] + ((int64_t)t.first / (G * G) + t.n + super) * D + c, h, 0.f);
        if (end && c < D && !more) end[(int64_t)t.n * D + c] = h;
        M.from[ch] = h;
    } else if (role == 2 || role == 3) {
        more_work(role, ch);
    }
    __syncthreads();
    return odd;
}

// An entry of the plan (of the chains) of a call that has none.
static __device__ __noinline__ int4 unplanned(const int32_t *cu, int64_t T, int64_t N, int L, layout how, int64_t i) {
    int64_t n = i, p = 0;
    lin::span s;
    const bool good = how == EQUAL ? lin::seq_span(cu, T, N, i, &s) : lin::find_slot(cu, T, N, L, i, &n, &p, &s);
    if (!good || (p > 0 && p >= (s.b - s.a + L - 1) / L)) return make_int4(0, -1, 0, 0);
    return make_int4((int)n, (int)p, (int)s.a, (int)s.b);
}

// Where a block is in its tiles, in shared memory: one warp asks for them, and in registers it would be in everybody's way.
struct progress {
    tile t;        // the last one
    int64_t item;  // the chain's or the tile's place among the call's (-1: none yet)
};
// The tiles that a block goes through, as one warp of it finds them (p = -1 behind the last).
template <int L, bool PLAN> struct course {
    const board &B;
    progress &at;
    const int32_t *cu;
    int64_t T, N;
    int blocks;
    layout how;
    bool back, chains;
    __device__ __forceinline__ course(const board &b, progress &at_, const int32_t *cu_, int64_t T_, int64_t N_, int blocks_, layout how_, bool back_)
        : B(b), at(at_), cu(cu_), T(T_), N(N_), blocks(blocks_), how(how_), back(back_) {
        chains = PLAN ? planned_chains(B) : how == EQUAL;
        if (threadIdx.x == 0) at = progress{tile{0, -1, 0, 0, 0, 0, 0}, -1};  // (a barrier follows)
    }
    __device__ __forceinline__ tile next() {
        tile t = at.t;
        int64_t item = at.item;
        __syncwarp();
        const int64_t items = (chains ? N : lin::chunk_slots(T, N, L)) * blocks;
        next_tile<L>(t, chains, back, [&](tile *to) {
            if (PLAN && chains) {
                int ticket = 0;
                if ((threadIdx.x & 31) == 0) ticket = atomicAdd(B.mode + 1, 1);
                item = __shfl_sync(0xffffffffu, ticket, 0);
            } else {
                item = item < 0 ? blockIdx.x : item + gridDim.x;
            }
            if (item >= items) return false;
            const int64_t r = back && !chains ? items - 1 - item : item, i = r / blocks;
            to->block = (int)(r - i * blocks);
            const int4 q = PLAN ? __ldcg((chains ? B.order : B.plan) + i) : unplanned(cu, T, N, L, how, i);
            to->n = q.x, to->p = q.y, to->a = q.z, to->b = q.w;
            return true;
        });
        if ((threadIdx.x & 31) == 0) at = progress{t, item};
        __syncwarp();
        return t;
    }
};

// Sets the error of a call that has no plan (make_plan() does it for the others).
__device__ __forceinline__ void check_all(const int32_t *cu, int64_t T, int64_t N, int *err) {
    if (blockIdx.x > 0) return;
    for (int64_t n = threadIdx.x; n < N; n += NT) {
        lin::span s;
        if (!lin::seq_span(cu, T, N, n, &s)) set_error(err, KDA_ERR_BAD_SEQLENS);
    }
}

// Boxes of NI tensors of two tiles, and which tiles come next
template <typename T, int NI, typename X> struct ring {
    T x[2][NI][X::L][X::W];
    uint64_t full[2];
    tile t[4];
    progress way;
};
template <int NI> struct row_maps {
    CUtensorMap m[NI];
};
template <typename X> inline bool make_row_map(CUtensorMap *m, const void *base, int64_t T, int D, int64_t stride, kda_dtype_t dtype) {
    return layer::make_row_map(m, base, T, D, stride, dtype, X::W, X::BOX);
}
// Asks for a tile's rows of one tensor
template <typename X, typename T> __device__ __forceinline__ void load_rows(T *to, const CUtensorMap &m, int block, int tok, uint64_t *full) {
#pragma unroll
    for (int r = 0; r < X::L; r += X::BOX) tc::tma_load_3d(to + r * X::W, &m, block * X::W, 0, tok + r, full);
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

// Channels of a tile.  64 cost least: each row of a tile is two sectors or more, a warp has no groups to join, and its reads of shared
// memory no bank conflicts.  Fewer make more chains, so that more blocks have whole ones, of which the last ends sooner, and
// tiles of more tokens, of which fewer join where they have to.  At 64 / 32 / 16 channels, bf16 (f32), D = 4096, us: forwards 16384 tokens of one
// sequence (64 chains of 64 channels) 193 / 202 / 177, 131072 of D = 256 (4) 116 / 110 / 107 (191 / 147 / 134), 4 sequences (256) 224 / 195 / 193,
// 6 (384) 301 / 245 / 257 (406 / 285 / 301), 8 (512) 349 / 345 / 370, 12 (768) 439 / 454 / 504 (558 / 567 / 583), 32 (2048) 1006 / 1082 / 1219;
// gradients 8192 of one 227 / 237 / 209, 3 sequences (192) 268 / 271 / 247, 6 (384) 455 / 384 / 401, 12 (768) 682 / 731 / 770.
inline int tile_width(int64_t N, int D) {
    const int64_t chains = N * ((D + 63) / 64);
    return chains < 2 * 152 ? 16 : chains < 4 * 152 ? 32 : 64;
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
