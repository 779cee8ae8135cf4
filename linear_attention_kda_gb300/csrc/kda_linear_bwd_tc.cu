// Gradients of linear attention with a decay per head on the tensor cores: bf16 tensors, chunks of 128 tokens.
//
//   linear_bwd_states_tc_kernel  the chains over chunks, forwards S <- e^{G_C} S + (K e^{G_C - G})^T V and backwards
//                                Lambda <- e^{G_C} Lambda + scale (Q e^G)^T dO; before every chunk the state as it is
//                                goes to the workspace as operand images in two bf16 parts (hi + lo).  The zeros that
//                                a chain begins with where it is given no state are neither written nor multiplied.
//   linear_grads_tc_kernel       per (chunk, head): with A = scale Tril[Q K^T * D], dA = scale Tril[dO V^T * D],
//                                D = e^{G_r - G_t},
//                                    dQ = scale e^G (dO S^T) + dA K,   dK = f (V Lambda^T) + dA^T Q,
//                                    dV = f (K Lambda) + A^T dO,       f = e^{G_C - G},
//                                and the decay's gradient.
//
// Numerics: the chains' terms are fp32 products in three bf16 parts.  A, dA and the first parts of S and Lambda are
// rounded to bf16 once; they make bf16 gradients.  The decay's
// gradient is an fp32 result: the products that it is summed from, Q K^T, dO V^T, dO S^T and V Lambda^T, have exact
// bf16 operands or both parts of a state (2^-16), and are taken in fp32 before any rounding.
#include <type_traits>

#include "kda_linear_tc.cuh"

namespace kda {
namespace lin {
namespace tcl {
namespace bw {

constexpr int THREADS = 640;  // warps 0-3: loads, products, decays, stores; 16 warps that work on the results

struct states_dir {
    CUtensorMap a, b;      // forwards k and v, backwards q and grad_o
    int ra, rb;            // states per head of each
    const float *init;     // [N, H, dk, dv] or NULL
    float *fin;            // likewise
    unsigned char *images; // [slots, H] x (hi, lo) images
    float scale;
};
struct states_maps {
    states_dir d[2];
};
struct states_args {
    const float *g;
    int g_stride;
    const int32_t *cu;
    int64_t T, N;
    int H, lo;             // lo: the images' second parts are wanted
    int64_t seg, slots;    // chunks of a segment and segment slots; 0: a chain is one piece
    float *sums;           // [2 directions][slots, H][dk, dv] state behind a segment that begins with zeros (with the
    float *decay;          // initial state, the chain's first one), and its whole decay [2][slots, H]
    bool sum_pass;         // these are made, and nothing else
    int *err;
};

constexpr int W = 64;      // value columns of a CTA
// Barriers that the chunks' images take in turn when they have left.  The loader waits for image i - 2 of the tiles i that
// it is to fetch, and image i - 1 may have left by then: on one barrier for all images that looks as if neither had, and
// image i needs the very tile.
constexpr int IMAGE_BARS = 3;

template <int DK> struct states_smem {
    static constexpr int AT = C * DK * 2, BT = C * W * 2, STAGE = AT + BT, IMG = DK * W * 2;
    static constexpr int PARTS = 3 * STAGE;  // three parts of the scaled rows of the second tile
    static constexpr int DEC = PARTS + 3 * BT;
    static constexpr int BAR = DEC + 3 * (int)sizeof(decays);
    static constexpr int BYTES = BAR + 256;
    static_assert(2 * IMG <= AT, "a chunk's images leave through the rows' tile of the chunk before");
};

// The chain of 64 value columns of one (sequence, head), S [dk rows][64 columns] in the threads' registers.  A chunk's
// factors go to the tile of 64 columns (half the values of the other), as three parts side by side (with two, 2^-16 of a
// term, the decay's gradient was off by 1e-5), which take one product of 192 columns, made anew in tensor memory and
// added in fp32 registers, smallest part first: an accumulator that the chain itself ran through would lose a little at
// every K-step, always in one direction (2.6e-6 of a slowly decaying state).  Under a chunk's product the state before
// it goes to memory as images and the next chunk's rows are scaled and split.  Three stages of tiles: with two, a
// chunk's tiles were asked for when the last product but one had ended.
// 4096 tokens of 32 heads, d = 128: 62 us, 1.9 us a step, 0.64 of HBM for the tiles and images (the factors on the other
// tile and three products of 64 columns, in one accumulator or in three: 71 us).  Bound by what lies between two
// products: sum, images, split, two fences.
template <int DK, int DV, bool CUT>
__global__ void __launch_bounds__(THREADS, 1)
linear_bwd_states_tc_kernel(const __grid_constant__ states_maps dirs, const __grid_constant__ states_args a) {
    using L = states_smem<DK>;
    extern __shared__ __align__(1024) unsigned char sm[];
    decays *dec = reinterpret_cast<decays *>(sm + L::DEC);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BAR);
    // in: a chunk's tiles and its decays
    uint64_t *in = bars, *dec_free = bars + 3, *s_ready = bars + 6, *u_done = bars + 7, *stg_full = bars + 8,
             *stg_done = bars + 9;
    constexpr int BARS = 9 + IMAGE_BARS;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + BARS);
    int *fail = reinterpret_cast<int *>(tmem_slot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool back = blockIdx.y == 1;
    const states_dir &D = dirs.d[back];
    const int col = blockIdx.x % (DV / W);
    const int64_t piece = blockIdx.x / (DV / W), slot = piece / a.H;
    const int h = (int)(piece % a.H);
    int64_t n, index = 0;
    span sp;
    if (!CUT) {
        n = longest_first(a.cu, a.N, slot, fail + 1);
        if (!seq_span(a.cu, a.T, a.N, n, &sp)) {
            if (tid == 0) set_error(a.err, KDA_ERR_BAD_SEQLENS);
            return;
        }
    } else {
        if (blockIdx.x == 0 && blockIdx.y == 0) check_seqlens(a.cu, a.T, a.N, a.err);
        if (!find_slot(a.cu, a.T, a.N, a.seg * C, slot, &n, &index, &sp)) return;
    }
    const int64_t u = n * a.H + h;
    const int whole = (int)((sp.b - sp.a + C - 1) / C), c0 = CUT ? (int)(index * a.seg) : 0;  // chunks, first one here
    if (index > 0 && c0 >= whole) return;
    const int nc = CUT && whole - c0 > a.seg ? (int)a.seg : whole - c0;
    const bool left = c0 == 0, right = c0 + nc == whole, first = back ? right : left, last = back ? left : right;
    float *fin = last ? D.fin : nullptr;
    const bool sum_pass = CUT && a.sum_pass;
    const int64_t sum_at = (back ? a.slots : 0) * a.H + piece;
    if (sum_pass) {
        if (last) return;
        fin = a.sums + sum_at * (DK * DV);
    }
    const int64_t slot0 = sp.a / C + n;
    const int np = fin ? nc : nc - 1;                         // chunks whose products are wanted
    const int i0 = sum_pass ? nc : first && !D.init ? 1 : 0;  // first chunk whose state before it is
    if (np <= 0 && i0 >= nc && !fin) return;
    auto chunk_of = [&](int i) { return c0 + (back ? nc - 1 - i : i); };
    auto tok_of = [&](int i) { return sp.a + (int64_t)chunk_of(i) * C; };
    auto len_of = [&](int i) { const int64_t r = sp.b - tok_of(i); return (int)(r < C ? r : C); };
    if (tid == 0) {
        for (int i = 0; i < BARS; ++i) mbar_init(bars + i, i < 3 ? 2 : i == 7 || i >= 9 ? 1 : 16);
        *fail = 0;
    }
    if (warp == 1) tmem_alloc(tmem_slot, 512);
    fence_proxy_async();
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tb = *tmem_slot;
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) { ok = ok && __all_sync(0xffffffffu, bar_wait(bar, parity)); };
    auto image_bar = [&](int j) { return stg_done + j % IMAGE_BARS; };  // j: images before it
    auto image_phase = [&](int j) { return (uint32_t)(j / IMAGE_BARS) & 1; };

    if (warp == 0) {
        if (lane == 0) {
            const int ha = h / D.ra, hb = h / D.rb;
            int i = 0;
            for (; i < np; ++i) {
                unsigned char *st = sm + i % 3 * L::STAGE;
                const int t = (int)tok_of(i);
                // chunk i - 2's images have left by this stage; where there are none, chunk i - 3 has been used
                if (sum_pass ? i >= 3 : i >= 2 + i0)
                    ok = sum_pass ? bar_wait(u_done, (i - 3) & 1) : bar_wait(image_bar(i - 2 - i0), image_phase(i - 2 - i0));
                if (!ok) break;
                mbar_arrive_expect_tx(in + i % 3, L::STAGE);
                for (int b = 0; b < DK / 64; ++b) tma_load_3d(st + b * C * 128, &D.a, 64 * b, ha, t, in + i % 3);
                tma_load_3d(st + L::AT, &D.b, W * col, hb, t, in + i % 3);
            }
            if (!ok)  // copies still in flight land before the block ends
                for (int j = i > 2 ? i - 2 : 0; j < i; ++j) bar_wait(in + j % 3, (j / 3) & 1);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            const uint32_t id = idesc_bf16(128, 3 * W, true, true), parts = smem_u32(sm + L::PARTS);
            constexpr uint32_t ALBO = DK == 128 ? 16384 : 0;  // dk = 64: lanes 64 .. 127 repeat lanes 0 .. 63, unread
            for (int i = 0; i < np; ++i) {
                ok = bar_wait(s_ready, i & 1) && bar_wait(in + i % 3, (i / 3) & 1);
                if (!ok) break;
                fence_after_sync();
                mma_bf16_mnmn(tb + (i & 1) * 256, smem_u32(sm + i % 3 * L::STAGE), ALBO, parts, L::BT, C / 16, id, false);
                mma_commit(u_done);
            }
        }
    } else if (warp == 2) {
        auto load = [&](int i) {
            const bool is = i < np;
            return load_log_decays(a.g && is ? a.g + tok_of(i) * a.g_stride + h : nullptr, a.g_stride, is ? len_of(i) : 0);
        };
        float4 g = load(0);
        for (int i = 0; i < np; ++i) {
            const float4 next = load(i + 1);
            if (i >= 3) wait(dec_free + i % 3, (i / 3 - 1) & 1);
            if (!ok) break;
            make_decays(g, dec[i % 3]);
            g = next;
            if (lane == 0) mbar_arrive(in + i % 3);
        }
    } else if (warp == 3) {
        if (lane == 0) {
            for (int i = i0; i < nc; ++i) {
                unsigned char *dst = D.images + ((slot0 + chunk_of(i)) * a.H + h) * (int64_t)(2 * DK * DV * 2) + col * L::IMG;
                const unsigned char *src = sm + (i + 2) % 3 * L::STAGE;
                ok = bar_wait(stg_full, (i - i0) & 1);
                if (!ok) break;
                bulk_s2g(dst, src, L::IMG);
                if (a.lo) bulk_s2g(dst + DK * DV * 2, src + L::IMG, L::IMG);
                bulk_commit();
                bulk_wait_read0();
                mbar_arrive(image_bar(i - i0));
            }
        }
    } else {
        constexpr int KC = DK / 32, VC = W / 32, CW = W / 4;
        const int quarter = warp & 3, part = (warp - 4) >> 2, row = 32 * quarter + lane;
        const bool mine = row < DK;
        const uint32_t ts = tmem_addr(tb, 32 * quarter, CW * part);
        const int own = row * DV + W * col + CW * part;
        const int64_t at = u * (int64_t)(DK * DV) + own;
        auto arrive = [&](uint64_t *bar) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        uint4 hi[VC], mid[VC], low[VC];  // of the next chunk's rows
        auto split_rows = [&](int i) {
            const int len = len_of(i);
            unsigned char *st = sm + i % 3 * L::STAGE;
            wait(in + i % 3, (i / 3) & 1);
            if (!ok) return;
            const decays &d = dec[i % 3];
            const float f = back ? D.scale * expf(ends(d, quarter - 1, -1) + d.rel[row]) : expf(ends(d, 3, quarter)) * d.w[row];
            const float m = row < len ? f : 0.f;
            split_chunks<VC>(st + L::AT, row, VC * part, m, hi, mid, low);
            if (m == 0.f) clear_chunks<KC>(st, row, KC * part);  // (zeros times no number would be none)
        };
        float x[CW];
#pragma unroll
        for (int c = 0; c < CW; c += 4) {
            float4 v = make_float4(0, 0, 0, 0);
            if (mine && first && D.init) v = *reinterpret_cast<const float4 *>(D.init + at + c);
            x[c] = v.x, x[c + 1] = v.y, x[c + 2] = v.z, x[c + 3] = v.w;
        }
        if (!first && !sum_pass) {  // what the segments before this one leave, in the chain's order
            const int before = back ? (whole + (int)a.seg - 1) / (int)a.seg - 1 - (int)index : (int)index;
#pragma unroll 2
            for (int j = before; j > 0; --j) {
                const int64_t s = sum_at + (back ? j : -j) * (int64_t)a.H;
                const float f = a.decay[s];
                if (!mine) continue;
                erase(x, f);
#pragma unroll
                for (int c = 0; c < CW; c += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(a.sums + s * (DK * DV) + own + c);
                    x[c] = fmaf(x[c], f, v.x), x[c + 1] = fmaf(x[c + 1], f, v.y);
                    x[c + 2] = fmaf(x[c + 2], f, v.z), x[c + 3] = fmaf(x[c + 3], f, v.w);
                }
            }
        }
        if (np > 0) split_rows(0);
        float all = 1.f, decay = 1.f;
        auto add_products = [&](int i) {  // of chunk i, behind the whole decay of it
            float y[CW], z[CW];
            tmem_load<CW>(ts + (i & 1) * 256 + 2 * W, y);
            tmem_load<CW>(ts + (i & 1) * 256 + W, z);
#pragma unroll
            for (int c = 0; c < CW; ++c) y[c] += z[c];
            tmem_load<CW>(ts + (i & 1) * 256, z);
            erase(x, all);
#pragma unroll
            for (int c = 0; c < CW; ++c) x[c] = fmaf(x[c], all, y[c] + z[c]);
        };
        for (int i = 0; i < nc; ++i) {
            if (i > 0) {
                wait(u_done, (i - 1) & 1);
                if (!ok) break;
                fence_after_sync();
            }
            if (i < np) {
#pragma unroll
                for (int j = 0; j < VC; ++j) {
                    unsigned char *p = sm + L::PARTS + img_chunk_off(C, row, VC * part + j);
                    *reinterpret_cast<uint4 *>(p) = hi[j];
                    *reinterpret_cast<uint4 *>(p + L::BT) = mid[j];
                    *reinterpret_cast<uint4 *>(p + 2 * L::BT) = low[j];
                }
                fence_proxy_async();
                arrive(s_ready);
            }
            if (i > 0) add_products(i - 1);
            fence_before_sync();
            if (i < np) {
                all = expf(dec[i % 3].hi[3]);
                if (sum_pass) decay *= all;
                arrive(dec_free + i % 3);
            }
            if (i >= i0) {  // the images, under the product, by way of the rows' tile of the chunk before
                // (those before them have left, so that stg_full is never two phases ahead of who waits for it)
                if (i > i0) wait(image_bar(i - 1 - i0), image_phase(i - 1 - i0));
                if (!ok) break;
                if (mine) {
#pragma unroll
                    for (int c = 0; c < CW; c += 8) {
                        uint4 hi, lo;  // of the state
                        split2(x[c], x[c + 1], hi.x, lo.x);
                        split2(x[c + 2], x[c + 3], hi.y, lo.y);
                        split2(x[c + 4], x[c + 5], hi.z, lo.z);
                        split2(x[c + 6], x[c + 7], hi.w, lo.w);
                        unsigned char *p = sm + (i + 2) % 3 * L::STAGE + img_chunk_off(DK, row, (CW * part + c) / 8);
                        *reinterpret_cast<uint4 *>(p) = hi;
                        *reinterpret_cast<uint4 *>(p + L::IMG) = lo;
                    }
                }
                fence_proxy_async();
                arrive(stg_full);
            }
            if (i + 1 < np) split_rows(i + 1);
            if (!ok) break;
        }
        if (ok && np == nc && nc > 0) {
            wait(u_done, (nc - 1) & 1);
            if (ok) {
                fence_after_sync();
                add_products(nc - 1);
            }
        }
        if (ok && fin && mine) {
            fin += sum_pass ? own : at;
#pragma unroll
            for (int c = 0; c < CW; c += 4)
                *reinterpret_cast<float4 *>(fin + c) = make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]);
            if (sum_pass && col == 0 && row == 0 && part == 0) a.decay[sum_at] = decay;
        }
    }
    if (!ok) atomicExch(fail, 1);
    fence_before_sync();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tb, 512);
    if (tid == 0 && *fail) set_error(a.err, KDA_ERR_DEVICE_TIMEOUT);
}

// ---------------------------------------------------------------------------------------------------- gradients
struct grads_maps {
    CUtensorMap q, k, v, o, dq, dk, dv;
};
struct grads_args {
    const float *g;
    int g_stride;
    float scale;
    const int32_t *cu;
    int64_t T, N;
    int H, rq, rk, rv;
    int r;                              // heads of a block, all of one head of q and of k, or of k and of v
    const unsigned char *states, *adj;  // images of S before and Lambda behind every chunk
    bool init, fin;                     // the first chunks have an S, the last ones a Lambda
    bf16 *dq, *dk, *dv;
    float *pq, *pk, *pv;                // fp32 parts [T, H or H / r, d] instead, where other blocks share the row
    float *dg, *dg_slot;                // [T, H], or sums over a chunk [slots, H]; neither: no decay gradient
    int sms;
    int *err;
};

struct grads_sums {                     // per column quarter (or row quarter) of the chunk's 128 x 128 pieces
    float row[4][C], col[4][C], qdq[4][C], kdk[4][C], dot[16];
};

template <int DK, int DV> struct grads_smem {
    static constexpr int QT = C * DK * 2, VT = C * DV * 2, SI = DK * DV * 2, SQ = C * C * 2;
    static constexpr int Q = 0, K = Q + QT, O = K + QT;
    static constexpr int V = O + VT;         // values, then A
    static constexpr int B0 = V + SQ;        // S hi, then Lambda lo
    static constexpr int B1 = B0 + SI;       // S lo, then dA
    static constexpr int B2 = B1 + SQ;       // Lambda hi
    static constexpr int DEC = B2 + (SI > 9216 ? SI : 9216);
    static constexpr int RLO = DEC + (int)sizeof(decays);
    static constexpr int BAR = RLO + C * 4;
    static constexpr int BYTES = BAR + 160;
    static_assert(sizeof(grads_sums) <= DEC - B2, "sums lie over Lambda hi once its products are done");
};
static_assert(grads_smem<128, 128>::BYTES <= 227 * 1024, "shared memory");

// Sum over the 32 lanes of x[c], for every c: lane c's result.
__device__ __forceinline__ float transpose_sum(float *x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 16; n > 0; n >>= 1) {
        const bool up = lane & n;
#pragma unroll
        for (int c = 0; c < n; ++c) {
            const float give = up ? x[c] : x[c + n], keep = up ? x[c + n] : x[c];
            x[c] = keep + __shfl_xor_sync(0xffffffffu, give, n);
        }
    }
    return x[0];
}
// Sum over channels of a row's fp32 values with the bf16 tile's.
template <int CW>
__device__ __forceinline__ float row_dot(const float *x, const unsigned char *tile, int row, int c0) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < CW; c += 8) {
        const uint4 u = *reinterpret_cast<const uint4 *>(tile + img_chunk_off(C, row, (c0 + c) / 8));
        s = fmaf(x[c], bf_lo(u.x), s), s = fmaf(x[c + 1], bf_hi(u.x), s);
        s = fmaf(x[c + 2], bf_lo(u.y), s), s = fmaf(x[c + 3], bf_hi(u.y), s);
        s = fmaf(x[c + 4], bf_lo(u.z), s), s = fmaf(x[c + 5], bf_hi(u.z), s);
        s = fmaf(x[c + 6], bf_lo(u.w), s), s = fmaf(x[c + 7], bf_hi(u.w), s);
    }
    return s;
}

// What a block's heads share: there is one, q and k, or k and v (the heads' own gradients leave with each of them).
enum { ONE = 0, QK = 1, KV = 2 };
// tensor memory: X, then V Lambda^T, then (KV) K Lambda; Y, then dO S^T, then dV or (KV) dQ; dQ or (KV) dV, and dK, summed
// over the block's heads
enum { T_X = 0, T_Y = 128, T_S = 256, T_K = 384 };

// A block takes a chunk and r heads, one after the other.  Bound by latency: of a head's 8 to 14 us the ten products hold
// the tensor pipe a fifth, tiles and images come (256 KB) and results leave (96 KB) while little is computed, since no
// second block fits an SM; 4096 tokens of 32 heads, d = 128: 90 us; 32768 of 32 heads that share 8, dv = 64: 471 us.
template <int DK, int DV, int MODE>
__global__ void __launch_bounds__(THREADS, 1)
linear_grads_tc_kernel(const __grid_constant__ grads_maps tm, const __grid_constant__ grads_args a) {
    using L = grads_smem<DK, DV>;
    extern __shared__ __align__(1024) unsigned char sm[];
    decays &d = *reinterpret_cast<decays *>(sm + L::DEC);
    float *rel_lo = reinterpret_cast<float *>(sm + L::RLO);
    grads_sums &sums = *reinterpret_cast<grads_sums *>(sm + L::B2);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BAR);
    uint64_t *f_qk = bars, *f_ov = bars + 1, *f_s = bars + 2, *f_l = bars + 3, *f_ll = bars + 4, *xy_done = bars + 5,
             *q_done = bars + 6, *k_done = bars + 7, *dot_done = bars + 8, *a_ready = bars + 9, *v_done = bars + 10,
             *d_ready = bars + 11, *out_done = bars + 12, *dec_ready = bars + 13, *clean = bars + 14, *t_free = bars + 15,
             *end = bars + 16, *xy_read = bars + 17;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 18);
    int *fail = reinterpret_cast<int *>(tmem_slot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = MODE == ONE ? 1 : a.r, groups = a.H / per, h0 = (int)(blockIdx.x % groups) * per;
    const int slot = (int)(blockIdx.x / groups);
    const bool decay = a.dg || a.dg_slot;
    chunk c;
    if (!find_chunk<C>(a.cu, a.T, a.N, slot, &c)) {
        if (a.dg_slot)
            for (int i = tid; i < per; i += THREADS) a.dg_slot[(int64_t)slot * a.H + h0 + i] = 0.f;
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < 18; ++i)
            mbar_init(bars + i, i == 8 || i == 9 || i == 11 || i == 14 || i == 15 || i == 17 ? 16 : i == 16 ? 2 : 1);
        *fail = 0;
    }
    if (warp == 1) tmem_alloc(tmem_slot, 512);
    fence_proxy_async();
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tb = *tmem_slot;
    const int len = c.len, tok0 = (int)c.tok0;
    const bool has_s = !c.first || a.init, has_l = !c.last || a.fin;  // zeros otherwise
    bool ok = true;
    // Head i of the block is the i-th phase of every barrier, but that shared q and k come once.
    auto wait = [&](uint64_t *bar, uint32_t ph) { ok = ok && __all_sync(0xffffffffu, bar_wait(bar, ph)); };

    if (warp == 0) {
        if (lane == 0) {
            const int t = tok0;
            int n_qk = 0, n_ov = 0, n_s = 0, n_l = 0, n_ll = 0;  // copies asked for
            for (int i = 0; i < per; ++i) {
                const int h = h0 + i, ph = i & 1;
                const int64_t image = ((int64_t)slot * a.H + h) * (2 * L::SI);
                const unsigned char *S = a.states + image, *G = a.adj + image;
                // (the states first: their product with one another is taken while the tiles are on their way)
                if (has_s) {
                    if (i && !(ok = bar_wait(k_done, ph ^ 1))) break;
                    mbar_arrive_expect_tx(f_s, decay ? 2 * L::SI : L::SI);
                    ++n_s;
                    bulk_g2s(sm + L::B0, S, L::SI, f_s);
                }
                if (i && !(ok = bar_wait(out_done, ph ^ 1))) break;
                if (has_s && decay) bulk_g2s(sm + L::B1, S + L::SI, L::SI, f_s);
                auto lambda = [&] {
                    mbar_arrive_expect_tx(f_l, L::SI);
                    ++n_l;
                    bulk_g2s(sm + L::B2, G, L::SI, f_l);
                };
                if (!i && has_l) lambda();
                if (!i || MODE == KV) {
                    mbar_arrive_expect_tx(f_qk, i ? L::QT : 2 * L::QT);
                    ++n_qk;
                    for (int b = 0; b < DK / 64; ++b) {
                        tma_load_3d(sm + L::Q + b * C * 128, &tm.q, 64 * b, h / a.rq, t, f_qk);
                        if (!i) tma_load_3d(sm + L::K + b * C * 128, &tm.k, 64 * b, h / a.rk, t, f_qk);
                    }
                }
                auto load_o = [&] {
                    for (int b = 0; b < DV / 64; ++b) tma_load_3d(sm + L::O + b * C * 128, &tm.o, 64 * b, h, t, f_ov);
                };
                auto load_v = [&] {
                    for (int b = 0; b < DV / 64; ++b) tma_load_3d(sm + L::V + b * C * 128, &tm.v, 64 * b, h / a.rv, t, f_ov);
                };
                mbar_arrive_expect_tx(f_ov, 2 * L::VT);
                ++n_ov;
                // (a head's own gradient leaves by way of dO's or V's place)
                if (MODE == KV) load_o();
                else load_v();
                if (i && !(ok = bar_wait(end, ph ^ 1))) break;
                if (MODE == KV) load_v();
                else load_o();
                if (i && has_l) lambda();
                if (decay && has_l) {
                    if (!(ok = bar_wait(q_done, ph) && bar_wait(dot_done, ph))) break;
                    mbar_arrive_expect_tx(f_ll, L::SI);
                    ++n_ll;
                    bulk_g2s(sm + L::B0, G + L::SI, L::SI, f_ll);
                }
            }
            // copies land before the block ends, whatever the others have given up on
            auto landed = [&](uint64_t *bar, int n) { ok = (n == 0 || bar_wait(bar, (n - 1) & 1)) && ok; };
            landed(f_qk, n_qk);
            landed(f_ov, n_ov);
            landed(f_s, n_s);
            landed(f_l, n_l);
            landed(f_ll, n_ll);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            const uint32_t q = smem_u32(sm + L::Q), k = smem_u32(sm + L::K), o = smem_u32(sm + L::O), v = smem_u32(sm + L::V),
                           b0 = smem_u32(sm + L::B0), b1 = smem_u32(sm + L::B1), b2 = smem_u32(sm + L::B2);
            const uint32_t id_c = idesc_bf16(128, 128), id_k = idesc_bf16(128, DK), id_v = idesc_bf16(128, DV, false, true),
                           id_dq = idesc_bf16(128, DK, false, true), id_dk = idesc_bf16(128, DK, true, true),
                           id_dv = idesc_bf16(128, DV, true, true);
            for (int i = 0; i < per; ++i) {
                const int ph = i & 1;
                // a ragged chunk's tiles are to be cleared first, those that come with this head
                if (i && !(ok = bar_wait(t_free, ph ^ 1))) break;
                if ((!i || MODE == KV) && !(ok = bar_wait(f_qk, ph) && (len == C || bar_wait(clean, ph)))) break;
                fence_after_sync();
                mma_bf16_k(tb + T_X, q, C, k, C, DK / 16, id_c, false);
                if (!(ok = bar_wait(f_ov, ph) && (len == C || bar_wait(clean, ph)))) break;
                mma_bf16_k(tb + T_Y, o, C, v, C, DV / 16, id_c, false);
                mma_commit(xy_done);
                if (!(ok = bar_wait(xy_read, ph))) break;
                fence_after_sync();
                if (has_s) {
                    if (!(ok = bar_wait(f_s, ph))) break;
                    mma_bf16_k(tb + T_Y, o, C, b0, DK, DV / 16, id_k, false);
                    if (decay) mma_bf16_k(tb + T_Y, o, C, b1, DK, DV / 16, id_k, true);
                }
                mma_commit(q_done);
                if (has_l) {
                    if (!(ok = bar_wait(f_l, ph))) break;
                    mma_bf16_k(tb + T_X, v, C, b2, DK, DV / 16, id_k, false);
                    if (decay) {
                        if (!(ok = bar_wait(f_ll, ph))) break;
                        mma_bf16_k(tb + T_X, v, C, b0, DK, DV / 16, id_k, true);
                    }
                }
                mma_commit(k_done);
                if (!(ok = bar_wait(a_ready, ph))) break;
                fence_after_sync();
                if (has_l) mma_bf16_kmn(tb + (MODE == KV ? T_X : T_Y), k, C, b2, DK * 128, DK / 16, id_v, false);
                mma_commit(v_done);
                if (!(ok = bar_wait(d_ready, ph))) break;
                fence_after_sync();
                mma_bf16_kmn(tb + (MODE == KV ? T_Y : T_S), b1, C, k, 16384, C / 16, id_dq, true);
                mma_bf16_mnmn(tb + T_K, b1, 16384, q, 16384, C / 16, id_dk, true);
                mma_bf16_mnmn(tb + (MODE == KV ? T_S : T_Y), v, 16384, o, 16384, C / 16, id_dv, true);
                mma_commit(out_done);
            }
        }
    } else if (warp == 2) {
        for (int i = 0; i < per; ++i) {
            const float4 g = load_log_decays(a.g ? a.g + (int64_t)tok0 * a.g_stride + h0 + i : nullptr, a.g_stride, len);
            if (i) wait(end, (i - 1) & 1);
            if (!ok) break;
            make_decays(g, d, rel_lo);
            if (lane == 0) mbar_arrive(dec_ready);
        }
    } else if (warp == 3) {
        // What the next head, or the block that runs here next, will load (blocks start in order, one on each SM): its
        // way from memory is half of a block's time otherwise, since all blocks load at once and then compute at once.
        for (int i = 0; i < per; ++i) {
            const bool more = i + 1 < per;
            const int64_t next = more ? blockIdx.x : (int64_t)blockIdx.x + a.sms, at = next / groups;
            const int g = more ? h0 + i + 1 : (int)(next % groups) * per;
            chunk x = c;
            if (!more && (next >= gridDim.x || !find_chunk<C>(a.cu, a.T, a.N, at, &x))) break;
            if (lane) continue;
            ok = bar_wait(f_ov, i & 1) && ok;
            if (more) mbar_arrive(end);  // (f_ov is never two phases ahead of this wait)
            const int t = (int)x.tok0;
            const int64_t image = (at * a.H + g) * (int64_t)(2 * L::SI);
            if (!more || MODE == KV)
                for (int b = 0; b < DK / 64; ++b) {
                    tma_prefetch_3d(&tm.q, 64 * b, g / a.rq, t);
                    if (!more) tma_prefetch_3d(&tm.k, 64 * b, g / a.rk, t);
                }
            for (int b = 0; b < DV / 64; ++b) {
                tma_prefetch_3d(&tm.o, 64 * b, g, t);
                tma_prefetch_3d(&tm.v, 64 * b, g / a.rv, t);
            }
            if (!x.first || a.init) bulk_prefetch_l2(a.states + image, decay ? 2 * L::SI : L::SI);
            if (!x.last || a.fin) bulk_prefetch_l2(a.adj + image, decay ? 2 * L::SI : L::SI);
        }
    } else if (warp >= 4) {
        constexpr int KW = DK / 4, VW = DV / 4;
        const int quarter = warp & 3, part = (warp - 4) >> 2, row = 32 * quarter + lane;
        const uint32_t tl = tmem_addr(tb, 32 * quarter, 0);
        auto arrive = [&](uint64_t *bar) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
#pragma unroll 1
        for (int it = 0; it < per; ++it) {
        const int h = h0 + it, ph = it & 1;
        auto add_store = [&](auto width, uint32_t t, float *x) {  // onto the sum over the heads before
            constexpr int N = decltype(width)::value;
            if (it) {
#pragma unroll
                for (int i = 0; i < N; i += 16) {
                    float y[16];
                    tmem_load<16>(t + i, y);
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[i + j] += y[j];
                }
            }
            tmem_store<N>(t, x);
        };
        using kw = std::integral_constant<int, KW>;
        using vw = std::integral_constant<int, VW>;
        float dot = 0.f, qdq = 0.f, kdk = 0.f, w_row = 0.f, w_col = 0.f;
        if (decay && !(has_s && has_l)) {
            arrive(dot_done);
        } else if (decay) {  // <S, Lambda>, both parts of each; Lambda's second one straight from memory
            constexpr int PER = L::SI / 16 / 512;  // 16-byte pieces of a thread
            uint4 l[PER];
            const unsigned char *G = a.adj + ((int64_t)slot * a.H + h) * (2 * L::SI);
#pragma unroll
            for (int i = 0; i < PER; ++i) l[i] = __ldg(reinterpret_cast<const uint4 *>(G + L::SI) + (tid - 128) + 512 * i);
            wait(f_s, ph);
            wait(f_l, ph);
            if (ok) {
                float acc = 0.f;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int at = ((tid - 128) + 512 * i) * 16;
                    const uint4 s0 = *reinterpret_cast<const uint4 *>(sm + L::B0 + at), s1 = *reinterpret_cast<const uint4 *>(sm + L::B1 + at),
                                l0 = *reinterpret_cast<const uint4 *>(sm + L::B2 + at);
                    const uint4 l1 = l[i];
                    auto two = [&](uint32_t sh, uint32_t sl, uint32_t lh, uint32_t ll) {
                        acc = fmaf(bf_lo(sh) + bf_lo(sl), bf_lo(lh) + bf_lo(ll), acc);
                        acc = fmaf(bf_hi(sh) + bf_hi(sl), bf_hi(lh) + bf_hi(ll), acc);
                    };
                    two(s0.x, s1.x, l0.x, l1.x);
                    two(s0.y, s1.y, l0.y, l1.y);
                    two(s0.z, s1.z, l0.z, l1.z);
                    two(s0.w, s1.w, l0.w, l1.w);
                }
                dot = acc;
            }
            arrive(dot_done);
        }
        if (len < C) {  // rows behind the sequence are another's: zeros from here on
            wait(f_qk, MODE == KV ? ph : 0);
            wait(f_ov, ph);
            if (ok && row >= len) {
                if (!it || MODE == KV) clear_chunks<DK / 32>(sm + L::Q, row, DK / 32 * part);
                if (!it) clear_chunks<DK / 32>(sm + L::K, row, DK / 32 * part);
                clear_chunks<DV / 32>(sm + L::O, row, DV / 32 * part);
                clear_chunks<DV / 32>(sm + L::V, row, DV / 32 * part);
            }
            fence_proxy_async();
            arrive(clean);
        }
        // ---- A and dA, columns 32 part .. of the chunk, and what the decay's gradient takes from their products
        wait(dec_ready, ph);
        wait(xy_done, ph);
        uint32_t pa[16], pd[16];
        const float rel = d.rel[row], rlo = rel_lo[row];
        if (ok) fence_after_sync();
        if (ok && part <= quarter) {
            float x[32], y[32];
            tmem_ld32(tl + T_X + 32 * part, x);
            tmem_ld32(tl + T_Y + 32 * part, y);
            fence_before_sync();
            arrive(xy_read);
            if (part < quarter) {  // all of it before the row's own block
                const float u = a.scale * __expf(ends(d, quarter - 1, part) + rel);
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 w4 = *reinterpret_cast<const float4 *>(&d.w[32 * part + e]);
                    const float f[4] = {u * w4.x, u * w4.y, u * w4.z, u * w4.w};
                    float q[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) q[j] = y[e + j] * f[j];
                    pa[e / 2] = pack_bf16(x[e] * f[0], x[e + 1] * f[1]);
                    pa[e / 2 + 1] = pack_bf16(x[e + 2] * f[2], x[e + 3] * f[3]);
                    pd[e / 2] = pack_bf16(q[0], q[1]);
                    pd[e / 2 + 1] = pack_bf16(q[2], q[3]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[e + j] *= q[j];  // what passes from t to r
                        w_row += x[e + j];
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float p[2], q[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int t = 32 * part + e + j;
                        const float f = a.scale * __expf((rel - d.rel[t]) + (rlo - rel_lo[t]));
                        p[j] = t <= row ? x[e + j] * f : 0.f;
                        q[j] = t <= row ? y[e + j] * f : 0.f;
                        // (t = r adds the same to both of its sums and is left out of them)
                        x[e + j] = t < row ? x[e + j] * q[j] : 0.f;
                        w_row += x[e + j];
                    }
                    pa[e / 2] = pack_bf16(p[0], p[1]);
                    pd[e / 2] = pack_bf16(q[0], q[1]);
                }
            }
            if (decay) w_col = transpose_sum(x);
        } else {
            arrive(xy_read);
#pragma unroll
            for (int e = 0; e < 16; ++e) pa[e] = pd[e] = 0;
        }
        wait(q_done, ph);  // S has been read: dA may lie where its second part was
        if (decay) wait(dot_done, ph);
        if (ok) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint4 *>(sm + L::B1 + img_chunk_off(C, row, 4 * part + j)) =
                    make_uint4(pd[4 * j], pd[4 * j + 1], pd[4 * j + 2], pd[4 * j + 3]);
            // ---- dQ's first part
            fence_after_sync();
            float x[KW] = {};
            if (has_s) tmem_load<KW>(tl + T_Y + KW * part, x);
            const float e = expf(ends(d, quarter - 1, -1) + rel), se = a.scale * e;
            erase(x, e);
#pragma unroll
            for (int i = 0; i < KW; ++i) x[i] *= se;
            if (decay) qdq = row_dot<KW>(x, sm + L::Q, row, KW * part);
            if (MODE == KV) tmem_store<KW>(tl + T_Y + KW * part, x);
            else add_store(kw{}, tl + T_S + KW * part, x);
        }
        wait(k_done, ph);  // the values have been read: A may lie over them
        const float f = expf(ends(d, 3, quarter)) * d.w[row];
        if (ok) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint4 *>(sm + L::V + img_chunk_off(C, row, 4 * part + j)) =
                    make_uint4(pa[4 * j], pa[4 * j + 1], pa[4 * j + 2], pa[4 * j + 3]);
            fence_proxy_async();
            fence_before_sync();
        }
        if (MODE != KV) arrive(a_ready);
        if (ok) {  // ---- dK's first part
            fence_after_sync();
            float x[KW] = {};
            if (has_l) tmem_load<KW>(tl + T_X + KW * part, x);
            if (MODE == KV) {  // K Lambda comes where this was
                fence_before_sync();
                arrive(a_ready);
            }
            erase(x, f);
#pragma unroll
            for (int i = 0; i < KW; ++i) x[i] *= f;
            if (decay) kdk = row_dot<KW>(x, sm + L::K, row, KW * part);
            add_store(kw{}, tl + T_K + KW * part, x);
        } else if (MODE == KV) {
            arrive(a_ready);
        }
        wait(v_done, ph);  // ---- dV's first part; Lambda has been read
        if (ok) {
            fence_after_sync();
            float x[VW] = {};
            if (has_l) tmem_load<VW>(tl + (MODE == KV ? T_X : T_Y) + VW * part, x);
            erase(x, f);
#pragma unroll
            for (int i = 0; i < VW; ++i) x[i] *= f;
            if (MODE == KV) add_store(vw{}, tl + T_S + VW * part, x);
            else tmem_store<VW>(tl + T_Y + VW * part, x);
            tmem_st_wait();
            fence_before_sync();
        }
        arrive(d_ready);
        if (decay) {
            sums.row[part][row] = w_row;
            sums.col[quarter][32 * part + lane] = w_col;
            sums.qdq[part][row] = qdq;
            sums.kdk[part][row] = kdk;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
            if (lane == 0) sums.dot[warp - 4] = dot;
            bar_sync(1, 512);
            if (warp == 4 && ok) {
                // dg_t = sum_{r >= t} (pairs inside the chunk + outputs of S) + sum_{j < t} keys into Lambda
                //        + e^{G_C} <S, Lambda>; four tokens a lane
                float p[4], kk[4], after = 0.f, before = 0.f, whole = lane < 16 ? sums.dot[lane] : 0.f;
#pragma unroll
                for (int off = 8; off > 0; off >>= 1) whole += __shfl_xor_sync(0xffffffffu, whole, off);
                const float left = expf(d.hi[3]);
                whole = __shfl_sync(0xffffffffu, whole, 0);
                whole = left == 0.f ? 0.f : whole * left;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 4 * lane + i;
                    p[i] = kk[i] = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        p[i] += (sums.row[j][r] - sums.col[j][r]) + sums.qdq[j][r];
                        kk[i] += sums.kdk[j][r];
                    }
                    after += p[i];
                    before += kk[i];
                }
                const float own_after = after, own_before = before;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const float x = __shfl_down_sync(0xffffffffu, after, off), y = __shfl_up_sync(0xffffffffu, before, off);
                    if (lane + off < 32) after += x;
                    if (lane >= off) before += y;
                }
                after -= own_after;    // of later lanes
                before -= own_before;  // of earlier lanes
                float out[4], total = 0.f;
#pragma unroll
                for (int i = 3; i >= 0; --i) {
                    after += p[i];
                    out[i] = after;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    out[i] += before + whole;
                    before += kk[i];
                    const int r = 4 * lane + i;
                    if (r < len) {
                        if (a.dg) a.dg[(int64_t)(tok0 + r) * a.H + h] = out[i];
                        total += out[i];
                    }
                }
                if (a.dg_slot) {
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
                    if (lane == 0) a.dg_slot[(int64_t)slot * a.H + h] = total;
                }
            }
        }
        wait(out_done, ph);
        if (ok) {
            fence_after_sync();
            // whole chunks leave by TMA from where the tiles were; ragged ends, and fp32 parts of shared heads, row by row
            auto put = [&](auto width, uint32_t t, unsigned char *stage, bf16 *out, float *shared, int D, int heads, int head) {
                constexpr int N = decltype(width)::value;
                float x[N];
                tmem_load<N>(tl + t + N * part, x);
                const int64_t at = ((int64_t)(tok0 + row) * heads + head) * D + N * part;
                if (shared) {
                    if (row < len) {
#pragma unroll
                        for (int i = 0; i < N; i += 4)
                            *reinterpret_cast<float4 *>(shared + at + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                    }
                    return;
                }
#pragma unroll
                for (int i = 0; i < N; i += 8) {
                    const uint4 u = make_uint4(pack_bf16(x[i], x[i + 1]), pack_bf16(x[i + 2], x[i + 3]),
                                               pack_bf16(x[i + 4], x[i + 5]), pack_bf16(x[i + 6], x[i + 7]));
                    if (len == C) *reinterpret_cast<uint4 *>(stage + img_chunk_off(C, row, (N * part + i) / 8)) = u;
                    else if (row < len) *reinterpret_cast<uint4 *>(out + at + i) = u;
                }
            };
            const bool done = it + 1 == per;
            if (MODE == KV) {
                put(kw{}, T_Y, sm + L::V, a.dq, a.pq, DK, a.H, h);
                if (done) put(vw{}, T_S, sm + L::O, a.dv, a.pv, DV, groups, h0 / per);
            } else {
                if (done) put(kw{}, T_S, sm + L::Q, a.dq, a.pq, DK, groups, h0 / per);
                put(vw{}, T_Y, sm + L::O, a.dv, a.pv, DV, a.H, h);
            }
            if (done) put(kw{}, T_K, sm + L::K, a.dk, a.pk, DK, groups, h0 / per);
            fence_before_sync();
            fence_proxy_async();
        }
        arrive(t_free);
        bar_sync(1, 512);
        if (warp == 4 && lane == 0) {
            if (ok && len == C) {
                const int t = tok0;
                const bool last = it + 1 == per;
                if (!a.pq && (MODE == KV || last))
                    for (int b = 0; b < DK / 64; ++b)
                        tma_store_3d(&tm.dq, sm + (MODE == KV ? L::V : L::Q) + b * C * 128, 64 * b, h / a.rq, t);
                if (!a.pk && last)
                    for (int b = 0; b < DK / 64; ++b) tma_store_3d(&tm.dk, sm + L::K + b * C * 128, 64 * b, h / a.rk, t);
                if (!a.pv && (MODE != KV || last))
                    for (int b = 0; b < DV / 64; ++b) tma_store_3d(&tm.dv, sm + L::O + b * C * 128, 64 * b, h / a.rv, t);
                bulk_commit();
                bulk_wait_read0();
            }
            mbar_arrive(end);
        }
        }
    }
    if (!ok) atomicExch(fail, 1);
    fence_before_sync();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tb, 512);
    if (tid == 0 && *fail) set_error(a.err, KDA_ERR_DEVICE_TIMEOUT);
}

// ---------------------------------------------------------------------------------------------------- launches
// Heads that a block takes in turn, a divisor of those that share a head of q and one of k (or of k and v): the sum over
// them then stays with the block, which also loads what they share once.  As many as leave a block for every second SM.
// Whole calls, 32 heads, d = 128, 4 heads to a block and one: 8 heads of q and k, 16384 tokens 539 / 845 us, 4096 tokens
// 159 / 235, 2048 tokens 84 / 132 (a block for every SM, two heads: 116); 8 of k and v 542 / 841, 158 / 232, 84 / 131; one
// head of q and k, 1024 tokens: 4 heads to a block 60, one or two 74, all 32 298.
static int heads_of_block(int64_t slots, int H, int rq, int rk) {
    int r = 1;
    for (int d = 2; d <= rq && d <= rk; ++d)
        if (rq % d == 0 && rk % d == 0 && slots * (H / d) >= 76) r = d;
    return r;
}

// Chunks of a segment, 0 for chains in one piece.  A chain is one CTA's (two, dv = 128, and two directions), so few of them
// leave the GPU idle.  Cut into `want` pieces each, they take a pass that sums the pieces and one that runs them, each
// chunks / want steps long, and a launch more, which pays off where chunks - 2 chunks / want is above ten steps.
// Measured, dv = 128 unless said, cut and whole: 8192 tokens of 2 heads, dv = 64, 69 / 119 us, 8 heads 131 / 172, 12 heads
// 175 / 193; 65536 of 8 heads 815 / 1224; 2048 of 1 head 37 / 42; 1280 of 2 heads 35 / 33; four sequences of 2048
// and 6 heads, dv = 64, 74 / 68.
static int64_t chain_segment(int64_t T, int64_t N, int H, int dv) {
    const int64_t want = 152 / (2 * N * H * (dv / W)), chunks = (T + C - 1) / C / N;  // of a sequence, on average
    if (chunks * (want - 2) <= 10 * want) return 0;
    const int64_t seg = (chunks + want - 1) / want;
    return seg < 2 ? 2 : seg;
}

struct layout {
    int64_t slots, seg, seg_slots;
    int r, mode, nq, nk, nv;  // heads of a block, what they share, parts of a row of dQ, dK and dV
    size_t states, adj, pq, pk, pv, dg, sums, decay, total;
    layout(int64_t T, int64_t N, int H, int Hq, int Hk, int Hv, int dk, int dv) {
        auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
        slots = chunk_slots(T, N, C);
        mode = QK, r = heads_of_block(slots, H, H / Hq, H / Hk);
        if (r == 1) mode = KV, r = heads_of_block(slots, H, H / Hk, H / Hv);
        if (r == 1) mode = ONE;
        nq = mode == KV ? H : H / r, nk = H / r, nv = mode == KV ? H / r : H;
        const size_t each = up((size_t)slots * H * dk * dv * 4);
        size_t at = 0;
        states = at, at += each;
        adj = at, at += each;
        pq = at, at += nq != Hq ? up((size_t)T * nq * dk * 4) : 0;
        pk = at, at += nk != Hk ? up((size_t)T * nk * dk * 4) : 0;
        pv = at, at += nv != Hv ? up((size_t)T * nv * dv * 4) : 0;
        dg = at, at += up((size_t)slots * H * 4);
        seg = chain_segment(T, N, H, dv);
        seg_slots = seg ? T / (seg * C) + N : N;
        sums = at, at += seg ? up((size_t)seg_slots * H * dk * dv * 8) : 0;
        decay = at, at += seg ? up((size_t)seg_slots * H * 8) : 0;
        total = at;
    }
};

template <int DK, int DV>
static kda_status_t run(const kda_linear_bwd_args *a, char *ws, cudaStream_t stream, int *err) {
    const layout L(a->T, a->N, a->H, a->Hq, a->Hk, a->Hv, DK, DV);
    const int gs = a->g_per_token ? a->H : 0;
    states_maps sm;
    grads_maps gm;
    if (!make_token_map(&gm.q, a->q, a->T, a->Hq, DK) || !make_token_map(&gm.k, a->k, a->T, a->Hk, DK) ||
        !make_token_map(&gm.v, a->v, a->T, a->Hv, DV) || !make_token_map(&gm.o, a->grad_o, a->T, a->H, DV) ||
        !make_token_map(&gm.dq, a->grad_q, a->T, a->Hq, DK) || !make_token_map(&gm.dk, a->grad_k, a->T, a->Hk, DK) ||
        !make_token_map(&gm.dv, a->grad_v, a->T, a->Hv, DV))
        return KDA_ERR_CUDA;
    const int rq = a->H / a->Hq, rk = a->H / a->Hk, rv = a->H / a->Hv;
    sm.d[0] = {gm.k, gm.v, rk, rv, a->initial_state, nullptr, (unsigned char *)ws + L.states, 1.f};
    sm.d[1] = {gm.q, gm.o, rq, 1, a->grad_final_state, a->grad_initial_state, (unsigned char *)ws + L.adj, a->scale};
    states_args s{};
    s.g = a->g, s.g_stride = gs, s.cu = a->cu_seqlens, s.T = a->T, s.N = a->N, s.H = a->H, s.lo = a->grad_g != nullptr;
    s.seg = L.seg, s.slots = L.seg_slots, s.err = err;
    if (L.seg) s.sums = (float *)(ws + L.sums), s.decay = (float *)(ws + L.decay);
    constexpr int smem1 = states_smem<DK>::BYTES, smem2 = grads_smem<DK, DV>::BYTES;
    static std::atomic<uint64_t> whole_allowed{0}, cut_allowed{0}, grads_allowed[3];
    const auto chains = L.seg ? linear_bwd_states_tc_kernel<DK, DV, true> : linear_bwd_states_tc_kernel<DK, DV, false>;
    cudaError_t e = allow_smem(chains, smem1, L.seg ? cut_allowed : whole_allowed);
    if (e != cudaSuccess) return kda_cuda_status(e);
    const dim3 grid((unsigned)(L.seg_slots * a->H * (DV / W)), 2);
    for (int pass = L.seg ? 0 : 1; pass < 2; ++pass) {
        s.sum_pass = pass == 0;
        chains<<<grid, THREADS, smem1, stream>>>(sm, s);
        e = cudaGetLastError();
        if (e != cudaSuccess) return kda_cuda_status(e);
    }
    grads_args g{};
    g.g = a->g, g.g_stride = gs, g.scale = a->scale, g.cu = a->cu_seqlens, g.T = a->T, g.N = a->N, g.H = a->H;
    g.rq = rq, g.rk = rk, g.rv = rv;
    g.states = (const unsigned char *)ws + L.states, g.adj = (const unsigned char *)ws + L.adj;
    g.init = a->initial_state != nullptr, g.fin = a->grad_final_state != nullptr;
    g.dq = (bf16 *)a->grad_q, g.dk = (bf16 *)a->grad_k, g.dv = (bf16 *)a->grad_v;
    g.r = L.r;
    g.pq = L.nq != a->Hq ? (float *)(ws + L.pq) : nullptr;
    g.pk = L.nk != a->Hk ? (float *)(ws + L.pk) : nullptr;
    g.pv = L.nv != a->Hv ? (float *)(ws + L.pv) : nullptr;
    if (a->grad_g) {
        if (a->g_per_token) g.dg = a->grad_g;
        else g.dg_slot = (float *)(ws + L.dg);
    }
    g.err = err;
    int dev = 0;
    g.sms = 152;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&g.sms, cudaDevAttrMultiProcessorCount, dev);
    const auto grads = L.mode == ONE  ? linear_grads_tc_kernel<DK, DV, ONE>
                       : L.mode == QK ? linear_grads_tc_kernel<DK, DV, QK>
                                      : linear_grads_tc_kernel<DK, DV, KV>;
    e = allow_smem(grads, smem2, grads_allowed[L.mode]);
    if (e != cudaSuccess) return kda_cuda_status(e);
    grads<<<(unsigned)(L.slots * (a->H / L.r)), THREADS, smem2, stream>>>(gm, g);
    e = cudaGetLastError();
    if (e != cudaSuccess) return kda_cuda_status(e);
    return kda_linear_sum_parts(a, {g.pq, L.nq}, {g.pk, L.nk}, {g.pv, L.nv}, g.dg_slot, L.slots, stream);
}

}  // namespace bw
}  // namespace tcl
}  // namespace lin
}  // namespace kda

size_t kda_linear_bwd_tc_bytes(int64_t T, int64_t N, int H, int Hq, int Hk, int Hv, int dk, int dv) {
    return kda::lin::tcl::bw::layout(T, N, H, Hq, Hk, Hv, dk, dv).total;
}

kda_status_t kda_launch_linear_bwd_tc(const kda_linear_bwd_args *a, void *ws, cudaStream_t stream, int *err) {
    using namespace kda::lin::tcl::bw;
    if (a->dk == 128)
        return a->dv == 128 ? run<128, 128>(a, (char *)ws, stream, err) : run<128, 64>(a, (char *)ws, stream, err);
    return a->dv == 128 ? run<64, 128>(a, (char *)ws, stream, err) : run<64, 64>(a, (char *)ws, stream, err);
}
