// Prefill of linear attention with a decay per head on the tensor cores: bf16 tensors, chunks of 128 tokens.
//
//   linear_fwd_tc_kernel      one CTA runs the chain of a (sequence, head), or of one segment of it: per chunk
//                                 X = Q K^T,  P = Tril[X * e^{G_r - G_j}],  O = scale (P V + e^G (Q S)),
//                                 S <- e^{G_C} S + (K e^{G_C - G})^T V
//                             with S in fp32 on the chip, so that q, k and v are read once and o is written once.
//   linear_segments_tc_kernel where there are few chains: what each segment adds to the state, (K f)^T V over its
//                             chunks; the first kernel then begins every segment from those before it.
//
// Numerics: products take bf16 operands and add in fp32.  P and the state that multiplies Q are rounded to bf16 once
// (they go into bf16 outputs); the keys that go into the fp32 state are kept as two bf16 parts, K f = hi + lo, and
// take two products, so that a state is good to 2^-16 of its terms instead of 2^-8, 3e-6 as a norm.  (A third part, in the
// outputs' place between their stores: 1.5e-7, and 64 us for 59 on 4096 tokens of 32 heads, 643 for 580 on 32 ragged
// sequences; bf16 k and v carry 2^-9, and fp32 calls have the exact state.)  The tensor cores make each chunk's
// (K f)^T V by itself, and the threads add it to the state: an accumulator that a whole chain runs through is cut at every
// K-step, always towards zero (without decay -7.4e-5 of the state after 16,384 tokens and growing with their number; now
// below 1e-6 at any length).  It costs 2 % of a chain's step and up to 6 % where loads are late.
#include "kda_linear_tc.cuh"

namespace kda {
namespace lin {
namespace tcl {

// cuTensorMapEncodeTiled through the runtime's driver entry point (no link-time libcuda dependency).
typedef CUresult (*encode_fn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

bool make_token_map(CUtensorMap *m, const void *base, int64_t T, int heads, int D) {
    static const encode_fn encode = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (encode_fn)p;
    }();
    if (!encode) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)heads * D * 2};
    const cuuint32_t box[3] = {64, 1, C};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct maps {
    CUtensorMap q, k, v, o;
};

struct chain_args {
    const float *g;
    int g_stride;              // elements between tokens (0: one decay per head)
    float scale;
    const int32_t *cu;
    int64_t T, N;
    int H, rq, rk, rv;         // states, and states per head of q, k, v
    const float *initial;
    float *final;
    bf16 *o;
    int64_t seg;               // chunks of a segment; 0: one CTA per sequence and head
    float *sums;               // per (segment slot, head): [dv / 4][dk][4] fp32, what the segment leaves
    double *sum_g;             // and its log-decay
    int *err;
};

// What a CTA works on.
struct work {
    int64_t n, slot, tok0, chunks, index;  // sequence, segment slot, first token, chunks, segment of the sequence
    int64_t end;                           // behind the sequence's last token
    bool last;                             // the sequence's last segment
    int h;
};
__device__ __forceinline__ bool find_work(const chain_args &a, work *w, int *n_smem) {
    w->h = (int)(blockIdx.x % a.H);
    w->slot = blockIdx.x / a.H;
    span s;
    if (a.seg == 0) {
        w->n = longest_first(a.cu, a.N, w->slot, n_smem);
        w->index = 0;
        if (!seq_span(a.cu, a.T, a.N, w->n, &s)) return false;
        w->tok0 = s.a;
        w->chunks = (s.b - s.a + C - 1) / C;
        w->last = true;
    } else {
        const int64_t W = a.seg * C;
        if (!find_slot(a.cu, a.T, a.N, W, w->slot, &w->n, &w->index, &s)) return false;
        w->tok0 = s.a + w->index * W;
        if (w->index > 0 && w->tok0 >= s.b) return false;
        const int64_t c = (s.b - w->tok0 + C - 1) / C;
        w->chunks = c < a.seg ? c : a.seg;
        w->last = w->tok0 + W >= s.b;
    }
    w->end = s.b;
    return true;
}
// ---------------------------------------------------------------------------------------------------- forward
template <int DK, int DV> struct fwd_smem {
    static constexpr int TILE = C * (DK > DV ? DK : DV) * 2;
    static constexpr int SLOTS = 4;
    static constexpr int SIMG = SLOTS * TILE;           // bf16 S, rows dk, 64-column halves of dv
    static constexpr int LO = SIMG + DK * DV * 2;       // second parts of the scaled keys
    static constexpr int OUT = LO + C * DK * 2;         // outputs on their way to memory
    static constexpr int DEC = OUT + C * DV * 2;
    static constexpr int BAR = DEC + 2 * (int)sizeof(decays);
    static constexpr int BYTES = BAR + 256;
};
static_assert(sizeof(decays) % 16 == 0, "alignment");
static_assert(fwd_smem<128, 128>::BYTES <= 227 * 1024, "shared memory");

constexpr int FWD_THREADS = 640;
// Tensor memory columns: two that take turns (a chunk's X, over which P lies as bf16, in one; what it adds to the state in
// the other, from after P V of the chunk before to before X of the next), outputs, state.
enum { T_X = 0, T_D = 256, T_S = 384 };

// Warps: 0 loads tiles, 1 issues the products, 2 makes the decays; 4-19 work on what the products leave, all of them on
// one thing after the other: warp w has lane quarter w % 4 and column quarter (w - 4) / 4 of every 128 x 128 piece.
// (With four warps on each of keys, P, state and outputs instead, every piece took four times as long, most of it
// one warp's own latency, and a step of the chain 8400 cycles.)
//
// Tiles of 128 tokens go through a ring of four slots in the order Q K V Q K V ..., each freed by the product that
// reads it last.  Products are issued in the order X, Q S, (K f)^T V twice, P V; X of the next chunk stands behind P V, in
// other columns, and is made while the state is added up and the outputs leave; the state's part of a chunk (products, sum,
// image) has the outputs and P made beside it.  Q S lands where P V adds to it, its rows multiplied by e^G in between.
template <int DK, int DV>
__global__ void __launch_bounds__(FWD_THREADS, 1)
linear_fwd_tc_kernel(const __grid_constant__ maps tm, const __grid_constant__ chain_args a) {
    using L = fwd_smem<DK, DV>;
    extern __shared__ __align__(1024) unsigned char sm[];
    decays *dec = reinterpret_cast<decays *>(sm + L::DEC);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::BAR), *free_ = full + L::SLOTS, *dec_ready = free_ + L::SLOTS,
             *dec_free = dec_ready + 2, *x_done = dec_free + 2, *p_ready = x_done + 1, *s_ready = p_ready + 1,
             *k_ready = s_ready + 1, *u_done = k_ready + 1, *o_done = u_done + 1, *o_read = o_done + 1, *o_staged = o_read + 1, *o_stored = o_staged + 1,
             *d_done = o_stored + 1, *u_read = d_done + 1, *x_read = u_read + 1;  // x_read: one for each lane quarter
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(x_read + 4);
    int *fail = reinterpret_cast<int *>(tmem_slot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (blockIdx.x == 0) check_seqlens(a.cu, a.T, a.N, a.err);
    work w;
    if (!find_work(a, &w, fail)) return;
    __syncthreads();  // the place that held the sequence's number is used again
    if (tid == 0) {
        for (int i = 0; i < L::SLOTS; ++i) {
            mbar_init(full + i, 1);
            mbar_init(free_ + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(dec_ready + i, 1);
            mbar_init(dec_free + i, 16);
        }
        mbar_init(x_done, 1);
        mbar_init(p_ready, 16);
        mbar_init(s_ready, 16);
        mbar_init(k_ready, 16);
        mbar_init(u_done, 1);
        mbar_init(o_done, 1);
        mbar_init(o_read, 16);
        mbar_init(o_staged, 16);
        mbar_init(o_stored, 1);
        mbar_init(d_done, 1);
        mbar_init(u_read, 16);
        for (int i = 0; i < 4; ++i) mbar_init(x_read + i, 4);
        *fail = 0;
    }
    if (warp == 1) tmem_alloc(tmem_slot, 512);
    fence_proxy_async();
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tb = *tmem_slot;
    const int nc = (int)w.chunks;
    bool ok = true;
    // every lane of a warp waits, and they go on or give up together
    auto wait = [&](uint64_t *bar, uint32_t parity) { ok = ok && __all_sync(0xffffffffu, bar_wait(bar, parity)); };
    auto tile = [&](int t) { return sm + (t % L::SLOTS) * L::TILE; };
    auto tile_phase = [&](int t) { return (uint32_t)(t / L::SLOTS) & 1; };
    auto len_of = [&](int i) { const int64_t r = w.end - (w.tok0 + (int64_t)i * C); return (int)(r < C ? r : C); };

    if (warp == 0) {
        if (lane == 0) {
            const int hs[3] = {w.h / a.rq, w.h / a.rk, w.h / a.rv};
            int sent = 0;
            for (int t = 0; t < 3 * nc; ++t) {
                if (t >= L::SLOTS) ok = bar_wait(free_ + t % L::SLOTS, tile_phase(t) ^ 1);
                if (!ok) break;
                const int kind = t % 3, D = kind == 2 ? DV : DK;
                const CUtensorMap *m = kind == 0 ? &tm.q : kind == 1 ? &tm.k : &tm.v;
                uint64_t *bar = full + t % L::SLOTS;
                mbar_arrive_expect_tx(bar, C * D * 2);
                for (int b = 0; b < D / 64; ++b)
                    tma_load_3d(tile(t) + b * C * 128, m, 64 * b, hs[kind], (int)(w.tok0 + (int64_t)(t / 3) * C), bar);
                sent = t + 1;
            }
            if (!ok)  // copies still in flight land before the block ends
                for (int t = sent > L::SLOTS ? sent - L::SLOTS : 0; t < sent; ++t) bar_wait(full + t % L::SLOTS, tile_phase(t));
        }
    } else if (warp == 1) {
        if (elect_one()) {
            const uint32_t id_x = idesc_bf16(128, 128), id_d1 = idesc_bf16(128, DV, false, true),
                           id_u = idesc_bf16(128, DV, true, true);
            constexpr uint32_t KLBO = DK == 128 ? 16384 : 0;  // dk = 64: rows 64 .. 127 repeat rows 0 .. 63, unread
            const uint32_t simg = smem_u32(sm + L::SIMG), klo = smem_u32(sm + L::LO);
            auto x_of = [&](int i) {
                const int t = 3 * i;
                ok = ok && bar_wait(full + t % L::SLOTS, tile_phase(t)) && bar_wait(full + (t + 1) % L::SLOTS, tile_phase(t + 1));
                if (!ok) return;
                fence_after_sync();
                mma_bf16_k(tb + T_X + 128 * (i & 1), smem_u32(tile(t)), C, smem_u32(tile(t + 1)), C, DK / 16, id_x, false);
                mma_commit(x_done);
            };
#pragma unroll 1
            for (int i = 0; i < nc; ++i) {
                const uint32_t k = smem_u32(tile(3 * i + 1)), v = smem_u32(tile(3 * i + 2));
                const uint32_t x = tb + T_X + 128 * (i & 1), u = tb + T_X + 128 * (~i & 1);
                if (i > 0) ok = bar_wait(u_read, (i - 1) & 1);  // X may lie where the state's last part was
                x_of(i);
                ok = ok && bar_wait(s_ready, i & 1) && (i == 0 || bar_wait(o_read, (i - 1) & 1));
                if (!ok) break;
                fence_after_sync();
                mma_bf16_kmn(tb + T_D, smem_u32(tile(3 * i)), C, simg, DK * 128, DK / 16, id_d1, false);
                mma_commit(d_done);
                mma_commit(free_ + (3 * i) % L::SLOTS);
                ok = bar_wait(k_ready, i & 1) && bar_wait(full + (3 * i + 2) % L::SLOTS, tile_phase(3 * i + 2));
                if (!ok) break;
                fence_after_sync();
                mma_bf16_mnmn(u, k, KLBO, v, 16384, C / 16, id_u, false);
                mma_bf16_mnmn(u, klo, KLBO, v, 16384, C / 16, id_u, true);
                mma_commit(u_done);
                mma_commit(free_ + (3 * i + 1) % L::SLOTS);
                ok = bar_wait(p_ready, i & 1);
                if (!ok) break;
                fence_after_sync();
                mma_ts_mn(tb + T_D, x, v, 16384, C / 16, id_d1, true);
                mma_commit(o_done);
                mma_commit(free_ + (3 * i + 2) % L::SLOTS);
            }
        }
    } else if (warp == 2) {
        auto load = [&](int i) {
            return load_log_decays(a.g ? a.g + (w.tok0 + (int64_t)i * C) * a.g_stride + w.h : nullptr, a.g_stride,
                                   i < nc ? len_of(i) : 0);
        };
        float4 g = load(0);
        for (int i = 0; i < nc; ++i) {
            const float4 next = load(i + 1);
            if (i >= 2) wait(dec_free + (i & 1), ((i >> 1) - 1) & 1);
            if (!ok) break;
            make_decays(g, dec[i & 1]);
            g = next;
            if (lane == 0) mbar_arrive(dec_ready + (i & 1));
        }
    } else if (warp == 3) {
        if (lane == 0) {  // whole chunks of outputs leave by TMA
            for (int i = 0; i < nc && len_of(i) == C; ++i) {
                ok = bar_wait(o_staged, i & 1);
                if (!ok) break;
                for (int b = 0; b < DV / 64; ++b)
                    tma_store_3d(&tm.o, sm + L::OUT + b * C * 128, 64 * b, w.h, (int)(w.tok0 + (int64_t)i * C));
                bulk_commit();
                bulk_wait_read0();
                mbar_arrive(o_stored);
            }
        }
    } else if (warp >= 4) {
        constexpr int KC = DK / 32;  // 16-byte chunks of a key row that a thread scales
        constexpr int VC = DV / 32;  // ... of a value row
        constexpr int CW = DV / 4;   // columns of the state and of the outputs
        const int quarter = warp & 3, part = (warp - 4) >> 2, row = 32 * quarter + lane;
        const bool wide = ((uintptr_t)a.o & 31) == 0, mine = row < DK;
        const uint32_t tl = tmem_addr(tb, 32 * quarter, 0), ts = tl + T_S + CW * part;
        const int64_t state = (w.n * a.H + w.h) * (int64_t)(DK * DV) + (int64_t)row * DV + CW * part;
        auto arrive = [&](uint64_t *bar) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        {   // entering state: the initial one, or what the sequence's earlier segments leave
            float x[CW];
#pragma unroll
            for (int c = 0; c < CW; ++c) x[c] = 0.f;
            if (mine && w.index == 0 && a.initial) {
#pragma unroll
                for (int c = 0; c < CW; c += 4) {
                    const float4 u = *reinterpret_cast<const float4 *>(a.initial + state + c);
                    x[c] = u.x, x[c + 1] = u.y, x[c + 2] = u.z, x[c + 3] = u.w;
                }
            }
            if (mine && w.index > 0) {
                for (int64_t s = w.slot - w.index; s < w.slot; ++s) {
                    const float f = expf((float)a.sum_g[s * a.H + w.h]);
                    const float *p = a.sums + (s * a.H + w.h) * (int64_t)(DK * DV) + (CW * part * DK + row * 4);
                    erase(x, f);
#pragma unroll
                    for (int c = 0; c < CW; c += 4) {
                        const float4 u = __ldcg(reinterpret_cast<const float4 *>(p + c * DK));
                        x[c] = fmaf(x[c], f, u.x), x[c + 1] = fmaf(x[c + 1], f, u.y);
                        x[c + 2] = fmaf(x[c + 2], f, u.z), x[c + 3] = fmaf(x[c + 3], f, u.w);
                    }
                }
            }
            tmem_store<CW>(ts, x);
            tmem_st_wait();
        }
        auto load_state = [&](int i, float *x) {  // before chunk i, with what chunk i - 1 adds to it
            if (i == 0) {
                tmem_load<CW>(ts, x);
                return;
            }
#pragma unroll
            for (int c = 0; c < CW; c += 16) {
                float y[16];
                tmem_load_pair(ts + c, tl + T_X + 128 * (i & 1) + CW * part + c, x + c, y);
#pragma unroll
                for (int j = 0; j < 16; ++j) x[c + j] += y[j];
            }
            fence_before_sync();
            arrive(u_read);
        };
        for (int i = 0; i <= nc; ++i) {
            // ---- the state after chunk i - 1: its bf16 image, and itself times the chunk's whole decay
            if (i > 0) wait(u_done, (i - 1) & 1);
            if (i < nc) wait(dec_ready + (i & 1), (i >> 1) & 1);
            if (!ok) break;
            fence_after_sync();
            const decays &d = dec[i & 1];
            if (i < nc) {
                float x[CW];
                load_state(i, x);
                if (mine) {
                    unsigned char *img = sm + L::SIMG + (CW * part >> 6) * (DK * 128) + row * 128;
#pragma unroll
                    for (int c = 0; c < CW; c += 8)
                        *reinterpret_cast<uint4 *>(img + ((((CW * part & 63) + c) / 8 ^ (row & 7)) << 4)) =
                            make_uint4(pack_bf16(x[c], x[c + 1]), pack_bf16(x[c + 2], x[c + 3]),
                                       pack_bf16(x[c + 4], x[c + 5]), pack_bf16(x[c + 6], x[c + 7]));
                }
                const float all = expf(d.hi[3]);
                erase(x, all);
#pragma unroll
                for (int c = 0; c < CW; ++c) x[c] *= all;
                tmem_store<CW>(ts, x);
                tmem_st_wait();
                fence_proxy_async();
                fence_before_sync();
                arrive(s_ready);
            }
            // ---- outputs of chunk i - 1
            if (i > 0) {
                const int len = len_of(i - 1);
                if (i > 1) wait(o_stored, i & 1);  // chunk i - 2's have left
                wait(o_done, (i - 1) & 1);
                if (!ok) break;
                fence_after_sync();
                float x[CW];
                tmem_load<CW>(tl + T_D + CW * part, x);
                fence_before_sync();
                arrive(o_read);
#pragma unroll
                for (int b = 0; b < CW; b += 16) {
                    uint32_t u[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c) u[c] = pack_bf16(a.scale * x[b + 2 * c], a.scale * x[b + 2 * c + 1]);
                    const int c0 = CW * part + b;
                    if (len == C) {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            *reinterpret_cast<uint4 *>(sm + L::OUT + img_chunk_off(C, row, c0 / 8 + j)) =
                                make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
                    } else if (row < len) {  // a sequence's ragged end: the rows behind it are another's
                        st_row_32B(a.o + ((w.tok0 + (int64_t)(i - 1) * C + row) * a.H + w.h) * DV + c0, u, wide);
                    }
                }
                if (len == C) {
                    fence_proxy_async();
                    arrive(o_staged);
                }
            }
            if (i == nc) break;
            // ---- keys of chunk i, scaled
            const int len = len_of(i), tk = 3 * i + 1, tv = tk + 1;
            wait(x_done, i & 1);  // X has read the keys
            if (!ok) break;
            fence_after_sync();
            scale_chunks<KC>(tile(tk), sm + L::LO, row, KC * part, row < len ? expf(ends(d, 3, quarter)) * d.w[row] : 0.f);
            if (len < C) {  // values behind the sequence are another's: they meet zeros, which an infinity would spoil
                wait(full + tv % L::SLOTS, tile_phase(tv));
                if (!ok) break;
                if (row >= len) clear_chunks<VC>(tile(tv), row, VC * part);
            }
            fence_proxy_async();
            arrive(k_ready);
            // ---- P of chunk i, columns 32 part .., and the rows of Q S times e^G
            {
                const uint32_t tx = tl + T_X + 128 * (i & 1);
                const float rel = d.rel[row];
                float x[32];
                uint32_t p[16];
                if (part <= quarter) tmem_ld32(tx + 32 * part, x);
                if (part < quarter) {
                    const float u = __expf(ends(d, quarter - 1, part) + rel);
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        const float4 w4 = *reinterpret_cast<const float4 *>(&d.w[32 * part + c]);
                        p[c / 2] = pack_bf16(x[c] * (u * w4.x), x[c + 1] * (u * w4.y));
                        p[c / 2 + 1] = pack_bf16(x[c + 2] * (u * w4.z), x[c + 3] * (u * w4.w));
                    }
                } else if (part == quarter) {
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        const float4 r4 = *reinterpret_cast<const float4 *>(&d.rel[32 * part + c]);
                        const float rs[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[c + j] = c + j <= lane ? x[c + j] * __expf(rel - rs[j]) : 0.f;
                        p[c / 2] = pack_bf16(x[c], x[c + 1]);
                        p[c / 2 + 1] = pack_bf16(x[c + 2], x[c + 3]);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 16; ++c) p[c] = 0;
                }
                fence_before_sync();
                // The quarter's X is read: P may lie over it.  (A wait with a limit, as all others here: at a hardware
                // barrier a warp would stay for good where another one's wait has run out before it.)
                arrive(x_read + quarter);
                wait(x_read + quarter, i & 1);
                if (!ok) break;
                fence_after_sync();
                tmem_st16u(tx + 16 * part, p);
                wait(d_done, i & 1);
                if (!ok) break;
                fence_after_sync();
                const float e = expf(ends(d, quarter - 1, -1) + rel);
                float y[CW];
                tmem_load<CW>(tl + T_D + CW * part, y);
                erase(y, e);
#pragma unroll
                for (int c = 0; c < CW; ++c) y[c] *= e;
                tmem_store<CW>(tl + T_D + CW * part, y);
                tmem_st_wait();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(p_ready);
                    mbar_arrive(dec_free + (i & 1));
                }
            }
        }
        if (ok && w.last && a.final) {  // the loop's last round has waited for the last state products
            float x[CW];
            load_state(nc, x);
            if (mine) {
#pragma unroll
                for (int c = 0; c < CW; c += 4)
                    *reinterpret_cast<float4 *>(a.final + state + c) = make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]);
            }
        }
    }
    if (!ok) atomicExch(fail, 1);
    fence_before_sync();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tb, 512);
    if (tid == 0 && *fail) set_error(a.err, KDA_ERR_DEVICE_TIMEOUT);
}

// ---------------------------------------------------------------------------------------------------- segments
template <int DK, int DV> struct seg_smem {
    static constexpr int KT = C * DK * 2, VT = C * DV * 2, STAGE = KT + VT;
    static constexpr int STAGES = 2;
    static constexpr int LO = STAGES * STAGE;
    static constexpr int DEC = LO + STAGES * KT;
    static constexpr int BAR = DEC + 2 * (int)sizeof(decays);
    static constexpr int BYTES = BAR + 128;
};
constexpr int SEG_THREADS = 640;

// Every segment but a sequence's last: the state that its tokens leave behind (the first one's begins from the
// initial state), in the threads' registers; a chunk's products are added to it as in the forward kernel.  Warps as there;
// each chunk's keys are scaled before the last one's products are waited for.
template <int DK, int DV>
__global__ void __launch_bounds__(SEG_THREADS, 1)
linear_segments_tc_kernel(const __grid_constant__ maps tm, const __grid_constant__ chain_args a) {
    using L = seg_smem<DK, DV>;
    extern __shared__ __align__(1024) unsigned char sm[];
    decays *dec = reinterpret_cast<decays *>(sm + L::DEC);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::BAR), *free_ = full + 2, *dec_ready = free_ + 2,
             *dec_free = dec_ready + 2, *ready = dec_free + 2, *u_done = ready + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(u_done + 1);
    int *fail = reinterpret_cast<int *>(tmem_slot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    work w;
    if (!find_work(a, &w, fail) || w.last) return;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(full + i, 1);
            mbar_init(free_ + i, 1);
            mbar_init(dec_ready + i, 1);
            mbar_init(dec_free + i, 16);
        }
        mbar_init(ready, 16);
        mbar_init(u_done, 1);
        *fail = 0;
    }
    if (warp == 1) tmem_alloc(tmem_slot, DV);
    fence_proxy_async();
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tb = *tmem_slot;
    const int nc = (int)w.chunks;
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) { ok = ok && __all_sync(0xffffffffu, bar_wait(bar, parity)); };

    if (warp == 0) {
        if (lane == 0) {
            const int hk = w.h / a.rk, hv = w.h / a.rv;
            int i = 0;
            for (; i < nc; ++i) {
                if (i >= 2) ok = bar_wait(free_ + (i & 1), ((i >> 1) - 1) & 1);
                if (!ok) break;
                unsigned char *st = sm + (i & 1) * L::STAGE;
                const int t = (int)(w.tok0 + (int64_t)i * C);
                mbar_arrive_expect_tx(full + (i & 1), L::STAGE);
                for (int b = 0; b < DK / 64; ++b) tma_load_3d(st + b * C * 128, &tm.k, 64 * b, hk, t, full + (i & 1));
                for (int b = 0; b < DV / 64; ++b) tma_load_3d(st + L::KT + b * C * 128, &tm.v, 64 * b, hv, t, full + (i & 1));
            }
            if (!ok)
                for (int j = i > 2 ? i - 2 : 0; j < i; ++j) bar_wait(full + (j & 1), (j >> 1) & 1);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            const uint32_t id_u = idesc_bf16(128, DV, true, true);
            constexpr uint32_t KLBO = DK == 128 ? 16384 : 0;
            for (int i = 0; i < nc; ++i) {
                const uint32_t st = smem_u32(sm + (i & 1) * L::STAGE);
                ok = bar_wait(ready, i & 1) && bar_wait(full + (i & 1), (i >> 1) & 1);
                if (!ok) break;
                fence_after_sync();
                mma_bf16_mnmn(tb, st, KLBO, st + L::KT, 16384, C / 16, id_u, false);
                mma_bf16_mnmn(tb, smem_u32(sm + L::LO + (i & 1) * L::KT), KLBO, st + L::KT, 16384, C / 16, id_u, true);
                mma_commit(u_done);
                mma_commit(free_ + (i & 1));
            }
        }
    } else if (warp == 2) {
        double total = 0.0;
        auto load = [&](int i) {
            return load_log_decays(a.g ? a.g + (w.tok0 + (int64_t)i * C) * a.g_stride + w.h : nullptr, a.g_stride,
                                   i < nc ? C : 0);
        };
        float4 g = load(0);
        for (int i = 0; i < nc; ++i) {
            const float4 next = load(i + 1);
            if (i >= 2) wait(dec_free + (i & 1), ((i >> 1) - 1) & 1);
            if (!ok) break;
            make_decays(g, dec[i & 1]);
            g = next;
            total += (double)dec[i & 1].hi[3] + (double)dec[i & 1].lo[3];
            if (lane == 0) mbar_arrive(dec_ready + (i & 1));
        }
        if (lane == 0) a.sum_g[w.slot * a.H + w.h] = total;
    } else if (warp >= 4) {
        constexpr int KC = DK / 32, CW = DV / 4;
        const int quarter = warp & 3, part = (warp - 4) >> 2, row = 32 * quarter + lane;
        const bool mine = row < DK;
        const uint32_t ts = tmem_addr(tb, 32 * quarter, CW * part);
        float x[CW];
        const float *s0 = w.index == 0 && a.initial && mine
                              ? a.initial + (w.n * a.H + w.h) * (int64_t)(DK * DV) + (int64_t)row * DV + CW * part : nullptr;
#pragma unroll
        for (int c = 0; c < CW; ++c) x[c] = s0 ? s0[c] : 0.f;
        auto add_products = [&](int i) {  // of chunk i
            wait(u_done, i & 1);
            if (!ok) return;
            fence_after_sync();
#pragma unroll
            for (int c = 0; c < CW; c += 16) {
                float y[16];
                tmem_load<16>(ts + c, y);
#pragma unroll
                for (int j = 0; j < 16; ++j) x[c + j] += y[j];
            }
        };
        for (int i = 0; i < nc; ++i) {
            wait(dec_ready + (i & 1), (i >> 1) & 1);
            wait(full + (i & 1), (i >> 1) & 1);
            if (!ok) break;
            const decays &d = dec[i & 1];
            scale_chunks<KC>(sm + (i & 1) * L::STAGE, sm + L::LO + (i & 1) * L::KT, row, KC * part,
                             expf(ends(d, 3, quarter)) * d.w[row]);
            const float all = expf(d.hi[3]);
            if (i > 0) add_products(i - 1);
            if (!ok) break;
            erase(x, all);
#pragma unroll
            for (int c = 0; c < CW; ++c) x[c] *= all;
            fence_proxy_async();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(ready);
                mbar_arrive(dec_free + (i & 1));
            }
        }
        if (ok) add_products(nc - 1);
        if (ok) {
            float *p = a.sums + (w.slot * a.H + w.h) * (int64_t)(DK * DV) + (CW * part * DK + row * 4);
            if (mine) {
#pragma unroll
                for (int c = 0; c < CW; c += 4)
                    *reinterpret_cast<float4 *>(p + c * DK) = make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]);
            }
        }
    }
    if (!ok) atomicExch(fail, 1);
    fence_before_sync();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tb, DV);
    if (tid == 0 && *fail) set_error(a.err, KDA_ERR_DEVICE_TIMEOUT);
}

// ---------------------------------------------------------------------------------------------------- launches
// Chunks of a segment, 0 for one chain per sequence and head.  A chain has one SM to itself, so fewer chains than
// half of the SMs leave the GPU idle; segments of at least two chunks are then cut until there is a CTA for every SM.
// Measured, d = 128, cut and whole: 4096 tokens of 1 head 28 / 106 us, 32 heads 55 / 110, 76 heads 96 / 111, 96 heads
// 154 / 112; 32 heads of 2048 tokens 33 / 59, 1024 24 / 33, 640 20 / 23, 512 22 / 20.
static int64_t segment_chunks(int64_t T, int64_t N, int H) {
    const int64_t chains = N * H, chunks = (T + C - 1) / C;  // of all sequences together
    if (chains > 76 || chunks <= 4 * N) return 0;
    const int64_t per_chain = (chunks + N - 1) / N, want = 152 / chains;
    const int64_t seg = (per_chain + want - 1) / want;
    return seg < 2 ? 2 : seg;
}
struct fwd_layout {
    int64_t seg, slots;
    size_t sums, sum_g, init, total;
    fwd_layout(int64_t T, int64_t N, int H, int dk, int dv) {
        auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
        seg = segment_chunks(T, N, H);
        slots = seg ? T / (seg * C) + N : N;
        size_t at = 0;
        sums = at, at += seg ? up((size_t)slots * H * dk * dv * 4) : 0;
        sum_g = at, at += seg ? up((size_t)slots * H * 8) : 0;
        init = at, at += seg ? up((size_t)N * H * dk * dv * 4) : 0;
        total = at;
    }
};

template <int DK, int DV>
static kda_status_t fwd(const kda_linear_args *a, char *ws, cudaStream_t stream, int *err) {
    const fwd_layout L(a->T, a->N, a->H, DK, DV);
    maps tm;
    if (!make_token_map(&tm.q, a->q, a->T, a->Hq, DK) || !make_token_map(&tm.k, a->k, a->T, a->Hk, DK) ||
        !make_token_map(&tm.v, a->v, a->T, a->Hv, DV) || !make_token_map(&tm.o, a->o, a->T, a->H, DV))
        return KDA_ERR_CUDA;
    chain_args c{};
    c.g = a->g, c.g_stride = a->g_per_token ? a->H : 0, c.scale = a->scale;
    c.cu = a->cu_seqlens, c.T = a->T, c.N = a->N, c.H = a->H;
    c.rq = a->H / a->Hq, c.rk = a->H / a->Hk, c.rv = a->H / a->Hv;
    c.initial = a->initial_state, c.final = a->final_state, c.o = (bf16 *)a->o;
    c.seg = L.seg, c.sums = (float *)(ws + L.sums), c.sum_g = (double *)(ws + L.sum_g), c.err = err;
    const unsigned grid = (unsigned)(L.slots * a->H);
    if (L.seg) {
        if (a->initial_state && a->initial_state == a->final_state) {
            // the last segments write final states while the first ones still read initial states: read a copy
            const cudaError_t e = cudaMemcpyAsync(ws + L.init, a->initial_state, (size_t)a->N * a->H * DK * DV * 4,
                                                  cudaMemcpyDeviceToDevice, stream);
            if (e != cudaSuccess) return kda_cuda_status(e);
            c.initial = (const float *)(ws + L.init);
        }
        constexpr int smem = seg_smem<DK, DV>::BYTES;
        static std::atomic<uint64_t> allowed{0};
        cudaError_t e = allow_smem(linear_segments_tc_kernel<DK, DV>, smem, allowed);
        if (e != cudaSuccess) return kda_cuda_status(e);
        linear_segments_tc_kernel<DK, DV><<<grid, SEG_THREADS, smem, stream>>>(tm, c);
        e = cudaGetLastError();
        if (e != cudaSuccess) return kda_cuda_status(e);
    }
    constexpr int smem = fwd_smem<DK, DV>::BYTES;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(linear_fwd_tc_kernel<DK, DV>, smem, allowed);
    if (e != cudaSuccess) return kda_cuda_status(e);
    linear_fwd_tc_kernel<DK, DV><<<grid, FWD_THREADS, smem, stream>>>(tm, c);
    return kda_cuda_status(cudaGetLastError());
}

}  // namespace tcl
}  // namespace lin
}  // namespace kda

size_t kda_linear_fwd_tc_bytes(int64_t T, int64_t N, int H, int dk, int dv) {
    return kda::lin::tcl::fwd_layout(T, N, H, dk, dv).total;
}

kda_status_t kda_launch_linear_fwd_tc(const kda_linear_args *a, void *ws, cudaStream_t stream, int *err) {
    using namespace kda::lin::tcl;
    if (a->dk == 128)
        return a->dv == 128 ? fwd<128, 128>(a, (char *)ws, stream, err) : fwd<128, 64>(a, (char *)ws, stream, err);
    return a->dv == 128 ? fwd<64, 128>(a, (char *)ws, stream, err) : fwd<64, 64>(a, (char *)ws, stream, err);
}
