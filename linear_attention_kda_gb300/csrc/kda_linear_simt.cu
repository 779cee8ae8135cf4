// Linear attention with a decay per head in fp32 on the CUDA cores: every product of the chunked form (chunks of
// C = 64 tokens), forward and backward, for fp32 tensors.  Bound by shared memory and FMA issue; 4096 tokens of 32
// heads, d = 128, replayed from a graph: 0.57 ms forward and 1.27 ms backward, where bf16 tensors take 0.056 and 0.162 on
// the tensor cores, and 64 tokens 29 / 70 us against 10 / 18, so that bf16 goes there at every length.
//
//   linear_states_kernel  the recurrence over chunks, S <- e^{G_C} S + (K e^{G_C - G})^T V, and backwards
//                         Lambda <- e^{G_C} Lambda + scale (Q e^G)^T dO; leaves each chunk's entering S and
//                         leaving Lambda in the workspace, the final S / the initial state's gradient in the outputs.
//                         Value columns are independent: a CTA takes 32 of one (sequence, head)'s.
//   linear_out_kernel     per (chunk, head): O = scale (Tril[Q K^T * D] V + e^G Q S), D = e^{G_r - G_j}
//   linear_grads_kernel   per (chunk, head): dQ, dK, dV and the decay's gradient
//   linear_sum_heads_kernel, linear_sum_decay_kernel   sums over the heads that share a row, and over tokens
//                         where g is one per head; in a fixed order, so that results repeat to the bit.
#include "kda_internal.h"
#include "kda_linear.cuh"

namespace kda {
namespace lin {

constexpr int C = 64;
constexpr int NT = 256;

// C x D tile (rows of `stride` elements in memory, zeros behind `len`) to shared memory rows of `pitch` floats.
template <int D>
__device__ __forceinline__ void load_tile(float *s, int pitch, const float *p, int64_t stride, int len) {
    constexpr int V = 4, PER = D / V;
#pragma unroll 4
    for (int e = threadIdx.x; e < C * PER; e += NT) {
        const int r = e / PER, c = (e % PER) * V;
        float4 x = r < len ? *reinterpret_cast<const float4 *>(p + r * stride + c) : make_float4(0, 0, 0, 0);
        *reinterpret_cast<float4 *>(s + r * pitch + c) = x;
    }
}

// ------------------------------------------------------------------------------------------- states
struct states_args {
    const void *k, *v;        // forwards k and v; backwards q and grad_o
    int Hk, Hv;               // their heads
    const float *init;        // [N, H, dk, dv] or NULL
    float *fin;               // likewise
    float *each;              // [slots, H, dk, dv] state before each chunk in this direction, or NULL
    float scale;              // of the products
};

template <int DK, int DV>
__global__ void __launch_bounds__(NT) linear_states_kernel(states_args fwd, states_args bwd, const float *g,
                                                           int g_stride, int g_tok, const int32_t *cu, int64_t tokens,
                                                           int64_t N, int H, int *err) {
    constexpr int CW = 32;               // value columns of a CTA
    constexpr int TN = DK / 32;          // columns of a thread (4 rows x TN columns)
    constexpr int CG = CW / TN;          // column groups
    constexpr int SPLIT = DV / CW;
    constexpr int V = 4;
    constexpr int KE = C * DK / V / NT, VE = C * CW / V / NT;  // 16-byte pieces of a thread
    __shared__ __align__(16) float s_k[C][DK], s_v[C][CW];
    __shared__ float s_hi[2][C], s_lo[2][C], s_f[2][C];
    const bool back = blockIdx.y == 1;
    const states_args &A = back ? bwd : fwd;
    const int part = blockIdx.x % SPLIT;
    const int64_t unit = blockIdx.x / SPLIT, n = unit / H;
    const int h = (int)(unit % H);
    const int tid = threadIdx.x, r0 = (tid / CG) * 4, c0 = (tid % CG) * TN;
    span sp;
    if (!seq_span(cu, tokens, N, n, &sp)) {
        if (tid == 0) set_error(err, KDA_ERR_BAD_SEQLENS);
        return;
    }
    const int64_t at = unit * (int64_t)(DK * DV) + part * CW + c0;
    const int rk = H / A.Hk, rv = H / A.Hv;
    const float *k = (const float *)A.k + (int64_t)(h / rk) * DK, *v = (const float *)A.v + (int64_t)(h / rv) * DV + part * CW;
    const int64_t chunks = (sp.b - sp.a + C - 1) / C, slot0 = sp.a / C + n;
    auto chunk_of = [&](int64_t i) { return back ? chunks - 1 - i : i; };
    // the next chunk's tiles wait in registers while this one's are used
    float4 kx[KE], vx[VE];
    float gx[C / 32];
    auto fetch = [&](int64_t i) {
        if (i >= chunks) return;
        const int64_t t0 = sp.a + chunk_of(i) * C;
        const int len = (int)(sp.b - t0 < C ? sp.b - t0 : C);
#pragma unroll
        for (int j = 0; j < KE; ++j) {
            const int e = tid + NT * j, r = e / (DK / V), c = (e % (DK / V)) * V;
            kx[j] = r < len ? *reinterpret_cast<const float4 *>(k + (t0 + r) * A.Hk * DK + c) : make_float4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < VE; ++j) {
            const int e = tid + NT * j, r = e / (CW / V), c = (e % (CW / V)) * V;
            vx[j] = r < len ? *reinterpret_cast<const float4 *>(v + (t0 + r) * A.Hv * DV + c) : make_float4(0, 0, 0, 0);
        }
        if (tid < 32) load_decays<C>(g ? g + t0 * g_tok + h : nullptr, g_stride, len, gx);
    };
    auto decays_of = [&](int64_t i) {  // of the chunk in the registers
        if (tid >= 32 || i >= chunks) return;
        const int b = i & 1;
        chunk_decays<C>(gx, s_hi[b], s_lo[b]);
        __syncwarp();
        const float eh = s_hi[b][C - 1], el = s_lo[b][C - 1];
        for (int r = tid; r < C; r += 32)
            s_f[b][r] = A.scale * (back ? expf(s_hi[b][r]) : expf((eh - s_hi[b][r]) + (el - s_lo[b][r])));
    };
    fetch(0);
    float S[4][TN];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) S[i][j] = A.init ? A.init[at + (int64_t)(r0 + i) * DV + j] : 0.f;
    decays_of(0);
    for (int64_t i = 0; i < chunks; ++i) {
        if (A.each) {
            float *e = A.each + ((slot0 + chunk_of(i)) * H + h) * (int64_t)(DK * DV) + part * CW + c0;
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int j = 0; j < TN; ++j) e[(int64_t)(r0 + a) * DV + j] = S[a][j];
        }
        __syncthreads();  // the chunk's decays are there; the last one's tiles are used
#pragma unroll
        for (int j = 0; j < KE; ++j) {
            const int e = tid + NT * j, r = e / (DK / V), c = (e % (DK / V)) * V;
            const float f = s_f[i & 1][r];
            *reinterpret_cast<float4 *>(&s_k[r][c]) = make_float4(kx[j].x * f, kx[j].y * f, kx[j].z * f, kx[j].w * f);
        }
#pragma unroll
        for (int j = 0; j < VE; ++j) {
            const int e = tid + NT * j;
            *reinterpret_cast<float4 *>(&s_v[e / (CW / V)][(e % (CW / V)) * V]) = vx[j];
        }
        const float all = expf(s_hi[i & 1][C - 1]);
        __syncthreads();
        fetch(i + 1);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            erase(S[a], all);
#pragma unroll
            for (int j = 0; j < TN; ++j) S[a][j] *= all;
        }
#pragma unroll 8
        for (int t = 0; t < C; ++t) {
            const float4 x = *reinterpret_cast<const float4 *>(&s_k[t][r0]);
            const float xs[4] = {x.x, x.y, x.z, x.w};
            float y[TN];
#pragma unroll
            for (int j = 0; j < TN; ++j) y[j] = s_v[t][c0 + j];
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int j = 0; j < TN; ++j) S[a][j] = fmaf(xs[a], y[j], S[a][j]);
        }
        decays_of(i + 1);
    }
    if (A.fin) {
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int j = 0; j < TN; ++j) A.fin[at + (int64_t)(r0 + a) * DV + j] = S[a][j];
    }
}

// ------------------------------------------------------------------------------------------- products
// Results of M x N products lie on 16 x 16 threads: thread (ty, tx) holds rows ty + 16 i and columns tx + 16 j.
// nt: += A[r][k] B[c][k];  nn: += A[r][k] B[k][c];  tn: += A[k][r] B[k][c].
template <int MI, int NJ, int K>
__device__ __forceinline__ void mm_nt(float (&acc)[MI][NJ], const float *A, int pa, const float *B, int pb) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll 2
    for (int k = 0; k < K; k += 4) {
        float4 a[MI];
#pragma unroll
        for (int i = 0; i < MI; ++i) a[i] = *reinterpret_cast<const float4 *>(A + (ty + 16 * i) * pa + k);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const float4 b = *reinterpret_cast<const float4 *>(B + (tx + 16 * j) * pb + k);
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                acc[i][j] = fmaf(a[i].x, b.x, acc[i][j]);
                acc[i][j] = fmaf(a[i].y, b.y, acc[i][j]);
                acc[i][j] = fmaf(a[i].z, b.z, acc[i][j]);
                acc[i][j] = fmaf(a[i].w, b.w, acc[i][j]);
            }
        }
    }
}
template <int MI, int NJ, int K>
__device__ __forceinline__ void mm_nn(float (&acc)[MI][NJ], const float *A, int pa, const float *B, int pb) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll 2
    for (int k = 0; k < K; k += 4) {
        float4 a[MI];
#pragma unroll
        for (int i = 0; i < MI; ++i) a[i] = *reinterpret_cast<const float4 *>(A + (ty + 16 * i) * pa + k);
#pragma unroll
        for (int l = 0; l < 4; ++l) {
            float b[NJ];
#pragma unroll
            for (int j = 0; j < NJ; ++j) b[j] = B[(k + l) * pb + tx + 16 * j];
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const float x = l == 0 ? a[i].x : l == 1 ? a[i].y : l == 2 ? a[i].z : a[i].w;
#pragma unroll
                for (int j = 0; j < NJ; ++j) acc[i][j] = fmaf(x, b[j], acc[i][j]);
            }
        }
    }
}
template <int MI, int NJ, int K>
__device__ __forceinline__ void mm_tn(float (&acc)[MI][NJ], const float *A, int pa, const float *B, int pb) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
        float a[MI], b[NJ];
#pragma unroll
        for (int i = 0; i < MI; ++i) a[i] = A[k * pa + ty + 16 * i];
#pragma unroll
        for (int j = 0; j < NJ; ++j) b[j] = B[k * pb + tx + 16 * j];
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
}
template <int MI, int NJ>
__device__ __forceinline__ void zero(float (&acc)[MI][NJ]) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = 0.f;
}

constexpr int PC = C + 4;  // pitch of C x C matrices

// ------------------------------------------------------------------------------------------- outputs
template <int DK, int DV> constexpr int out_smem_floats() {
    return C * (DK + 4) + C * ((DK > DV ? DK : DV) + 4) + C * (DV + 4) + C * PC + 2 * C;
}

template <int DK, int DV>
__global__ void __launch_bounds__(NT) linear_out_kernel(const float *q, const float *k, const float *v, int Hq, int Hk, int Hv,
                                                        const float *g, int g_stride, int g_tok, const float *states,
                                                        float scale, const int32_t *cu, int64_t tokens, int64_t N,
                                                        int H, float *o) {
    constexpr int PK = DK + 4, PV = DV + 4, PB = (DK > DV ? DK : DV) + 4;
    extern __shared__ __align__(16) float smem[];
    float *s_q = smem, *s_b = s_q + C * PK, *s_v = s_b + C * PB, *s_a = s_v + C * PV, *s_hi = s_a + C * PC,
          *s_lo = s_hi + C;
    const int64_t slot = blockIdx.x / H;
    const int h = (int)(blockIdx.x % H);
    chunk c;
    if (!find_chunk<C>(cu, tokens, N, slot, &c)) return;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    if (tid < 32) {
        float x[C / 32];
        load_decays<C>(g ? g + c.tok0 * g_tok + h : nullptr, g_stride, c.len, x);
        chunk_decays<C>(x, s_hi, s_lo);
    }
    load_tile<DK>(s_q, PK, q + (c.tok0 * Hq + h / (H / Hq)) * DK, (int64_t)Hq * DK, c.len);
    load_tile<DK>(s_b, PK, k + (c.tok0 * Hk + h / (H / Hk)) * DK, (int64_t)Hk * DK, c.len);
    load_tile<DV>(s_v, PV, v + (c.tok0 * Hv + h / (H / Hv)) * DV, (int64_t)Hv * DV, c.len);
    __syncthreads();
    {
        float x[4][4];
        zero(x);
        mm_nt<4, 4, DK>(x, s_q, PK, s_b, PK);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = ty + 16 * i, t = tx + 16 * j;
                s_a[r * PC + t] = t <= r ? x[i][j] * expf((s_hi[r] - s_hi[t]) + (s_lo[r] - s_lo[t])) : 0.f;
            }
    }
    __syncthreads();
    float acc[4][DV / 16];
    zero(acc);
    const float *S = states + (slot * H + h) * (int64_t)(DK * DV);
    for (int p = 0; p < DK; p += C) {  // the state, C rows at a time
        load_tile<DV>(s_b, PV, S + (int64_t)p * DV, DV, C);
        __syncthreads();
        mm_nn<4, DV / 16, C>(acc, s_q + p, PK, s_b, PV);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float e = expf(s_hi[ty + 16 * i]);
        erase(acc[i], e);
#pragma unroll
        for (int j = 0; j < DV / 16; ++j) acc[i][j] *= e;
    }
    mm_nn<4, DV / 16, C>(acc, s_a, PC, s_v, PV);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i;
        if (r < c.len) {
#pragma unroll
            for (int j = 0; j < DV / 16; ++j) st(o + ((c.tok0 + r) * H + h) * DV + tx + 16 * j, scale * acc[i][j]);
        }
    }
}

// ------------------------------------------------------------------------------------------- gradients
struct grads_args {
    const void *q, *k, *v, *go;
    int Hq, Hk, Hv;
    const float *g;
    int g_stride, g_tok;
    const float *states, *adj;           // [slots, H, dk, dv]
    float scale;
    const int32_t *cu;
    int64_t tokens, N;
    int H;
    void *dq, *dk, *dv;                  // with the heads of q, k, v where those are H, else:
    float *pq, *pk, *pv;                 // fp32 [T, H, d], summed over heads afterwards
    float *dg;                           // [T, H], or
    float *dg_slot;                      // [slots, H] sums over a chunk
};

constexpr int PR = 32;  // state rows staged at a time

template <int DK, int DV> constexpr int grads_smem_floats() {
    return 2 * C * (DK + 4) + 2 * C * (DV + 4) + 3 * C * PC + 2 * PR * (DV + 4) + 5 * C + 8;
}

// x (rows r = ty + 16 i of a chunk) to the gradient: rounded to its dtype where its heads are the states', else fp32
template <int D>
__device__ __forceinline__ void put_rows(const float (&x)[4][D / 16], float *out, float *part, int64_t tok0, int len, int H,
                                         int h) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i;
        if (r < len) {
            const int64_t at = ((tok0 + r) * H + h) * D + tx;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                (part ? part : out)[at + 16 * j] = x[i][j];
            }
        }
    }
}

template <int DK, int DV>
__global__ void __launch_bounds__(NT) linear_grads_kernel(grads_args A) {
    constexpr int PK = DK + 4, PV = DV + 4;
    extern __shared__ __align__(16) float smem[];
    float *s_q = smem, *s_k = s_q + C * PK, *s_v = s_k + C * PK, *s_o = s_v + C * PV, *s_a = s_o + C * PV,
          *s_da = s_a + C * PC, *s_w = s_da + C * PC, *s_S = s_w + C * PC, *s_L = s_S + PR * PV, *s_hi = s_L + PR * PV,
          *s_lo = s_hi + C, *s_row = s_lo + C, *s_qdq = s_row + C, *s_kdk = s_qdq + C, *s_dot = s_kdk + C;
    const int H = A.H;
    const int64_t slot = blockIdx.x / H;
    const int h = (int)(blockIdx.x % H);
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    chunk c;
    if (!find_chunk<C>(A.cu, A.tokens, A.N, slot, &c)) {
        if (A.dg_slot && tid == 0) A.dg_slot[slot * H + h] = 0.f;
        return;
    }
    if (tid < 32) {
        float x[C / 32];
        load_decays<C>(A.g ? A.g + c.tok0 * A.g_tok + h : nullptr, A.g_stride, c.len, x);
        chunk_decays<C>(x, s_hi, s_lo);
    }
    load_tile<DK>(s_q, PK, (const float *)A.q + (c.tok0 * A.Hq + h / (H / A.Hq)) * DK, (int64_t)A.Hq * DK, c.len);
    load_tile<DK>(s_k, PK, (const float *)A.k + (c.tok0 * A.Hk + h / (H / A.Hk)) * DK, (int64_t)A.Hk * DK, c.len);
    load_tile<DV>(s_v, PV, (const float *)A.v + (c.tok0 * A.Hv + h / (H / A.Hv)) * DV, (int64_t)A.Hv * DV, c.len);
    load_tile<DV>(s_o, PV, (const float *)A.go + (c.tok0 * H + h) * DV, (int64_t)H * DV, c.len);
    __syncthreads();
    const float scale = A.scale;
    {
        float x[4][4], y[4][4];
        zero(x);
        zero(y);
        mm_nt<4, 4, DK>(x, s_q, PK, s_k, PK);
        mm_nt<4, 4, DV>(y, s_o, PV, s_v, PV);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = ty + 16 * i, t = tx + 16 * j;
                const float d = t <= r ? scale * expf((s_hi[r] - s_hi[t]) + (s_lo[r] - s_lo[t])) : 0.f;
                s_a[r * PC + t] = x[i][j] * d;
                s_da[r * PC + t] = y[i][j] * d;
                // what passes from t to r; t = r adds the same to both of its sums below and is left out of them
                s_w[r * PC + t] = t < r ? x[i][j] * y[i][j] * d : 0.f;
            }
    }
    __syncthreads();
    // dL/dG_r of the chunk's own pairs: what r receives less what it hands on
    if (tid < C) {
        float in = 0.f, out = 0.f;
        for (int t = 0; t < tid; ++t) in += s_w[tid * PC + t];
        for (int r = tid + 1; r < C; ++r) out += s_w[r * PC + tid];
        s_row[tid] = in - out;
    }
    float dq[4][DK / 16], dk[4][DK / 16], dv[4][DV / 16], dot = 0.f;
    zero(dq);
    zero(dk);
    zero(dv);
    const float *S = A.states + (slot * H + h) * (int64_t)(DK * DV), *L = A.adj + (slot * H + h) * (int64_t)(DK * DV);
#pragma unroll
    for (int p = 0; p < DK / PR; ++p) {
        for (int e = tid; e < PR * DV / 4; e += NT) {
            const int r = e / (DV / 4), cc = (e % (DV / 4)) * 4;
            const float4 x = *reinterpret_cast<const float4 *>(S + (p * PR + r) * DV + cc);
            const float4 y = *reinterpret_cast<const float4 *>(L + (p * PR + r) * DV + cc);
            *reinterpret_cast<float4 *>(s_S + r * PV + cc) = x;
            *reinterpret_cast<float4 *>(s_L + r * PV + cc) = y;
            dot += x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
        }
        __syncthreads();
        float t[4][PR / 16];
        zero(t);
        mm_nt<4, PR / 16, DV>(t, s_o, PV, s_S, PV);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < PR / 16; ++j) dq[i][p * (PR / 16) + j] = t[i][j];
        zero(t);
        mm_nt<4, PR / 16, DV>(t, s_v, PV, s_L, PV);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < PR / 16; ++j) dk[i][p * (PR / 16) + j] = t[i][j];
        mm_nn<4, DV / 16, PR>(dv, s_k + p * PR, PK, s_L, PV);
        __syncthreads();
    }
    const float Gh = s_hi[C - 1], Gl = s_lo[C - 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i;
        const float w = expf(s_hi[r]), e = scale * w, f = expf((Gh - s_hi[r]) + (Gl - s_lo[r]));
        float a = 0.f, b = 0.f;
        erase(dq[i], w);
        erase(dk[i], f);
        erase(dv[i], f);
#pragma unroll
        for (int j = 0; j < DK / 16; ++j) {
            dq[i][j] *= e;
            dk[i][j] *= f;
            a = fmaf(s_q[r * PK + tx + 16 * j], dq[i][j], a);
            b = fmaf(s_k[r * PK + tx + 16 * j], dk[i][j], b);
        }
#pragma unroll
        for (int j = 0; j < DV / 16; ++j) dv[i][j] *= f;
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, off);
            b += __shfl_xor_sync(0xffffffffu, b, off);
        }
        if (tx == 0) {
            s_qdq[r] = a;
            s_kdk[r] = b;
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    if ((tid & 31) == 0) s_dot[tid >> 5] = dot;
    mm_nn<4, DK / 16, C>(dq, s_da, PC, s_k, PK);
    mm_tn<4, DK / 16, C>(dk, s_da, PC, s_q, PK);
    mm_tn<4, DV / 16, C>(dv, s_a, PC, s_o, PV);
    put_rows<DK>(dq, (float *)A.dq, A.pq, c.tok0, c.len, H, h);
    put_rows<DK>(dk, (float *)A.dk, A.pk, c.tok0, c.len, H, h);
    put_rows<DV>(dv, (float *)A.dv, A.pv, c.tok0, c.len, H, h);
    if (!A.dg && !A.dg_slot) return;
    __syncthreads();
    // dg_t = sum_{r >= t} (own pairs + outputs of the entering state) + sum_{j < t} keys into the leaving state
    //        + e^{G_C} <S, Lambda>
    if (tid < 32) {
        ff whole{0.f, 0.f};
        for (int w = 0; w < NT / 32; ++w) whole = ff_add(whole, {s_dot[w], 0.f});
        const float left = expf(Gh), all = left == 0.f ? 0.f : (whole.h + whole.l) * left;
        const ff x0 = ff_add({s_row[2 * tid], 0.f}, {s_qdq[2 * tid], 0.f});
        const ff own = ff_add(x0, ff_add({s_row[2 * tid + 1], 0.f}, {s_qdq[2 * tid + 1], 0.f}));
        const float k0 = s_kdk[2 * tid];
        const ff keys = ff_add({k0, 0.f}, {s_kdk[2 * tid + 1], 0.f});
        ff after = own, before = keys;
        for (int off = 1; off < 32; off <<= 1) {
            const ff a = ff_shfl(after, (tid + off) & 31), b = ff_shfl(before, (tid - off) & 31);
            if (tid + off < 32) after = ff_add(after, a);
            if (tid >= off) before = ff_add(b, before);
        }
        before = ff_add(before, {-keys.h, -keys.l});
        const ff base = ff_add(before, {all, 0.f});
        const ff g0 = ff_add(after, base), g1 = ff_add(ff_add(after, {-x0.h, -x0.l}), ff_add(base, {k0, 0.f}));
        if (A.dg) {
            if (2 * tid < c.len) A.dg[(c.tok0 + 2 * tid) * H + h] = g0.h + g0.l;
            if (2 * tid + 1 < c.len) A.dg[(c.tok0 + 2 * tid + 1) * H + h] = g1.h + g1.l;
        } else {
            ff sum{0.f, 0.f};
            if (2 * tid < c.len) sum = g0;
            if (2 * tid + 1 < c.len) sum = ff_add(sum, g1);
            for (int off = 16; off > 0; off >>= 1) sum = ff_add(sum, ff_shfl(sum, (tid + off) & 31));
            if (tid == 0) A.dg_slot[slot * H + h] = sum.h + sum.l;
        }
    }
}

// out[t][x][c] = sum of part[t][x * R + i][c] over i, in order; rows behind the last sequence stay as they were
template <typename T>
__global__ void __launch_bounds__(NT) linear_sum_heads_kernel(const float *part, T *out, int64_t tokens, int64_t N,
                                                              const int32_t *cu, int Hx, int R, int D) {
    const int64_t last = seq_start(cu, tokens, N, N), rows = (last < tokens ? last : tokens) * Hx;
    for (int64_t e = (int64_t)blockIdx.x * NT + threadIdx.x; e < rows * D; e += (int64_t)gridDim.x * NT) {
        const int64_t row = e / D;
        const float *p = part + row * R * D + (e - row * D);
        float s = 0.f;
        for (int i = 0; i < R; ++i) s += p[(int64_t)i * D];
        st(out + e, s);
    }
}

__global__ void __launch_bounds__(NT) linear_sum_decay_kernel(const float *part, float *out, int64_t slots, int H) {
    __shared__ double s[NT];
    const int h = blockIdx.x;
    double x = 0.0;
    for (int64_t i = threadIdx.x; i < slots; i += NT) x += (double)part[i * H + h];
    s[threadIdx.x] = x;
    __syncthreads();
    for (int n = NT / 2; n > 0; n >>= 1) {
        if (threadIdx.x < n) s[threadIdx.x] += s[threadIdx.x + n];
        __syncthreads();
    }
    if (threadIdx.x == 0) out[h] = (float)s[0];
}

// ------------------------------------------------------------------------------------------- launches
static size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

template <int DK, int DV>
static cudaError_t fwd(const kda_linear_args *a, char *ws, cudaStream_t stream, int *err) {
    float *states = (float *)ws;
    const int64_t slots = chunk_slots(a->T, a->N, C);
    const int gs = a->g_per_token ? a->H : 0, gt = a->g_per_token ? a->H : 0;
    const states_args f{a->k, a->v, a->Hk, a->Hv, a->initial_state, a->final_state, a->T ? states : nullptr, 1.f};
    linear_states_kernel<DK, DV><<<dim3((unsigned)(a->N * a->H * (DV / 32)), 1), NT, 0, stream>>>(
        f, f, a->g, gs, gt, a->cu_seqlens, a->T, a->N, a->H, err);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a->T == 0) return e;
    constexpr int smem = out_smem_floats<DK, DV>() * 4;
    static std::atomic<uint64_t> allowed{0};
    e = allow_smem(linear_out_kernel<DK, DV>, smem, allowed);
    if (e != cudaSuccess) return e;
    linear_out_kernel<DK, DV><<<(unsigned)(slots * a->H), NT, smem, stream>>>(
        (const float *)a->q, (const float *)a->k, (const float *)a->v, a->Hq, a->Hk, a->Hv, a->g, gs, gt, states, a->scale,
        a->cu_seqlens, a->T, a->N, a->H, (float *)a->o);
    return cudaGetLastError();
}

struct bwd_layout {
    size_t states, adj, pq, pk, pv, dg, total;
    bwd_layout(int64_t T, int64_t N, int H, int Hq, int Hk, int Hv, int dk, int dv) {
        const size_t each = up256((size_t)chunk_slots(T, N, C) * H * dk * dv * 4);
        const size_t rk = up256((size_t)T * H * dk * 4), rv = up256((size_t)T * H * dv * 4);
        size_t at = 0;
        states = at, at += each;
        adj = at, at += each;
        pq = at, at += Hq != H ? rk : 0;
        pk = at, at += Hk != H ? rk : 0;
        pv = at, at += Hv != H ? rv : 0;
        dg = at, at += up256((size_t)chunk_slots(T, N, C) * H * 4);
        total = at;
    }
};

template <typename T>
static cudaError_t sum_heads(const kda_row_parts &p, void *out, const kda_linear_bwd_args *a, int Hx, int D, cudaStream_t stream) {
    if (!p.part) return cudaSuccess;
    const int64_t want = (a->T * Hx * D + NT - 1) / NT;
    linear_sum_heads_kernel<T><<<(unsigned)(want < 4096 ? want : 4096), NT, 0, stream>>>(
        p.part, (T *)out, a->T, a->N, a->cu_seqlens, Hx, p.parts / Hx, D);
    return cudaGetLastError();
}
template <typename T>
static cudaError_t sum_parts(const kda_linear_bwd_args *a, const kda_row_parts &pq, const kda_row_parts &pk, const kda_row_parts &pv,
                             const float *dg_slot, int64_t slots, cudaStream_t stream) {
    cudaError_t e = sum_heads<T>(pq, a->grad_q, a, a->Hq, a->dk, stream);
    if (e == cudaSuccess) e = sum_heads<T>(pk, a->grad_k, a, a->Hk, a->dk, stream);
    if (e == cudaSuccess) e = sum_heads<T>(pv, a->grad_v, a, a->Hv, a->dv, stream);
    if (e == cudaSuccess && dg_slot) {
        linear_sum_decay_kernel<<<(unsigned)a->H, NT, 0, stream>>>(dg_slot, a->grad_g, slots, a->H);
        e = cudaGetLastError();
    }
    return e;
}

template <int DK, int DV>
static cudaError_t bwd(const kda_linear_bwd_args *a, char *ws, cudaStream_t stream, int *err) {
    const bwd_layout L(a->T, a->N, a->H, a->Hq, a->Hk, a->Hv, DK, DV);
    const int64_t slots = chunk_slots(a->T, a->N, C);
    const int gs = a->g_per_token ? a->H : 0;
    float *states = a->T ? (float *)(ws + L.states) : nullptr, *adj = a->T ? (float *)(ws + L.adj) : nullptr;
    const states_args f{a->k, a->v, a->Hk, a->Hv, a->initial_state, nullptr, states, 1.f};
    const states_args b{a->q, a->grad_o, a->Hq, a->H, a->grad_final_state, a->grad_initial_state, adj, a->scale};
    linear_states_kernel<DK, DV><<<dim3((unsigned)(a->N * a->H * (DV / 32)), 2), NT, 0, stream>>>(
        f, b, a->g, gs, gs, a->cu_seqlens, a->T, a->N, a->H, err);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (a->T == 0) {
        if (a->grad_g && !a->g_per_token) return cudaMemsetAsync(a->grad_g, 0, (size_t)a->H * 4, stream);
        return cudaSuccess;
    }
    grads_args G{};
    G.q = a->q, G.k = a->k, G.v = a->v, G.go = a->grad_o;
    G.Hq = a->Hq, G.Hk = a->Hk, G.Hv = a->Hv, G.H = a->H;
    G.g = a->g, G.g_stride = gs, G.g_tok = gs;
    G.states = states, G.adj = adj, G.scale = a->scale;
    G.cu = a->cu_seqlens, G.tokens = a->T, G.N = a->N;
    G.dq = a->grad_q, G.dk = a->grad_k, G.dv = a->grad_v;
    G.pq = a->Hq != a->H ? (float *)(ws + L.pq) : nullptr;
    G.pk = a->Hk != a->H ? (float *)(ws + L.pk) : nullptr;
    G.pv = a->Hv != a->H ? (float *)(ws + L.pv) : nullptr;
    if (a->grad_g) {
        if (a->g_per_token) G.dg = a->grad_g;
        else G.dg_slot = (float *)(ws + L.dg);
    }
    constexpr int smem = grads_smem_floats<DK, DV>() * 4;
    static_assert(smem <= 227 * 1024, "shared memory");
    static std::atomic<uint64_t> allowed{0};
    e = allow_smem(linear_grads_kernel<DK, DV>, smem, allowed);
    if (e != cudaSuccess) return e;
    linear_grads_kernel<DK, DV><<<(unsigned)(slots * a->H), NT, smem, stream>>>(G);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return sum_parts<float>(a, {G.pq, a->H}, {G.pk, a->H}, {G.pv, a->H}, G.dg_slot, slots, stream);
}

static cudaError_t fwd_d(const kda_linear_args *a, char *ws, cudaStream_t s, int *err) {
    if (a->dk == 128) return a->dv == 128 ? fwd<128, 128>(a, ws, s, err) : fwd<128, 64>(a, ws, s, err);
    return a->dv == 128 ? fwd<64, 128>(a, ws, s, err) : fwd<64, 64>(a, ws, s, err);
}
static cudaError_t bwd_d(const kda_linear_bwd_args *a, char *ws, cudaStream_t s, int *err) {
    if (a->dk == 128) return a->dv == 128 ? bwd<128, 128>(a, ws, s, err) : bwd<128, 64>(a, ws, s, err);
    return a->dv == 128 ? bwd<64, 128>(a, ws, s, err) : bwd<64, 64>(a, ws, s, err);
}

}  // namespace lin
}  // namespace kda

size_t kda_linear_fwd_layout_bytes(int64_t T, int64_t N, int H, int dk, int dv, kda_dtype_t dtype) {
    if (dtype == KDA_BF16) return kda_linear_fwd_tc_bytes(T, N, H, dk, dv);
    return kda::lin::up256((size_t)kda::lin::chunk_slots(T, N, kda::lin::C) * H * dk * dv * 4);
}

size_t kda_linear_bwd_layout_bytes(int64_t T, int64_t N, int H, int Hq, int Hk, int Hv, int dk, int dv,
                                   kda_dtype_t dtype) {
    if (dtype == KDA_BF16) return kda_linear_bwd_tc_bytes(T, N, H, Hq, Hk, Hv, dk, dv);
    return kda::lin::bwd_layout(T, N, H, Hq, Hk, Hv, dk, dv).total;
}

kda_status_t kda_launch_linear_fwd(const kda_linear_args *a, void *ws, cudaStream_t stream) {
    int *err = kda_device_error_ptr();
    if (!err) return KDA_ERR_CUDA;
    if (a->dtype == KDA_BF16 && a->T > 0) return kda_launch_linear_fwd_tc(a, ws, stream, err);
    return kda_cuda_status(kda::lin::fwd_d(a, (char *)ws, stream, err));  // (no tokens: no elements of their type)
}

kda_status_t kda_launch_linear_bwd(const kda_linear_bwd_args *a, void *ws, cudaStream_t stream) {
    int *err = kda_device_error_ptr();
    if (!err) return KDA_ERR_CUDA;
    if (a->dtype == KDA_BF16 && a->T > 0) return kda_launch_linear_bwd_tc(a, ws, stream, err);
    return kda_cuda_status(kda::lin::bwd_d(a, (char *)ws, stream, err));
}

kda_status_t kda_linear_sum_parts(const kda_linear_bwd_args *a, const kda_row_parts &pq, const kda_row_parts &pk,
                                  const kda_row_parts &pv, const float *dg_slot, int64_t slots, cudaStream_t stream) {
    return kda_cuda_status(a->dtype == KDA_BF16 ? kda::lin::sum_parts<kda::bf16>(a, pq, pk, pv, dg_slot, slots, stream)
                                                : kda::lin::sum_parts<float>(a, pq, pk, pv, dg_slot, slots, stream));
}
