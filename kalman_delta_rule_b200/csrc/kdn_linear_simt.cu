// Linear attention with a decay for each head for fp32 inputs: CUDA cores, in chunks of 64 tokens
// (the recurrence unrolled as in kdn_linear.cuh).  Every step is parallel over chunks but one:
//   delta  per (chunk, head, d_v tile): the chunk's own contribution U = K^T diag(w) V (w = decay to
//          the chunk's end) or, for the gradient, E = scale Q^T diag(e^G) dO, and the chunk's decay
//   scan   per state element: the contributions become the states at the chunks' starts
//          (S <- decay S + U, forwards), or the state gradients at the chunks' ends (backwards);
//          left out for sequences of a few chunks, whose CTAs add up what they need themselves
//   out    per (chunk, head, d_v tile): o
//   grad   per (chunk, head): dq, dk, dv and the decay's gradient
// The scan reads and writes each chunk's state once, which costs about the token tensors' own
// traffic at d = 128, and in exchange no step but its multiply-add chain is serial: a problem of
// few, long sequences fills the GPU as well as one of many short ones.  The backward's two
// directions share the first two launches; a launch starts while the one before runs out, with the
// caller's rows read before its results are waited for.  256 tokens of 2 heads of 32: 10.4 us, two
// launches' latency.  Gradient of 24 ragged sequences, 5003 tokens of 4 heads of 64: 95-97 us, bound by
// the fp32 products of `grad` (1.4 waves of its 408 CTAs, two per SM by shared memory; 54% issue activity).  At size the products
// are bound by their reads of shared memory (a 4 x 4 tile per thread, single elements of B): 256 tokens of 1024 heads of 128
// 1650 us, their gradient 2530, against some 350 for the multiply-adds of the forward.
#include "kdn_common.cuh"
#include "kdn_launch.h"

namespace kdn {

namespace {

constexpr int C = 64;          // tokens of a chunk
constexpr int NT = 256;
constexpr int PAD = 4;         // floats behind each shared-memory row: 16 rows' float4 reads hit 16 banks groups

__device__ __forceinline__ float4 scale4(float4 x, float f) { return make_float4(x.x * f, x.y * f, x.z * f, x.w * f); }

// acc[i][j] += sum_k A(m_i, k) B(k, n_j) for m_i = 4 ty + i, n_j = tx + 16 j (16 x 16 threads).
// TA: A is stored [k][m]; TB: B is stored [n][k].  Row strides lda, ldb; K a multiple of 4.
template <int NJ, bool TA, bool TB>
__device__ __forceinline__ void mm(float (&acc)[4][NJ], const float *A, int lda, const float *B, int ldb, int K, int ty,
                                   int tx) {
#pragma unroll 2
    for (int k = 0; k < K; k += 4) {
        float av[4][4];        // [i][k]
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 x = TA ? *reinterpret_cast<const float4 *>(A + (k + i) * lda + ty * 4)
                                : *reinterpret_cast<const float4 *>(A + (ty * 4 + i) * lda + k);
            const float e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                if (TA) av[m][i] = e[m]; else av[i][m] = e[m];
            }
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            float bv[4];
            if (TB) {
                const float4 x = *reinterpret_cast<const float4 *>(B + (tx + 16 * j) * ldb + k);
                bv[0] = x.x; bv[1] = x.y; bv[2] = x.z; bv[3] = x.w;
            } else {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) bv[kk] = B[(k + kk) * ldb + tx + 16 * j];
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i][j] = fmaf(av[i][kk], bv[kk], acc[i][j]);
        }
    }
}

// rows [0, L) of W columns from a token tensor ([ntok, H, d], column col) to shared memory [C][W + PAD];
// rows behind the piece's end are zero, whatever the next sequence's rows hold
template <int W>
__device__ __forceinline__ void load_rows(float *dst, const void *src, int tok, int L, int H, int h, int d, int col) {
    const float *p = static_cast<const float *>(src) + ((size_t)tok * H + h) * d + col;
    const size_t rs = (size_t)H * d;
    for (int i = threadIdx.x; i < C * (W / 4); i += NT) {
        const int r = i / (W / 4), c = (i % (W / 4)) * 4;
        *reinterpret_cast<float4 *>(dst + r * (W + PAD) + c) = r < L ? ldf4(p + r * rs + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}
// a [DK][W] block of a state (row stride dv) to shared memory [DK][W + PAD]
template <int DK, int W>
__device__ __forceinline__ void load_state(float *dst, const float *src, int dv) {
    for (int i = threadIdx.x; i < DK * (W / 4); i += NT) {
        const int r = i / (W / 4), c = (i % (W / 4)) * 4;
        *reinterpret_cast<float4 *>(dst + r * (W + PAD) + c) = *reinterpret_cast<const float4 *>(src + (size_t)r * dv + c);
    }
}

// G (log2, inclusive) of the chunk's C tokens to shared memory by warp 0; decay 1 behind the end.  A NaN
// among the log decays is put where every factor of the chunk meets it.
struct ChunkDecay {
    Log2 G[C];
    float one;                 // 1, or NaN
};
__device__ __forceinline__ void chunk_log_decay(const LinArgs &a, int tok, int L, int h, ChunkDecay *d) {
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        float g[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) g[i] = 2 * lane + i < L ? lin_load_decay(a, tok + 2 * lane + i, h) : 0.f;
        const bool bad = __any_sync(0xffffffffu, g[0] != g[0] || g[1] != g[1]);
        const Log2 x0 = lin_log2(g[0]), x1 = x0 + lin_log2(g[1]);
        Log2 s = x1;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const Log2 y = {__shfl_up_sync(0xffffffffu, s.hi, off), __shfl_up_sync(0xffffffffu, s.lo, off)};
            if (lane >= off) s = y + s;
        }
        Log2 before = {__shfl_up_sync(0xffffffffu, s.hi, 1), __shfl_up_sync(0xffffffffu, s.lo, 1)};
        if (lane == 0) before = {0.f, 0.f};
        d->G[2 * lane] = before + x0;
        d->G[2 * lane + 1] = s;
        if (lane == 0) d->one = bad ? __int_as_float(0x7fc00000) : 1.f;
    }
    __syncthreads();
}
// sum over the 16 threads of a row (lanes tx = 0..15)
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// A [DK][DVT] tile of a state (row stride dv) in the registers of a CTA, to which chunks' contributions are added.
template <int DK, int DVT>
struct Fold {
    static constexpr int N = DK * DVT / 4 / NT;
    float4 x[N];
    static __device__ __forceinline__ size_t at(int e, int dv) {
        const int i = threadIdx.x + e * NT;
        return (size_t)(i / (DVT / 4)) * dv + (i % (DVT / 4)) * 4;
    }
    static __device__ __forceinline__ float4 *in(float *tile, int e) {        // its place in shared memory
        const int i = threadIdx.x + e * NT;
        return reinterpret_cast<float4 *>(tile + (i / (DVT / 4)) * (DVT + PAD) + (i % (DVT / 4)) * 4);
    }
    __device__ __forceinline__ void start(const float *p, size_t off, int dv) {
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = p ? ldf4(p + off + at(e, dv)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ void add(float2 f, const float *U, int dv) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float4 y = *reinterpret_cast<const float4 *>(U + at(e, dv));
            x[e] = make_float4(lin_carry(f, x[e].x, y.x), lin_carry(f, x[e].y, y.y), lin_carry(f, x[e].z, y.z), lin_carry(f, x[e].w, y.w));
        }
    }
    __device__ __forceinline__ void store(float *p, int dv) const {
#pragma unroll
        for (int e = 0; e < N; ++e) stf4(p + at(e, dv), x[e]);
    }
};

struct Ws {
    float *U, *E;              // [slots, H, dk, dv]: states at the chunks' starts; state gradients at their ends
    float2 *dec;               // [slots, H] decay of the whole chunk
    float *dgc;                // [slots, H] the chunk's share of a per-head decay's gradient
};

}  // namespace

// ------------------------------------------------------------------ delta
// What a launch of the first two steps works on; the backward's two directions are independent and share launches
// (blockIdx.z): 0 forwards, 1 backwards.
struct Walk {
    const void *X, *Y;         // K, V;  Q, dO
    float *U;                  // contributions, then states
    const float *first;        // state before the first chunk;  gradient of the last state
    float *last;               // state behind the last chunk;  gradient of the first state
};
struct Walks {
    Walk w[2];
};

template <int DK, int DVT>
__global__ void __launch_bounds__(NT) linear_delta_kernel(LinArgs a, Walks ws, float2 *dec)
{
    let_next_launch();
    extern __shared__ __align__(16) float sm[];
    float *Xs = sm, *Ys = sm + C * (DK + PAD);
    __shared__ ChunkDecay dec_s;
    const Log2 *G = dec_s.G;
    const bool rev = blockIdx.z != 0;
    const Walk &wk = ws.w[blockIdx.z];
    const int u = blockIdx.x / a.H, h = blockIdx.x % a.H, col = blockIdx.y * DVT;
    LinPiece p;
    if (!lin_piece(a, u, C, p) || p.len == 0) return;
    const int tok = p.t0 + p.j * C, L = min(C, p.len - p.j * C);
    load_rows<DK>(Xs, wk.X, tok, L, a.H, h, DK, 0);
    load_rows<DVT>(Ys, wk.Y, tok, L, a.H, h, a.dv, col);
    chunk_log_decay(a, tok, L, h, &dec_s);
    for (int i = threadIdx.x; i < L * (DVT / 4); i += NT) {
        const int r = i / (DVT / 4);
        float4 *y = reinterpret_cast<float4 *>(Ys + r * (DVT + PAD) + (i % (DVT / 4)) * 4);
        *y = scale4(*y, dec_s.one * (rev ? a.scale * lin_exp2(G[r]) : lin_exp2_between(G[C - 1], G[r])));
    }
    if (!rev && blockIdx.y == 0 && threadIdx.x == 0) {
        const float2 f = lin_chunk_decay(G[C - 1]);
        dec[(size_t)u * a.H + h] = make_float2(f.x * dec_s.one, f.y);
    }
    __syncthreads();
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    float *dst = wk.U + ((size_t)u * a.H + h) * DK * a.dv + col;
#pragma unroll
    for (int m0 = 0; m0 < DK; m0 += 64) {
        if (ty * 4 >= DK) break;
        float acc[4][DVT / 16] = {};
        mm<DVT / 16, true, false>(acc, Xs + m0, DK + PAD, Ys, DVT + PAD, C, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < DVT / 16; ++j) dst[(size_t)(m0 + ty * 4 + i) * a.dv + tx + 16 * j] = acc[i][j];
    }
}

// ------------------------------------------------------------------ scan
// thread = four elements of one (sequence, head)'s state; the chunks' contributions are fetched
// eight at a time, so that the loads of a group overlap and only its multiply-adds are serial
__global__ void __launch_bounds__(256) linear_scan_kernel(LinArgs a, Walks ws, const float2 *dec)
{
    let_next_launch();
    wait_for_launch();
    const bool rev = blockIdx.z != 0;
    const Walk &wk = ws.w[blockIdx.z];
    const int per = a.dk * a.dv / 4;
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    const int sh = (int)(id / per), e = (int)(id % per) * 4;
    if (sh >= a.nseq * a.H) return;
    const int s = sh / a.H, h = sh % a.H;
    int t0, len;
    lin_seq(a, s, t0, len);
    const int n = (len + C - 1) / C;
    const size_t st = (size_t)a.H * a.dk * a.dv;
    float *p = wk.U + ((size_t)lin_first_slot(a, s, t0, C) * a.H + h) * a.dk * a.dv + e;
    const float2 *d = dec + (size_t)lin_first_slot(a, s, t0, C) * a.H + h;
    const size_t se = (size_t)sh * a.dk * a.dv + e;
    float4 x = wk.first ? *reinterpret_cast<const float4 *>(wk.first + se) : make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int B = 8;
    for (int c0 = 0; c0 < n; c0 += B) {
        float4 y[B];
        float2 f[B];
#pragma unroll
        for (int i = 0; i < B; ++i) {
            if (c0 + i < n) {
                const int c = rev ? n - 1 - c0 - i : c0 + i;
                y[i] = *reinterpret_cast<const float4 *>(p + c * st);
                f[i] = d[(size_t)c * a.H];
            }
        }
#pragma unroll
        for (int i = 0; i < B; ++i) {
            if (c0 + i < n) {
                const int c = rev ? n - 1 - c0 - i : c0 + i;
                *reinterpret_cast<float4 *>(p + c * st) = x;
                x = make_float4(lin_carry(f[i], x.x, y[i].x), lin_carry(f[i], x.y, y[i].y), lin_carry(f[i], x.z, y[i].z),
                                lin_carry(f[i], x.w, y[i].w));
            }
        }
    }
    if (wk.last) *reinterpret_cast<float4 *>(wk.last + se) = x;
}

// ------------------------------------------------------------------ out
// FOLD: of the chunks' own contributions each CTA forms its state itself, and a sequence's last one S_out: no scan.
template <int DK, int DVT, bool FOLD>
__global__ void __launch_bounds__(NT) linear_out_kernel(LinArgs a, const float *S, const float2 *dec)
{
    extern __shared__ __align__(16) float sm[];
    float *Qs = sm, *Ks = Qs + C * (DK + PAD), *Vs = Ks + C * (DK + PAD), *Ss = Vs + C * (DVT + PAD),
          *Ps = Ss + DK * (DVT + PAD);
    __shared__ ChunkDecay dec_s;
    const Log2 *G = dec_s.G;
    const int u = blockIdx.x / a.H, h = blockIdx.x % a.H, col = blockIdx.y * DVT;
    LinPiece p;
    if (!lin_piece(a, u, C, p) || (p.len == 0 && !FOLD)) return wait_for_launch();
    const int tok = p.t0 + p.j * C, L = min(C, p.len - p.j * C);
    load_rows<DK>(Qs, a.q, tok, L, a.H, h, DK, 0);
    load_rows<DK>(Ks, a.k, tok, L, a.H, h, DK, 0);
    load_rows<DVT>(Vs, a.v, tok, L, a.H, h, a.dv, col);
    chunk_log_decay(a, tok, L, h, &dec_s);
    const float scale = a.scale * dec_s.one;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    {
        float acc[4][4] = {};
        mm<4, false, true>(acc, Qs, DK + PAD, Ks, DK + PAD, DK, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = ty * 4 + i, s = tx + 16 * j;
                Ps[t * (C + PAD) + s] = s <= t ? scale * acc[i][j] * lin_exp2_between(G[t], G[s]) : 0.f;
            }
    }
    wait_for_launch();                     // the states, or the contributions, are complete
    const size_t slot = (size_t)u * a.H + h, per = (size_t)DK * a.dv;
    if constexpr (FOLD) {
        const size_t seq = ((size_t)p.s * a.H + h) * per + col;
        Fold<DK, DVT> x;
        x.start(a.S0, seq, a.dv);
        auto add = [&](int c) {            // chunk c's contribution
            const size_t from = slot - (size_t)(p.j - c) * a.H;
            x.add(dec[from], S + from * per + col, a.dv);
        };
#pragma unroll 2
        for (int c = 0; c < p.j; ++c) add(c);
#pragma unroll
        for (int e = 0; e < x.N; ++e) *x.in(Ss, e) = x.x[e];
        if (a.S_out && p.j * C + C >= p.len) {
            if (L > 0) add(p.j);
            x.store(a.S_out + seq, a.dv);
        }
    } else {
        load_state<DK, DVT>(Ss, S + slot * per + col, a.dv);
    }
    __syncthreads();
    float acc[4][DVT / 16] = {};
    mm<DVT / 16, false, false>(acc, Qs, DK + PAD, Ss, DVT + PAD, DK, ty, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float f = scale * lin_exp2(G[ty * 4 + i]);
#pragma unroll
        for (int j = 0; j < DVT / 16; ++j) acc[i][j] *= f;
    }
    mm<DVT / 16, false, false>(acc, Ps, C + PAD, Vs, DVT + PAD, C, ty, tx);
    float *o = static_cast<float *>(a.o) + ((size_t)tok * a.H + h) * a.dv + col;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = ty * 4 + i;
        if (t >= L) continue;
#pragma unroll
        for (int j = 0; j < DVT / 16; ++j) stf(o + (size_t)t * a.H * a.dv + tx + 16 * j, acc[i][j]);
    }
}

// ------------------------------------------------------------------ grad
// With P = scale QK^T o D, dP = dO V^T, dA = scale dP o D, Z = P o dP, S the state at the chunk's start,
// R the gradient of the state at its end, a_t = scale e^{G_t}, w_t = e^{G_C - G_t}:
//   dQ = dA K + a (dO S^T),  dK = dA^T Q + w (V R^T),  dV = P^T dO + w (K R)
//   dg_t = sum over pairs (query i >= t, key j < t), in the chunk, before and behind it:
//        sum_{i >= t, j < t} Z_ij + sum_{s >= t} q_s.(a dO S^T)_s + sum_{s < t} k_s.(w V R^T)_s + e^{G_C} <S, R>
// No term is divided by a decay, and every sum is formed from its own terms (a difference of larger ones would leave their
// roundings where a reset's gradient is zero).
template <int DK, int DVT, bool FOLD>
__global__ void __launch_bounds__(NT, DK <= 64 ? 2 : 1) linear_grad_kernel(LinBwdArgs b, Ws ws)
{
    const LinArgs &a = b.a;
    constexpr int NK = DK / 16, NV = DVT / 16;
    extern __shared__ __align__(16) float sm[];
    float *Qs = sm, *Ks = Qs + C * (DK + PAD), *Vs = Ks + C * (DK + PAD), *Os = Vs + C * (DVT + PAD),
          *Ss = Os + C * (DVT + PAD), *Ps = Ss + DK * (DVT + PAD);
    float *const Rs = Ss, *const As = Ps, *const Zs = Vs;   // each takes the other's place once that has been read
    constexpr int ZR = C + 1;              // Z's row stride
    static_assert(C * ZR <= 2 * C * (DVT + PAD) + DK * (DVT + PAD), "Z takes the place of V, dO and the states");
    __shared__ ChunkDecay dec_s;
    const Log2 *G = dec_s.G;
    __shared__ float zc[4][C], xi[C], yi[C], wsum[8];
    const int u = blockIdx.x / a.H, h = blockIdx.x % a.H;
    LinPiece p;
    if (!lin_piece(a, u, C, p)) return wait_for_launch();
    const size_t seq = ((size_t)p.s * a.H + h) * DK * a.dv;
    if (p.len == 0) {
        if (FOLD && b.dS0)
            for (int e = threadIdx.x * 4; e < DK * a.dv; e += NT * 4)
                stf4(b.dS0 + seq + e, b.dS_T ? ldf4(b.dS_T + seq + e) : make_float4(0.f, 0.f, 0.f, 0.f));
        return wait_for_launch();
    }
    const int tok = p.t0 + p.j * C, L = min(C, p.len - p.j * C);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const size_t sbase = ((size_t)u * a.H + h) * DK * a.dv;
    load_rows<DK>(Qs, a.q, tok, L, a.H, h, DK, 0);
    load_rows<DK>(Ks, a.k, tok, L, a.H, h, DK, 0);
    chunk_log_decay(a, tok, L, h, &dec_s);

    const float scale = a.scale * dec_s.one;
    float pv[4][4] = {};
    mm<4, false, true>(pv, Qs, DK + PAD, Ks, DK + PAD, DK, ty, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = ty * 4 + i, s = tx + 16 * j;
            pv[i][j] = s <= t ? scale * pv[i][j] * lin_exp2_between(G[t], G[s]) : 0.f;
            Ps[t * (C + PAD) + s] = pv[i][j];
        }

    float dp[4][4] = {}, dqi[4][NK] = {}, dki[4][NK] = {};
    float sr = 0.f;
    wait_for_launch();                     // the states and their gradients are complete
    for (int col = 0; col < a.dv; col += DVT) {
        __syncthreads();       // the previous tile is read; Ps is written
        load_rows<DVT>(Vs, a.v, tok, L, a.H, h, a.dv, col);
        load_rows<DVT>(Os, b.d_o, tok, L, a.H, h, a.dv, col);
        // chunk c's slot is slot + (c - j) H
        const size_t slot = (size_t)u * a.H + h, per = (size_t)DK * a.dv;
        if constexpr (FOLD) {
            Fold<DK, DVT> x;
            x.start(a.S0, seq + col, a.dv);
#pragma unroll 2
            for (int c = p.j; c > 0; --c) x.add(ws.dec[slot - (size_t)c * a.H], ws.U + (slot - (size_t)c * a.H) * per + col, a.dv);
#pragma unroll
            for (int e = 0; e < x.N; ++e) *x.in(Ss, e) = x.x[e];
        } else {
            load_state<DK, DVT>(Ss, ws.U + sbase + col, a.dv);
        }
        __syncthreads();
        mm<4, false, true>(dp, Os, DVT + PAD, Vs, DVT + PAD, DVT, ty, tx);
        mm<NK, false, true>(dqi, Os, DVT + PAD, Ss, DVT + PAD, DVT, ty, tx);
        __syncthreads();
        if constexpr (FOLD) {                                      // R over S, and their inner product
            Fold<DK, DVT> y;
            y.start(b.dS_T, seq + col, a.dv);
#pragma unroll 2
            for (int c = (p.len - 1) / C - p.j; c > 0; --c) y.add(ws.dec[slot + (size_t)c * a.H], ws.E + (slot + (size_t)c * a.H) * per + col, a.dv);
#pragma unroll
            for (int e = 0; e < y.N; ++e) {
                float4 *at = y.in(Ss, e);
                sr = fmaf(at->x, y.x[e].x, fmaf(at->y, y.x[e].y, fmaf(at->z, y.x[e].z, fmaf(at->w, y.x[e].w, sr))));
                *at = y.x[e];
            }
            if (b.dS0 && p.j == 0) {
                y.add(ws.dec[slot], ws.E + slot * per + col, a.dv);
                y.store(b.dS0 + seq + col, a.dv);
            }
        } else {
            for (int i = threadIdx.x; i < DK * (DVT / 4); i += NT) {
                const int r = i / (DVT / 4), c = (i % (DVT / 4)) * 4;
                float4 *at = reinterpret_cast<float4 *>(Ss + r * (DVT + PAD) + c);
                const float4 x = *at, y = *reinterpret_cast<const float4 *>(ws.E + sbase + col + (size_t)r * a.dv + c);
                sr = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, sr))));
                *at = y;
            }
        }
        __syncthreads();
        mm<NK, false, true>(dki, Vs, DVT + PAD, Rs, DVT + PAD, DVT, ty, tx);
        float acc[4][NV] = {};
        mm<NV, false, false>(acc, Ks, DK + PAD, Rs, DVT + PAD, DK, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float w = lin_exp2_between(G[C - 1], G[ty * 4 + i]);
#pragma unroll
            for (int j = 0; j < NV; ++j) acc[i][j] *= w;
        }
        mm<NV, true, false>(acc, Ps, C + PAD, Os, DVT + PAD, C, ty, tx);
        float *dv = static_cast<float *>(b.dv) + ((size_t)tok * a.H + h) * a.dv + col;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = ty * 4 + i;
            if (t >= L) continue;
#pragma unroll
            for (int j = 0; j < NV; ++j) stf(dv + (size_t)t * a.H * a.dv + tx + 16 * j, acc[i][j]);
        }
    }

    // ---- dA and Z to shared memory; the boundary terms of the decay's gradient
    __syncthreads();           // P and the last tile have been read
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = ty * 4 + i;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int s = tx + 16 * j;
            As[t * (C + PAD) + s] = s <= t ? scale * dp[i][j] * lin_exp2_between(G[t], G[s]) : 0.f;
            Zs[t * ZR + s] = s <= t ? pv[i][j] * dp[i][j] : 0.f;
        }
        const float fa = scale * lin_exp2(G[t]), fw = lin_exp2_between(G[C - 1], G[t]);
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            dqi[i][j] *= fa;
            dki[i][j] *= fw;
            x = fmaf(dqi[i][j], Qs[t * (DK + PAD) + tx + 16 * j], x);
            y = fmaf(dki[i][j], Ks[t * (DK + PAD) + tx + 16 * j], y);
        }
        x = row_sum(x);
        y = row_sum(y);
        if (tx == 0) { xi[t] = x; yi[t] = y; }
    }
    sr = warp_sum(sr);
    if (lane == 0) wsum[warp] = sr;
    __syncthreads();
    if (b.dg) {                // sum_{i >= t, j < t} Z_ij: Z's rows become the sums of the columns before, then columns from the diagonal down
        float *z = Zs + (threadIdx.x >> 2) * ZR + (threadIdx.x & 3) * 16, run = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) run += z[j];
        const float a1 = __shfl_up_sync(0xffffffffu, run, 1, 4), a2 = __shfl_up_sync(0xffffffffu, run, 2, 4), a3 = __shfl_up_sync(0xffffffffu, run, 3, 4);
        const int part = threadIdx.x & 3;
        run = part == 0 ? 0.f : part == 1 ? a1 : part == 2 ? a2 + a1 : (a3 + a2) + a1;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float own = z[j];
            z[j] = run;
            run += own;
        }
        __syncthreads();
        const int t = threadIdx.x % C, i0 = (threadIdx.x / C) * 16;
        run = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) run += i0 + i >= t ? Zs[(i0 + i) * ZR + t] : 0.f;
        zc[threadIdx.x / C][t] = run;
        __syncthreads();
    }

    mm<NK, false, false>(dqi, As, C + PAD, Ks, DK + PAD, C, ty, tx);
    mm<NK, true, false>(dki, As, C + PAD, Qs, DK + PAD, C, ty, tx);
    float *dq = static_cast<float *>(b.dq) + ((size_t)tok * a.H + h) * DK, *dk = static_cast<float *>(b.dk) + ((size_t)tok * a.H + h) * DK;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = ty * 4 + i;
        if (t >= L) continue;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            stf(dq + (size_t)t * a.H * DK + tx + 16 * j, dqi[i][j]);
            stf(dk + (size_t)t * a.H * DK + tx + 16 * j, dki[i][j]);
        }
    }
    if (b.dg && warp == 0) {   // two tokens per lane, sums over the tokens from t on and before t in fp64
        float s0 = 0.f;
        for (int w = 0; w < 8; ++w) s0 += wsum[w];
        const double whole = (double)lin_exp2(G[C - 1]) * s0;
        double pairs[2], later[2], earlier[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            pairs[e] = (zc[0][t] + zc[1][t]) + (zc[2][t] + zc[3][t]);
            later[e] = xi[t];
            earlier[e] = yi[t];
        }
        double fl = later[0] + later[1], fe = earlier[0] + earlier[1];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const double yl = __shfl_down_sync(0xffffffffu, fl, off), ye = __shfl_up_sync(0xffffffffu, fe, off);
            if (lane + off < 32) fl += yl;
            if (lane >= off) fe += ye;
        }
        fl = __shfl_down_sync(0xffffffffu, fl, 1);   // tokens of the lanes above
        fe = __shfl_up_sync(0xffffffffu, fe, 1);     // tokens of the lanes below
        if (lane == 31) fl = 0.0;
        if (lane == 0) fe = 0.0;
        const double d1 = whole + pairs[1] + fl + later[1] + fe + earlier[0], d0 = whole + pairs[0] + fl + later[1] + later[0] + fe;
        if (a.decay == KDN_DECAY_TOKEN) {
            if (2 * lane < L) b.dg[(size_t)(tok + 2 * lane) * a.H + h] = (float)d0;
            if (2 * lane + 1 < L) b.dg[(size_t)(tok + 2 * lane + 1) * a.H + h] = (float)d1;
        } else {
            double d = (2 * lane < L ? d0 : 0.0) + (2 * lane + 1 < L ? d1 : 0.0);
            for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
            if (lane == 0) ws.dgc[(size_t)u * a.H + h] = (float)d;
        }
    }
}

// dg[h] of a per-head decay: the chunks' shares in a fixed order
__global__ void __launch_bounds__(256) linear_head_decay_kernel(LinArgs a, const float *dgc, float *dg, int slots, int tokens)
{
    __shared__ double part[256];
    const int h = blockIdx.x;
    double s = 0.0;
    for (int u = threadIdx.x; u < slots; u += 256) {
        LinPiece p;
        if (lin_piece(a, u, tokens, p) && p.len > 0) s += dgc[(size_t)u * a.H + h];
    }
    part[threadIdx.x] = s;
    __syncthreads();
    for (int off = 128; off > 0; off >>= 1) {
        if ((int)threadIdx.x < off) part[threadIdx.x] += part[threadIdx.x + off];
        __syncthreads();
    }
    if (threadIdx.x == 0) dg[h] = (float)part[0];
}

// ------------------------------------------------------------------ host side
cudaError_t launch_linear_head_decay(const LinArgs &a, const float *share, float *dg, int tokens, cudaStream_t st) {
    return launch(linear_head_decay_kernel, dim3((unsigned)a.H), 256, 0, st, a, share, dg, (int)lin_slots(a.cu != nullptr, a.T, a.ntok, a.nseq, tokens), tokens);
}

namespace {

size_t round256(size_t x) { return (x + 255) / 256 * 256; }
long long slots_of(const LinArgs &a) { return lin_slots(a.cu != nullptr, a.T, a.ntok, a.nseq, C); }
size_t state_bytes(const LinArgs &a) { return round256((size_t)slots_of(a) * a.H * a.dk * a.dv * 4); }
size_t head_bytes(const LinArgs &a) { return round256((size_t)slots_of(a) * a.H * 8); }

// the first two steps for one direction or both
template <int DK, int DVT>
cudaError_t deltas(const LinArgs &a, const Walks &ws, int walks, float2 *dec, cudaStream_t st) {
    constexpr size_t smem = sizeof(float) * C * (DK + DVT + 2 * PAD);
    KernelSetup ks;
    auto kern = linear_delta_kernel<DK, DVT>;
    const cudaError_t e = kernel_setup(reinterpret_cast<const void *>(kern), smem, NT, false, &ks);
    if (e != cudaSuccess) return e;
    return launch(kern, dim3((unsigned)(slots_of(a) * a.H), a.dv / DVT, walks), NT, smem, st, a, ws, dec);
}
cudaError_t scans(const LinArgs &a, const Walks &ws, int walks, const float2 *dec, cudaStream_t st) {
    const long long threads = (long long)a.nseq * a.H * (a.dk * a.dv / 4);
    return launch_next(linear_scan_kernel, dim3((unsigned)((threads + 255) / 256), 1, walks), 256, 0, st, a, ws, dec);
}

// Sequences of a few chunks go without the scan: its launch costs more than reading their contributions again does (256
// tokens of 2 heads of 32: 14.4 -> 10.4 us; 512 of 1024 heads of 128, where most is read again: 4032 -> 3592; the gradient
// of 5003 tokens in 24 sequences, H4 d64: 96 -> 86).  Packed lengths are known on the device only: a few chunks on
// average, and so little to read that one sequence of nearly all tokens, whose chunk j reads j contributions again, still costs
// no more than about a quarter (4990 tokens beside 11 single ones, H4 d64: 61 -> 64 us, gradient 105 -> 132).  Both bounds are on
// that sequence: what its last CTA reads in turn (past 1.5 MB: 4080 tokens of one head of 128 x 256, 8 MB: 67 -> 120 us) and what
// all of them read (past 256 MB: 8170 tokens of 16 heads of 128 x 256, 17 GB: 2.3 -> 4.3 ms, gradient 2.9 -> 6.7).
bool folded(const LinArgs &a) {
    constexpr int FEW = 8 * C;
    if (!a.cu) return a.T <= FEW;
    if (a.ntok <= FEW) return true;
    if (a.ntok > 16 * FEW || a.ntok / FEW >= a.nseq) return false;
    const long long chunks = a.ntok / C, one = chunks * a.dk * a.dv * 4;
    return one <= 3ll << 19 && one * chunks / 2 * a.H <= 256ll << 20;
}

template <int DK, int DVT, bool FOLD>
cudaError_t outputs(const LinArgs &a, const float *U, const float2 *dec, cudaStream_t st) {
    constexpr size_t smem = sizeof(float) * (C * (2 * DK + DVT + C + 4 * PAD) + DK * (DVT + PAD));
    KernelSetup ks;
    auto kern = linear_out_kernel<DK, DVT, FOLD>;
    const cudaError_t e = kernel_setup(reinterpret_cast<const void *>(kern), smem, NT, false, &ks);
    if (e != cudaSuccess) return e;
    return launch_next(kern, dim3((unsigned)(slots_of(a) * a.H), a.dv / DVT), NT, smem, st, a, U, dec);
}

template <int DK, int DVT>
cudaError_t forward(const LinArgs &a, uint8_t *ws, cudaStream_t st) {
    float *U = reinterpret_cast<float *>(ws);
    float2 *dec = reinterpret_cast<float2 *>(ws + state_bytes(a));
    const Walks wk{{{a.k, a.v, U, a.S0, a.S_out}, {}}};
    cudaError_t e = deltas<DK, DVT>(a, wk, 1, dec, st);
    if (e != cudaSuccess) return e;
    if (folded(a)) return outputs<DK, DVT, true>(a, U, dec, st);
    e = scans(a, wk, 1, dec, st);
    return e != cudaSuccess ? e : outputs<DK, DVT, false>(a, U, dec, st);
}

template <int DK, int DVT>
cudaError_t backward(const LinBwdArgs &b, uint8_t *wsp, cudaStream_t st) {
    const LinArgs &a = b.a;
    Ws ws;
    ws.U = reinterpret_cast<float *>(wsp);
    ws.E = reinterpret_cast<float *>(wsp + state_bytes(a));
    ws.dec = reinterpret_cast<float2 *>(wsp + 2 * state_bytes(a));
    ws.dgc = reinterpret_cast<float *>(wsp + 2 * state_bytes(a) + head_bytes(a));
    const Walks wk{{{a.k, a.v, ws.U, a.S0, nullptr}, {a.q, b.d_o, ws.E, b.dS_T, b.dS0}}};
    cudaError_t e = deltas<DK, DVT>(a, wk, 2, ws.dec, st);
    const bool fold = folded(a);
    if (e == cudaSuccess && !fold) e = scans(a, wk, 2, ws.dec, st);
    if (e != cudaSuccess) return e;
    constexpr size_t smem = sizeof(float) * (C * (2 * DK + 2 * DVT + C + 5 * PAD) + DK * (DVT + PAD));
    KernelSetup ks;
    auto kern = fold ? linear_grad_kernel<DK, DVT, true> : linear_grad_kernel<DK, DVT, false>;
    e = kernel_setup(reinterpret_cast<const void *>(kern), smem, NT, false, &ks);
    if (e != cudaSuccess) return e;
    e = launch_next(kern, dim3((unsigned)(slots_of(a) * a.H)), NT, smem, st, b, ws);
    if (e != cudaSuccess || !b.dg || a.decay != KDN_DECAY_HEAD) return e;
    return launch_linear_head_decay(a, ws.dgc, b.dg, C, st);
}

#define KDN_LINEAR_SIZES(FN, ARG)                                          \
    if (a.dv == 32) {                                                      \
        if (a.dk == 32) return FN<32, 32>(ARG, w, st);                     \
        return a.dk == 64 ? FN<64, 32>(ARG, w, st) : FN<128, 32>(ARG, w, st); \
    }                                                                      \
    if (a.dk == 32) return FN<32, 64>(ARG, w, st);                         \
    return a.dk == 64 ? FN<64, 64>(ARG, w, st) : FN<128, 64>(ARG, w, st);

}  // namespace

size_t linear_simt_workspace_bytes(const LinArgs &a) { return state_bytes(a) + head_bytes(a); }
size_t linear_simt_backward_workspace_bytes(const LinArgs &a) { return 2 * state_bytes(a) + 2 * head_bytes(a); }

cudaError_t launch_linear_simt(const LinArgs &a, void *workspace, cudaStream_t st) {
    uint8_t *w = static_cast<uint8_t *>(workspace);
    KDN_LINEAR_SIZES(forward, a)
}
cudaError_t launch_linear_simt_backward(const LinBwdArgs &b, void *workspace, cudaStream_t st) {
    const LinArgs &a = b.a;
    uint8_t *w = static_cast<uint8_t *>(workspace);
    KDN_LINEAR_SIZES(backward, b)
}

}  // namespace kdn
