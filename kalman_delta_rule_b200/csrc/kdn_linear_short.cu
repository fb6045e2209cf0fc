// Backward of linear attention with a decay for each head for sequences of at most 32 tokens, fp32 arithmetic on CUDA
// cores.  Such a sequence is one chunk, so the state at its start and the gradient at its end are the caller's own S0 and
// dS_T, nothing has to be walked, and one launch does: a CTA per (sequence, head), with the formulas of the chunk
// (kdn_linear_grad_tc.cu) over the tokens that there are,
//     dQ = dA K + a (dO S0^T),   dK = dA^T Q + w (V dS_T^T),   dV = P^T dO + w (K dS_T),
//     dS0 = e^{G_T} dS_T + (a Q)^T dO,
//     dg_t = sum_{i >= t, j < t} Z_ij + sum_{s >= t} q_s.(a dO S0^T)_s + sum_{s < t} k_s.(w V dS_T^T)_s + e^{G_T} <S0, dS_T>.
// Only the outputs are rounded to the type.  Room for CS = 16 tokens (two CTAs of 256 threads per SM, one loads its two
// states while the other multiplies) or 32 (one CTA of 512).  Bound by the latency of loading two states and by shared
// memory's reads: one head of 128 x 128 takes 14 us with a token, 24 with 16, 39 with 32; 2048 heads 154, 271 and 584, of
// which HBM's share for the three states is 62.
#include "kdn_common.cuh"
#include "kdn_launch.h"
#include "kdn_linear.cuh"

namespace kdn {

namespace {

constexpr int PAD = 4;

template <int CS, int DK, int DVT>
struct Tiles {
    float q[CS][DK + PAD], k[CS][DK + PAD], v[CS][DVT + PAD], o[CS][DVT + PAD];
    float s[DK][DVT + PAD], r[DK][DVT + PAD];
};

// rows [0, len) of W columns from a token tensor, zeros behind them
template <int CS, int W, typename Tin>
__device__ __forceinline__ void load_rows(float (&dst)[CS][W + PAD], const void *src, int t0, int len, int H, int h, int d, int col) {
    const Tin *p = static_cast<const Tin *>(src) + ((size_t)t0 * H + h) * d + col;
    for (int e = threadIdx.x; e < CS * (W / 4); e += 16 * CS) {
        const int t = e / (W / 4), c = (e % (W / 4)) * 4;
        *reinterpret_cast<float4 *>(&dst[t][c]) = t < len ? ldf4(p + (size_t)t * H * d + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}
__device__ __forceinline__ float dot4(float4 x, float4 y, float s) {
    return fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s))));
}

// N neighbours of a row in shared memory, as few loads as their alignment allows
template <int N>
struct Row {
    float x[N];
    __device__ __forceinline__ explicit Row(const float *p) {
        if constexpr (N % 4 == 0) {
#pragma unroll
            for (int j = 0; j < N; j += 4) *reinterpret_cast<float4 *>(x + j) = *reinterpret_cast<const float4 *>(p + j);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = p[j];
        }
    }
};

}  // namespace

template <int CS, int DK, int DVT, typename Tin>
__global__ void __launch_bounds__(16 * CS, 32 / CS) linear_short_backward_kernel(LinBwdArgs b, float *share)
{
    constexpr int NT = 16 * CS, NP = CS / 16;   // threads; pairs of tokens per thread
    constexpr int TG = CS * DK / NT;       // tokens of a thread's channel in dQ, dK
    constexpr int SG = CS * DVT / NT;      // tokens of a thread's column in dV
    constexpr int C4 = DVT / 4, RP = NT / C4;   // threads per row of a state, rows per pass
    constexpr int NR = DK > RP ? DK / RP : 1;
    extern __shared__ __align__(16) uint8_t raw[];
    Tiles<CS, DK, DVT> &m = *reinterpret_cast<Tiles<CS, DK, DVT> *>(raw);
    __shared__ __align__(16) float P[CS][CS + 4], dA[CS][CS + 4], dAt[CS][CS + 4];   // (dAt: keys by queries)
    __shared__ float Z[CS][CS + 1];
    __shared__ float since[CS], until[CS], xs[NT / 32][TG], ys[NT / 32][TG], srs[NT / 32];
    __shared__ Log2 G[CS];
    __shared__ float one_s;
    const LinArgs &a = b.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int s = blockIdx.x / a.H, h = blockIdx.x % a.H;
    int t0, len;
    lin_seq(a, s, t0, len);
    const size_t state = (size_t)blockIdx.x * DK * a.dv;
    const bool has_s = a.S0 != nullptr, has_r = b.dS_T != nullptr;

    load_rows<CS, DK, Tin>(m.q, a.q, t0, len, a.H, h, DK, 0);
    load_rows<CS, DK, Tin>(m.k, a.k, t0, len, a.H, h, DK, 0);
    if (warp == 0) {                       // log2 decays since the start; 1 behind the end; a NaN meets every factor
        const float g = lane < len ? lin_load_decay(a, t0 + lane, h) : 0.f;
        const unsigned nan = __ballot_sync(0xffffffffu, isnan(g));
        Log2 x = lin_log2(g);
#pragma unroll
        for (int off = 1; off < CS; off <<= 1) {
            const Log2 y = {__shfl_up_sync(0xffffffffu, x.hi, off), __shfl_up_sync(0xffffffffu, x.lo, off)};
            if (lane >= off) x = x + y;
        }
        if (lane < CS) G[lane] = x;
        if (lane == 0) one_s = nan ? __int_as_float(0x7fc00000) : 1.f;
    }
    __syncthreads();
    const float one = one_s, whole = one * lin_exp2(G[CS - 1]);
    if (tid < CS) {
        since[tid] = a.scale * one * lin_exp2(G[tid]);
        until[tid] = one * lin_exp2_between(G[CS - 1], G[tid]);
    }
    const int pt = tid / 16;                                      // this thread's pairs: a query, NP keys
    float D[NP], dp[NP] = {}, p[NP] = {}, sr = 0.f;
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        const int ps = tid % 16 + 16 * n;
        D[n] = ps <= pt ? a.scale * one * lin_exp2_between(G[pt], G[ps]) : 0.f;
        if (ps <= pt && pt < len) {
#pragma unroll 8
            for (int c = 0; c < DK; c += 4) p[n] = dot4(*reinterpret_cast<float4 *>(&m.q[pt][c]), *reinterpret_cast<float4 *>(&m.k[ps][c]), p[n]);
            p[n] *= D[n];
        }
        P[pt][ps] = p[n];
    }
    const int ch = tid % DK, ct = (tid / DK) * TG;                // this thread's channel and first token
    float X[TG] = {}, Y[TG] = {};
    for (int col = 0; col < a.dv; col += DVT) {
        __syncthreads();
        load_rows<CS, DVT, Tin>(m.v, a.v, t0, len, a.H, h, a.dv, col);
        load_rows<CS, DVT, Tin>(m.o, b.d_o, t0, len, a.H, h, a.dv, col);
        const int c4 = (tid % C4) * 4;
#pragma unroll 4
        for (int i = tid / C4; i < DK; i += RP) {
            const size_t at = state + (size_t)i * a.dv + col + c4;
            const float4 x = has_s ? ldf4(a.S0 + at) : make_float4(0.f, 0.f, 0.f, 0.f);
            const float4 y = has_r ? ldf4(b.dS_T + at) : make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4 *>(&m.s[i][c4]) = x;
            *reinterpret_cast<float4 *>(&m.r[i][c4]) = y;
            sr = dot4(x, y, sr);
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            const int ps = tid % 16 + 16 * n;
            if (ps > pt || pt >= len) continue;
#pragma unroll 8
            for (int c = 0; c < DVT; c += 4) dp[n] = dot4(*reinterpret_cast<float4 *>(&m.o[pt][c]), *reinterpret_cast<float4 *>(&m.v[ps][c]), dp[n]);
        }
        if (ct < len) {
#pragma unroll 2
            for (int c = 0; c < DVT; c += 4) {
                if (has_s) {
                    const float4 x = *reinterpret_cast<float4 *>(&m.s[ch][c]);
#pragma unroll
                    for (int j = 0; j < TG; ++j) X[j] = dot4(x, *reinterpret_cast<float4 *>(&m.o[ct + j][c]), X[j]);
                }
                if (has_r) {
                    const float4 x = *reinterpret_cast<float4 *>(&m.r[ch][c]);
#pragma unroll
                    for (int j = 0; j < TG; ++j) Y[j] = dot4(x, *reinterpret_cast<float4 *>(&m.v[ct + j][c]), Y[j]);
                }
            }
        }
        const int vc = tid % DVT, vt = (tid / DVT) * SG;          // this thread's column of dV and first token
        if (vt < len) {
            float x[SG] = {}, y[SG] = {};
            for (int t = vt; t < len; ++t) {
                const float o = m.o[t][vc];
                const Row<SG> w(&P[t][vt]);
#pragma unroll
                for (int j = 0; j < SG; ++j) x[j] = fmaf(w.x[j], o, x[j]);
            }
            if (has_r) {
#pragma unroll 4
                for (int i = 0; i < DK; i += 4) {
                    const float r0 = m.r[i][vc], r1 = m.r[i + 1][vc], r2 = m.r[i + 2][vc], r3 = m.r[i + 3][vc];
#pragma unroll
                    for (int j = 0; j < SG; ++j) y[j] = dot4(*reinterpret_cast<float4 *>(&m.k[vt + j][i]), make_float4(r0, r1, r2, r3), y[j]);
                }
            }
            Tin *dst = static_cast<Tin *>(b.dv) + ((size_t)t0 * a.H + h) * a.dv + col + vc;
#pragma unroll
            for (int j = 0; j < SG; ++j)
                if (vt + j < len) stf(dst + (size_t)(vt + j) * a.H * a.dv, fmaf(until[vt + j], y[j], x[j]));
        }
        if (b.dS0 && tid / C4 < DK) {
            float4 acc[NR];
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                const float4 r = *reinterpret_cast<float4 *>(&m.r[tid / C4 + j * RP][c4]);
                acc[j] = make_float4(whole * r.x, whole * r.y, whole * r.z, whole * r.w);
            }
            for (int t = 0; t < len; ++t) {
                const float4 o = *reinterpret_cast<float4 *>(&m.o[t][c4]);
                const float f = since[t];
                const float4 fo = make_float4(f * o.x, f * o.y, f * o.z, f * o.w);
#pragma unroll
                for (int j = 0; j < NR; ++j) {
                    const float q = m.q[t][tid / C4 + j * RP];
                    acc[j] = make_float4(fmaf(q, fo.x, acc[j].x), fmaf(q, fo.y, acc[j].y), fmaf(q, fo.z, acc[j].z), fmaf(q, fo.w, acc[j].w));
                }
            }
#pragma unroll
            for (int j = 0; j < NR; ++j) stf4(b.dS0 + state + (size_t)(tid / C4 + j * RP) * a.dv + col + c4, acc[j]);
        }
    }
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        dA[pt][tid % 16 + 16 * n] = dAt[tid % 16 + 16 * n][pt] = D[n] * dp[n];
        Z[pt][tid % 16 + 16 * n] = p[n] * dp[n];
    }
    sr = warp_sum(sr);
    if (lane == 0) srs[warp] = sr;
    __syncthreads();
    // dQ, dK: a channel of TG tokens per thread
    Tin *dq = static_cast<Tin *>(b.dq) + ((size_t)t0 * a.H + h) * DK + ch, *dk = static_cast<Tin *>(b.dk) + ((size_t)t0 * a.H + h) * DK + ch;
    float x[TG], y[TG];
#pragma unroll
    for (int j = 0; j < TG; ++j) {
        x[j] = X[j] * since[ct + j];
        y[j] = Y[j] * until[ct + j];
        const float xq = warp_sum(x[j] * m.q[ct + j][ch]), yk = warp_sum(y[j] * m.k[ct + j][ch]);
        if (lane == 0) {
            xs[warp][j] = xq;
            ys[warp][j] = yk;
        }
    }
    for (int t = 0; t < len; ++t) {
        const float q = m.q[t][ch], k = m.k[t][ch];
        const Row<TG> wq(&dAt[t][ct]), wk(&dA[t][ct]);
#pragma unroll
        for (int j = 0; j < TG; ++j) {
            x[j] = fmaf(wq.x[j], k, x[j]);
            y[j] = fmaf(wk.x[j], q, y[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < TG; ++j) {
        if (ct + j >= len) continue;
        stf(dq + (size_t)(ct + j) * a.H * DK, x[j]);
        stf(dk + (size_t)(ct + j) * a.H * DK, y[j]);
    }
    if (!b.dg) return;
    __syncthreads();
    if (warp > 0) return;
    // the decay's gradient, a token per lane: every sum over its own terms.  Z's rows become their prefix sums
    constexpr int WG = DK / 32;            // warps that share a group of TG tokens
    float g = 0.f, later = 0.f, before = 0.f, s0 = 0.f;
    if (lane < len) {
        float row = 0.f;
        for (int j = 0; j <= lane; ++j) {
            const float z = Z[lane][j];
            Z[lane][j] = row;
            row += z;
        }
#pragma unroll
        for (int w = 0; w < WG; ++w) {
            later += xs[lane / TG * WG + w][lane % TG];
            before += ys[lane / TG * WG + w][lane % TG];
        }
    }
#pragma unroll
    for (int off = 1; off < CS; off <<= 1) {
        const float x = __shfl_down_sync(0xffffffffu, later, off), y = __shfl_up_sync(0xffffffffu, before, off);
        if (lane + off < 32) later += x;
        if (lane >= off) before += y;
    }
    before = __shfl_up_sync(0xffffffffu, before, 1);     // of the tokens before
    if (lane == 0) before = 0.f;
    __syncwarp();
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) s0 += srs[w];
    if (lane < len) {
        for (int i = lane; i < len; ++i) g += Z[i][lane];
        g = fmaf(whole, s0, (g + later) + before);
        if (a.decay == KDN_DECAY_TOKEN) b.dg[(size_t)(t0 + lane) * a.H + h] = g;
    }
    if (a.decay == KDN_DECAY_HEAD) {
        g = warp_sum(g);
        if (lane == 0) share[(size_t)lin_first_slot(a, s, t0, kLinearShort) * a.H + h] = g;
    }
}

namespace {

template <int CS, int DK, int DVT, typename Tin>
cudaError_t run(const LinBwdArgs &b, float *share, cudaStream_t st) {
    constexpr size_t smem = sizeof(Tiles<CS, DK, DVT>);
    KernelSetup ks;
    auto kern = linear_short_backward_kernel<CS, DK, DVT, Tin>;
    const cudaError_t e = kernel_setup(reinterpret_cast<const void *>(kern), smem, 16 * CS, false, &ks);
    if (e != cudaSuccess) return e;
    return launch(kern, dim3((unsigned)((long long)b.a.nseq * b.a.H)), 16 * CS, smem, st, b, share);
}
template <int DK, int DVT, typename Tin>
cudaError_t by_length(const LinBwdArgs &b, float *share, cudaStream_t st) {
    return (b.a.cu ? b.a.ntok : b.a.T) <= 16 ? run<16, DK, DVT, Tin>(b, share, st) : run<kLinearShort, DK, DVT, Tin>(b, share, st);
}
template <int DK, typename Tin>
cudaError_t by_tile(const LinBwdArgs &b, float *share, cudaStream_t st) {
    return b.a.dv == 32 ? by_length<DK, 32, Tin>(b, share, st) : by_length<DK, 64, Tin>(b, share, st);
}
template <typename Tin>
cudaError_t by_size(const LinBwdArgs &b, float *share, cudaStream_t st) {
    return b.a.dk == 32 ? by_tile<32, Tin>(b, share, st) : b.a.dk == 64 ? by_tile<64, Tin>(b, share, st) : by_tile<128, Tin>(b, share, st);
}

}  // namespace

size_t linear_short_backward_workspace_bytes(const LinArgs &a) {     // the heads' shares of a per-head decay's gradient
    return ((size_t)lin_slots(a.cu != nullptr, a.T, a.ntok, a.nseq, kLinearShort) * a.H * 4 + 255) / 256 * 256;
}
cudaError_t launch_linear_short_backward(const LinBwdArgs &b, bool bf16_in, void *workspace, cudaStream_t st) {
    float *share = static_cast<float *>(workspace);
    const cudaError_t e = bf16_in ? by_size<bf16>(b, share, st) : by_size<float>(b, share, st);
    if (e != cudaSuccess || !b.dg || b.a.decay != KDN_DECAY_HEAD) return e;
    return launch_linear_head_decay(b.a, share, b.dg, kLinearShort, st);
}

}  // namespace kdn
