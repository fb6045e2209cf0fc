// Linear attention with a decay for each head, recurrent form: the tokens of each sequence applied in order to a state
// that is read once and written back once (in place, for single tokens).  Per token
//     S <- e^g S + k v^T,   o = scale S^T q.
// A CTA owns a d_v tile of one (sequence, head); its part of S stays in registers as float4 rows between the tokens.
// Columns of S never meet, so the tile width is free: the widest one that still gives every SM two CTAs (few sequences:
// narrow tiles, more CTAs, shorter loads per CTA; many: whole rows, so that q, k and the sums over rows are shared by all
// columns).  All arithmetic is fp32, two elements per instruction; only o is rounded to the type.
//
// One token: bound by the state's read and write (131 KB per head at d = 128, against 1 KB of token data): 256 sequences
// of 32 heads take 164 us, 6.6 TB/s; 4 sequences of 16 heads 2.8 us, the latency of its chain of loads and sums.  (Tiles of
// 64 columns at 256 sequences: 188 us; three CTAs per SM, which costs the registers spills: 169.)  Several tokens are taken
// GT at a time, so that the two barriers and the sums over the warps' rows are shared by the group, with the next
// group's rows on their way: 0.20 us a token for a single head, 0.5 when taken one by one; 256 sequences of 32 heads take
// 169 us for 2 tokens, 194 for 4 and 249 for 8 (the state and the tokens once: 167, 170 and 175), from 4 on the tokens' own time.
#include "kdn_common.cuh"
#include "kdn_launch.h"

namespace kdn {

namespace {
constexpr int NT = 256;
}

template <int DK, int DVT, int GT, typename Tin>
__global__ void __launch_bounds__(NT, GT == 1 ? 1 : 2) linear_recurrent_kernel(LinArgs a)
{
    constexpr int TPR = DVT / 4;           // threads per row of S
    constexpr int RPP = NT / TPR;          // rows per pass
    constexpr int NP = DK / RPP;
    static_assert(DK % RPP == 0, "row passes");
    constexpr int NW = NT / 32;
    constexpr int NQ = (GT * DK + NT - 1) / NT, NV = (GT * DVT + NT - 1) / NT;   // elements of a group's q (k), v per thread
    const int tiles = a.dv / DVT;
    const int sh = blockIdx.x / tiles, col = (blockIdx.x % tiles) * DVT;
    const int s = sh / a.H, h = sh % a.H;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c4 = (tid % TPR) * 4, rs = tid / TPR;
    __shared__ __align__(16) float2 qk[GT][DK];
    __shared__ __align__(16) float vs[GT][DVT], red[GT][NW][DVT];
    __shared__ float fs[GT];
    int t0, len;
    lin_seq(a, s, t0, len);

    const size_t base = (size_t)sh * DK * a.dv + col + c4;
    float4 S[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int row = p * RPP + rs;
        S[p] = a.S0 ? __ldcs(reinterpret_cast<const float4 *>(a.S0 + base + (size_t)row * a.dv)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // the next group of tokens, on its way while this one is at work (behind the end: whatever was there before)
    float q1[NQ] = {}, k1[NQ] = {}, v1[NV] = {}, g1 = 0.f;
    auto fetch = [&](int i0) {
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const int e = j * NT + tid, i = i0 + e / DK;
            if (e < GT * DK && i < len) {
                const size_t at = ((size_t)(t0 + i) * a.H + h) * DK + e % DK;
                q1[j] = ldf(static_cast<const Tin *>(a.q) + at);
                k1[j] = ldf(static_cast<const Tin *>(a.k) + at);
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = j * NT + tid, i = i0 + e / DVT;
            if (e < GT * DVT && i < len) v1[j] = ldf(static_cast<const Tin *>(a.v) + ((size_t)(t0 + i) * a.H + h) * a.dv + col + e % DVT);
        }
        if (tid < GT && i0 + tid < len) g1 = lin_load_decay(a, t0 + i0 + tid, h);
    };
    fetch(0);
    for (int i0 = 0; i0 < len; i0 += GT) {
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const int e = j * NT + tid;
            if (e < GT * DK) qk[e / DK][e % DK] = make_float2(q1[j], k1[j]);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = j * NT + tid;
            if (e < GT * DVT) vs[e / DVT][e % DVT] = v1[j];
        }
        if (tid < GT) fs[tid] = expf(g1);
        fetch(i0 + GT);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < GT; ++j) {
            if (i0 + j >= len) break;
            const float4 v = *reinterpret_cast<const float4 *>(&vs[j][c4]);
            const float f = fs[j];
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            if constexpr (GT == 1) {       // HBM's time, not arithmetic's: one element at a time takes fewer registers
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    const float2 c = qk[j][p * RPP + rs];
                    float4 &x = S[p];
                    x = make_float4(fmaf(c.y, v.x, f * x.x), fmaf(c.y, v.y, f * x.y), fmaf(c.y, v.z, f * x.z), fmaf(c.y, v.w, f * x.w));
                    o = make_float4(fmaf(c.x, x.x, o.x), fmaf(c.x, x.y, o.y), fmaf(c.x, x.z, o.z), fmaf(c.x, x.w, o.w));
                }
            } else {
                const f32x2 f2 = pk2(f, f), v01 = pk2(v.x, v.y), v23 = pk2(v.z, v.w);
                f32x2 o01 = 0, o23 = 0;
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    const float2 c = qk[j][p * RPP + rs];
                    const f32x2 q2 = pk2(c.x, c.x), k2 = pk2(c.y, c.y);
                    const f32x2 x01 = fma2(k2, v01, mul2(f2, pk2(S[p].x, S[p].y))), x23 = fma2(k2, v23, mul2(f2, pk2(S[p].z, S[p].w)));
                    o01 = fma2(q2, x01, o01);
                    o23 = fma2(q2, x23, o23);
                    S[p] = make_float4(x2(x01), y2(x01), x2(x23), y2(x23));
                }
                o = make_float4(x2(o01), y2(o01), x2(o23), y2(o23));
            }
#pragma unroll
            for (int off = TPR; off < 32; off <<= 1) {    // rows of the same warp
                o.x += __shfl_xor_sync(0xffffffffu, o.x, off);
                o.y += __shfl_xor_sync(0xffffffffu, o.y, off);
                o.z += __shfl_xor_sync(0xffffffffu, o.z, off);
                o.w += __shfl_xor_sync(0xffffffffu, o.w, off);
            }
            if (lane < TPR) *reinterpret_cast<float4 *>(&red[j][warp][c4]) = o;
        }
        __syncthreads();
        for (int e = tid; e < GT * DVT; e += NT) {
            const int j = e / DVT, c = e % DVT;
            if (i0 + j >= len) break;
            float x = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) x += red[j][w][c];
            stf(static_cast<Tin *>(a.o) + ((size_t)(t0 + i0 + j) * a.H + h) * a.dv + col + c, a.scale * x);
        }
    }
    if (!a.S_out) return;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int row = p * RPP + rs;
        __stcs(reinterpret_cast<float4 *>(a.S_out + base + (size_t)row * a.dv), S[p]);
    }
}

namespace {
template <int DK, int DVT, typename Tin>
cudaError_t run(const LinArgs &a, cudaStream_t st) {
    const unsigned grid = (unsigned)((long long)a.nseq * a.H * (a.dv / DVT));
    return launch(!a.cu && a.T == 1 ? linear_recurrent_kernel<DK, DVT, 1, Tin> : linear_recurrent_kernel<DK, DVT, 4, Tin>, grid, NT, 0, st, a);
}
template <int DK, typename Tin>
cudaError_t by_tile(const LinArgs &a, cudaStream_t st) {
    const long long heads = (long long)a.nseq * a.H;
    if (a.dv >= 128 && heads * (a.dv / 128) >= 2 * 148) return run<DK, 128, Tin>(a, st);
    if (a.dv >= 64 && heads * (a.dv / 64) >= 2 * 148) return run<DK, 64, Tin>(a, st);
    return run<DK, 32, Tin>(a, st);
}
}  // namespace

cudaError_t launch_linear_recurrent(const LinArgs &a, bool bf16_in, cudaStream_t st) {
    switch (a.dk) {
        case 32: return bf16_in ? by_tile<32, bf16>(a, st) : by_tile<32, float>(a, st);
        case 64: return bf16_in ? by_tile<64, bf16>(a, st) : by_tile<64, float>(a, st);
        default: return bf16_in ? by_tile<128, bf16>(a, st) : by_tile<128, float>(a, st);
    }
}

}  // namespace kdn
