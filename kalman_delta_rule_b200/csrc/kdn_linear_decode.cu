// Linear attention with a decay for each head, recurrent form: n tokens of each sequence applied in
// order to a state in HBM that is read once and written back once, in place.  Per token
//     S <- e^g S + k v^T,   o = scale S^T q.
// A CTA owns a d_v tile of one (sequence, head); its part of S stays in registers as float4 rows
// between the tokens.  Columns of S never meet, so the tile width is free: the widest one that still
// gives every SM two CTAs (few sequences: narrow tiles, more CTAs, shorter loads per CTA; many: whole
// rows, so that q, k and the sums over rows are shared by all columns).
// Bound by the state's read and write (131 KB per head at d = 128, against 1 KB of token data).
#include "kdn_common.cuh"
#include "kdn_launch.h"

namespace kdn {

namespace {
constexpr int NT = 256;
}

template <int DK, int DVT, typename Tin>
__global__ void __launch_bounds__(NT) linear_decode_kernel(LinArgs a)
{
    constexpr int TPR = DVT / 4;           // threads per row of S
    constexpr int RPP = NT / TPR;          // rows per pass
    constexpr int NP = DK / RPP;
    static_assert(DK % RPP == 0, "row passes");
    constexpr int NW = NT / 32;
    const int tiles = a.dv / DVT;
    const int sh = blockIdx.x / tiles, col = (blockIdx.x % tiles) * DVT;
    const int s = sh / a.H, h = sh % a.H;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c4 = (tid % TPR) * 4, rs = tid / TPR;
    __shared__ float qk[2][2][DK];                       // [buffer][q, k]
    __shared__ __align__(16) float red[2][NW][DVT];

    const size_t base = (size_t)sh * DK * a.dv + col + c4;
    float4 S[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int row = p * RPP + rs;
        S[p] = __ldcs(reinterpret_cast<const float4 *>(a.S0 + base + (size_t)row * a.dv));
    }
    for (int i = 0; i < a.T; ++i) {
        const int buf = i & 1;
        const size_t th = ((size_t)s * a.T + i) * a.H + h;
        if (tid < DK) {
            qk[buf][0][tid] = ldf(static_cast<const Tin *>(a.q) + th * DK + tid);
            qk[buf][1][tid] = ldf(static_cast<const Tin *>(a.k) + th * DK + tid);
        }
        const float4 v = ldf4(static_cast<const Tin *>(a.v) + th * a.dv + col + c4);
        const float f = a.decay == KDN_DECAY_NONE ? 1.f : expf(a.decay == KDN_DECAY_HEAD ? __ldg(a.g + h) : __ldg(a.g + th));
        __syncthreads();
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int row = p * RPP + rs;
            const float q = qk[buf][0][row], k = qk[buf][1][row];
            float4 x = S[p];
            x = make_float4(fmaf(k, v.x, f * x.x), fmaf(k, v.y, f * x.y), fmaf(k, v.z, f * x.z), fmaf(k, v.w, f * x.w));
            o = make_float4(fmaf(q, x.x, o.x), fmaf(q, x.y, o.y), fmaf(q, x.z, o.z), fmaf(q, x.w, o.w));
            S[p] = x;
        }
#pragma unroll
        for (int off = TPR; off < 32; off <<= 1) {        // rows of the same warp
            o.x += __shfl_xor_sync(0xffffffffu, o.x, off);
            o.y += __shfl_xor_sync(0xffffffffu, o.y, off);
            o.z += __shfl_xor_sync(0xffffffffu, o.z, off);
            o.w += __shfl_xor_sync(0xffffffffu, o.w, off);
        }
        if (lane < TPR) *reinterpret_cast<float4 *>(&red[buf][warp][c4]) = o;
        __syncthreads();
        if (tid < DVT) {
            float x = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) x += red[buf][w][tid];
            stf(static_cast<Tin *>(a.o) + th * a.dv + col + tid, a.scale * x);
        }
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int row = p * RPP + rs;
        __stcs(reinterpret_cast<float4 *>(a.S_out + base + (size_t)row * a.dv), S[p]);
    }
}

namespace {
template <int DK, int DVT, typename Tin>
cudaError_t run(const LinArgs &a, cudaStream_t st) {
    linear_decode_kernel<DK, DVT, Tin><<<(unsigned)((long long)a.nseq * a.H * (a.dv / DVT)), NT, 0, st>>>(a);
    return cudaGetLastError();
}
template <int DK, typename Tin>
cudaError_t by_tile(const LinArgs &a, cudaStream_t st) {
    const long long heads = (long long)a.nseq * a.H;
    if (a.dv >= 128 && heads * (a.dv / 128) >= 2 * 148) return run<DK, 128, Tin>(a, st);
    if (a.dv >= 64 && heads * (a.dv / 64) >= 2 * 148) return run<DK, 64, Tin>(a, st);
    return run<DK, 32, Tin>(a, st);
}
}  // namespace

cudaError_t launch_linear_decode(const LinArgs &a, bool bf16_in, cudaStream_t st) {
    switch (a.dk) {
        case 32: return bf16_in ? by_tile<32, bf16>(a, st) : by_tile<32, float>(a, st);
        case 64: return bf16_in ? by_tile<64, bf16>(a, st) : by_tile<64, float>(a, st);
        default: return bf16_in ? by_tile<128, bf16>(a, st) : by_tile<128, float>(a, st);
    }
}

}  // namespace kdn
