// What the tensor-core kernels of linear attention share: chunks of 128 tokens, the decay factors of
// a chunk, the weighted rows of the state update as three bf16 terms, and bounded waits that see each
// other's failures.
#pragma once

#include "kdn_linear.cuh"
#include "kdn_tc.cuh"

namespace kdn {
namespace lin {

using namespace tc;

constexpr int C = 128;             // tokens of a chunk: the M of every MMA
constexpr int DVT = 64;            // columns of d_v per tile: one 128-byte swizzle atom
constexpr int DKP = 128;           // key channels, padded with zeros where d_k is smaller
constexpr int ATOM = C * 128;      // bytes of a [128 rows][64 bf16] swizzled tile

// ------------------------------------------------------------------ waits
// Every wait gives up after ~0.5 s of SM clocks, or as soon as another wait of the CTA has; the
// kernels then stop issuing work and drain what is in flight.
struct Waits {
    volatile int *abort_flag;
    __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity) const {
        if (mbar_try_wait(bar, parity)) return true;
        const long long t0 = clock64();
        while (!mbar_try_wait(bar, parity)) {
            if (*abort_flag) return false;
            if (clock64() - t0 > 1000000000ll) {
                *abort_flag = 1;
                return false;
            }
        }
        return true;
    }
};
// all lanes' writes before this are behind the arrival of the warp's one lane
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// ------------------------------------------------------------------ decay of a chunk
// With G the chunk's inclusive log2 decays (fp64): where |G| <= 60 throughout, e^{-G_s} is stored and
// every factor is a product of stored ones (no exponential per pair); in a chunk that decays further
// (or a reset) G itself is stored in two floats and the factors are formed pair by pair, so that none
// exceeds one.
struct Decay {
    float b[C];                    // factored: 2^{-G_s};  pairwise: high part of G_s
    float lo[C];                   // pairwise: low part
};
struct DecayMeta {
    float2 whole;                  // the whole chunk's decay, in two floats
    int factored;
    int pad;
};
__device__ __forceinline__ float decay_since(const Decay &d, bool factored, int t) {   // 2^{G_t}
    return factored ? 1.f / d.b[t] : exp2f(d.b[t] + d.lo[t]);
}
__device__ __forceinline__ float decay_until(const Decay &d, const DecayMeta &m, int s) {   // 2^{G_C - G_s}
    return m.factored ? m.whole.x * d.b[s] : exp2f((d.b[C - 1] - d.b[s]) + (d.lo[C - 1] - d.lo[s]));
}
__device__ __forceinline__ float decay_pair(const Decay &d, int t, int s) {   // 2^{G_t - G_s}, pairwise chunks
    return exp2f((d.b[t] - d.b[s]) + (d.lo[t] - d.lo[s]));
}

// one warp: the factors of the chunk whose tokens' log2 decays x (four per lane) were fetched before
__device__ __forceinline__ void decay_fetch(const LinArgs &a, int tok, int L, int h, double (&x)[4]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = lane * 4 + i < L ? lin_log2_decay(a, tok + lane * 4 + i, h) : 0.0;
}
__device__ __forceinline__ void decay_write(const double (&x)[4], Decay *d, DecayMeta *m) {
    const int lane = threadIdx.x & 31;
    double G[4];
    G[0] = x[0];
#pragma unroll
    for (int i = 1; i < 4; ++i) G[i] = G[i - 1] + x[i];
    double s = G[3];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += y;
    }
    const double before = s - G[3];
    bool in = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        G[i] += before;
        in = in && G[i] >= -60.0 && G[i] <= 60.0;
    }
    const bool factored = __all_sync(0xffffffffu, in);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float hi = (float)G[i];
        d->b[lane * 4 + i] = factored ? lin_exp2(-G[i]) : hi;
        if (!factored) d->lo[lane * 4 + i] = (float)(G[i] - (double)hi);
    }
    if (lane == 31) {
        m->whole = lin_chunk_decay(s);
        m->factored = factored;
    }
}

// ------------------------------------------------------------------ three bf16 terms of an fp32 value
// x = t0 + t1 + t2 up to 2^-24 |x|: the products that fp32 states are summed from keep fp32's accuracy
// through bf16 operands (two terms alone would leave 2^-17)
__device__ __forceinline__ void split3(float x, float y, uint32_t (&t)[3]) {
    t[0] = pack_bf16x2(x, y);
    x -= bf16_lo(t[0]);
    y -= bf16_hi(t[0]);
    t[1] = pack_bf16x2(x, y);
    t[2] = pack_bf16x2(x - bf16_lo(t[1]), y - bf16_hi(t[1]));
}

// half a row of a [128][64] bf16 tile, weighted, as three terms in three tiles (thread = row x half)
__device__ __forceinline__ void weigh_row(const uint8_t *src, uint8_t *dst, int row, int half, float w) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t off = swz(row, (half * 4 + j) * 16);
        const uint4 u = *reinterpret_cast<const uint4 *>(src + off);
        const uint32_t x[4] = {u.x, u.y, u.z, u.w};
        uint32_t o[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t t[3];
            split3(bf16_lo(x[i]) * w, bf16_hi(x[i]) * w, t);
            o[0][i] = t[0]; o[1][i] = t[1]; o[2][i] = t[2];
        }
#pragma unroll
        for (int k = 0; k < 3; ++k)
            *reinterpret_cast<uint4 *>(dst + k * ATOM + off) = make_uint4(o[k][0], o[k][1], o[k][2], o[k][3]);
    }
}
__device__ __forceinline__ void zero_row(uint8_t *dst, int row, int first, int n) {   // n 16-byte pieces
    for (int j = 0; j < n; ++j) *reinterpret_cast<uint4 *>(dst + swz(row, (first + j) * 16)) = make_uint4(0, 0, 0, 0);
}

// ------------------------------------------------------------------ MMAs (one thread)
// D[128, n] (+)= A B over 16-element K steps; shared-memory operands in 128-byte swizzled tiles
__device__ __forceinline__ uint64_t kmajor(uint32_t tile, int step) {   // K along the rows' 128 bytes, 64 elements per tile
    return sdesc(tile + (uint32_t)(step >> 2) * ATOM + (uint32_t)(step & 3) * 32u, 16, 1024);
}
__device__ __forceinline__ uint64_t mnmajor(uint32_t tile, int step) {  // K along the tile's rows, MN in blocks of 64
    return sdesc(tile + (uint32_t)step * 2048u, ATOM, 1024);
}

// delta[dk, dv tile] = X^T (Y0 + Y1 + Y2): columns 0..63 take the first term, 64..127 the other two
__device__ __forceinline__ void mma_delta(uint32_t d, uint32_t x, uint32_t y) {
    constexpr uint32_t ID2 = idesc_bf16(128, 128, true, true), ID1 = idesc_bf16(128, 64, true, true);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) mma_bf16(d, mnmajor(x, ks), mnmajor(y, ks), ID2, ks > 0);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) mma_bf16(d + 64, mnmajor(x, ks), mnmajor(y + 2 * ATOM, ks), ID1, 1);
}

// ------------------------------------------------------------------ states in the workspace
// One tile of 64 columns of a [d_k, d_v] fp32 state: [16 column quads][128 rows][4].  A warp whose lanes
// are rows of S (TMEM lanes) moves 512 contiguous bytes per access.
constexpr size_t TILE_FLOATS = 128 * 64;
__device__ __forceinline__ size_t tile_at(size_t slot, int H, int h, int tiles, int tile) {
    return ((slot * H + h) * tiles + tile) * TILE_FLOATS;
}

}  // namespace lin
}  // namespace kdn
