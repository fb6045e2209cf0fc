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
// (The slow path is a call, the hot loops are kept rolled and the sizes template arguments: the roles of a
// kernel run side by side, and together they have to stay in the instruction cache.)
static __device__ __noinline__ bool wait_slowly(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    const long long t0 = clock64();
    while (!mbar_try_wait_for(bar, parity, 1000000u)) {
        if (*abort_flag) return false;
        if (clock64() - t0 > 1000000000ll) {
            *abort_flag = 1;
            return false;
        }
    }
    return true;
}
struct Waits {
    volatile int *abort_flag;
    __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity) const {
        return mbar_try_wait_for(bar, parity, 1000000u) || wait_slowly(bar, parity, abort_flag);
    }
    // one answer for the warp
    __device__ __forceinline__ bool wait_all(uint64_t *bar, uint32_t parity) const { return __all_sync(0xffffffffu, wait(bar, parity)); }
};
// A value that is the same in every lane, in a form that shows it to the compiler: around the MMAs every
// branch and loop has to be provably one for the warp, or each of their operands is moved to uniform registers
// lane by lane (see elect_one)
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
// all lanes' writes before this are behind the arrival of the warp's one lane
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// ------------------------------------------------------------------ decay of a chunk
// A small launch ahead (linear_decay_kernel) forms one record per (chunk, head), which every kernel that walks
// the chunk fetches with a bulk copy: the factors' arithmetic is long for one warp between two chunks, and
// would be repeated by every tile of d_v and by the backward's three walks.
// With G the chunk's inclusive log2 decays: where |G| <= 60 throughout, 2^{-G_s} is stored and every factor is
// a product of stored ones (no exponential per pair); in a chunk that decays further (or a reset) G itself is
// stored in two floats and the factors are formed pair by pair, so that none exceeds one.  Behind the
// sequence's end the decay is 1.  A NaN among the log decays makes all of the chunk's factors NaN.
struct __align__(16) Decay {
    float b[C];                    // factored: 2^{-G_s};  pairwise: high part of G_s
    float lo[C];                   // pairwise: low part
    float2 whole;                  // the whole chunk's decay, in two floats
    Log2 total;                    // its log2
    int factored;
    int pad[3];
};
static_assert(sizeof(Decay) % 16 == 0, "bulk copies");
__device__ __forceinline__ float decay_since(const Decay &d, int t) {   // 2^{G_t}
    return d.factored ? 1.f / d.b[t] : exp2f(d.b[t] + d.lo[t]);
}
__device__ __forceinline__ float decay_until(const Decay &d, int s) {   // 2^{G_C - G_s}
    return d.factored ? d.whole.x * d.b[s] : exp2f((d.b[C - 1] - d.b[s]) + (d.lo[C - 1] - d.lo[s]));
}
__device__ __forceinline__ float decay_pair(const Decay &d, int t, int s) {   // 2^{G_t - G_s}, pairwise chunks
    return exp2f((d.b[t] - d.b[s]) + (d.lo[t] - d.lo[s]));
}

// ------------------------------------------------------------------ three bf16 terms of an fp32 value
__device__ __forceinline__ f32x2 unpack2(uint32_t u) { return pk2(bf16_lo(u), bf16_hi(u)); }
__device__ __forceinline__ uint32_t round_bf16x2(f32x2 x) { return pack_bf16x2(x2(x), y2(x)); }
// x = t0 + t1 + t2 exactly (barring underflow): each term is the nearest bf16 to what is left of the 24 bits.  So
// the products that fp32 states are summed from keep fp32's accuracy through bf16 operands (two terms would
// leave 2^-17); the first term alone is x rounded to bf16.
__device__ __forceinline__ void split3(f32x2 x, uint32_t (&t)[3]) {
    t[0] = round_bf16x2(x);
    x = sub2(x, unpack2(t[0]));
    t[1] = round_bf16x2(x);
    x = sub2(x, unpack2(t[1]));
    t[2] = round_bf16x2(x);
}

// half a row of a [128][64] bf16 tile, weighted, as three terms in three tiles (thread = row x half)
__device__ __forceinline__ void weigh_row(const uint8_t *src, uint8_t *dst, int row, int half, float w) {
#pragma unroll 2
    for (int j = 0; j < 4; ++j) {
        const uint32_t off = swz(row, (half * 4 + j) * 16);
        const uint4 u = *reinterpret_cast<const uint4 *>(src + off);
        const uint32_t x[4] = {u.x, u.y, u.z, u.w};
        uint32_t o[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t t[3];
            split3(mul2(unpack2(x[i]), pk2(w, w)), t);
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
// D[128, n] (+)= A B over 16-element K steps; shared-memory operands in 128-byte swizzled tiles.  The
// steps' descriptors differ from the tile's by a constant (the address field holds address / 16), so the
// issuing thread spends one addition per operand and step.
__device__ __forceinline__ uint64_t tile_kmajor(uint32_t tile) { return sdesc(tile, 16, 1024); }    // K along the rows' 128 bytes, 64 elements per tile
__device__ __forceinline__ uint64_t tile_mnmajor(uint32_t tile) { return sdesc(tile, ATOM, 1024); } // K along the tile's rows, MN in blocks of 64
__host__ __device__ constexpr uint32_t step_kmajor(int ks) { return ((ks >> 2) * ATOM + (ks & 3) * 32) >> 4; }
__host__ __device__ constexpr uint32_t step_mnmajor(int ks) { return ks * 2048 >> 4; }

// D (+)= A B over STEPS K steps, both operands in shared memory.  Unrolled: with the tile's address uniform over the
// warp the descriptors are uniform registers plus constants, and a step costs the issuing thread some 20 cycles
template <int STEPS, bool A_MN, bool B_MN, int N>
__device__ __forceinline__ void mma_tiles(uint32_t d, uint32_t a, uint32_t b, bool acc) {
    constexpr uint32_t ID = idesc_bf16(128, N, A_MN, B_MN);
    const uint64_t da = A_MN ? tile_mnmajor(a) : tile_kmajor(a), db = B_MN ? tile_mnmajor(b) : tile_kmajor(b);
#pragma unroll
    for (int ks = 0; ks < STEPS; ++ks)
        mma_bf16(d, da + (A_MN ? step_mnmajor(ks) : step_kmajor(ks)), db + (B_MN ? step_mnmajor(ks) : step_kmajor(ks)), ID, acc || ks > 0);
}

// delta[dk, dv tile] = X^T [Y0 Y1 Y2]: 64 columns for each term, so that X is read from shared memory once
__device__ __forceinline__ void mma_delta(uint32_t d, uint32_t x, uint32_t y) { mma_tiles<8, true, true, 192>(d, x, y, false); }

// ------------------------------------------------------------------ states in the workspace
// One tile of 64 columns of a [d_k, d_v] fp32 state: [16 column quads][128 rows][4].  A warp whose lanes
// are rows of S (TMEM lanes) moves 512 contiguous bytes per access.
constexpr size_t TILE_FLOATS = 128 * 64;
__device__ __forceinline__ size_t tile_at(size_t slot, int H, int h, int tiles, int tile) {
    return ((slot * H + h) * tiles + tile) * TILE_FLOATS;
}

// thread of a TMA issuer: a [128 tokens][64 channels] tile as two boxes of 64 tokens
__device__ __forceinline__ void load_tile(uint8_t *dst, const CUtensorMap *m, int c0, int h, int tok, uint64_t *bar) {
    tma_load_3d(dst, m, c0, h, tok, bar);
    tma_load_3d(dst + ATOM / 2, m, c0, h, tok + 64, bar);
}
// the same tile brought into L2
__device__ __forceinline__ void prefetch_tile(const CUtensorMap *m, int c0, int h, int tok) {
    tma_prefetch_3d(m, c0, h, tok);
    tma_prefetch_3d(m, c0, h, tok + 64);
}
// after a wait gave up: one more bounded wait for a barrier that copies or MMAs in flight still arrive on
static __device__ __noinline__ void drain(uint64_t *bar, uint32_t parity) { mbar_wait(bar, parity, 100000000ll); }

// What the backward's first launches leave in the workspace for its last one
struct States {
    const Decay *decay;            // [slots of C][H]
    const float *S, *R;            // [slots of C][H][tiles]: states at the chunks' starts, state gradients at their ends
    float *share;                  // [slots of C][H]: the chunks' shares of a per-head decay's gradient
};
size_t states_workspace_bytes(const LinArgs &a);
cudaError_t launch_states(const LinBwdArgs &b, void *workspace, States *out, cudaStream_t st);

}  // namespace lin
}  // namespace kdn
