// Linear attention with a decay for each head on the tensor cores (tcgen05, bf16 inputs): forward, and
// the states at the chunks' boundaries that the backward reads.  Chunks of C = 128 tokens; per chunk,
// with the factors of kdn_linear_tc.cuh and S the fp32 state at the chunk's start,
//     O  = scale ((Q K^T o D) V + diag(e^G) Q S),     S' = e^{G_C} S + K^T diag(e^{G_C - G}) V
//
// Forward (linear_forward_kernel): a CTA walks one segment of a sequence for one head and 64 columns of
// d_v, chunk by chunk, with everything but the inputs and outputs on chip.  Warp roles, each a loop over
// the chunks that meets the others at mbarriers:
//   TMA      refills Q, K, the V tile and the decay record for chunk c + 2, each as soon as chunk c is done with it
//   MMA      one thread: scores = Q K^T, delta = K^T V', OS = Q S, OI = P V (P from TMEM)
//   W (8)    V' = diag(e^{G_C - G}) V as three bf16 terms; scores (TMEM) -> decayed, masked, bf16 -> P (TMEM)
//   S (8)    S <- e^{G_C} S + delta in registers (fp32), its bf16 copy for Q S
//   O (4)    o = scale (OI + e^G OS)
// Its floor is one pass over q, k, v and o at HBM's rate.  The MMAs take about 1950 cycles per chunk and tile (scores
// 512, Q S 384, delta 800 -- its A operand, K, meets three terms of the weighted rows in one product of 192 columns --, P V
// 256), shared memory's reads for them and the warps' passes about 2900, and a chunk 3450: a role's own latencies (TMEM
// loads, conversions, the fence before its mbarrier) do not overlap with themselves.  B4 H16 T4096 d128: 79 us, tensor pipe
// 37% active, DRAM 38%; with the decays' launch a call takes 88 to 92, 3.0 to 3.1 TB/s.  One CTA per SM; that problem's 128 chains leave 20 SMs idle.
// Rounding: P and the copy of S that Q reads are bf16 (o itself is); the state never is -- its products
// take three-term weighted rows and it stays in fp32 registers, so it keeps fp32's accuracy over any length.
//
// Few chains (sequence x head x tile) would leave SMs idle, so a sequence can be cut into segments: a first
// launch (linear_state_kernel, TOTALS) forms each earlier sub-segment's contribution to the state from k and
// v alone, and a segment's CTA starts from their decayed sum.
#include <mutex>

#include "kdn_launch.h"
#include "kdn_linear_tc.cuh"

namespace kdn {

using namespace lin;

namespace {

// warps: W weighted rows (forward: and scores), S state, O outputs (forward); then MMA and TMA
constexpr int NW_W = 8, NW_S = 8, NW_O = 4;
constexpr int NT_F = (NW_W + NW_S + NW_O + 2) * 32;
constexpr int NT_S = (NW_W + NW_S + 2) * 32;

struct FwdSmem {
    static constexpr int Q = 0, K = Q + 2 * 2 * ATOM, V = K + 2 * 2 * ATOM, VP = V + 2 * ATOM, S = VP + 3 * ATOM,
                         DEC = S + ATOM, BAR = DEC + 2 * (int)sizeof(Decay), NBAR = 20, CTL = BAR + NBAR * 8, TOTAL = CTL + 16;
};
static_assert(FwdSmem::TOTAL <= 227 * 1024, "shared memory");

struct StateSmem {
    static constexpr int X = 0, Y = X + 2 * 2 * ATOM, VP = Y + 2 * ATOM, DEC = VP + 2 * 3 * ATOM,
                         BAR = DEC + 2 * (int)sizeof(Decay), NBAR = 18,
                         CTL = BAR + NBAR * 8, TOTAL = CTL + 16;
};
static_assert(StateSmem::TOTAL <= 227 * 1024, "shared memory");

// segments of `seg` tokens; the totals of sub-segments of `sub` tokens (seg a multiple of sub)
struct Split {
    int seg, sub;
    const float *U;                // [slots of sub][H][tiles] state tiles
    const float2 *dec;             // [slots of sub][H] decay of the sub-segment
};

struct FwdArgs {
    LinArgs a;
    Split sp;
    const Decay *decay;            // [slots of C][H]
    CUtensorMap tq, tk, tv;
};

struct StateArgs {
    LinArgs a;                     // q, k, v, S0 unused
    Split sp;                      // STATES: where the walk starts from
    int piece;                     // tokens per CTA: sp.sub (TOTALS) or sp.seg (STATES)
    const float *first;            // STATES: state before the first (REV: gradient behind the last) chunk, or NULL
    float *last;                   // STATES: state behind the last (REV: gradient before the first) chunk, or NULL
    float *tiles;                  // TOTALS: [slots of sub]; STATES: [slots of C][H][tiles]
    float2 *dec;                   // TOTALS
    const Decay *decay;            // [slots of C][H]
    CUtensorMap tx, ty;
};

// 32 columns of row `row` of a state, in pairs: from the caller's [dk, dv] layout (zero outside it) ...
__device__ __forceinline__ void load_caller(f32x2 (&S)[16], const float *src, int dk, int dv, int row, int col) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float4 x = src && row < dk && col < dv ? __ldg(reinterpret_cast<const float4 *>(src + (size_t)row * dv + col) + j)
                                                     : make_float4(0.f, 0.f, 0.f, 0.f);
        S[2 * j] = pk2(x.x, x.y);
        S[2 * j + 1] = pk2(x.z, x.w);
    }
}
__device__ __forceinline__ float4 quad(const f32x2 (&S)[16], int j) { return make_float4(x2(S[2 * j]), y2(S[2 * j]), x2(S[2 * j + 1]), y2(S[2 * j + 1])); }
__device__ __forceinline__ void store_caller(const f32x2 (&S)[16], float *dst, int dk, int dv, int row, int col) {
    if (row >= dk || col >= dv) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) *(reinterpret_cast<float4 *>(dst + (size_t)row * dv + col) + j) = quad(S, j);
}
// ... and to a workspace tile
__device__ __forceinline__ void store_tile(const f32x2 (&S)[16], float *tile, int row, int half) {
#pragma unroll
    for (int j = 0; j < 8; ++j) *reinterpret_cast<float4 *>(tile + ((half * 8 + j) * 128 + row) * 4) = quad(S, j);
}
// S <- decay S + x: the decay in two floats (see lin_chunk_decay)
__device__ __forceinline__ f32x2 carry2(f32x2 hi, f32x2 lo, f32x2 s, f32x2 x) { return fma2(hi, s, fma2(lo, s, x)); }
// ... with the tile of a sub-segment
__device__ __forceinline__ void fold_tile(f32x2 (&S)[16], const float *tile, float2 dec, int row, int half) {
    const f32x2 hi = pk2(dec.x, dec.x), lo = pk2(dec.y, dec.y);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float4 x = __ldg(reinterpret_cast<const float4 *>(tile + ((half * 8 + j) * 128 + row) * 4));
        S[2 * j] = carry2(hi, lo, S[2 * j], pk2(x.x, x.y));
        S[2 * j + 1] = carry2(hi, lo, S[2 * j + 1], pk2(x.z, x.w));
    }
}
// ... with a chunk's delta from TMEM
__device__ __forceinline__ void add_delta(f32x2 (&S)[16], uint32_t d, float2 dec) {
    const f32x2 hi = pk2(dec.x, dec.x), lo = pk2(dec.y, dec.y);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        float x[8], y[8], z[8];
        tmem_ld8x3(d + p * 8, d + 64 + p * 8, d + 128 + p * 8, x, y, z);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f32x2 low = add2(pk2(y[2 * j], y[2 * j + 1]), pk2(z[2 * j], z[2 * j + 1]));
            S[p * 4 + j] = carry2(hi, lo, S[p * 4 + j], add2(pk2(x[2 * j], x[2 * j + 1]), low));
        }
    }
}

}  // namespace

// ================================================================= decay records
// a warp per (chunk, head), four tokens per lane
__global__ void __launch_bounds__(256) linear_decay_kernel(LinArgs a, Decay *rec, long long n)
{
    let_next_launch();                        // the walk that follows may set itself up meanwhile
    const long long id = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (id >= n) return;
    const int u = (int)(id / a.H), h = (int)(id % a.H);
    LinPiece p;
    if (!lin_piece(a, u, C, p) || p.len == 0) return;
    const int tok = p.t0 + p.j * C, L = min(C, p.len - p.j * C);
    Decay *d = rec + id;
    float g[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        g[i] = 0.f;
        if (lane * 4 + i < L) g[i] = lin_load_decay(a, tok + lane * 4 + i, h);
    }
    Log2 G[4];
    bool bad = false, in = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bad = bad || g[i] != g[i];
        G[i] = i ? G[i - 1] + lin_log2(g[i]) : lin_log2(g[i]);
    }
    Log2 s = G[3];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const Log2 y = {__shfl_up_sync(0xffffffffu, s.hi, off), __shfl_up_sync(0xffffffffu, s.lo, off)};
        if (lane >= off) s = y + s;
    }
    Log2 before = {__shfl_up_sync(0xffffffffu, s.hi, 1), __shfl_up_sync(0xffffffffu, s.lo, 1)};
    if (lane == 0) before = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        G[i] = before + G[i];
        in = in && fabsf(G[i].hi) <= 60.f;
    }
    const bool factored = __all_sync(0xffffffffu, in);
    bad = __any_sync(0xffffffffu, bad);
    float b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        b[i] = factored ? lin_exp2({-G[i].hi, -G[i].lo}) : G[i].hi;
        if (bad) b[i] = __int_as_float(0x7fc00000);
    }
    *reinterpret_cast<float4 *>(d->b + lane * 4) = make_float4(b[0], b[1], b[2], b[3]);
    *reinterpret_cast<float4 *>(d->lo + lane * 4) = make_float4(G[0].lo, G[1].lo, G[2].lo, G[3].lo);
    if (lane == 31) {
        d->whole = bad ? make_float2(__int_as_float(0x7fc00000), 0.f) : lin_chunk_decay(s);
        d->total = s;
        d->factored = factored;
    }
}

// ================================================================= forward
template <int KATOMS>       // 64-channel tiles of q and k in use
__global__ void __launch_bounds__(NT_F, 1) linear_forward_kernel(const __grid_constant__ FwdArgs f)
{
    using L_ = FwdSmem;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    const LinArgs &a = f.a;
    const int tiles = (a.dv + DVT - 1) / DVT;
    const int tile = blockIdx.x % tiles, h = (blockIdx.x / tiles) % a.H, u = blockIdx.x / tiles / a.H;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    constexpr int W_S = NW_W, W_O = W_S + NW_S, W_MMA = W_O + NW_O, W_TMA = W_MMA + 1;   // MMA beside the rows with the fewest scores
    LinPiece pc;
    if (!uniform(lin_piece(a, u, f.sp.seg, pc))) return wait_for_launch();
    const int tok0 = pc.t0 + pc.j * f.sp.seg, len = min(f.sp.seg, pc.len - pc.j * f.sp.seg);
    const int n = uniform((len + C - 1) / C);

    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L_::BAR);
    uint64_t *qk_full = bar, *v_full = bar + 2, *q_free = bar + 4, *k_free = bar + 6, *v_free = bar + 8, *dec_full = bar + 10,
             *dec_free = bar + 12, *sc_full = bar + 14, *p_full = bar + 15, *o_full = bar + 16, *dl_full = bar + 17,
             *delta_ok = bar + 18,             // the weighted rows are there, and the delta before has been read
             *qs_ok = bar + 19;                // the state's copy is there, and the outputs before have been read
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L_::CTL);
    int *abort_flag = reinterpret_cast<int *>(sm + L_::CTL + 4);
    const Waits w{abort_flag};
    Decay *dec = reinterpret_cast<Decay *>(sm + L_::DEC);

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(qk_full + i, 1);
            mbar_init(v_full + i, 1);
            mbar_init(q_free + i, 1);
            mbar_init(k_free + i, NW_S);
            mbar_init(v_free + i, NW_O);
            mbar_init(dec_full + i, 1);
            mbar_init(dec_free + i, NW_W + NW_S + NW_O);
        }
        mbar_init(sc_full, 1);
        mbar_init(p_full, NW_W);
        mbar_init(o_full, 1);
        mbar_init(dl_full, 1);
        mbar_init(delta_ok, NW_W + NW_S);
        mbar_init(qs_ok, NW_S + NW_O);
        mbar_fence_init();
        *abort_flag = (sb & 1023u) ? 1 : 0;   // the swizzled tiles need 1 KB alignment
        tma_prefetch_desc(&f.tq);
        tma_prefetch_desc(&f.tk);
        tma_prefetch_desc(&f.tv);
    }
    if (KATOMS == 1) {                        // channels 64..127 of K and Q: zeros, never written again
        for (int i = threadIdx.x; i < 4 * (ATOM / 16); i += NT_F) {
            const int t = i / (ATOM / 16);
            *reinterpret_cast<uint4 *>(sm + ((t & 1) ? L_::K : L_::Q) + (t >> 1) * 2 * ATOM + ATOM + (i % (ATOM / 16)) * 16) =
                make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
    }
    if (warp == W_MMA) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const uint32_t T_SC = tmem, T_P = tmem + 128, T_OI = tmem + 192, T_OS = tmem + 256, T_DL = tmem + 320;
    const uint32_t lanes = ((uint32_t)(warp & 3) * 32u) << 16;
    const int row = (warp & 3) * 32 + lane;

    if (warp < W_S) {
        // ---------------------------------------------------------- W: weighted rows of V, then the scores
        const int half = warp >> 2, q4 = warp & 3;
        for (int c = 0; c < n; ++c) {
            const int st = c & 1, L = min(C, len - c * C);
            if (!w.wait(dec_full + st, (c >> 1) & 1) || !w.wait(v_full + st, (c >> 1) & 1)) break;
            const Decay &d = dec[st];
            const bool factored = d.factored;
            const float until = decay_until(d, row), since = factored ? 1.f / d.b[row] : 1.f;
            if (c >= 1 && !w.wait(dl_full, (c - 1) & 1)) break;   // the MMAs that read the weighted rows before
            if (row < L) {
                weigh_row(sm + L_::V + st * ATOM, sm + L_::VP, row, half, until);
            } else {                          // rows behind the sequence's end: zeros in every operand that is summed over rows
#pragma unroll 1
                for (int k = 0; k < 3; ++k) zero_row(sm + L_::VP + k * ATOM, row, half * 4, 4);
                zero_row(sm + L_::V + st * ATOM, row, half * 4, 4);
                if (w.wait(qk_full + st, (c >> 1) & 1)) zero_row(sm + L_::K + (st * 2 + half) * ATOM, row, 0, 8);
            }
            fence_async_smem();
            warp_arrive(delta_ok);

            if (!w.wait(sc_full, c & 1)) break;
            tc_fence_after();
            // P: pieces of 16 columns, every other one is this warp's; zero above the diagonal
#pragma unroll 1
            for (int c16 = half * 16; c16 < C; c16 += 32) {
                uint32_t p[8] = {};
                if (c16 <= q4 * 32 + 31) {
                    float x[16];
                    tmem_ld16(T_SC + lanes + c16, x);
                    if (factored) {                   // (the factors first: their product is at most one, 2^{-G_s} alone up to 2^60)
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 b = *reinterpret_cast<const float4 *>(d.b + c16 + j);
                            if constexpr (KATOMS == 1) {      // (in pairs it costs this instance 16 bytes of spills: 65.8 -> 67.5 us)
                                x[j] *= since * b.x; x[j + 1] *= since * b.y; x[j + 2] *= since * b.z; x[j + 3] *= since * b.w;
                            } else {
                                const f32x2 y = mul2(pk2(x[j], x[j + 1]), mul2(pk2(since, since), pk2(b.x, b.y))),
                                            z = mul2(pk2(x[j + 2], x[j + 3]), mul2(pk2(since, since), pk2(b.z, b.w)));
                                x[j] = x2(y); x[j + 1] = y2(y); x[j + 2] = x2(z); x[j + 3] = y2(z);
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) x[j] *= decay_pair(d, row, c16 + j);
                    }
                    if (c16 + 15 > q4 * 32) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) x[j] = c16 + j <= row ? x[j] : 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) p[j] = round_bf16x2(pk2(x[2 * j], x[2 * j + 1]));
                }
                tmem_st8(T_P + lanes + c16 / 2, p);
            }
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(p_full);
            warp_arrive(dec_free + st);
        }
    } else if (warp < W_O) {
        // ---------------------------------------------------------- S: the state
        const int half = (warp - W_S) >> 2;
        const int col = tile * DVT + half * 32;
        const size_t se = ((size_t)pc.s * a.H + h) * a.dk * a.dv;
        f32x2 S[16];
        load_caller(S, a.S0 ? a.S0 + se : nullptr, a.dk, a.dv, row, col);
        const int before = pc.j * (f.sp.seg / f.sp.sub), s0 = lin_first_slot(a, pc.s, pc.t0, f.sp.sub);
        for (int i = 0; i < before; ++i)
            fold_tile(S, f.sp.U + tile_at(s0 + i, a.H, h, tiles, tile), f.sp.dec[(size_t)(s0 + i) * a.H + h], row, half);
        bool ok = true;
        warp_arrive(delta_ok);                // (there is no delta before the first)
        for (int c = 0; c < n; ++c) {
            const int st = c & 1;
            // the bf16 copy that chunk c's Q S reads, once the Q S before has
            if (c > 0) ok = w.wait(q_free + (st ^ 1), ((c - 1) >> 1) & 1);
            if (!ok) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t z[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = round_bf16x2(S[j * 4 + i]);
                *reinterpret_cast<uint4 *>(sm + L_::S + swz(row, (half * 4 + j) * 16)) = make_uint4(z[0], z[1], z[2], z[3]);
            }
            fence_async_smem();
            warp_arrive(qs_ok);
            ok = w.wait(dec_full + st, (c >> 1) & 1);
            if (!ok) break;
            const float2 whole = dec[st].whole;
            warp_arrive(dec_free + st);
            ok = w.wait(dl_full, c & 1);
            if (!ok) break;
            tc_fence_after();
            warp_arrive(k_free + st);
            add_delta(S, T_DL + lanes + half * 32, whole);
            tc_fence_before();
            warp_arrive(delta_ok);
        }
        if (ok && a.S_out && (long long)(pc.j + 1) * f.sp.seg >= pc.len) store_caller(S, a.S_out + se, a.dk, a.dv, row, col);
    } else if (warp < W_MMA) {
        // ---------------------------------------------------------- O: the outputs, through the chunk's V tile, which its MMAs
        // are done with: a warp's 32 rows x 128 bytes there and back, so that eight lanes share a row's 128 bytes in memory
        // (a row per lane costs 8 times the LSU cycles, and the fences of the other roles wait behind them)
        const int col = tile * DVT + (lane & 7) * 8;
        bf16 *o = static_cast<bf16 *>(a.o) + ((size_t)(tok0 + (warp & 3) * 32 + (lane >> 3)) * a.H + h) * a.dv + col;
        warp_arrive(qs_ok);                   // (there are no outputs before the first)
        for (int c = 0; c < n; ++c) {
            const int st = c & 1, L = min(C, len - c * C);
            if (!w.wait(dec_full + st, (c >> 1) & 1)) break;
            const float fs = a.scale * decay_since(dec[st], row);
            warp_arrive(dec_free + st);
            const f32x2 fs2 = pk2(fs, fs), fi2 = pk2(a.scale, a.scale);
            if (!w.wait(o_full, c & 1)) break;
            tc_fence_after();
#pragma unroll 2
            for (int p = 0; p < 64; p += 16) {
                float x[16], y[16];
                tmem_ld16x2(T_OI + lanes + p, T_OS + lanes + p, x, y);
                if (p == 48) {
                    tc_fence_before();
                    warp_arrive(qs_ok);
                }
#pragma unroll
                for (int j = 0; j < 16; j += 8) {
                    uint32_t z[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        z[i] = round_bf16x2(fma2(fi2, pk2(x[j + 2 * i], x[j + 2 * i + 1]), mul2(fs2, pk2(y[j + 2 * i], y[j + 2 * i + 1]))));
                    *reinterpret_cast<uint4 *>(sm + L_::V + st * ATOM + swz(row, (p + j) * 2)) = make_uint4(z[0], z[1], z[2], z[3]);
                }
            }
            __syncwarp();
#pragma unroll
            for (int r = 0; r < 32; r += 4) {
                const int t = (warp & 3) * 32 + r + (lane >> 3);
                const uint4 z = *reinterpret_cast<const uint4 *>(sm + L_::V + st * ATOM + swz(t, (lane & 7) * 16));
                if (t < L && col < a.dv) *reinterpret_cast<uint4 *>(o + (size_t)r * a.H * a.dv) = z;
            }
            o += (size_t)C * a.H * a.dv;
            fence_async_smem();
            warp_arrive(v_free + st);
        }
    } else if (warp == W_TMA) {
        // ---------------------------------------------------------- TMA: Q, K and V are refilled as each is free
        if (lane == 0) {
            wait_for_launch();                // the decay records are complete
            const Decay *decay = f.decay + (size_t)(lin_first_slot(a, pc.s, pc.t0, C) + pc.j * (f.sp.seg / C)) * a.H + h;
            for (int c = 0; c < n; ++c) {
                const int st = c & 1, tok = tok0 + c * C;
                const uint32_t before = ((c >> 1) - 1) & 1;
                // two stages are one chunk ahead, less than DRAM's latency: the chunk two further on is brought into L2
                if (c + 2 < n) {
#pragma unroll 1
                    for (int k = 0; k < KATOMS; ++k) {
                        prefetch_tile(&f.tq, k * 64, h, tok + 2 * C);
                        prefetch_tile(&f.tk, k * 64, h, tok + 2 * C);
                    }
                    prefetch_tile(&f.tv, tile * DVT, h, tok + 2 * C);
                }
                if (c >= 2 && !w.wait(q_free + st, before)) break;
                if (*w.abort_flag) break;
                mbar_expect_tx(qk_full + st, (uint32_t)(2 * KATOMS) * ATOM);
                for (int k = 0; k < KATOMS; ++k) load_tile(sm + L_::Q + (st * 2 + k) * ATOM, &f.tq, k * 64, h, tok, qk_full + st);
                if (c >= 2 && !w.wait(k_free + st, before)) break;
                for (int k = 0; k < KATOMS; ++k) load_tile(sm + L_::K + (st * 2 + k) * ATOM, &f.tk, k * 64, h, tok, qk_full + st);
                if (c >= 2 && !w.wait(dec_free + st, before)) break;
                mbar_expect_tx(dec_full + st, sizeof(Decay));
                bulk_load(dec + st, decay + (size_t)c * a.H, sizeof(Decay), dec_full + st);
                if (c >= 2 && !w.wait(v_free + st, before)) break;
                mbar_expect_tx(v_full + st, ATOM);
                load_tile(sm + L_::V + st * ATOM, &f.tv, tile * DVT, h, tok, v_full + st);
            }
        }
    } else if (warp == W_MMA) {
        // ---------------------------------------------------------- MMA (the warp waits, one lane issues)
        for (int c = 0; c < n; ++c) {
            const int st = c & 1;
            if (!w.wait_all(qk_full + st, (c >> 1) & 1)) break;
            tc_fence_after();
            if (elect_one()) {                        // (the scores before were read before P V of the chunk before)
                mma_tiles<4 * KATOMS, false, false, 128>(T_SC, sb + L_::Q + st * 2 * ATOM, sb + L_::K + st * 2 * ATOM, false);
                mma_commit(sc_full);
            }
            if (!w.wait_all(delta_ok, c & 1)) break;
            tc_fence_after();
            if (elect_one()) {
                mma_delta(T_DL, sb + L_::K + st * 2 * ATOM, sb + L_::VP);
                mma_commit(dl_full);
            }
            if (!w.wait_all(qs_ok, c & 1)) break;
            tc_fence_after();
            if (elect_one()) {
                mma_tiles<4 * KATOMS, false, true, 64>(T_OS, sb + L_::Q + st * 2 * ATOM, sb + L_::S, false);
                mma_commit(q_free + st);
            }
            if (!w.wait_all(p_full, c & 1)) break;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t dv = tile_mnmajor(sb + L_::V + st * ATOM);
#pragma unroll 4
                for (int ks = 0; ks < 8; ++ks)
                    mma_bf16_ta(T_OI, T_P + ks * 8, dv + step_mnmajor(ks), idesc_bf16(128, 64, false, true), ks > 0);
                mma_commit(o_full);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // a wait gave up: bounded waits for the copies and MMAs in flight, before their memory goes
        if (threadIdx.x == 0) {
            raise_error(a.err, ERR_TIMEOUT);
            for (int i = 0; i < 2; ++i) {     // whichever phase is under way
                for (uint32_t ph = 0; ph < 2; ++ph) {
                    drain(qk_full + i, ph);
                    drain(v_full + i, ph);
                    drain(dec_full + i, ph);
                }
            }
        }
        if (warp == W_MMA && elect_one()) {
            mbar_init(qs_ok, 1);
            mbar_fence_init();
            mma_commit(qs_ok);
            drain(qs_ok, 0);
        }
        __syncthreads();
    }
    if (warp == W_MMA) tmem_dealloc(tmem, 512);
}

// ================================================================= states
// S <- e^{G_C} S + X^T diag(w) Y chunk by chunk for one (piece of a sequence, head, 64 columns of d_v):
//   forwards   X = K, Y = V, w = e^{G_C - G}:         S at the chunks' starts
//   REV        X = Q, Y = dO, w = scale e^G, from the last chunk on:  the state's gradient at their ends
// TOTALS: from zero, only the piece's final value and decay are kept (what a segment hands on); pieces of a
// sequence's last (REV: first) segment have nobody to hand on to and are left out.  STATES: from the given
// state and the totals of the segments before, every chunk's value is stored.
// The delta MMAs (800 cycles per chunk) hide the two epilogues: prep and state each have their own eight
// warps and a second buffer of weighted rows and of TMEM columns.
template <bool REV, bool TOTALS, int KATOMS>
__global__ void __launch_bounds__(NT_S, 1) linear_state_kernel(const __grid_constant__ StateArgs f)
{
    using L_ = StateSmem;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    const LinArgs &a = f.a;
    const int tiles = (a.dv + DVT - 1) / DVT;
    const int tile = blockIdx.x % tiles, h = (blockIdx.x / tiles) % a.H, u = blockIdx.x / tiles / a.H;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    constexpr int W_MMA = NW_W + NW_S, W_TMA = W_MMA + 1;
    LinPiece pc;
    if (!uniform(lin_piece(a, u, f.piece, pc))) return wait_for_launch();
    const int per = f.sp.seg / f.sp.sub;
    if (TOTALS) {
        const int seg = pc.j / per, last = pc.len > 0 ? (pc.len - 1) / f.sp.seg : 0;
        if (uniform(REV ? seg == 0 : seg == last)) return wait_for_launch();
    }
    const int tok0 = pc.t0 + pc.j * f.piece, len = min(f.piece, pc.len - pc.j * f.piece);
    const int n = uniform((len + C - 1) / C);
    auto chunk = [&](int c) { return REV ? n - 1 - c : c; };
    const int c0 = lin_first_slot(a, pc.s, pc.t0, C) + pc.j * (f.piece / C);   // the piece's first chunk's slot

    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L_::BAR);
    uint64_t *x_full = bar, *x_free = bar + 2, *y_full = bar + 4, *y_free = bar + 6, *vp_full = bar + 8, *dl_full = bar + 10,
             *dl_free = bar + 12, *dec_full = bar + 14, *dec_empty = bar + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L_::CTL);
    int *abort_flag = reinterpret_cast<int *>(sm + L_::CTL + 4);
    const Waits w{abort_flag};
    Decay *dec = reinterpret_cast<Decay *>(sm + L_::DEC);

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(x_full + i, 1);
            mbar_init(x_free + i, 1);
            mbar_init(y_full + i, 1);
            mbar_init(y_free + i, NW_W);
            mbar_init(vp_full + i, NW_W);
            mbar_init(dl_full + i, 1);
            mbar_init(dl_free + i, NW_S);
            mbar_init(dec_full + i, 1);
            mbar_init(dec_empty + i, NW_W + NW_S);
        }
        mbar_fence_init();
        *abort_flag = (sb & 1023u) ? 1 : 0;
        tma_prefetch_desc(&f.tx);
        tma_prefetch_desc(&f.ty);
    }
    if (KATOMS == 1) {
        for (int i = threadIdx.x; i < 2 * (ATOM / 16); i += NT_S)
            *reinterpret_cast<uint4 *>(sm + L_::X + (i / (ATOM / 16)) * 2 * ATOM + ATOM + (i % (ATOM / 16)) * 16) = make_uint4(0, 0, 0, 0);
        fence_async_smem();
    }
    if (warp == W_MMA) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const uint32_t lanes = ((uint32_t)(warp & 3) * 32u) << 16;
    const int row = (warp & 3) * 32 + lane;

    if (warp < NW_W) {
        // ---------------------------------------------------------- weighted rows
        const int vrow = threadIdx.x & 127, vhalf = threadIdx.x >> 7;
        for (int c = 0; c < n; ++c) {
            const int st = c & 1, L = min(C, len - chunk(c) * C);
            if (!w.wait(dec_full + st, (c >> 1) & 1) || !w.wait(y_full + st, (c >> 1) & 1)) break;
            if (c >= 2 && !w.wait(dl_full + st, ((c >> 1) - 1) & 1)) break;   // the MMAs that read this buffer
            uint8_t *vp = sm + L_::VP + st * 3 * ATOM;
            if (vrow < L) {
                weigh_row(sm + L_::Y + st * ATOM, vp, vrow, vhalf,
                          REV ? a.scale * decay_since(dec[st], vrow) : decay_until(dec[st], vrow));
            } else {
#pragma unroll
                for (int k = 0; k < 3; ++k) zero_row(vp + k * ATOM, vrow, vhalf * 4, 4);
                if (w.wait(x_full + st, (c >> 1) & 1)) zero_row(sm + L_::X + (st * 2 + vhalf) * ATOM, vrow, 0, 8);
            }
            fence_async_smem();
            warp_arrive(vp_full + st);
            warp_arrive(y_free + st);
            warp_arrive(dec_empty + st);
        }
    } else if (warp < W_MMA) {
        // ---------------------------------------------------------- the state
        const int half = (warp - NW_W) >> 2;
        const int col = tile * DVT + half * 32;
        const size_t se = ((size_t)pc.s * a.H + h) * a.dk * a.dv;
        f32x2 S[16];
        load_caller(S, !TOTALS && f.first ? f.first + se : nullptr, a.dk, a.dv, row, col);
        if (!TOTALS) {
            const int s0 = lin_first_slot(a, pc.s, pc.t0, f.sp.sub);
            const int lo = REV ? (pc.j + 1) * per : 0, hi = REV ? (pc.len + f.sp.sub - 1) / f.sp.sub : pc.j * per;
            for (int i = lo; i < hi; ++i) {
                const size_t slot = s0 + (REV ? hi - 1 - (i - lo) : i);
                fold_tile(S, f.sp.U + tile_at(slot, a.H, h, tiles, tile), f.sp.dec[slot * a.H + h], row, half);
            }
        }
        Log2 total = {0.f, 0.f};
        bool ok = true, bad = false;
        for (int c = 0; c < n; ++c) {
            const int st = c & 1;
            if (!TOTALS) store_tile(S, f.tiles + tile_at(c0 + chunk(c), a.H, h, tiles, tile), row, half);
            ok = w.wait(dec_full + st, (c >> 1) & 1);
            if (!ok) break;
            const float2 whole = dec[st].whole;
            total = total + dec[st].total;
            bad = bad || whole.x != whole.x;
            warp_arrive(dec_empty + st);
            ok = w.wait(dl_full + st, (c >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            add_delta(S, tmem + st * 192 + lanes + half * 32, whole);
            tc_fence_before();
            warp_arrive(dl_free + st);
        }
        if (ok && TOTALS) {
            store_tile(S, f.tiles + tile_at(u, a.H, h, tiles, tile), row, half);
            if (warp == NW_W && lane == 0 && tile == 0)
                f.dec[(size_t)u * a.H + h] = bad ? make_float2(__int_as_float(0x7fc00000), 0.f) : lin_chunk_decay(total);
        } else if (ok && f.last && (REV ? pc.j == 0 : (long long)(pc.j + 1) * f.piece >= pc.len)) {
            store_caller(S, f.last + se, a.dk, a.dv, row, col);
        }
    } else if (warp == W_TMA) {
        if (lane == 0) {
            wait_for_launch();
            for (int c = 0; c < n; ++c) {
                const int st = c & 1, tok = tok0 + chunk(c) * C;
                if (c + 2 < n) {              // (as in the forward)
                    const int far = tok0 + chunk(c + 2) * C;
                    for (int k = 0; k < KATOMS; ++k) prefetch_tile(&f.tx, k * 64, h, far);
                    prefetch_tile(&f.ty, tile * DVT, h, far);
                }
                const uint32_t before = ((c >> 1) - 1) & 1;
                if (c >= 2 && !w.wait(dec_empty + st, before)) break;
                if (*w.abort_flag) break;
                mbar_expect_tx(dec_full + st, sizeof(Decay));
                bulk_load(dec + st, f.decay + (size_t)(c0 + chunk(c)) * a.H + h, sizeof(Decay), dec_full + st);
                if (c >= 2 && !w.wait(y_free + st, before)) break;      // (read once, early: refilled a good chunk ahead)
                mbar_expect_tx(y_full + st, ATOM);
                load_tile(sm + L_::Y + st * ATOM, &f.ty, tile * DVT, h, tok, y_full + st);
                if (c >= 2 && !w.wait(x_free + st, before)) break;
                mbar_expect_tx(x_full + st, (uint32_t)KATOMS * ATOM);
                for (int k = 0; k < KATOMS; ++k) load_tile(sm + L_::X + (st * 2 + k) * ATOM, &f.tx, k * 64, h, tok, x_full + st);
            }
        }
    } else if (warp == W_MMA) {
        for (int c = 0; c < n; ++c) {
            const int st = c & 1;
            if (!w.wait_all(x_full + st, (c >> 1) & 1) || !w.wait_all(vp_full + st, (c >> 1) & 1)) break;
            if (c >= 2 && !w.wait_all(dl_free + st, ((c >> 1) - 1) & 1)) break;
            tc_fence_after();
            if (elect_one()) {
                mma_delta(tmem + st * 192, sb + L_::X + st * 2 * ATOM, sb + L_::VP + st * 3 * ATOM);
                mma_commit(dl_full + st);
                mma_commit(x_free + st);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        if (threadIdx.x == 0) {
            raise_error(a.err, ERR_TIMEOUT);
            for (int i = 0; i < 2; ++i) {
                for (uint32_t ph = 0; ph < 2; ++ph) {
                    drain(x_full + i, ph);
                    drain(y_full + i, ph);
                    drain(dec_full + i, ph);
                }
            }
        }
        if (warp == W_MMA && elect_one()) {
            mbar_init(dl_free, 1);
            mbar_fence_init();
            mma_commit(dl_free);
            drain(dl_free, 0);
        }
        __syncthreads();
    }
    if (warp == W_MMA) tmem_dealloc(tmem, 512);
}

// ================================================================= host side
namespace {

constexpr int SMS = 148;

size_t round256(size_t x) { return (x + 255) / 256 * 256; }
int tiles_of(const LinArgs &a) { return (a.dv + DVT - 1) / DVT; }
long long slots(const LinArgs &a, int L) { return lin_slots(a.cu != nullptr, a.T, a.ntok, a.nseq, L); }

// Segment and sub-segment lengths.  One CTA per SM, so the SMs take SMS chains (sequence x head x tile) at a
// time: with fewer, each sequence is cut into as many segments as keep every CTA on an SM of its own, none
// shorter than MIN_SEG tokens (a cut costs another launch and a second read of the earlier segments' k and v).
// The totals' own launch takes sub-segments that fill the SMs in turn.
constexpr int MIN_SEG = 8 * C;
void split_of(const LinArgs &a, int *seg, int *sub) {
    const int longest = a.cu ? a.ntok : a.T;
    const long long per = (long long)a.H * tiles_of(a);          // CTAs of one segment of one sequence
    long long parts = a.cu ? SMS / per - (a.nseq - 1) : SMS / (per * (a.nseq > 0 ? a.nseq : 1));
    if (parts > longest / MIN_SEG) parts = longest / MIN_SEG;
    if (parts <= 1) {
        *seg = *sub = (longest + C) / C * C;                     // one segment holds any sequence
        return;
    }
    *seg = (int)(((long long)longest + parts - 1) / parts + C - 1) / C * C;
    // parts - 1 of the parts' tokens are summed up ahead: two sub-segments for each segment where half the SMs or
    // fewer would be at work
    const int halves = 2 * per * (parts - 1) * (a.cu ? 1 : a.nseq) <= SMS && *seg % (2 * C) == 0 ? 2 : 1;
    *sub = *seg / halves;
}
bool is_split(const LinArgs &a, int seg) { return (a.cu ? a.ntok : a.T) > seg; }
size_t totals_bytes(const LinArgs &a, int sub) {
    return round256((size_t)slots(a, sub) * a.H * tiles_of(a) * TILE_FLOATS * 4) + round256((size_t)slots(a, sub) * a.H * 8);
}

size_t decay_bytes(const LinArgs &a) { return round256((size_t)slots(a, C) * a.H * sizeof(Decay)); }
cudaError_t decays(const LinArgs &a, void *ws, cudaStream_t st) {
    const long long n = slots(a, C) * a.H;
    return launch(linear_decay_kernel, dim3((unsigned)((n + 7) / 8)), 256, 0, st, a, static_cast<Decay *>(ws), n);
}

template <typename K>
cudaError_t setup(K kern, size_t smem, int threads) {
    KernelSetup ks;
    return kernel_setup(reinterpret_cast<const void *>(kern), smem, threads, false, &ks);
}

// `early`: right behind the decay launch; the CTAs may then start before it is done (they wait for it before they read
// its records, and touch nothing else that it does)
template <bool REV, bool TOTALS>
cudaError_t states(const StateArgs &f, bool early, cudaStream_t st) {
    auto kern = f.a.dk > 64 ? linear_state_kernel<REV, TOTALS, 2> : linear_state_kernel<REV, TOTALS, 1>;
    const cudaError_t e = setup(kern, StateSmem::TOTAL, NT_S);
    if (e != cudaSuccess) return e;
    return launch_with(early, kern, dim3((unsigned)(slots(f.a, f.piece) * f.a.H * tiles_of(f.a))), NT_S, StateSmem::TOTAL, st, f);
}

// totals of the earlier segments into ws, if the sequences are cut
template <bool REV>
cudaError_t totals(StateArgs f, uint8_t *ws, Split *sp, bool early, cudaStream_t st) {
    split_of(f.a, &sp->seg, &sp->sub);
    sp->U = nullptr;
    sp->dec = nullptr;
    if (!is_split(f.a, sp->seg)) return cudaSuccess;
    float *U = reinterpret_cast<float *>(ws);
    float2 *dec = reinterpret_cast<float2 *>(ws + round256((size_t)slots(f.a, sp->sub) * f.a.H * tiles_of(f.a) * TILE_FLOATS * 4));
    f.sp = *sp;
    f.piece = sp->sub;
    f.tiles = U;
    f.dec = dec;
    f.first = nullptr;
    f.last = nullptr;
    sp->U = U;
    sp->dec = dec;
    return states<REV, true>(f, early, st);
}

}  // namespace

size_t linear_tc_workspace_bytes(const LinArgs &a) {
    int seg, sub;
    split_of(a, &seg, &sub);
    return decay_bytes(a) + (is_split(a, seg) ? totals_bytes(a, sub) : 0);
}

cudaError_t launch_linear_tc(const LinArgs &a, void *workspace, cudaStream_t st) {
    FwdArgs f;
    f.a = a;
    if (!make_token_map(&f.tq, a.q, a.dk, a.H, a.ntok) || !make_token_map(&f.tk, a.k, a.dk, a.H, a.ntok) ||
        !make_token_map(&f.tv, a.v, a.dv, a.H, a.ntok))
        return cudaErrorInvalidValue;
    StateArgs s{};
    s.a = a;
    s.tx = f.tk;
    s.ty = f.tv;
    s.decay = f.decay = static_cast<const Decay *>(workspace);
    cudaError_t e = decays(a, workspace, st);
    if (e == cudaSuccess) e = totals<false>(s, static_cast<uint8_t *>(workspace) + decay_bytes(a), &f.sp, true, st);
    auto kern = a.dk > 64 ? linear_forward_kernel<2> : linear_forward_kernel<1>;
    if (e == cudaSuccess) e = setup(kern, FwdSmem::TOTAL, NT_F);
    if (e != cudaSuccess) return e;
    return launch_with(!is_split(a, f.sp.seg), kern, dim3((unsigned)(slots(a, f.sp.seg) * a.H * tiles_of(a))), NT_F, FwdSmem::TOTAL, st, f);
}

namespace lin {

size_t states_workspace_bytes(const LinArgs &a) {
    int seg, sub;
    split_of(a, &seg, &sub);
    const size_t n = (size_t)slots(a, C) * a.H;
    return decay_bytes(a) + (is_split(a, seg) ? totals_bytes(a, sub) : 0) + 2 * round256(n * tiles_of(a) * TILE_FLOATS * 4) + round256(n * 4);
}

cudaError_t launch_states(const LinBwdArgs &b, void *workspace, States *out, cudaStream_t st) {
    const LinArgs &a = b.a;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    int seg, sub;
    split_of(a, &seg, &sub);
    const size_t n = (size_t)slots(a, C) * a.H, tile_bytes = round256(n * tiles_of(a) * TILE_FLOATS * 4);
    uint8_t *tot = ws + decay_bytes(a);
    float *S = reinterpret_cast<float *>(tot + (is_split(a, seg) ? totals_bytes(a, sub) : 0)), *R = S + tile_bytes / 4;
    out->decay = static_cast<const Decay *>(workspace);
    out->S = S;
    out->R = R;
    out->share = R + tile_bytes / 4;
    cudaError_t e = decays(a, workspace, st);
    if (e != cudaSuccess) return e;
    StateArgs f{};
    f.a = a;
    f.decay = out->decay;
    // forwards: the states at the chunks' starts
    if (!make_token_map(&f.tx, a.k, a.dk, a.H, a.ntok) || !make_token_map(&f.ty, a.v, a.dv, a.H, a.ntok)) return cudaErrorInvalidValue;
    e = totals<false>(f, tot, &f.sp, true, st);
    if (e != cudaSuccess) return e;
    f.piece = f.sp.seg;
    f.tiles = S;
    f.first = a.S0;
    e = states<false, false>(f, !is_split(a, f.sp.seg), st);
    if (e != cudaSuccess) return e;
    // backwards: the state's gradient at their ends
    if (!make_token_map(&f.tx, a.q, a.dk, a.H, a.ntok) || !make_token_map(&f.ty, b.d_o, a.dv, a.H, a.ntok)) return cudaErrorInvalidValue;
    e = totals<true>(f, tot, &f.sp, false, st);
    if (e != cudaSuccess) return e;
    f.piece = f.sp.seg;
    f.tiles = R;
    f.first = b.dS_T;
    f.last = b.dS0;
    return states<true, false>(f, false, st);
}

}  // namespace lin

}  // namespace kdn
