// Linear attention with a decay for each head on the tensor cores (tcgen05, bf16 inputs): forward, and
// the states at the chunks' boundaries that the backward reads.  Chunks of C = 128 tokens; per chunk,
// with the factors of kdn_linear_tc.cuh and S the fp32 state at the chunk's start,
//     O  = scale ((Q K^T o D) V + diag(e^G) Q S),     S' = e^{G_C} S + K^T diag(e^{G_C - G}) V
//
// Forward (linear_forward_kernel): a CTA walks one segment of a sequence for one head and 64 columns of
// d_v, chunk by chunk, with everything but the inputs and outputs on chip.  Warp roles, each a loop over
// the chunks that meets the others at mbarriers:
//   TMA      loads Q, K and the V tile of chunk c + 2 as soon as chunk c's MMAs have read theirs
//   decay    sums the log decays of chunk c + 1, forms its factors
//   MMA      one thread: OS = Q S, delta = K^T V', OI = P V (P from TMEM), scores of c + 1 = Q K^T
//   A (8)    scores (TMEM) -> decayed, masked, bf16 -> P (TMEM, in place); o = scale (OI + e^G OS)
//   B (8)    V' = diag(e^{G_C - G}) V as three bf16 terms; S <- e^{G_C} S + delta in registers (fp32),
//            its bf16 copy for the next Q S
// What bounds it is one pass over q, k, v and o at HBM's rate; the MMAs take about 2050 cycles per chunk
// and tile (scores 512, Q S 384, delta 896 -- its A operand is read from shared memory three times --,
// P V 256), which is about what the chunk's bytes take at an SM's share of the bandwidth.
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

constexpr int NW_A = 8, NW_B = 8;                     // epilogue warps
constexpr int NT_F = (NW_A + NW_B + 3) * 32;          // and the TMA, MMA and decay warps

struct FwdSmem {
    static constexpr int Q = 0, K = Q + 2 * 2 * ATOM, V = K + 2 * 2 * ATOM, VP = V + 2 * ATOM, S = VP + 3 * ATOM,
                         DEC = S + ATOM, META = DEC + 2 * (int)sizeof(Decay), BAR = META + 2 * (int)sizeof(DecayMeta),
                         NBAR = 17, CTL = BAR + NBAR * 8, TOTAL = CTL + 16;
};
static_assert(FwdSmem::TOTAL <= 227 * 1024, "shared memory");

struct StateSmem {
    static constexpr int X = 0, Y = X + 2 * 2 * ATOM, VP = Y + 2 * ATOM, DEC = VP + 2 * 3 * ATOM,
                         META = DEC + 2 * (int)sizeof(Decay), BAR = META + 2 * (int)sizeof(DecayMeta), NBAR = 14,
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
    CUtensorMap tx, ty;
};

// 32 columns of row `row` of a state: from the caller's [dk, dv] layout (zero outside it) ...
__device__ __forceinline__ void load_caller(float (&S)[32], const float *src, int dk, int dv, int row, int col) {
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
        const float4 x = src && row < dk && col < dv ? __ldg(reinterpret_cast<const float4 *>(src + (size_t)row * dv + col + j))
                                                     : make_float4(0.f, 0.f, 0.f, 0.f);
        S[j] = x.x; S[j + 1] = x.y; S[j + 2] = x.z; S[j + 3] = x.w;
    }
}
__device__ __forceinline__ void store_caller(const float (&S)[32], float *dst, int dk, int dv, int row, int col) {
    if (row >= dk || col >= dv) return;
#pragma unroll
    for (int j = 0; j < 32; j += 4)
        *reinterpret_cast<float4 *>(dst + (size_t)row * dv + col + j) = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
}
// ... and to a workspace tile
__device__ __forceinline__ void store_tile(const float (&S)[32], float *tile, int row, int half) {
#pragma unroll
    for (int q = 0; q < 8; ++q)
        *reinterpret_cast<float4 *>(tile + ((half * 8 + q) * 128 + row) * 4) = make_float4(S[4 * q], S[4 * q + 1], S[4 * q + 2], S[4 * q + 3]);
}
// S <- decay S + the tile of a sub-segment
__device__ __forceinline__ void fold_tile(float (&S)[32], const float *tile, float2 dec, int row, int half) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const float4 x = __ldg(reinterpret_cast<const float4 *>(tile + ((half * 8 + q) * 128 + row) * 4));
        S[4 * q] = lin_carry(dec, S[4 * q], x.x);
        S[4 * q + 1] = lin_carry(dec, S[4 * q + 1], x.y);
        S[4 * q + 2] = lin_carry(dec, S[4 * q + 2], x.z);
        S[4 * q + 3] = lin_carry(dec, S[4 * q + 3], x.w);
    }
}
__device__ __forceinline__ void add_delta(float (&S)[32], uint32_t d, float2 dec) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        float x[16], y[16];
        tmem_ld16(d + p * 16, x);
        tmem_ld16(d + 64 + p * 16, y);
#pragma unroll
        for (int j = 0; j < 16; ++j) S[p * 16 + j] = lin_carry(dec, S[p * 16 + j], x[j] + y[j]);
    }
}

// meeting of the two warps of a quadrant: whether both came with `ok`, the same answer for both (a warp
// whose wait gave up still comes, so that the other is not left behind)
__device__ __forceinline__ bool both(int id, bool ok) {
    int r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.and.pred q, %2, 64, p;\n selp.b32 %0, 1, 0, q;\n}"
                 : "=r"(r) : "r"((int)ok), "r"(id) : "memory");
    return r != 0;
}

// thread 0 of the TMA warp: a [128 tokens][64 channels] tile as two boxes of 64 tokens
__device__ __forceinline__ void load_tile(uint8_t *dst, const CUtensorMap *m, int c0, int h, int tok, uint64_t *bar) {
    tma_load_3d(dst, m, c0, h, tok, bar);
    tma_load_3d(dst + ATOM / 2, m, c0, h, tok + 64, bar);
}

// after a wait gave up: one more bounded wait for a barrier that copies or MMAs in flight still arrive on
__device__ __noinline__ void drain(uint64_t *bar, uint32_t parity) { mbar_wait(bar, parity, 100000000ll); }

}  // namespace

// ================================================================= forward
__global__ void __launch_bounds__(NT_F, 1) linear_forward_kernel(const __grid_constant__ FwdArgs f)
{
    using L_ = FwdSmem;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    const LinArgs &a = f.a;
    const int tiles = (a.dv + DVT - 1) / DVT;
    const int tile = blockIdx.x % tiles, h = (blockIdx.x / tiles) % a.H, u = blockIdx.x / tiles / a.H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    LinPiece pc;
    if (!lin_piece(a, u, f.sp.seg, pc)) return;
    const int tok0 = pc.t0 + pc.j * f.sp.seg, len = min(f.sp.seg, pc.len - pc.j * f.sp.seg);
    const int n = (len + C - 1) / C;
    const int katoms = a.dk > 64 ? 2 : 1;

    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L_::BAR);
    uint64_t *full = bar, *empty = bar + 2, *sc_full = bar + 4, *p_full = bar + 6, *dec_full = bar + 8, *dec_empty = bar + 10,
             *o_full = bar + 12, *o_free = bar + 13, *dl_full = bar + 14, *vp_full = bar + 15, *s_full = bar + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L_::CTL);
    int *abort_flag = reinterpret_cast<int *>(sm + L_::CTL + 4);
    const Waits w{abort_flag};
    Decay *dec = reinterpret_cast<Decay *>(sm + L_::DEC);
    DecayMeta *meta = reinterpret_cast<DecayMeta *>(sm + L_::META);

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
            mbar_init(sc_full + i, 1);
            mbar_init(p_full + i, NW_A);
            mbar_init(dec_full + i, 1);
            mbar_init(dec_empty + i, NW_A + NW_B);
        }
        mbar_init(o_full, 1);
        mbar_init(o_free, NW_A);
        mbar_init(dl_full, 1);
        mbar_init(vp_full, NW_B);
        mbar_init(s_full, NW_B);
        mbar_fence_init();
        *abort_flag = (sb & 1023u) ? 1 : 0;   // the swizzled tiles need 1 KB alignment
        tma_prefetch_desc(&f.tq);
        tma_prefetch_desc(&f.tk);
        tma_prefetch_desc(&f.tv);
    }
    if (katoms == 1) {                        // channels 64..127 of K and Q: zeros, never written again
        for (int i = threadIdx.x; i < 4 * (ATOM / 16); i += NT_F) {
            const int t = i / (ATOM / 16);
            *reinterpret_cast<uint4 *>(sm + ((t & 1) ? L_::K : L_::Q) + (t >> 1) * 2 * ATOM + ATOM + (i % (ATOM / 16)) * 16) =
                make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
    }
    if (warp == NW_A + NW_B + 1) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t T_SC = tmem, T_OI = tmem + 256, T_OS = tmem + 320, T_DL = tmem + 384;
    const uint32_t lanes = ((uint32_t)(warp & 3) * 32u) << 16;
    const int row = (warp & 3) * 32 + lane;

    if (warp < NW_A) {
        // ---------------------------------------------------------- A: scores -> P, and the outputs
        const int half = warp >> 2, q4 = warp & 3;
        float since[2];                       // 2^{G_t} of the row, for the chunk's output
        bool fact[2];
        auto scores = [&](int c) -> bool {
            const int st = c & 1;
            bool ok = w.wait(dec_full + st, (c >> 1) & 1);
            const Decay &d = dec[st];
            const bool factored = meta[st].factored;
            fact[st] = factored;
            since[st] = decay_since(d, factored, row);
            ok = ok && w.wait(sc_full + st, (c >> 1) & 1);
            tc_fence_after();
            // column blocks of 32: this warp takes blocks half and half + 2; blocks above the diagonal are zero
            uint32_t p[2][16];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int blk = half + 2 * i;
                if (blk > q4) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) p[i][j] = 0u;
                    continue;
                }
                float x[32];
                tmem_ld32(T_SC + st * 128 + lanes + blk * 32, x);
                if (factored) {
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 b = *reinterpret_cast<const float4 *>(d.b + blk * 32 + j);
                        x[j] *= b.x; x[j + 1] *= b.y; x[j + 2] *= b.z; x[j + 3] *= b.w;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[j] *= blk * 32 + j <= row ? decay_pair(d, row, blk * 32 + j) : 0.f;
                }
                if (blk == q4) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[j] = j <= lane ? x[j] : 0.f;
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) p[i][j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
            }
            // P takes the place of the scores' first 64 columns: the quadrant's other warp has read them too
            if (!both(1 + q4, ok)) return false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float y[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) y[j] = __uint_as_float(p[i][j]);
                tmem_st16(T_SC + st * 128 + lanes + (half + 2 * i) * 16, y);
            }
            tc_fence_before();
            warp_arrive(p_full + st);
            warp_arrive(dec_empty + st);
            return true;
        };
        auto output = [&](int c) -> bool {
            const int st = c & 1, L = min(C, len - c * C), col = tile * DVT + half * 32;
            if (!w.wait(o_full, c & 1)) return false;
            tc_fence_after();
            // factored: the row's 2^{G_t} is common to both parts (P holds the columns' 2^{-G_s})
            const float fs = a.scale * since[st], fi = fact[st] ? fs : a.scale;
            bf16 *o = static_cast<bf16 *>(a.o) + ((size_t)(tok0 + c * C + row) * a.H + h) * a.dv + col;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float x[16], y[16];
                tmem_ld16(T_OI + lanes + half * 32 + p * 16, x);
                tmem_ld16(T_OS + lanes + half * 32 + p * 16, y);
                if (p == 1) {
                    tc_fence_before();
                    warp_arrive(o_free);
                }
                if (row < L && col < a.dv) {
#pragma unroll
                    for (int j = 0; j < 16; j += 8) {
                        uint32_t z[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            z[i] = pack_bf16x2(fmaf(fi, x[j + 2 * i], fs * y[j + 2 * i]), fmaf(fi, x[j + 2 * i + 1], fs * y[j + 2 * i + 1]));
                        *reinterpret_cast<uint4 *>(o + p * 16 + j) = make_uint4(z[0], z[1], z[2], z[3]);
                    }
                }
            }
            return true;
        };
        bool ok = n == 0 || scores(0);
        for (int c = 0; c < n && ok; ++c) {
            if (c + 1 < n) ok = scores(c + 1);
            ok = ok && output(c);
        }
    } else if (warp < NW_A + NW_B) {
        // ---------------------------------------------------------- B: weighted rows of V, the state
        const int half = (warp - NW_A) >> 2;
        const int vrow = (threadIdx.x - NW_A * 32) & 127, vhalf = (threadIdx.x - NW_A * 32) >> 7;
        const int col = tile * DVT + half * 32;
        const size_t se = ((size_t)pc.s * a.H + h) * a.dk * a.dv;
        float S[32];
        load_caller(S, a.S0 ? a.S0 + se : nullptr, a.dk, a.dv, row, col);
        const int before = pc.j * (f.sp.seg / f.sp.sub), s0 = lin_first_slot(a, pc.s, pc.t0, f.sp.sub);
        for (int i = 0; i < before; ++i)
            fold_tile(S, f.sp.U + tile_at(s0 + i, a.H, h, tiles, tile), f.sp.dec[(size_t)(s0 + i) * a.H + h], row, half);
        auto publish = [&]() {                // the bf16 copy that Q S reads
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t z[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = pack_bf16x2(S[j * 8 + 2 * i], S[j * 8 + 2 * i + 1]);
                *reinterpret_cast<uint4 *>(sm + L_::S + swz(row, (half * 4 + j) * 16)) = make_uint4(z[0], z[1], z[2], z[3]);
            }
            fence_async_smem();
            warp_arrive(s_full);
        };
        if (n > 0) publish();
        bool ok = true;
        for (int c = 0; c < n; ++c) {
            const int st = c & 1, L = min(C, len - c * C);
            ok = w.wait(dec_full + st, (c >> 1) & 1) && w.wait(full + st, (c >> 1) & 1);
            if (!ok) break;
            const float2 whole = meta[st].whole;
            if (vrow < L) {
                weigh_row(sm + L_::V + st * ATOM, sm + L_::VP, vrow, vhalf, decay_until(dec[st], meta[st], vrow));
            } else {                          // rows behind the sequence's end: zeros in every operand that is summed over rows
#pragma unroll
                for (int k = 0; k < 3; ++k) zero_row(sm + L_::VP + k * ATOM, vrow, vhalf * 4, 4);
                zero_row(sm + L_::V + st * ATOM, vrow, vhalf * 4, 4);
                zero_row(sm + L_::K + (st * 2 + vhalf) * ATOM, vrow, 0, 8);
            }
            fence_async_smem();
            warp_arrive(vp_full);
            warp_arrive(dec_empty + st);
            ok = w.wait(dl_full, c & 1);
            if (!ok) break;
            tc_fence_after();
            add_delta(S, T_DL + lanes + half * 32, whole);
            tc_fence_before();
            if (c + 1 < n) publish();
        }
        if (ok && a.S_out && (long long)(pc.j + 1) * f.sp.seg >= pc.len) store_caller(S, a.S_out + se, a.dk, a.dv, row, col);
    } else if (warp == NW_A + NW_B) {
        // ---------------------------------------------------------- TMA
        if (lane == 0) {
            const uint32_t bytes = (uint32_t)(2 * katoms + 1) * ATOM;
            for (int c = 0; c < n; ++c) {
                const int st = c & 1, tok = tok0 + c * C;
                if (c >= 2 && !w.wait(empty + st, ((c >> 1) - 1) & 1)) break;
                if (*w.abort_flag) break;
                mbar_expect_tx(full + st, bytes);
                for (int k = 0; k < katoms; ++k) {
                    load_tile(sm + L_::Q + (st * 2 + k) * ATOM, &f.tq, k * 64, h, tok, full + st);
                    load_tile(sm + L_::K + (st * 2 + k) * ATOM, &f.tk, k * 64, h, tok, full + st);
                }
                load_tile(sm + L_::V + st * ATOM, &f.tv, tile * DVT, h, tok, full + st);
            }
        }
    } else if (warp == NW_A + NW_B + 1) {
        // ---------------------------------------------------------- MMA
        if (lane == 0) {
            constexpr uint32_t ID_QK = idesc_bf16(128, 128, false, false), ID_QS = idesc_bf16(128, 64, false, true);
            auto qk = [&](int c) -> bool {
                const int st = c & 1;
                if (!w.wait(full + st, (c >> 1) & 1)) return false;
                tc_fence_after();
                for (int ks = 0; ks < 4 * katoms; ++ks)
                    mma_bf16(T_SC + st * 128, kmajor(sb + L_::Q + st * 2 * ATOM, ks), kmajor(sb + L_::K + st * 2 * ATOM, ks), ID_QK, ks > 0);
                mma_commit(sc_full + st);
                return true;
            };
            bool ok = n == 0 || qk(0);
            for (int c = 0; c < n && ok; ++c) {
                const int st = c & 1;
                ok = w.wait(s_full, c & 1) && (c == 0 || w.wait(o_free, (c - 1) & 1));
                if (!ok) break;
                tc_fence_after();
                for (int ks = 0; ks < 4 * katoms; ++ks)
                    mma_bf16(T_OS, kmajor(sb + L_::Q + st * 2 * ATOM, ks), mnmajor(sb + L_::S, ks), ID_QS, ks > 0);
                ok = w.wait(vp_full, c & 1);
                if (!ok) break;
                tc_fence_after();
                mma_delta(T_DL, sb + L_::K + st * 2 * ATOM, sb + L_::VP);
                mma_commit(dl_full);
                ok = w.wait(p_full + st, (c >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                for (int ks = 0; ks < 8; ++ks)
                    mma_bf16_ta(T_OI, T_SC + st * 128 + ks * 8, mnmajor(sb + L_::V + st * ATOM, ks), ID_QS, ks > 0);
                mma_commit(o_full);
                mma_commit(empty + st);
                if (c + 1 < n) ok = qk(c + 1);
            }
        }
    } else {
        // ---------------------------------------------------------- decay
        double x[4];
        if (n > 0) decay_fetch(a, tok0, min(C, len), h, x);
        for (int c = 0; c < n; ++c) {
            const int st = c & 1;
            if (c >= 2 && !w.wait(dec_empty + st, ((c >> 1) - 1) & 1)) break;
            decay_write(x, dec + st, meta + st);
            warp_arrive(dec_full + st);
            if (c + 1 < n) decay_fetch(a, tok0 + (c + 1) * C, min(C, len - (c + 1) * C), h, x);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // a wait gave up: bounded waits for the copies and MMAs in flight, before their memory goes
        if (threadIdx.x == 0) {
            raise_error(a.err, ERR_TIMEOUT);
            for (int i = 0; i < 2; ++i) drain(full + i, 0);
            for (int i = 0; i < 2; ++i) drain(full + i, 1);
        }
        if (warp == NW_A + NW_B + 1 && lane == 0) {
            mbar_init(o_free, 1);
            mbar_fence_init();
            mma_commit(o_free);
            drain(o_free, 0);
        }
        __syncthreads();
    }
    if (warp == NW_A + NW_B + 1) tmem_dealloc(tmem, 512);
}

// ================================================================= states
// S <- e^{G_C} S + X^T diag(w) Y chunk by chunk for one (piece of a sequence, head, 64 columns of d_v):
//   forwards   X = K, Y = V, w = e^{G_C - G}:         S at the chunks' starts
//   REV        X = Q, Y = dO, w = scale e^G, from the last chunk on:  the state's gradient at their ends
// TOTALS: from zero, only the piece's final value and decay are kept (what a segment hands on); pieces of a
// sequence's last (REV: first) segment have nobody to hand on to and are left out.  STATES: from the given
// state and the totals of the segments before, every chunk's value is stored.
// The delta MMAs (896 cycles per chunk) hide the two epilogues: prep and state each have their own eight
// warps and a second buffer of weighted rows and of TMEM columns.
template <bool REV, bool TOTALS>
__global__ void __launch_bounds__(NT_F, 1) linear_state_kernel(const __grid_constant__ StateArgs f)
{
    using L_ = StateSmem;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    const LinArgs &a = f.a;
    const int tiles = (a.dv + DVT - 1) / DVT;
    const int tile = blockIdx.x % tiles, h = (blockIdx.x / tiles) % a.H, u = blockIdx.x / tiles / a.H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    LinPiece pc;
    if (!lin_piece(a, u, f.piece, pc)) return;
    const int per = f.sp.seg / f.sp.sub;
    if (TOTALS) {
        const int seg = pc.j / per, last = pc.len > 0 ? (pc.len - 1) / f.sp.seg : 0;
        if (REV ? seg == 0 : seg == last) return;
    }
    const int tok0 = pc.t0 + pc.j * f.piece, len = min(f.piece, pc.len - pc.j * f.piece);
    const int n = (len + C - 1) / C;
    const int katoms = a.dk > 64 ? 2 : 1;
    auto chunk = [&](int c) { return REV ? n - 1 - c : c; };

    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L_::BAR);
    uint64_t *full = bar, *empty = bar + 2, *vp_full = bar + 4, *dl_full = bar + 6, *dl_free = bar + 8, *dec_full = bar + 10,
             *dec_empty = bar + 12;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L_::CTL);
    int *abort_flag = reinterpret_cast<int *>(sm + L_::CTL + 4);
    const Waits w{abort_flag};
    Decay *dec = reinterpret_cast<Decay *>(sm + L_::DEC);
    DecayMeta *meta = reinterpret_cast<DecayMeta *>(sm + L_::META);

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
            mbar_init(vp_full + i, NW_A);
            mbar_init(dl_full + i, 1);
            mbar_init(dl_free + i, NW_B);
            mbar_init(dec_full + i, 1);
            mbar_init(dec_empty + i, NW_A + NW_B);
        }
        mbar_fence_init();
        *abort_flag = (sb & 1023u) ? 1 : 0;
        tma_prefetch_desc(&f.tx);
        tma_prefetch_desc(&f.ty);
    }
    if (katoms == 1) {
        for (int i = threadIdx.x; i < 2 * (ATOM / 16); i += NT_F)
            *reinterpret_cast<uint4 *>(sm + L_::X + (i / (ATOM / 16)) * 2 * ATOM + ATOM + (i % (ATOM / 16)) * 16) = make_uint4(0, 0, 0, 0);
        fence_async_smem();
    }
    if (warp == NW_A + NW_B + 1) tmem_alloc(tmem_slot, 256);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t lanes = ((uint32_t)(warp & 3) * 32u) << 16;
    const int row = (warp & 3) * 32 + lane;

    if (warp < NW_A) {
        // ---------------------------------------------------------- weighted rows
        const int vrow = threadIdx.x & 127, vhalf = threadIdx.x >> 7;
        for (int c = 0; c < n; ++c) {
            const int st = c & 1, L = min(C, len - chunk(c) * C);
            if (!w.wait(dec_full + st, (c >> 1) & 1) || !w.wait(full + st, (c >> 1) & 1)) break;
            if (c >= 2 && !w.wait(dl_full + st, ((c >> 1) - 1) & 1)) break;   // the MMAs that read this buffer
            uint8_t *vp = sm + L_::VP + st * 3 * ATOM;
            if (vrow < L) {
                weigh_row(sm + L_::Y + st * ATOM, vp, vrow, vhalf,
                          REV ? a.scale * decay_since(dec[st], meta[st].factored, vrow) : decay_until(dec[st], meta[st], vrow));
            } else {
#pragma unroll
                for (int k = 0; k < 3; ++k) zero_row(vp + k * ATOM, vrow, vhalf * 4, 4);
                zero_row(sm + L_::X + (st * 2 + vhalf) * ATOM, vrow, 0, 8);
            }
            fence_async_smem();
            warp_arrive(vp_full + st);
            warp_arrive(dec_empty + st);
        }
    } else if (warp < NW_A + NW_B) {
        // ---------------------------------------------------------- the state
        const int half = (warp - NW_A) >> 2;
        const int col = tile * DVT + half * 32;
        const size_t se = ((size_t)pc.s * a.H + h) * a.dk * a.dv;
        float S[32];
        load_caller(S, !TOTALS && f.first ? f.first + se : nullptr, a.dk, a.dv, row, col);
        if (!TOTALS) {
            const int s0 = lin_first_slot(a, pc.s, pc.t0, f.sp.sub);
            const int lo = REV ? (pc.j + 1) * per : 0, hi = REV ? (pc.len + f.sp.sub - 1) / f.sp.sub : pc.j * per;
            for (int i = lo; i < hi; ++i) {
                const size_t slot = s0 + (REV ? hi - 1 - (i - lo) : i);
                fold_tile(S, f.sp.U + tile_at(slot, a.H, h, tiles, tile), f.sp.dec[slot * a.H + h], row, half);
            }
        }
        const int c0 = lin_first_slot(a, pc.s, pc.t0, C) + pc.j * (f.piece / C);
        double log_whole = 0.0;
        bool ok = true;
        for (int c = 0; c < n; ++c) {
            const int st = c & 1;
            if (!TOTALS) store_tile(S, f.tiles + tile_at(c0 + chunk(c), a.H, h, tiles, tile), row, half);
            ok = w.wait(dec_full + st, (c >> 1) & 1);
            if (!ok) break;
            const float2 whole = meta[st].whole;
            warp_arrive(dec_empty + st);
            if (TOTALS && warp == NW_A) {     // the piece's decay: the product of the chunks', in fp64
                const double x = (double)whole.x + (double)whole.y;
                log_whole = c == 0 ? x : log_whole * x;
            }
            ok = w.wait(dl_full + st, (c >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            add_delta(S, tmem + st * 128 + lanes + half * 32, whole);
            tc_fence_before();
            warp_arrive(dl_free + st);
        }
        if (ok && TOTALS) {
            store_tile(S, f.tiles + tile_at(u, a.H, h, tiles, tile), row, half);
            if (warp == NW_A && lane == 0 && tile == 0) {
                const float hi = (float)log_whole;
                f.dec[(size_t)u * a.H + h] = make_float2(hi, (float)(log_whole - (double)hi));
            }
        } else if (ok && f.last && (REV ? pc.j == 0 : (long long)(pc.j + 1) * f.piece >= pc.len)) {
            store_caller(S, f.last + se, a.dk, a.dv, row, col);
        }
    } else if (warp == NW_A + NW_B) {
        if (lane == 0) {
            for (int c = 0; c < n; ++c) {
                const int st = c & 1, tok = tok0 + chunk(c) * C;
                if (c >= 2 && !w.wait(empty + st, ((c >> 1) - 1) & 1)) break;
                if (*w.abort_flag) break;
                mbar_expect_tx(full + st, (uint32_t)(katoms + 1) * ATOM);
                for (int k = 0; k < katoms; ++k) load_tile(sm + L_::X + (st * 2 + k) * ATOM, &f.tx, k * 64, h, tok, full + st);
                load_tile(sm + L_::Y + st * ATOM, &f.ty, tile * DVT, h, tok, full + st);
            }
        }
    } else if (warp == NW_A + NW_B + 1) {
        if (lane == 0) {
            for (int c = 0; c < n; ++c) {
                const int st = c & 1;
                if (!w.wait(full + st, (c >> 1) & 1) || !w.wait(vp_full + st, (c >> 1) & 1)) break;
                if (c >= 2 && !w.wait(dl_free + st, ((c >> 1) - 1) & 1)) break;
                tc_fence_after();
                mma_delta(tmem + st * 128, sb + L_::X + st * 2 * ATOM, sb + L_::VP + st * 3 * ATOM);
                mma_commit(dl_full + st);
                mma_commit(empty + st);
            }
        }
    } else {
        double x[4];
        if (n > 0) decay_fetch(a, tok0 + chunk(0) * C, min(C, len - chunk(0) * C), h, x);
        for (int c = 0; c < n; ++c) {
            const int st = c & 1;
            if (c >= 2 && !w.wait(dec_empty + st, ((c >> 1) - 1) & 1)) break;
            decay_write(x, dec + st, meta + st);
            warp_arrive(dec_full + st);
            if (c + 1 < n) decay_fetch(a, tok0 + chunk(c + 1) * C, min(C, len - chunk(c + 1) * C), h, x);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        if (threadIdx.x == 0) {
            raise_error(a.err, ERR_TIMEOUT);
            for (int i = 0; i < 2; ++i) drain(full + i, 0);
            for (int i = 0; i < 2; ++i) drain(full + i, 1);
        }
        if (warp == NW_A + NW_B + 1 && lane == 0) {
            mbar_init(dl_free, 1);
            mbar_fence_init();
            mma_commit(dl_free);
            drain(dl_free, 0);
        }
        __syncthreads();
    }
    if (warp == NW_A + NW_B + 1) tmem_dealloc(tmem, 256);
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

template <typename K>
cudaError_t setup(K kern, size_t smem) {
    KernelSetup ks;
    return kernel_setup(reinterpret_cast<const void *>(kern), smem, NT_F, false, &ks);
}

template <bool REV, bool TOTALS>
cudaError_t states(const StateArgs &f, cudaStream_t st) {
    auto kern = linear_state_kernel<REV, TOTALS>;
    const cudaError_t e = setup(kern, StateSmem::TOTAL);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)(slots(f.a, f.piece) * f.a.H * tiles_of(f.a)), NT_F, StateSmem::TOTAL, st>>>(f);
    return cudaGetLastError();
}

// totals of the earlier segments into ws, if the sequences are cut
template <bool REV>
cudaError_t totals(StateArgs f, uint8_t *ws, Split *sp, cudaStream_t st) {
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
    return states<REV, true>(f, st);
}

}  // namespace

size_t linear_tc_workspace_bytes(const LinArgs &a) {
    int seg, sub;
    split_of(a, &seg, &sub);
    return is_split(a, seg) ? totals_bytes(a, sub) : 0;
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
    cudaError_t e = totals<false>(s, static_cast<uint8_t *>(workspace), &f.sp, st);
    if (e == cudaSuccess) e = setup(linear_forward_kernel, FwdSmem::TOTAL);
    if (e != cudaSuccess) return e;
    linear_forward_kernel<<<(unsigned)(slots(a, f.sp.seg) * a.H * tiles_of(a)), NT_F, FwdSmem::TOTAL, st>>>(f);
    return cudaGetLastError();
}

}  // namespace kdn
