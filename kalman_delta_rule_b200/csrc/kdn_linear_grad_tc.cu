// Backward of linear attention with a decay for each head on the tensor cores (tcgen05, bf16 inputs).
// The states S at the chunks' starts and the state gradients R at their ends come from two walks over the
// sequence (kdn_linear_tc.cu); everything else is parallel over (chunk, head), one CTA each.  With
// a_t = scale e^{G_t}, w_t = e^{G_C - G_t}, P = scale Q K^T o D, dP = dO V^T, dA = scale dP o D, Z = P o dP:
//     dQ = dA K + a (dO S^T),   dK = dA^T Q + w (V R^T),   dV = P^T dO + w (K R)
//     dg_t = sum_{i >= t, j < t} Z_ij + sum_{s >= t} q_s.(a dO S^T)_s + sum_{s < t} k_s.(w V R^T)_s + e^{G_C} <S, R>
// (no term is divided by a decay, and every sum is formed from its own terms: as a difference of larger sums -- rows of Z less
// columns of Z, say -- a reset's gradient would be their roundings instead of zero).
//
// TMEM holds four accumulators of 128 columns: the scores, dP, dO S^T and V R^T.  The last two are scaled
// by their rows' decays in place, and dA K and dA^T Q are added to them; the first two are replaced by the
// two parts of dV.  Rounding: P and dA, and R in K R, are bf16 (dq, dk and dv are); S and R enter the
// products that dg is summed from as three bf16 terms, so dg keeps fp32's accuracy.
// Per chunk and head at d = 128: 12 products of 128 x 128 x 128 (6100 cycles of MMA), 256 KB in (half of it the two fp32
// states) and 96 KB out, 15000 cycles at an SM's share of HBM.  Its operands fill shared memory, so one CTA per SM walks its
// phases one after the other -- the states' terms, P and dA, the decay's sums, the outputs -- in about 29000: 220 us for B4 H16
// T4096 (tensor pipe 22% active, DRAM 39%), behind 58 to 61 and 60 to 63 us for the two walks; a call takes 344 to 360.
#include "kdn_launch.h"
#include "kdn_linear_tc.cuh"

namespace kdn {

using namespace lin;

namespace {

constexpr int NT = 512;
constexpr int SMS = 148;

struct Smem {
    static constexpr int Q = 0, K = Q + 2 * ATOM, DO = K + 2 * ATOM, V = DO + 2 * ATOM, ST = V + 2 * ATOM, R1 = ST + 3 * ATOM,
                         DEC = R1 + 2 * ATOM, SUM = DEC + (int)sizeof(Decay), CTL = SUM + (4 * 4 * C + 32) * 4, TOTAL = CTL + 48;
    static constexpr int P = ST, DA = V;      // once the states' terms and V have been used
    static constexpr int R2 = Q;              // the second and third terms of R, between the scores and the second load of q
};
static_assert(Smem::TOTAL <= 227 * 1024, "shared memory");

struct GradArgs {
    LinBwdArgs b;
    States s;
    CUtensorMap tq, tk, tv, to;
};

// sums over the 32 lanes of 16 values each: lane l returns the sum of value l / 2
__device__ __forceinline__ float sum16(float (&x)[16], int lane) {
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) {
        const bool up = lane & (2 * w);       // lanes of the upper half keep the upper values
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float send = up ? x[i] : x[i + w], keep = up ? x[i + w] : x[i];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, send, 2 * w);
        }
    }
    return x[0] + __shfl_xor_sync(0xffffffffu, x[0], 1);
}

}  // namespace

template <int KATOMS>       // 64-channel tiles of q and k in use
__global__ void __launch_bounds__(NT, 1) linear_grad_tc_kernel(const __grid_constant__ GradArgs f)
{
    using L_ = Smem;
    constexpr int NK = 64 * KATOMS;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    const LinArgs &a = f.b.a;
    const int u = blockIdx.x / a.H, h = blockIdx.x % a.H;
    LinPiece pc;
    if (!uniform(lin_piece(a, u, C, pc) && pc.len > 0)) return;
    const int tok = pc.t0 + pc.j * C, L = min(C, pc.len - pc.j * C);
    const int tiles = (a.dv + DVT - 1) / DVT, nt = min(tiles, 2);        // tiles of d_v, of a half that is resident
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, q4 = warp & 3, cg = warp >> 2;
    const int row = q4 * 32 + lane;
    const uint32_t lanes = ((uint32_t)q4 * 32u) << 16;

    uint64_t *bar_tma = reinterpret_cast<uint64_t *>(sm + L_::CTL), *bar_a = bar_tma + 1, *bar_b = bar_tma + 2, *bar_c = bar_tma + 3;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar_tma + 4);
    int *abort_flag = reinterpret_cast<int *>(tmem_slot + 1);
    const Waits w{abort_flag};
    const Decay &d = *reinterpret_cast<const Decay *>(sm + L_::DEC);
    float *zr = reinterpret_cast<float *>(sm + L_::SUM), *zc = zr + 4 * C, *xi = zc + 4 * C, *yi = xi + 4 * C, *sr_w = yi + 4 * C;

    auto load = [&](const CUtensorMap *m, int region, int c0, int n) {   // (thread 0)
        for (int t = 0; t < n; ++t) load_tile(sm + region + t * ATOM, m, c0 + t * 64, h, tok, bar_tma);
    };
    if (threadIdx.x == 0) {
        mbar_init(bar_tma, 1);
        mbar_init(bar_a, 1);
        mbar_init(bar_b, 1);
        mbar_init(bar_c, 1);
        mbar_fence_init();
        *abort_flag = (sb & 1023u) ? 1 : 0;
        mbar_expect_tx(bar_tma, (uint32_t)(2 * KATOMS + 2 * nt) * ATOM + (uint32_t)sizeof(Decay));
        bulk_load(sm + L_::DEC, f.s.decay + (size_t)u * a.H + h, sizeof(Decay), bar_tma);
        load(&f.tq, L_::Q, 0, KATOMS);
        load(&f.tk, L_::K, 0, KATOMS);
        load(&f.to, L_::DO, 0, nt);
        load(&f.tv, L_::V, 0, nt);
    }
    // 16 columns of a state tile's row in registers
    auto fetch = [&](const float *base, int t, float4 (&x)[4]) {
        const float *tile = base + tile_at(u, a.H, h, tiles, t);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __ldg(reinterpret_cast<const float4 *>(tile + ((cg * 4 + j) * 128 + row) * 4));
    };
    float4 S[4], R[4];
    fetch(f.s.S, 0, S);
    fetch(f.s.R, 0, R);
    if (warp == 0) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const uint32_t T_SC = tmem, T_DP = tmem + 128, T_DQ = tmem + 256, T_DK = tmem + 384;
    // every thread takes every wait and every barrier; after a wait that gave up the rest give up at once
    uint32_t ph_tma = 0, ph_a = 0, ph_b = 0;  // MMAs are committed to two barriers in turn
    auto wait_tma = [&]() { w.wait(bar_tma, ph_tma); ph_tma ^= 1; };
    auto wait_a = [&]() { w.wait(bar_a, ph_a); ph_a ^= 1; tc_fence_after(); };
    auto wait_b = [&]() { w.wait(bar_b, ph_b); ph_b ^= 1; tc_fence_after(); };
    auto publish = [&]() {                    // this thread's shared-memory and TMEM work, before the next MMAs
        fence_async_smem();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    };
    // 16 columns of a state tile's row, as terms in shared memory
    auto terms = [&](const float4 (&x)[4], int p0, int p1, int p2) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t o[3][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 y = x[2 * j + (i >> 1)];
                uint32_t t[3];
                split3(i & 1 ? pk2(y.z, y.w) : pk2(y.x, y.y), t);
                o[0][i] = t[0]; o[1][i] = t[1]; o[2][i] = t[2];
            }
            const uint32_t off = swz(row, (cg * 2 + j) * 16);
            *reinterpret_cast<uint4 *>(sm + p0 + off) = make_uint4(o[0][0], o[0][1], o[0][2], o[0][3]);
            *reinterpret_cast<uint4 *>(sm + p1 + off) = make_uint4(o[1][0], o[1][1], o[1][2], o[1][3]);
            *reinterpret_cast<uint4 *>(sm + p2 + off) = make_uint4(o[2][0], o[2][1], o[2][2], o[2][3]);
        }
    };
    auto zero_tail = [&](int tile, int n) {   // rows behind the sequence's end
        if (L < C && row >= L)
            for (int t = 0; t < n; ++t) zero_row(sm + tile + t * ATOM, row, cg * 2, 2);
    };

    // ---- products with the states, tile after tile of d_v (two are resident); the scores with the first.  The terms of
    // the next operand are formed while the products of the one before run: S's in ST, R's in R1 and where q was
    float sr = 0.f;
    for (int t = 0; t < tiles; ++t) {
        const int i = t & 1;
        if (i == 0) {
            if (t > 0) {                      // the second half: nothing reads the first one's tiles any more
                wait_b();
                __syncthreads();
                if (threadIdx.x == 0) {
                    mbar_expect_tx(bar_tma, (uint32_t)(2 * nt) * ATOM);
                    load(&f.to, L_::DO, t * DVT, nt);
                    load(&f.tv, L_::V, t * DVT, nt);
                }
            }
            wait_tma();
            if (t == 0) {
                zero_tail(L_::Q, KATOMS);
                zero_tail(L_::K, KATOMS);
            }
            zero_tail(L_::V, nt);
            zero_tail(L_::DO, nt);
        }
        if (t > 0) wait_a();
        terms(S, L_::ST, L_::ST + ATOM, L_::ST + 2 * ATOM);
        publish();
        if (warp == 0 && elect_one()) {
            if (t == 0) {
                mma_tiles<4 * KATOMS, false, false, 128>(T_SC, sb + L_::Q, sb + L_::K, false);
                mma_commit(bar_b);
            }
#pragma unroll 1
            for (int p = 0; p < 3; ++p) mma_tiles<4, false, false, NK>(T_DQ, sb + L_::DO + i * ATOM, sb + L_::ST + p * ATOM, t + p > 0);
            mma_tiles<4, false, false, 128>(T_DP, sb + L_::DO + i * ATOM, sb + L_::V + i * ATOM, t > 0);
            mma_commit(bar_a);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sr += S[j].x * R[j].x + S[j].y * R[j].y + S[j].z * R[j].z + S[j].w * R[j].w;
        if (t + 1 < tiles) fetch(f.s.S, t + 1, S);
        if (i == 1 || t == 0) wait_b();       // the scores (q's place is free), or the products of R's terms before
        terms(R, L_::R1 + i * ATOM, L_::R2, L_::R2 + ATOM);
        publish();
        if (warp == 0 && elect_one()) {
            mma_tiles<4, false, false, NK>(T_DK, sb + L_::V + i * ATOM, sb + L_::R1 + i * ATOM, t > 0);
#pragma unroll 1
            for (int p = 0; p < 2; ++p) mma_tiles<4, false, false, NK>(T_DK, sb + L_::V + i * ATOM, sb + L_::R2 + p * ATOM, true);
            mma_commit(bar_b);
        }
        if (t + 1 < tiles) fetch(f.s.R, t + 1, R);
    }
    wait_a();
    wait_b();
    if (threadIdx.x == 0) {                   // q again (from L2)
        mbar_expect_tx(bar_tma, (uint32_t)KATOMS * ATOM);
        load(&f.tq, L_::Q, 0, KATOMS);
    }

    if (threadIdx.x == 32 && blockIdx.x + SMS < gridDim.x) {
        // one CTA per SM has nobody to hide its loads behind: what the CTA a wave later reads is brought into L2, now that
        // this wave's loads are done
        const int u2 = (int)((blockIdx.x + SMS) / a.H), h2 = (int)((blockIdx.x + SMS) % a.H);
        LinPiece p2;
        if (lin_piece(a, u2, C, p2) && p2.len > 0) {
            const int tok2 = p2.t0 + p2.j * C;
            for (int k = 0; k < KATOMS; ++k) {
                prefetch_tile(&f.tq, k * 64, h2, tok2);
                prefetch_tile(&f.tk, k * 64, h2, tok2);
            }
            for (int t = 0; t < tiles; ++t) {
                prefetch_tile(&f.to, t * DVT, h2, tok2);
                prefetch_tile(&f.tv, t * DVT, h2, tok2);
                bulk_prefetch(f.s.S + tile_at(u2, a.H, h2, tiles, t), TILE_FLOATS * 4);
                bulk_prefetch(f.s.R + tile_at(u2, a.H, h2, tiles, t), TILE_FLOATS * 4);
            }
        }
    }
    // ---- P and dA (bf16) to shared memory; of Z, per block of 32 rows (q4) x 32 columns (cg): the rows' sums (zr), and for each
    // column t the sum over the rows from t on of the block's columns before t (zc); the sums of whole blocks behind the diagonal's
    // neighbours
    const float since = decay_since(d, row), until = decay_until(d, row);
    {
        float z = 0.f;                        // of the row's columns so far
        const float fs = a.scale * since;
        const f32x2 fs2 = pk2(fs, fs);
#pragma unroll 1
        for (int p = 0; p < 32; p += 16) {
            const int c0 = cg * 32 + p;
            uint32_t pb[8] = {}, ab[8] = {};
            if (cg <= q4) {
                float x[16], y[16];
                tmem_ld16x2(T_SC + lanes + c0, T_DP + lanes + c0, x, y);
                if (cg == q4) {               // the diagonal's block: zero above it, whatever the products hold there
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        x[j] = p + j <= lane ? x[j] : 0.f;
                        y[j] = p + j <= lane ? y[j] : 0.f;
                    }
                }
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    f32x2 g[2];
                    if (d.factored) {
                        const float4 b = *reinterpret_cast<const float4 *>(d.b + c0 + j);
                        g[0] = mul2(fs2, pk2(b.x, b.y));
                        g[1] = mul2(fs2, pk2(b.z, b.w));
                    } else {                  // (above the diagonal a factor may be infinite)
                        float e[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) e[i] = c0 + j + i <= row ? a.scale * decay_pair(d, row, c0 + j + i) : 0.f;
                        g[0] = pk2(e[0], e[1]);
                        g[1] = pk2(e[2], e[3]);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int k = j + 2 * i;
                        const f32x2 v = pk2(y[k], y[k + 1]), pp = mul2(pk2(x[k], x[k + 1]), g[i]), zz = mul2(pp, v);
                        const float before = z + x2(zz);
                        pb[k / 2] = round_bf16x2(pp);
                        ab[k / 2] = round_bf16x2(mul2(v, g[i]));
                        x[k] = z;
                        x[k + 1] = before;
                        z = before + y2(zz);
                    }
                }
                if (cg == q4) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[j] = p + j <= lane ? x[j] : 0.f;
                }
                const float s = sum16(x, lane);
                if (!(lane & 1)) zc[q4 * C + c0 + (lane >> 1)] = s;
            } else if (!(lane & 1)) {
                zc[q4 * C + c0 + (lane >> 1)] = 0.f;
            }
            const int tile = (c0 >> 6) * ATOM;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t off = swz(row, (c0 & 63) * 2 + j * 16);
                *reinterpret_cast<uint4 *>(sm + L_::P + tile + off) = make_uint4(pb[4 * j], pb[4 * j + 1], pb[4 * j + 2], pb[4 * j + 3]);
                *reinterpret_cast<uint4 *>(sm + L_::DA + tile + off) = make_uint4(ab[4 * j], ab[4 * j + 1], ab[4 * j + 2], ab[4 * j + 3]);
            }
        }
        zr[cg * C + row] = z;
        if (q4 > cg + 1) {                    // (cg, q4) = (0, 2), (0, 3), (1, 3)
            z = warp_sum(z);
            if (lane == 0) sr_w[26 + cg + q4] = z;
        }
    }
    wait_tma();
    zero_tail(L_::Q, KATOMS);
    // ---- dV's parts for the resident (last) half of d_v
    const int last = (tiles - 1) & ~1;
    auto value_parts = [&]() {                // P^T dO into the scores' columns, K R into dP's
        if (nt == 2) {
            mma_tiles<8, true, true, 128>(T_SC, sb + L_::P, sb + L_::DO, false);
            mma_tiles<4 * KATOMS, false, true, 128>(T_DP, sb + L_::K, sb + L_::R1, false);
        } else {
            mma_tiles<8, true, true, 64>(T_SC, sb + L_::P, sb + L_::DO, false);
            mma_tiles<4 * KATOMS, false, true, 64>(T_DP, sb + L_::K, sb + L_::R1, false);
        }
        mma_commit(bar_a);
    };
    publish();
    if (warp == 0 && elect_one()) value_parts();
    // ---- meanwhile the states' parts of dQ and dK: dot products with q and k, rows scaled in place
    if (cg < 2 * KATOMS) {
        const float fa = a.scale * since, fw = until;
        float xs = 0.f, ys = 0.f;
#pragma unroll 1
        for (int p = 0; p < 32; p += 16) {
            const int c0 = cg * 32 + p;
            float x[16], y[16];
            tmem_ld16x2(T_DQ + lanes + c0, T_DK + lanes + c0, x, y);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t off = (c0 >> 6) * ATOM + swz(row, (c0 & 63) * 2 + j * 16);
                const uint4 qv = *reinterpret_cast<const uint4 *>(sm + L_::Q + off), kv = *reinterpret_cast<const uint4 *>(sm + L_::K + off);
                const uint32_t qw[4] = {qv.x, qv.y, qv.z, qv.w}, kw[4] = {kv.x, kv.y, kv.z, kv.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    xs = fmaf(bf16_lo(qw[i]), x[8 * j + 2 * i], xs);
                    xs = fmaf(bf16_hi(qw[i]), x[8 * j + 2 * i + 1], xs);
                    ys = fmaf(bf16_lo(kw[i]), y[8 * j + 2 * i], ys);
                    ys = fmaf(bf16_hi(kw[i]), y[8 * j + 2 * i + 1], ys);
                }
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                x[j] *= fa;
                y[j] *= fw;
            }
            tmem_st16(T_DQ + lanes + c0, x);
            tmem_st16(T_DK + lanes + c0, y);
        }
        xi[cg * C + row] = fa * xs;
        yi[cg * C + row] = fw * ys;
    }
    sr = warp_sum(sr);
    if (lane == 0) sr_w[warp] = sr;
    publish();

    // ---- dQ, dK
    if (warp == 0 && elect_one()) {
        mma_tiles<8, false, true, NK>(T_DQ, sb + L_::DA, sb + L_::K, true);
        mma_commit(bar_b);
        mma_tiles<8, true, true, NK>(T_DK, sb + L_::DA, sb + L_::Q, true);
        mma_commit(bar_c);                    // (a barrier of its own: it must not run a phase ahead of a waiter)
    }
    // meanwhile four warps sum up the decay's gradient, a token per thread: sums over the tokens from t on and before t.  Pairs
    // (i, j): within the warp's columns (zc), its rows from t on with the columns before them, later rows with those
    if (f.b.dg && warp < 4) {
        const int t = threadIdx.x;
        float pairs = 0.f, rows = 0.f, later = 0.f, earlier = 0.f, s0 = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            pairs += zc[i * C + t];
            if (i < warp) rows += zr[i * C + t];
        }
        if (warp == 1 || warp == 2) pairs += sr_w[27 + warp] + sr_w[28 + warp];
#pragma unroll
        for (int i = 0; i < 2 * KATOMS; ++i) {
            later += xi[i * C + t];
            earlier += yi[i * C + t];
        }
#pragma unroll
        for (int i = 0; i < NT / 32; i += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(sr_w + i);
            s0 += (x.x + x.y) + (x.z + x.w);
        }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const float yr = __shfl_down_sync(0xffffffffu, rows, off), yl = __shfl_down_sync(0xffffffffu, later, off),
                        ye = __shfl_up_sync(0xffffffffu, earlier, off);
            if (lane + off < 32) {
                rows += yr;
                later += yl;
            }
            if (lane >= off) earlier += ye;
        }
        if (lane == 0) sr_w[16 + warp] = later;          // the warp's sums
        if (lane == 31) sr_w[20 + warp] = earlier;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        earlier = __shfl_up_sync(0xffffffffu, earlier, 1);   // of the tokens before
        if (lane == 0) earlier = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i > warp) later += sr_w[16 + i];
            if (i < warp) earlier += sr_w[20 + i];
        }
        const float g = ((pairs + rows) + later) + earlier + d.whole.x * s0;
        if (a.decay == KDN_DECAY_TOKEN) {
            if (t < L) f.b.dg[(size_t)(tok + t) * a.H + h] = g;
        } else {
            const float sum = warp_sum(t < L ? g : 0.f);
            if (lane == 0) sr_w[24 + warp] = sum;
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (t == 0) f.s.share[(size_t)u * a.H + h] = (sr_w[24] + sr_w[25]) + (sr_w[26] + sr_w[27]);
        }
    }

    // ---- out, each as its products are done: 32 columns of a warp's 32 rows at a time through shared memory that no MMA
    // reads any more, so that four lanes share a row's 64 bytes in memory.  which: 0 dv, 1 dq, 2 dk (one piece of code:
    // a CTA passes here once, and what it executes has to be fetched)
    auto put = [&](int which, int t0) {
        const int width = which ? a.dk : a.dv, col = t0 * DVT + cg * 32, in = cg * 32;
        if (col >= width || in >= (which ? NK : nt * DVT)) return;
        uint8_t *tile = sm + (which == 0 ? L_::DO : which == 1 ? L_::R1 : L_::DA) + (in >> 6) * ATOM;
        const uint32_t acc = (which == 0 ? T_SC : which == 1 ? T_DQ : T_DK) + lanes + in;
        bf16 *dst = static_cast<bf16 *>(which == 0 ? f.b.dv : which == 1 ? f.b.dq : f.b.dk);
#pragma unroll
        for (int p = 0; p < 32; p += 16) {
            float x[16], y[16];
            tmem_ld16x2(acc + p, T_DP + lanes + in + p, x, y);
            const f32x2 f2 = pk2(until, until);
            uint32_t z[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                f32x2 v = pk2(x[2 * j], x[2 * j + 1]);
                if (which == 0) v = fma2(f2, pk2(y[2 * j], y[2 * j + 1]), v);
                z[j] = round_bf16x2(v);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
                *reinterpret_cast<uint4 *>(tile + swz(row, (in & 63) * 2 + p * 2 + j * 16)) = make_uint4(z[4 * j], z[4 * j + 1], z[4 * j + 2], z[4 * j + 3]);
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < 32; r += 8) {
            const int t = q4 * 32 + r + (lane >> 2);
            const uint4 z = *reinterpret_cast<const uint4 *>(tile + swz(t, (in & 63) * 2 + (lane & 3) * 16));
            if (t < L) *reinterpret_cast<uint4 *>(dst + ((size_t)(tok + t) * a.H + h) * width + col + (lane & 3) * 8) = z;
        }
    };
#pragma unroll 1
    for (int which = 0; which < 3; ++which) {
        if (which == 0) wait_a();
        if (which == 1) wait_b();
        if (which == 2) {
            w.wait(bar_c, 0);
            tc_fence_after();
        }
        put(which, which == 0 ? last : 0);
    }
    // ---- the first half's dV (d_v = 256)
    for (int t0 = last - 2; t0 >= 0; t0 -= 2) {
        publish();                            // the tiles that were written through are read, TMEM too
        if (threadIdx.x == 0) {
            mbar_expect_tx(bar_tma, (uint32_t)nt * ATOM);
            load(&f.to, L_::DO, t0 * DVT, nt);
        }
        for (int t = 0; t < nt; ++t) {
            fetch(f.s.R, t0 + t, R);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 y0 = R[2 * j], y1 = R[2 * j + 1];
                *reinterpret_cast<uint4 *>(sm + L_::R1 + t * ATOM + swz(row, (cg * 2 + j) * 16)) =
                    make_uint4(round_bf16x2(pk2(y0.x, y0.y)), round_bf16x2(pk2(y0.z, y0.w)), round_bf16x2(pk2(y1.x, y1.y)), round_bf16x2(pk2(y1.z, y1.w)));
            }
        }
        wait_tma();
        zero_tail(L_::DO, nt);
        publish();
        if (warp == 0 && elect_one()) value_parts();
        wait_a();
        put(0, t0);
    }

    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {                        // a wait gave up: bounded waits for what is in flight, before its memory goes
        if (threadIdx.x == 0) {
            raise_error(a.err, ERR_TIMEOUT);
            drain(bar_tma, 0);
            drain(bar_tma, 1);
        }
        if (warp == 0 && elect_one()) {
            mbar_init(bar_a, 1);
            mbar_fence_init();
            mma_commit(bar_a);
            drain(bar_a, 0);
        }
        __syncthreads();
    }
    if (warp == 0) tmem_dealloc(tmem, 512);
}

size_t linear_tc_backward_workspace_bytes(const LinArgs &a) { return states_workspace_bytes(a); }

cudaError_t launch_linear_tc_backward(const LinBwdArgs &b, void *workspace, cudaStream_t st) {
    const LinArgs &a = b.a;
    GradArgs f;
    f.b = b;
    cudaError_t e = launch_states(b, workspace, &f.s, st);
    if (e != cudaSuccess) return e;
    if (!make_token_map(&f.tq, a.q, a.dk, a.H, a.ntok) || !make_token_map(&f.tk, a.k, a.dk, a.H, a.ntok) ||
        !make_token_map(&f.tv, a.v, a.dv, a.H, a.ntok) || !make_token_map(&f.to, b.d_o, a.dv, a.H, a.ntok))
        return cudaErrorInvalidValue;
    auto kern = a.dk > 64 ? linear_grad_tc_kernel<2> : linear_grad_tc_kernel<1>;
    KernelSetup ks;
    e = kernel_setup(reinterpret_cast<const void *>(kern), Smem::TOTAL, NT, false, &ks);
    if (e != cudaSuccess) return e;
    e = launch(kern, dim3((unsigned)(lin_slots(a.cu != nullptr, a.T, a.ntok, a.nseq, C) * a.H)), NT, Smem::TOTAL, st, f);
    if (e != cudaSuccess || !b.dg || a.decay != KDN_DECAY_HEAD) return e;
    return launch_linear_head_decay(a, f.s.share, b.dg, C, st);
}

}  // namespace kdn
