// Linear attention with a decay for each head: argument packs, launchers and the device helpers
// its kernels share.  Per head, with a log decay g_t (natural logarithm, <= 0),
//     S_t = e^{g_t} S_{t-1} + k_t v_t^T,    o_t = scale S_t^T q_t.
// A sequence is cut into chunks of C tokens; with G_t = sum_{j <= t} g_j from the chunk's start the
// recurrence unrolls to
//     O  = scale ((Q K^T o D) V + diag(e^G) Q S),   D_ts = e^{G_t - G_s} for t >= s, else 0
//     S' = e^{G_C} S + K^T diag(e^{G_C - G}) V
// Every factor that the kernels form from a difference of G is at most one (for g <= 0).  G is
// summed in fp64: a difference of two partial sums of a strongly decaying chunk keeps its bits.
#pragma once

#include "kdn_common.cuh"

namespace kdn {

struct LinArgs {
    const void *q, *k, *v;     // [ntok, H, dk], [ntok, H, dk], [ntok, H, dv]
    const float *g;            // log decay: [ntok, H] (KDN_DECAY_TOKEN), [H] (KDN_DECAY_HEAD) or NULL
    int decay;                 // kdn_decay_t
    float scale;
    const float *S0;           // [N, H, dk, dv] or NULL (zero)
    void *o;                   // [ntok, H, dv]
    float *S_out;              // [N, H, dk, dv] or NULL
    const int32_t *cu;         // device [N + 1] or NULL (dense: sequence s = [s T, (s + 1) T))
    int T, nseq, H, dk, dv;
    int ntok;
    unsigned *err;
};

struct LinBwdArgs {
    LinArgs a;                 // forward inputs (o, S_out unused)
    const void *d_o;           // [ntok, H, dv]
    const float *dS_T;         // [N, H, dk, dv] or NULL (zero)
    void *dq, *dk, *dv;        // token layouts, input dtype
    float *dg;                 // [ntok, H], [H] or NULL
    float *dS0;                // [N, H, dk, dv] or NULL
};

// ------------------------------------------------------------ sequences cut into pieces of L tokens
// Slot u of a problem holds piece j of sequence s.  Packed sequences: sequence s owns the slots from
// cu[s] / L + s on -- at least as many as it has pieces, and at least one -- so a piece's slot needs
// no table, ntok / L + N slots are enough for any lengths, and some slots stay empty.
struct LinPiece {
    int s, j;                  // sequence, piece
    int t0, len;               // the sequence's first token and length
};

__host__ __device__ __forceinline__ long long lin_slots(bool packed, int T, long long ntok, int nseq, int L) {
    return packed ? ntok / L + nseq : (long long)nseq * (T > L ? (T + L - 1) / L : 1);
}

// the sequence's tokens; a malformed cu_seqlens cannot lead outside the token tensors
__device__ __forceinline__ void lin_seq(const LinArgs &a, int s, int &t0, int &len) {
    if (a.cu) {
        t0 = min(max(__ldg(a.cu + s), 0), a.ntok);
        len = max(min(__ldg(a.cu + s + 1), a.ntok) - t0, 0);
    } else {
        t0 = s * a.T;
        len = a.T;
    }
}
__device__ __forceinline__ int lin_first_slot(const LinArgs &a, int s, int t0, int L) {
    return a.cu ? t0 / L + s : s * (a.T > L ? (a.T + L - 1) / L : 1);
}
// piece of slot u; false: the slot is empty (a sequence without tokens has one piece, of length 0)
__device__ __forceinline__ bool lin_piece(const LinArgs &a, int u, int L, LinPiece &p) {
    if (a.cu) {
        int lo = 0, hi = a.nseq - 1;      // the last sequence whose first slot is <= u
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (min(max(__ldg(a.cu + mid), 0), a.ntok) / L + mid <= u) lo = mid; else hi = mid - 1;
        }
        p.s = lo;
    } else {
        p.s = u / (a.T > L ? (a.T + L - 1) / L : 1);
    }
    lin_seq(a, p.s, p.t0, p.len);
    p.j = u - lin_first_slot(a, p.s, p.t0, L);
    return p.j == 0 || (p.j > 0 && (long long)p.j * L < p.len);
}

// log2 of a token's decay factor in fp64.  Below 2^-4096 (a reset, g = -inf, included) every fp32
// factor across the token is 0 either way; the floor keeps differences of sums free of inf - inf.
__device__ __forceinline__ double lin_log2_decay(const LinArgs &a, int t, int h) {
    if (a.decay == KDN_DECAY_NONE) return 0.0;
    const float g = a.decay == KDN_DECAY_HEAD ? __ldg(a.g + h) : __ldg(a.g + (size_t)t * a.H + h);
    const double x = (double)g * 1.4426950408889634;
    return x < -4096.0 ? -4096.0 : x;     // a NaN stays a NaN
}
// 2^x for x <= 0; the fp64 argument is split so that its fraction keeps fp32's relative accuracy
__device__ __forceinline__ float lin_exp2(double x) {
    const float hi = (float)x;
    return exp2f(hi) * (1.f + 0.693147180559945f * (float)(x - (double)hi));
}

// A whole chunk's decay 2^x in two floats.  One float would be off by up to half a unit in the last
// place, the same way in every chunk of a constant decay: over the thousands of chunks of a long memory
// that adds up to several 1e-6 of the state.
__device__ __forceinline__ float2 lin_chunk_decay(double x) {
    const double f = exp2(x);
    const float hi = (float)f;
    return make_float2(hi, (float)(f - (double)hi));
}
__device__ __forceinline__ float lin_carry(float2 decay, float s, float u) { return fmaf(decay.x, s, fmaf(decay.y, s, u)); }

}  // namespace kdn
