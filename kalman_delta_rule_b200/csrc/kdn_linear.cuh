// Linear attention with a decay for each head: argument packs, launchers and the device helpers
// its kernels share.  Per head, with a log decay g_t (natural logarithm, <= 0),
//     S_t = e^{g_t} S_{t-1} + k_t v_t^T,    o_t = scale S_t^T q_t.
// A sequence is cut into chunks of C tokens; with G_t = sum_{j <= t} g_j from the chunk's start the
// recurrence unrolls to
//     O  = scale ((Q K^T o D) V + diag(e^G) Q S),   D_ts = e^{G_t - G_s} for t >= s, else 0
//     S' = e^{G_C} S + K^T diag(e^{G_C - G}) V
// Every factor that the kernels form from a difference of G is at most one (for g <= 0).
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

// Sums of log2 decays are kept in two floats (about 48 bits): a constant decay near one leaves its mark only
// after thousands of tokens, and a strongly decaying chunk must not cost two neighbours' difference its bits.
// (fp64 or 64-bit integers would do too, but take ten times as long: the GPU has few units for them.)  Below
// e^-2839 (a reset, g = -inf, included) every fp32 factor across a token is 0 either way; the floor keeps
// differences of sums free of inf - inf.
struct Log2 {
    float hi, lo;
};
__device__ __forceinline__ Log2 lin_log2(float g) {          // from the natural logarithm; a NaN gives -2839, see the callers
    const float x = fmaxf(g, -2839.f);
    const float hi = x * 1.44269504f;
    return {hi, fmaf(x, 1.44269504f, -hi) + x * 1.92596299e-8f};
}
__device__ __forceinline__ Log2 operator+(Log2 a, Log2 b) {   // (Knuth's two-sum, then renormalised)
    const float s = a.hi + b.hi, t = s - a.hi;
    const float e = ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo);
    const float hi = s + e;
    return {hi, e - (hi - s)};
}
__device__ __forceinline__ Log2 operator-(Log2 a, Log2 b) { return a + Log2{-b.hi, -b.lo}; }
__device__ __forceinline__ float lin_load_decay(const LinArgs &a, int t, int h) {
    if (a.decay == KDN_DECAY_NONE) return 0.f;
    return a.decay == KDN_DECAY_HEAD ? __ldg(a.g + h) : __ldg(a.g + (size_t)t * a.H + h);
}
__device__ __forceinline__ float lin_exp2(Log2 x) { return exp2f(x.hi) * fmaf(x.lo, 0.693147181f, 1.f); }
// 2^(a - b); the difference is rounded to fp32, an error of 2^-24 of the exponent (where that is large the factor is tiny)
__device__ __forceinline__ float lin_exp2_between(Log2 a, Log2 b) { return exp2f((a.hi - b.hi) + (a.lo - b.lo)); }
// A whole chunk's decay 2^x in two floats, 1 + expm1.  One float would be off by up to half a unit in the
// last place, the same way in every chunk of a constant decay: over the chunks that a decay near one lets
// the memory last that adds up to several 1e-6 of the state.  What is left is relative to 1 - 2^x.  Below
// one half, where nothing lasts, one float and its exponential do (1 + expm1 would cancel).
__device__ __forceinline__ float2 lin_chunk_decay(Log2 x) {
    if (x.hi < -1.f) return make_float2(lin_exp2(x), 0.f);
    const float z = expm1f(fmaf(x.hi, 0.693147181f, fmaf(x.hi, -1.90465421e-9f, x.lo * 0.693147181f)));
    const float hi = 1.f + z;
    return make_float2(hi, z - (hi - 1.f));
}
__device__ __forceinline__ float lin_carry(float2 decay, float s, float u) { return fmaf(decay.x, s, fmaf(decay.y, s, u)); }

// Launches of a call follow one another programmatically: a CTA of the next one may start, set itself up and read the
// caller's inputs once every CTA of this one runs (or is done).  Every CTA waits for the launch before it, one without
// work too, before it reads what any earlier launch wrote: no launch is complete before those that precede it.
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void wait_for_launch() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// (The status is the launch's own: cudaGetLastError() after <<< >>> may be that of an earlier call, and a decode step reported
// as failed has taken its token all the same.)
template <typename... P, typename... A>
cudaError_t launch_with(bool early, void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}
// a call's first launch, or one that starts when the launch before is done ...
template <typename... P, typename... A>
cudaError_t launch(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A &...args) {
    return launch_with(false, kern, grid, threads, smem, st, args...);
}
// ... and one that follows programmatically
template <typename... P, typename... A>
cudaError_t launch_next(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A &...args) {
    return launch_with(true, kern, grid, threads, smem, st, args...);
}

}  // namespace kdn
