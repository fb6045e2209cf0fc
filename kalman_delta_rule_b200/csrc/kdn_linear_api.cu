// C ABI of the linear-attention and layer-norm entry points: argument validation, workspace sizing
// and dispatch.  Declarations and the contract are in include/kdn.h.
#include <math.h>

#include <initializer_list>

#include "kdn_common.cuh"
#include "kdn_launch.h"

namespace {

bool dk_ok(int d) { return d == 32 || d == 64 || d == 128; }
bool dv_ok(int d) { return d == 32 || d == 64 || d == 128 || d == 256; }
bool aligned(std::initializer_list<const void *> ptrs) {   // 16 bytes; NULL passes
    for (const void *p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & 15u) return false;
    return true;
}
struct Span {
    const void *p;
    size_t bytes;
};
bool overlap(const Span &a, const Span &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}
// no output (or workspace) shares a byte with an input or another output (kernels read inputs while other CTAs write)
bool distinct(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (const Span &in : ins)
            if (overlap(*o, in)) return false;
        for (auto other = outs.begin(); other != o; ++other)
            if (overlap(*o, *other)) return false;
    }
    return true;
}
// bytes of a problem's arrays
struct Sizes {
    size_t qk, vo, g, state;
    Sizes(const kdn::LinArgs &a, kdn_dtype_t dtype) {
        const size_t rows = (size_t)a.ntok * a.H, e = dtype == KDN_DTYPE_BF16 ? 2 : 4;
        qk = rows * a.dk * e;
        vo = rows * a.dv * e;
        g = a.decay == KDN_DECAY_TOKEN ? rows * 4 : a.decay == KDN_DECAY_HEAD ? (size_t)a.H * 4 : 0;
        state = (size_t)a.nseq * a.H * a.dk * a.dv * 4;
    }
};
kdn_status_t cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return KDN_OK;
    (void)cudaGetLastError();              // reported by the status, not to whichever launch asks next
    return KDN_ERR_CUDA;
}

kdn_status_t check_sizes(int H, int d_k, int d_v, kdn_dtype_t dtype, float scale, int decay) {
    if (H <= 0 || !isfinite(scale)) return KDN_ERR_INVALID_ARG;
    if (dtype != KDN_DTYPE_F32 && dtype != KDN_DTYPE_BF16) return KDN_ERR_INVALID_ARG;
    if (decay != KDN_DECAY_NONE && decay != KDN_DECAY_TOKEN && decay != KDN_DECAY_HEAD) return KDN_ERR_INVALID_ARG;
    if (!dk_ok(d_k) || !dv_ok(d_v)) return KDN_ERR_UNSUPPORTED;
    return KDN_OK;
}

// validates `p` and fills the sizes of `a`
kdn_status_t check_problem(const kdn_linear_problem_t *p, kdn::LinArgs *a) {
    if (!p) return KDN_ERR_INVALID_ARG;
    if (p->B < 0 || p->T < 0) return KDN_ERR_INVALID_ARG;
    const kdn_status_t st = check_sizes(p->H, p->d_k, p->d_v, p->in_dtype, p->scale, p->decay);
    if (st != KDN_OK) return st;
    if (p->cu_seqlens && (p->B != 1 || p->num_seqs < 0)) return KDN_ERR_INVALID_ARG;
    *a = kdn::LinArgs{};
    a->cu = p->cu_seqlens;
    a->nseq = p->cu_seqlens ? p->num_seqs : p->B;
    a->T = p->T; a->H = p->H; a->dk = p->d_k; a->dv = p->d_v;
    a->scale = p->scale; a->decay = p->decay;
    const long long ntok = (long long)p->B * p->T;
    if (ntok > (1ll << 30)) return KDN_ERR_UNSUPPORTED;
    // grids are one-dimensional in (slots x heads) or (sequences x heads x tiles of d_v)
    if ((ntok / 64 + a->nseq) * a->H >= (1ll << 31) || (long long)a->nseq * a->H * (a->dv / 32) >= (1ll << 31)) return KDN_ERR_UNSUPPORTED;
    a->ntok = (int)ntok;
    return KDN_OK;
}

// Which kernels run a problem.  Short sequences, whose lengths are bounded by T (packed: by all the tokens, the lengths
// being known on the device only), have paths of their own: one launch instead of two to five, no states written and read
// between launches, and fp32 arithmetic whatever the type -- with a few hundred scores nothing averages the tensor cores'
// roundings of them.  At d = 128, with 1 / 64 / 2048 heads in all:
// Forward, token after token: 16 tokens 5.7 / 7.6 / 100 us in bf16 against 9.2 / 9.7 / 231 on the tensor cores, 32 tokens
// 9.0 / 12.2 / 178 against 9.2 / 9.6 / 230, 64 tokens 15.5 / 21 / 319 against 9.2 / 9.7 / 232.  fp32, 64 tokens: 14.7 / 20.8 / 294
// against 21.3 / 22.3 / 851 in chunks, d = 64: 12.7 / 13.1 / 103 against 14.7 / 15.4 / 190.  At d = 32 alone the chunks are the
// quicker ones from about 40 tokens on (64 tokens: 13.5 / 14.7 / 77 against 8.6 / 9.6 / 80).
// Backward, the whole sequence as one chunk: 16 tokens 24 / 24 / 273 us against 28 / 28 / 548 on the tensor cores, 24 tokens
// 31 / 32 / 469 against 28 / 28 / 550, 32 tokens 40 / 40 / 587 against 28 / 28 / 545 (d = 64: 17 / 17 / 257 against 23 / 23 / 303;
// fp32 in chunks: 55 / 67 / 1135).  Above some 20 tokens at d = 128 the bf16 call pays for its accuracy, not for its time.
constexpr int kShortForwardBf16 = 32, kShortForwardF32 = 64;
enum Path { SHORT, CUDA_CORES, TENSOR_CORES };
int longest(const kdn::LinArgs &a) { return a.cu ? a.ntok : a.T; }
Path forward_path(const kdn_linear_problem_t *p, const kdn::LinArgs &a) {
    const bool bf16 = p->in_dtype == KDN_DTYPE_BF16;
    if (longest(a) <= (bf16 ? kShortForwardBf16 : kShortForwardF32)) return SHORT;
    return bf16 ? TENSOR_CORES : CUDA_CORES;
}
Path backward_path(const kdn_linear_problem_t *p, const kdn::LinArgs &a) {
    if (longest(a) <= kdn::kLinearShort) return SHORT;
    return p->in_dtype == KDN_DTYPE_BF16 ? TENSOR_CORES : CUDA_CORES;
}
size_t forward_bytes(const kdn_linear_problem_t *p, const kdn::LinArgs &a) {
    const Path path = forward_path(p, a);
    return path == SHORT ? 0 : path == TENSOR_CORES ? kdn::linear_tc_workspace_bytes(a) : kdn::linear_simt_workspace_bytes(a);
}
size_t backward_bytes(const kdn_linear_problem_t *p, const kdn::LinArgs &a) {
    const Path path = backward_path(p, a);
    return path == SHORT ? kdn::linear_short_backward_workspace_bytes(a)
                         : path == TENSOR_CORES ? kdn::linear_tc_backward_workspace_bytes(a) : kdn::linear_simt_backward_workspace_bytes(a);
}

kdn_status_t check_norm(long long n, int G, int d, kdn_dtype_t dtype, float eps) {
    if (n < 0 || G <= 0 || d <= 0 || !(eps >= 0.f) || !isfinite(eps)) return KDN_ERR_INVALID_ARG;
    if (dtype != KDN_DTYPE_F32 && dtype != KDN_DTYPE_BF16) return KDN_ERR_INVALID_ARG;
    if (d > kdn::kNormMaxWidth || G > 65535 || n > (1ll << 40) / G) return KDN_ERR_UNSUPPORTED;
    return KDN_OK;
}

}  // namespace

extern "C" {

kdn_status_t kdn_linear_workspace_size(const kdn_linear_problem_t *p, size_t *bytes) {
    kdn::LinArgs a;
    const kdn_status_t st = check_problem(p, &a);
    if (st != KDN_OK) return st;
    if (!bytes) return KDN_ERR_INVALID_ARG;
    *bytes = forward_bytes(p, a);
    return KDN_OK;
}

kdn_status_t kdn_linear_forward(const kdn_linear_problem_t *p, const void *q, const void *k, const void *v,
                                const float *g, const float *S0, void *o, float *S_out, void *workspace,
                                size_t workspace_bytes, void *stream) {
    kdn::LinArgs a;
    const kdn_status_t st = check_problem(p, &a);
    if (st != KDN_OK) return st;
    if (a.nseq == 0 || (a.ntok == 0 && !S_out)) return KDN_OK;
    if (a.ntok > 0 && (!q || !k || !v || !o || (a.decay != KDN_DECAY_NONE && !g))) return KDN_ERR_INVALID_ARG;
    if (!aligned({q, k, v, g, S0, o, S_out})) return KDN_ERR_INVALID_ARG;
    const size_t need = forward_bytes(p, a);
    if (need && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))) return KDN_ERR_WORKSPACE;
    const Sizes n(a, p->in_dtype);
    if (!distinct({{o, n.vo}, {S_out, n.state}, {workspace, need}}, {{q, n.qk}, {k, n.qk}, {v, n.vo}, {g, n.g}, {S0, n.state}}))
        return KDN_ERR_INVALID_ARG;
    a.q = q; a.k = k; a.v = v; a.g = g; a.S0 = S0; a.o = o; a.S_out = S_out;
    a.err = kdn::error_word();
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    switch (forward_path(p, a)) {
        case SHORT: return cuda_status(kdn::launch_linear_recurrent(a, p->in_dtype == KDN_DTYPE_BF16, cs));
        case CUDA_CORES: return cuda_status(kdn::launch_linear_simt(a, workspace, cs));
        default: return cuda_status(kdn::launch_linear_tc(a, workspace, cs));
    }
}

kdn_status_t kdn_linear_decode_tokens(int N, int n_tokens, int H, int d_k, int d_v, kdn_dtype_t in_dtype, float scale,
                                      int decay, const void *q, const void *k, const void *v, const float *g, float *S,
                                      void *o, void *stream) {
    if (N < 0 || n_tokens < 0) return KDN_ERR_INVALID_ARG;
    const kdn_status_t st = check_sizes(H, d_k, d_v, in_dtype, scale, decay);
    if (st != KDN_OK) return st;
    if (N == 0 || n_tokens == 0) return KDN_OK;
    if ((long long)N * n_tokens > (1ll << 30) || (long long)N * H * (d_v / 32) >= (1ll << 31)) return KDN_ERR_UNSUPPORTED;
    if (!q || !k || !v || !S || !o || (decay != KDN_DECAY_NONE && !g)) return KDN_ERR_INVALID_ARG;
    if (!aligned({q, k, v, g, S, o})) return KDN_ERR_INVALID_ARG;
    kdn::LinArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.decay = decay; a.scale = scale;
    a.S0 = S; a.S_out = S; a.o = o;
    a.T = n_tokens; a.nseq = N; a.H = H; a.dk = d_k; a.dv = d_v; a.ntok = N * n_tokens;
    const Sizes n(a, in_dtype);
    if (!distinct({{o, n.vo}, {S, n.state}}, {{q, n.qk}, {k, n.qk}, {v, n.vo}, {g, n.g}})) return KDN_ERR_INVALID_ARG;
    return cuda_status(kdn::launch_linear_recurrent(a, in_dtype == KDN_DTYPE_BF16, static_cast<cudaStream_t>(stream)));
}

kdn_status_t kdn_linear_backward_workspace_size(const kdn_linear_problem_t *p, size_t *bytes) {
    kdn::LinArgs a;
    const kdn_status_t st = check_problem(p, &a);
    if (st != KDN_OK) return st;
    if (!bytes) return KDN_ERR_INVALID_ARG;
    *bytes = backward_bytes(p, a);
    return KDN_OK;
}

kdn_status_t kdn_linear_backward(const kdn_linear_problem_t *p, const void *q, const void *k, const void *v,
                                 const float *g, const float *S0, const void *d_o, const float *dS_T, void *dq, void *dk,
                                 void *dv, float *dg, float *dS0, void *workspace, size_t workspace_bytes, void *stream) {
    kdn::LinBwdArgs b{};
    kdn::LinArgs &a = b.a;
    const kdn_status_t st = check_problem(p, &a);
    if (st != KDN_OK) return st;
    if (dg && a.decay == KDN_DECAY_NONE) return KDN_ERR_INVALID_ARG;
    if (!aligned({q, k, v, g, S0, d_o, dS_T, dq, dk, dv, dg, dS0})) return KDN_ERR_INVALID_ARG;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (a.nseq == 0 || a.ntok == 0) {
        if (dg && a.decay == KDN_DECAY_HEAD && cuda_status(cudaMemsetAsync(dg, 0, sizeof(float) * a.H, cs)) != KDN_OK) return KDN_ERR_CUDA;
        if (a.nseq == 0 || !dS0) return KDN_OK;
    }
    if (a.ntok > 0 && (!q || !k || !v || !d_o || !dq || !dk || !dv || (a.decay != KDN_DECAY_NONE && !g)))
        return KDN_ERR_INVALID_ARG;
    const size_t need = backward_bytes(p, a);
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return KDN_ERR_WORKSPACE;
    const Sizes n(a, p->in_dtype);
    if (!distinct({{dq, n.qk}, {dk, n.qk}, {dv, n.vo}, {dg, n.g}, {dS0, n.state}, {workspace, need}},
                  {{q, n.qk}, {k, n.qk}, {v, n.vo}, {g, n.g}, {S0, n.state}, {d_o, n.vo}, {dS_T, n.state}}))
        return KDN_ERR_INVALID_ARG;
    a.q = q; a.k = k; a.v = v; a.g = g; a.S0 = S0;
    a.err = kdn::error_word();
    b.d_o = d_o; b.dS_T = dS_T; b.dq = dq; b.dk = dk; b.dv = dv; b.dg = dg; b.dS0 = dS0;
    switch (backward_path(p, a)) {
        case SHORT: return cuda_status(kdn::launch_linear_short_backward(b, p->in_dtype == KDN_DTYPE_BF16, workspace, cs));
        case CUDA_CORES: return cuda_status(kdn::launch_linear_simt_backward(b, workspace, cs));
        default: return cuda_status(kdn::launch_linear_tc_backward(b, workspace, cs));
    }
}

kdn_status_t kdn_layer_norm(long long n, int G, int d, kdn_dtype_t dtype, float eps, const void *x, const float *weight,
                            const float *bias, void *y, float *mean, float *rstd, void *stream) {
    const kdn_status_t st = check_norm(n, G, d, dtype, eps);
    if (st != KDN_OK) return st;
    if (n == 0) return KDN_OK;
    if (!x || !y || !aligned({x, weight, bias, y, mean, rstd})) return KDN_ERR_INVALID_ARG;
    const size_t par = (size_t)G * d * 4, rows = (size_t)n * G, all = rows * d * (dtype == KDN_DTYPE_BF16 ? 2 : 4);
    if (!distinct({{y, all}, {mean, rows * 4}, {rstd, rows * 4}}, {{x, all}, {weight, par}, {bias, par}})) return KDN_ERR_INVALID_ARG;
    kdn::NormArgs a{};
    a.x = x; a.weight = weight; a.bias = bias; a.y = y; a.mean = mean; a.rstd = rstd;
    a.n = n; a.G = G; a.d = d; a.eps = eps;
    return cuda_status(kdn::launch_norm(a, dtype == KDN_DTYPE_BF16, static_cast<cudaStream_t>(stream)));
}

kdn_status_t kdn_layer_norm_backward_workspace_size(long long n, int G, int d, size_t *bytes) {
    const kdn_status_t st = check_norm(n, G, d, KDN_DTYPE_F32, 0.f);
    if (st != KDN_OK) return st;
    if (!bytes) return KDN_ERR_INVALID_ARG;
    *bytes = kdn::norm_backward_workspace_bytes(n, G, d);
    return KDN_OK;
}

kdn_status_t kdn_layer_norm_backward(long long n, int G, int d, kdn_dtype_t dtype, const void *dy, const void *x,
                                     const float *weight, const float *mean, const float *rstd, void *dx, float *dweight,
                                     float *dbias, void *workspace, size_t workspace_bytes, void *stream) {
    const kdn_status_t st = check_norm(n, G, d, dtype, 0.f);
    if (st != KDN_OK) return st;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (!aligned({dy, x, weight, mean, rstd, dx, dweight, dbias})) return KDN_ERR_INVALID_ARG;
    if (n == 0) {   // no rows: the sums are zero
        for (float *out : {dweight, dbias})
            if (out && cuda_status(cudaMemsetAsync(out, 0, sizeof(float) * (size_t)G * d, cs)) != KDN_OK) return KDN_ERR_CUDA;
        return KDN_OK;
    }
    if (!dy || !x || !mean || !rstd || !dx) return KDN_ERR_INVALID_ARG;
    kdn::NormArgs a{};
    size_t need = 0;
    if (dweight || dbias) {
        need = kdn::norm_backward_workspace_bytes(n, G, d);
        if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return KDN_ERR_WORKSPACE;
        a.part = static_cast<float *>(workspace);
    }
    const size_t par = (size_t)G * d * 4, rows = (size_t)n * G, all = rows * d * (dtype == KDN_DTYPE_BF16 ? 2 : 4);
    if (!distinct({{dx, all}, {dweight, par}, {dbias, par}, {workspace, need}},
                  {{dy, all}, {x, all}, {weight, par}, {mean, rows * 4}, {rstd, rows * 4}}))
        return KDN_ERR_INVALID_ARG;
    a.x = x; a.dy = dy; a.weight = weight; a.dx = dx;
    a.mean = const_cast<float *>(mean); a.rstd = const_cast<float *>(rstd);
    a.dweight = dweight; a.dbias = dbias;
    a.n = n; a.G = G; a.d = d;
    return cuda_status(kdn::launch_norm_backward(a, dtype == KDN_DTYPE_BF16, cs));
}

}  // extern "C"
