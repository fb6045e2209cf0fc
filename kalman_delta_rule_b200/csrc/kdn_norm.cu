// Layer norm over the last axis of rows [n, G, d], with a weight and a bias row for each of the G
// groups (G = 1: one pair for all rows; G = heads: the norm of a layer's readout), and its gradient:
//     m = mean(x),  r = (mean((x - m)^2) + eps)^{-1/2},  y = (x - m) r w + b
//     dx = r (u - mean(u) - xh mean(u xh)),  u = w dy,  xh = (x - m) r;   dw = sum xh dy,  db = sum dy
//
// A row is held in the registers of LPR threads, EPL elements each, so x (and dy) is read once and
// the variance is the mean of squared deviations from a mean that is already known.  LPR <= 32: a row
// per part of a warp, sums by shuffles; LPR >= 64: a row per CTA.  All sums are fp32.
// Both directions are bound by HBM: the forward moves 2 d elements per row, the backward 3 d.  A row's
// reductions are a chain of latencies, so the next rows' loads are issued before them; its arithmetic is packed
// (two fp32 per instruction: with one, issue bounds the kernels before HBM does); and the launch has as
// many CTAs as are resident at once (a second, partial wave cost up to a third).  bf16: 16384 x 16 rows of 128
// take 26.9 us (5.1 TB/s), their gradient 39.0 (5.2); the gradient of 16384 rows of 4096 87.7 (4.6), of which the sums
// of the CTAs' shares of dw and db 7.
//
// dw and db: a row's threads always own the same columns of the same group, so each keeps its columns'
// two sums in registers over all the rows it walks; the CTA's rows join in shared memory, and the CTA
// writes one share per column to the workspace, which a second launch adds in a fixed order.  No
// atomics: the result does not depend on the order in which CTAs run.
#include "kdn_common.cuh"
#include "kdn_launch.h"

namespace kdn {

namespace {

constexpr int kMaxBlocks = 148 * 8;   // CTAs of a launch (backward: shares of dw, db in the workspace)

// VEC elements as they are in memory (16 bytes, a pair of bf16, or one element), and widened
template <typename T, int VEC> struct Raw { typedef uint4 type; };
template <> struct Raw<float, 1> { typedef float type; };
template <> struct Raw<bf16, 1> { typedef unsigned short type; };
template <> struct Raw<bf16, 2> { typedef unsigned type; };
template <typename T, int VEC>
__device__ __forceinline__ typename Raw<T, VEC>::type load_raw(const T *src) {
    return __ldg(reinterpret_cast<const typename Raw<T, VEC>::type *>(src));
}
template <typename T, int VEC>
__device__ __forceinline__ void widen(float *dst, const typename Raw<T, VEC>::type &u) {
    if constexpr (VEC == 8) {
        const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            dst[2 * i] = __uint_as_float(w[i] << 16);
            dst[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else if constexpr (VEC == 4) {
        dst[0] = __uint_as_float(u.x); dst[1] = __uint_as_float(u.y);
        dst[2] = __uint_as_float(u.z); dst[3] = __uint_as_float(u.w);
    } else if constexpr (VEC == 2) {
        dst[0] = __uint_as_float(u << 16);
        dst[1] = __uint_as_float(u & 0xffff0000u);
    } else if constexpr (sizeof(T) == 4) {
        dst[0] = u;
    } else {
        dst[0] = __uint_as_float((unsigned)u << 16);
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T *dst, const float *src) {
    if constexpr (VEC == 8) {
        uint4 u;
        unsigned *w = reinterpret_cast<unsigned *>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __nv_bfloat162 h = __floats2bfloat162_rn(src[2 * i], src[2 * i + 1]);
            w[i] = *reinterpret_cast<unsigned *>(&h);
        }
        *reinterpret_cast<uint4 *>(dst) = u;
    } else if constexpr (VEC == 4) {
        stf4(dst, make_float4(src[0], src[1], src[2], src[3]));
    } else if constexpr (VEC == 2) {
        *reinterpret_cast<__nv_bfloat162 *>(dst) = __floats2bfloat162_rn(src[0], src[1]);
    } else {
        stf(dst, src[0]);
    }
}

template <int LPR>
struct Shape {
    static constexpr int NT = LPR <= 32 ? 256 : LPR;
    static constexpr int ROWS = NT / LPR;                // rows of a CTA at a time
    // CTAs per SM that the registers must allow: 768 threads forwards, 512 backwards
    static constexpr int FWD = NT >= 768 ? 1 : 768 / NT, BWD = NT >= 512 ? 1 : 512 / NT;
};

// A thread's rows on their way: NA arrays' elements of its columns and NS fp32 values per row.  Rows within a warp are
// copied, if in 16-byte pieces, to slots of the thread's own in shared memory, DEPTH rows ahead, which costs no registers and, as
// no other thread reads them, no barrier (16384 x 16 rows of 128: 28.7 -> 26.9 us, the gradient 42.9 -> 39.1).  Rows over
// a CTA, and pieces of other sizes, wait in registers, one row ahead: there a barrier per row sets the pace, and
// the detour costs more than it brings (gradient of 16384 x 4096: 88 us, through shared memory 91).
__device__ __forceinline__ void copy16(void *dst, const void *src, bool there) {   // (zeros where there is no element)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(void *dst, const void *src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src), "r"(there ? 4 : 0) : "memory");
}
template <typename T, int VEC, int LPR, int EPL, int NA, int NS>
struct Ahead {
    static constexpr bool ASYNC = VEC * sizeof(T) == 16 && LPR <= 32;
    static constexpr int NT = Shape<LPR>::NT, NV = EPL / VEC, ROW = NT * (NA * NV * 16 + NS * 4);
    static constexpr int ROOM = 110 * 1024 / ROW;          // two CTAs per SM
    static constexpr int DEPTH = !ASYNC ? 1 : ROOM < 4 ? ROOM : 4;
    static constexpr size_t BYTES = ASYNC ? (size_t)DEPTH * ROW : 0;
    static_assert(DEPTH >= 1, "shared memory");
    typedef typename Raw<T, VEC>::type raw_t;
    uint8_t *mem;
    int turn = 0;
    raw_t raw[ASYNC ? 1 : NA * NV] = {};
    float val[ASYNC || NS == 0 ? 1 : NS] = {};

    __device__ __forceinline__ uint4 *piece(int st, int k) const { return reinterpret_cast<uint4 *>(mem) + (st * NA * NV + k) * NT + threadIdx.x; }
    __device__ __forceinline__ float *value(int st, int k) const {
        return reinterpret_cast<float *>(mem + (size_t)DEPTH * NA * NV * NT * 16) + (st * NS + k) * NT + threadIdx.x;
    }
    // row `row` of the arrays, if it is there; zeros where there is no row or no element
    __device__ __forceinline__ void fetch(const void *const (&arr)[NA], const float *const (&vals)[NS > 0 ? NS : 1], size_t row, int d, int lane, bool there) {
        if constexpr (ASYNC) {
#pragma unroll
            for (int n = 0; n < NA; ++n) {
                const T *base = static_cast<const T *>(arr[n]) + (there ? row * d : 0);
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int c = (j * LPR + lane) * VEC;
                    copy16(piece(turn, n * NV + j), there && c < d ? base + c : base, there && c < d);
                }
            }
#pragma unroll
            for (int n = 0; n < NS; ++n) copy4(value(turn, n), vals[n] + (there ? row : 0), there);
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (++turn == DEPTH) turn = 0;
        } else {
            if (!there) {
#pragma unroll
                for (int k = 0; k < NA * NV; ++k) raw[k] = raw_t();
#pragma unroll
                for (int n = 0; n < NS; ++n) val[n] = 0.f;
                return;
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * LPR + lane) * VEC;
                if (c >= d) continue;
#pragma unroll
                for (int n = 0; n < NA; ++n) raw[n * NV + j] = load_raw<T, VEC>(static_cast<const T *>(arr[n]) + row * d + c);
            }
#pragma unroll
            for (int n = 0; n < NS; ++n) val[n] = __ldg(vals[n] + row);
        }
    }
    // the row fetched DEPTH calls ago
    __device__ __forceinline__ void take(float (&x)[NA][EPL], float (&v)[NS > 0 ? NS : 1]) {
        if constexpr (ASYNC) asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
#pragma unroll
        for (int n = 0; n < NA; ++n)
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if constexpr (ASYNC) widen<T, VEC>(x[n] + j * VEC, *piece(turn, n * NV + j));
                else widen<T, VEC>(x[n] + j * VEC, raw[n * NV + j]);
            }
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            if constexpr (ASYNC) v[n] = *value(turn, n);
            else v[n] = val[n];
        }
    }
};

// N sums over the LPR threads of a row; every one of them gets them.  Over a CTA: one barrier, on two buffers in
// turn (who writes a buffer again has passed a barrier that its readers reached after reading)
template <int LPR, int N>
struct RowSum {
    float (*red)[N][LPR > 32 ? LPR / 32 : 1];   // [2][N][warps]
    int turn = 0;
    __device__ __forceinline__ void operator()(float (&x)[N]) {
#pragma unroll
        for (int o = (LPR < 32 ? LPR : 32) / 2; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
        if constexpr (LPR > 32) {
            turn ^= 1;
            if ((threadIdx.x & 31) == 0) {
#pragma unroll
                for (int i = 0; i < N; ++i) red[turn][i][threadIdx.x >> 5] = x[i];
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < N; ++i) {
                x[i] = 0.f;
#pragma unroll
                for (int w = 0; w < LPR / 32; ++w) x[i] += red[turn][i][w];
            }
        }
    }
};

// the rows of a group that a thread's place in its CTA walks: i = first, first + step, ... < n (all threads of a CTA
// take the same number of turns: the sums over a row shuffle or synchronise)
template <int LPR>
struct Rows {
    long long first, step;
    __device__ __forceinline__ Rows(const NormArgs &a)
        : first((long long)(blockIdx.x / a.G) * Shape<LPR>::ROWS), step((long long)(gridDim.x / a.G) * Shape<LPR>::ROWS) {}
};

// A CTA serves one group.
template <typename T, int VEC, int LPR, int EPL>
__global__ void __launch_bounds__(Shape<LPR>::NT, Shape<LPR>::FWD) norm_kernel(NormArgs a)
{
    constexpr int NV = EPL / VEC;
    __shared__ float red[2][1][LPR > 32 ? LPR / 32 : 1];
    RowSum<LPR, 1> sum{red};
    const int g = blockIdx.x % a.G, lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
    const Rows<LPR> rows(a);
    const float width = (float)a.d, inv = 1.f / width;
    f32x2 w[EPL / 2], b[EPL / 2];
    auto param = [&](const float *p, int e, float other) {
        const int c = (e / VEC * LPR + lane) * VEC + e % VEC;
        return p && c < a.d ? __ldg(p + (size_t)g * a.d + c) : other;
    };
#pragma unroll
    for (int e = 0; e < EPL; e += 2) {
        w[e / 2] = pk2(param(a.weight, e, 1.f), param(a.weight, e + 1, 1.f));
        b[e / 2] = pk2(param(a.bias, e, 0.f), param(a.bias, e + 1, 0.f));
    }
    extern __shared__ __align__(16) uint8_t mem[];
    typedef Ahead<T, VEC, LPR, EPL, 1, 0> Next;
    Next next{mem};
    auto fetch = [&](long long i0) { next.fetch({a.x}, {nullptr}, (size_t)(i0 + sub) * a.G + g, a.d, lane, i0 + sub < a.n); };
#pragma unroll
    for (int k = 0; k < Next::DEPTH; ++k) fetch(rows.first + k * rows.step);
    for (long long i0 = rows.first; i0 < a.n; i0 += rows.step) {
        const long long i = i0 + sub;
        float vs[1][EPL], none[1], s[1];
        next.take(vs, none);               // (zero behind the row's end)
        fetch(i0 + Next::DEPTH * rows.step);
        const float (&v)[EPL] = vs[0];
        f32x2 x[EPL / 2], s2 = 0;
#pragma unroll
        for (int e = 0; e < EPL / 2; ++e) {
            x[e] = pk2(v[2 * e], v[2 * e + 1]);
            s2 = add2(s2, x[e]);
        }
        s[0] = x2(s2) + y2(s2);
        sum(s);
        const float mean = s[0] / width;      // (not a product with 1 / d: a constant row's mean is its value)
        const f32x2 mean2 = pk2(mean, mean);
        s2 = 0;
#pragma unroll
        for (int e = 0; e < EPL / 2; ++e) {
            x[e] = sub2(x[e], mean2);
            const f32x2 in = pk2((2 * e / VEC * LPR + lane) * VEC < a.d ? x2(x[e]) : 0.f,
                                 ((2 * e + 1) / VEC * LPR + lane) * VEC < a.d ? y2(x[e]) : 0.f);
            s2 = fma2(in, in, s2);
        }
        s[0] = x2(s2) + y2(s2);
        sum(s);
        const float rstd = rsqrtf(fmaf(s[0], inv, a.eps));
        const f32x2 rstd2 = pk2(rstd, rstd);
        if (i >= a.n) continue;
        const size_t row = (size_t)i * a.G + g;
        T *y = static_cast<T *>(a.y) + row * a.d;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LPR + lane) * VEC;
            if (c >= a.d) continue;
            float o[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int k = (j * VEC + e) / 2;
                const f32x2 r = fma2(mul2(x[k], rstd2), w[k], b[k]);
                o[e] = (j * VEC + e) % 2 ? y2(r) : x2(r);
            }
            store_vec<T, VEC>(y + c, o);
        }
        if (lane == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

template <typename T, int VEC, int LPR, int EPL>
__global__ void __launch_bounds__(Shape<LPR>::NT, Shape<LPR>::BWD) norm_backward_kernel(NormArgs a)
{
    constexpr int ROWS = Shape<LPR>::ROWS, NV = EPL / VEC;
    __shared__ float red[2][2][LPR > 32 ? LPR / 32 : 1];
    __shared__ float join[ROWS > 1 ? ROWS : 1][ROWS > 1 ? LPR * VEC : 1];
    RowSum<LPR, 2> sum{red};
    const int g = blockIdx.x % a.G, lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
    const Rows<LPR> rows(a);
    const float inv = 1.f / (float)a.d;
    f32x2 w[EPL / 2], dw[EPL / 2], db[EPL / 2];
    auto param = [&](int e) {
        const int c = (e / VEC * LPR + lane) * VEC + e % VEC;
        return a.weight && c < a.d ? __ldg(a.weight + (size_t)g * a.d + c) : 1.f;
    };
#pragma unroll
    for (int e = 0; e < EPL / 2; ++e) {
        w[e] = pk2(param(2 * e), param(2 * e + 1));
        dw[e] = db[e] = 0;
    }
    // a place without an element or a row holds zeros: dy's make every term of it vanish, but for 0 times an xh that has left
    // fp32's range (a large mean in a row that hardly varies), which is looked for behind the sum
    extern __shared__ __align__(16) uint8_t mem[];
    typedef Ahead<T, VEC, LPR, EPL, 2, 2> Next;
    Next next{mem};
    auto fetch = [&](long long i0) {
        next.fetch({a.x, a.dy}, {a.mean, a.rstd}, (size_t)(i0 + sub) * a.G + g, a.d, lane, i0 + sub < a.n);
    };
#pragma unroll
    for (int k = 0; k < Next::DEPTH; ++k) fetch(rows.first + k * rows.step);
    for (long long i0 = rows.first; i0 < a.n; i0 += rows.step) {
        const long long i = i0 + sub;
        float in[2][EPL], stat[2], s[2];
        next.take(in, stat);
        fetch(i0 + Next::DEPTH * rows.step);
        const float (&vx)[EPL] = in[0], (&vy)[EPL] = in[1];
        const f32x2 mean2 = pk2(stat[0], stat[0]), rstd2 = pk2(stat[1], stat[1]);
        f32x2 xh[EPL / 2], u[EPL / 2], s1 = 0, s2 = 0;
#pragma unroll
        for (int e = 0; e < EPL / 2; ++e) {
            xh[e] = mul2(sub2(pk2(vx[2 * e], vx[2 * e + 1]), mean2), rstd2);
            u[e] = pk2(vy[2 * e], vy[2 * e + 1]);
            dw[e] = fma2(xh[e], u[e], dw[e]);
            db[e] = add2(db[e], u[e]);
            u[e] = mul2(u[e], w[e]);
            s1 = add2(s1, u[e]);
            s2 = fma2(u[e], xh[e], s2);
        }
        s[0] = x2(s1) + y2(s1);
        s[1] = x2(s2) + y2(s2);
        if (__builtin_expect(s[1] != s[1], 0)) {
            s[1] = 0.f;
#pragma unroll
            for (int e = 0; e < EPL / 2; ++e) {
                if ((2 * e / VEC * LPR + lane) * VEC < a.d) s[1] = fmaf(x2(u[e]), x2(xh[e]), s[1]);
                if (((2 * e + 1) / VEC * LPR + lane) * VEC < a.d) s[1] = fmaf(y2(u[e]), y2(xh[e]), s[1]);
            }
        }
        sum(s);
        if (i >= a.n) continue;
        const f32x2 m1 = pk2(s[0] * inv, s[0] * inv), m2 = pk2(-s[1] * inv, -s[1] * inv);
        T *dx = static_cast<T *>(a.dx) + ((size_t)i * a.G + g) * a.d;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LPR + lane) * VEC;
            if (c >= a.d) continue;
            float o[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int k = (j * VEC + e) / 2;
                const f32x2 r = mul2(rstd2, fma2(xh[k], m2, sub2(u[k], m1)));
                o[e] = (j * VEC + e) % 2 ? y2(r) : x2(r);
            }
            store_vec<T, VEC>(dx + c, o);
        }
    }
    asm volatile("griddepcontrol.launch_dependents;");
    if (!a.part) return;
    // the CTA's share: [CTA][2][d]
    auto value = [&](int which, int e) { const f32x2 p = which ? db[e / 2] : dw[e / 2]; return e % 2 ? y2(p) : x2(p); };
    float *part = a.part + (size_t)blockIdx.x * 2 * a.d;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (ROWS > 1) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < VEC; ++e) join[sub][lane * VEC + e] = value(which, j * VEC + e);
                __syncthreads();
                for (int c = threadIdx.x; c < LPR * VEC; c += Shape<LPR>::NT) {
                    float s = 0.f;
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) s += join[r][c];
                    if (j * LPR * VEC + c < a.d) part[which * a.d + j * LPR * VEC + c] = s;
                }
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int c = (j * LPR + lane) * VEC + e;
                    if (c < a.d) part[which * a.d + c] = value(which, j * VEC + e);
                }
            }
        }
    }
}

// dw (blockIdx.z = 0) and db (1) [G, d] from the CTAs' shares: thread = (column, one of 32 parts of the CTAs)
__global__ void __launch_bounds__(1024) norm_params_kernel(NormArgs a, int blocks)
{
    __shared__ float red[32][33];
    const int g = blockIdx.y, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, part = threadIdx.x >> 5;
    float *out = blockIdx.z ? a.dbias : a.dweight;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // (launched while the rows' kernel runs out)
    if (!out) return;
    float s = 0.f;
    if (c < a.d) {
        const float *p = a.part + (size_t)blockIdx.z * a.d + c;
#pragma unroll 8
        for (int b = g + part * a.G; b < blocks; b += 32 * a.G) s += __ldcg(p + (size_t)b * 2 * a.d);   // (not __ldg: written while this kernel waited)
    }
    red[part][lane] = s;
    __syncthreads();
    // warp w joins the parts of column w
    s = warp_sum(red[lane][part]);
    const int cw = blockIdx.x * 32 + part;
    if (lane == 0 && cw < a.d) out[(size_t)g * a.d + cw] = s;
}

// CTAs of a launch: as many as are resident at once, a multiple of the groups, no more than the rows need
template <typename K>
cudaError_t blocks_for(K kern, size_t smem, int threads, const NormArgs &a, int rows, int *blocks) {
    KernelSetup ks;
    const cudaError_t e = kernel_setup(reinterpret_cast<const void *>(kern), smem, threads, false, &ks);
    if (e != cudaSuccess) return e;
    long long per = (long long)ks.sms * ks.blocks_per_sm;
    if (per > kMaxBlocks) per = kMaxBlocks;
    per /= a.G;
    if (per < 1) per = 1;
    const long long need = (a.n + rows - 1) / rows;
    *blocks = (int)((per < need ? per : need) * a.G);
    return cudaSuccess;
}

template <typename T, int VEC, int LPR, int EPL>
cudaError_t run(const NormArgs &a, bool back, cudaStream_t st) {
    using Sh = Shape<LPR>;
    int blocks = 0;
    auto kern = back ? norm_backward_kernel<T, VEC, LPR, EPL> : norm_kernel<T, VEC, LPR, EPL>;
    const size_t smem = back ? Ahead<T, VEC, LPR, EPL, 2, 2>::BYTES : Ahead<T, VEC, LPR, EPL, 1, 0>::BYTES;
    cudaError_t e = blocks_for(kern, smem, Sh::NT, a, Sh::ROWS, &blocks);
    if (e != cudaSuccess) return e;
    e = launch(kern, dim3((unsigned)blocks), Sh::NT, smem, st, a);
    if (e != cudaSuccess || !back || !a.part) return e;
    return launch_next(norm_params_kernel, dim3((a.d + 31) / 32, a.G, 2), 1024, 0, st, a, blocks);
}

// Within a warp 16 elements per thread (8 for the narrowest rows): against 8, a row of 128 costs a quarter fewer
// instructions, which is what bounds short rows.  Across a CTA the rows in flight per SM count, so CTAs are small: 16
// elements per thread against 8 bring rows of 2048 bf16 from 21.6 to 15.9 us (10000 of them; gradient of 15000 x 1602 from
// 65 to 43).  Odd widths, an element per load, are bound by their instructions, and 8 per thread are quicker (20000 x 1001
// bf16 24.7 us against 31.2).  Above 8192 the 1024 threads of a row have 64 registers each, and the gradient spills: 2048
// rows of 16384 bf16 take 134 us (forward 39), 4096 of 8192 61.
template <typename T, int VEC>
cudaError_t by_width(const NormArgs &a, bool back, cudaStream_t st) {
    if (a.d <= 64) return run<T, VEC, 8, 8>(a, back, st);
    if (a.d <= 128) return run<T, VEC, 8, 16>(a, back, st);
    if (a.d <= 256) return run<T, VEC, 16, 16>(a, back, st);
    if (a.d <= 512) return run<T, VEC, 32, 16>(a, back, st);
    constexpr int N = VEC > 1 ? 16 : 8;    // elements per thread
    if (a.d <= 1024) return run<T, VEC, 1024 / N, N>(a, back, st);
    if (a.d <= 2048) return run<T, VEC, 2048 / N, N>(a, back, st);
    if (a.d <= 4096) return run<T, VEC, 256, 16>(a, back, st);
    if (a.d <= 8192) return run<T, VEC, 512, 16>(a, back, st);
    return run<T, VEC, 1024, 16>(a, back, st);
}
// (bf16 rows of an even width in pairs: 50000 x 510 21.4 us, element by element 38.6)
cudaError_t by_type(const NormArgs &a, bool bf16_in, bool back, cudaStream_t st) {
    if (bf16_in) {
        if (a.d % 8 == 0) return by_width<bf16, 8>(a, back, st);
        return a.d % 2 == 0 ? by_width<bf16, 2>(a, back, st) : by_width<bf16, 1>(a, back, st);
    }
    return a.d % 4 == 0 ? by_width<float, 4>(a, back, st) : by_width<float, 1>(a, back, st);
}

}  // namespace

size_t norm_backward_workspace_bytes(long long n, int G, int d) {
    return (size_t)(G > kMaxBlocks ? G : kMaxBlocks / G * G) * 2 * d * sizeof(float);
}
cudaError_t launch_norm(const NormArgs &a, bool bf16_in, cudaStream_t st) { return by_type(a, bf16_in, false, st); }
cudaError_t launch_norm_backward(const NormArgs &a, bool bf16_in, cudaStream_t st) { return by_type(a, bf16_in, true, st); }

}  // namespace kdn
