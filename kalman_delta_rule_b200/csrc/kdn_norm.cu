// Layer norm over the last axis of rows [n, G, d], with a weight and a bias row for each of the G
// groups (G = 1: one pair for all rows; G = heads: the norm of a layer's readout), and its gradient:
//     m = mean(x),  r = (mean((x - m)^2) + eps)^{-1/2},  y = (x - m) r w + b
//     dx = r (u - mean(u) - xh mean(u xh)),  u = w dy,  xh = (x - m) r;   dw = sum xh dy,  db = sum dy
//
// A row is held in the registers of LPR threads, EPL elements each, so x (and dy) is read once and
// the variance is the mean of squared deviations from a mean that is already known.  LPR <= 32: a row
// per part of a warp, sums by shuffles; LPR = 256 or 512: a row per CTA.  All sums are fp32.
// Both directions are bound by HBM: the forward moves 2 d elements per row, the backward 3 d.
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

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(float *dst, const T *src) {
    if constexpr (VEC == 8) {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(src));
        const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            dst[2 * i] = __uint_as_float(w[i] << 16);
            dst[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else if constexpr (VEC == 4) {
        const float4 f = ldf4(src);
        dst[0] = f.x; dst[1] = f.y; dst[2] = f.z; dst[3] = f.w;
    } else {
        dst[0] = ldf(src);
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
    } else {
        stf(dst, src[0]);
    }
}

template <int LPR>
struct Shape {
    static constexpr int NT = LPR <= 32 ? 256 : LPR;
    static constexpr int ROWS = NT / LPR;                // rows of a CTA at a time
};

// sum over the LPR threads of a row; every one of them gets it
template <int LPR>
__device__ __forceinline__ float row_sum(float x, float *red) {
#pragma unroll
    for (int o = (LPR < 32 ? LPR : 32) / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if constexpr (LPR > 32) {
        __syncthreads();       // the previous sum has been read
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
        __syncthreads();
        x = 0.f;
#pragma unroll
        for (int w = 0; w < LPR / 32; ++w) x += red[w];
    }
    return x;
}

// A CTA serves one group; its rows are i = first, first + step, ... of the n rows of that group.
template <typename T, int VEC, int LPR, int EPL>
__global__ void __launch_bounds__(Shape<LPR>::NT) norm_kernel(NormArgs a)
{
    constexpr int ROWS = Shape<LPR>::ROWS, NV = EPL / VEC;
    __shared__ float red[LPR > 32 ? LPR / 32 : 1];
    const int g = blockIdx.x % a.G, lane = threadIdx.x % LPR;
    const long long step = (long long)(gridDim.x / a.G) * ROWS;
    const float width = (float)a.d;   // a division, not a product with 1 / d: a constant row's mean is its value
    float w[EPL], b[EPL];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * LPR + lane) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            w[j * VEC + e] = a.weight && c < a.d ? __ldg(a.weight + (size_t)g * a.d + c + e) : 1.f;
            b[j * VEC + e] = a.bias && c < a.d ? __ldg(a.bias + (size_t)g * a.d + c + e) : 0.f;
        }
    }
    // all threads of a CTA take the same number of turns: the sums over a row shuffle or synchronise
    for (long long i0 = (long long)(blockIdx.x / a.G) * ROWS; i0 < a.n; i0 += step) {
        const long long i = i0 + threadIdx.x / LPR;
        const bool live = i < a.n;
        const size_t row = (size_t)(live ? i : 0) * a.G + g;
        const T *x = static_cast<const T *>(a.x) + row * a.d;
        float v[EPL];
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LPR + lane) * VEC;
            if (live && c < a.d) {
                load_vec<T, VEC>(v + j * VEC, x + c);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[j * VEC + e] = 0.f;
            }
        }
#pragma unroll
        for (int e = 0; e < EPL; ++e) s += v[e];
        const float mean = row_sum<LPR>(s, red) / width;
        s = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool in = (j * LPR + lane) * VEC < a.d;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                v[j * VEC + e] -= mean;
                if (in) s = fmaf(v[j * VEC + e], v[j * VEC + e], s);
            }
        }
        const float rstd = rsqrtf(row_sum<LPR>(s, red) / width + a.eps);
        if (!live) continue;
        T *y = static_cast<T *>(a.y) + row * a.d;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LPR + lane) * VEC;
            if (c >= a.d) continue;
            float o[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = fmaf(v[j * VEC + e] * rstd, w[j * VEC + e], b[j * VEC + e]);
            store_vec<T, VEC>(y + c, o);
        }
        if (lane == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

template <typename T, int VEC, int LPR, int EPL>
__global__ void __launch_bounds__(Shape<LPR>::NT) norm_backward_kernel(NormArgs a)
{
    constexpr int ROWS = Shape<LPR>::ROWS, NV = EPL / VEC;
    __shared__ float red[LPR > 32 ? LPR / 32 : 1];
    __shared__ float join[ROWS > 1 ? ROWS : 1][ROWS > 1 ? LPR * VEC : 1];
    const int g = blockIdx.x % a.G, lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
    const long long step = (long long)(gridDim.x / a.G) * ROWS;
    const float width = (float)a.d;
    const bool params = a.part != nullptr;
    float w[EPL], dw[EPL], db[EPL];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * LPR + lane) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            w[j * VEC + e] = a.weight && c < a.d ? __ldg(a.weight + (size_t)g * a.d + c + e) : 1.f;
            dw[j * VEC + e] = db[j * VEC + e] = 0.f;
        }
    }
    for (long long i0 = (long long)(blockIdx.x / a.G) * ROWS; i0 < a.n; i0 += step) {
        const long long i = i0 + sub;
        const bool live = i < a.n;
        const size_t row = (size_t)(live ? i : 0) * a.G + g;
        const T *x = static_cast<const T *>(a.x) + row * a.d, *dy = static_cast<const T *>(a.dy) + row * a.d;
        float xh[EPL], u[EPL];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LPR + lane) * VEC;
            if (live && c < a.d) {
                load_vec<T, VEC>(xh + j * VEC, x + c);
                load_vec<T, VEC>(u + j * VEC, dy + c);
            }
        }
        const float mean = live ? __ldg(a.mean + row) : 0.f, rstd = live ? __ldg(a.rstd + row) : 0.f;
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool in = live && (j * LPR + lane) * VEC < a.d;
#pragma unroll
            for (int e = j * VEC; e < (j + 1) * VEC; ++e) {
                xh[e] = in ? (xh[e] - mean) * rstd : 0.f;
                u[e] = in ? u[e] : 0.f;
                dw[e] = fmaf(xh[e], u[e], dw[e]);
                db[e] += u[e];
                u[e] *= w[e];
                s1 += u[e];
                s2 = fmaf(u[e], xh[e], s2);
            }
        }
        s1 = row_sum<LPR>(s1, red) / width;
        s2 = row_sum<LPR>(s2, red) / width;
        if (!live) continue;
        T *dx = static_cast<T *>(a.dx) + row * a.d;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LPR + lane) * VEC;
            if (c >= a.d) continue;
            float o[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = rstd * (u[j * VEC + e] - s1 - xh[j * VEC + e] * s2);
            store_vec<T, VEC>(dx + c, o);
        }
    }
    if (!params) return;
    // the CTA's share: [CTA][2][d]
    float *part = a.part + (size_t)blockIdx.x * 2 * a.d;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (ROWS > 1) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < VEC; ++e) join[sub][lane * VEC + e] = which ? db[j * VEC + e] : dw[j * VEC + e];
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
                    if (c < a.d) part[which * a.d + c] = which ? db[j * VEC + e] : dw[j * VEC + e];
                }
            }
        }
    }
}

// dw, db [G, d] from the CTAs' shares: thread = (column, one of 8 parts of the CTAs)
__global__ void __launch_bounds__(256) norm_params_kernel(NormArgs a, int blocks)
{
    __shared__ float red[2][8][32];
    const int g = blockIdx.y, c = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
    float s0 = 0.f, s1 = 0.f;
    if (c < a.d)
        for (int b = g + part * a.G; b < blocks; b += 8 * a.G) {
            s0 += a.part[(size_t)b * 2 * a.d + c];
            s1 += a.part[(size_t)b * 2 * a.d + a.d + c];
        }
    red[0][part][threadIdx.x & 31] = s0;
    red[1][part][threadIdx.x & 31] = s1;
    __syncthreads();
    if (part < 2 && c < a.d) {
        float s = 0.f;
#pragma unroll
        for (int p = 0; p < 8; ++p) s += red[part][p][threadIdx.x & 31];
        float *dst = part ? a.dbias : a.dweight;
        if (dst) dst[(size_t)g * a.d + c] = s;
    }
}

// CTAs of a launch: a multiple of the groups, no more than the rows need, at most `most`
int blocks_for(long long n, int G, int rows, int most) {
    const long long need = (n + rows - 1) / rows;
    long long per = most / G;
    if (per < 1) per = 1;
    if (per > need) per = need;
    return (int)(per * G);
}

template <typename T, int VEC, int LPR, int EPL>
cudaError_t run(const NormArgs &a, bool back, cudaStream_t st) {
    using Sh = Shape<LPR>;
    if (!back) {
        const int blocks = blocks_for(a.n, a.G, Sh::ROWS, kMaxBlocks);
        norm_kernel<T, VEC, LPR, EPL><<<blocks, Sh::NT, 0, st>>>(a);
        return cudaGetLastError();
    }
    const int blocks = blocks_for(a.n, a.G, Sh::ROWS, kMaxBlocks);
    norm_backward_kernel<T, VEC, LPR, EPL><<<blocks, Sh::NT, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.part) return e;
    norm_params_kernel<<<dim3((a.d + 31) / 32, a.G), 256, 0, st>>>(a, blocks);
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t by_width(const NormArgs &a, bool back, cudaStream_t st) {
    if (a.d <= 64) return run<T, VEC, 8, 8>(a, back, st);
    if (a.d <= 128) return run<T, VEC, 16, 8>(a, back, st);
    if (a.d <= 256) return run<T, VEC, 32, 8>(a, back, st);
    if (a.d <= 512) return run<T, VEC, 32, 16>(a, back, st);
    if (a.d <= 1024) return run<T, VEC, 32, 32>(a, back, st);
    if (a.d <= 2048) return run<T, VEC, 256, 8>(a, back, st);
    if (a.d <= 4096) return run<T, VEC, 256, 16>(a, back, st);
    if (a.d <= 8192) return run<T, VEC, 256, 32>(a, back, st);
    return run<T, VEC, 512, 32>(a, back, st);
}
cudaError_t launch(const NormArgs &a, bool bf16_in, bool back, cudaStream_t st) {
    if (bf16_in) return a.d % 8 == 0 ? by_width<bf16, 8>(a, back, st) : by_width<bf16, 1>(a, back, st);
    return a.d % 4 == 0 ? by_width<float, 4>(a, back, st) : by_width<float, 1>(a, back, st);
}

}  // namespace

size_t norm_backward_workspace_bytes(long long n, int G, int d) {
    return (size_t)(G > kMaxBlocks ? G : kMaxBlocks / G * G) * 2 * d * sizeof(float);
}
cudaError_t launch_norm(const NormArgs &a, bool bf16_in, cudaStream_t st) { return launch(a, bf16_in, false, st); }
cudaError_t launch_norm_backward(const NormArgs &a, bool bf16_in, cudaStream_t st) { return launch(a, bf16_in, true, st); }

}  // namespace kdn
