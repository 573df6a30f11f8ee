// Root-mean-square norms around a block with its gate and residual scale, forward and backward.
//
// With rows r of canvas b = r / C, n(v) = v rsqrt(mean(v^2) + eps) over the d columns:
//   x'_r = x_r + s g_b w_post n(y_r)         (after the block; g_b = 1 without a gate)
//   h_r  = w_pre n(x'_r)                     (before the next block)
// and, from the gradients dx' (residual stream) and dh, with v = y rstd_y, m = x' rstd_x,
// t = dh w_pre, c = s g_b w_post:
//   dx = dx' + rstd_x (t - m mean(t m))
//   dy = rstd_y (c dx - v mean(c dx v))
//   dw_pre = sum_r dh m,  P_b = sum_{r in b} dx v,  dw_post = s sum_b g_b P_b,  dgate_b = s w_post P_b.
// Sums, statistics and everything between a load and a store are fp32; x', h, dx and dy are rounded
// once, to the activations' type (h is taken of the unrounded x').
#include <algorithm>

#include "common.cuh"
#include "kernels.cuh"

namespace dg {

namespace {

// Sixteen bytes of a row: 8 bf16 or 4 fp32 values.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int kN = 4;
    static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                          pack_bf16x2(f[6], f[7]));
    }
};

template <typename T>
__device__ __forceinline__ uint4 load16(const T* p) {
    return *reinterpret_cast<const uint4*>(p);
}
// kN parameters (weights, a gate row) as fp32: kN fp32 or bf16 values, kN * sizeof(P)-byte aligned.
template <int kN>
__device__ __forceinline__ void load_params(const float* p, float (&f)[kN]) {
#pragma unroll
    for (int i = 0; i < kN; i += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
        f[i] = v.x;
        f[i + 1] = v.y;
        f[i + 2] = v.z;
        f[i + 3] = v.w;
    }
}
template <int kN>
__device__ __forceinline__ void load_params(const __nv_bfloat16* p, float (&f)[kN]) {
#pragma unroll
    for (int i = 0; i < kN; i += 4) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p + i));
        f[i] = bf16_lo(v.x);
        f[i + 1] = bf16_hi(v.x);
        f[i + 2] = bf16_lo(v.y);
        f[i + 3] = bf16_hi(v.y);
    }
}

// kV sums over the threads of one row, every thread receiving all of them.  kWarps warps per row
// (1: no barrier); `sh` holds kV * kWarps floats and is not reused before the next barrier.
template <int kWarps, int kV>
__device__ __forceinline__ void row_sums(float (&v)[kV], float* sh) {
#pragma unroll
    for (int i = 0; i < kV; ++i) v[i] = warp_sum(v[i]);
    if (kWarps == 1) return;
    const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
    if (l == 0) {
#pragma unroll
        for (int i = 0; i < kV; ++i) sh[i * kWarps + w] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kV; ++i) v[i] = warp_sum(l < kWarps ? sh[i * kWarps + l] : 0.f);
}

// 1 / sqrt(mean f^2 + eps) of a row held in its threads' registers.  Squares leave fp32's range where values
// are beyond about 1e19 or, with hardly any eps, below 1e-15; such a row (the choice is the same in all
// its threads) is summed again in fp64.
template <int kWarps, int kNV, int kN>
__device__ __forceinline__ float row_rstd(const float (&f)[kNV][kN], float inv_d, float eps, float* sh, double* sh64) {
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < kNV; ++k)
#pragma unroll
        for (int i = 0; i < kN; ++i) s[0] = fmaf(f[k][i], f[k][i], s[0]);
    row_sums<kWarps>(s, sh);
    const float ms = fmaf(s[0], inv_d, eps);
    if (ms > 1e-30f && ms < INFINITY) return 1.0f / sqrtf(ms);
    double a = 0.0;
#pragma unroll
    for (int k = 0; k < kNV; ++k)
#pragma unroll
        for (int i = 0; i < kN; ++i) a = fma(static_cast<double>(f[k][i]), static_cast<double>(f[k][i]), a);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (kWarps > 1) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0) sh64[threadIdx.x >> 5] = a;
        __syncthreads();
        a = 0.0;
        for (int w = 0; w < kWarps; ++w) a += sh64[w];
    }
    return static_cast<float>(1.0 / sqrt(fma(a, static_cast<double>(inv_d), static_cast<double>(eps))));
}

// ------------------------------------------------------------------------------------ forward
// One row per group of kWarps warps, kNV 16-byte vectors per thread, everything in registers: each
// input is read once.  kWarps == 1: four rows per CTA, no barrier; else one row per CTA.
template <typename T, typename P, int kWarps, int kNV>
__global__ void __launch_bounds__(kWarps == 1 ? 128 : 32 * kWarps) block_norm_kernel(const __grid_constant__ BlockNormParams p) {
    constexpr int kN = Vec<T>::kN;
    constexpr int kThreads = 32 * kWarps;
    __shared__ float sh[2][kWarps];
    __shared__ double sh64[kWarps];
    const int64_t r = kWarps == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5) : blockIdx.x;
    if (r >= p.R) return;  // kWarps == 1 only: a whole warp leaves
    const int t = kWarps == 1 ? threadIdx.x & 31 : threadIdx.x;
    const int n_vec = p.d / kN;
    const T* x = static_cast<const T*>(p.x) + r * p.ld_x;
    float fx[kNV][kN];
    {
        uint4 v[kNV];
#pragma unroll
        for (int k = 0; k < kNV; ++k) {
            const int c = t + k * kThreads;
            v[k] = c < n_vec ? load16(x + c * kN) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < kNV; ++k) Vec<T>::unpack(v[k], fx[k]);
    }
    const float inv_d = 1.0f / static_cast<float>(p.d);
    if (p.y) {
        const T* y = static_cast<const T*>(p.y) + r * p.ld_y;
        float fy[kNV][kN];
        {
            uint4 v[kNV];
#pragma unroll
            for (int k = 0; k < kNV; ++k) {
                const int c = t + k * kThreads;
                v[k] = c < n_vec ? load16(y + c * kN) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int k = 0; k < kNV; ++k) Vec<T>::unpack(v[k], fy[k]);
        }
        const float rstd = row_rstd<kWarps>(fy, inv_d, p.eps, sh[0], sh64);
        if (t == 0 && p.rstd_y) p.rstd_y[r] = rstd;
        const P* w = static_cast<const P*>(p.w_post);
        const P* g = p.gate ? static_cast<const P*>(p.gate) + (r / p.C) * p.d : nullptr;
        T* xo = static_cast<T*>(p.x_out) + r * p.d;
#pragma unroll
        for (int k = 0; k < kNV; ++k) {
            const int c = t + k * kThreads;
            if (c < n_vec) {
                float fw[kN];
                load_params<kN>(w + c * kN, fw);
                if (g) {
                    float fg[kN];
                    load_params<kN>(g + c * kN, fg);
#pragma unroll
                    for (int i = 0; i < kN; ++i) fw[i] *= fg[i];
                }
#pragma unroll
                for (int i = 0; i < kN; ++i) fx[k][i] = fmaf(p.res_scale * (fy[k][i] * rstd), fw[i], fx[k][i]);
                *reinterpret_cast<uint4*>(xo + c * kN) = Vec<T>::pack(fx[k]);
            }
        }
    }
    if (!p.w_pre) return;
    const float rstd = row_rstd<kWarps>(fx, inv_d, p.eps, sh[1], sh64);
    if (t == 0 && p.rstd_x) p.rstd_x[r] = rstd;
    const P* w = static_cast<const P*>(p.w_pre);
    T* h = static_cast<T*>(p.h) + r * p.d;
#pragma unroll
    for (int k = 0; k < kNV; ++k) {
        const int c = t + k * kThreads;
        if (c < n_vec) {
            float f[kN], fw[kN];
            load_params<kN>(w + c * kN, fw);
#pragma unroll
            for (int i = 0; i < kN; ++i) f[i] = fx[k][i] * rstd * fw[i];
            *reinterpret_cast<uint4*>(h + c * kN) = Vec<T>::pack(f);
        }
    }
}

template <typename T, typename P, int kWarps, int kNV>
cudaError_t launch_forward(const BlockNormParams& p, cudaStream_t st) {
    const unsigned grid = static_cast<unsigned>(kWarps == 1 ? (static_cast<int64_t>(p.R) + 3) / 4 : p.R);
    block_norm_kernel<T, P, kWarps, kNV><<<grid, kWarps == 1 ? 128 : 32 * kWarps, 0, st>>>(p);
    note_launches(1);
    return cudaGetLastError();
}

template <typename T, typename P>
cudaError_t forward_by_width(const BlockNormParams& p, cudaStream_t st) {
    const int n_vec = p.d / Vec<T>::kN;
    if (n_vec <= 32) return launch_forward<T, P, 1, 1>(p, st);
    if (n_vec <= 64) return launch_forward<T, P, 1, 2>(p, st);
    if (n_vec <= 128) return launch_forward<T, P, 2, 2>(p, st);
    if (n_vec <= 256) return launch_forward<T, P, 4, 2>(p, st);
    if (n_vec <= 512) return launch_forward<T, P, 8, 2>(p, st);
    if (n_vec <= 1024) return launch_forward<T, P, 16, 2>(p, st);
    if (n_vec <= 2048) return launch_forward<T, P, 16, 4>(p, st);
    return launch_forward<T, P, 32, 4>(p, st);
}

// ------------------------------------------------------------------------------------ backward
// The second mean needs dx, which needs the first; expanding it,
//   sum c dx v = sum c (dx' + rstd_x t) v - rstd_x mean(t m) sum c m v,
// so the three sums  sum t m,  sum c (dx' + rstd_x t) v,  sum c m v  take one exchange per row.
// A CTA walks a run of rows of one canvas and keeps its columns' sums of dh m and dx v in
// registers; the runs' partial sums go to the workspace and are added in a fixed order.
template <typename T, typename P, int kWarps, int kNV>
__global__ void __launch_bounds__(32 * kWarps) block_norm_backward_kernel(const __grid_constant__ BlockNormBackwardParams p) {
    constexpr int kN = Vec<T>::kN;
    constexpr int kThreads = 32 * kWarps;
    __shared__ float sh[2][3 * kWarps];
    const int t = threadIdx.x;
    const int n_vec = p.d / kN;
    const int b = blockIdx.x / p.runs, run = blockIdx.x - b * p.runs;
    const int64_t r0 = static_cast<int64_t>(b) * p.C + static_cast<int64_t>(run) * p.run_rows;
    const int64_t r1 = min(r0 + p.run_rows, static_cast<int64_t>(b + 1) * p.C);
    const bool pre = p.w_pre != nullptr, post = p.y != nullptr;
    const float inv_d = 1.0f / static_cast<float>(p.d);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    float acc_pre[kNV][kN], acc_post[kNV][kN];
#pragma unroll
    for (int k = 0; k < kNV; ++k)
#pragma unroll
        for (int i = 0; i < kN; ++i) acc_pre[k][i] = acc_post[k][i] = 0.f;

    int parity = 0;
    for (int64_t r = r0; r < r1; ++r, parity ^= 1) {
        uint4 gv[kNV], hv[kNV], xv[kNV], yv[kNV];
#pragma unroll
        for (int k = 0; k < kNV; ++k) {
            const int c = t + k * kThreads;
            const bool in = c < n_vec;
            gv[k] = in && p.dx_out ? load16(static_cast<const T*>(p.dx_out) + r * p.ld_dx_out + c * kN) : zero;
            hv[k] = in && pre ? load16(static_cast<const T*>(p.dh) + r * p.ld_dh + c * kN) : zero;
            xv[k] = in && pre ? load16(static_cast<const T*>(p.x) + r * p.ld_x + c * kN) : zero;
            yv[k] = in && post ? load16(static_cast<const T*>(p.y) + r * p.ld_y + c * kN) : zero;
        }
        const float rx = pre ? p.rstd_x[r] : 0.f, ry = post ? p.rstd_y[r] : 0.f;
        const P* gate = p.gate ? static_cast<const P*>(p.gate) + static_cast<int64_t>(b) * p.d : nullptr;
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < kNV; ++k) {
            const int c = t + k * kThreads;
            if (c < n_vec) {
                float fg[kN], fh[kN], fx[kN], fy[kN], wp[kN], wc[kN];
                Vec<T>::unpack(gv[k], fg);
                Vec<T>::unpack(hv[k], fh);
                Vec<T>::unpack(xv[k], fx);
                Vec<T>::unpack(yv[k], fy);
                if (pre) load_params<kN>(static_cast<const P*>(p.w_pre) + c * kN, wp);
                if (post) load_params<kN>(static_cast<const P*>(p.w_post) + c * kN, wc);
                if (gate) {
                    float g[kN];
                    load_params<kN>(gate + c * kN, g);
#pragma unroll
                    for (int i = 0; i < kN; ++i) wc[i] *= g[i];
                }
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    const float m = fx[i] * rx, tt = pre ? fh[i] * wp[i] : 0.f;
                    s[0] = fmaf(tt, m, s[0]);
                    if (post) {
                        const float cv = wc[i] * (fy[i] * ry);
                        s[1] = fmaf(cv, fmaf(rx, tt, fg[i]), s[1]);
                        s[2] = fmaf(cv, m, s[2]);
                    }
                }
            }
        }
        row_sums<kWarps>(s, sh[parity]);
        const float m1 = s[0] * inv_d;
        const float m2 = p.res_scale * fmaf(-rx * m1, s[2], s[1]) * inv_d;
#pragma unroll
        for (int k = 0; k < kNV; ++k) {
            const int c = t + k * kThreads;
            if (c < n_vec) {
                float fg[kN], fh[kN], fx[kN], fy[kN], wp[kN], wc[kN];
                Vec<T>::unpack(gv[k], fg);
                Vec<T>::unpack(hv[k], fh);
                Vec<T>::unpack(xv[k], fx);
                Vec<T>::unpack(yv[k], fy);
                if (pre) load_params<kN>(static_cast<const P*>(p.w_pre) + c * kN, wp);
                if (post) load_params<kN>(static_cast<const P*>(p.w_post) + c * kN, wc);
                if (gate) {
                    float g[kN];
                    load_params<kN>(gate + c * kN, g);
#pragma unroll
                    for (int i = 0; i < kN; ++i) wc[i] *= g[i];
                }
                float dx[kN], dy[kN];
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    const float m = fx[i] * rx, tt = pre ? fh[i] * wp[i] : 0.f;
                    dx[i] = fmaf(rx, fmaf(-m, m1, tt), fg[i]);
                    acc_pre[k][i] = fmaf(fh[i], m, acc_pre[k][i]);
                    if (post) {
                        const float v = fy[i] * ry;
                        acc_post[k][i] = fmaf(dx[i], v, acc_post[k][i]);
                        dy[i] = ry * fmaf(-v, m2, p.res_scale * wc[i] * dx[i]);
                    }
                }
                *reinterpret_cast<uint4*>(static_cast<T*>(p.dx) + r * p.d + c * kN) = Vec<T>::pack(dx);
                if (post) *reinterpret_cast<uint4*>(static_cast<T*>(p.dy) + r * p.d + c * kN) = Vec<T>::pack(dy);
            }
        }
    }
    grid_launch_dependents();
    // partial sums of the run: [B * runs, d] for each of the two (the absent one is not stored)
#pragma unroll
    for (int k = 0; k < kNV; ++k) {
        const int c = t + k * kThreads;
        if (c < n_vec) {
            const int64_t at = static_cast<int64_t>(blockIdx.x) * p.d + c * kN;
#pragma unroll
            for (int i = 0; i < kN; i += 4) {
                if (pre)
                    *reinterpret_cast<float4*>(p.part_pre + at + i) =
                        make_float4(acc_pre[k][i], acc_pre[k][i + 1], acc_pre[k][i + 2], acc_pre[k][i + 3]);
                if (post)
                    *reinterpret_cast<float4*>(p.part_post + at + i) =
                        make_float4(acc_post[k][i], acc_post[k][i + 1], acc_post[k][i + 2], acc_post[k][i + 3]);
            }
        }
    }
}

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ float4 shfl_add4(float4 v, int o) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
    v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
    return v;
}
__device__ __forceinline__ float4 param4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 param4(const __nv_bfloat16* p) {
    float f[4];
    load_params<4>(p, f);
    return make_float4(f[0], f[1], f[2], f[3]);
}

// Adds the runs' partial sums.  One warp per four columns: `sub` lanes share a canvas (a power of
// two), 32 / sub canvases at a time; every sum has a fixed order.
template <typename P>
__global__ void __launch_bounds__(128) block_norm_params_kernel(const __grid_constant__ BlockNormBackwardParams p, int sub) {
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int c = (blockIdx.x * 4 + (threadIdx.x >> 5)) * 4;
    if (c >= p.d) return;
    if (p.w_pre) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        const int n = p.B * p.runs;
#pragma unroll 4
        for (int j = lane; j < n; j += 32) a = add4(a, __ldcg(reinterpret_cast<const float4*>(p.part_pre + static_cast<int64_t>(j) * p.d + c)));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a = shfl_add4(a, o);
        if (lane == 0) *reinterpret_cast<float4*>(p.dw_pre + c) = a;
    }
    if (p.y) {
        const float4 w = param4(static_cast<const P*>(p.w_post) + c);
        float4 total = make_float4(0.f, 0.f, 0.f, 0.f);
        const int first = lane / sub, l = lane % sub;
        for (int b0 = 0; b0 < p.B; b0 += 32 / sub) {
            const int b = b0 + first;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            if (b < p.B) {
#pragma unroll 4
                for (int j = l; j < p.runs; j += sub)
                    a = add4(a, __ldcg(reinterpret_cast<const float4*>(p.part_post + (static_cast<int64_t>(b) * p.runs + j) * p.d + c)));
            }
            for (int o = sub >> 1; o > 0; o >>= 1) a = shfl_add4(a, o);
            a = make_float4(p.res_scale * a.x, p.res_scale * a.y, p.res_scale * a.z, p.res_scale * a.w);
            if (p.gate && b < p.B) {
                const int64_t at = static_cast<int64_t>(b) * p.d + c;
                const float4 g = param4(static_cast<const P*>(p.gate) + at);
                if (l == 0) *reinterpret_cast<float4*>(p.dgate + at) = make_float4(w.x * a.x, w.y * a.y, w.z * a.z, w.w * a.w);
                a = make_float4(g.x * a.x, g.y * a.y, g.z * a.z, g.w * a.w);
            }
            total = add4(total, a);
        }
        for (int o = 16; o >= sub; o >>= 1) total = shfl_add4(total, o);
        if (lane == 0) *reinterpret_cast<float4*>(p.dw_post + c) = total;
    }
}

template <typename T, typename P, int kWarps, int kNV>
cudaError_t launch_backward(const BlockNormBackwardParams& p, cudaStream_t st) {
    block_norm_backward_kernel<T, P, kWarps, kNV><<<static_cast<unsigned>(p.B) * p.runs, 32 * kWarps, 0, st>>>(p);
    note_launches(1);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    int sub = 32;  // lanes per canvas: as many as keep a canvas for every group of lanes
    while (sub > 1 && 32 / sub < p.B) sub >>= 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.d / 4 + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, block_norm_params_kernel<P>, p, sub);
    if (e != cudaSuccess) return e;
    note_launches(1);
    return cudaGetLastError();
}

template <typename T, typename P>
cudaError_t backward_by_width(const BlockNormBackwardParams& p, cudaStream_t st) {
    const int n_vec = p.d / Vec<T>::kN;
    if (n_vec <= 32) return launch_backward<T, P, 1, 1>(p, st);
    if (n_vec <= 64) return launch_backward<T, P, 2, 1>(p, st);
    if (n_vec <= 128) return launch_backward<T, P, 4, 1>(p, st);
    if (n_vec <= 256) return launch_backward<T, P, 8, 1>(p, st);
    if (n_vec <= 512) return launch_backward<T, P, 16, 1>(p, st);
    if (n_vec <= 1024) return launch_backward<T, P, 16, 2>(p, st);
    if (n_vec <= 2048) return launch_backward<T, P, 32, 2>(p, st);
    return launch_backward<T, P, 32, 4>(p, st);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormParams& p, int act_bf16, int param_bf16, cudaStream_t st) {
    if (act_bf16)
        return param_bf16 ? forward_by_width<__nv_bfloat16, __nv_bfloat16>(p, st) : forward_by_width<__nv_bfloat16, float>(p, st);
    return param_bf16 ? forward_by_width<float, __nv_bfloat16>(p, st) : forward_by_width<float, float>(p, st);
}

// Runs of rows per canvas: about four CTAs of work per SM, never more runs than rows.
int32_t block_norm_runs(int32_t B, int32_t C) {
    const int want = (4 * num_sms() + B - 1) / B;
    return std::max(1, std::min<int32_t>(want, C));
}

cudaError_t launch_block_norm_backward(const BlockNormBackwardParams& p, int act_bf16, int param_bf16, cudaStream_t st) {
    if (act_bf16)
        return param_bf16 ? backward_by_width<__nv_bfloat16, __nv_bfloat16>(p, st) : backward_by_width<__nv_bfloat16, float>(p, st);
    return param_bf16 ? backward_by_width<float, __nv_bfloat16>(p, st) : backward_by_width<float, float>(p, st);
}

}  // namespace dg
