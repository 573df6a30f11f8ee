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
//
// Times below are of launches back to back in one graph that rotate over inputs and outputs of 500 MB together,
// so that rows come from memory; those marked [L2] rotate over four sets, which L2 holds where they are small.
#include <algorithm>

#include "common.cuh"
#include "kernels.cuh"
#include "tensor_core.cuh"

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

// 1 / sqrt(x): the hardware's approximation and one Newton step (error about 2^-23).
__device__ __forceinline__ float rsqrt_newton(float x) {
    const float r = rsqrtf(x);
    return r * fmaf(-0.5f * x * r, r, 1.5f);
}

// 1 / sqrt(mean f^2 + eps) of a row held in its threads' registers.  Squares leave fp32's range where values
// are beyond about 1e19 or, with hardly any eps, below 1e-15; such a row (the choice is the same in all
// its threads) is summed again in fp64.
template <int kWarps, int kNV, int kN>
__device__ __forceinline__ float row_rstd(const float (&f)[kNV][kN], float inv_d, float eps, float* sh, double* sh64) {
    float a4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kNV; ++k)
#pragma unroll
        for (int i = 0; i < kN; ++i) a4[i & 3] = fmaf(f[k][i], f[k][i], a4[i & 3]);
    float s[1] = {(a4[0] + a4[1]) + (a4[2] + a4[3])};
    row_sums<kWarps>(s, sh);
    const float ms = fmaf(s[0], inv_d, eps);
    if (ms > 1e-30f && ms < INFINITY) return rsqrt_newton(ms);
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
// input is read once.  kWarps == 1: four rows per CTA, no barrier; else one row per CTA.  Every step is
// rounded as in the ring below, so that a row's results do not depend on the number of rows.  Few rows cost
// the launch and one trip to memory (64 x 256 bf16: 2.4 us); a row too wide for the ring is bound by the
// two sums that stand between its loads and its stores (512 x 16384 fp32: 30.9 us, 4.3 TB/s).
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
                for (int i = 0; i < kN; ++i) fx[k][i] = fmaf(fy[k][i] * rstd, fw[i] * p.res_scale, fx[k][i]);
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

// ------------------------------------------------------------------------------------ rows in a ring
// A group of kW warps walks a run of rows, the next rows' bulk copies in flight in a ring of
// shared-memory slots with a barrier each.  Beside memory it is instructions that bound such a
// walk, so the parameters stay in registers, as fp32 pairs for the packed fma.rn.f32x2, and widths
// that fill every thread's vectors (kFull) have no column checks.  A CTA has kGroups groups, each with
// its own ring and named barrier.  bf16, both norms with a gate, 2048 columns: 256 rows 3.9 us, 4096 rows
// 15.6 us (4.3 TB/s: 7 rows a group barely fill the ring once, and the loads' latency bounds it), 12288 rows
// 38.0 us (5.3 TB/s).  Without the packed arithmetic and with ordinary loads 4096 rows took 18 us where this takes
// 13.7 [L2].  Two CTAs an SM: three, with 80 registers a thread, were no faster.
template <typename T, int kP>
__device__ __forceinline__ void unpack_pairs(const uint4& v, Pair (&p)[kP]) {
    float f[2 * kP];
    Vec<T>::unpack(v, f);
#pragma unroll
    for (int i = 0; i < kP; ++i) p[i] = pair(f[2 * i], f[2 * i + 1]);
}
template <typename T, int kP>
__device__ __forceinline__ uint4 pack_pairs(const Pair (&p)[kP]) {
    float f[2 * kP];
#pragma unroll
    for (int i = 0; i < kP; ++i) unpair(p[i], f[2 * i], f[2 * i + 1]);
    return Vec<T>::pack(f);
}
template <typename P, int kP>
__device__ __forceinline__ void load_pairs(const P* src, Pair (&p)[kP]) {
    float f[2 * kP];
    load_params<2 * kP>(src, f);
#pragma unroll
    for (int i = 0; i < kP; ++i) p[i] = pair(f[2 * i], f[2 * i + 1]);
}

constexpr int kMaxSlots = 8;
constexpr int kNormCtas = 2;  // per SM, of the backward pass: its parameters and sums take 124 registers
template <int kGroups>
struct Rings {
    uint64_t full[kGroups][kMaxSlots];
    WaitCtl wc;
};
template <int kGroups>
__device__ __forceinline__ void rings_init(Rings<kGroups>& rings, long long wait_limit) {
    if (threadIdx.x == 0) {
        for (int g = 0; g < kGroups; ++g)
            for (int s = 0; s < kMaxSlots; ++s) mbar_init(&rings.full[g][s], 1);
        rings.wc.abort = 0;
        rings.wc.limit = wait_limit > 0 ? wait_limit : kWaitLimitCycles;
        fence_barrier_init();
    }
    __syncthreads();
}
// A row that never arrives: the error is recorded, nothing more is fetched, and the walk goes on (its
// waits end at once), so that every thread keeps to the same barriers.  At the end the threads that
// fill slots wait for the last copy that each has issued.
template <int kGroups>
__device__ __forceinline__ void rings_drain(Rings<kGroups>& rings, int group, int slot, int fills) {
    if (fills > 0 && aborted(&rings.wc)) {
        const long long t0 = clock64();
        while (!mbar_try_wait(&rings.full[group][slot], (fills - 1) & 1) && clock64() - t0 < rings.wc.limit) {
        }
    }
    __syncthreads();
}
// Barrier of a group of kW warps.
template <int kW>
__device__ __forceinline__ void group_barrier(int group) {
    if (kW == 1)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * kW) : "memory");
}
// kV sums over the group's threads, every thread receiving all of them; `sh`: kV * kW floats, not
// reused before the group's next barrier.  Every thread has passed a group barrier (kW > 1).
template <int kW, int kV>
__device__ __forceinline__ void group_sums(float (&v)[kV], float* sh, int group) {
#pragma unroll
    for (int i = 0; i < kV; ++i) v[i] = warp_sum(v[i]);
    if (kW == 1) return;
    const int w = (threadIdx.x >> 5) % kW;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int i = 0; i < kV; ++i) sh[i * kW + w] = v[i];
    }
    group_barrier<kW>(group);
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        if (kW % 4 == 0) {
            v[i] = 0.f;
#pragma unroll
            for (int q = 0; q < kW; q += 4) {
                const float4 w4 = *reinterpret_cast<const float4*>(sh + i * kW + q);
                v[i] += (w4.x + w4.y) + (w4.z + w4.w);
            }
        } else {
            v[i] = sh[i * kW];
#pragma unroll
            for (int q = 1; q < kW; ++q) v[i] += sh[i * kW + q];
        }
    }
}
// row_rstd for a group (see there), of values held as pairs or as raw vectors.
template <typename T, int kP>
__device__ __forceinline__ void as_pairs(const Pair (&f)[kP], Pair (&p)[kP]) {
#pragma unroll
    for (int i = 0; i < kP; ++i) p[i] = f[i];
}
template <typename T, int kP>
__device__ __forceinline__ void as_pairs(const uint4& v, Pair (&p)[kP]) {
    unpack_pairs<T>(v, p);
}
template <typename T, int kW, int kNV, typename V>
__device__ __forceinline__ float group_rstd(const V (&v)[kNV], float inv_d, float eps, float* sh, double* sh64, int group) {
    constexpr int kP = Vec<T>::kN / 2;
    Pair two[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < kNV; ++k) {
        Pair f[kP];
        as_pairs<T>(v[k], f);
#pragma unroll
        for (int i = 0; i < kP; ++i) two[i & 1] = fma2(f[i], f[i], two[i & 1]);
    }
    float s[1] = {sum2(two[0]) + sum2(two[1])};
    group_sums<kW>(s, sh, group);
    const float ms = fmaf(s[0], inv_d, eps);
    if (ms > 1e-30f && ms < INFINITY) return rsqrt_newton(ms);
    double a = 0.0;
#pragma unroll
    for (int k = 0; k < kNV; ++k) {
        Pair f[kP];
        as_pairs<T>(v[k], f);
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            float lo, hi;
            unpair(f[i], lo, hi);
            a = fma(static_cast<double>(lo), static_cast<double>(lo), fma(static_cast<double>(hi), static_cast<double>(hi), a));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (kW > 1) {
        group_barrier<kW>(group);
        if ((threadIdx.x & 31) == 0) sh64[(threadIdx.x >> 5) % kW] = a;
        group_barrier<kW>(group);
        a = 0.0;
        for (int w = 0; w < kW; ++w) a += sh64[w];
    }
    return static_cast<float>(1.0 / sqrt(fma(a, static_cast<double>(inv_d), static_cast<double>(eps))));
}

template <typename T, typename P, int kW, int kGroups, int kNV, int kCtas, bool kFull>
__global__ void __launch_bounds__(32 * kW * kGroups, kCtas)
    block_norm_rows_kernel(const __grid_constant__ BlockNormParams p, int slots, int run) {
    constexpr int kN = Vec<T>::kN, kP = kN / 2, kThreads = 32 * kW;
    extern __shared__ __align__(128) uint8_t slots_mem[];
    __shared__ Rings<kGroups> rings;
    __shared__ __align__(16) float sh[kGroups][2][kW];
    __shared__ double sh64[kGroups][kW];
    const int group = threadIdx.x / kThreads, t = threadIdx.x % kThreads;
    const int n_vec = kFull ? kNV * kThreads : p.d / kN, d = kFull ? kNV * kThreads * kN : p.d;
    const bool pre = p.w_pre != nullptr, post = p.y != nullptr;
    const uint32_t row_bytes = static_cast<uint32_t>(d) * sizeof(T), slot_bytes = row_bytes * (post ? 2 : 1);
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * kGroups + group) * run;
    const int r0 = static_cast<int>(min(first, static_cast<int64_t>(p.R))), n = min(run, p.R - r0);
    const float inv_d = 1.0f / static_cast<float>(d);
    uint8_t* ring = slots_mem + group * slots * slot_bytes;
    rings_init(rings, p.wait_limit);
    const int ahead = min(n, slots);  // rows fetched before the walk; slot s is always filled by thread s
    const T* next_x = static_cast<const T*>(p.x) + (static_cast<int64_t>(r0) + (t < ahead ? t : 0)) * p.ld_x;
    const T* next_y = static_cast<const T*>(p.y) + (static_cast<int64_t>(r0) + (t < ahead ? t : 0)) * p.ld_y;
    int fills = 0;
    const auto fetch = [&](int slot) {  // the next row, into a free slot
        if (aborted(&rings.wc)) return;
        uint64_t* bar = &rings.full[group][slot];
        uint8_t* dst = ring + slot * slot_bytes;
        mbar_arrive_expect_tx(bar, slot_bytes);
        bulk_load(dst, next_x, row_bytes, bar);
        if (post) bulk_load(dst + row_bytes, next_y, row_bytes, bar);
        next_x += slots * p.ld_x;
        next_y += slots * p.ld_y;
        ++fills;
    };
    if (t < ahead && !(p.wait_limit > 0 && r0 == 0 && t == 0)) fetch(t);  // (the test hook leaves row 0 out)
    Pair wc[kNV][kP], wpre[kNV][kP];  // res_scale gate w_post, w_pre
    int canvas = r0 / p.C, left = 0;  // rows before wc is of the next canvas
    const auto load_post = [&]() {
        const Pair scale = pair(p.res_scale, p.res_scale);
#pragma unroll
        for (int k = 0; k < kNV; ++k) {
            const int c = t + k * kThreads;
            if (kFull || c < n_vec) {
                load_pairs(static_cast<const P*>(p.w_post) + c * kN, wc[k]);
                if (p.gate && DG_CHECKED(g_device_error, canvas < p.R / p.C)) {
                    Pair g[kP];
                    load_pairs(static_cast<const P*>(p.gate) + static_cast<int64_t>(canvas) * d + c * kN, g);
#pragma unroll
                    for (int j = 0; j < kP; ++j) wc[k][j] = mul2(wc[k][j], g[j]);
                }
#pragma unroll
                for (int j = 0; j < kP; ++j) wc[k][j] = mul2(wc[k][j], scale);
            }
        }
    };
    if (post && n > 0) load_post();  // (a group past the last row has no canvas)
    left = p.gate ? p.C - r0 % p.C : 0x7fffffff;
#pragma unroll
    for (int k = 0; k < kNV; ++k) {
        const int c = t + k * kThreads;
        if (pre && (kFull || c < n_vec)) load_pairs(static_cast<const P*>(p.w_pre) + c * kN, wpre[k]);
    }
    T* xo = static_cast<T*>(p.x_out) + static_cast<int64_t>(r0) * d + t * kN;
    T* h = static_cast<T*>(p.h) + static_cast<int64_t>(r0) * d + t * kN;
    const uint8_t* src0 = ring + t * 16;
    int slot = 0, phase = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i, --left, xo += d, h += d) {
        if (left == 0) {
            ++canvas;
            left = p.C;
            load_post();
        }
        DG_CHECK(g_device_error, r0 + i < p.R && (!p.gate || canvas == (r0 + i) / p.C));
        mbar_wait(&rings.full[group][slot], phase, &rings.wc);
        const uint8_t* src = src0 + slot * slot_bytes;
        Pair fx[kNV][kP], fy[kNV][kP];
        const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < kNV; ++k) {
            const bool in = kFull || t + k * kThreads < n_vec;
            unpack_pairs<T>(in ? *reinterpret_cast<const uint4*>(src + k * (16 * kThreads)) : zero, fx[k]);
            if (post) unpack_pairs<T>(in ? *reinterpret_cast<const uint4*>(src + row_bytes + k * (16 * kThreads)) : zero, fy[k]);
        }
        if (post) {
            const float rstd = group_rstd<T, kW>(fy, inv_d, p.eps, sh[group][0], sh64[group], group);
            if (t == 0 && p.rstd_y) p.rstd_y[r0 + i] = rstd;
            const Pair rstd2 = pair(rstd, rstd);
#pragma unroll
            for (int k = 0; k < kNV; ++k) {
                if (kFull || t + k * kThreads < n_vec) {
#pragma unroll
                    for (int j = 0; j < kP; ++j) fx[k][j] = fma2(mul2(fy[k][j], rstd2), wc[k][j], fx[k][j]);
                    *reinterpret_cast<uint4*>(xo + k * (kN * kThreads)) = pack_pairs<T>(fx[k]);
                }
            }
        }
        float rstd = 0.f;
        if (pre) rstd = group_rstd<T, kW>(fx, inv_d, p.eps, sh[group][1], sh64[group], group);
        // between this barrier and the last row's, the slot and the exchange's floats have been read
        if (kW == 1 || !post || !pre) group_barrier<kW>(group);
        if (t == slot && i + slots < n) fetch(slot);
        if (pre) {
            if (t == 0 && p.rstd_x) p.rstd_x[r0 + i] = rstd;
            const Pair rstd2 = pair(rstd, rstd);
#pragma unroll
            for (int k = 0; k < kNV; ++k) {
                if (kFull || t + k * kThreads < n_vec) {
#pragma unroll
                    for (int j = 0; j < kP; ++j) fx[k][j] = mul2(mul2(fx[k][j], rstd2), wpre[k][j]);
                    *reinterpret_cast<uint4*>(h + k * (kN * kThreads)) = pack_pairs<T>(fx[k]);
                }
            }
        }
        if (++slot == slots) {
            slot = 0;
            phase ^= 1;
        }
    }
    rings_drain(rings, group, t, fills);
}

// kCtas CTAs per SM share its shared memory.
template <typename T, typename P, int kW, int kGroups, int kNV, int kCtas, bool kFull>
cudaError_t launch_rows_as(const BlockNormParams& p, cudaStream_t st) {
    constexpr int kRingBytes = 200 * 1024 / kCtas;
    const int slot = p.d * static_cast<int>(sizeof(T)) * (p.y ? 2 : 1);
    const int64_t groups = static_cast<int64_t>(kCtas) * num_sms() * kGroups;
    const int run = static_cast<int>((p.R + groups - 1) / groups);
    const int slots = std::min({kMaxSlots, run, kRingBytes / (slot * kGroups)});
    const int64_t ctas = (p.R + static_cast<int64_t>(run) * kGroups - 1) / (static_cast<int64_t>(run) * kGroups);
    static DeviceOnce once;
    const cudaError_t attr_err = allow_shared_memory(once, block_norm_rows_kernel<T, P, kW, kGroups, kNV, kCtas, kFull>, kRingBytes);
    if (attr_err != cudaSuccess) return attr_err;
    block_norm_rows_kernel<T, P, kW, kGroups, kNV, kCtas, kFull><<<static_cast<unsigned>(ctas), 32 * kW * kGroups, kGroups * slots * slot, st>>>(p, slots, run);
    note_launches(1);
    return cudaGetLastError();
}
template <typename T, typename P, int kW, int kGroups, int kNV, int kCtas>
cudaError_t launch_rows(const BlockNormParams& p, cudaStream_t st) {
    if (p.d == kNV * kW * 32 * Vec<T>::kN) return launch_rows_as<T, P, kW, kGroups, kNV, kCtas, true>(p, st);
    return launch_rows_as<T, P, kW, kGroups, kNV, kCtas, false>(p, st);
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
    // Which form (us, bf16, both norms with a gate).  Up to 32 vectors a warp has a row, and the direct form's
    // one load per thread is all there is to wait for (256 columns, 64, 4096 and 16384 rows: 2.4, 4.3, 10.8;
    // the ring 2.9, 5.3, 10.5) until the rows are so many that memory is (65536 rows: 33.7, ring 27.6).  Wider,
    // the ring, at any number of rows (2048 columns, 64, 4096 and 16384 rows: 3.0, 15.6, 52.1; direct 3.3,
    // 19.4, 63.4), as long as the parameters of a thread's columns fit its registers and three rows the
    // shared memory.  (The test hook's bounded waits are the ring's.)
    if (n_vec <= 32 && p.R < 256 * num_sms() && p.wait_limit <= 0) return launch_forward<T, P, 1, 1>(p, st);
    if (n_vec <= 32) return launch_rows<T, P, 1, 8, 1, 3>(p, st);
    if (n_vec <= 64) return launch_rows<T, P, 1, 8, 2, 2>(p, st);
    if (n_vec <= 128) return launch_rows<T, P, 2, 4, 2, 2>(p, st);
    if (n_vec <= 256) return launch_rows<T, P, 4, 2, 2, 2>(p, st);
    if (n_vec <= 512) return launch_rows<T, P, 8, 1, 2, 2>(p, st);
    if (n_vec <= 1024) return launch_rows<T, P, 16, 1, 2, 1>(p, st);
    if constexpr (sizeof(T) == 4)  // (bf16 rows have 2048 vectors at most)
        if (n_vec > 2048) return launch_forward<T, P, 32, 4>(p, st);
    return launch_forward<T, P, 16, 4>(p, st);
}

// ------------------------------------------------------------------------------------ backward
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
// The second mean needs dx, which needs the first; expanding it,
//   sum c dx v = sum c (dx' + rstd_x t) v - rstd_x mean(t m) sum c m v,
// so the three sums  sum t m,  sum c (dx' + rstd_x t) v,  sum c m v  take one exchange per row.
// A CTA walks a run of rows of one canvas and keeps its columns' sums of dh m and dx v in registers;
// the runs' partial sums go to the workspace and are added in a fixed order.
// This form is for rows too wide for the ring further down: a row is read twice, from memory (the next
// row is on its way to L2 meanwhile) and then from L1, as registers hold the columns' sums only
// (1024 x 8192 fp32, gated: 61 us, 3.3 TB/s).
template <typename T, typename P, int kWarps, int kNV>
__global__ void __launch_bounds__(32 * kWarps, 1) block_norm_backward_kernel(const __grid_constant__ BlockNormBackwardParams p) {
    constexpr int kN = Vec<T>::kN;
    constexpr int kThreads = 32 * kWarps;
    __shared__ float sh[2][3 * kWarps];
    grid_launch_dependents();  // (the sums' kernel waits for this one's end)
    const int t = threadIdx.x;
    const int n_vec = p.d / kN;
    const int b = blockIdx.x / p.runs, run = blockIdx.x - b * p.runs;
    const int64_t r0 = static_cast<int64_t>(b) * p.C + static_cast<int64_t>(run) * p.run_rows;
    const int64_t r1 = min(r0 + p.run_rows, static_cast<int64_t>(b + 1) * p.C);
    const bool pre = p.w_pre != nullptr, post = p.y != nullptr;
    const float inv_d = 1.0f / static_cast<float>(p.d);
    const P* gate = p.gate ? static_cast<const P*>(p.gate) + static_cast<int64_t>(b) * p.d : nullptr;
    float acc_pre[kNV][kN], acc_post[kNV][kN];
#pragma unroll
    for (int k = 0; k < kNV; ++k)
#pragma unroll
        for (int i = 0; i < kN; ++i) acc_pre[k][i] = acc_post[k][i] = 0.f;

    int parity = 0;
#pragma unroll 1
    for (int64_t r = r0; r < r1; ++r, parity ^= 1) {
        if (t == 0 && r + 1 < r1) {
            const uint32_t bytes = static_cast<uint32_t>(p.d) * sizeof(T);
            if (p.dx_out) prefetch_l2(static_cast<const T*>(p.dx_out) + (r + 1) * p.ld_dx_out, bytes);
            if (pre) prefetch_l2(static_cast<const T*>(p.dh) + (r + 1) * p.ld_dh, bytes);
            if (pre) prefetch_l2(static_cast<const T*>(p.x) + (r + 1) * p.ld_x, bytes);
            if (post) prefetch_l2(static_cast<const T*>(p.y) + (r + 1) * p.ld_y, bytes);
        }
        const float rx = pre ? p.rstd_x[r] : 0.f, ry = post ? p.rstd_y[r] : 0.f;
        // a vector's columns: the gradients, m, v and t = dh w_pre, c = gate w_post (zero where the call has none)
        const auto read = [&](int c, float(&g)[kN], float(&h)[kN], float(&m)[kN], float(&v)[kN], float(&tt)[kN], float(&cc)[kN]) {
            const uint4 zero = make_uint4(0, 0, 0, 0);
            Vec<T>::unpack(p.dx_out ? load16(static_cast<const T*>(p.dx_out) + r * p.ld_dx_out + c * kN) : zero, g);
            Vec<T>::unpack(pre ? load16(static_cast<const T*>(p.dh) + r * p.ld_dh + c * kN) : zero, h);
            Vec<T>::unpack(pre ? load16(static_cast<const T*>(p.x) + r * p.ld_x + c * kN) : zero, m);
            Vec<T>::unpack(post ? load16(static_cast<const T*>(p.y) + r * p.ld_y + c * kN) : zero, v);
            if (pre) load_params<kN>(static_cast<const P*>(p.w_pre) + c * kN, tt);
            if (post) load_params<kN>(static_cast<const P*>(p.w_post) + c * kN, cc);
            if (gate) {
                float f[kN];
                load_params<kN>(gate + c * kN, f);
#pragma unroll
                for (int i = 0; i < kN; ++i) cc[i] *= f[i];
            }
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                m[i] *= rx;
                v[i] *= ry;
                tt[i] = pre ? tt[i] * h[i] : 0.f;
                cc[i] = post ? cc[i] * p.res_scale : 0.f;
            }
        };
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll 2
        for (int k = 0; k < kNV; ++k) {
            const int c = t + k * kThreads;
            if (c < n_vec) {
                float g[kN], h[kN], m[kN], v[kN], tt[kN], cc[kN];
                read(c, g, h, m, v, tt, cc);
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    const float cv = cc[i] * v[i];
                    s[0] = fmaf(tt[i], m[i], s[0]);
                    s[1] = fmaf(cv, fmaf(rx, tt[i], g[i]), s[1]);
                    s[2] = fmaf(cv, m[i], s[2]);
                }
            }
        }
        row_sums<kWarps>(s, sh[parity]);
        const float m1 = s[0] * inv_d, m2 = fmaf(-rx * m1, s[2], s[1]) * inv_d;
#pragma unroll
        for (int k = 0; k < kNV; ++k) {
            const int c = t + k * kThreads;
            if (c < n_vec) {
                float g[kN], h[kN], m[kN], v[kN], tt[kN], cc[kN];
                read(c, g, h, m, v, tt, cc);
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    g[i] = fmaf(rx, fmaf(-m[i], m1, tt[i]), g[i]);  // dx
                    acc_pre[k][i] = fmaf(h[i], m[i], acc_pre[k][i]);
                    acc_post[k][i] = fmaf(g[i], v[i], acc_post[k][i]);
                    cc[i] = ry * fmaf(-v[i], m2, cc[i] * g[i]);  // dy
                }
                *reinterpret_cast<uint4*>(static_cast<T*>(p.dx) + r * p.d + c * kN) = Vec<T>::pack(g);
                if (post) *reinterpret_cast<uint4*>(static_cast<T*>(p.dy) + r * p.d + c * kN) = Vec<T>::pack(cc);
            }
        }
    }
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
__device__ __forceinline__ void store_pairs(float* to, Pair a, Pair b) {
    float4 v;
    unpair(a, v.x, v.y);
    unpair(b, v.z, v.w);
    *reinterpret_cast<float4*>(to) = v;
}

// The same with the rows' bulk copies kept in flight (see block_norm_rows_kernel).  A CTA's rows are of
// one canvas; its groups take them in turn, and their columns' sums are added at the end, in the
// order of the groups.  12288 x 2048 bf16, gated: 61.4 us with the sums below (4.9 TB/s);
// an instruction is issued in 59 % of the cycles, so arithmetic and the exchange of a row's sums bound it as
// much as memory (55 % busy).  1024 x 4096 fp32: 25.5 us, read twice as above 31.  Rows of up to 32 vectors are
// too small for bulk copies (four of 128 bytes a row: 16384 x 64 bf16 took 19.3 us [L2]) and come by loads two rows ahead
// (14.0 [L2], from memory 19.2; three spill).
template <typename T, typename P, int kW, int kGroups, int kNV, int kCtas, bool kFull>
__global__ void __launch_bounds__(32 * kW * kGroups, kCtas)
    block_norm_backward_rows_kernel(const __grid_constant__ BlockNormBackwardParams p, int slots) {
    constexpr int kN = Vec<T>::kN, kP = kN / 2, kThreads = 32 * kW;
    constexpr bool kRing = kNV > 1;  // one vector per thread: rows come straight into registers
    constexpr int kAhead = 2;        // so many of them
    extern __shared__ __align__(128) uint8_t slots_mem[];
    __shared__ Rings<kGroups> rings;
    __shared__ __align__(16) float sh[kGroups][2][3 * kW];
    grid_launch_dependents();  // (the sums' kernel waits for this one's end)
    const int group = threadIdx.x / kThreads, t = threadIdx.x % kThreads;
    const int n_vec = kFull ? kNV * kThreads : p.d / kN, d = kFull ? kNV * kThreads * kN : p.d;
    const int b = blockIdx.x / p.runs, part = blockIdx.x - b * p.runs;
    const int rows = min(p.run_rows, p.C - part * p.run_rows), n = rows > group ? (rows - group + kGroups - 1) / kGroups : 0;
    const int64_t r0 = static_cast<int64_t>(b) * p.C + part * p.run_rows + group;  // then every kGroups-th row
    const bool pre = p.w_pre != nullptr, post = p.y != nullptr, up = p.dx_out != nullptr;
    const float inv_d = 1.0f / static_cast<float>(d);
    // a slot: the rows of dx_out, dh, x and y that the call has
    const uint32_t row_bytes = static_cast<uint32_t>(d) * sizeof(T);
    const uint32_t at_h = up ? row_bytes : 0, at_x = at_h + (pre ? row_bytes : 0), at_y = at_x + (pre ? row_bytes : 0);
    const uint32_t slot_bytes = at_y + (post ? row_bytes : 0);
    uint8_t* ring = slots_mem + group * slots * slot_bytes;
    if (kRing) rings_init(rings, p.wait_limit);
    const int ahead = min(n, slots);  // rows fetched before the walk; slot s is always filled by thread s
    int64_t next = r0 + (t < ahead ? t : 0) * kGroups;
    int fills = 0;
    const auto fetch = [&](int slot) {  // the next row, into a free slot
        if (aborted(&rings.wc)) return;
        uint64_t* bar = &rings.full[group][slot];
        uint8_t* dst = ring + slot * slot_bytes;
        mbar_arrive_expect_tx(bar, slot_bytes);
        if (up) bulk_load(dst, static_cast<const T*>(p.dx_out) + next * p.ld_dx_out, row_bytes, bar);
        if (pre) {
            bulk_load(dst + at_h, static_cast<const T*>(p.dh) + next * p.ld_dh, row_bytes, bar);
            bulk_load(dst + at_x, static_cast<const T*>(p.x) + next * p.ld_x, row_bytes, bar);
        }
        if (post) bulk_load(dst + at_y, static_cast<const T*>(p.y) + next * p.ld_y, row_bytes, bar);
        next += slots * kGroups;
        ++fills;
    };
    // (the test hook leaves the first row out)
    if (kRing && t < ahead && !(p.wait_limit > 0 && blockIdx.x == 0 && threadIdx.x == 0)) fetch(t);
    uint4 row[kAhead][4];
    const auto load_row = [&](int i, uint4(&v)[4]) {
        const int64_t r = r0 + static_cast<int64_t>(i) * kGroups;
        const bool in = i < n && t < n_vec;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        v[0] = in && up ? load16(static_cast<const T*>(p.dx_out) + r * p.ld_dx_out + t * kN) : zero;
        v[1] = in && pre ? load16(static_cast<const T*>(p.dh) + r * p.ld_dh + t * kN) : zero;
        v[2] = in && pre ? load16(static_cast<const T*>(p.x) + r * p.ld_x + t * kN) : zero;
        v[3] = in && post ? load16(static_cast<const T*>(p.y) + r * p.ld_y + t * kN) : zero;
    };
    if (!kRing) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load_row(i, row[i]);
    }
    Pair wp[kNV][kP], wc[kNV][kP], acc_pre[kNV][kP], acc_post[kNV][kP];
    const Pair scale = pair(p.res_scale, p.res_scale);
#pragma unroll
    for (int k = 0; k < kNV; ++k) {
        const int c = t + k * kThreads;
#pragma unroll
        for (int i = 0; i < kP; ++i) wp[k][i] = wc[k][i] = acc_pre[k][i] = acc_post[k][i] = 0;
        if (kFull || c < n_vec) {
            if (pre) load_pairs(static_cast<const P*>(p.w_pre) + c * kN, wp[k]);
            if (post) {
                load_pairs(static_cast<const P*>(p.w_post) + c * kN, wc[k]);
                Pair g[kP];
                if (p.gate) load_pairs(static_cast<const P*>(p.gate) + static_cast<int64_t>(b) * d + c * kN, g);
#pragma unroll
                for (int i = 0; i < kP; ++i) wc[k][i] = mul2(wc[k][i], p.gate ? mul2(scale, g[i]) : scale);
            }
        }
    }
    const float* rstd_x = p.rstd_x + r0;
    const float* rstd_y = p.rstd_y + r0;
    float rx = 0.f, ry = 0.f;  // of the row at hand, read a row ahead
    if (n > 0) {
        if (pre) rx = *rstd_x;
        if (post) ry = *rstd_y;
    }
    T* dxo = static_cast<T*>(p.dx) + r0 * d + t * kN;
    T* dyo = static_cast<T*>(p.dy) + r0 * d + t * kN;
    const uint8_t* src0 = ring + t * 16;
    int slot = 0, phase = 0, parity = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i, parity ^= 1, dxo += kGroups * d, dyo += kGroups * d) {
        const bool more = i + 1 < n;
        rstd_x += kGroups;
        rstd_y += kGroups;
        const float rx_next = pre && more ? *rstd_x : 0.f, ry_next = post && more ? *rstd_y : 0.f;
        const Pair rx2 = pair(rx, rx), ry2 = pair(ry, ry);
        DG_CHECK(g_device_error, (r0 + i * kGroups) / p.C == b && b < p.B);
        if (kRing) mbar_wait(&rings.full[group][slot], phase, &rings.wc);
        const uint8_t* src = src0 + slot * slot_bytes;
        // a vector's columns of the four rows (zero where the call has none)
        const auto read = [&](int k, Pair(&g)[kP], Pair(&h)[kP], Pair(&x)[kP], Pair(&y)[kP]) {
            if (!kRing) {
                unpack_pairs<T>(row[0][0], g);
                unpack_pairs<T>(row[0][1], h);
                unpack_pairs<T>(row[0][2], x);
                unpack_pairs<T>(row[0][3], y);
                return;
            }
            const bool in = kFull || t + k * kThreads < n_vec;
            const uint8_t* at = src + k * (16 * kThreads);
            const uint4 zero = make_uint4(0, 0, 0, 0);
            unpack_pairs<T>(in && up ? *reinterpret_cast<const uint4*>(at) : zero, g);
            unpack_pairs<T>(in && pre ? *reinterpret_cast<const uint4*>(at + at_h) : zero, h);
            unpack_pairs<T>(in && pre ? *reinterpret_cast<const uint4*>(at + at_x) : zero, x);
            unpack_pairs<T>(in && post ? *reinterpret_cast<const uint4*>(at + at_y) : zero, y);
        };
        Pair sum0 = 0, sum1 = 0, sum2_ = 0;
#pragma unroll
        for (int k = 0; k < kNV; ++k) {
            Pair g[kP], h[kP], x[kP], y[kP];
            read(k, g, h, x, y);
#pragma unroll
            for (int j = 0; j < kP; ++j) {
                const Pair m = mul2(x[j], rx2), tt = mul2(h[j], wp[k][j]), cv = mul2(wc[k][j], mul2(y[j], ry2));
                sum0 = fma2(tt, m, sum0);
                sum1 = fma2(cv, fma2(rx2, tt, g[j]), sum1);
                sum2_ = fma2(cv, m, sum2_);
            }
        }
        float s[3] = {sum2(sum0), sum2(sum1), sum2(sum2_)};
        group_sums<kW>(s, sh[group][parity], group);
        if (kW == 1) group_barrier<kW>(group);
        // past this barrier every thread is done with the row before: its slot is free
        const int before = slot == 0 ? slots - 1 : slot - 1;
        if (kRing && t == before && i > 0 && i - 1 + slots < n) fetch(before);
        const float a = -rx * s[0] * inv_d, e = -ry * fmaf(a, s[2], s[1]) * inv_d;
        const Pair a2 = pair(a, a), e2 = pair(e, e);
#pragma unroll
        for (int k = 0; k < kNV; ++k) {
            if (kFull || t + k * kThreads < n_vec) {
                // (read again: kept in registers, the row would spill)
                Pair g[kP], h[kP], x[kP], y[kP], dx[kP], dy[kP];
                read(k, g, h, x, y);
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    const Pair m = mul2(x[j], rx2), v = mul2(y[j], ry2);
                    dx[j] = fma2(a2, m, fma2(rx2, mul2(h[j], wp[k][j]), g[j]));
                    acc_pre[k][j] = fma2(h[j], m, acc_pre[k][j]);
                    acc_post[k][j] = fma2(dx[j], v, acc_post[k][j]);
                    dy[j] = fma2(e2, v, mul2(wc[k][j], mul2(dx[j], ry2)));
                }
                *reinterpret_cast<uint4*>(dxo + k * (kN * kThreads)) = pack_pairs<T>(dx);
                if (post) *reinterpret_cast<uint4*>(dyo + k * (kN * kThreads)) = pack_pairs<T>(dy);
            }
        }
        rx = rx_next;
        ry = ry_next;
        if (!kRing) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int q = 1; q < kAhead; ++q) row[q - 1][j] = row[q][j];
            }
            load_row(i + kAhead, row[kAhead - 1]);
        }
        if (++slot == slots) {
            slot = 0;
            phase ^= 1;
        }
    }
    if (kRing) rings_drain(rings, group, t, fills);
    // the columns' sums: of one group as they are, of more by way of the ring's memory, [2, kGroups, d]
    const int64_t out = static_cast<int64_t>(blockIdx.x) * p.d;
    float* sums = reinterpret_cast<float*>(slots_mem);
    float* to_pre = kGroups == 1 ? p.part_pre + out : sums + group * p.d;
    float* to_post = kGroups == 1 ? p.part_post + out : sums + (kGroups + group) * p.d;
#pragma unroll
    for (int k = 0; k < kNV; ++k) {
        const int c = t + k * kThreads;
        if (kFull || c < n_vec) {
#pragma unroll
            for (int i = 0; i < kP; i += 2) {
                if (pre) store_pairs(to_pre + c * kN + 2 * i, acc_pre[k][i], acc_pre[k][i + 1]);
                if (post) store_pairs(to_post + c * kN + 2 * i, acc_post[k][i], acc_post[k][i + 1]);
            }
        }
    }
    if (kGroups > 1) {
        __syncthreads();
#pragma unroll 1
        for (int c = 4 * threadIdx.x; c < p.d; c += 4 * kThreads * kGroups) {
            for (int which = 0; which < 2; ++which) {
                if (which == 0 ? !pre : !post) continue;
                const float* src = sums + which * kGroups * p.d + c;
                float4 v = *reinterpret_cast<const float4*>(src);
#pragma unroll
                for (int q = 1; q < kGroups; ++q) v = add4(v, *reinterpret_cast<const float4*>(src + q * p.d));
                *reinterpret_cast<float4*>((which == 0 ? p.part_pre : p.part_post) + out + c) = v;
            }
        }
    }
}

__device__ __forceinline__ float4 param4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 param4(const __nv_bfloat16* p) {
    float f[4];
    load_params<4>(p, f);
    return make_float4(f[0], f[1], f[2], f[3]);
}

// Adds the runs' partial sums, blockIdx.y 0: dw_pre, 1: dw_post and dgate.  A CTA takes 32 columns:
// eight threads of four columns (a 128-byte line of a run's sums) by 32 lanes that share the runs.  Of
// the lanes, `sub` (a power of two) share a canvas, or with more than 16 canvases each has every 32nd, four at
// a time; every sum has a fixed order.  Bound by the trips to L2 of a lane's run of loads: 2 to 3 us behind the
// kernel above for 2 x 296 rows of 2048 sums (4.8 MB).
template <typename P, int kTurns>
__global__ void __launch_bounds__(256) block_norm_params_kernel(const __grid_constant__ BlockNormBackwardParams p, int sub) {
    __shared__ float4 sh[32][8];
    const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
    const int c = blockIdx.x * 32 + tx * 4;
    const bool in = c < p.d, post = p.w_pre == nullptr || blockIdx.y == 1;
    const float* part = post ? p.part_post : p.part_pre;
    if (!post) sub = 32;
    const int canvases = post ? p.B : 1, runs = post ? p.runs : p.B * p.runs;
    const int first = ty / sub, l = ty % sub;
    const bool gated = post && p.gate;
    const float4 one = make_float4(1.f, 1.f, 1.f, 1.f), zero = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 w = gated && in ? param4(static_cast<const P*>(p.w_post) + c) : one;
    float4 total = zero;
    grid_dependency_wait();
    for (int b0 = 0; b0 < canvases; b0 += kTurns * 32) {  // one turn, and its first canvas only, unless sub == 1
        float4 a[kTurns], g[kTurns];
#pragma unroll
        for (int k = 0; k < kTurns; ++k) {
            const int b = b0 + first + k * 32;
            a[k] = zero;
            g[k] = gated && in && b < canvases ? param4(static_cast<const P*>(p.gate) + static_cast<int64_t>(b) * p.d + c) : one;
        }
        const auto add_run = [&](int k, int j) {
            const int b = b0 + first + k * 32;
            if (in && b < canvases) a[k] = add4(a[k], __ldcg(reinterpret_cast<const float4*>(part + (static_cast<int64_t>(b) * runs + j) * p.d + c)));
        };
        if (kTurns == 1 || sub > 1) {
#pragma unroll 8
            for (int j = l; j < runs; j += sub) add_run(0, j);
        } else {
#pragma unroll 2
            for (int j = 0; j < runs; ++j) {
#pragma unroll
                for (int k = 0; k < kTurns; ++k) add_run(k, j);
            }
        }
        if (sub > 1) {
            sh[ty][tx] = a[0];
            __syncthreads();
            if (l == 0)
                for (int q = 1; q < sub; ++q) a[0] = add4(a[0], sh[ty + q][tx]);
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < kTurns; ++k) {
            const int b = b0 + first + k * 32;
            if (l != 0 || !in || b >= canvases) continue;
            if (post) {
                a[k] = make_float4(p.res_scale * a[k].x, p.res_scale * a[k].y, p.res_scale * a[k].z, p.res_scale * a[k].w);
                if (gated)
                    *reinterpret_cast<float4*>(p.dgate + static_cast<int64_t>(b) * p.d + c) =
                        make_float4(w.x * a[k].x, w.y * a[k].y, w.z * a[k].z, w.w * a[k].w);
                a[k] = make_float4(g[k].x * a[k].x, g[k].y * a[k].y, g[k].z * a[k].z, g[k].w * a[k].w);
            }
            total = add4(total, a[k]);
        }
    }
    sh[ty][tx] = total;
    __syncthreads();
    if (ty == 0 && in) {
        for (int q = sub; q < 32; q += sub) total = add4(total, sh[q][tx]);
        *reinterpret_cast<float4*>((post ? p.dw_post : p.dw_pre) + c) = total;
    }
}

template <typename P>
cudaError_t launch_params(const BlockNormBackwardParams& p, cudaStream_t st) {
    note_launches(1);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    int sub = 32;  // lanes per canvas: as many as leave a group of lanes for every canvas
    while (sub > 1 && 32 / sub < p.B) sub >>= 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.d + 31) / 32), p.w_pre && p.y ? 2u : 1u);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // With one canvas to a lane and more CTAs than the SMs hold at 96 registers, the form of 40 (1024 x 8192 fp32 in
    // four canvases: 60.5 us, else 63.7; with fewer CTAs it is the slower one, 4096 x 1024 in 16: 22.2 and 19.6 [L2]).
    e = sub > 1 && static_cast<int>(cfg.gridDim.x * cfg.gridDim.y) > 2 * num_sms()
            ? cudaLaunchKernelEx(&cfg, block_norm_params_kernel<P, 1>, p, sub)
            : cudaLaunchKernelEx(&cfg, block_norm_params_kernel<P, 4>, p, sub);
    if (e != cudaSuccess) return e;
    note_launches(1);
    return cudaGetLastError();
}

template <typename T, typename P, int kWarps, int kNV>
cudaError_t launch_backward(const BlockNormBackwardParams& p, cudaStream_t st) {
    block_norm_backward_kernel<T, P, kWarps, kNV><<<static_cast<unsigned>(p.B) * p.runs, 32 * kWarps, 0, st>>>(p);
    return launch_params<P>(p, st);
}

template <typename T, typename P, int kW, int kGroups, int kNV, int kCtas, bool kFull>
cudaError_t launch_backward_rows_as(const BlockNormBackwardParams& p, cudaStream_t st) {
    constexpr int kRingBytes = 200 * 1024 / kCtas;
    const int slot = p.d * static_cast<int>(sizeof(T)) * ((p.dx_out ? 1 : 0) + (p.w_pre ? 2 : 0) + (p.y ? 1 : 0));
    const int slots = std::min({kMaxSlots, (p.run_rows + kGroups - 1) / kGroups, kRingBytes / (slot * kGroups)});
    const int bytes = std::max(kNV > 1 ? kGroups * slots * slot : 0, kGroups > 1 ? 2 * kGroups * p.d * 4 : 0);
    static DeviceOnce once;
    const cudaError_t attr_err = allow_shared_memory(once, block_norm_backward_rows_kernel<T, P, kW, kGroups, kNV, kCtas, kFull>, kRingBytes);
    if (attr_err != cudaSuccess) return attr_err;
    block_norm_backward_rows_kernel<T, P, kW, kGroups, kNV, kCtas, kFull><<<static_cast<unsigned>(p.B) * p.runs, 32 * kW * kGroups, bytes, st>>>(p, slots);
    return launch_params<P>(p, st);
}

template <typename T, typename P, int kW, int kGroups, int kNV, int kCtas>
cudaError_t launch_backward_rows(const BlockNormBackwardParams& p, cudaStream_t st) {
    if (p.d == kNV * kW * 32 * Vec<T>::kN) return launch_backward_rows_as<T, P, kW, kGroups, kNV, kCtas, true>(p, st);
    return launch_backward_rows_as<T, P, kW, kGroups, kNV, kCtas, false>(p, st);
}

template <typename T, typename P>
cudaError_t backward_by_width(const BlockNormBackwardParams& p, cudaStream_t st) {
    const int n_vec = p.d / Vec<T>::kN;
    if (n_vec <= 32) return launch_backward_rows<T, P, 1, 8, 1, kNormCtas>(p, st);
    if (n_vec <= 64) return launch_backward_rows<T, P, 1, 8, 2, kNormCtas>(p, st);
    if (n_vec <= 128) return launch_backward_rows<T, P, 2, 4, 2, kNormCtas>(p, st);
    if (n_vec <= 256) return launch_backward_rows<T, P, 4, 2, 2, kNormCtas>(p, st);
    if (n_vec <= 512) return launch_backward_rows<T, P, 8, 1, 2, kNormCtas>(p, st);
    if (n_vec <= 1024) return launch_backward_rows<T, P, 16, 1, 2, 1>(p, st);
    if constexpr (sizeof(T) == 4)  // (bf16 rows have 2048 vectors at most)
        if (n_vec > 2048) return launch_backward<T, P, 16, 8>(p, st);
    return launch_backward<T, P, 16, 4>(p, st);
}

}  // namespace

cudaError_t read_and_clear_norm_error(int* out) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int));
    if (e != cudaSuccess) return e;
    if (v) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
    }
    *out = v;
    return e;
}

cudaError_t launch_block_norm(const BlockNormParams& p, int act_bf16, int param_bf16, cudaStream_t st) {
    if (act_bf16)
        return param_bf16 ? forward_by_width<__nv_bfloat16, __nv_bfloat16>(p, st) : forward_by_width<__nv_bfloat16, float>(p, st);
    return param_bf16 ? forward_by_width<float, __nv_bfloat16>(p, st) : forward_by_width<float, float>(p, st);
}

// Runs of rows per canvas: as many CTAs as the SMs hold at once, but two rows to a run, so that there
// are not more partial sums than need be (256 rows of 2048 in runs of one, two, four: 11.9, 9.4, 9.8 us [L2]).
int32_t block_norm_runs(int32_t B, int32_t C, int32_t d, int act_bf16) {
    const int n_vec = d / (act_bf16 ? 8 : 4);
    const int per_sm = n_vec <= 512 ? kNormCtas : 1;
    return std::max(1, std::min<int32_t>(per_sm * num_sms() / B, C / 2 + C % 2));
}

cudaError_t launch_block_norm_backward(const BlockNormBackwardParams& p, int act_bf16, int param_bf16, cudaStream_t st) {
    if (act_bf16)
        return param_bf16 ? backward_by_width<__nv_bfloat16, __nv_bfloat16>(p, st) : backward_by_width<__nv_bfloat16, float>(p, st);
    return param_bf16 ? backward_by_width<float, __nv_bfloat16>(p, st) : backward_by_width<float, float>(p, st);
}

}  // namespace dg
