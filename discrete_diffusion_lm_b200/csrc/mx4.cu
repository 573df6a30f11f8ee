// Microscaled 4-bit floating point (OCP Microscaling Formats, MXFP4): quantisation, reading back, and
// products on the sm_100a tensor cores.
//
// Thirty-two consecutive values of a row share the scale 2^(c - 127), kept as the byte c (E8M0); a
// value is E2M1: 0, 0.5, 1, 1.5, 2, 3, 4 or 6 with a sign, two to a byte, the lower index in the low
// half.  For a block of largest magnitude A,
//   e = max(floor(log2 A) - 2, -127), c = e + 127, q_i = round-to-nearest-even(x_i 2^-e), |q_i| <= 6
// (6 = 1.5 2^2 is the largest E2M1 value, so e puts A between 4 and 8); A = 0 gives c = 0; a block
// with a NaN or an infinity gets c = 255, which stands for NaN.
// Scale bytes lie as the tensor core takes them: tiles of 128 rows x 4 blocks (128 values), 512
// bytes, byte (r % 32) * 16 + (r / 32 % 4) * 4 + block % 4; tiles of one row group are consecutive.
// Padding in a tile (rows or blocks past the matrix) holds 127.
//
// Times below are of launches back to back in one graph that rotate over inputs and outputs of 500 MB together;
// those marked [L2], the rules' among them, rotate over three or four sets, which L2 mostly holds.
#include <cuda_fp16.h>
#include <cuda_fp4.h>

#include <algorithm>
#include <atomic>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "kernels.cuh"
#include "tensor_core.cuh"

namespace dg {

namespace {

constexpr uint32_t kUnitScale = 127;  // the scale byte of 2^0

// The scale byte of a block whose largest magnitude has the bit pattern `top` (sign cleared).
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    if (top >= 0x7F800000u) return 255u;  // an infinity, or a NaN of either sign
    const uint32_t ex = top >> 23;  // biased exponent; 0 for zero and subnormal values, whose e is -127
    return ex > 2u ? ex - 2u : 0u;
}
// 2^-e as a float for a scale byte c = e + 127 in [0, 252]: exponents 127 down to -125, all normal.
__device__ __forceinline__ float inverse_scale(uint32_t c) { return __uint_as_float((254u - c) << 23); }

// Values times `inv`, rounded to E2M1 (nearest, ties to even, saturating), packed low to high.
__device__ __forceinline__ uint32_t pack_e2m1(const float (&f)[8], float inv) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(f[0] * inv), "f"(f[1] * inv), "f"(f[2] * inv), "f"(f[3] * inv), "f"(f[4] * inv), "f"(f[5] * inv),
          "f"(f[6] * inv), "f"(f[7] * inv));
    return r;
}
__device__ __forceinline__ uint16_t pack_e2m1(const float (&f)[4], float inv) {
    uint16_t r;
    asm("{\n\t.reg .b8 a, b;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "mov.b16 %0, {a, b};\n\t}"
        : "=h"(r)
        : "f"(f[0] * inv), "f"(f[1] * inv), "f"(f[2] * inv), "f"(f[3] * inv));
    return r;
}

// ------------------------------------------------------------------------------------ quantisation
// Both directions are bound by memory.  A warp takes kMx4Cols columns of a row: vectors of 16 bytes per
// lane, contiguous over the warp (4 fp32 or 8 bf16 values), all loaded before the first is used; a
// block of 32 lies in 8 or 4 lanes.  8192 x 2048 fp32 takes 16.0 us (4.7 TB/s), and 15.1 us back.
constexpr int kMx4Cols = 512;

__device__ __forceinline__ uint8_t* scale_word(uint8_t* scales, int32_t r, int32_t k_tiles, int32_t k) {
    return scales + (static_cast<int64_t>(r / 128) * k_tiles + k / 128) * 512 + (r % 32) * 16 + (r / 32 % 4) * 4;
}

// Rows up to a multiple of 128 are walked, so that every scale tile is written whole.
template <typename T>
__global__ void __launch_bounds__(256) mx4_quantize_kernel(const T* __restrict__ x, int64_t ld, int32_t rows, int32_t K,
                                                           uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    constexpr int kN = 16 / sizeof(T), kLanes = 32 / kN;  // values of a vector, lanes of a block
    constexpr int kVecs = kMx4Cols / (32 * kN);
    const int lane = threadIdx.x & 31;
    const int32_t r = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int32_t k0 = blockIdx.y * kMx4Cols + lane * kN, k_end = (K + 127) / 128 * 128;
    grid_launch_dependents();
    uint4 v[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        const int32_t k = k0 + j * 32 * kN;
        v[j] = r < rows && k < K ? ld_stream_v4(x + static_cast<int64_t>(r) * ld + k) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        const int32_t k = k0 + j * 32 * kN;
        if (k - lane * kN >= k_end) break;  // the whole warp
        float f[kN];
        if constexpr (sizeof(T) == 2) {
            const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = bf16_lo(w[i]);
                f[2 * i + 1] = bf16_hi(w[i]);
            }
        } else {
            f[0] = __uint_as_float(v[j].x);
            f[1] = __uint_as_float(v[j].y);
            f[2] = __uint_as_float(v[j].z);
            f[3] = __uint_as_float(v[j].w);
        }
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kN; ++i) top = max(top, __float_as_uint(f[i]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        uint32_t c = kUnitScale;
        if (r < rows && k < K) {  // K is a multiple of 32: a block's lanes agree
            c = scale_byte(top);
            DG_CHECK(g_device_error, k + kN <= K && ld >= K);
            const auto q = pack_e2m1(f, inverse_scale(c == 255u ? kUnitScale : c));
            using Code = std::remove_const_t<decltype(q)>;
            *reinterpret_cast<Code*>(codes + static_cast<int64_t>(r) * (K / 2) + k / 2) = c == 255u ? Code(0) : q;
        }
        // the scale bytes of four blocks (4 kLanes lanes) as one word of their tile
        uint32_t word = c << (8 * (lane / kLanes & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, kLanes);
        word |= __shfl_xor_sync(0xffffffffu, word, 2 * kLanes);
        if (lane % (4 * kLanes) == 0 && k < k_end) *reinterpret_cast<uint32_t*>(scale_word(scales, r, (K + 127) / 128, k)) = word;
    }
}

// ------------------------------------------------------------------------------------ reading back
// Eight codes to their values (E2M1 values are exact in fp16).
__device__ __forceinline__ void unpack_e2m1(uint32_t q, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(q >> (8 * i)), __NV_E2M1);
        const float2 v = __half22float2(__half2(h));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}

template <typename T>
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                             int32_t rows, int32_t K, T* __restrict__ out) {
    constexpr int kN = 16 / sizeof(T), kVecs = kMx4Cols / (32 * kN);
    using Code = std::conditional_t<kN == 8, uint32_t, uint16_t>;
    const int lane = threadIdx.x & 31;
    const int32_t r = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int32_t k0 = blockIdx.y * kMx4Cols + lane * kN;
    if (r >= rows) return;
    uint32_t q[kVecs], word[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        const int32_t k = k0 + j * 32 * kN;
        q[j] = word[j] = 0;
        if (k < K) {
            q[j] = __ldg(reinterpret_cast<const Code*>(codes + static_cast<int64_t>(r) * (K / 2) + k / 2));
            word[j] = __ldg(reinterpret_cast<const uint32_t*>(scale_word(const_cast<uint8_t*>(scales), r, (K + 127) / 128, k)));
        }
    }
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        const int32_t k = k0 + j * 32 * kN;
        if (k >= K) break;
        const uint32_t c = word[j] >> (8 * (k / 32 & 3)) & 255u;
        // 2^(c - 127): c = 0 is the subnormal 2^-127, 255 is NaN
        const float s = c == 255u ? __uint_as_float(0x7FC00000u) : c ? __uint_as_float(c << 23) : __uint_as_float(0x00400000u);
        float f[8];
        unpack_e2m1(q[j], f);
#pragma unroll
        for (int i = 0; i < kN; ++i) f[i] *= s;
        T* o = out + static_cast<int64_t>(r) * K + k;
        if constexpr (kN == 8)
            *reinterpret_cast<uint4*>(o) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                                      pack_bf16x2(f[6], f[7]));
        else
            *reinterpret_cast<float4*>(o) = make_float4(f[0], f[1], f[2], f[3]);
    }
}

// ------------------------------------------------------------------------------------ product
// out[M, N] = A[M, K] W[N, K]^T, both operands MXFP4 with K-contiguous rows, fp32 accumulation.
//
// A CTA computes 128 rows x 128 columns over a run of 256-value blocks of K.  Per block, one thread
// copies the W tile (128-byte rows, 128-byte swizzle) and its scale tiles, another the A tile and
// its scale tiles (it waits for the preceding kernel first: A may be that kernel's output); a third
// moves the scales into tensor memory (tcgen05.cp), and a fourth issues four
// tcgen05.mma.kind::mxf4 of K = 64, two scale bytes per row and instruction.  (tcgen05.cp and the
// products that follow it in one thread run one after the other: with both in one thread a stage took
// 1100 to 1300 cycles instead of about 560.)
// With few rows A may be bf16 (kFew): the epilogue's warps, idle until the products are done, quantise
// each stage of it into shared memory, a block of 32 values per thread, in the place of its copies.
// With few tiles K is split over the CTAs of a cluster: each sends every other its share of the rows
// of its fp32 tile (bulk copies into that CTA's inbox), and adds the shares it is sent in a fixed order.
// Few rows cost latency, not bandwidth: 1 x 8192 x 2048 (8.9 MB of W) takes 7.6 us, 1 x 2048 x 8192 8.3 (6.9
// [L2], without the split 13.0 [L2]).
constexpr int kMTile = 128, kNTile = 128, kKStage = 256;
constexpr int kMx4Threads = 384;  // W copies, products, A copies, scale copies; eight epilogue warps
constexpr uint32_t kOperandBytes = 128 * kKStage / 2;
constexpr uint32_t kScaleBytes = 1024;  // two tiles
constexpr uint32_t kStageBytes = 2 * (kOperandBytes + kScaleBytes);
constexpr int kMx4Stages = 6;       // of the ring; a split of K keeps kSplitStages and has the rest as inbox
constexpr int kSplitStages = 4;
constexpr uint32_t kTmemCols = 256;  // 128 accumulator columns, 16 per stage of scales
constexpr int kTilePitch = kNTile + 4;  // floats; rows 16 bytes off the banks of the row before
constexpr uint32_t kMx4Smem = kMx4Stages * kStageBytes + 512 + 1024;
static_assert(kMx4Stages * 16 + kNTile <= static_cast<int>(kTmemCols), "scales and accumulator fit");
static_assert(kMTile * kTilePitch * 4 <= kSplitStages * kStageBytes, "the fp32 tile fits the drained ring");
// an inbox holds splits - 1 shares of up to 128 / splits rows: 3 x 32 or 64
static_assert(3 * 32 * kTilePitch * 4 <= (kMx4Stages - kSplitStages) * kStageBytes, "the inbox fits the rest");

enum Mx4Out : int { kOutBf16 = 0, kOutF32 = 1, kOutGeluMx4 = 2 };

struct alignas(64) Mx4Kernel {
    CUtensorMap tm_a, tm_w;  // bytes [rows, K / 2], box 128 rows x 128 bytes
    const uint8_t *sa, *sw;
    const __nv_bfloat16* a_bf16;  // kFew: A [M, K]
    void* out;            // bf16 or fp32 [M, N], or codes [M, N / 2]
    uint8_t* out_scales;  // kOutGeluMx4
    int32_t M, N, K;
    int32_t n_tiles, k_tiles, k_blocks;  // 128-column tiles; 128-value and 256-value steps of K
    long long wait_limit;
    int32_t fault_block;  // test hook: W's copies of this 256-value block are never issued (-1: none)
};

// kind::mxf4 instruction descriptor: E2M1 operands (type 1), E8M0 scales, M = 128, N = 128; the scale
// bytes of operand A at bit 29, of B at bit 4 (which two of a word's four).
__device__ __forceinline__ uint32_t idesc_mx4(uint32_t pair) {
    return (pair << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(kNTile >> 3) << 17) | (1u << 23) |
           (static_cast<uint32_t>(kMTile >> 7) << 27) | (pair << 29);
}
__device__ __forceinline__ void umma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}
// 32 rows x 16 bytes of shared memory (no swizzle, groups of 8 rows 128 bytes apart) to four
// tensor-memory columns, repeated for the four lane groups.
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t d) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(d) : "memory");
}
// Shared memory of this CTA to another CTA's of the cluster, counted on that CTA's barrier.
__device__ __forceinline__ void bulk_send(uint32_t dst_cluster, uint32_t src, uint32_t bytes, uint32_t bar_cluster) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst_cluster),
                 "r"(src), "r"(bytes), "r"(bar_cluster)
                 : "memory");
}
// (relaxed: mbarrier initialisation is released by its own fence, shares by the barrier they complete on)
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}

// GELU, tanh form, as x T / (1 + T) with T = exp(2u), two values at a time.  The hidden layer is rounded to 4
// bits by comparisons with the E2M1 midpoints, so an error here moves values across them: the hardware
// tanh's 2^-11 would move one value in a few hundred, ex2 and a reciprocal (about 2^-22) one in a
// million.  The special-function unit bounds the epilogue (a block on 4096 rows of 1024 x 4096 takes 32.1 us,
// without the gelu 26.7), so two values share a reciprocal: 1 / a = b (1 / ab); with one each 33.8 us, with
// Newton's iteration instead no less.  T is kept below 2^62, so that ab and its reciprocal are normal numbers (from
// 2^24 on T / (1 + T) is 1 anyway); below, T goes to zero as it should, at 2^-126.  A sum that left fp32 gives no
// number on either side; taking -infinity for 0, two instructions more for each pair, cost 0.9 us.
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ Pair gelu_pair(Pair x) {
    const float k0 = 2.0f * 0.7978845608028654f * kLog2e;  // 2 sqrt(2 / pi) log2 e
    const float k1 = k0 * 0.044715f;
    float lo, hi;
    unpair(mul2(x, fma2(mul2(x, x), pair(k1, k1), pair(k0, k0))), lo, hi);
    lo = ex2_approx(fminf(lo, 62.0f));
    hi = ex2_approx(fminf(hi, 62.0f));
    const float a = 1.0f + lo, b = 1.0f + hi, r = rcp_approx(a * b);
    return mul2(x, mul2(pair(lo, hi), mul2(pair(r, r), pair(b, a))));  // (x T alone could leave fp32)
}
// max(a, |b|) that keeps a NaN.
__device__ __forceinline__ float max_abs_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
    return r;
}

// Sixteen bytes of codes and the scale byte of a block of 32 bf16 values.
__device__ __forceinline__ uint4 quantize_block(const __nv_bfloat16* x, uint32_t& c) {
    uint32_t w[16], q[4], top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(x) + i);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, max(w[i] << 16 & 0x7FFFFFFFu, w[i] & 0x7FFF0000u));
    c = scale_byte(top);
    const float inv = inverse_scale(c == 255u ? kUnitScale : c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float f[8] = {bf16_lo(w[4 * i]),     bf16_hi(w[4 * i]),     bf16_lo(w[4 * i + 1]), bf16_hi(w[4 * i + 1]),
                            bf16_lo(w[4 * i + 2]), bf16_hi(w[4 * i + 2]), bf16_lo(w[4 * i + 3]), bf16_hi(w[4 * i + 3])};
        q[i] = c == 255u ? 0u : pack_e2m1(f, inv);
    }
    return make_uint4(q[0], q[1], q[2], q[3]);
}

template <int kOut, bool kFew>
__global__ void __launch_bounds__(kMx4Threads, 1) mx4_matmul_kernel(const __grid_constant__ Mx4Kernel p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kMx4Stages * kStageBytes);
    uint64_t* scaled = full + kMx4Stages;
    uint64_t* empty = scaled + kMx4Stages;
    uint64_t* accum = empty + kMx4Stages;
    uint64_t* inbox_full = accum + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(inbox_full + 1);
    WaitCtl* wc = reinterpret_cast<WaitCtl*>(tmem_slot + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int splits = static_cast<int>(cluster_size()), split = static_cast<int>(cluster_rank());
    const int stages = splits > 1 ? kSplitStages : kMx4Stages;
    const int32_t tile = blockIdx.x / splits;
    const int32_t mt = tile / p.n_tiles, nt = tile - mt * p.n_tiles;
    const int32_t kb0 = static_cast<int32_t>(static_cast<int64_t>(p.k_blocks) * split / splits);
    const int32_t kb1 = static_cast<int32_t>(static_cast<int64_t>(p.k_blocks) * (split + 1) / splits);
    const int32_t m_valid = min(kMTile, p.M - mt * kMTile);
    const int32_t share = (m_valid + splits - 1) / splits;  // rows of the tile that a split adds up

    // one stage's copy of an operand: W (or A) rows and their scale tiles
    const auto load_stage = [&](int32_t kb, int s, bool is_a) {
        const int32_t rt = is_a ? mt : nt;
        uint8_t* st = smem + s * kStageBytes;
        uint64_t* bar = &full[s];
        const uint32_t scale_bytes = min(2, p.k_tiles - 2 * kb) * 512;
        mbar_arrive_expect_tx(bar, kOperandBytes + scale_bytes);
        tma_load_2d(st + (is_a ? 0 : kOperandBytes), is_a ? &p.tm_a : &p.tm_w, kb * (kKStage / 2), rt * 128, bar);
        bulk_load(st + 2 * kOperandBytes + (is_a ? 0 : kScaleBytes),
                  (is_a ? p.sa : p.sw) + static_cast<int64_t>(rt) * p.k_tiles * 512 + static_cast<int64_t>(kb) * 1024, scale_bytes, bar);
    };
    if (threadIdx.x == 96) {
        prefetch_map(&p.tm_w);
        if (!kFew) prefetch_map(&p.tm_a);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kMx4Stages; ++s) {
            mbar_init(&full[s], kFew ? 9 : 2);  // W's copies, and A's or the eight warps that write it
            mbar_init(&scaled[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(accum, 1);
        mbar_init(inbox_full, 1);
        wc->abort = 0;
        wc->limit = p.wait_limit;
        fence_barrier_init();
    }
    __syncthreads();
    if (splits > 1) cluster_arrive();  // this CTA's inbox barrier is initialised
    // The copies start at once; the warps that use the tensor memory meet when it is there.
    if (warp != 0 && warp != 2) {
        if (warp == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(kTmemCols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
        tcgen05_before_sync();
        asm volatile("bar.sync 1, %0;" ::"n"(kMx4Threads - 64) : "memory");
        tcgen05_after_sync();
    }
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);

    if ((warp == 0 || (warp == 2 && !kFew)) && lane == 0) {
        // ---------------------------------------------------------------- producers: W, A
        const bool is_a = warp == 2;
        int32_t kb = kb0;
        if (is_a) grid_dependency_wait();  // A may be the preceding kernel's output; the weights are not
        for (int s = 0, phase = 0; kb < kb1; ++kb) {
            if (s == stages) {
                s = 0;
                phase ^= 1;
            }
            if (!mbar_wait(&empty[s], phase ^ 1, wc)) break;
            if (is_a || kb != p.fault_block) load_stage(kb, s, is_a);
            ++s;
        }
        if (aborted(wc)) {  // let the copies in flight land before the shared memory goes away
            const long long t0 = clock64();
            for (int i = max(0, kb - kb0 - stages); i < kb - kb0; ++i)  // (a block left out by the test hook never lands)
                while (kb0 + i != p.fault_block && !mbar_try_wait(&full[i % stages], (i / stages) & 1) && clock64() - t0 < wc->limit) {
                }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        // The whole warp walks the loop, so that descriptors stay in uniform registers; one lane issues.
        const uint64_t da0 = smem_desc(smem_u32(smem), 16, 1024, kLayoutSw128);
        int s = 0, phase = 0;
        for (int32_t kb = kb0; kb < kb1; ++kb) {
            if (!__all_sync(0xffffffffu, mbar_wait(&scaled[s], phase, wc))) break;
            tcgen05_after_sync();
            const uint64_t da = da0 + static_cast<uint64_t>(s * (kStageBytes / 16)), dw = da + kOperandBytes / 16;
            const uint32_t sf = tmem + kNTile + s * 16;  // two tiles of A, two of W, four columns each
            const int32_t steps = min(4, (p.K - kb * kKStage + 63) / 64);
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    if (ks < steps)
                        umma_mx4(tmem, da + 2 * ks, dw + 2 * ks, idesc_mx4((ks & 1) * 2), sf + 4 * (ks >> 1), sf + 8 + 4 * (ks >> 1),
                                 (kb > kb0 || ks > 0) ? 1u : 0u);
                umma_commit(&empty[s]);
                if (kb == kb1 - 1) umma_commit(accum);
            }
            __syncwarp();
            if (++s == stages) {
                s = 0;
                phase ^= 1;
            }
        }
    } else if (warp == 3) {
        // ---------------------------------------------------------------- scale copies
        const uint64_t d0 = smem_desc(smem_u32(smem) + 2 * kOperandBytes, 16, 128, 0);
        int s = 0, phase = 0;
        for (int32_t kb = kb0; kb < kb1; ++kb) {
            if (!__all_sync(0xffffffffu, mbar_wait(&full[s], phase, wc))) break;
            tcgen05_after_sync();
            const uint64_t d = d0 + static_cast<uint64_t>(s * (kStageBytes / 16));
            const uint32_t sf = tmem + kNTile + s * 16;
            const int32_t tiles = min(2, p.k_tiles - 2 * kb);
            if (elect_one()) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (j < tiles) {
                        copy_scales(sf + 4 * j, d + 32 * j);
                        copy_scales(sf + 8 + 4 * j, d + kScaleBytes / 16 + 32 * j);
                    }
                umma_commit(&scaled[s]);
            }
            __syncwarp();
            if (++s == stages) {
                s = 0;
                phase ^= 1;
            }
        }
    }
    __syncwarp();
    if (kFew && warp >= 4) {
        // ---------------------------------------------------------------- A, quantised
        int s = 0, phase = 0;
        for (int32_t kb = kb0; kb < kb1; ++kb) {
            if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], phase ^ 1, wc))) break;
            uint8_t* st = smem + s * kStageBytes;
            for (int i = threadIdx.x - 128; i < m_valid * 8; i += 256) {
                const int row = i >> 3, j = i & 7;  // the stage's block j of a row: its 16-byte chunk j
                const int32_t k = kb * kKStage + j * 32;
                uint4 q = make_uint4(0, 0, 0, 0);
                uint32_t c = kUnitScale;
                if (k < p.K) q = quantize_block(p.a_bf16 + (static_cast<int64_t>(mt) * kMTile + row) * p.K + k, c);
                *reinterpret_cast<uint4*>(st + row * 128 + ((j ^ (row & 7)) << 4)) = q;
                st[2 * kOperandBytes + (j >> 2) * 512 + (row & 31) * 16 + (row >> 5) * 4 + (j & 3)] = static_cast<uint8_t>(c);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[s]);
            if (++s == stages) {
                s = 0;
                phase ^= 1;
            }
        }
        __syncwarp();
    }

    // ---------------------------------------------------------------- epilogue: fp32 tile, then rows
    float* tile_f = reinterpret_cast<float*>(smem);
    bool ok = true;
    if (warp >= 4) {
        ok = __all_sync(0xffffffffu, mbar_wait(accum, 0, wc));
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        if (ok && quarter * 32 < m_valid) {
            tcgen05_after_sync();
            const int row = quarter * 32 + lane;
            const uint32_t acc = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * (kNTile / 2);
            uint32_t v[64];
            tmem_ld_32x32b_x32_nowait(acc, v);
            tmem_ld_32x32b_x32_nowait(acc + 32, v + 32);
            tmem_ld_wait();
            if (row < m_valid) {  // rows of kTilePitch floats
                const uint32_t at = smem_u32(tile_f + row * kTilePitch + half * (kNTile / 2));
#pragma unroll
                for (int q = 0; q < 16; ++q) st_shared_v4(at + 16 * q, make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
            }
        }
    }
    grid_launch_dependents();
    if (splits > 1) fence_proxy_async_smem();  // the tile's rows, visible to the bulk copies
    ok = __syncthreads_and(ok);
    const int32_t row0 = min(split * share, m_valid), rows = min(share, m_valid - row0);
    float* inbox = reinterpret_cast<float*>(smem + kSplitStages * kStageBytes);  // (splits - 1) shares
    if (splits > 1) {
        cluster_wait();  // every inbox barrier is initialised
        if (warp == 0 && elect_one()) {
            mbar_arrive_expect_tx(inbox_full, static_cast<uint32_t>((splits - 1) * rows * kTilePitch * 4));
            for (int d = 1; d < splits; ++d) {  // to split `to`, its share; slots are in the order of the senders
                const int to = (split + d) % splits;
                const int32_t first = min(to * share, m_valid), n = min(share, m_valid - first);
                if (n > 0)
                    bulk_send(map_to_rank(smem_u32(inbox + (split < to ? split : split - 1) * n * kTilePitch), to),
                              smem_u32(tile_f + first * kTilePitch), static_cast<uint32_t>(n * kTilePitch * 4), map_to_rank(smem_u32(inbox_full), to));
            }
        }
        __syncwarp();
        if (rows > 0 && !mbar_wait(inbox_full, 0, wc)) {
            // given up elsewhere in this CTA: the other splits' shares are under way all the same
            const long long t0 = clock64();
            while (!mbar_try_wait(inbox_full, 0) && clock64() - t0 < wc->limit) {
            }
            ok = false;
        }
        ok = __syncthreads_and(ok);
        cluster_arrive();  // every share sent to this CTA is here
    }
    const int32_t col = nt * kNTile + lane * 4;
    // The CTA's rows over its warps; a lane takes four columns.  A quantised output's scale tile is
    // written whole: the last split also takes the rows past M.  (Kept as tight loops: code that runs
    // once per launch costs its instruction fetches.  Unrolled over rows and splits this part took
    // 7000 cycles, so 1000.)
    const int32_t last = kOut == kOutGeluMx4 && split == splits - 1 ? kMTile : row0 + rows;
    if (ok) {
#pragma unroll 1
        for (int32_t i = row0 + warp; i < last; i += kMx4Threads / 32) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < row0 + rows) {
                const float* own = tile_f + i * kTilePitch + lane * 4;
                const float* sent = inbox + (i - row0) * kTilePitch + lane * 4;
#pragma unroll 1
                for (int q = 0; q < splits; ++q) {
                    const float4 w = *reinterpret_cast<const float4*>(q == split ? own : sent);
                    if (q != split) sent += rows * kTilePitch;
                    v.x += w.x;
                    v.y += w.y;
                    v.z += w.z;
                    v.w += w.w;
                }
            }
            const int64_t r = static_cast<int64_t>(mt) * kMTile + i;
            DG_CHECK(g_device_error, i < kMTile && (i >= m_valid || (r < p.M && share * splits >= m_valid)));
            if (kOut == kOutF32) {
                if (col < p.N) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + r * p.N + col) = v;
            } else if (kOut == kOutBf16) {
                if (col < p.N)
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + r * p.N + col) =
                        make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
            } else {
                // eight lanes hold a block of 32 hidden values
                float f[4];
                unpair(gelu_pair(pair(v.x, v.y)), f[0], f[1]);
                unpair(gelu_pair(pair(v.z, v.w)), f[2], f[3]);
                uint32_t top = __float_as_uint(max_abs_nan(max_abs_nan(max_abs_nan(fabsf(f[0]), f[1]), f[2]), f[3]));
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                const bool in = i < m_valid && col < p.N;
                const uint32_t c = in ? scale_byte(top) : kUnitScale;
                if (in) {
                    const uint16_t q = pack_e2m1(f, inverse_scale(c == 255u ? kUnitScale : c));
                    *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(p.out) + r * (p.N / 2) + col / 2) = c == 255u ? uint16_t(0) : q;
                }
                uint32_t word = c << (8 * (lane >> 3));
                word |= __shfl_xor_sync(0xffffffffu, word, 8);
                word |= __shfl_xor_sync(0xffffffffu, word, 16);
                if (lane == 0)
                    *reinterpret_cast<uint32_t*>(p.out_scales + (static_cast<int64_t>(mt) * p.n_tiles + nt) * 512 + (i % 32) * 16 + (i / 32) * 4) = word;
            }
        }
    }
    tcgen05_before_sync();
    __syncthreads();
    if (splits > 1) cluster_wait();  // this CTA's shares have arrived: none is still read from its tile
    tcgen05_after_sync();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

template <int kOut, bool kFew = false>
cudaError_t launch_product(const Mx4Kernel& kp, int grid, int splits, bool dependent, cudaStream_t st) {
    static DeviceOnce once;
    const cudaError_t attr_err = allow_shared_memory(once, mx4_matmul_kernel<kOut, kFew>, static_cast<int>(kMx4Smem));
    if (attr_err != cudaSuccess) return attr_err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kMx4Threads);
    cfg.dynamicSmemBytes = kMx4Smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, mx4_matmul_kernel<kOut, kFew>, kp);
    if (e != cudaSuccess) return e;
    note_launches(1);
    return cudaGetLastError();
}

// ------------------------------------------------------------------------------------ product, many tiles
// The same product for many tiles: persistent clusters of two CTAs, each pair computing 256 rows x kN
// columns at a time with tcgen05.mma.cta_group::2 (M = 256): a CTA stages its own 128 rows of A and
// half of the W rows, so an operand byte read from L2 serves twice the products of a single CTA's tile;
// the scales of W are staged by both, as both tensor memories hold them.  All copies of a stage
// complete on the leader's barrier (box copies of cta_group::2, no multicast); the leader's MMA
// thread commits a stage to both CTAs' empty barriers and a finished tile to both accumulator
// barriers.  256 accumulator columns are two buffers of 128 or one of 256; eight epilogue warps
// drain a buffer while the copies, and with two buffers the products, of the next tile run.
// 4096 x 8192 x 2048 bf16 takes 33.5 us (4.1 PFLOP/s; the first form, of single CTAs, 133).  With K = 1024, 4096
// and 8192 it is 24.1, 55.1 and 99.1: a stage (28 to a pair and 1024 of K) takes 0.34 to 0.39 us, 650 to 760 cycles at
// 1.965 GHz, of which its products fill 512.  Probably the feed bounds it: 35 KB a stage into every SM are 13 TB/s
// from L2.  The other 12 to 15 us are the launch, the first stages and the drains of seven tiles into registers,
// which are not hidden.  In a loop of half a second the power cap takes the clock to 1.7 GHz: 36.8 us.
template <int kN>
struct PairTile {
    static constexpr int kBuffers = 256 / kN;
    static constexpr uint32_t kABytes = kOperandBytes;
    static constexpr uint32_t kWBytes = (kN / 2) * (kKStage / 2);
    static constexpr uint32_t kSwBytes = (kN / 128) * kScaleBytes;
    static constexpr uint32_t kStage = kABytes + kWBytes + kScaleBytes + kSwBytes;
    static constexpr uint32_t kSlabBytes = 16384;            // 128 rows x 128 bytes
    static constexpr uint32_t kStaging = 2 * kSlabBytes;  // one per epilogue group: a fifth stage is worth more
    static constexpr uint32_t kBudget = 226u * 1024u;
    static constexpr int kFit = static_cast<int>((kBudget - kStaging) / kStage);
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr uint32_t kSmem = kStaging + kStages * kStage + 512 + 1024;
    static constexpr uint32_t kScaleCols = 8 + 8 * (kN / 128);  // of one stage: A, then W
    static_assert(256 + kStages * kScaleCols <= 512, "accumulators and scales fit the tensor memory");
    static_assert(kStage % 1024 == 0, "stages keep the 1024-byte alignment of the swizzle");
    static_assert(kSmem <= 232448, "shared memory of a CTA");
};
constexpr int kPairThreads = 64 + 256 + 32;  // producer, MMA issuer, two groups of four epilogue warps, scale copies

struct alignas(64) Mx4PairKernel {
    CUtensorMap tm_a, tm_w;    // bytes [rows, K / 2], boxes of 128 and kN / 2 rows x 128 bytes
    CUtensorMap tm_sa, tm_sw;  // scale tiles as [tiles, 128] words, boxes of two tiles
    CUtensorMap tm_out;        // bf16 (box 64 columns x 32 rows) or fp32 (32 x 32) [M, N]
    uint8_t* out_codes;        // kOutGeluMx4
    uint8_t* out_scales;
    int32_t M, N, K;
    int32_t m_tiles, n_tiles, k_tiles, k_blocks;
    long long wait_limit;
    int32_t fault_block;  // test hook: the copies of this block are never issued (-1: none)
};

template <int kN>
__device__ __forceinline__ uint32_t idesc_mx4_pair(uint32_t pair) {
    return (pair << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(kN >> 3) << 17) | (1u << 23) | (2u << 27) | (pair << 29);
}
__device__ __forceinline__ void umma_mx4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}
// As copy_scales, in both CTAs of the pair: each from its own shared memory to its own tensor memory.
__device__ __forceinline__ void copy_scales_pair(uint32_t tmem, uint64_t d) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(d) : "memory");
}
// Barrier of one epilogue group (128 threads) that also ORs a flag over it: one exit decision.
__device__ __forceinline__ bool group_sync_or(int group, bool flag) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(flag)), "r"(1 + group)
        : "memory");
    return r != 0;
}

template <int kOut, int kN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    mx4_matmul_pair_kernel(const __grid_constant__ Mx4PairKernel p) {
    using G = PairTile<kN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* staging = smem + G::kStages * G::kStage;
    uint64_t* full = reinterpret_cast<uint64_t*>(staging + G::kStaging);  // leader's: both CTAs' copies
    uint64_t* empty = full + G::kStages;                                  // own stage free
    uint64_t* scaled = empty + G::kStages;                                // leader's: scales in both tensor memories
    uint64_t* acc_full = scaled + G::kStages;                             // own accumulator buffer final
    uint64_t* acc_empty = acc_full + G::kBuffers;                         // leader's: both CTAs drained the buffer
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + G::kBuffers);
    WaitCtl* wc = reinterpret_cast<WaitCtl*>(tmem_slot + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int32_t tiles = p.m_tiles * p.n_tiles, first = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < G::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&scaled[s], 1);
        }
        for (int b = 0; b < G::kBuffers; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 16);  // eight epilogue warps in each CTA
        }
        wc->abort = 0;
        wc->limit = p.wait_limit;
        fence_barrier_init();
    }
    __syncthreads();
    cluster_arrive();
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    cluster_wait();  // barriers of both CTAs initialised before any remote arrival
    if (warp != 0) {  // the copies start at once; the other warps meet when the tensor memory is there
        tcgen05_before_sync();
        asm volatile("bar.sync 3, %0;" ::"n"(kPairThreads - 32) : "memory");
        tcgen05_after_sync();
    }
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);

    if (warp == 0 && lane == 0) {
        // ---------------------------------------------------------------- producer (both CTAs)
        const uint32_t leader_full = map_to_rank(smem_u32(&full[0]), 0);
        grid_dependency_wait();  // A may be the preceding kernel's output
        int i = 0;
        bool ok = true;
        for (int32_t t = first; ok && t < tiles; t += step) {
            const int32_t nt = t / p.m_tiles, mt = t - nt * p.m_tiles;
            const int32_t rt = 2 * mt + static_cast<int32_t>(rank);  // this CTA's group of 128 rows
            for (int32_t kb = 0; kb < p.k_blocks; ++kb, ++i) {
                const int s = i % G::kStages;
                ok = mbar_wait(&empty[s], ((i / G::kStages) & 1) ^ 1, wc);
                if (!ok) break;
                if (kb == p.fault_block) continue;
                if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * G::kStage);
                uint8_t* st = smem + s * G::kStage;
                const uint32_t bar = leader_full + s * 8;
                tma_load_2d_pair(st, &p.tm_a, kb * (kKStage / 2), rt * 128, bar);
                tma_load_2d_pair(st + G::kABytes, &p.tm_w, kb * (kKStage / 2), nt * kN + static_cast<int32_t>(rank) * (kN / 2), bar);
                uint8_t* sc = st + G::kABytes + G::kWBytes;
                tma_load_2d_pair(sc, &p.tm_sa, 0, rt * p.k_tiles + 2 * kb, bar);
#pragma unroll
                for (int j = 0; j < kN / 128; ++j)
                    tma_load_2d_pair(sc + kScaleBytes * (1 + j), &p.tm_sw, 0, (nt * (kN / 128) + j) * p.k_tiles + 2 * kb, bar);
            }
        }
        if (aborted(wc) && rank == 0) {  // copies in flight land on the leader's barriers: wait for them (bounded)
            const long long t0 = clock64();
            for (int k = max(0, i - G::kStages); k < i; ++k)
                while (k % p.k_blocks != p.fault_block && !mbar_try_wait(&full[k % G::kStages], (k / G::kStages) & 1) && clock64() - t0 < wc->limit) {
                }
        }
    } else if (warp == 1 && rank == 0) {
        // ---------------------------------------------------------------- MMA issuer (leader)
        // The whole warp walks the loop, so that addresses and descriptors stay in uniform registers, and
        // one elected lane issues: a product is issued in fewer cycles than the 128 it takes.
        const uint64_t da0 = smem_desc(smem_u32(smem), 16, 1024, kLayoutSw128);
        const uint64_t dw0 = smem_desc(smem_u32(smem) + G::kABytes, 16, 1024, kLayoutSw128);
        int s = 0, phase = 0, n = 0;
        bool ok = true;
        for (int32_t t = first; ok && t < tiles; t += step, ++n) {
            const int b = n % G::kBuffers;
            ok = __all_sync(0xffffffffu, mbar_wait(&acc_empty[b], ((n / G::kBuffers) & 1) ^ 1, wc));
            if (!ok) break;
            tcgen05_after_sync();
            const uint32_t acc = tmem + b * kN;
            for (int32_t kb = 0; kb < p.k_blocks; ++kb) {
                ok = __all_sync(0xffffffffu, mbar_wait(&scaled[s], phase, wc));
                if (!ok) break;
                tcgen05_after_sync();
                const uint64_t da = da0 + static_cast<uint64_t>(s * (G::kStage / 16)), dw = dw0 + static_cast<uint64_t>(s * (G::kStage / 16));
                const uint32_t sf = tmem + 256 + s * G::kScaleCols;  // A: 2 tiles x 4 columns; W: 2 x 4 kN / 128
                const uint32_t bar = smem_u32(&empty[s]), done = smem_u32(&acc_full[b]);
                const int32_t steps = min(4, (p.K - kb * kKStage + 63) / 64);
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        if (ks < steps)
                            umma_mx4_pair(acc, da + 2 * ks, dw + 2 * ks, idesc_mx4_pair<kN>((ks & 1) * 2), sf + 4 * (ks >> 1),
                                          sf + 8 + (ks >> 1) * (kN / 128) * 4, (kb > 0 || ks > 0) ? 1u : 0u);
                    umma_commit_pair_both(bar);
                    if (kb == p.k_blocks - 1) umma_commit_pair_both(done);
                }
                __syncwarp();
                if (++s == G::kStages) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
    } else if (warp == 10) {
        // ---------------------------------------------------------------- scale copies (leader)
        // A thread of their own: tcgen05.cp and the products that follow it in one thread run one after
        // the other, which cost 1300 cycles per stage against the products' 512.
        if (rank == 0) {
            const uint64_t d0 = smem_desc(smem_u32(smem) + G::kABytes + G::kWBytes, 16, 128, 0);
            const uint32_t own_scaled = map_to_rank(smem_u32(&scaled[0]), 0);
            int s = 0, phase = 0;
            bool ok = true;
            for (int32_t t = first; ok && t < tiles; t += step) {
                for (int32_t kb = 0; kb < p.k_blocks; ++kb) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&full[s], phase, wc));
                    if (!ok) break;
                    tcgen05_after_sync();
                    const uint64_t d = d0 + static_cast<uint64_t>(s * (G::kStage / 16));
                    const uint32_t sf = tmem + 256 + s * G::kScaleCols, bar = own_scaled + s * 8;
                    const int32_t halves = min(2, p.k_tiles - 2 * kb);
                    if (elect_one()) {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (j < halves) {
                                copy_scales_pair(sf + 4 * j, d + 32 * j);
#pragma unroll
                                for (int q = 0; q < kN / 128; ++q)
                                    copy_scales_pair(sf + 8 + (j * (kN / 128) + q) * 4, d + 64 * (1 + q) + 32 * j);
                            }
                        umma_commit_pair(bar);
                    }
                    __syncwarp();
                    if (++s == G::kStages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
        }
    } else if (warp >= 2) {
        // ---------------------------------------------------------------- epilogue (both CTAs)
        const int quarter = warp & 3, group = (warp - 2) >> 2;
        const int row = quarter * 32 + lane;
        const bool issuer = threadIdx.x == 64 + 128 * group;
        const uint32_t leader_empty = map_to_rank(smem_u32(&acc_empty[0]), 0);
        const uint32_t area = smem_u32(staging) + group * G::kSlabBytes;
        const uint32_t row_base = area + row * 128;
        const uint32_t sw = row & 7;
        constexpr int kCols = kN / 2;  // of the group
        int n = 0;
        for (int32_t t = first; t < tiles; t += step, ++n) {
            const int32_t nt = t / p.m_tiles, mt = t - nt * p.m_tiles;
            const int b = n % G::kBuffers;
            const bool got = mbar_wait(&acc_full[b], (n / G::kBuffers) & 1, wc);
            if (group_sync_or(group, !got)) break;  // (and the issuer has seen the last slab read out)
            tcgen05_after_sync();
            const uint32_t acc = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + b * kN + group * kCols;
            const int32_t row0 = (2 * mt + static_cast<int32_t>(rank)) * 128;
            const int32_t col0 = nt * kN + group * kCols;
            if (kOut == kOutGeluMx4) {
                const bool valid = row0 + row < p.M;
                const int64_t r = row0 + row;
                uint32_t word = 0, all[kCols];
#pragma unroll
                for (int c = 0; c < kCols; c += 32) tmem_ld_32x32b_x32_nowait(acc + c, all + c);
                tmem_ld_wait();
                tcgen05_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(leader_empty + b * 8);
#pragma unroll
                for (int c = 0; c < kCols; c += 32) {
                    const uint32_t* v = all + c;
                    float f[32], most[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int q = 0; q < 32; q += 2) {
                        unpair(gelu_pair(pair(__uint_as_float(v[q]), __uint_as_float(v[q + 1]))), f[q], f[q + 1]);
                        most[q & 3] = max_abs_nan(most[q & 3], f[q]);
                        most[(q & 3) + 1] = max_abs_nan(most[(q & 3) + 1], f[q + 1]);
                    }
                    const uint32_t top = __float_as_uint(max_abs_nan(max_abs_nan(most[0], most[1]), max_abs_nan(most[2], most[3])));
                    const bool in = valid && col0 + c < p.N;
                    const uint32_t sb = in ? scale_byte(top) : kUnitScale;
                    if (in && DG_CHECKED(g_device_error, r < p.M && col0 + c + 32 <= p.N)) {
                        const float inv = inverse_scale(sb == 255u ? 127u : sb);
                        uint32_t q4[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float(&g)[8] = *reinterpret_cast<const float(*)[8]>(&f[8 * q]);
                            q4[q] = sb == 255u ? 0u : pack_e2m1(g, inv);
                        }
                        *reinterpret_cast<uint4*>(p.out_codes + r * (p.N / 2) + (col0 + c) / 2) = make_uint4(q4[0], q4[1], q4[2], q4[3]);
                    }
                    word |= sb << (8 * ((col0 + c) / 32 & 3));
                    // whole tiles of 128 rows x 4 blocks; a group of 64 columns writes its half of the words
                    if (kCols == 64 ? c == 32 : (c & 127) == 96) {
                        const int32_t kt = (col0 + c) / 128, kts = (p.N + 127) / 128;
                        if (kt < kts && row0 < (p.M + 127) / 128 * 128) {
                            uint8_t* at = p.out_scales + (static_cast<int64_t>(row0 / 128) * kts + kt) * 512 + lane * 16 + quarter * 4;
                            if (kCols == 64)
                                *reinterpret_cast<uint16_t*>(at + 2 * group) = static_cast<uint16_t>(word >> (16 * group));
                            else
                                *reinterpret_cast<uint32_t*>(at) = word;
                        }
                        word = 0;
                    }
                }
            } else {
                // The whole share of the accumulator goes to registers first: the next tile's products wait
                // only for that.  Then slab by slab through shared memory, in boxes of 32 rows with one in
                // flight: a burst of stores would hold up the copies behind it (42 us instead of 35).
                constexpr int kSlabCols = kOut == kOutBf16 ? 64 : 32;
                uint32_t v[kCols];
#pragma unroll
                for (int c = 0; c < kCols; c += 32) tmem_ld_32x32b_x32_nowait(acc + c, v + c);
                tmem_ld_wait();
                tcgen05_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(leader_empty + b * 8);
#pragma unroll
                for (int s0 = 0; s0 < kCols; s0 += kSlabCols) {
                    if (s0 > 0) group_sync_or(group, false);  // the issuer has seen the slab before read out
#pragma unroll
                    for (int c = 0; c < kSlabCols; c += 32) {
                        const uint32_t* w = v + s0 + c;
                        if (kOut == kOutBf16) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                st_shared_v4(row_base + (((c / 8 + k) ^ sw) << 4),
                                             make_uint4(pack_bf16x2(__uint_as_float(w[8 * k]), __uint_as_float(w[8 * k + 1])),
                                                        pack_bf16x2(__uint_as_float(w[8 * k + 2]), __uint_as_float(w[8 * k + 3])),
                                                        pack_bf16x2(__uint_as_float(w[8 * k + 4]), __uint_as_float(w[8 * k + 5])),
                                                        pack_bf16x2(__uint_as_float(w[8 * k + 6]), __uint_as_float(w[8 * k + 7]))));
                        } else {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                st_shared_v4(row_base + ((k ^ sw) << 4), make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
                        }
                    }
                    fence_proxy_async_smem();
                    group_sync_or(group, false);
                    if (issuer && col0 + s0 < p.N) {
#pragma unroll 1
                        for (int q = 0; q < 4 && row0 + 32 * q < p.M; ++q) {
                            if (!DG_CHECKED(g_device_error, col0 + s0 < p.N && row0 + 32 * q < p.M && t < tiles)) continue;
                            tma_store_2d(&p.tm_out, col0 + s0, row0 + 32 * q, area + q * 4096);
                            bulk_commit();
                            bulk_wait_read_all();
                        }
                    }
                }
            }
        }
        if (issuer) bulk_wait_all();  // complete before the CTA may exit
    }
    __syncwarp();
    grid_launch_dependents();
    // neither CTA leaves (or frees its tensor memory) while its peer may still use it
    tcgen05_before_sync();
    __syncthreads();
    cluster_sync();
    tcgen05_after_sync();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

template <int kOut, int kN>
cudaError_t launch_pair(const Mx4MatmulParams& q, cudaStream_t st) {
    using G = PairTile<kN>;
    static DeviceOnce once;
    const cudaError_t attr_err = allow_shared_memory(once, mx4_matmul_pair_kernel<kOut, kN>, static_cast<int>(G::kSmem));
    if (attr_err != cudaSuccess) return attr_err;
    Mx4PairKernel kp;
    std::memset(&kp, 0, sizeof(kp));
    kp.M = q.M;
    kp.N = q.N;
    kp.K = q.K;
    kp.m_tiles = (q.M + 255) / 256;
    kp.n_tiles = (q.N + kN - 1) / kN;
    kp.k_tiles = (q.K + 127) / 128;
    kp.k_blocks = (q.K + kKStage - 1) / kKStage;
    kp.wait_limit = q.wait_limit > 0 ? q.wait_limit : kWaitLimitCycles;
    kp.fault_block = q.wait_limit > 0 ? q.fault_block : -1;
    kp.out_codes = static_cast<uint8_t*>(q.out);
    kp.out_scales = q.out_scales;
    const uint64_t ta = static_cast<uint64_t>((q.M + 127) / 128) * kp.k_tiles, tw = static_cast<uint64_t>((q.N + 127) / 128) * kp.k_tiles;
    const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8, u32 = CU_TENSOR_MAP_DATA_TYPE_UINT32;
    cudaError_t e = encode_2d(&kp.tm_a, u8, q.a, q.K / 2, q.M, q.K / 2, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess) e = encode_2d(&kp.tm_w, u8, q.w, q.K / 2, q.N, q.K / 2, 128, kN / 2, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess) e = encode_2d(&kp.tm_sa, u32, q.a_scales, 128, ta, 512, 128, 2, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (e == cudaSuccess) e = encode_2d(&kp.tm_sw, u32, q.w_scales, 128, tw, 512, 128, 2, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (e == cudaSuccess && kOut == kOutBf16)
        e = encode_2d(&kp.tm_out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, q.out, q.N, q.M, static_cast<uint64_t>(q.N) * 2, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess && kOut == kOutF32)
        e = encode_2d(&kp.tm_out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, q.out, q.N, q.M, static_cast<uint64_t>(q.N) * 4, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    const int64_t tiles = static_cast<int64_t>(kp.m_tiles) * kp.n_tiles;
    if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<int64_t>(tiles, num_sms() / 2)));
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = G::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = q.dependent ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, mx4_matmul_pair_kernel<kOut, kN>, kp);
    if (e != cudaSuccess) return e;
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace

size_t mx4_scale_bytes(int32_t rows, int32_t K) {
    return static_cast<size_t>((static_cast<int64_t>(rows) + 127) / 128) * ((static_cast<int64_t>(K) + 127) / 128) * 512;
}

cudaError_t launch_mx4_quantize(const void* x, int64_t ld, int is_bf16, int32_t rows, int32_t K, uint8_t* codes, uint8_t* scales,
                                cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(rows) + 127) / 128 * 16), static_cast<unsigned>((K + kMx4Cols - 1) / kMx4Cols));
    if (grid.y > 65535u) return cudaErrorInvalidValue;
    if (is_bf16)
        mx4_quantize_kernel<<<grid, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(x), ld, rows, K, codes, scales);
    else
        mx4_quantize_kernel<<<grid, 256, 0, st>>>(static_cast<const float*>(x), ld, rows, K, codes, scales);
    note_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int32_t rows, int32_t K, void* out, int is_bf16,
                                  cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>((rows + 7LL) / 8), static_cast<unsigned>((K + kMx4Cols - 1) / kMx4Cols));
    if (grid.y > 65535u) return cudaErrorInvalidValue;
    if (is_bf16)
        mx4_dequantize_kernel<<<grid, 256, 0, st>>>(codes, scales, rows, K, static_cast<__nv_bfloat16*>(out));
    else
        mx4_dequantize_kernel<<<grid, 256, 0, st>>>(codes, scales, rows, K, static_cast<float*>(out));
    note_launches(1);
    return cudaGetLastError();
}

Mx4Plan mx4_plan(int32_t M, int32_t N, int32_t K) {
    // Which kernel, from sizes alone (us a product [L2], K = 2048 unless said):
    //  * more 256 x 128 tiles than pairs: 256 x 256 tiles (96 tiles: 8.6, with 128 columns 10.2, single
    //    CTAs 14.7; a block on 4096 rows of 2048: 70, with 128 columns 83);
    //  * fewer: 256 x 128 tiles (64 tiles: 7.0, single CTAs 8.2), unless splitting K makes up for it, which takes
    //    K > 2048 (32 tiles at K = 8192: 14.9, split in two 12.5);
    //  * up to 128 rows half of a pair's tile is empty, and single CTAs do better where they fit one wave
    //    (128 tiles of 64 rows, K = 8192: 17.1, pairs 19.1; 256 tiles, K = 2048: 16.0, pairs 12.8) or four splits
    //    shorten K > 1024 (16 tiles of 17 rows: 5.3, pairs 6.1; 32 tiles of 64 rows, K = 1024: 6.0, pairs 5.2; 64
    //    tiles of 64 rows, two splits: 7.2, pairs 6.7);
    //  * up to kMx4FewRows rows single CTAs, which alone take A as bf16: their epilogue is as short as the pairs' (8
    //    tiles of a row: 4.7, pairs 4.8).
    const int64_t pairs = static_cast<int64_t>((M + 255) / 256) * ((N + 127) / 128);
    const int64_t singles = static_cast<int64_t>((M + kMTile - 1) / kMTile) * ((N + kNTile - 1) / kNTile);
    const int32_t k_blocks = (K + kKStage - 1) / kKStage;
    // single CTAs: split K while the clusters fit one wave and every split keeps a block.  (Clusters of
    // eight are placed two to a GPC at most: 200 x 1000 x 4096 took 10.8 us split in eight, 7.5 in four.  GPCs
    // hold unequal numbers of SMs, so not all 148 take clusters of four: 33 tiles in four splits, K = 6624, 100
    // rows, 9.8 us, 34 tiles 16.1, and 38 in two 11.3.  Every GPC of 16 SMs or more has room for four.)
    int splits = 1;
    while (splits < 4 && 2 * splits * singles <= (splits == 1 ? num_sms() : 128) && 2 * splits <= k_blocks) splits *= 2;
    const bool paired = M > 128 ? splits == 1 || k_blocks <= 8
                                : M > kMx4FewRows && (k_blocks <= 4 || (k_blocks <= 8 && splits == 2) || singles > num_sms());
    if (paired) return {0, 2 * pairs > num_sms() ? 256 : 128};
    return {splits, kNTile};
}

cudaError_t launch_mx4_matmul(const Mx4MatmulParams& q, cudaStream_t st) {
    const Mx4Plan plan = mx4_plan(q.M, q.N, q.K);
    if (plan.splits == 0) {
        const bool wide = plan.columns == 256;
        if (q.out_kind == kMx4OutF32) return wide ? launch_pair<kOutF32, 256>(q, st) : launch_pair<kOutF32, 128>(q, st);
        if (q.out_kind == kMx4OutBf16) return wide ? launch_pair<kOutBf16, 256>(q, st) : launch_pair<kOutBf16, 128>(q, st);
        return wide ? launch_pair<kOutGeluMx4, 256>(q, st) : launch_pair<kOutGeluMx4, 128>(q, st);
    }
    const int splits = plan.splits;
    Mx4Kernel kp;
    std::memset(&kp, 0, sizeof(kp));
    cudaError_t e = cudaSuccess;
    if (!q.a_bf16) e = encode_2d(&kp.tm_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, q.a, q.K / 2, q.M, q.K / 2, 128, kMTile, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess)
        e = encode_2d(&kp.tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, q.w, q.K / 2, q.N, q.K / 2, 128, kNTile, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    kp.sa = q.a_scales;
    kp.sw = q.w_scales;
    kp.a_bf16 = static_cast<const __nv_bfloat16*>(q.a_bf16);
    kp.out = q.out;
    kp.out_scales = q.out_scales;
    kp.M = q.M;
    kp.N = q.N;
    kp.K = q.K;
    kp.n_tiles = (q.N + kNTile - 1) / kNTile;
    kp.k_tiles = (q.K + 127) / 128;
    kp.k_blocks = (q.K + kKStage - 1) / kKStage;
    kp.wait_limit = q.wait_limit > 0 ? q.wait_limit : kWaitLimitCycles;
    kp.fault_block = q.wait_limit > 0 ? q.fault_block : -1;
    const int64_t grid = static_cast<int64_t>((q.M + kMTile - 1) / kMTile) * kp.n_tiles * splits;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (q.out_kind == kMx4OutF32) return launch_product<kOutF32>(kp, static_cast<int>(grid), splits, q.dependent != 0, st);
    if (q.out_kind == kMx4OutBf16) return launch_product<kOutBf16>(kp, static_cast<int>(grid), splits, q.dependent != 0, st);
    if (q.a_bf16) return launch_product<kOutGeluMx4, true>(kp, static_cast<int>(grid), splits, q.dependent != 0, st);
    return launch_product<kOutGeluMx4>(kp, static_cast<int>(grid), splits, q.dependent != 0, st);
}

cudaError_t read_and_clear_mx4_error(int* out) {
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

}  // namespace dg
