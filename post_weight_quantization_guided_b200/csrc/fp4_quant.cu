// fp4_quant.cu -- quantising a matrix to a microscaled 4-bit format and reading it back.
//
//   MX: s = 2^(floor(log2 amax) - 2) over blocks of 32;  NV: s = E4M3(amax / (6 t)) over 16;
//   code = E2M1(x / (s t)), nearest, ties to even, at most 6 in magnitude.
//
// Bound: HBM (read x, write half a byte an element). One pass: a lane takes 8 consecutive
// elements (one or two 16-byte loads, 4 bytes of codes out), 4 (MX) or 2 (NV) neighbouring lanes
// hold a block and agree on its largest element by shuffles, a warp covers 256 elements of a row.
//
// Exact decisions. MX quotients are exact (a power of two). An NV quotient x / (s t) is estimated
// in 32 bits and rounded to a code twice, a little below and a little above the estimate; where
// both give one code it is the right one. Where they differ the quotient is near the border b of
// two codes, and the sign of |x| - (b s) t decides: b s has at most 7 bits, so one fused
// multiply-add gives that sign exactly. The block scale is found in 64 bits (below).
#include <cuda_fp8.h>

#include "fp4.cuh"
#include "profile.cuh"

namespace lnq {

constexpr int kQuantThreads = 256;
constexpr int kSpan = 256;  // elements of a row that a warp takes at a time (8 a lane)

// ------------------------------------------------------------------------------------------
// Rows of 8 elements
// ------------------------------------------------------------------------------------------
// x[0..7], zeros from element `left` on. `wide`: 16-byte loads are possible (and left >= 8).
template <typename T>
__device__ __forceinline__ void load8(const T *__restrict__ p, int left, bool wide, float (&v)[8])
{
    if (wide && left >= 8) {
        alignas(16) T e[8];
        constexpr int kLoads = sizeof(T) * 8 / 16;
#pragma unroll
        for (int k = 0; k < kLoads; ++k)
            reinterpret_cast<uint4 *>(e)[k] = __ldg(reinterpret_cast<const uint4 *>(p) + k);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = to_f32<T>(e[k]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = k < left ? to_f32<T>(p[k]) : 0.f;
    }
}

template <typename T>
__device__ __forceinline__ void store8(T *__restrict__ p, int left, bool wide, const float (&v)[8])
{
    if (wide && left >= 8) {
        alignas(16) T e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            e[k] = from_f32<T>(v[k]);
        constexpr int kStores = sizeof(T) * 8 / 16;
#pragma unroll
        for (int k = 0; k < kStores; ++k)
            reinterpret_cast<uint4 *>(p)[k] = reinterpret_cast<const uint4 *>(e)[k];
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < left)
                p[k] = from_f32<T>(v[k]);
    }
}

// The codes of 8 numbers (nearest, ties to even, saturating), element k in bits 4k+3 .. 4k.
__device__ __forceinline__ uint32_t e2m1x8(const float (&q)[8])
{
    uint32_t out;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(out)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    return out;
}

// q as a float that rounds to few bits as q itself would: towards zero, and the last bit set if
// anything was lost.
__device__ __forceinline__ float to_odd(double q)
{
    const float f = __double2float_rz(q);
    return static_cast<double>(f) == q ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// ------------------------------------------------------------------------------------------
// Block scales
// ------------------------------------------------------------------------------------------
// What a thread keeps of the matrix scale t.
struct MatrixScale {
    float t, rt;       // t, about 1 / t
    double r6;         // 1 / (6 t)
    bool valid, fast;  // t positive and finite; s t and 1 / (s t) normal 32-bit numbers for every s
};

__device__ __forceinline__ MatrixScale matrix_scale(const float *t)
{
    MatrixScale m;
    m.t = t == nullptr ? 1.f : __ldg(t);
    m.valid = m.t > 0.f && m.t < __uint_as_float(0x7F800000u);
    m.fast = m.t >= 0x1p-100f && m.t <= 0x1p115f;
    m.rt = 1.f / m.t;
    m.r6 = 1.0 / (6.0 * static_cast<double>(m.t));
    return m;
}

// E4M3(amax / (6 t)). The 64-bit quotient is within 2^-51 of the exact one. It is rounded to 40
// bits, which puts a quotient on the border of two E4M3 numbers back on it, and moves none that
// is not there onto it: amax and 6 t b (b a border, 5 bits) are whole numbers of at most 24 and 31
// bits on one scale, so a quotient off the border is at least 2^-31 away from it.
__device__ __forceinline__ uint32_t nv_scale_byte(float amax, const MatrixScale &m)
{
    const double q = static_cast<double>(amax) * m.r6;
    double q40 = q;
    if (q < 1024.0) {
        const double big = __dmul_rn(q, 8193.0);
        q40 = __dsub_rn(big, __dsub_rn(big, q));
    }
    return __nv_cvt_float_to_fp8(to_odd(fmin(q40, 1024.0)), __NV_SATFINITE, __NV_E4M3);
}

// The 8 codes of an NV block with scale s, any t: quotients in 64 bits. A quotient on a border of
// two codes is exact; any other is at least 2^-31 away from it, further than its rounding.
__device__ __noinline__ uint32_t nv_codes_slow(const float (&v)[8], float s, float t)
{
    const double step = static_cast<double>(s) * static_cast<double>(t);
    float q[8];
    for (int k = 0; k < 8; ++k)
        q[k] = to_odd(fmax(-8.0, fmin(8.0, static_cast<double>(v[k]) / step)));
    return e2m1x8(q);
}

__device__ __forceinline__ uint32_t nv_codes(const float (&v)[8], float s, const MatrixScale &m)
{
    if (!m.fast)
        return nv_codes_slow(v, s, m.t);
    // relative error of v * r below 2^-21: three roundings and the approximate reciprocal
    const float r = __frcp_rn(s) * m.rt;
    const float below = r * (1.f - 0x1p-20f), above = r * (1.f + 0x1p-20f);
    float lo[8], hi[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        lo[k] = v[k] * below;
        hi[k] = v[k] * above;
    }
    uint32_t codes = e2m1x8(lo);
    const uint32_t upper = e2m1x8(hi);
    if (codes != upper) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t c = (codes >> (4 * k)) & 7u;
            if (((upper >> (4 * k)) & 7u) != c) {
                // the border between codes c and c + 1
                const float b = 0.5f * (fp4_code_value(c) + fp4_code_value(c + 1u));
                const float d = fmaf(-b * s, m.t, fabsf(v[k]));
                if (d > 0.f || (d == 0.f && (c & 1u)))
                    codes += 1u << (4 * k);
            }
        }
    }
    return codes;
}

// ------------------------------------------------------------------------------------------
// Kernels
// ------------------------------------------------------------------------------------------
template <typename T, int FMT>
__global__ void __launch_bounds__(kQuantThreads)
    fp4_quantize_kernel(const T *__restrict__ x, int64_t rows, int64_t d, int64_t ldx, bool wide,
                        const float *__restrict__ t, uint8_t *__restrict__ codes,
                        uint8_t *__restrict__ scales)
{
    constexpr int kLanes = fp4_block(FMT) / 8;  // lanes that hold one block
    const int lane = threadIdx.x & 31;
    const int64_t padded = fp4_padded(d), spans = (padded + kSpan - 1) / kSpan;
    const int64_t total = rows * spans;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (kQuantThreads / 32);
    MatrixScale m;
    if (FMT == LNQ_FP4_NV)
        m = matrix_scale(t);
    for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kQuantThreads / 32) + (threadIdx.x >> 5);
         w < total; w += stride) {
        const int64_t row = w / spans;
        const int64_t i0 = (w - row * spans) * kSpan + lane * 8;
        const int left = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(8), d - i0)));
        float v[8];
        load8(x + row * ldx + i0, left, wide, v);
        // largest magnitude, as bits: a NaN or an infinity is above every finite number
        uint32_t amax = 0u;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            amax = max(amax, __float_as_uint(v[k]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1)
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        uint32_t byte, word = 0u;
        if (FMT == LNQ_FP4_MX) {
            byte = 255u;
            if (amax < 0x7F800000u) {
                // exponent field of the scale: that of amax, less 2
                byte = max(static_cast<int>(amax >> 23) - 2, 0);
                const float r = __uint_as_float((254u - byte) << 23);
                float q[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    q[k] = v[k] * r;
                word = e2m1x8(q);
            }
        } else {
            byte = 127u;
            if (amax < 0x7F800000u && m.valid) {
                byte = nv_scale_byte(__uint_as_float(amax), m);
                if (byte != 0u)
                    word = nv_codes(v, fp4_scale_value<FMT>(byte), m);
            }
        }
        if (i0 < padded) {
            reinterpret_cast<uint32_t *>(codes + row * (padded / 2))[i0 / 8] = word;
            if (lane % kLanes == 0)
                scales[row * (padded / fp4_block(FMT)) + i0 / fp4_block(FMT)] =
                    static_cast<uint8_t>(i0 < d ? byte : 0u);
        }
    }
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kQuantThreads)
    fp4_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                          int64_t rows, int64_t d, const float *__restrict__ t, T *__restrict__ y,
                          int64_t ldy, bool wide)
{
    const int lane = threadIdx.x & 31;
    const int64_t padded = fp4_padded(d), spans = (padded + kSpan - 1) / kSpan;
    const int64_t total = rows * spans;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (kQuantThreads / 32);
    const float tv = t == nullptr ? 1.f : __ldg(t);
    for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kQuantThreads / 32) + (threadIdx.x >> 5);
         w < total; w += stride) {
        const int64_t row = w / spans;
        const int64_t i0 = (w - row * spans) * kSpan + lane * 8;
        if (i0 >= d)
            continue;
        const uint32_t word =
            __ldg(reinterpret_cast<const uint32_t *>(codes + row * (padded / 2)) + i0 / 8);
        const float s = fp4_scale_value<FMT>(
            __ldg(scales + row * (padded / fp4_block(FMT)) + i0 / fp4_block(FMT)));
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = fp4_code_value((word >> (4 * k)) & 15u) * s * tv;
        store8(y + row * ldy + i0, static_cast<int>(min(static_cast<int64_t>(8), d - i0)), wide, v);
    }
}

// The largest finite magnitude, as bits, into *top (zero before): an integer maximum, so the
// order of the blocks does not matter.
template <typename T>
__global__ void __launch_bounds__(kQuantThreads)
    fp4_absmax_kernel(const T *__restrict__ x, int64_t rows, int64_t d, int64_t ldx, bool wide,
                      uint32_t *__restrict__ top)
{
    const int lane = threadIdx.x & 31;
    const int64_t spans = (d + kSpan - 1) / kSpan, total = rows * spans;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (kQuantThreads / 32);
    uint32_t amax = 0u;
    for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kQuantThreads / 32) + (threadIdx.x >> 5);
         w < total; w += stride) {
        const int64_t row = w / spans;
        const int64_t i0 = (w - row * spans) * kSpan + lane * 8;
        const int left = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(8), d - i0)));
        float v[8];
        load8(x + row * ldx + i0, left, wide, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t b = __float_as_uint(v[k]) & 0x7FFFFFFFu;
            amax = max(amax, b < 0x7F800000u ? b : 0u);
        }
    }
    __shared__ uint32_t part[kQuantThreads / 32];
    amax = __reduce_max_sync(0xffffffffu, amax);
    if (lane == 0)
        part[threadIdx.x >> 5] = amax;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int k = 1; k < kQuantThreads / 32; ++k)
            amax = max(amax, part[k]);
        if (amax != 0u)
            atomicMax(top, amax);
    }
}

__global__ void fp4_scale_from_absmax_kernel(float *t)
{
    const float s = *t / 2688.f;
    *t = s > 0.f ? s : 1.f;
}

// ------------------------------------------------------------------------------------------
// Host launchers
// ------------------------------------------------------------------------------------------
static bool wide_rows(const void *p, int64_t ld, int size)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * size) % 16 == 0;
}

static unsigned span_blocks(int64_t rows, int64_t d, int num_sms)
{
    const int64_t spans = rows * ((fp4_padded(d) + kSpan - 1) / kSpan);
    const int64_t blocks = (spans + kQuantThreads / 32 - 1) / (kQuantThreads / 32);
    return static_cast<unsigned>(min(blocks, static_cast<int64_t>(num_sms) * 8));
}

template <typename F>
static cudaError_t by_type(int type, F f)
{
    switch (type) {
    case LNQ_F32: return f(static_cast<float *>(nullptr));
    case LNQ_BF16: return f(static_cast<__nv_bfloat16 *>(nullptr));
    case LNQ_F16: return f(static_cast<__half *>(nullptr));
    }
    return cudaErrorInvalidValue;
}

cudaError_t fp4_tensor_scale_launch(const void *x, int xt, int64_t rows, int64_t d, int64_t ldx,
                                    float *t, int num_sms, cudaStream_t s)
{
    cudaError_t e = cudaMemsetAsync(t, 0, sizeof(float), s);
    if (e != cudaSuccess)
        return e;
    if (rows > 0) {
        KernelTimer timer("lnq_fp4_absmax", s);
        e = by_type(xt, [&](auto *p) {
            using T = std::remove_pointer_t<decltype(p)>;
            fp4_absmax_kernel<T><<<span_blocks(rows, d, num_sms), kQuantThreads, 0, s>>>(
                static_cast<const T *>(x), rows, d, ldx, wide_rows(x, ldx, sizeof(T)),
                reinterpret_cast<uint32_t *>(t));
            return cudaGetLastError();
        });
        if (e != cudaSuccess)
            return e;
    }
    fp4_scale_from_absmax_kernel<<<1, 1, 0, s>>>(t);
    return cudaGetLastError();
}

cudaError_t fp4_quantize_launch(const void *x, int xt, int64_t rows, int64_t d, int64_t ldx,
                                int fmt, const float *t, uint8_t *codes, uint8_t *scales,
                                int num_sms, cudaStream_t s)
{
    KernelTimer timer("lnq_fp4_quantize", s);
    return by_type(xt, [&](auto *p) {
        using T = std::remove_pointer_t<decltype(p)>;
        auto *kernel = fmt == LNQ_FP4_MX ? fp4_quantize_kernel<T, LNQ_FP4_MX>
                                         : fp4_quantize_kernel<T, LNQ_FP4_NV>;
        kernel<<<span_blocks(rows, d, num_sms), kQuantThreads, 0, s>>>(
            static_cast<const T *>(x), rows, d, ldx, wide_rows(x, ldx, sizeof(T)), t, codes, scales);
        return cudaGetLastError();
    });
}

cudaError_t fp4_dequantize_launch(const uint8_t *codes, const uint8_t *scales, int64_t rows,
                                  int64_t d, int fmt, const float *t, void *y, int yt, int64_t ldy,
                                  int num_sms, cudaStream_t s)
{
    KernelTimer timer("lnq_fp4_dequantize", s);
    return by_type(yt, [&](auto *p) {
        using T = std::remove_pointer_t<decltype(p)>;
        auto *kernel = fmt == LNQ_FP4_MX ? fp4_dequantize_kernel<T, LNQ_FP4_MX>
                                         : fp4_dequantize_kernel<T, LNQ_FP4_NV>;
        kernel<<<span_blocks(rows, d, num_sms), kQuantThreads, 0, s>>>(
            codes, scales, rows, d, t, static_cast<T *>(y), ldy, wide_rows(y, ldy, sizeof(T)));
        return cudaGetLastError();
    });
}

}  // namespace lnq
