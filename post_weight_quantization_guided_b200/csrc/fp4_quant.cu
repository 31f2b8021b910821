// fp4_quant.cu -- quantising a matrix to a microscaled 4-bit format and reading it back.
//
//   MX: s = 2^(floor(log2 amax) - 2) over blocks of 32;  NV: s = E4M3(amax / (6 t)) over 16;
//   code = E2M1(x / (s t)), nearest, ties to even, at most 6 in magnitude.
//
// Bound: HBM (read x, write half a byte an element). One pass: a lane takes 16 consecutive
// elements, an NV block or half an MX one (whose two lanes agree on its largest element by a
// shuffle), a warp 512 elements of a row. One B200, 16384 x 4096 bf16: MX 28 us (the bytes alone 26 at
// the copy rate), NV 37 to 40 us (a span is loaded and then worked on, with nothing in flight
// meanwhile: issue slots 60 to 65% busy, integer pipe 51 to 56%, DRAM 27%), reading back 34 us, the matrix
// scale 24.5 and 2 for its quotient; 4096 x 11008 f32: 34 to 38, reading back 36, the scale 32.
// Rows whose pitch is no multiple of 16 bytes go element by element: 16384 x 4095 bf16 takes 71
// (MX) and 73 us, reading back 206, the scale 74; 4096 x 11007 f32 96 (MX) and 88, 67, 85.
//
// Exact decisions. MX quotients are exact (a power of two). An NV quotient is estimated in 32 bits
// and rounded twice, a little below and a little above the estimate; where both agree that is the
// answer. Where they differ the quotient is near the border b of two codes or of two scales (ties
// are frequent: 16-bit elements over a t that comes from one of them). The sign of |x| - (b s) t, or
// of amax - (6 b) t, then decides: b s and 6 b have at most 7 bits, so one fused multiply-add gives
// it exactly. Only a t near the ends of the 32-bit range takes 64-bit quotients.
#include <cuda_fp8.h>

#include <type_traits>

#include "fp4.cuh"
#include "profile.cuh"

namespace lnq {

constexpr int kQuantThreads = 256;
constexpr int kLane = 16;          // elements a lane takes at a time
constexpr int kSpan = 32 * kLane;  // and a warp, of one row

// ------------------------------------------------------------------------------------------
// A lane's 16 elements
// ------------------------------------------------------------------------------------------
template <typename T>
struct Elements {
    static constexpr int kWords = kLane * sizeof(T) / 16;
    uint4 w[kWords];
    __device__ __forceinline__ T get(int k) const
    {
        if constexpr (sizeof(T) == 4) {
            return __uint_as_float(reinterpret_cast<const uint32_t *>(w)[k]);
        } else {
            const uint32_t u = reinterpret_cast<const uint32_t *>(w)[k / 2];
            const unsigned short h = static_cast<unsigned short>(k & 1 ? u >> 16 : u);
            return *reinterpret_cast<const T *>(&h);
        }
    }
    // x[0..15], zeros from element `left` on; `wide`: 16-byte loads are possible
    __device__ __forceinline__ void load(const T *__restrict__ p, int left, bool wide)
    {
        if (wide && left >= kLane) {
#pragma unroll
            for (int k = 0; k < kWords; ++k)
                w[k] = __ldg(reinterpret_cast<const uint4 *>(p) + k);
            return;
        }
        uint32_t *u = reinterpret_cast<uint32_t *>(w);
#pragma unroll
        for (int k = 0; k < kLane; ++k) {
            if constexpr (sizeof(T) == 4) {
                u[k] = k < left ? __float_as_uint(p[k]) : 0u;
            } else {
                const uint32_t h = k < left ? reinterpret_cast<const unsigned short *>(p)[k] : 0u;
                u[k / 2] = k & 1 ? u[k / 2] | (h << 16) : h;
            }
        }
    }
    // The largest magnitude as the bits of a 32-bit number: above every finite one where there is
    // a NaN or an infinity.
    __device__ __forceinline__ uint32_t top() const
    {
        const uint32_t *u = reinterpret_cast<const uint32_t *>(w);
        if constexpr (sizeof(T) == 4) {
            uint32_t m = u[0] & 0x7FFFFFFFu;
#pragma unroll
            for (int k = 1; k < kLane; ++k)
                m = max(m, u[k] & 0x7FFFFFFFu);
            return m;
        } else {
            // pairs; the maximum with a NaN is a NaN, whose bits are above an infinity's
            uint32_t m = u[0] & 0x7FFF7FFFu;
#pragma unroll
            for (int k = 1; k < kLane / 2; ++k) {
                const uint32_t a = u[k] & 0x7FFF7FFFu;
                if constexpr (std::is_same_v<T, __nv_bfloat16>)
                    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(a));
                else
                    asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(m) : "r"(a));
            }
            const unsigned short h = static_cast<unsigned short>(max(m & 0xFFFFu, m >> 16));
            return __float_as_uint(to_f32<T>(*reinterpret_cast<const T *>(&h)));
        }
    }
};

// The spans of a matrix (kSpan elements of a row each), every hop-th for a warp. Rows and spans are
// carried along: one division a thread, where one a span took a third of the time.
struct SpanWalk {
    int64_t row, hop_rows, rows;
    int span, spans, hop_spans;  // a row has at most 2^24 elements
    __device__ __forceinline__ SpanWalk(int64_t rows_, int64_t width)
    {
        const int64_t warps = static_cast<int64_t>(gridDim.x) * (kQuantThreads / 32);
        const int64_t at = static_cast<int64_t>(blockIdx.x) * (kQuantThreads / 32) + (threadIdx.x >> 5);
        rows = rows_;
        spans = static_cast<int>((width + kSpan - 1) / kSpan);
        row = at / spans;
        span = static_cast<int>(at - row * spans);
        hop_rows = warps / spans;
        hop_spans = static_cast<int>(warps - hop_rows * spans);
    }
    __device__ __forceinline__ bool more() const { return row < rows; }
    // this lane's first element of the row
    __device__ __forceinline__ int element() const { return span * kSpan + (threadIdx.x & 31) * kLane; }
    __device__ __forceinline__ void next()
    {
        row += hop_rows;
        span += hop_spans;
        if (span >= spans) {
            span -= spans;
            ++row;
        }
    }
};

// The codes of 8 numbers (nearest, ties to even, saturating), element k in bits 4k+3 .. 4k.
__device__ __forceinline__ uint32_t e2m1x8(const float *q)
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

// The values of a word's 8 codes. (All are used: with four of them unused the compiler was seen to
// give zeros for the others.)
__device__ __forceinline__ void code_values(uint32_t w, float *v)
{
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[k]));
        v[2 * k] = f.x;
        v[2 * k + 1] = f.y;
    }
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
    float t, rt, rt6;  // t, about 1 / t, about 1 / (6 t)
    bool valid, fast;  // t positive and finite; s t and 1 / (s t) normal 32-bit numbers for every s
};

__device__ __forceinline__ MatrixScale matrix_scale(const float *t)
{
    MatrixScale m;
    m.t = t == nullptr ? 1.f : __ldg(t);
    m.valid = m.t > 0.f && m.t < __uint_as_float(0x7F800000u);
    m.fast = m.t >= 0x1p-100f && m.t <= 0x1p115f;
    m.rt = 1.f / m.t;
    m.rt6 = m.rt * (1.f / 6.f);
    return m;
}

// E4M3(amax / (6 t)). The 64-bit quotient is within 2^-51 of the exact one. It is rounded to 40
// bits, which puts a quotient on the border of two E4M3 numbers back on it, and moves none that
// is not there onto it: amax and 6 t b (b a border, 5 bits) are whole numbers of at most 24 and 31
// bits on one scale, so a quotient off the border is at least 2^-31 away from it.
__device__ __noinline__ uint32_t nv_scale_exact(float amax, float t)
{
    const double q = static_cast<double>(amax) / (6.0 * static_cast<double>(t));
    double q40 = q;
    if (q < 1024.0) {
        const double big = __dmul_rn(q, 8193.0);
        q40 = __dsub_rn(big, __dsub_rn(big, q));
    }
    return __nv_cvt_float_to_fp8(to_odd(fmin(q40, 1024.0)), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ uint32_t nv_scale_byte(float amax, const MatrixScale &m)
{
    // relative error of amax * rt6 below 2^-21: three roundings and that of the constant
    const float below = amax * (m.rt6 * (1.f - 0x1p-20f)), above = amax * (m.rt6 * (1.f + 0x1p-20f));
    unsigned short both;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(both) : "f"(above), "f"(below));
    const uint32_t byte = both & 255u, next = both >> 8;
    if (!m.fast)
        return nv_scale_exact(amax, m.t);
    if (byte == next)
        return byte;
    // near the border b of two neighbours: 6 b has at most 7 bits, so the sign of amax - 6 b t is exact
    const float b6 = 3.f * (fp4_scale_value<LNQ_FP4_NV>(byte) + fp4_scale_value<LNQ_FP4_NV>(next));
    const float d = fmaf(-b6, m.t, amax);
    return d > 0.f || (d == 0.f && (byte & 1u)) ? next : byte;
}

// The codes of an NV block (its first `left` elements at x) with scale s, any t: quotients in 64
// bits. A quotient on a border of two codes is exact; any other is at least 2^-31 away from it,
// further than its rounding. (The elements are read again: handing over registers would have
// every block written to local memory, which took half of the kernel's time.)
template <typename T>
__device__ __noinline__ uint2 nv_codes_slow(const T *__restrict__ x, int left, float s, float t)
{
    const double step = static_cast<double>(s) * static_cast<double>(t);
    uint32_t word[2] = {0u, 0u};
    for (int k = 0; k < min(left, kLane); ++k) {
        float q[8] = {};
        q[0] = to_odd(fmax(-8.0, fmin(8.0, static_cast<double>(to_f32<T>(x[k])) / step)));
        word[k >> 3] |= e2m1x8(q) << (4 * (k & 7));
    }
    return make_uint2(word[0], word[1]);
}

// v[k] * r for pairs, packed.
__device__ __forceinline__ void scale16(const float (&v)[kLane], float r, float (&q)[kLane])
{
    uint64_t rr;
    asm("mov.b64 %0, {%1, %1};" : "=l"(rr) : "f"(r));
#pragma unroll
    for (int k = 0; k < kLane; k += 2) {
        uint64_t pair;
        asm("mov.b64 %0, {%1, %2};" : "=l"(pair) : "f"(v[k]), "f"(v[k + 1]));
        asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(pair) : "l"(rr));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(q[k]), "=f"(q[k + 1]) : "l"(pair));
    }
}

// The codes of an NV block with scale s; v are its elements, x where they (the first `left`) are.
template <typename T>
__device__ __forceinline__ uint2 nv_codes(const float (&v)[kLane], const T *__restrict__ x, int left, float s,
                                          const MatrixScale &m)
{
    if (!m.fast)
        return nv_codes_slow<T>(x, left, s, m.t);
    // relative error of v * r below 2^-21: three roundings and the approximate reciprocal
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    r *= m.rt;
    float q[kLane];
    scale16(v, r * (1.f - 0x1p-20f), q);
    uint2 codes = make_uint2(e2m1x8(q), e2m1x8(q + 8));
    scale16(v, r * (1.f + 0x1p-20f), q);
    uint32_t d0 = codes.x ^ e2m1x8(q), d1 = codes.y ^ e2m1x8(q + 8);
    // Where they differ the border between codes c and c + 1 decides, one element at a time (few
    // lanes have more than one).
    while ((d0 | d1) != 0u) {
        const bool second = d0 == 0u;
        const int shift = (__ffs(static_cast<int>(second ? d1 : d0)) - 1) & ~3;
        const uint32_t c = ((second ? codes.y : codes.x) >> shift) & 7u;
        const float e = fabsf(to_f32<T>(x[(second ? 8 : 0) + shift / 4]));
        const float b = 0.5f * (fp4_code_value(c) + fp4_code_value(c + 1u));
        const float d = fmaf(-b * s, m.t, e);
        const uint32_t up = d > 0.f || (d == 0.f && (c & 1u)) ? 1u << shift : 0u;
        const uint32_t done = ~(15u << shift);
        if (second) {
            codes.y += up;
            d1 &= done;
        } else {
            codes.x += up;
            d0 &= done;
        }
    }
    return codes;
}

// ------------------------------------------------------------------------------------------
// Kernels
// ------------------------------------------------------------------------------------------
template <typename T, int FMT>
__global__ void __launch_bounds__(kQuantThreads)
    fp4_quantize_kernel(const T *__restrict__ x, int64_t rows, int d, int64_t ldx, bool wide,
                        const float *__restrict__ t, uint8_t *__restrict__ codes,
                        uint8_t *__restrict__ scales)
{
    const int padded = static_cast<int>(fp4_padded(d));
    MatrixScale m;
    if (FMT == LNQ_FP4_NV)
        m = matrix_scale(t);
    for (SpanWalk walk(rows, padded); walk.more(); walk.next()) {
        const int i0 = walk.element();
        Elements<T> e;
        e.load(x + walk.row * ldx + i0, d - i0, wide);
        uint32_t amax = e.top(), byte;
        uint2 word = make_uint2(0u, 0u);
        float v[kLane];
#pragma unroll
        for (int k = 0; k < kLane; ++k)
            v[k] = to_f32<T>(e.get(k));
        if (FMT == LNQ_FP4_MX) {
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            byte = 255u;
            if (amax < 0x7F800000u) {
                // exponent field of the scale: that of amax, less 2
                byte = max(static_cast<int>(amax >> 23) - 2, 0);
                float q[kLane];
                scale16(v, __uint_as_float((254u - byte) << 23), q);
                word = make_uint2(e2m1x8(q), e2m1x8(q + 8));
            }
        } else {
            byte = 127u;
            if (amax < 0x7F800000u && m.valid) {
                byte = nv_scale_byte(__uint_as_float(amax), m);
                if (byte != 0u)
                    word = nv_codes<T>(v, x + walk.row * ldx + i0, d - i0,
                                       __uint_as_float(byte << 20) * 0x1p120f, m);
            }
        }
        if (i0 < padded) {
            *reinterpret_cast<uint2 *>(codes + walk.row * (padded / 2) + i0 / 2) = word;
            if (FMT == LNQ_FP4_NV || (threadIdx.x & 1) == 0)
                scales[walk.row * (padded / fp4_block(FMT)) + i0 / fp4_block(FMT)] =
                    static_cast<uint8_t>(i0 < d ? byte : 0u);
        }
    }
}

// A lane writes 16 bytes at a time, its neighbours the next, so that a warp's store is 512 bytes in
// a row (two stores of alternate 16-byte pieces were a quarter slower).
template <typename T, int FMT>
__global__ void __launch_bounds__(kQuantThreads)
    fp4_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                          int64_t rows, int d, const float *__restrict__ t, T *__restrict__ y,
                          int64_t ldy, bool wide)
{
    constexpr int kPiece = 16 / sizeof(T), kPieces = kSpan / 32 / kPiece;
    const int padded = static_cast<int>(fp4_padded(d));
    const int lane = threadIdx.x & 31;
    const float tv = t == nullptr ? 1.f : __ldg(t);
    for (SpanWalk walk(rows, padded); walk.more(); walk.next()) {
        const uint8_t *c = codes + walk.row * (padded / 2), *s = scales + walk.row * (padded / fp4_block(FMT));
        T *out = y + walk.row * ldy;
        const int i0 = walk.span * kSpan + lane * kPiece;
        uint32_t word[kPieces], byte[kPieces];
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const int i = i0 + p * 32 * kPiece;
            word[p] = byte[p] = 0u;
            if (i < d) {
                word[p] = __ldg(reinterpret_cast<const uint32_t *>(c) + i / 8) >> (4 * (i & 4));
                byte[p] = __ldg(s + i / fp4_block(FMT));
            }
        }
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const int i = i0 + p * 32 * kPiece;
            const float scale = fp4_scale_value<FMT>(byte[p]);
            float v[8];
            if constexpr (kPiece == 8) {
                code_values(word[p], v);
            } else {
#pragma unroll
                for (int k = 0; k < kPiece; ++k)
                    v[k] = fp4_code_value((word[p] >> (4 * k)) & 15u);
            }
            alignas(16) T e[kPiece];
#pragma unroll
            for (int k = 0; k < kPiece; ++k)
                e[k] = from_f32<T>(v[k] * scale * tv);
            if (wide && i + kPiece <= d) {
                *reinterpret_cast<uint4 *>(out + i) = *reinterpret_cast<const uint4 *>(e);
            } else {
#pragma unroll
                for (int k = 0; k < kPiece; ++k)
                    if (i + k < d)
                        out[i + k] = e[k];
            }
        }
    }
}

// The largest finite magnitude, as bits, into *top (zero before): an integer maximum, so the
// order of the blocks does not matter.
template <typename T>
__global__ void __launch_bounds__(kQuantThreads)
    fp4_absmax_kernel(const T *__restrict__ x, int64_t rows, int d, int64_t ldx, bool wide,
                      uint32_t *__restrict__ top)
{
    constexpr int kSpansAhead = 2;  // loaded before the first is worked on
    uint32_t amax = 0u;
    SpanWalk walk(rows, d);
    while (walk.more()) {
        Elements<T> e[kSpansAhead];
#pragma unroll
        for (int u = 0; u < kSpansAhead; ++u) {
            const int i0 = walk.element();
            const bool more = walk.more();
            e[u].load(x + (more ? walk.row * ldx + i0 : 0), more ? d - i0 : 0, wide);
            walk.next();
        }
#pragma unroll
        for (int u = 0; u < kSpansAhead; ++u) {
            uint32_t m = e[u].top();
            if (m >= 0x7F800000u) {
                m = 0u;
#pragma unroll
                for (int k = 0; k < kLane; ++k) {
                    const uint32_t b = __float_as_uint(to_f32<T>(e[u].get(k))) & 0x7FFFFFFFu;
                    m = max(m, b < 0x7F800000u ? b : 0u);
                }
            }
            amax = max(amax, m);
        }
    }
    __shared__ uint32_t part[kQuantThreads / 32];
    amax = __reduce_max_sync(0xffffffffu, amax);
    if ((threadIdx.x & 31) == 0)
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
                static_cast<const T *>(x), rows, static_cast<int>(d), ldx, wide_rows(x, ldx, sizeof(T)),
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
            static_cast<const T *>(x), rows, static_cast<int>(d), ldx, wide_rows(x, ldx, sizeof(T)), t,
            codes, scales);
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
            codes, scales, rows, static_cast<int>(d), t, static_cast<T *>(y), ldy,
            wide_rows(y, ldy, sizeof(T)));
        return cudaGetLastError();
    });
}

}  // namespace lnq
