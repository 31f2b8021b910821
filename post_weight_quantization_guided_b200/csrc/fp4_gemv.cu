// fp4_gemv.cu -- unquantised activations times a quantised matrix, for few rows, and the same
// with the rows grouped by expert.
//
//   y[b][j] = t sum_k s[j][k] sum_{i in block k} x[b][i] code[j][i]
//
// Bound: HBM, the codes and scales read once (half a byte and 1/16 (NV) or 1/32 (MX) of a byte an
// element); in practice also the decoding, which every element passes once.
//
// The products run on mma.sync m16n8k16 in bf16 with 32-bit sums: with at most a few rows the
// work is decoding weights, and the instruction takes them straight from registers, where
// tcgen05.mma would want them written to shared memory first. Nothing is rounded: code * scale
// has at most 6 bits, and x enters as one bf16 number (bf16), the sum of two (f16) or of three (f32),
// each piece a column of its own, so 8, 4 or 2 rows of x fill the 8 columns.
//
// A CTA computes 16 outputs; its 8 warps take chunks of 128 elements in turn. Lane 4 g + t holds 32
// consecutive elements of outputs g and g + 8 (one 16-byte load each): one MX block, two NV
// blocks. A word's elements i and i + 4 become one register of two bf16 numbers by two shifts and
// two masks: sign to bit 15, the other three bits to exponent and mantissa, which reads as
// code * 2^-126; the multiplication by s 2^119 that follows leaves code * s * 2^-7 (a factor taken
// out of the finished sum). The order of elements within the instruction's K is free, and x is
// paired alike. Last, the warps' sums are added in order.
#include "fp4.cuh"
#include "profile.cuh"

namespace lnq {

namespace gv {
constexpr int kWarps = 8;
constexpr int kRows = 16;   // outputs of a CTA
constexpr int kChunk = 128; // elements of K a warp takes at a time
constexpr int kBatch = 4;   // chunks whose codes a warp has in flight

template <typename T> struct Pieces;
template <> struct Pieces<__nv_bfloat16> { static constexpr int n = 1; };
template <> struct Pieces<__half> { static constexpr int n = 2; };
template <> struct Pieces<float> { static constexpr int n = 3; };
}  // namespace gv

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                 "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Elements i and i + 4 of a word of codes, as two bf16 numbers times 2^-126.
template <int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t w)
{
    const uint32_t sign = w << (12 - 4 * I);
    const uint32_t rest = I < 2 ? w << (6 - 4 * I) : w >> (4 * I - 6);
    return (sign & 0x80008000u) | (rest & 0x01C001C0u);
}

// Both halves: a power of two or a short number as bf16.
__device__ __forceinline__ uint32_t twice_bf16(float v)
{
    const uint32_t h = __float_as_uint(v) >> 16;
    return h | (h << 16);
}

// Piece p of v (p < pieces): the leading 8 bits, the next 8, the last 8. An infinity is all in
// piece 0; a NaN is in the last.
__device__ __forceinline__ uint32_t piece_bits(float v, int p)
{
    const float a = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
    if (p == 0)
        return __float_as_uint(a) >> 16;
    const float r = fabsf(v) == __uint_as_float(0x7F800000u) ? 0.f : v - a;
    const float b = __uint_as_float(__float_as_uint(r) & 0xFFFF0000u);
    return __float_as_uint(p == 1 ? (isnan(r) ? r : b) : r - b) >> 16;
}

// x[0..7] (zeros from element `left` on) as one word's part of the instruction's column: register i
// holds elements i and i + 4, of piece p.
template <typename TX>
__device__ __forceinline__ void load_column(const TX *__restrict__ x, int left, bool wide, int p,
                                            uint32_t (&b)[4])
{
    alignas(16) TX e[8];
    if (wide && left >= 8) {
#pragma unroll
        for (int k = 0; k < static_cast<int>(sizeof(TX)) / 2; ++k)
            reinterpret_cast<uint4 *>(e)[k] = __ldg(reinterpret_cast<const uint4 *>(x) + k);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            e[k] = k < left ? x[k] : from_f32<TX>(0.f);
    }
    if constexpr (gv::Pieces<TX>::n == 1) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(e);
        b[0] = __byte_perm(w[0], w[2], 0x5410);
        b[1] = __byte_perm(w[0], w[2], 0x7632);
        b[2] = __byte_perm(w[1], w[3], 0x5410);
        b[3] = __byte_perm(w[1], w[3], 0x7632);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            b[i] = piece_bits(to_f32<TX>(e[i]), p) | (piece_bits(to_f32<TX>(e[i + 4]), p) << 16);
    }
}

// One word of codes of two outputs, scaled: the instruction's A registers of its eight elements.
__device__ __forceinline__ void decode_word(uint32_t w0, uint32_t w1, uint32_t m0, uint32_t m1,
                                            uint32_t (&lo)[4], uint32_t (&hi)[4])
{
    lo[0] = mul_bf16x2(code_pair<0>(w0), m0);
    lo[1] = mul_bf16x2(code_pair<0>(w1), m1);
    lo[2] = mul_bf16x2(code_pair<1>(w0), m0);
    lo[3] = mul_bf16x2(code_pair<1>(w1), m1);
    hi[0] = mul_bf16x2(code_pair<2>(w0), m0);
    hi[1] = mul_bf16x2(code_pair<2>(w1), m1);
    hi[2] = mul_bf16x2(code_pair<3>(w0), m0);
    hi[3] = mul_bf16x2(code_pair<3>(w1), m1);
}

// NT column tiles (of 8 / pieces rows of x) per pass over the weights.
template <typename TX, int FMT, int NT>
__global__ void __launch_bounds__(gv::kWarps * 32, 2)
    fp4_gemv_kernel(const TX *__restrict__ x, int n, int64_t ldx, bool wide,
                    const int32_t *__restrict__ offsets, Fp4Matrix w, int d_in, void *__restrict__ y,
                    int yt, int64_t ldy)
{
    using namespace gv;
    constexpr int P = Pieces<TX>::n, kTok = 8 / P;   // rows of x per column tile
    constexpr int kPass = NT * kTok;                 // and per pass
    constexpr int kBlocks = 32 / fp4_block(FMT);     // blocks of a lane's 32 elements
    __shared__ float sums[kWarps][NT][kRows][8];
    const int e = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int2 rows = offsets == nullptr ? make_int2(0, n) : fp4_group_rows(offsets, e, n);
    if (rows.x >= rows.y)
        return;
    const int j0 = blockIdx.x * kRows;
    const int d_out = static_cast<int>(w.rows);
    const int64_t code_pitch = fp4_code_pitch(d_in), scale_pitch = fp4_scale_pitch(d_in, FMT);
    const int chunks = (d_in + kChunk - 1) / kChunk;
    const int blocks = (d_in + fp4_block(FMT) - 1) / fp4_block(FMT);
    // outputs behind the last (nobody writes their sums) repeat it
    const int64_t first = static_cast<int64_t>(e) * d_out;
    const int64_t r0 = first + min(j0 + g, d_out - 1), r1 = first + min(j0 + g + 8, d_out - 1);
    const uint8_t *codes0 = w.codes + r0 * code_pitch + t * 16;
    const uint8_t *codes1 = w.codes + r1 * code_pitch + t * 16;
    const uint8_t *scales0 = w.scales + r0 * scale_pitch + t * kBlocks;
    const uint8_t *scales1 = w.scales + r1 * scale_pitch + t * kBlocks;
    const float scale = (w.t == nullptr ? 1.f : __ldg(w.t + e)) * 128.f;
    const int token = g / P, piece = g - token * P;  // of this lane's column
    for (int b0 = rows.x; b0 < rows.y; b0 += kPass) {
        float acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                acc[nt][k] = 0.f;
        for (int c0 = warp; c0 < chunks; c0 += kWarps * kBatch) {
            uint4 q0[kBatch], q1[kBatch];
            uint32_t s0[kBatch], s1[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int c = c0 + u * kWarps;
                q0[u] = q1[u] = make_uint4(0u, 0u, 0u, 0u);
                s0[u] = s1[u] = 0u;
                if (c < chunks) {
                    q0[u] = __ldg(reinterpret_cast<const uint4 *>(codes0 + static_cast<int64_t>(c) * 64));
                    q1[u] = __ldg(reinterpret_cast<const uint4 *>(codes1 + static_cast<int64_t>(c) * 64));
                    if (kBlocks == 2) {
                        s0[u] = __ldg(reinterpret_cast<const uint16_t *>(scales0 + c * 8));
                        s1[u] = __ldg(reinterpret_cast<const uint16_t *>(scales1 + c * 8));
                    } else {
                        s0[u] = __ldg(scales0 + c * 4);
                        s1[u] = __ldg(scales1 + c * 4);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int c = c0 + u * kWarps;
                if (c >= chunks)
                    break;
                const int i0 = c * kChunk + t * 32, block0 = c * (kChunk / fp4_block(FMT)) + t * kBlocks;
                // s 2^119 of each block, as bf16 twice; 0 behind the row's last block
                uint32_t m0[kBlocks], m1[kBlocks];
                bool usual = true;
#pragma unroll
                for (int k = 0; k < kBlocks; ++k) {
                    uint32_t v0 = (s0[u] >> (8 * k)) & 255u, v1 = (s1[u] >> (8 * k)) & 255u;
                    const bool in = block0 + k < blocks;
                    if (FMT == LNQ_FP4_MX) {
                        // 2^(v - 8), a normal number that keeps code * s * 2^-7 one for 9 <= v <= 135
                        usual = !in || ((v0 - 9u <= 126u || v0 == 255u) && (v1 - 9u <= 126u || v1 == 255u));
                        m0[k] = v0 == 255u ? 0x7FC07FC0u : (v0 + 119u) * 0x00800080u;
                        m1[k] = v1 == 255u ? 0x7FC07FC0u : (v1 + 119u) * 0x00800080u;
                    } else {
                        m0[k] = twice_bf16(fp4_scale_value<FMT>(v0) * 0x1p119f);
                        m1[k] = twice_bf16(fp4_scale_value<FMT>(v1) * 0x1p119f);
                    }
                    if (!in)
                        m0[k] = m1[k] = 0u;
                }
                const uint32_t w0[4] = {q0[u].x, q0[u].y, q0[u].z, q0[u].w};
                const uint32_t w1[4] = {q1[u].x, q1[u].y, q1[u].z, q1[u].w};
                if (FMT == LNQ_FP4_NV || __all_sync(0xffffffffu, usual)) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t lo[4], hi[4];
                        decode_word(w0[j], w1[j], m0[j * kBlocks / 4], m1[j * kBlocks / 4], lo, hi);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const int b = b0 + nt * kTok + token;
                            const int left = b < rows.y && g < kTok * P ? d_in - i0 - 8 * j : 0;
                            uint32_t v[4];
                            load_column<TX>(x + (left > 0 ? b * ldx + i0 + 8 * j : 0), left, wide, piece, v);
                            mma_bf16(acc[nt], lo, v[0], v[1]);
                            mma_bf16(acc[nt], hi, v[2], v[3]);
                        }
                    }
                } else {
                    // An MX scale outside that range: codes alone (times 2^126, exact), the four
                    // lanes' blocks one after another, each sum scaled in 32 bits. (The other
                    // lanes' x is left out too: an infinity of another block stays there.)
                    const uint32_t one = twice_bf16(0x1p126f);
                    const bool in = block0 < blocks;
                    const float f0 = in ? fp4_scale_value<FMT>(s0[u] & 255u) * 0x1p-7f : 0.f;
                    const float f1 = in ? fp4_scale_value<FMT>(s1[u] & 255u) * 0x1p-7f : 0.f;
#pragma unroll 1
                    for (int i = 0; i < 4 * NT; ++i) {
                        const int tt = i & 3, nt = i >> 2;
                        const bool on = t == tt && in;
                        const int b = b0 + nt * kTok + token;
                        const int left = b < rows.y && g < kTok * P && on ? d_in - i0 : 0;
                        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                        for (int j = 0; j < 4; ++j) {
                            uint32_t lo[4], hi[4], v[4];
                            const uint32_t c0w = j == 0 ? w0[0] : (j == 1 ? w0[1] : (j == 2 ? w0[2] : w0[3]));
                            const uint32_t c1w = j == 0 ? w1[0] : (j == 1 ? w1[1] : (j == 2 ? w1[2] : w1[3]));
                            decode_word(c0w, c1w, on ? one : 0u, on ? one : 0u, lo, hi);
                            load_column<TX>(x + (left > 8 * j ? b * ldx + i0 + 8 * j : 0), left - 8 * j,
                                            wide, piece, v);
                            mma_bf16(part, lo, v[0], v[1]);
                            mma_bf16(part, hi, v[2], v[3]);
                        }
                        const float h0 = __shfl_sync(0xffffffffu, f0, (lane & ~3) + tt);
                        const float h1 = __shfl_sync(0xffffffffu, f1, (lane & ~3) + tt);
#pragma unroll
                        for (int k = 0; k < NT; ++k)
                            if (k == nt) {
                                acc[k][0] = fmaf(part[0], h0, acc[k][0]);
                                acc[k][1] = fmaf(part[1], h0, acc[k][1]);
                                acc[k][2] = fmaf(part[2], h1, acc[k][2]);
                                acc[k][3] = fmaf(part[3], h1, acc[k][3]);
                            }
                    }
                }
            }
        }
        __syncthreads();  // the last pass's sums are read
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            *reinterpret_cast<float2 *>(&sums[warp][nt][g][2 * t]) = make_float2(acc[nt][0], acc[nt][1]);
            *reinterpret_cast<float2 *>(&sums[warp][nt][g + 8][2 * t]) = make_float2(acc[nt][2], acc[nt][3]);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kPass * kRows; i += kWarps * 32) {
            const int j = i % kRows, b = i / kRows, nt = b / kTok, col = (b % kTok) * P;
            if (b0 + b < rows.y && j0 + j < d_out) {
                float sum = 0.f;
#pragma unroll
                for (int p = P - 1; p >= 0; --p)  // the small pieces first
#pragma unroll
                    for (int k = 0; k < kWarps; ++k)
                        sum += sums[k][nt][j][col + p];
                sum *= scale;
                const int64_t o = static_cast<int64_t>(b0 + b) * ldy + j0 + j;
                if (yt == LNQ_BF16)
                    static_cast<__nv_bfloat16 *>(y)[o] = from_f32<__nv_bfloat16>(sum);
                else if (yt == LNQ_F16)
                    static_cast<__half *>(y)[o] = from_f32<__half>(sum);
                else
                    static_cast<float *>(y)[o] = sum;
            }
        }
    }
}

template <typename TX, int FMT>
static cudaError_t gemv_fmt(const void *x, int n, int64_t ldx, const int32_t *offsets,
                            int64_t experts, const Fp4Matrix &w, int64_t d_in, void *y, int yt,
                            int64_t ldy, cudaStream_t s)
{
    const dim3 grid(static_cast<unsigned>((w.rows + gv::kRows - 1) / gv::kRows),
                    static_cast<unsigned>(experts));
    const bool wide = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && ldx * sizeof(TX) % 16 == 0;
    // column tiles of a pass: enough for a group of average size, at most 4
    const int64_t mean = (n + experts - 1) / experts, tiles = (mean * gv::Pieces<TX>::n + 7) / 8;
    auto *kernel = tiles <= 1 ? fp4_gemv_kernel<TX, FMT, 1>
                              : (tiles <= 2 ? fp4_gemv_kernel<TX, FMT, 2> : fp4_gemv_kernel<TX, FMT, 4>);
    KernelTimer timer("lnq_fp4_gemv", s);
    kernel<<<grid, gv::kWarps * 32, 0, s>>>(static_cast<const TX *>(x), n, ldx, wide, offsets, w,
                                           static_cast<int>(d_in), y, yt, ldy);
    return cudaGetLastError();
}

template <typename TX>
static cudaError_t gemv_in(const void *x, int n, int64_t ldx, const int32_t *offsets,
                           int64_t experts, const Fp4Matrix &w, int64_t d_in, int fmt, void *y,
                           int yt, int64_t ldy, cudaStream_t s)
{
    return fmt == LNQ_FP4_MX
               ? gemv_fmt<TX, LNQ_FP4_MX>(x, n, ldx, offsets, experts, w, d_in, y, yt, ldy, s)
               : gemv_fmt<TX, LNQ_FP4_NV>(x, n, ldx, offsets, experts, w, d_in, y, yt, ldy, s);
}

cudaError_t fp4_gemv_launch(const void *x, int xt, int64_t n, int64_t ldx, const int32_t *offsets,
                            int64_t experts, const Fp4Matrix &w, int64_t d_in, int fmt, void *y,
                            int yt, int64_t ldy, cudaStream_t s)
{
    const int rows = static_cast<int>(n);
    switch (xt) {
    case LNQ_F32: return gemv_in<float>(x, rows, ldx, offsets, experts, w, d_in, fmt, y, yt, ldy, s);
    case LNQ_BF16:
        return gemv_in<__nv_bfloat16>(x, rows, ldx, offsets, experts, w, d_in, fmt, y, yt, ldy, s);
    case LNQ_F16: return gemv_in<__half>(x, rows, ldx, offsets, experts, w, d_in, fmt, y, yt, ldy, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace lnq
