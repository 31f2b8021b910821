// fp4_gemv.cu -- unquantised activations times a quantised matrix, for few rows, and the same
// with the rows grouped by expert.
//
//   y[b][j] = t sum_k s[j][k] sum_{i in block k} x[b][i] code[j][i]
//
// One warp per output j; the lanes take 8 consecutive elements of the row in turn, eight rows of
// x at a time, and add their sums by a fixed shuffle butterfly.
#include "fp4.cuh"
#include "profile.cuh"

namespace lnq {

constexpr int kGemvWarps = 8;
constexpr int kGemvRows = 8;  // rows of x per pass over the weights

template <typename TX, typename TY, int FMT>
__global__ void __launch_bounds__(kGemvWarps * 32)
    fp4_gemv_kernel(const TX *__restrict__ x, int n, int64_t ldx,
                    const int32_t *__restrict__ offsets, Fp4Matrix w, int64_t d_in,
                    TY *__restrict__ y, int64_t ldy)
{
    const int e = blockIdx.y, lane = threadIdx.x & 31;
    const int2 rows = offsets == nullptr ? make_int2(0, n) : fp4_group_rows(offsets, e, n);
    if (rows.x >= rows.y)
        return;
    const int64_t j = static_cast<int64_t>(blockIdx.x) * kGemvWarps + (threadIdx.x >> 5);
    if (j >= w.rows)
        return;
    const int64_t padded = fp4_padded(d_in);
    const int64_t row = e * w.rows + j;
    const uint32_t *codes = reinterpret_cast<const uint32_t *>(w.codes + row * (padded / 2));
    const uint8_t *scales = w.scales + row * (padded / fp4_block(FMT));
    const float t = w.t == nullptr ? 1.f : w.t[e];
    for (int b0 = rows.x; b0 < rows.y; b0 += kGemvRows) {
        float acc[kGemvRows];
        for (int b = 0; b < kGemvRows; ++b)
            acc[b] = 0.f;
        for (int64_t i0 = lane * 8; i0 < d_in; i0 += 256) {
            const uint32_t word = codes[i0 / 8];
            const float s = fp4_scale_value<FMT>(scales[i0 / fp4_block(FMT)]);
            for (int k = 0; k < 8; ++k) {
                if (i0 + k >= d_in)
                    break;
                const float v = fp4_code_value((word >> (4 * k)) & 15u) * s;
#pragma unroll
                for (int b = 0; b < kGemvRows; ++b)
                    if (b0 + b < rows.y)
                        acc[b] = fmaf(v, to_f32<TX>(x[(b0 + b) * ldx + i0 + k]), acc[b]);
            }
        }
#pragma unroll
        for (int b = 0; b < kGemvRows; ++b) {
            for (int o = 16; o >= 1; o >>= 1)
                acc[b] += __shfl_xor_sync(0xffffffffu, acc[b], o);
            if (lane == 0 && b0 + b < rows.y)
                y[(b0 + b) * ldy + j] = from_f32<TY>(acc[b] * t);
        }
    }
}

template <typename TX, typename TY>
static cudaError_t gemv_types(const void *x, int n, int64_t ldx, const int32_t *offsets,
                              int64_t experts, const Fp4Matrix &w, int64_t d_in, int fmt, void *y,
                              int64_t ldy, cudaStream_t s)
{
    const dim3 grid(static_cast<unsigned>((w.rows + kGemvWarps - 1) / kGemvWarps),
                    static_cast<unsigned>(experts));
    KernelTimer timer("lnq_fp4_gemv", s);
    auto *kernel = fmt == LNQ_FP4_MX ? fp4_gemv_kernel<TX, TY, LNQ_FP4_MX>
                                     : fp4_gemv_kernel<TX, TY, LNQ_FP4_NV>;
    kernel<<<grid, kGemvWarps * 32, 0, s>>>(static_cast<const TX *>(x), n, ldx, offsets, w, d_in,
                                           static_cast<TY *>(y), ldy);
    return cudaGetLastError();
}

template <typename TX>
static cudaError_t gemv_out(const void *x, int n, int64_t ldx, const int32_t *offsets,
                            int64_t experts, const Fp4Matrix &w, int64_t d_in, int fmt, void *y,
                            int yt, int64_t ldy, cudaStream_t s)
{
    switch (yt) {
    case LNQ_F32: return gemv_types<TX, float>(x, n, ldx, offsets, experts, w, d_in, fmt, y, ldy, s);
    case LNQ_BF16:
        return gemv_types<TX, __nv_bfloat16>(x, n, ldx, offsets, experts, w, d_in, fmt, y, ldy, s);
    case LNQ_F16: return gemv_types<TX, __half>(x, n, ldx, offsets, experts, w, d_in, fmt, y, ldy, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t fp4_gemv_launch(const void *x, int xt, int64_t n, int64_t ldx, const int32_t *offsets,
                            int64_t experts, const Fp4Matrix &w, int64_t d_in, int fmt, void *y,
                            int yt, int64_t ldy, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    const int rows = static_cast<int>(n);
    switch (xt) {
    case LNQ_F32: return gemv_out<float>(x, rows, ldx, offsets, experts, w, d_in, fmt, y, yt, ldy, s);
    case LNQ_BF16:
        return gemv_out<__nv_bfloat16>(x, rows, ldx, offsets, experts, w, d_in, fmt, y, yt, ldy, s);
    case LNQ_F16: return gemv_out<__half>(x, rows, ldx, offsets, experts, w, d_in, fmt, y, yt, ldy, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace lnq
