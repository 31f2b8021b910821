// fp4_api.cu -- the extern "C" entry points declared in include/lnq_fp4.h: argument checks, then
// the launchers. No device memory is allocated here.
#include "fp4.cuh"

namespace lnq {
namespace {


bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool valid_fmt(int fmt) { return fmt == LNQ_FP4_MX || fmt == LNQ_FP4_NV; }
bool valid_type(int t) { return t == LNQ_F32 || t == LNQ_BF16 || t == LNQ_F16; }
bool valid_d(int64_t d) { return d >= 1 && d <= LNQ_FP4_MAX_D; }
bool valid_rows(int64_t n) { return n >= 0 && n <= LNQ_FP4_MAX_ROWS; }

// An unquantised matrix of n rows and d columns.
bool valid_dense(const void *p, int type, int64_t n, int64_t d, int64_t ld)
{
    return valid_type(type) && ld >= d && ld <= (int64_t(1) << 40) &&
           (n == 0 || (p != nullptr && aligned(p, type == LNQ_F32 ? 4 : 2)));
}

// A quantised matrix of n rows.
bool valid_codes(const uint8_t *codes, const uint8_t *scales, const float *t, int64_t n, int fmt)
{
    if (fmt == LNQ_FP4_MX && t != nullptr)
        return false;
    if (n == 0)
        return true;
    return codes != nullptr && scales != nullptr && aligned(codes, 16) &&
           aligned(scales, fmt == LNQ_FP4_MX ? 4 : 8) && aligned(t, 4);
}

lnq_status status_of(cudaError_t e)
{
    return e == cudaSuccess ? LNQ_OK
                            : (e == cudaErrorNotSupported ? LNQ_ERR_UNSUPPORTED : LNQ_ERR_CUDA);
}

// Both forms of both products: the sizes they share.
bool valid_product(int64_t n, int64_t d_out, int64_t d_in, int64_t experts, int fmt)
{
    return valid_rows(n) && valid_d(d_in) && valid_fmt(fmt) && d_out >= 1 && experts >= 1 &&
           experts <= LNQ_FP4_MAX_EXPERTS && d_out <= LNQ_FP4_MAX_ROWS && d_out * experts <= LNQ_FP4_MAX_ROWS;
}

lnq_status gemv(const void *x, int xt, int64_t n, int64_t ldx, const int32_t *offsets,
                int64_t experts, const uint8_t *codes, const uint8_t *scales, const float *t,
                int64_t d_out, int64_t d_in, int fmt, void *y, int yt, int64_t ldy,
                lnq_stream_t stream)
{
    if (!valid_product(n, d_out, d_in, experts, fmt) || !valid_dense(x, xt, n, d_in, ldx) ||
        !valid_dense(y, yt, n, d_out, ldy) || !valid_codes(codes, scales, t, n, fmt))
        return LNQ_ERR_INVALID_ARG;
    if (n == 0)
        return LNQ_OK;
    return status_of(fp4_gemv_launch(x, xt, n, ldx, offsets, experts,
                                     Fp4Matrix{codes, scales, t, d_out}, d_in, fmt, y, yt, ldy,
                                     device_sm_count(), reinterpret_cast<cudaStream_t>(stream)));
}

lnq_status gemm(const uint8_t *a_codes, const uint8_t *a_scales, const float *ta, int64_t n,
                const int32_t *offsets, int64_t experts, const uint8_t *w_codes,
                const uint8_t *w_scales, const float *tw, int64_t d_out, int64_t d_in, int fmt,
                void *y, int yt, int64_t ldy, lnq_stream_t stream)
{
    if (!valid_product(n, d_out, d_in, experts, fmt) ||
        !valid_codes(a_codes, a_scales, ta, n, fmt) || !valid_codes(w_codes, w_scales, tw, n, fmt) ||
        !valid_dense(y, yt, n, d_out, ldy))
        return LNQ_ERR_INVALID_ARG;
    if (n == 0)
        return LNQ_OK;
    return status_of(fp4_gemm_launch(Fp4Matrix{a_codes, a_scales, ta, n}, offsets, experts,
                                     Fp4Matrix{w_codes, w_scales, tw, d_out}, d_in, fmt, y, yt,
                                     ldy, wait_limit(), device_sm_count(),
                                     reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace
}  // namespace lnq

using namespace lnq;

extern "C" {

int64_t lnq_fp4_code_bytes(int64_t d) { return valid_d(d) ? fp4_code_pitch(d) : 0; }

int64_t lnq_fp4_scale_bytes(int64_t d, lnq_fp4_format fmt)
{
    return valid_d(d) && valid_fmt(fmt) ? fp4_scale_pitch(d, fmt) : 0;
}

lnq_status lnq_fp4_tensor_scale(const void *x, lnq_dtype xt, int64_t rows, int64_t d, int64_t ldx,
                                float *t, lnq_stream_t stream)
{
    if (!valid_rows(rows) || !valid_d(d) || !valid_dense(x, xt, rows, d, ldx) || t == nullptr ||
        !aligned(t, 4))
        return LNQ_ERR_INVALID_ARG;
    return status_of(fp4_tensor_scale_launch(x, xt, rows, d, ldx, t, device_sm_count(),
                                             reinterpret_cast<cudaStream_t>(stream)));
}

lnq_status lnq_fp4_quantize(const void *x, lnq_dtype xt, int64_t rows, int64_t d, int64_t ldx,
                            lnq_fp4_format fmt, const float *t, uint8_t *codes, uint8_t *scales,
                            lnq_stream_t stream)
{
    if (!valid_rows(rows) || !valid_d(d) || !valid_fmt(fmt) || !valid_dense(x, xt, rows, d, ldx) ||
        !valid_codes(codes, scales, t, rows, fmt))
        return LNQ_ERR_INVALID_ARG;
    if (rows == 0)
        return LNQ_OK;
    return status_of(fp4_quantize_launch(x, xt, rows, d, ldx, fmt, t, codes, scales,
                                         device_sm_count(),
                                         reinterpret_cast<cudaStream_t>(stream)));
}

lnq_status lnq_fp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t d,
                              lnq_fp4_format fmt, const float *t, void *y, lnq_dtype yt,
                              int64_t ldy, lnq_stream_t stream)
{
    if (!valid_rows(rows) || !valid_d(d) || !valid_fmt(fmt) || !valid_dense(y, yt, rows, d, ldy) ||
        !valid_codes(codes, scales, t, rows, fmt))
        return LNQ_ERR_INVALID_ARG;
    if (rows == 0)
        return LNQ_OK;
    return status_of(fp4_dequantize_launch(codes, scales, rows, d, fmt, t, y, yt, ldy,
                                           device_sm_count(),
                                           reinterpret_cast<cudaStream_t>(stream)));
}

lnq_status lnq_fp4_gemv(const void *x, lnq_dtype xt, int64_t nb, int64_t ldx, const uint8_t *codes,
                        const uint8_t *scales, const float *t, int64_t d_out, int64_t d_in,
                        lnq_fp4_format fmt, void *y, lnq_dtype yt, int64_t ldy,
                        lnq_stream_t stream)
{
    return gemv(x, xt, nb, ldx, nullptr, 1, codes, scales, t, d_out, d_in, fmt, y, yt, ldy, stream);
}

lnq_status lnq_fp4_grouped_gemv(const void *x, lnq_dtype xt, int64_t n, int64_t ldx,
                                const int32_t *offsets, int64_t experts, const uint8_t *codes,
                                const uint8_t *scales, const float *t, int64_t d_out,
                                int64_t d_in, lnq_fp4_format fmt, void *y, lnq_dtype yt,
                                int64_t ldy, lnq_stream_t stream)
{
    if (offsets == nullptr || !aligned(offsets, 4))
        return LNQ_ERR_INVALID_ARG;
    return gemv(x, xt, n, ldx, offsets, experts, codes, scales, t, d_out, d_in, fmt, y, yt, ldy,
                stream);
}

lnq_status lnq_fp4_gemm(const uint8_t *a_codes, const uint8_t *a_scales, const float *ta,
                        int64_t n, const uint8_t *w_codes, const uint8_t *w_scales,
                        const float *tw, int64_t d_out, int64_t d_in, lnq_fp4_format fmt, void *y,
                        lnq_dtype yt, int64_t ldy, lnq_stream_t stream)
{
    return gemm(a_codes, a_scales, ta, n, nullptr, 1, w_codes, w_scales, tw, d_out, d_in, fmt, y,
                yt, ldy, stream);
}

lnq_status lnq_fp4_grouped_gemm(const uint8_t *a_codes, const uint8_t *a_scales, const float *ta,
                                int64_t n, const int32_t *offsets, int64_t experts,
                                const uint8_t *w_codes, const uint8_t *w_scales, const float *tw,
                                int64_t d_out, int64_t d_in, lnq_fp4_format fmt, void *y,
                                lnq_dtype yt, int64_t ldy, lnq_stream_t stream)
{
    if (offsets == nullptr || !aligned(offsets, 4))
        return LNQ_ERR_INVALID_ARG;
    return gemm(a_codes, a_scales, ta, n, offsets, experts, w_codes, w_scales, tw, d_out, d_in, fmt,
                y, yt, ldy, stream);
}

lnq_status lnq_fp4_check(lnq_stream_t stream)
{
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    Fp4GiveUps counts = {0u, 0u, 0u};
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess || fp4_give_ups(&counts, s) != cudaSuccess)
        return LNQ_ERR_CUDA;
    return fp4_report_news(device, s, counts) ? LNQ_ERR_TIMEOUT : LNQ_OK;
}

}  // extern "C"
