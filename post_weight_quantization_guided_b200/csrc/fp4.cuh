// fp4.cuh -- the microscaled 4-bit formats: layout, decoding, launchers of the operators.
#pragma once

#include "../../include/lnq_fp4.h"
#include "common.cuh"

namespace lnq {

constexpr int kFp4Pad = 128;  // a row's pitch covers d rounded up to a multiple of this

__host__ __device__ constexpr int fp4_block(int fmt) { return fmt == LNQ_FP4_MX ? 32 : 16; }
__host__ __device__ constexpr int64_t fp4_padded(int64_t d)
{
    return (d + kFp4Pad - 1) / kFp4Pad * kFp4Pad;
}
__host__ __device__ constexpr int64_t fp4_code_pitch(int64_t d) { return fp4_padded(d) / 2; }
__host__ __device__ constexpr int64_t fp4_scale_pitch(int64_t d, int fmt)
{
    return fp4_padded(d) / fp4_block(fmt);
}

// The value of a scale byte. MX: 2^(b - 127), subnormal for b = 0. NV: the byte's exponent and
// mantissa fields at the head of a float's, times 2^(127 - 7), which also makes the subnormals.
template <int FMT>
__device__ __forceinline__ float fp4_scale_value(uint32_t b)
{
    if (FMT == LNQ_FP4_MX) {
        const uint32_t bits = b == 0u ? 0x00400000u : (b == 255u ? 0x7FC00000u : b << 23);
        return __uint_as_float(bits);
    }
    b &= 0x7Fu;
    return b == 0x7Fu ? __uint_as_float(0x7FC00000u)
                      : __uint_as_float(b << 20) * __uint_as_float((127u + 120u) << 23);
}

// The value of the code in bits 3..0 of c: its exponent and mantissa bits at a float's, times
// 2^(127 - 1), and the sign.
__device__ __forceinline__ float fp4_code_value(uint32_t c)
{
    const uint32_t bits = ((c & 7u) << 22) | ((c & 8u) << 28);
    return __uint_as_float(bits) * __uint_as_float((127u + 126u) << 23);
}

// One element of a type given at run time or as a template argument.
template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v)
{
    return __bfloat162float(v);
}
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v)
{
    return __float2bfloat16_rn(v);
}
template <> __device__ __forceinline__ __half from_f32<__half>(float v)
{
    return __float2half_rn(v);
}

// offsets[] as the grouped operators read it: each value limited to 0 .. n and to no less than
// the largest before it. Returns group e's first row and the row behind its last. For whole warps.
__device__ __forceinline__ int2 fp4_group_rows(const int32_t *__restrict__ offsets, int e, int n)
{
    int lo = 0;
    for (int i = threadIdx.x & 31; i <= e; i += 32)
        lo = max(lo, min(offsets[i], n));
    lo = __reduce_max_sync(0xffffffffu, lo);
    return make_int2(lo, max(lo, min(offsets[e + 1], n)));
}

// A quantised matrix (or `experts` of them, one after another).
struct Fp4Matrix {
    const uint8_t *codes, *scales;
    const float *t;  // matrix scale(s), or nullptr
    int64_t rows;    // rows of one matrix
};

cudaError_t fp4_tensor_scale_launch(const void *x, int xt, int64_t rows, int64_t d, int64_t ldx,
                                    float *t, int num_sms, cudaStream_t s);
cudaError_t fp4_quantize_launch(const void *x, int xt, int64_t rows, int64_t d, int64_t ldx,
                                int fmt, const float *t, uint8_t *codes, uint8_t *scales,
                                int num_sms, cudaStream_t s);
cudaError_t fp4_dequantize_launch(const uint8_t *codes, const uint8_t *scales, int64_t rows,
                                  int64_t d, int fmt, const float *t, void *y, int yt, int64_t ldy,
                                  int num_sms, cudaStream_t s);
// offsets == nullptr: one group of all n rows and one matrix.
cudaError_t fp4_gemv_launch(const void *x, int xt, int64_t n, int64_t ldx, const int32_t *offsets,
                            int64_t experts, const Fp4Matrix &w, int64_t d_in, int fmt, void *y,
                            int yt, int64_t ldy, int num_sms, cudaStream_t s);
cudaError_t fp4_gemm_launch(const Fp4Matrix &a, const int32_t *offsets, int64_t experts,
                            const Fp4Matrix &w, int64_t d_in, int fmt, void *y, int yt,
                            int64_t ldy, long long wait_limit, int num_sms, cudaStream_t s);
// The products' bounded waits that gave up on a device since the library was loaded (modulo 2^32): of
// products on one stream (and on those that share its slot), of products captured into graphs, of all.
struct Fp4GiveUps {
    uint32_t own, captured, all;
};
constexpr int kFp4ReportSlots = 1024;
// The counts as they are once `s` has been synchronised, on the current device.
cudaError_t fp4_give_ups(Fp4GiveUps *counts, cudaStream_t s);
// fp4_report.cu: the slot of a stream's count; whether the counts hold something this stream has not
// been told of, and that it has been told now (the default stream: of all of the device's).
int fp4_report_slot(cudaStream_t s);
bool fp4_report_news(int device, cudaStream_t s, const Fp4GiveUps &now);

// api.cu
int device_sm_count();
long long wait_limit();

}  // namespace lnq
