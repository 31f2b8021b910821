// fp4_gemm.cu -- the product of two quantised matrices, and the same with the rows grouped by
// expert.
//
//   y[b][j] = ta tw sum_i (code sa)[b][i] (code sw)[j][i]
//
// A CTA computes a 64 x 64 tile: it decodes 32 columns of both operands into shared memory at a
// time, and each thread accumulates a 4 x 4 piece.
#include "fp4.cuh"
#include "profile.cuh"

namespace lnq {

__device__ uint32_t g_fp4_error[2];

constexpr int kTile = 64, kDepth = 32;

template <int FMT>
__device__ __forceinline__ void decode_tile(float (&out)[kDepth][kTile + 1], const Fp4Matrix &m,
                                            int64_t first, int64_t behind, int64_t i0, int64_t d)
{
    const int64_t padded = fp4_padded(d);
    const int r = threadIdx.x >> 2, c = (threadIdx.x & 3) * 8;  // 256 threads: 64 rows x 4 words
    const int64_t row = first + r;
    uint32_t word = 0u;
    float s = 0.f;
    if (row < behind && i0 + c < d) {
        word = reinterpret_cast<const uint32_t *>(m.codes + row * (padded / 2))[(i0 + c) / 8];
        s = fp4_scale_value<FMT>(
            m.scales[row * (padded / fp4_block(FMT)) + (i0 + c) / fp4_block(FMT)]);
    }
    for (int k = 0; k < 8; ++k)
        out[c + k][r] = i0 + c + k < d ? fp4_code_value((word >> (4 * k)) & 15u) * s : 0.f;
}

template <typename TY, int FMT>
__global__ void __launch_bounds__(256)
    fp4_gemm_kernel(Fp4Matrix a, const int32_t *__restrict__ offsets, Fp4Matrix w, int64_t d_in,
                    TY *__restrict__ y, int64_t ldy)
{
    __shared__ float as[kDepth][kTile + 1], bs[kDepth][kTile + 1];
    const int e = blockIdx.z;
    const int n = static_cast<int>(a.rows);
    const int2 rows = offsets == nullptr ? make_int2(0, n) : fp4_group_rows(offsets, e, n);
    const int64_t j0 = static_cast<int64_t>(blockIdx.x) * kTile;
    const float ta = a.t == nullptr ? 1.f : *a.t, tw = w.t == nullptr ? 1.f : w.t[e];
    const int tr = (threadIdx.x >> 4) * 4, tc = (threadIdx.x & 15) * 4;
    for (int64_t b0 = rows.x + static_cast<int64_t>(blockIdx.y) * kTile; b0 < rows.y;
         b0 += static_cast<int64_t>(gridDim.y) * kTile) {
        float acc[4][4] = {};
        for (int64_t i0 = 0; i0 < d_in; i0 += kDepth) {
            __syncthreads();
            decode_tile<FMT>(as, a, b0, rows.y, i0, d_in);
            decode_tile<FMT>(bs, w, e * w.rows + j0, (e + 1) * w.rows, i0, d_in);
            __syncthreads();
            for (int k = 0; k < kDepth; ++k)
                for (int p = 0; p < 4; ++p)
                    for (int q = 0; q < 4; ++q)
                        acc[p][q] = fmaf(as[k][tr + p], bs[k][tc + q], acc[p][q]);
        }
        for (int p = 0; p < 4; ++p)
            for (int q = 0; q < 4; ++q)
                if (b0 + tr + p < rows.y && j0 + tc + q < w.rows)
                    y[(b0 + tr + p) * ldy + j0 + tc + q] = from_f32<TY>(acc[p][q] * ta * tw);
    }
}

cudaError_t fp4_gemm_launch(const Fp4Matrix &a, const int32_t *offsets, int64_t experts,
                            const Fp4Matrix &w, int64_t d_in, int fmt, void *y, int yt,
                            int64_t ldy, long long wait_limit, int num_sms, cudaStream_t s)
{
    (void)wait_limit, (void)num_sms;
    const dim3 grid(static_cast<unsigned>((w.rows + kTile - 1) / kTile),
                    static_cast<unsigned>(min((a.rows + kTile - 1) / kTile, int64_t(64))),
                    static_cast<unsigned>(experts));
    KernelTimer timer("lnq_fp4_gemm", s);
    const bool mx = fmt == LNQ_FP4_MX;
    switch (yt) {
    case LNQ_F32:
        (mx ? fp4_gemm_kernel<float, LNQ_FP4_MX> : fp4_gemm_kernel<float, LNQ_FP4_NV>)
            <<<grid, 256, 0, s>>>(a, offsets, w, d_in, static_cast<float *>(y), ldy);
        break;
    case LNQ_BF16:
        (mx ? fp4_gemm_kernel<__nv_bfloat16, LNQ_FP4_MX> : fp4_gemm_kernel<__nv_bfloat16, LNQ_FP4_NV>)
            <<<grid, 256, 0, s>>>(a, offsets, w, d_in, static_cast<__nv_bfloat16 *>(y), ldy);
        break;
    case LNQ_F16:
        (mx ? fp4_gemm_kernel<__half, LNQ_FP4_MX> : fp4_gemm_kernel<__half, LNQ_FP4_NV>)
            <<<grid, 256, 0, s>>>(a, offsets, w, d_in, static_cast<__half *>(y), ldy);
        break;
    default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

cudaError_t fp4_take_error_flags(uint32_t *flags, cudaStream_t s)
{
    const uint32_t zero[2] = {0u, 0u};
    cudaError_t e = cudaMemcpyFromSymbolAsync(flags, g_fp4_error, sizeof(uint32_t), 0,
                                              cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && flags[0] != 0u) {
        e = cudaMemcpyToSymbolAsync(g_fp4_error, zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess)
            e = cudaStreamSynchronize(s);
    }
    return e;
}

}  // namespace lnq
