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
// A CTA first writes its rows of x to shared memory as the instruction's B registers, pieces and
// all. Its 8 warps then stream tiles of 16 outputs, a register ring of chunks of 128 elements ahead:
// lane 4 g + t holds 32 consecutive elements of outputs g and g + 8 (one 16-byte load each): one MX
// block, two NV blocks. A word's elements i and i + 4 become one register of two bf16 numbers: a
// mask, one multiplication that puts the sign at bit 15 and the other three bits at exponent and
// mantissa, and a mask, which reads as code * 2^-126; the multiplication by the scale that follows
// leaves code * s times a power of two (taken out of the finished sum). The order of elements within the
// instruction's K is free, and x is paired alike.
//
// With few outputs the CTAs of a cluster take shares of K and add their sums in order through
// distributed shared memory.
#include "fp4.cuh"
#include "profile.cuh"

namespace lnq {

namespace gv {
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kRows = 16;        // outputs of a tile
constexpr int kChunk = 128;      // elements of K a warp takes at a time
constexpr int kAhead = 4;        // chunks whose codes a warp has in flight
constexpr int kMaxShares = 8;    // CTAs of a cluster
constexpr int kXBytes = 100000;  // shared memory for x: two CTAs fit an SM

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

// Elements i and i + 4 (i = 0, 1) of a word of codes, as two bf16 numbers times 2^-126: the code
// n = 8 sign + rest, times 2^12 + 2^6, has the sign at bit 15 and the rest at bits 8 .. 6.
template <int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t w)
{
    return ((w & (0x000F000Fu << (4 * I))) * (4160u >> (4 * I))) & 0x81C081C0u;
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
    hi[0] = mul_bf16x2(code_pair<0>(w0 >> 8), m0);
    hi[1] = mul_bf16x2(code_pair<0>(w1 >> 8), m1);
    hi[2] = mul_bf16x2(code_pair<1>(w0 >> 8), m0);
    hi[3] = mul_bf16x2(code_pair<1>(w1 >> 8), m1);
}

// One chunk of one lane: codes and scale bytes of outputs g and g + 8.
struct Chunk {
    uint4 q0, q1;
    uint32_t s0, s1;
};

// Weights enter as code * s * 2^kShift. NV: s 2^119 is a normal number for every s. MX: with a factor
// 2^-2 every code * s is a bf16 number (6 2^127 2^-2 .. 0.5 2^-127 2^-2, the smallest subnormal), and
// its multiplier 2^(v - 127 + 124) one while v <= kTopScale; a larger v takes a second factor.
template <int FMT> constexpr float kUnshift = FMT == LNQ_FP4_MX ? 4.f : 128.f;
constexpr uint32_t kTopScale = 130u;

// The (first) multiplier of a scale byte, as bf16 twice.
template <int FMT>
__device__ __forceinline__ uint32_t scale_pair(uint32_t v)
{
    if (FMT == LNQ_FP4_MX)
        return v == 255u ? 0x7FC07FC0u : (min(v, kTopScale) + 124u) * 0x00800080u;
    // exponent and mantissa bits at a bf16's, which reads as s 2^-120, then 2^120 and 2^119
    const uint32_t m = mul_bf16x2(mul_bf16x2((v & 127u) * 0x00100010u, 0x7B807B80u), 0x7B007B00u);
    return (v & 127u) == 127u ? 0x7FC07FC0u : m;
}
// The second one of a large MX scale: 2^(v - 130).
__device__ __forceinline__ uint32_t scale_rest(uint32_t v)
{
    return (max(v, kTopScale) - kTopScale + 127u) * 0x00800080u;
}

// NT column tiles (of 8 / pieces rows of x) per pass over the weights. Grid: x = clusters per
// expert times the cluster's CTAs, y = experts.
template <typename TX, int FMT, int NT>
__global__ void __launch_bounds__(gv::kThreads, 2)
    fp4_gemv_kernel(const TX *__restrict__ x, int n, int64_t ldx, bool wide,
                    const int32_t *__restrict__ offsets, Fp4Matrix w, int d_in, void *__restrict__ y,
                    int yt, int64_t ldy, int shares, int panel)
{
    using namespace gv;
    constexpr int P = Pieces<TX>::n, kTok = 8 / P;   // rows of x per column tile
    constexpr int kPass = NT * kTok;                 // and per pass
    constexpr int kBlocks = 32 / fp4_block(FMT);     // blocks of a lane's 32 elements
    extern __shared__ uint4 xs[];                    // [panel][NT][4 words][32 lanes]
    __shared__ float sums[kWarps][kRows][NT * 8 + 1];
    const int e = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int2 rows = offsets == nullptr ? make_int2(0, n) : fp4_group_rows(offsets, e, n);
    if (rows.x >= rows.y)
        return;
    const int share = shares > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int cluster = static_cast<int>(blockIdx.x) / shares, clusters = static_cast<int>(gridDim.x) / shares;
    const int d_out = static_cast<int>(w.rows), tiles = (d_out + kRows - 1) / kRows;
    const int64_t code_pitch = fp4_code_pitch(d_in), scale_pitch = fp4_scale_pitch(d_in, FMT);
    const int chunks = (d_in + kChunk - 1) / kChunk;
    const int blocks = (d_in + fp4_block(FMT) - 1) / fp4_block(FMT);
    const int c_begin = static_cast<int>(static_cast<int64_t>(share) * chunks / shares);
    const int c_end = static_cast<int>(static_cast<int64_t>(share + 1) * chunks / shares);
    const int64_t first = static_cast<int64_t>(e) * d_out;
    const float scale = (w.t == nullptr ? 1.f : __ldg(w.t + e)) * kUnshift<FMT>;
    // this warp's tiles: tile0, tile0 + hop, ...; the CTA's rounds
    const int tile0 = cluster + warp * clusters, hop = kWarps * clusters;
    const int rounds = (tiles - cluster + hop - 1) / hop;
    const bool once = c_end - c_begin <= panel;  // x fits at once

    for (int b0 = rows.x; b0 < rows.y; b0 += kPass) {
        auto stage = [&](int c0, int c1) {  // x of chunks c0 .. c1 - 1
            for (int i = threadIdx.x; i < (c1 - c0) * NT * 128; i += kThreads) {
                const int c = i / (NT * 128), nt = i / 128 % NT, j = (i >> 5) & 3, l = i & 31;
                const int col = l >> 2, b = b0 + nt * kTok + col / P;
                const int k = (c0 + c) * kChunk + (l & 3) * 32 + j * 8;
                const int left = col < kTok * P && b < rows.y ? d_in - k : 0;
                uint32_t v[4];
                load_column<TX>(x + (left > 0 ? b * ldx + k : 0), left, wide, col % P, v);
                xs[i] = make_uint4(v[0], v[1], v[2], v[3]);
            }
        };
        __syncthreads();  // the last pass has read x
        if (once) {
            stage(c_begin, c_end);
            __syncthreads();
        }
        for (int round = 0; round < rounds; ++round) {
            const int tile = tile0 + round * hop;
            const bool mine = tile < tiles;
            // outputs behind the last (nobody writes their sums) repeat it
            const int j0 = tile * kRows;
            const int64_t r0 = first + min(j0 + g, d_out - 1), r1 = first + min(j0 + g + 8, d_out - 1);
            const uint8_t *codes0 = w.codes + r0 * code_pitch + t * 16;
            const uint8_t *codes1 = w.codes + r1 * code_pitch + t * 16;
            const uint8_t *scales0 = w.scales + r0 * scale_pitch + t * kBlocks;
            const uint8_t *scales1 = w.scales + r1 * scale_pitch + t * kBlocks;
            auto fetch = [&](Chunk &q, int c, int c1) {
                if (c >= c1)
                    return;
                q.q0 = __ldg(reinterpret_cast<const uint4 *>(codes0 + static_cast<int64_t>(c) * 64));
                q.q1 = __ldg(reinterpret_cast<const uint4 *>(codes1 + static_cast<int64_t>(c) * 64));
                if (kBlocks == 2) {
                    q.s0 = __ldg(reinterpret_cast<const uint16_t *>(scales0 + c * 8));
                    q.s1 = __ldg(reinterpret_cast<const uint16_t *>(scales1 + c * 8));
                } else {
                    q.s0 = __ldg(scales0 + c * 4);
                    q.s1 = __ldg(scales1 + c * 4);
                }
            };
            float acc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    acc[nt][k] = 0.f;
            for (int p0 = c_begin; p0 < c_end; p0 += panel) {
                const int p1 = min(p0 + panel, c_end);
                if (!once) {
                    __syncthreads();
                    stage(p0, p1);
                    __syncthreads();
                }
                if (!mine)
                    continue;
                Chunk ring[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    fetch(ring[u], p0 + u, p1);
                for (int cc = p0; cc < p1; cc += kAhead) {
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {
                        const int c = cc + u;
                        if (c >= p1)
                            break;
                        const Chunk q = ring[u];
                        fetch(ring[u], c + kAhead, p1);
                        const uint32_t w0[4] = {q.q0.x, q.q0.y, q.q0.z, q.q0.w};
                        const uint32_t w1[4] = {q.q1.x, q.q1.y, q.q1.z, q.q1.w};
                        const int block0 = c * (kChunk / fp4_block(FMT)) + t * kBlocks;
                        const uint4 *xc = xs + (c - p0) * (NT * 128) + lane;
                        uint32_t m0[kBlocks], m1[kBlocks];
#pragma unroll
                        for (int k = 0; k < kBlocks; ++k) {
                            const bool in = block0 + k < blocks;  // else behind the row
                            m0[k] = in ? scale_pair<FMT>((q.s0 >> (8 * k)) & 255u) : 0u;
                            m1[k] = in ? scale_pair<FMT>((q.s1 >> (8 * k)) & 255u) : 0u;
                        }
                        const bool large = FMT == LNQ_FP4_MX &&
                                           __any_sync(0xffffffffu, max(q.s0, q.s1) > kTopScale);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t lo[4], hi[4];
                            decode_word(w0[j], w1[j], m0[j * kBlocks / 4], m1[j * kBlocks / 4], lo, hi);
                            if (large) {
                                const uint32_t h0 = scale_rest(q.s0), h1 = scale_rest(q.s1);
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    lo[k] = mul_bf16x2(lo[k], k & 1 ? h1 : h0);
                                    hi[k] = mul_bf16x2(hi[k], k & 1 ? h1 : h0);
                                }
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const uint4 v = xc[nt * 128 + j * 32];
                                mma_bf16(acc[nt], lo, v.x, v.y);
                                mma_bf16(acc[nt], hi, v.z, v.w);
                            }
                        }
                    }
                }
            }
            if (mine) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    sums[warp][g][nt * 8 + 2 * t] = acc[nt][0];
                    sums[warp][g][nt * 8 + 2 * t + 1] = acc[nt][1];
                    sums[warp][g + 8][nt * 8 + 2 * t] = acc[nt][2];
                    sums[warp][g + 8][nt * 8 + 2 * t + 1] = acc[nt][3];
                }
            }
            // output i of the round: tile i / (16 kPass) of the CTA, row of x, output of the tile
            auto finish = [&](int i, auto &&sum_at) {
                const int k = i / (kRows * kPass), b = i / kRows % kPass, r = i % kRows;
                const int j = (tile0 + (k - warp) * clusters + round * hop) * kRows + r;
                if (b0 + b >= rows.y || j >= d_out)
                    return;
                float sum = 0.f;
#pragma unroll
                for (int p = P - 1; p >= 0; --p)  // the small pieces first
                    sum = sum_at(sum, k, r, b / kTok * 8 + b % kTok * P + p);
                sum *= scale;
                const int64_t o = static_cast<int64_t>(b0 + b) * ldy + j;
                if (yt == LNQ_BF16)
                    static_cast<__nv_bfloat16 *>(y)[o] = from_f32<__nv_bfloat16>(sum);
                else if (yt == LNQ_F16)
                    static_cast<__half *>(y)[o] = from_f32<__half>(sum);
                else
                    static_cast<float *>(y)[o] = sum;
            };
            if (shares == 1) {  // a warp has its tile's whole sums
                __syncwarp();
                for (int i = lane; i < kRows * kPass; i += 32)
                    finish(warp * kRows * kPass + i,
                           [&](float s, int k, int r, int c) { return s + sums[k][r][c]; });
                __syncwarp();
            } else {
                cluster_sync();
                for (int i = share * kThreads + threadIdx.x; i < kWarps * kRows * kPass; i += shares * kThreads)
                    finish(i, [&](float s, int k, int r, int c) {
                        float v[kMaxShares];
#pragma unroll
                        for (int q = 0; q < kMaxShares; ++q)
                            if (q < shares)
                                asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                             : "=f"(v[q])
                                             : "r"(cluster_addr(&sums[k][r][c], static_cast<uint32_t>(q))));
#pragma unroll
                        for (int q = 0; q < kMaxShares; ++q)
                            if (q < shares)
                                s += v[q];
                        return s;
                    });
                cluster_sync();  // the sums have been read
            }
        }
    }
}

template <typename TX, int FMT, int NT>
static cudaError_t gemv_tiles(const void *x, int n, int64_t ldx, const int32_t *offsets,
                              int64_t experts, const Fp4Matrix &w, int64_t d_in, void *y, int yt,
                              int64_t ldy, int num_sms, cudaStream_t s)
{
    using namespace gv;
    const bool wide = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && ldx * sizeof(TX) % 16 == 0;
    const int64_t tiles = (w.rows + kRows - 1) / kRows, chunks = (d_in + kChunk - 1) / kChunk;
    const int64_t busy = offsets == nullptr ? 1 : min(experts, static_cast<int64_t>(n));  // experts
    const int64_t room = 2 * num_sms;  // CTAs that run at once
    constexpr int kChunkBytes = NT * 128 * 16;
    // K is shared while there are fewer tiles than warps, or while a share of x does not fit
    int shares = 1;
    while (shares < kMaxShares && chunks >= shares * 4 &&
           (tiles * busy * shares < room * kWarps || chunks * kChunkBytes > static_cast<int64_t>(shares) * kXBytes))
        shares *= 2;
    const int panel = static_cast<int>(min((chunks + shares - 1) / shares, static_cast<int64_t>(kXBytes / kChunkBytes)));
    const int64_t clusters = max(int64_t(1), min((tiles + kWarps - 1) / kWarps,
                                                 (room + busy * shares - 1) / (busy * shares)));
    auto *kernel = fp4_gemv_kernel<TX, FMT, NT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kXBytes);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(shares);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * shares), static_cast<unsigned>(experts));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(panel) * kChunkBytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    KernelTimer timer("lnq_fp4_gemv", s);
    e = cudaLaunchKernelEx(&cfg, kernel, static_cast<const TX *>(x), n, ldx, wide, offsets, w,
                           static_cast<int>(d_in), y, yt, ldy, shares, panel);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename TX, int FMT>
static cudaError_t gemv_fmt(const void *x, int n, int64_t ldx, const int32_t *offsets,
                            int64_t experts, const Fp4Matrix &w, int64_t d_in, void *y, int yt,
                            int64_t ldy, int num_sms, cudaStream_t s)
{
    // column tiles of a pass: enough for a group of average size, at most 4
    const int64_t mean = (n + experts - 1) / experts, tiles = (mean * gv::Pieces<TX>::n + 7) / 8;
    if (tiles <= 1)
        return gemv_tiles<TX, FMT, 1>(x, n, ldx, offsets, experts, w, d_in, y, yt, ldy, num_sms, s);
    if (tiles <= 2)
        return gemv_tiles<TX, FMT, 2>(x, n, ldx, offsets, experts, w, d_in, y, yt, ldy, num_sms, s);
    return gemv_tiles<TX, FMT, 4>(x, n, ldx, offsets, experts, w, d_in, y, yt, ldy, num_sms, s);
}

template <typename TX>
static cudaError_t gemv_in(const void *x, int n, int64_t ldx, const int32_t *offsets,
                           int64_t experts, const Fp4Matrix &w, int64_t d_in, int fmt, void *y,
                           int yt, int64_t ldy, int num_sms, cudaStream_t s)
{
    return fmt == LNQ_FP4_MX
               ? gemv_fmt<TX, LNQ_FP4_MX>(x, n, ldx, offsets, experts, w, d_in, y, yt, ldy, num_sms, s)
               : gemv_fmt<TX, LNQ_FP4_NV>(x, n, ldx, offsets, experts, w, d_in, y, yt, ldy, num_sms, s);
}

cudaError_t fp4_gemv_launch(const void *x, int xt, int64_t n, int64_t ldx, const int32_t *offsets,
                            int64_t experts, const Fp4Matrix &w, int64_t d_in, int fmt, void *y,
                            int yt, int64_t ldy, int num_sms, cudaStream_t s)
{
    const int rows = static_cast<int>(n);
    switch (xt) {
    case LNQ_F32:
        return gemv_in<float>(x, rows, ldx, offsets, experts, w, d_in, fmt, y, yt, ldy, num_sms, s);
    case LNQ_BF16:
        return gemv_in<__nv_bfloat16>(x, rows, ldx, offsets, experts, w, d_in, fmt, y, yt, ldy, num_sms, s);
    case LNQ_F16:
        return gemv_in<__half>(x, rows, ldx, offsets, experts, w, d_in, fmt, y, yt, ldy, num_sms, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace lnq
