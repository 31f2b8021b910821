// fp4_gemv.cu -- unquantised activations times a quantised matrix, for few rows, and the same
// with the rows grouped by expert.
//
//   y[b][j] = t sum_k s[j][k] sum_{i in block k} x[b][i] code[j][i]
//
// Bound: HBM, the codes and scales read once (half a byte and 1/16 (NV) or 1/32 (MX) of a byte an
// element). Large calls take instructions instead, about 3.4 an element: 16 rows over 8 experts 4096 ->
// 14336 75 us (3.5 TB/s of codes and scales), no unit full over the whole kernel (issue slots 67%,
// integer pipe 60%), but more than one warp ready where one issues. Small ones take their fixed
// parts, one after the other (x to shared memory, decoding, the join), and a last round of tiles that
// does not fill the warps: 1 x 4096 -> 14336 16 us, 16 x 4096 -> 14336 29 us, 1 x 4096 -> 4096 8.7 us,
// 7 x 11008 -> 4101 in 32 bits 22 us.
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
// With few tiles several warps of a CTA share a tile's K, and where x does not fit its shared
// memory several CTAs of a cluster do; the sums are added in order.
#include "fp4.cuh"
#include "profile.cuh"
#include "resident.h"

namespace lnq {

namespace gv {
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kRows = 16;        // outputs of a tile
constexpr int kChunk = 128;      // elements of K a warp takes at a time
constexpr int kAhead = 4;        // chunks whose codes a warp has in flight
constexpr int kSumPitch = kRows + 4;  // a warp's two columns by 8 outputs fall into different banks
constexpr int kMaxShares = 8;    // CTAs of a cluster
constexpr int kXBytes = 92 << 10;  // shared memory for x: two CTAs fit an SM

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

// The pieces of v, as bf16 bits: the leading 8 bits, the next 8, the last 8. An infinity is all in
// the first; a NaN is in the last too.
template <int P>
__device__ __forceinline__ void split_bf16(float v, uint32_t (&bits)[P])
{
    bits[0] = __float_as_uint(v) >> 16;
    if constexpr (P > 1) {
        const float r = fabsf(v) == __uint_as_float(0x7F800000u)
                            ? 0.f
                            : v - __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
        if constexpr (P == 2) {
            bits[1] = __float_as_uint(r) >> 16;  // of a 16-bit v the rest has 3 bits
        } else {
            const float b = __uint_as_float(__float_as_uint(r) & 0xFFFF0000u);
            bits[1] = __float_as_uint(b) >> 16;
            bits[2] = __float_as_uint(r - b) >> 16;
        }
    }
}

// x[0..7] (zeros from element `left` on) as one word's part of the instruction's columns, one for
// each piece: register i holds elements i and i + 4.
template <typename TX>
__device__ __forceinline__ void load_columns(const TX *__restrict__ x, int left, bool wide,
                                             uint4 (&col)[gv::Pieces<TX>::n])
{
    constexpr int P = gv::Pieces<TX>::n;
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
    if constexpr (P == 1) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(e);
        col[0] = make_uint4(__byte_perm(w[0], w[2], 0x5410), __byte_perm(w[0], w[2], 0x7632),
                            __byte_perm(w[1], w[3], 0x5410), __byte_perm(w[1], w[3], 0x7632));
    } else {
        uint32_t b[8][P];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            split_bf16<P>(to_f32<TX>(e[k]), b[k]);
#pragma unroll
        for (int p = 0; p < P; ++p)
            col[p] = make_uint4(b[0][p] | (b[4][p] << 16), b[1][p] | (b[5][p] << 16),
                                b[2][p] | (b[6][p] << 16), b[3][p] | (b[7][p] << 16));
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
// 2^-2 every code * s is a bf16 number (6 2^127 2^-2 .. 0.5 2^-127 2^-2 = 2^-130, a subnormal one), and
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

// A round of a CTA: 2^log warps to each of its next tiles; the last tiles (1 or more) take all the
// warps they can, as long as `chunks` of K give each two (16 rows over 8 experts 4096 -> 14336:
// 73 us, 80 with its last tiles' other warps idle).
__host__ __device__ __forceinline__ int gemv_round_log(int log, int tiles_left, int chunks)
{
    while (tiles_left > 0 && (tiles_left << (log + 1)) <= gv::kWarps && (chunks >> (log + 2)) > 0)
        ++log;
    return log;
}

// NT tiles of 8 columns (pieces of rows of x) per pass over the weights. Grid: x = clusters per
// expert times the cluster's CTAs, y = experts. 2^`part_log` warps (more in the last round) share a
// tile's K within a CTA, `shares` CTAs within a cluster; `panel` chunks of x fit at a time.
template <typename TX, int FMT, int NT>
__global__ void __launch_bounds__(gv::kThreads, 2)
    fp4_gemv_kernel(const TX *__restrict__ x, int n, int64_t ldx, bool wide,
                    const int32_t *__restrict__ offsets, Fp4Matrix w, int d_in, void *__restrict__ y,
                    int yt, int64_t ldy, int part_log, int shares, int panel)
{
    using namespace gv;
    constexpr int P = Pieces<TX>::n, kPass = NT * 8 / P;  // rows of x per pass: P columns each
    constexpr int kBlocks = 32 / fp4_block(FMT);     // blocks of a lane's 32 elements
    // x: a word's 8 columns by 4 lanes t in the order of the lanes that read them
    extern __shared__ uint4 xs[];  // [panel][NT][4 words][8 columns][4 lanes t]
    __shared__ float sums[kWarps][NT * 8][kSumPitch];
    // the multiplier of each scale byte (76 us where computing them takes 80, 16 rows over 8 experts
    // 4096 -> 14336; 117 and 121, 64 rows; the same where there is one matrix)
    __shared__ uint32_t multiplier[256];
    const int e = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int2 rows = offsets == nullptr ? make_int2(0, n) : fp4_group_rows(offsets, e, n);
    if (rows.x >= rows.y)
        return;
    multiplier[threadIdx.x] = scale_pair<FMT>(threadIdx.x);
    const int share = shares > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int cluster = static_cast<int>(blockIdx.x) / shares, clusters = static_cast<int>(gridDim.x) / shares;
    const int d_out = static_cast<int>(w.rows), tiles = (d_out + kRows - 1) / kRows;
    const int64_t code_pitch = fp4_code_pitch(d_in), scale_pitch = fp4_scale_pitch(d_in, FMT);
    const int chunks = (d_in + kChunk - 1) / kChunk;
    const int c_begin = static_cast<int>(static_cast<int64_t>(share) * chunks / shares);
    const int c_end = static_cast<int>(static_cast<int64_t>(share + 1) * chunks / shares);
    // this lane's scale bytes of the last chunk: zeros behind the row's last block
    const int left_blocks = (d_in - (chunks - 1) * kChunk - t * 32 + fp4_block(FMT) - 1) / fp4_block(FMT);
    const uint32_t tail = left_blocks >= kBlocks ? 0xFFFFu : (left_blocks == 1 ? 0xFFu : 0u);
    const int64_t first = static_cast<int64_t>(e) * d_out;
    // the power of two goes to the sum before a large t, with which it might overflow
    const float t_e = w.t == nullptr ? 1.f : __ldg(w.t + e);
    const bool t_large = fabsf(t_e) >= 1.f;
    const float scale0 = t_large ? kUnshift<FMT> : 1.f, scale1 = t_large ? t_e : t_e * kUnshift<FMT>;
    const int own = (chunks + shares - 1) / shares;  // chunks of the cluster's largest share
    const int count = (tiles - cluster + clusters - 1) / clusters;  // tiles: every clusters-th
    const bool once = c_end - c_begin <= panel;  // x fits at once

    for (int b0 = rows.x; b0 < rows.y; b0 += kPass) {
        const int tokens = min(kPass, rows.y - b0);
        auto stage = [&](int c0, int c1) {  // x of chunks c0 .. c1 - 1
#pragma unroll 2
            for (int i = threadIdx.x; i < (c1 - c0) * 16 * tokens; i += kThreads) {
                const int q = i & 15, r = i / 16, c = r / tokens, token = r - c * tokens;  // q: [word][t]
                const int k = (c0 + c) * kChunk + (q & 3) * 32 + (q >> 2) * 8;
                uint4 col[P];
                load_columns<TX>(x + (k < d_in ? (b0 + token) * ldx + k : 0), d_in - k, wide, col);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const int at = token * P + p;  // column of the pass
                    xs[((c * NT + at / 8) * 4 + (q >> 2)) * 32 + at % 8 * 4 + (q & 3)] = col[p];
                }
            }
        };
        const uint8_t *codes0, *codes1, *scales0, *scales1;
        Chunk ring[kAhead];
        auto fetch = [&](Chunk &q, int ahead, int left) {
            if (left <= 0)
                return;
            q.q0 = __ldg(reinterpret_cast<const uint4 *>(codes0 + ahead * 64));
            q.q1 = __ldg(reinterpret_cast<const uint4 *>(codes1 + ahead * 64));
            if (kBlocks == 2) {
                q.s0 = __ldg(reinterpret_cast<const uint16_t *>(scales0 + ahead * 8));
                q.s1 = __ldg(reinterpret_cast<const uint16_t *>(scales1 + ahead * 8));
            } else {
                q.s0 = __ldg(scales0 + ahead * 4);
                q.s1 = __ldg(scales1 + ahead * 4);
            }
        };
        // this warp's tile of a round that begins at the CTA's tile `done`, and its part of chunks
        // p0 .. p1 - 1
        auto tile_of = [&](int done, int log) { return cluster + (done + (warp >> log)) * clusters; };
        auto part_of = [&](int log, int p0, int p1) {
            const int part = warp & ((1 << log) - 1);
            return make_int2(p0 + (part * (p1 - p0) >> log), p0 + ((part + 1) * (p1 - p0) >> log));
        };
        // the first chunks of it
        auto begin = [&](int done, int log, int p0, int p1) {
            const int tile = tile_of(done, log);
            if (tile >= tiles)
                return;
            const int2 part = part_of(log, p0, p1);
            const int w_begin = part.x, w_end = part.y;
            // outputs behind the last (nobody writes their sums) repeat it
            const int64_t r0 = first + min(tile * kRows + g, d_out - 1);
            const int64_t r1 = first + min(tile * kRows + g + 8, d_out - 1);
            codes0 = w.codes + r0 * code_pitch + static_cast<int64_t>(w_begin) * 64 + t * 16;
            codes1 = w.codes + r1 * code_pitch + static_cast<int64_t>(w_begin) * 64 + t * 16;
            scales0 = w.scales + r0 * scale_pitch + (w_begin * 4 + t) * kBlocks;
            scales1 = w.scales + r1 * scale_pitch + (w_begin * 4 + t) * kBlocks;
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                fetch(ring[u], u, w_end - w_begin - u);
        };
        int log = gemv_round_log(part_log, count, own);
        if (once)
            begin(0, log, c_begin, c_end);  // its loads run while x is written
        __syncthreads();  // the last pass has read x; the multipliers are written
        if (once) {
            stage(c_begin, c_end);
            __syncthreads();
        }
        for (int done = 0, slots, next; done < count; done += slots, log = next) {
            const int parts = 1 << log;
            slots = kWarps >> log;
            next = gemv_round_log(part_log, count - done - slots, own);
            const bool mine = tile_of(done, log) < tiles;
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
                    begin(done, log, p0, p1);
                }
                if (!mine)
                    continue;
                const int2 part = part_of(log, p0, p1);
                const int w_begin = part.x, w_end = part.y;
                // (the columns behind the last row's hold anything: nobody reads their sums)
                const uint4 *xc = xs + (w_begin - p0) * (NT * 128) + lane;
                for (int c0 = w_begin; c0 < w_end; c0 += kAhead) {
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {
                        const int c = c0 + u;
                        if (c >= w_end)
                            break;
                        Chunk &q = ring[u];
                        if (c == chunks - 1) {
                            q.s0 &= tail;
                            q.s1 &= tail;
                        }
                        uint32_t m0[kBlocks], m1[kBlocks];
#pragma unroll
                        for (int k = 0; k < kBlocks; ++k) {
                            const uint32_t v0 = (q.s0 >> (8 * k)) & 255u, v1 = (q.s1 >> (8 * k)) & 255u;
                            m0[k] = multiplier[v0];
                            m1[k] = multiplier[v1];
                        }
                        const bool large = FMT == LNQ_FP4_MX &&
                                           __any_sync(0xffffffffu, max(q.s0, q.s1) > kTopScale);
                        const uint32_t h0 = large ? scale_rest(q.s0) : 0u, h1 = large ? scale_rest(q.s1) : 0u;
                        const uint32_t w0[4] = {q.q0.x, q.q0.y, q.q0.z, q.q0.w};
                        const uint32_t w1[4] = {q.q1.x, q.q1.y, q.q1.z, q.q1.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t lo[4], hi[4];
                            decode_word(w0[j], w1[j], m0[j * kBlocks / 4], m1[j * kBlocks / 4], lo, hi);
                            if (large) {
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
                        xc += NT * 128;
                        fetch(q, u + kAhead, w_end - c - kAhead);
                    }
                    codes0 += kAhead * 64;
                    codes1 += kAhead * 64;
                    scales0 += kAhead * 4 * kBlocks;
                    scales1 += kAhead * 4 * kBlocks;
                }
            }
            if (once && done + slots < count)  // the next tile's loads run while this one's sums are added
                begin(done + slots, next, c_begin, c_end);
            if (mine) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    sums[warp][nt * 8 + 2 * t][g] = acc[nt][0];
                    sums[warp][nt * 8 + 2 * t + 1][g] = acc[nt][1];
                    sums[warp][nt * 8 + 2 * t][g + 8] = acc[nt][2];
                    sums[warp][nt * 8 + 2 * t + 1][g + 8] = acc[nt][3];
                }
            }
            // Output i of the round: tile slot k, row b of x, output r of the tile.
            // This CTA's sum: the small pieces first, of each the warps that share the tile.
            auto own_sum = [&](int k, int b, int r) {
                float sum = 0.f;
#pragma unroll
                for (int p = P - 1; p >= 0; --p)
                    for (int q = 0; q < parts; ++q)
                        sum += sums[k * parts + q][b * P + p][r];
                return sum;
            };
            auto put = [&](int k, int b, int r, float sum) {
                const int j = (cluster + (done + k) * clusters) * kRows + r;
                if (b0 + b >= rows.y || j >= d_out)
                    return;
                sum = sum * scale0 * scale1;
                const int64_t o = static_cast<int64_t>(b0 + b) * ldy + j;
                if (yt == LNQ_BF16)
                    static_cast<__nv_bfloat16 *>(y)[o] = from_f32<__nv_bfloat16>(sum);
                else if (yt == LNQ_F16)
                    static_cast<__half *>(y)[o] = from_f32<__half>(sum);
                else
                    static_cast<float *>(y)[o] = sum;
            };
            __syncthreads();
            for (int i = threadIdx.x; i < slots * kRows * kPass; i += kThreads) {
                const int k = i / (kRows * kPass), b = i / kRows % kPass, r = i % kRows;
                const float sum = own_sum(k, b, r);
                if (shares == 1)
                    put(k, b, r, sum);
                else
                    sums[k * parts][b * P][r] = sum;
            }
            if (shares == 1) {
                __syncthreads();
                continue;
            }
            cluster_sync();
            for (int i = share * kThreads + threadIdx.x; i < slots * kRows * kPass; i += shares * kThreads) {
                const int k = i / (kRows * kPass), b = i / kRows % kPass, r = i % kRows;
                float v[kMaxShares], sum = 0.f;
#pragma unroll
                for (int q = 0; q < kMaxShares; ++q)
                    if (q < shares)
                        asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                     : "=f"(v[q])
                                     : "r"(cluster_addr(&sums[k * parts][b * P][r], static_cast<uint32_t>(q))));
#pragma unroll
                for (int q = 0; q < kMaxShares; ++q)
                    if (q < shares)
                        sum += v[q];
                put(k, b, r, sum);
            }
            cluster_sync();  // the sums have been read
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
    constexpr int64_t kChunkBytes = NT * 128 * 16;
    auto *kernel = fp4_gemv_kernel<TX, FMT, NT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kXBytes);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // How K is shared: by `shares` CTAs of a cluster (less of x for each to write) and 2^`part_log`
    // warps of a CTA. The least cost: a chunk of a column of x staged, a chunk of a tile, and a
    // round's fixed costs, which are larger where a cluster's CTAs wait for one another. The weights
    // were fitted to measured times and rank plans; they do not tell the time (from cold caches
    // 1.2 to 5 times 6.5 ns a unit). Against all shares and parts at 16 sizes (1 to 64 rows, bf16, fp16
    // and fp32, 2048 .. 11008 -> 1408 .. 14336, 1 to 64 experts) it takes the fastest plan or one within
    // 2% of it at 14, 4% more at 16 x 4096 -> 14336 bf16 (33 us where four CTAs to a tile take 32) and 6%
    // at 4 x 2048 -> 1408 fp32 (12.3, 11.6).
    constexpr int64_t kWork = 62 + 13 * NT, kRound = 390, kClusterRound = 530;
    const int64_t stage = min((n + experts - 1) / experts, int64_t(NT * 8 / Pieces<TX>::n)) * Pieces<TX>::n * 4;
    static ResidentClusters resident[4];  // by their size
    const int device = current_device();
    int shares = 1, part_log = 0;
    int64_t clusters = 1, best = INT64_MAX;
    for (int i = 0, c = 1; c <= kMaxShares && (c == 1 || chunks >= c * 2); ++i, c *= 2) {
        const int whole_sms = 2 * num_sms / c;
        const int room = c == 1 ? whole_sms : resident[i].get(device, whole_sms, [&]() {
            attr[0].val.clusterDim.x = static_cast<unsigned>(c);
            cfg.gridDim = dim3(static_cast<unsigned>(whole_sms * c));
            cfg.dynamicSmemBytes = kXBytes / kChunkBytes * kChunkBytes;
            return max_active_clusters(kernel, cfg);
        });
        const int64_t own = (chunks + c - 1) / c, m = max(int64_t(1), min(tiles, room / busy));
        const int64_t per_cta = (tiles + m - 1) / m, waves = (m * busy + room - 1) / room;
        for (int k = 0; k < 4 && (k == 0 || own >= 2 << k); ++k) {
            const int64_t whole = per_cta / (kWarps >> k), left = per_cta % (kWarps >> k);
            const int last = gemv_round_log(k, static_cast<int>(left), static_cast<int>(own));
            const int64_t rounds = whole + (left > 0), stagings = own * kChunkBytes > kXBytes ? rounds : 1;
            const int64_t work = whole * ((own + (1 << k) - 1) >> k) +
                                 (left > 0 ? (own + (1 << last) - 1) >> last : 0);
            const int64_t cost = waves * (stagings * own * stage + work * kWork +
                                          rounds * (c > 1 ? kClusterRound : kRound));
            if (cost < best)
                best = cost, shares = c, part_log = k, clusters = m;
        }
    }
    const int64_t panel = min((chunks + shares - 1) / shares, kXBytes / kChunkBytes);
    attr[0].val.clusterDim.x = static_cast<unsigned>(shares);
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * shares), static_cast<unsigned>(experts));
    cfg.dynamicSmemBytes = static_cast<size_t>(panel * kChunkBytes);
    KernelTimer timer("lnq_fp4_gemv", s);
    e = cudaLaunchKernelEx(&cfg, kernel, static_cast<const TX *>(x), n, ldx, wide, offsets, w,
                           static_cast<int>(d_in), y, yt, ldy, part_log, shares, static_cast<int>(panel));
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
    if (tiles <= 3)
        return gemv_tiles<TX, FMT, 3>(x, n, ldx, offsets, experts, w, d_in, y, yt, ldy, num_sms, s);
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
