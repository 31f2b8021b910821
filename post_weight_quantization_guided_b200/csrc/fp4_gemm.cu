// fp4_gemm.cu -- the product of two quantised matrices, and the same with the rows grouped by
// expert, on the block-scaled tensor cores.
//
//   y[b][j] = ta tw sum_i (code sa)[b][i] (code sw)[j][i]
//
// The weights are the MMA's M side (its rows are outputs j), the activations its N side, so that
// few rows cost narrow tiles, not padded ones. A cluster pair of CTAs computes 256 outputs x BN
// rows (BN = 32 .. 256) with tcgen05.mma.cta_group::2.kind::mxf4nvf4 (M = 256, N = BN, K = 64 per
// instruction); each CTA holds its 128 outputs' codes and half of the BN rows' codes.
//
// Codes come by TMA in stages of 256 elements of K (128 bytes a row, 128-byte swizzle, zeros
// outside the matrix), the block scales of a CTA's 128 outputs and of all BN rows by TMA in steps
// of two stages, in a ring of their own. A warp rearranges the scales in place: row r's four scales
// of 64 (NV) or 128 (MX) elements go where the tensor core wants them, to byte 16 (r % 32) +
// 4 (r / 32 % 4) of a 512-byte atom per 128 rows. (Nothing but TMA may be in flight for the proxy
// fence that follows: it waits for asynchronous copies of the CTA's other warps and for loads of its
// own, which cost 1.2 us a step.) The MMA thread copies the atoms to TMEM (tcgen05.cp, 4 columns
// each, a slot per stage so that no copy overtakes an MMA that still reads) and issues four MMAs
// a stage. All K-wise bounds are in these copies: codes and scales behind the row's end arrive as
// zeros.
//
// Warps: 0-7 epilogue (two per TMEM lane quarter, alternate 32-column chunks), 8 loads, 9-10 scales,
// 11 MMA. Persistent over tiles, outputs fastest, so that neighbouring pairs
// share the rows' tile.
// With few tiles, two pairs of one cluster take half of K each and add their sums through
// distributed shared memory in a fixed order.
//
// What bounds it: the way from stage to stage. One B200, operands in L2: a stage takes 0.36 to 0.38 us
// (about 700 cycles; the slope of the time from K = 4096 to 16384), in 64-row tiles, whose MMAs take
// 128 cycles, as in 256-row ones, whose MMAs take 512, and with 4 pairs at work as with 32. Neither
// the tensor core nor memory sets that pace, nor shared memory (88 KB a stage and CTA in 256-row
// tiles, 690 cycles at 128 bytes a cycle, but 56 KB in 64-row ones), but the chain of TMA, rearranging
// warp, fence, arrival, copy to TMEM, MMA and commit over rings of this depth. With all 74 pairs at
// work it is 0.39 to 0.45 us from L2 and, of operands that L2 does not hold, 0.52 to 0.61.
// 16384 x 4096 -> 14336 NV: 418 us (4.6 PFLOP/s) at the clock that the power limit leaves; at an earlier
// 389 us it was 295 without its code loads, 350 without its stores, 360 without tcgen05.cp. (256-row
// tiles of two accumulators do not fit TMEM beside the scales; stores through shared memory in
// 16-byte pieces were no faster.)
// Few rows: 3 us to the first stage, a tile's stages, the last stores: 32 x 4096 -> 14336 13.5 us.
#include <cstring>

#include "fp4.cuh"
#include "fp4_mma.cuh"
#include "lnq_internal.cuh"
#include "profile.cuh"
#include "resident.h"

namespace lnq {

// Waits that gave up: by the slot of the product's stream, [kCapturedSlot] of products captured into
// a graph, which runs on any stream, and [kAllSlot] of all.
constexpr int kCapturedSlot = kFp4ReportSlots, kAllSlot = kFp4ReportSlots + 1;
__device__ uint32_t g_fp4_gave_up[kFp4ReportSlots + 2];

__device__ __forceinline__ void give_up(int slot)
{
    atomicAdd(&g_fp4_gave_up[slot], 1u);
    atomicAdd(&g_fp4_gave_up[kAllSlot], 1u);
}

namespace f4 {
constexpr int BM = 128, PM = 256;       // outputs of a CTA, of a pair
constexpr int BK = 256;                 // elements of K per stage: 128 bytes of codes a row
constexpr int kEpiWarps = 8;
constexpr int kTmaWarp = 8, kLoadWarp = 9, kScaleWarp = 10, kMmaWarp = 11;
constexpr int kThreads = 12 * 32;       // 168 registers a thread
constexpr int kScaleRing = 4;           // steps (two stages each) of scales in flight
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxSplit = 2;            // pairs of a cluster
constexpr int kAtom = 512;              // bytes of scales of 128 rows x 4 blocks

template <int BN, int FMT>
struct Tile {
    static constexpr int kAtomsK = BK / fp4_block(FMT) / 4;       // scale atoms per stage along K
    static constexpr int kAtomsN = (BN + 127) / 128;              // along the rows
    static constexpr int kABytes = BM * 128, kBBytes = BN / 2 * 128;
    static constexpr int kScaleBytes = kAtomsK * (1 + kAtomsN) * kAtom;
    static constexpr int kRowBytes = 8 * kAtomsK;                  // scales of a row and step
    static constexpr int kStepBytes = 2 * kScaleBytes;
    // Offset of 16-byte chunk c of row i of a step's scales as they come (see the load warp).
    static __device__ __forceinline__ uint32_t chunk_at(int i, int c)
    {
        return kRowBytes == 32 ? static_cast<uint32_t>(i * 32 + ((c ^ (i >> 2)) & 1) * 16)
                               : static_cast<uint32_t>(i * 16);
    }
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kSlotCols = kAtomsK * 4 * (1 + kAtomsN);  // TMEM columns of a stage's scales
    static constexpr int kAcc = BN == 256 ? 1 : 2;                 // accumulators
    static constexpr int kStages = BN == 256 ? 5 : (BN == 128 ? 7 : 8);
    static constexpr int kLimInts = LNQ_FP4_MAX_EXPERTS + 1;
    static constexpr int kBars = 2 * kStages + 3 * kScaleRing + 2 * kAcc + 1;
    static constexpr size_t kSmem = static_cast<size_t>(kStages) * kStageBytes +
                                    kScaleRing * kStepBytes + 2 * kLimInts * 4 + kBars * 8 + 32 + 1024 /* alignment */;
    static_assert(kSmem <= 232448, "shared memory");
    static_assert(kStages * kSlotCols + kAcc * BN <= static_cast<int>(kTmemCols), "TMEM");
    static_assert(kStageBytes % 1024 == 0, "stages");
    static_assert(BN > 128 || BN * BM * 4 <= kStages * kStageBytes, "partial sums of a split");
};
}  // namespace f4

struct Fp4GemmParams {
    const uint8_t *a_scales, *w_scales;  // rows (activations), outputs (weights)
    const float *ta, *tw;
    const int32_t *offsets;
    void *y;
    int64_t ldy;
    int64_t w_total;       // outputs of all matrices
    int n, experts, d_out;
    int yt;
    int nk;                // stages of K
    int blocks;            // scale blocks of a row
    int scale_pitch;       // bytes
    int mt;                // output tiles of one matrix
    int split;             // pairs that share a tile's K
    int sf_tma;            // scales by TMA: rows are multiples of 16 bytes
    int report;            // where a wait that gives up is counted
    long long limit;
};

// What a finished sum v is multiplied by, one after the other: v * f2 * f0 * f1 is v * ta * tw, where
// neither ta nor tw alone takes it out of the 32-bit range. f2 is a power of two, 1 in all ordinary
// cases (and then left out). For the sums that there can be, 0 and 2^-20 to 2^47 (six bits a code and
// scale, 2^24 products): f0 takes an exponent of -60 to 60, so v * f2 is inexact or infinite only where
// the result is 0 or infinite.
struct Fp4Factors {
    float f0, f1, f2;
    __device__ __forceinline__ Fp4Factors(float ta, float tw) : f0(ta), f1(tw), f2(1.f)
    {
        auto ordinary = [](float t) { return t >= 0x1p-60f && t <= 0x1p60f; };
        auto valid = [](float t) { return t > 0.f && t < __uint_as_float(0x7F800000u); };
        if ((ordinary(ta) && ordinary(tw)) || !valid(ta) || !valid(tw))
            return;
        int e = 0;
        auto mantissa = [&](float t) {  // of t, 1 .. 2, its exponent added to e
            const float n = t < 0x1p-126f ? t * 0x1p64f : t;
            e += static_cast<int>(__float_as_uint(n) >> 23) - 127 - (t < 0x1p-126f ? 64 : 0);
            return __uint_as_float((__float_as_uint(n) & 0x007FFFFFu) | 0x3F800000u);
        };
        f0 = mantissa(ta);
        f1 = mantissa(tw);
        const int near = max(-60, min(e, 60)), rest = min(e - near, 127);  // 2^127 is infinite already
        f0 *= __uint_as_float(static_cast<uint32_t>(near + 127) << 23);
        f2 = __uint_as_float(rest >= -126 ? static_cast<uint32_t>(rest + 127) << 23
                                          : (rest >= -149 ? 1u << (rest + 149) : 0u));
    }
    __device__ __forceinline__ float operator()(float v) const { return v * f0 * f1; }
};

template <typename T>
__device__ __forceinline__ void store_column(T *__restrict__ y, int64_t ldy, int count,
                                             const uint32_t (&v)[32], const Fp4Factors &f)
{
    if (count >= 32) {
#pragma unroll
        for (int c = 0; c < 32; ++c)
            y[c * ldy] = from_f32<T>(f(__uint_as_float(v[c])));
    } else {
#pragma unroll
        for (int c = 0; c < 32; ++c)
            if (c < count)
                y[c * ldy] = from_f32<T>(f(__uint_as_float(v[c])));
    }
}

// Where a tile lies: group, first row and the row behind the group's last, first output.
struct Fp4TileAt {
    int e, b0, b1, j0;
};

template <int BN>
__device__ __forceinline__ Fp4TileAt tile_at(int64_t tile, const Fp4GemmParams &p, const int *lim,
                                             const int *pre)
{
    const int q = static_cast<int>(tile / p.mt), m = static_cast<int>(tile - int64_t(q) * p.mt);
    int lo = 0, hi = p.experts;  // pre[lo] <= q < pre[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= q)
            lo = mid;
        else
            hi = mid;
    }
    return Fp4TileAt{lo, lim[lo] + (q - pre[lo]) * BN, lim[lo + 1], m * f4::PM};
}

template <int BN, int FMT>
__global__ void __launch_bounds__(f4::kThreads, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap wmap,
                    const __grid_constant__ CUtensorMap amap,
                    const __grid_constant__ CUtensorMap wsmap,
                    const __grid_constant__ CUtensorMap asmap, const Fp4GemmParams p)
{
    using namespace f4;
    using T = Tile<BN, FMT>;
    constexpr int W = T::kAtomsK;            // words of scales per row and stage
    constexpr int kGroups = 1 + T::kAtomsN;  // of 128 rows of scales: outputs, then the tile's rows
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(align_up(reinterpret_cast<uintptr_t>(smem_raw), 1024));
    uint8_t *sf = smem + T::kStages * T::kStageBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sf + kScaleRing * T::kStepBytes);
    uint64_t *full = bars;                           // codes landed (leader's: both CTAs')
    uint64_t *empty = full + T::kStages;             // stage and TMEM slot free (each CTA's)
    uint64_t *sf_raw = empty + T::kStages;           // a step's scales landed (each CTA's)
    uint64_t *sf_ready = sf_raw + kScaleRing;        // and are in place (leader's: both CTAs')
    uint64_t *sf_empty = sf_ready + kScaleRing;      // and are in TMEM (each CTA's)
    uint64_t *tfull = sf_empty + kScaleRing;         // accumulator done (each CTA's)
    uint64_t *tempty = tfull + T::kAcc;              // accumulator read (leader's: both CTAs')
    uint64_t *drain = tempty + T::kAcc;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 1);
    uint64_t *loaded = drain + 2;  // 1 + stages of codes this CTA loaded, once its loads are over
    int *lim = reinterpret_cast<int *>(tmem_holder + 4);  // [experts + 1] group boundaries
    int *pre = lim + T::kLimInts;                         // [experts + 1] row tiles before group e

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank(), cr = rank & 1u, leader = rank & ~1u;
    const int part = static_cast<int>(rank >> 1);          // this pair's share of K
    const uint16_t pair_mask = static_cast<uint16_t>(3u << leader);
    const int64_t first = blockIdx.x / (2 * p.split), step = gridDim.x / (2 * p.split);
    const int steps = (p.nk + 1) / 2;  // of two stages
    const int kb0 = part * steps / p.split * 2;
    const int kb1 = min((part + 1) * steps / p.split * 2, p.nk);
    // for what ends by itself, or with a wait of `limit` elsewhere in the cluster
    const long long last_limit = (p.limit < (1LL << 62) ? p.limit : 1LL << 62) + kDrainLimit;

    if (threadIdx.x == 32) {
        *loaded = 0u;
        for (int s = 0; s < T::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < kScaleRing; ++s) {
            mbar_init(&sf_raw[s], 1);
            mbar_init(&sf_ready[s], 2);
            mbar_init(&sf_empty[s], 1);
        }
        for (int a = 0; a < T::kAcc; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], 2 * kEpiWarps);
        }
        mbar_init(drain, 1);
        fence_barrier_init();
        tma_prefetch_desc(&wmap);
        tma_prefetch_desc(&amap);
        if (p.sf_tma) {
            tma_prefetch_desc(&wsmap);
            tma_prefetch_desc(&asmap);
        }
    }
    if (warp == kMmaWarp)
        tmem_alloc_pair(tmem_holder, kTmemCols);
    if (warp == 0) {
        // group boundaries: offsets limited to 0 .. n and to no less than the largest before
        int top = 0, tiles = 0;
        if (p.offsets == nullptr) {
            if (lane < 2)
                lim[lane] = lane * p.n;
        } else {
            for (int i = lane; i - lane <= p.experts; i += 32) {
                int v = i <= p.experts ? min(p.offsets[i], p.n) : 0;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(0xffffffffu, v, o);
                    v = lane >= o ? max(v, u) : v;
                }
                v = max(v, top);
                top = __shfl_sync(0xffffffffu, v, 31);
                if (i <= p.experts)
                    lim[i] = v;
            }
        }
        __syncwarp();
        if (lane == 0)
            pre[0] = 0;
        for (int i = lane; i - lane < p.experts; i += 32) {
            int v = i < p.experts ? (lim[i + 1] - lim[i] + BN - 1) / BN : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                v += lane >= o ? u : 0;
            }
            v += tiles;
            tiles = __shfl_sync(0xffffffffu, v, 31);
            if (i < p.experts)
                pre[i + 1] = v;
        }
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    const int64_t num_tiles = static_cast<int64_t>(pre[p.experts]) * p.mt;

    if (warp == kTmaWarp) {
        // ------------------------------------------------------------------ loads by TMA
        // One thread serves two rings, whichever has room: codes in stages, and scales in steps of
        // two stages (8 W bytes of a row: 32 (NV, their 16-byte halves exchanged in every second
        // four rows: TMA's 32-byte swizzle) or 16 (MX)).
        if (lane == 0) {
            int64_t tile = first, sf_tile = p.sf_tma ? first : num_tiles;
            int kb = kb0, sf_kb = kb0, stage = 0, slot = 0;
            uint32_t par = 1u, sf_par = 1u, sf_used = 0u;
            Fp4TileAt at = {0, 0, 0, 0}, sf_at = {0, 0, 0, 0};
            if (first < num_tiles)
                at = sf_at = tile_at<BN>(first, p, lim, pre);
            uint64_t count = 0u;  // stages of codes loaded
            auto load_stage = [&]() {
                uint8_t *st = smem + stage * T::kStageBytes;
                if (cr == 0)
                    mbar_arrive_expect_tx(&full[stage], 2 * T::kStageBytes);
                const uint32_t fb = cluster_addr(&full[stage], leader);
                tma_load_2d_pair(st, &wmap, fb, kb * 128, at.e * p.d_out + at.j0 + static_cast<int>(cr) * BM);
                tma_load_2d_pair(st + T::kABytes, &amap, fb, kb * 128, at.b0 + static_cast<int>(cr) * (BN / 2));
                ++count;
                stage = stage + 1 == T::kStages ? 0 : stage + 1;
                par ^= stage == 0 ? 1u : 0u;
                if (++kb == kb1) {
                    kb = kb0;
                    tile += step;
                    if (tile < num_tiles)
                        at = tile_at<BN>(tile, p, lim, pre);
                }
            };
            long long since = clock64();
            while (tile < num_tiles || sf_tile < num_tiles) {
                bool moved = false;
                if (sf_tile < num_tiles && mbar_test(&sf_empty[slot], sf_par)) {
                    uint8_t *st = sf + slot * T::kStepBytes;
                    mbar_arrive_expect_tx(&sf_raw[slot], (BM + BN) * T::kRowBytes);
                    tma_load_2d(st, &wsmap, &sf_raw[slot], sf_kb * 4 * W,
                                sf_at.e * p.d_out + sf_at.j0 + static_cast<int>(cr) * BM);
                    tma_load_2d(st + BM * T::kRowBytes, &asmap, &sf_raw[slot], sf_kb * 4 * W, sf_at.b0);
                    sf_used |= 1u << slot;
                    slot = slot + 1 == kScaleRing ? 0 : slot + 1;
                    sf_par ^= slot == 0 ? 1u : 0u;
                    sf_kb += 2;
                    if (sf_kb >= kb1) {
                        sf_kb = kb0;
                        sf_tile += step;
                        if (sf_tile < num_tiles)
                            sf_at = tile_at<BN>(sf_tile, p, lim, pre);
                    }
                    moved = true;
                }
                if (tile < num_tiles && mbar_test(&empty[stage], par)) {
                    load_stage();
                    moved = true;
                }
                if (moved) {
                    since = clock64();
                } else if (clock64() - since >= p.limit) {
                    give_up(p.report);
                    break;
                }
            }
            // No copy may be in flight when this CTA exits, whichever thread of the pair gave up: all
            // that was loaded is waited for here, which costs nothing where it is multiplied too.
            // The codes of both CTAs are counted together, on the leader's barriers. So a CTA that
            // gave up first loads the stages that its peer has loaded and it has not: the peer saw
            // them empty, and so they are (one commit tells both).
            st_release_cluster(loaded, count + 1u);
            if (tile < num_tiles) {
                const uint64_t theirs = wait_nonzero_cluster(cluster_addr(loaded, rank ^ 1u), last_limit);
                while (count + 1u < theirs)
                    load_stage();
            }
            for (int s = 0; s < kScaleRing; ++s)
                if ((sf_used >> s) & 1u)
                    mbar_wait(&sf_raw[s], s < slot ? sf_par ^ 1u : sf_par, last_limit);
            for (int s = 0; s < T::kStages && cr == 0; ++s)
                if (static_cast<uint64_t>(s) < count)
                    mbar_wait(&full[s], s < stage ? par ^ 1u : par, last_limit);
        }
    } else if ((warp == kScaleWarp || warp == kLoadWarp) && !p.sf_tma) {
        // ------------------------------------------------------------------ scales without TMA
        // Rows that are no multiples of 16 bytes. The two warps take steps in turn: loads of half a
        // stage's bytes, four lanes to a row's step and eight rows at a time, into registers
        // while the step before is in use; then each word to its place in its atom.
        constexpr int kSets = kGroups * 16, N = W / 2;  // N: words a lane loads of a row
        const uint32_t ready_leader = cluster_addr(&sf_ready[0], leader);
        const int unit = lane & 3, r = lane >> 2;
        uint32_t v[kSets][N];
        int64_t tile = first;
        int kb = kb0, slot = 0;
        uint32_t phase = 1u;
        auto advance = [&]() {
            kb += 2;
            if (kb >= kb1) {
                kb = kb0;
                tile += step;
            }
            slot = slot + 1 == kScaleRing ? 0 : slot + 1;
            phase ^= slot == 0 ? 1u : 0u;
        };
        auto fetch = [&]() {
            if (tile >= num_tiles)
                return;
            const Fp4TileAt at = tile_at<BN>(tile, p, lim, pre);
            // rows outside the arrays (nobody reads their sums) repeat the last one
            const int64_t w0 = min(static_cast<int64_t>(at.e) * p.d_out + at.j0 + static_cast<int>(cr) * BM,
                                   p.w_total - 1);
            const int wtop = static_cast<int>(min(p.w_total - 1 - w0, static_cast<int64_t>(BM)));
            const int atop = min(p.n - 1 - at.b0, BN), o = (kb * W + unit * N) * 4;
            const uint8_t *wsrc = p.w_scales + w0 * p.scale_pitch + o;
            const uint8_t *asrc = p.a_scales + static_cast<int64_t>(at.b0) * p.scale_pitch + o;
#pragma unroll
            for (int g = 0; g < kSets; ++g) {
                const int row = g < 16 ? min(g * 8 + r, wtop) : min((g - 16) * 8 + r, atop);
#pragma unroll
                for (int k = 0; k < N; ++k)
                    v[g][k] = 0u;
                if (o < p.scale_pitch && (g - 16) * 8 < BN)
                    ldg_words<N>(v[g], (g < 16 ? wsrc : asrc) + static_cast<int64_t>(row) * p.scale_pitch);
            }
        };
        if (warp == kLoadWarp)
            advance();
        fetch();
        while (tile < num_tiles) {
            if (!__all_sync(0xffffffffu, mbar_wait(&sf_empty[slot], phase, p.limit))) {
                if (lane == 0)
                    give_up(p.report);
                break;
            }
            const uint32_t st = smem_u32(sf) + static_cast<uint32_t>(slot * T::kStepBytes);
#pragma unroll
            for (int g = 0; g < kSets; ++g) {
                if ((g - 16) * 8 >= BN)
                    continue;
                const int i = g % 16 * 8 + r, group = g / 16;  // row of its 128
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const int word = unit * N + k;  // of the row's step
                    const int h = word / W, a = word % W;
                    const int atom = h * W * kGroups + (group == 0 ? a : W + a * T::kAtomsN + group - 1);
                    // nothing behind the row's last block
                    sts_word(st + static_cast<uint32_t>(atom * kAtom + (i & 31) * 16 + (i >> 5) * 4),
                             v[g][k] & first_bytes(p.blocks - (kb * W + word) * 4));
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_smem_written(ready_leader + static_cast<uint32_t>(slot * 8));
            advance();
            advance();
            fetch();
        }
    } else if (warp == kScaleWarp || warp == kLoadWarp) {
        // ------------------------------------------------------------------ scales into atoms
        // Lane l takes rows l, l + 32, l + 64, l + 96 of each 128 and writes, for each word of
        // the rows, the four rows' words as 16 bytes of the word's atom: in place, so everything is
        // read before anything is written. The two warps take steps in turn.
        const uint32_t ready_leader = cluster_addr(&sf_ready[0], leader);
        const int my_turn = warp == kScaleWarp ? 0 : 1;
        int slot = 0, turn = 0;
        uint32_t phase = 0u;
        bool ok = true;
        for (int64_t tile = first; tile < num_tiles && ok; tile += step) {
            for (int kb = kb0; kb < kb1; kb += 2) {
                const int at_slot = slot;
                const uint32_t at_phase = phase;
                const bool mine = turn == my_turn;
                slot = slot + 1 == kScaleRing ? 0 : slot + 1;
                phase ^= slot == 0 ? 1u : 0u;
                turn ^= 1;
                if (!mine)
                    continue;
                if (!__all_sync(0xffffffffu, mbar_wait(&sf_raw[at_slot], at_phase, p.limit))) {
                    if (lane == 0)
                        give_up(p.report);
                    ok = false;
                    break;
                }
                const uint32_t st = smem_u32(sf) + static_cast<uint32_t>(at_slot * T::kStepBytes);
                uint32_t v[kGroups * 4][2 * W];
#pragma unroll
                for (int g = 0; g < kGroups * 4; ++g)
#pragma unroll
                    for (int c = 0; c < W / 2; ++c)
                        lds_words4(v[g] + 4 * c, st + T::chunk_at(g * 32 + lane, c));
                __syncwarp();
#pragma unroll
                for (int g = 0; g < kGroups; ++g)
#pragma unroll
                    for (int k = 0; k < 2 * W; ++k) {
                        const int h = k / W, a = k % W;  // stage of the step, atom of the stage
                        const int atom = h * W * kGroups + (g == 0 ? a : W + a * T::kAtomsN + g - 1);
                        sts_words4(st + atom * kAtom + lane * 16, v[g * 4][k], v[g * 4 + 1][k],
                                   v[g * 4 + 2][k], v[g * 4 + 3][k]);
                    }
                // The leader's thread has the tensor core of this CTA read these stores.
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_smem_written(ready_leader + static_cast<uint32_t>(at_slot * 8));
            }
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------------ MMA issue (leader)
        if (cr == 0 && elect_one()) {
            constexpr bool kNv = FMT == LNQ_FP4_NV;
            int stage = 0, slot = 0, acc = 0;
            uint32_t fph = 0u, sph = 0u, aph = 1u;  // parities: codes, scales, accumulators
            bool ok = true;
            for (int64_t tile = first; tile < num_tiles && ok; tile += step) {
                if (!mbar_wait_cluster(&tempty[acc], aph, p.limit)) {
                    give_up(p.report);
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
                for (int kb = kb0; kb < kb1; ++kb) {
                    const int h = (kb - kb0) & 1;  // stage of the step
                    if ((h == 0 && !mbar_wait_cluster(&sf_ready[slot], sph, p.limit)) ||
                        !mbar_wait(&full[stage], fph, p.limit)) {
                        give_up(p.report);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_u32(smem + stage * T::kStageBytes);
                    const uint64_t ad = umma_desc_sw128(sa, 16, 1024);
                    const uint64_t bd = umma_desc_sw128(sa + T::kABytes, 16, 1024);
                    const uint64_t sd = smem_desc_plain(
                        smem_u32(sf + slot * T::kStepBytes + h * T::kScaleBytes));
                    const uint32_t st =
                        tmem_base + static_cast<uint32_t>(T::kAcc * BN + stage * T::kSlotCols);
#pragma unroll
                    for (int c = 0; c < T::kAtomsK * (1 + T::kAtomsN); ++c)
                        tmem_cp_32x128b_pair(st + c * 4, sd + c * (kAtom >> 4));
#pragma unroll
                    for (int kk = 0; kk < BK / 64; ++kk) {  // 32 bytes of K each
                        const int atom = kNv ? kk : kk / 2;
                        const uint32_t idesc = umma_idesc_f4(PM, BN, !kNv, kNv ? 0u : (kk & 1) * 2u);
                        umma_f4_pair<kNv>(d_tmem, ad + kk * 2, bd + kk * 2, idesc, st + atom * 4,
                                          st + (T::kAtomsK + atom * T::kAtomsN) * 4,
                                          (kb != kb0 || kk != 0) ? 1u : 0u);
                    }
                    umma_commit_pair(&empty[stage], pair_mask);
                    if (h == 1 || kb + 1 == kb1) {
                        umma_commit_pair(&sf_empty[slot], pair_mask);
                        slot = slot + 1 == kScaleRing ? 0 : slot + 1;
                        sph ^= slot == 0 ? 1u : 0u;
                    }
                    stage = stage + 1 == T::kStages ? 0 : stage + 1;
                    fph ^= stage == 0 ? 1u : 0u;
                }
                if (!ok)
                    break;
                umma_commit_pair(&tfull[acc], pair_mask);
                acc = acc + 1 == T::kAcc ? 0 : acc + 1;
                aph ^= acc == 0 ? 1u : 0u;
            }
            // every MMA of this thread has completed, and its commits have arrived, once `drain`
            // flips
            umma_commit_pair(drain, pair_mask);
            mbar_wait(drain, 0, last_limit);
        } else if (cr != 0 && lane == 0) {
            mbar_wait(drain, 0, last_limit);
        }
    } else {
        // ------------------------------------------------------------------ epilogue
        constexpr int kChunks = (BN / 32 + 1) / 2;  // 32-column chunks of a warp
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t tempty_leader = cluster_addr(&tempty[0], leader);
        const float ta = p.ta == nullptr ? 1.f : __ldg(p.ta);
        int it = 0;
        for (int64_t tile = first; tile < num_tiles; tile += step, ++it) {
            const int acc = it % T::kAcc, use = it / T::kAcc;
            int ok = 0;
            if (lane == 0)
                ok = mbar_wait(&tfull[acc], use & 1, p.limit) ? 1 : 0;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) {
                if (lane == 0)
                    give_up(p.report);
                break;
            }
            __syncwarp();
            tc_fence_after();
            const Fp4TileAt at = tile_at<BN>(tile, p, lim, pre);
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                   static_cast<uint32_t>(acc * BN);
            const int rows = min(at.b1 - at.b0, BN);  // rows of this tile
            // the accumulator is read whole before anything is stored: the next tile may begin
            uint32_t v[kChunks][32];
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const int col = (2 * c + half) * 32;
                if (col < BN && col < rows)
                    tmem_ld_32x32b_x32_nowait(taddr + col, v[c]);
            }
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                tmem_ld_fence(v[c]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_tmem_read(tempty_leader + static_cast<uint32_t>(acc * 8));
            if (p.split > 1) {
                // this pair's share of the sums, [row][128 outputs], over the finished stages
                float *sums = reinterpret_cast<float *>(smem);
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    const int col = (2 * c + half) * 32;
                    if (BN <= 128 && col < BN && col < rows)
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            sums[(col + k) * BM + quarter * 32 + lane] = __uint_as_float(v[c][k]);
                }
                continue;
            }
            const int j = at.j0 + static_cast<int>(cr) * BM + quarter * 32 + lane;
            if (j >= p.d_out)
                continue;
            const Fp4Factors f(ta, p.tw == nullptr ? 1.f : __ldg(p.tw + at.e));
            if (f.f2 != 1.f) {
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        v[c][k] = __float_as_uint(__uint_as_float(v[c][k]) * f.f2);
            }
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const int col = (2 * c + half) * 32, count = rows - col;
                if (col >= BN || count <= 0)
                    continue;
                const int64_t o = static_cast<int64_t>(at.b0 + col) * p.ldy + j;
                if (p.yt == LNQ_BF16)
                    store_column(static_cast<__nv_bfloat16 *>(p.y) + o, p.ldy, count, v[c], f);
                else if (p.yt == LNQ_F16)
                    store_column(static_cast<__half *>(p.y) + o, p.ldy, count, v[c], f);
                else
                    store_column(static_cast<float *>(p.y) + o, p.ldy, count, v[c], f);
            }
        }
    }

    if (p.split > 1) {
        // One tile per cluster. Each pair adds and writes its share of the rows, over the pairs
        // in order. (After a wait that gave up they may add anything: nothing is being copied to the
        // stages any more, and the call is reported.)
        cluster_sync();
        const Fp4TileAt at = tile_at<BN>(first, p, lim, pre);
        const int rows = min(at.b1 - at.b0, BN);
        const int r0 = part * rows / p.split, r1 = (part + 1) * rows / p.split;
        const Fp4Factors f(p.ta == nullptr ? 1.f : __ldg(p.ta), p.tw == nullptr ? 1.f : __ldg(p.tw + at.e));
        uint32_t peer[kMaxSplit];
#pragma unroll
        for (int s = 0; s < kMaxSplit; ++s)
            peer[s] = cluster_addr(smem, 2u * (s < p.split ? s : 0) + cr);
        // four consecutive outputs a thread
        for (int i = r0 * (BM / 4) + static_cast<int>(threadIdx.x); i < r1 * (BM / 4); i += kThreads) {
            float u[kMaxSplit][4];
#pragma unroll
            for (int s = 0; s < kMaxSplit; ++s)
                if (s < p.split)
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(u[s][0]), "=f"(u[s][1]), "=f"(u[s][2]), "=f"(u[s][3])
                                 : "r"(peer[s] + i * 16)
                                 : "memory");
            const int j = at.j0 + static_cast<int>(cr) * BM + i % (BM / 4) * 4;
            const int64_t o = static_cast<int64_t>(at.b0 + i / (BM / 4)) * p.ldy + j;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float sum = u[0][k];
#pragma unroll
                for (int s = 1; s < kMaxSplit; ++s)
                    if (s < p.split)
                        sum += u[s][k];
                sum = f(sum * f.f2);
                if (j + k >= p.d_out)
                    break;
                if (p.yt == LNQ_BF16)
                    static_cast<__nv_bfloat16 *>(p.y)[o + k] = from_f32<__nv_bfloat16>(sum);
                else if (p.yt == LNQ_F16)
                    static_cast<__half *>(p.y)[o + k] = from_f32<__half>(sum);
                else
                    static_cast<float *>(p.y)[o + k] = sum;
            }
        }
    }

    // All CTAs stay until the cluster is done: the MMAs read both CTAs' shared memory, barriers
    // in the leader are signalled by both, partial sums are read by all.
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (warp == kMmaWarp)
        tmem_dealloc_pair(tmem_base, kTmemCols);
}

// ------------------------------------------------------------------------------------------
// Host launcher
// ------------------------------------------------------------------------------------------
// Codes of `rows` rows as a byte matrix; boxes of 128 bytes x `box` rows.
static bool encode_codes(CUtensorMap *map, const uint8_t *codes, int64_t rows, int64_t d, int box)
{
    auto encode = tensor_map_encoder();
    cuuint64_t dims[2] = {static_cast<cuuint64_t>((d + 1) / 2), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(fp4_code_pitch(d))};
    cuuint32_t boxes[2] = {128, static_cast<cuuint32_t>(box)};
    cuuint32_t estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(codes), dims, strides,
                  boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scales of `rows` rows as a byte matrix; boxes of a step's bytes (`width`) x `box` rows.
static bool encode_scales(CUtensorMap *map, const uint8_t *scales, int64_t rows, int blocks, int pitch,
                          int width, int box)
{
    auto encode = tensor_map_encoder();
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(blocks), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
    cuuint32_t boxes[2] = {static_cast<cuuint32_t>(width), static_cast<cuuint32_t>(box)};
    cuuint32_t estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(scales), dims, strides,
                  boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  width == 32 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, int FMT>
static cudaError_t gemm_tile(const Fp4Matrix &a, const Fp4Matrix &w, int64_t d_in, Fp4GemmParams p,
                             int64_t tiles, int num_sms, cudaStream_t s)
{
    using T = f4::Tile<BN, FMT>;
    CUtensorMap wmap, amap, wsmap = {}, asmap = {};
    if (!encode_codes(&wmap, w.codes, p.w_total, d_in, f4::BM) ||
        !encode_codes(&amap, a.codes, a.rows, d_in, BN / 2))
        return cudaErrorInvalidValue;
    p.sf_tma = p.scale_pitch % 16 == 0 && ((reinterpret_cast<uintptr_t>(w.scales) |
                                            reinterpret_cast<uintptr_t>(a.scales)) & 15) == 0;
    if (p.sf_tma &&
        (!encode_scales(&wsmap, w.scales, p.w_total, p.blocks, p.scale_pitch, T::kRowBytes, f4::BM) ||
         !encode_scales(&asmap, a.scales, a.rows, p.blocks, p.scale_pitch, T::kRowBytes, BN)))
        return cudaErrorInvalidValue;
    auto kernel = fp4_gemm_kernel<BN, FMT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(T::kSmem));
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * p.split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.blockDim = dim3(f4::kThreads);
    cfg.dynamicSmemBytes = T::kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (p.split == 1) {
        static ResidentClusters pairs;  // one CTA per SM
        const int resident = pairs.get(current_device(), num_sms / 2, [&]() {
            cfg.gridDim = dim3(static_cast<unsigned>(num_sms & ~1));
            return max_active_clusters(kernel, cfg);
        });
        tiles = tiles < resident ? tiles : resident;
    }
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * 2 * p.split));
    KernelTimer timer("lnq_fp4_gemm", s);
    e = cudaLaunchKernelEx(&cfg, kernel, wmap, amap, wsmap, asmap, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t fp4_gemm_launch(const Fp4Matrix &a, const int32_t *offsets, int64_t experts,
                            const Fp4Matrix &w, int64_t d_in, int fmt, void *y, int yt,
                            int64_t ldy, long long wait_limit, int num_sms, cudaStream_t s)
{
    if (tensor_map_encoder() == nullptr)
        return cudaErrorNotSupported;
    Fp4GemmParams p;
    p.a_scales = a.scales;
    p.w_scales = w.scales;
    p.ta = a.t;
    p.tw = w.t;
    p.offsets = offsets;
    p.y = y;
    p.ldy = ldy;
    p.w_total = w.rows * experts;
    p.n = static_cast<int>(a.rows);
    p.experts = static_cast<int>(experts);
    p.d_out = static_cast<int>(w.rows);
    p.yt = yt;
    p.nk = static_cast<int>((d_in + f4::BK - 1) / f4::BK);
    p.blocks = static_cast<int>((d_in + fp4_block(fmt) - 1) / fp4_block(fmt));
    p.scale_pitch = static_cast<int>(fp4_scale_pitch(d_in, fmt));
    p.mt = static_cast<int>((w.rows + f4::PM - 1) / f4::PM);
    p.limit = wait_limit;
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &capture) != cudaSuccess)
        return cudaErrorInvalidValue;
    p.report = capture == cudaStreamCaptureStatusNone ? fp4_report_slot(s) : kCapturedSlot;
    // an upper bound of the row tiles where the groups are not known here
    auto tiles_of = [&](int rows) {
        return p.mt * (offsets == nullptr ? (a.rows + rows - 1) / rows
                                          : min(a.rows, a.rows / rows + experts));
    };
    const int64_t pairs = num_sms / 2;
    int bn = 32;
    p.split = 1;
    if (offsets != nullptr) {
        // Twice a group of average size, 64 at least: a tile's time depends little on its width,
        // and a group larger than the tile reads its weights again (2000 rows over 32 experts,
        // 2048 -> 2048, largest group 493: 31 us with 64 rows a tile, 24 with 128, 25 with 256).
        const int64_t mean = (a.rows + experts - 1) / experts;
        bn = 64;
        while (bn < 256 && bn < 2 * mean)
            bn *= 2;
    } else {
        // Rows per tile and pairs that share a tile's K: the least time, in hundredths of a
        // microsecond, from the times measured for a tile's fixed parts (first loads, last sums;
        // joining the shares) and for a stage, which depends little on the width. (Four pairs to
        // a tile, clusters of 8, were slower than two at every size.)
        constexpr int kFixed[4] = {540, 590, 690, 820}, kStage[4] = {38, 39, 40, 43};
        int64_t best = INT64_MAX;
        for (int w = 0; w < 4; ++w) {
            const int rows = 32 << w;
            const int64_t tiles = tiles_of(rows);
            for (int split = 1; split <= (rows <= 128 ? f4::kMaxSplit : 1); split *= 2) {
                if (split > 1 && (tiles * split > pairs || p.nk < split * 2))
                    break;
                const int64_t cost = (tiles * split + pairs - 1) / pairs *
                                         ((p.nk + split - 1) / split * kStage[w]) + kFixed[w] +
                                     (split > 1 ? 60 : 0);
                if (cost < best)
                    best = cost, bn = rows, p.split = split;
            }
        }
    }
    const int64_t tiles = tiles_of(bn);
    const bool nv = fmt == LNQ_FP4_NV;
    switch (bn) {
    case 32:
        return nv ? gemm_tile<32, LNQ_FP4_NV>(a, w, d_in, p, tiles, num_sms, s)
                  : gemm_tile<32, LNQ_FP4_MX>(a, w, d_in, p, tiles, num_sms, s);
    case 64:
        return nv ? gemm_tile<64, LNQ_FP4_NV>(a, w, d_in, p, tiles, num_sms, s)
                  : gemm_tile<64, LNQ_FP4_MX>(a, w, d_in, p, tiles, num_sms, s);
    case 128:
        return nv ? gemm_tile<128, LNQ_FP4_NV>(a, w, d_in, p, tiles, num_sms, s)
                  : gemm_tile<128, LNQ_FP4_MX>(a, w, d_in, p, tiles, num_sms, s);
    default:
        return nv ? gemm_tile<256, LNQ_FP4_NV>(a, w, d_in, p, tiles, num_sms, s)
                  : gemm_tile<256, LNQ_FP4_MX>(a, w, d_in, p, tiles, num_sms, s);
    }
}

cudaError_t fp4_give_ups(Fp4GiveUps *counts, cudaStream_t s)
{
    auto read = [&](uint32_t *to, int slot) {
        return cudaMemcpyFromSymbolAsync(to, g_fp4_gave_up, sizeof(uint32_t), slot * sizeof(uint32_t),
                                         cudaMemcpyDeviceToHost, s);
    };
    cudaError_t e = read(&counts->own, fp4_report_slot(s));
    if (e == cudaSuccess)
        e = read(&counts->captured, kCapturedSlot);
    if (e == cudaSuccess)
        e = read(&counts->all, kAllSlot);
    return e != cudaSuccess ? e : cudaStreamSynchronize(s);
}

}  // namespace lnq
